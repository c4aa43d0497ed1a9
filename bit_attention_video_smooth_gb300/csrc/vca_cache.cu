// vca_cache.cu -- writing the 8-bit cache: new K/V rows into pages (append) and
// the tokens that stay after an eviction into fresh pages (evict).
//
// A page of one head has one scale s, a power of two with max|x| <= 448 s, so
// x / s is exact and an E4M3 code keeps its significant bits when the scale
// grows: only values that become subnormal round again.
//
// Both are bound by the bytes they move.  Append reads 4 and writes 2 bytes a
// channel of K and V: 17,664 rows of 40 heads 87 us, 6.2 TB/s.  Evict reads every
// weight once and moves what stays: 4 x 8 heads of up to 32,768 tokens cut to
// 4,096 in 41 us, the selection 20 and the move 23 (they overlap); a thousand tokens
// in 11 us.
#include "vca_cache.cuh"

namespace vca {

namespace {

using namespace cache;

constexpr int kThreads = 256;
constexpr int kRowsPerPass = kThreads / 16;         // 16 threads a row, 8 channels each
constexpr int kPasses = kBlk / kRowsPerPass;

// Eight codes of eight fp32 values times inv (a power of two: exact above the
// subnormal codes); `odd`: some may not be finite.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv, bool odd) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], inv);
    if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = scaled_or_nan(x[i], inv);
    }
    return make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
}
// The values of eight codes at scale s: exact, the smallest (2^-9 2^-120) as a
// subnormal.
__device__ __forceinline__ void decode8(const uint2 &w, float s, float (&x)[8]) {
    float a[4], b[4];
    e4m3x4_decode(w.x, a);
    e4m3x4_decode(w.y, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = __fmul_rn(a[i], s);
        x[4 + i] = __fmul_rn(b[i], s);
    }
}

// ---------------------------------------------------------------------------
// Append: one CTA per (page that gets new rows, head, K or V)
// ---------------------------------------------------------------------------
// The page's rows stay in registers between the maximum and the codes, 64 bytes a
// thread with all loads in flight, four CTAs to an SM.
struct AppendParams {
    CacheView c;
    CacheRows k, v;
    const int32_t *start;
    int T;
    float *weight;          // [pages][H][128] or null
    int32_t *dev_status;
};

__global__ void __launch_bounds__(kThreads, 4) append_kernel(const AppendParams p) {
    __shared__ int s_at[4];                 // sequence, page column, its first new row (of the call), page
    __shared__ uint32_t red[kThreads / 32];
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        // the blockIdx.x-th page that gets new rows, counted over the sequences in order
        int before = 0, found = -1;
        const bool reports = blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0;
        if (lane == 0) s_at[0] = -1;
        bool more = true;
        for (int b0 = 0; more && (found < 0 || reports); b0 += 32) {
            const int b = b0 + lane;
            Seq s;
            more = load_seqs(p.c, p.start, p.T, b0, s);
            if (s.n > s.len) s.bad = true;      // the cache's length counts the new rows
            if (reports && s.bad) report(p.dev_status, kErrInvalid);
            const int first = s.len - s.n, cnt = s.bad || s.n == 0 ? 0 : (s.len - 1) / kBlk - first / kBlk + 1;
            int incl = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const int j = static_cast<int>(blockIdx.x) - before - (incl - cnt);
            if (found < 0 && j >= 0 && j < cnt) {
                const int col = first / kBlk + j;
                s_at[1] = col;
                s_at[2] = s.row0 - first;           // row of slot t: t + s_at[2]
                s_at[3] = first;
                s_at[0] = b;
            }
            found = __ballot_sync(0xffffffffu, j >= 0 && j < cnt) != 0 ? 1 : found;
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    __syncthreads();
    const int b = s_at[0];
    if (b < 0) return;
    const int col = s_at[1], shift = s_at[2], first = s_at[3], h = blockIdx.y;
    const int page = load_page(p.c, b, col, p.dev_status);
    if (page < 0) return;
    const bool is_v = blockIdx.z != 0;
    const CacheRows x = is_v ? p.v : p.k;
    uint8_t *codes = (is_v ? p.c.v8 : p.c.k8) + (static_cast<int64_t>(page) * p.c.H + h) * (kBlk * kD);
    float *scale = (is_v ? p.c.sv : p.c.sk) + static_cast<int64_t>(page) * p.c.H + h;
    const int lo = max(first - col * kBlk, 0), hi = min(p.c.len[b] - col * kBlk, kBlk);   // new slots of this page
    const int r = threadIdx.x >> 4, ch = (threadIdx.x & 15) * 8;
    // a page that is used again holds another token's weights
    if (p.weight && !is_v && static_cast<int>(threadIdx.x) >= lo && static_cast<int>(threadIdx.x) < hi)
        p.weight[(static_cast<int64_t>(page) * p.c.H + h) * kBlk + threadIdx.x] = 0.0f;

    uint4 v[kPasses];
    uint32_t m = 0;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int slot = r + i * kRowsPerPass;
        v[i] = make_uint4(0, 0, 0, 0);
        if (slot >= lo && slot < hi)
            v[i] = *reinterpret_cast<const uint4 *>(x.p + (col * kBlk + slot + shift) * x.tok + h * x.head + ch);
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) m = max(m, amax_bf16x8(v[i], odd));
    const float s_old = lo > 0 ? *scale : 0.0f;
    const uint32_t sb = max(scale_bits(block_max<kThreads>(m, red)), __float_as_uint(s_old) & 0x7f800000u);
    const float inv = pow2_inverse(sb);
    if (threadIdx.x == 0) *scale = __uint_as_float(sb);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int slot = r + i * kRowsPerPass;
        if (slot < lo || slot >= hi) continue;
        float f[8];
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(w[e] << 16);
            f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
        *reinterpret_cast<uint2 *>(codes + slot * kD + ch) = encode8(f, inv, odd);
    }
    // the scale grew: the codes that were there move with it
    if (lo > 0 && __uint_as_float(sb) != s_old) {
        for (int slot = r; slot < lo; slot += kRowsPerPass) {
            uint2 *at = reinterpret_cast<uint2 *>(codes + slot * kD + ch);
            float f[8];
            decode8(*at, s_old, f);
            *at = encode8(f, inv, false);      // a NaN code stays one
        }
    }
}

// ---------------------------------------------------------------------------
// Evict
// ---------------------------------------------------------------------------
struct EvictParams {
    CacheView c;
    float *weight;
    const int32_t *dst;
    int dst_cols, budget, recent;
    int32_t *new_len, *kept, *dev_status;
};

// Unsigned keys in the order of the weights; NaN counts as the lowest, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    uint32_t u = __float_as_uint(w);
    if ((u & 0x7fffffffu) > 0x7f800000u) u = 0xff800000u;
    if (u == 0x80000000u) u = 0u;
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024;
constexpr int kSelKeys = 40960;         // keys that a CTA can keep in shared memory: 160 KB

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// A word of another CTA's shared memory.
__device__ __forceinline__ int cluster_read(const int *p, uint32_t rank) {
    uint32_t at;
    int v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// A cluster of kCluster CTAs (of four; of eight 43 us where four took 19, of
// sixteen 210) per (sequence, head), each over an equal run of the older slots: the
// key of the last weight that stays by a radix select over four bytes (the CTAs'
// histograms are added through distributed shared memory), then
// the slots that stay, in order.  Each weight is read once, unless a CTA's run
// does not fit its shared memory.  Weights crowd into few bins (their first byte
// is most of the exponent, and many are 0), and equal lanes' atomics take turns:
// eight copies of the histogram, in different banks, cut the turns by eight.
template <int kCluster>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictParams p, int keep) {
    extern __shared__ uint32_t sKeys[];
    constexpr int kCopy = 257;
    __shared__ int copies[8 * kCopy], hist[2][256], total[256], s_bin, s_left, counts[2];
    __shared__ int wsum[2][kSelThreads / 32];
    const int rank = kCluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int h = blockIdx.x / kCluster, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    let_next_start();
    int len = p.c.len[b];
    if (len < 0 || len > static_cast<int64_t>(p.c.cols) * kBlk) {
        if (tid == 0) report(p.dev_status, kErrInvalid);
        len = 0;
    }
    const int stay = min(len, p.budget), recent = min(min(len, p.recent), stay);
    if (h == 0 && tid == 0 && rank == 0) p.new_len[b] = stay;
    const int older = len - recent, want = stay - recent;
    int32_t *kept = p.kept + (static_cast<int64_t>(b) * p.c.H + h) * p.budget;
    for (int j = rank * kSelThreads + tid; j < recent; j += kCluster * kSelThreads) kept[want + j] = older + j;
    if (want == older) {
        // all of them stay
        for (int j = rank * kSelThreads + tid; j < want; j += kCluster * kSelThreads) kept[j] = j;
        return;
    }
    if (want == 0) return;
    const int run = (older + kCluster * 32 - 1) / (kCluster * 32) * 32;      // a multiple of a warp's
    const int t0 = min(older, rank * run), n = min(older, t0 + run) - t0;
    // the key of slot t of the run; a page that does not exist counts as the lowest weights
    auto load_key = [&](int i) -> uint32_t {
        const int t = t0 + i, page = p.c.table[static_cast<int64_t>(b) * p.c.cols + t / kBlk];
        if (page < 0 || page >= p.c.pages) {
            report(p.dev_status, kErrInvalid);
            return 0u;
        }
        return weight_key(p.weight[(static_cast<int64_t>(page) * p.c.H + h) * kBlk + t % kBlk]);
    };
    const bool kept_keys = n <= keep;
    auto key_of = [&](int i) -> uint32_t { return kept_keys ? sKeys[i] : load_key(i); };
    if (kept_keys) {
        // eight at once: the table entries' loads side by side, then the weights'
        for (int i0 = tid; i0 < n; i0 += 8 * kSelThreads) {
            int page[8];
            float w[8];
            bool bad = false;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = i0 + k * kSelThreads;
                page[k] = i < n ? p.c.table[static_cast<int64_t>(b) * p.c.cols + (t0 + i) / kBlk] : 0;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = i0 + k * kSelThreads;
                const bool there = page[k] >= 0 && page[k] < p.c.pages;
                bad |= !there;
                if (i < n && there) w[k] = p.weight[(static_cast<int64_t>(page[k]) * p.c.H + h) * kBlk + (t0 + i) % kBlk];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = i0 + k * kSelThreads;
                if (i < n) sKeys[i] = page[k] >= 0 && page[k] < p.c.pages ? weight_key(w[k]) : 0u;
            }
            if (bad) report(p.dev_status, kErrInvalid);
        }
    }
    for (int i = tid; i < 8 * kCopy; i += kSelThreads) copies[i] = 0;
    __syncthreads();
    uint32_t prefix = 0, mask = 0;
    int left = want;               // how many of those whose key starts with `prefix` stay
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        int *mine = hist[pass & 1];
        for (int i = tid; i < n; i += kSelThreads) {
            const uint32_t k = key_of(i);
            if ((k & mask) == prefix) atomicAdd(&copies[(lane & 7) * kCopy + ((k >> shift) & 255)], 1);
        }
        __syncthreads();
        if (tid < 256) {
            int sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum += copies[i * kCopy + tid];
                copies[i * kCopy + tid] = 0;
            }
            mine[tid] = sum;
        }
        __syncthreads();
        if constexpr (kCluster > 1) cluster_sync();
        if constexpr (kCluster > 1) {
            if (tid < 256) {
                int sum = 0;
#pragma unroll
                for (int r = 0; r < kCluster; ++r) sum += cluster_read(&mine[tid], r);
                total[tid] = sum;
            }
            __syncthreads();
        }
        if (warp == 0) {
            // bins from the top: lane i holds bins 255 - 8 i .. 248 - 8 i
            const int *bins = kCluster > 1 ? total : mine;
            int c[8], s = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += c[e] = bins[255 - 8 * lane - e];
            int incl = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            int above = incl - s;
            if (above < left && left <= incl) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (above < left && left <= above + c[e]) {
                        s_bin = 255 - 8 * lane - e;
                        s_left = left - above;
                    }
                    above += c[e];
                }
            }
        }
        // the next pass writes the other histogram, which every CTA of the cluster has read by now
        __syncthreads();
        prefix |= static_cast<uint32_t>(s_bin) << shift;
        mask |= 255u << shift;
        left = s_left;
    }
    // keys above `prefix` stay, and the first `left` of those equal to it.  A warp
    // takes a run of its own: counts first, then places
    const int per = (n + kSelThreads - 1) / kSelThreads * 32;       // slots of a warp
    const int w0 = min(n, warp * per), w1 = min(n, w0 + per);
    int gt = 0, eq = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t k = key_of(i);
        gt += k > prefix;
        eq += k == prefix;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        wsum[0][warp] = gt;
        wsum[1][warp] = eq;
    }
    __syncthreads();
    int g0 = 0, e0 = 0, g_all = 0, e_all = 0;      // before this warp, and of the CTA
    for (int i = 0; i < kSelThreads / 32; ++i) {
        const int x = wsum[0][i], y = wsum[1][i];
        if (i < warp) {
            g0 += x;
            e0 += y;
        }
        g_all += x;
        e_all += y;
    }
    if constexpr (kCluster > 1) {
        if (tid == 0) {
            counts[0] = g_all;
            counts[1] = e_all;
        }
        __syncthreads();
        cluster_sync();
        for (int r = 0; r < rank; ++r) {
            g0 += cluster_read(&counts[0], r);
            e0 += cluster_read(&counts[1], r);
        }
        cluster_sync();      // no CTA leaves while another reads its counts
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int i = w0; i < w1; i += 32) {
        const bool there = i + lane < w1;
        const uint32_t k = there ? key_of(i + lane) : 0u;
        const uint32_t bg = __ballot_sync(0xffffffffu, there && k > prefix), be = __ballot_sync(0xffffffffu, there && k == prefix);
        const int tie = e0 + __popc(be & below);      // ties before this slot
        if (there && (k > prefix || (k == prefix && tie < left))) kept[g0 + __popc(bg & below) + min(tie, left)] = t0 + i + lane;
        g0 += __popc(bg);
        e0 += __popc(be);
    }
}

// The largest magnitude among eight codes, NaN apart.
__device__ __forceinline__ uint32_t top_code(const uint2 &w) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = (i ? w.y : w.x) & 0x7f7f7f7fu;
        m = __vmaxu4(m, x & ~(((x + 0x01010101u) & 0x80808080u) - (((x + 0x01010101u) & 0x80808080u) >> 7)));
    }
    m = __vmaxu4(m, m >> 16);
    return max(m & 0xffu, (m >> 8) & 0xffu);
}

// One CTA per (page that is written, head): K by the first 256 threads, V by the
// others.  A token whose scale stays the page's is copied without decoding.
__global__ void __launch_bounds__(2 * kThreads, 3) move_kernel(const EvictParams p) {
    __shared__ uint32_t red[2][kThreads / 32];
    __shared__ int s_row[kBlk];         // place of the token's row of codes in the pool, in tiles of 128; -1: none
    __shared__ int s_slot[kBlk];
    __shared__ float s_scale[2][kBlk];
    const int col = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const bool is_v = tid >= kThreads;
    const int32_t *kept = p.kept + (static_cast<int64_t>(b) * p.c.H + h) * p.budget + col * kBlk;
    const int page = p.dst[static_cast<int64_t>(b) * p.dst_cols + col];
    wait_for_results();
    const int rows = min(p.new_len[b] - col * kBlk, kBlk);
    if (rows <= 0) return;
    if (page < 0 || page >= p.c.pages) {
        if (tid == 0) report(p.dev_status, kErrInvalid);
        return;
    }
    const int to = page * p.c.H + h;
    if (tid < 2 * kBlk) {
        const int j = tid & (kBlk - 1);
        int from = -1, t = 0;
        if (j < rows) {
            t = kept[j];
            from = load_page(p.c, b, t / kBlk, p.dev_status);
            if (from >= 0) from = from * p.c.H + h;
        }
        s_scale[tid / kBlk][j] = from >= 0 ? (tid < kBlk ? p.c.sk : p.c.sv)[from] : 0.0f;
        if (tid < kBlk) {
            s_row[j] = from;
            s_slot[j] = t % kBlk;
            if (from >= 0)
                p.weight[static_cast<int64_t>(to) * kBlk + j] = p.weight[static_cast<int64_t>(from) * kBlk + t % kBlk];
        }
    }
    __syncthreads();
    const uint8_t *codes = is_v ? p.c.v8 : p.c.k8;
    const float *s = s_scale[is_v];
    const int r = (tid >> 4) & 15, ch = (tid & 15) * 8;
    uint2 v[kPasses];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int j = r + i * kRowsPerPass, from = s_row[j];
        v[i] = make_uint2(0, 0);
        if (from >= 0) v[i] = *reinterpret_cast<const uint2 *>(codes + (static_cast<int64_t>(from) * kBlk + s_slot[j]) * kD + ch);
    }
    // the largest value of a row: magnitudes of codes are in the order of their bits (NaN apart)
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const float top = __fmul_rn(e4m3_to_f32(top_code(v[i])), s[r + i * kRowsPerPass]);
        m = max(m, __float_as_uint(top));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) red[is_v][(tid >> 5) & 7] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, red[is_v][i]);
    const uint32_t sb = scale_bits(m);
    const float inv = pow2_inverse(sb);
    if ((tid & (kThreads - 1)) == 0) (is_v ? p.c.sv : p.c.sk)[to] = __uint_as_float(sb);
    uint8_t *out = (is_v ? p.c.v8 : p.c.k8) + static_cast<int64_t>(to) * kBlk * kD;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int j = r + i * kRowsPerPass;
        if (s_row[j] < 0) continue;
        if (__float_as_uint(s[j]) != sb) {
            float f[8];
            decode8(v[i], s[j], f);
            v[i] = encode8(f, inv, false);     // a NaN code stays one
        }
        *reinterpret_cast<uint2 *>(out + j * kD + ch) = v[i];
    }
}

}  // namespace

cudaError_t launch_cache_append(const CacheView &c, const CacheRows &k, const CacheRows &v, const int32_t *start, int T,
                                float *weight, int32_t *dev_status, cudaStream_t st) {
    // n rows touch at most n pages and at most (n - 1) / 128 + 2
    const int64_t bound = static_cast<int64_t>(T) / kBlk + 2ll * c.B;
    const AppendParams p{c, k, v, start, T, weight, dev_status};
    append_kernel<<<dim3(static_cast<unsigned>(bound < T ? bound : T), c.H, 2), kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_cache_evict(const CacheView &c, float *weight, const int32_t *dst_table, int dst_cols, int budget,
                               int recent, int32_t *new_len, int32_t *kept, int32_t *dev_status, cudaStream_t st) {
    const EvictParams p{c, weight, dst_table, dst_cols, budget, recent, new_len, kept, dev_status};
    const int64_t tokens = static_cast<int64_t>(c.cols) * kBlk;      // of a sequence, at most
    // a cluster of four CTAs for each head where one CTA would not hold the keys, or
    // where they are many and all clusters run at once (a CTA fills an SM): 2 x 8
    // heads of 32,000 tokens 23 us against 39, of 8,000 18 against 17; 16 x 8 heads of
    // 32,000 tokens 88 against 58, of 64,000 (past kSelKeys) 118 against 210
    const int parts = tokens > kSelKeys || (tokens > 12288 && 4ll * c.B * c.H <= 152) ? 4 : 1;
    const int64_t run = (tokens + parts - 1) / parts + 32;
    const int keep = static_cast<int>(run < kSelKeys ? run : kSelKeys);
    const auto kernel = parts == 4 ? select_kernel<4> : select_kernel<1>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = parts;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(c.H * parts, c.B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(keep) * 4;
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, p, keep);
    if (e != cudaSuccess) return e;
    const int64_t most = budget < tokens ? budget : tokens;      // that stay
    return launch_after(move_kernel, dim3(static_cast<unsigned>((most + kBlk - 1) / kBlk), c.H, c.B), 2 * kThreads, 0, st, p);
}

}  // namespace vca
