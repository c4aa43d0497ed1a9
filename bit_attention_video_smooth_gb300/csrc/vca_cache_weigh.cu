// vca_cache_weigh.cu -- the attention weight that each cached token receives:
//   weight[key] += sum over the rows r that see it of 2^(x(r, key) - lse(r) log2 e),
// x the score in log2 units, as vca_cache_attention.cu has it.
//
// The scores come from the tensor core with keys as rows: S^T = K Q^T, K's E4M3
// codes straight from TMA, so a thread owns one key and adds its row of S^T up in
// registers; no sum crosses threads.  A query row is hi + lo E4M3 with a factor
// per 32 channels, as in vca_cache_chunk.cu, here the B operand.  A first kernel
// writes every tile of N query rows (16 where sequences have few, else 128) as
// an image of what the second one wants in shared memory: the two code
// matrices, their factors, and for each row its lse.
//
// The second kernel runs one CTA per SM over an equal share of the (sequence,
// KV head, page) list.  Up to four pages of a head stay in shared memory while the
// head's tiles stream past them: a page is read once, and a tile once for four
// pages.  Few rows are bound by reading K (128 B a token) and the weights; many
// by the tensor core's two FP8 products, 2 x 2 rows keys d flops, and the sums'
// exp2 and adds.  One row for each of 5 heads over 8, 32 sequences of up to
// 32,768 tokens: 118 us, 5.4 TB/s; 1,104 rows over 70,656 tokens, 8 heads: 178 us, 896
// TFLOP/s of one product's, the tensor pipe 39 % busy.  Four sets of sum warps took
// 264 us, two with the next scores loaded ahead 237 (registers spill).
// Warps: 0 producer, 1-2 MMA issuers, 3-10 sums (two sets of four).  Every wait is
// bounded, as in vca_attention.cu.
#include "vca_attention_common.cuh"
#include "vca_cache.cuh"

namespace vca {

namespace {

using namespace attn;
using namespace cache;

constexpr uint32_t kTile = kBlk * kD;
constexpr int kKP = 4;                       // pages of a unit
constexpr int kKStages = 8, kSlots = 32;
constexpr int kSets = 2;                     // sets of four sum warps
constexpr int kIssuers = 2;                  // MMA issuers, for the even and the odd pages of a unit
constexpr int kThreads = 32 * (1 + kIssuers + 4 * kSets);
constexpr uint32_t kBarSums = 1;             // named barrier of the sum warps

// A tile of N rows as it lies in the workspace and in shared memory: hi, lo
// codes [N][128], swizzled; the factors of hi and of lo, 32 rows of 16 bytes each
// (row i: rows i, i + 32, i + 64, i + 96; for N = 16 in the first of the two: row
// i the factors of hi i, row 16 + i those of lo i); -lse log2 e of each row; and
// how many keys it sees.
template <int N>
struct Image {
    static constexpr uint32_t lo = N * kD, sf = 2 * N * kD, consts = sf + 1024, seen = consts + 4 * N, bytes = seen + 4 * N;
    static constexpr uint32_t stride = (bytes + 1023) / 1024 * 1024;
};

// S^T takes a column per row; of 16 rows, two: hi and lo are then one product of
// 32 columns, since issuing an MMA costs the same for few columns as for many.
template <int N>
struct Layout {
    static constexpr int qstages = N == 128 ? 2 : 4, cols = N == 128 ? 128 : 32, sbufs = N == 128 ? 3 : 8;
    static constexpr uint32_t tmem_sfa = sbufs * cols, tmem_sfb = tmem_sfa + 4, tmem_cols = 512;
    static constexpr uint32_t offQ = kKStages * kTile, offSlot = offQ + qstages * Image<N>::stride;
    static constexpr uint32_t offSum = offSlot + kSlots * 8, offBar = offSum + 2 * kKP * kBlk * 4;   // fp32 [2][pages][128]
    static constexpr int bars = 2 * kKStages + 2 * qstages + 2 * sbufs + kIssuers;
    static constexpr uint32_t offMisc = offBar + bars * 8, smem = offMisc + 16 + 1024;
    static_assert(smem <= 232448, "shared memory budget");
    static_assert(tmem_sfb + 8 * qstages * kIssuers <= tmem_cols, "TMEM plan");
    // The producer lists a unit's pages once every reader has left the unit qstages before the last one
    static_assert(kSlots >= (qstages + 1) * kKP, "page slots");
    // S^T buffers: of 16 rows every issuer and its set of sum warps have a ring of
    // their own; of 128 one ring serves both issuers, and one may come to a buffer
    // before the other has used it.  It has waited for its page two before, or else
    // for the tile's q_full, which tells that the tile qstages before is summed up: at
    // most max(sbufs + 1, (qstages - 1) kKP + 1) uses are not, which must be fewer than
    // two rounds for the barrier's parity to be unambiguous.
    static constexpr int ring = N == 128 ? sbufs : sbufs / kIssuers;
    static_assert(N == 16 || (sbufs + 1 < 2 * ring && (qstages - 1) * kKP + 1 < 2 * ring), "S^T buffers");
};

struct WeighParams {
    AttnParams a;
    const float *lse;
    float *weight;
    uint8_t *images;
    int tiles;           // images of one head at most
};

// A sequence's rows and pages.
struct Work {
    Seq s;
    int tiles, pages;
};
template <int N>
__device__ __forceinline__ Work work_of(const AttnParams &p, const Seq &s) {
    Work w;
    w.s = s;
    w.tiles = static_cast<int>((static_cast<int64_t>(w.s.n) * p.G + N - 1) / N);
    w.pages = w.s.bad || w.tiles == 0 ? 0 : (w.s.len + kBlk - 1) / kBlk;
    return w;
}
template <int N>
__device__ __forceinline__ Work work_of(const AttnParams &p, int b) {
    return work_of<N>(p, load_seq(p.c, p.start, p.T, b));
}
// The first tile with a row that sees page j: with c = len - n, a causal row sees
// it when its token is at least the (128 j - c)-th new one, so its row at least
// G (128 j - c) and its tile floor of that by N = 128 j G / N - ceil(c G / N).
template <int N>
__device__ __forceinline__ int64_t hidden_tiles(const AttnParams &p, const Seq &s) {      // ceil(c G / N)
    const int64_t r = static_cast<int64_t>(s.len - s.n) * p.G;
    return r >= 0 ? (r + N - 1) / N : -(-r / N);
}
template <int N>
__device__ __forceinline__ int first_tile(const AttnParams &p, const Seq &s, int page) {
    if (!p.causal) return 0;
    const int64_t t = static_cast<int64_t>(page) * (kBlk / N) * p.G - hidden_tiles<N>(p, s);
    return static_cast<int>(t > 0 ? t : 0);
}

// How many of `count` pages from `page` on the rows of a tile see.
template <int N>
__device__ __forceinline__ int pages_seen(const AttnParams &p, const Seq &s, int tile, int page, int count) {
    if (!p.causal) return count;
    const int last = min(s.n * p.G, (tile + 1) * N) - 1;
    return min(count, (min(seen_by_row(p, s, last), s.len) + kBlk - 1) / kBlk - page);
}

__device__ __forceinline__ int64_t scan64(int64_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// Tiles of work in the pages [0, upto) of one head: upto * tiles less what
// first_tile leaves out, an arithmetic series.  Of few rows all tiles count for
// every page: but for the last pages they do.
template <int N>
struct Cost {
    int64_t tiles, hidden, from;      // from: the first page that leaves some out
    int G;
    bool even;
    __device__ Cost(const AttnParams &p, const Work &w) : tiles(w.tiles), hidden(0), from(0), G(p.G), even(N == 16 || !p.causal) {
        if (even) return;
        hidden = hidden_tiles<N>(p, w.s);
        from = hidden >= 0 ? hidden / G + 1 : 0;
    }
    __device__ int64_t before(int64_t upto) const {
        const int64_t m = even ? 0 : upto - from;
        return upto * tiles - (m > 0 ? G * (m * (from + upto - 1) / 2) - hidden * m : 0);
    }
    // The first page before which at least `find` tiles lie.
    __device__ int page_at(int64_t find, int pages) const {
        if (even) return static_cast<int>((find + tiles - 1) / tiles);
        int lo = 0, hi = pages;
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (before(mid) >= find)
                hi = mid;
            else
                lo = mid + 1;
        }
        return lo;
    }
};

// Place in the list of (sequence, head, page).
struct Place {
    int64_t linear;      // pages before it
    int64_t at;          // its place among its sequence's H * pages
    int b, tile0;        // the sequence, the tiles of those before
};
// The first place before which at least `pos` tiles of work lie (a warp's work).
template <int N>
__device__ Place find_place(const AttnParams &p, int64_t pos) {
    Place r{};
    bool more = true;
    for (int b0 = 0; more; b0 += 32) {
        Seq s;
        more = load_seqs(p.c, p.start, p.T, b0, s);
        Work w = work_of<N>(p, s);
        const int64_t cost = Cost<N>(p, w).before(w.pages) * p.c.H, pages = static_cast<int64_t>(p.c.H) * w.pages;
        const int64_t tiles = w.tiles;
        const int64_t ci = scan64(cost), pi = scan64(pages), ti = scan64(tiles);
        const uint32_t hit = __ballot_sync(0xffffffffu, pos < ci);
        if (hit) {
            const int l = __ffs(hit) - 1;
            r.b = b0 + l;
            r.tile0 += static_cast<int>(__shfl_sync(0xffffffffu, ti - tiles, l));
            r.linear += __shfl_sync(0xffffffffu, pi - pages, l);
            const int64_t rest = pos - __shfl_sync(0xffffffffu, ci - cost, l);
            w = work_of<N>(p, r.b);
            const Cost<N> head(p, w);
            const int64_t one = head.before(w.pages), h = rest / one;
            r.at = h * w.pages + head.page_at(rest - h * one, w.pages);
            r.linear += r.at;
            if (r.at == static_cast<int64_t>(p.c.H) * w.pages) {
                r.tile0 += w.tiles;
                ++r.b;
                r.at = 0;
            }
            return r;
        }
        pos -= __shfl_sync(0xffffffffu, ci, 31);
        r.linear += __shfl_sync(0xffffffffu, pi, 31);
        r.tile0 += static_cast<int>(__shfl_sync(0xffffffffu, ti, 31));
    }
    r.b = p.c.B;
    return r;
}
template <int N>
__device__ int64_t all_work(const AttnParams &p) {
    int64_t sum = 0;
    bool more = true;
    for (int b0 = 0; more; b0 += 32) {
        Seq s;
        more = load_seqs(p.c, p.start, p.T, b0, s);
        const Work w = work_of<N>(p, s);
        sum += Cost<N>(p, w).before(w.pages);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum * p.c.H;
}

// A CTA's walk over its share, up to kKP pages of one head at a time.
template <int N>
struct Walk {
    int64_t left;
    int b, h, page, tile0;       // tile0: the sequence's first image
    Work w;
    __device__ void begin(const AttnParams &p, const Place &from, int64_t pages) {
        left = pages;
        b = from.b;
        tile0 = from.tile0;
        w = work_of<N>(p, b);
        skip(p);
        h = static_cast<int>(from.at / w.pages);
        page = static_cast<int>(from.at - static_cast<int64_t>(h) * w.pages);
    }
    __device__ void skip(const AttnParams &p) {
        while (w.pages == 0 && b + 1 < p.c.B) {
            tile0 += w.tiles;
            w = work_of<N>(p, ++b);
        }
    }
    __device__ int count() const { return static_cast<int>(min(left, static_cast<int64_t>(min(kKP, w.pages - page)))); }
    __device__ void next(const AttnParams &p, int done) {
        left -= done;
        page += done;
        if (page < w.pages || left <= 0) return;
        page = 0;
        if (++h < p.c.H) return;
        h = 0;
        tile0 += w.tiles;
        w = work_of<N>(p, ++b);
        skip(p);
    }
};

// The pages of a share and their scales, in order, for a whole warp: three
// batches of up to 32 pages of one head, one page per lane -- the one being
// used, one whose scales are being loaded, one whose table entries are.
template <int N>
struct Feed {
    Walk<N> ahead;
    int page[3], count[3], head[3], used;
    float sk[2];
    __device__ void begin(const AttnParams &p, const Walk<N> &w) {
        ahead = w;
        used = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) fetch(p, i);
        sk[0] = scale(p, 0);
        sk[1] = scale(p, 1);
    }
    // The next batch's table entries.
    __device__ void fetch(const AttnParams &p, int i) {
        page[i] = -1;
        count[i] = 0;
        if (ahead.left <= 0) return;
        count[i] = static_cast<int>(min(ahead.left, static_cast<int64_t>(min(32, ahead.w.pages - ahead.page))));
        head[i] = ahead.h;
        const int lane = threadIdx.x & 31;
        if (lane < count[i]) page[i] = load_page(p.c, ahead.b, ahead.page + lane, p.dev_status);
        ahead.next(p, count[i]);
    }
    __device__ float scale(const AttnParams &p, int i) const {
        return page[i] >= 0 ? p.c.sk[static_cast<int64_t>(page[i]) * p.c.H + head[i]] : 0.0f;
    }
    __device__ void take(const AttnParams &p, int &pg, float &ks) {
        if (used == count[0]) {
            used = 0;
            page[0] = page[1];
            count[0] = count[1];
            head[0] = head[1];
            sk[0] = sk[1];
            page[1] = page[2];
            count[1] = count[2];
            head[1] = head[2];
            sk[1] = scale(p, 1);
            fetch(p, 2);
        }
        pg = __shfl_sync(0xffffffffu, page[0], used);
        ks = __shfl_sync(0xffffffffu, sk[0], used);
        ++used;
    }
};

// ---------------------------------------------------------------------------
// The images
// ---------------------------------------------------------------------------
// One CTA per (tile, head): 16 threads a row, 8 channels each.
template <int N>
__global__ void __launch_bounds__(256) image_kernel(const WeighParams wp) {
    let_next_start();
    const AttnParams &p = wp.a;
    const int h = blockIdx.y, lane16 = threadIdx.x & 15;
    // the tile's sequence
    int b = 0, rest = blockIdx.x;
    {
        const int lane = threadIdx.x & 31;
        int before = 0;
        bool found = false, more = true;
        if (blockIdx.x == 0 && h == 0)
            for (int i = threadIdx.x; i < p.c.B; i += 256)
                if (load_seq(p.c, p.start, p.T, i).bad) report(p.dev_status, kErrInvalid);
        for (int b0 = 0; more && !found; b0 += 32) {
            Seq s;
            more = load_seqs(p.c, p.start, p.T, b0, s);
            const int t = work_of<N>(p, s).tiles;
            int incl = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, static_cast<int>(blockIdx.x) < before + incl);
            if (hit) {
                const int l = __ffs(hit) - 1;
                b = b0 + l;
                rest = blockIdx.x - before - __shfl_sync(0xffffffffu, incl - t, l);
                found = true;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (!found) return;
    }
    const Seq s = load_seq(p.c, p.start, p.T, b);
    const int R = s.n * p.G;
    uint8_t *img = wp.images + (static_cast<int64_t>(h) * wp.tiles + blockIdx.x) * Image<N>::stride;
    uint8_t *sf = img + Image<N>::sf;
    if (N == 16) {
        // the columns of TMEM that no row takes get factors too
        reinterpret_cast<uint32_t *>(sf)[threadIdx.x] = 0x7f7f7f7fu;
        __syncthreads();
    }
    for (int n = threadIdx.x >> 4; n < N; n += 16) {
        const int r = rest * N + n;
        const bool real = r < R;
        const int seen = real ? min(seen_by_row(p, s, r), s.len) : 0;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (real) v = *reinterpret_cast<const uint4 *>(query_row(p, s, h, r) + 8 * lane16);
        bool odd = false;
        uint32_t m = amax_bf16x8(v, odd);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const int e = max(static_cast<int>(m >> 23) - 127 - 7, -100);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float x[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = __uint_as_float(w[k] << 16) * down;
            x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u) * down;
        }
        if (odd) {      // the conversion would turn an infinity into a number
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = scaled_or_nan(x[k], 1.0f);
        }
        uint2 hi, lo;
        float d[4];
        hi.x = e4m3x4(x[0], x[1], x[2], x[3]);
        hi.y = e4m3x4(x[4], x[5], x[6], x[7]);
        e4m3x4_decode(hi.x, d);
        lo.x = e4m3x4(32.0f * (x[0] - d[0]), 32.0f * (x[1] - d[1]), 32.0f * (x[2] - d[2]), 32.0f * (x[3] - d[3]));
        e4m3x4_decode(hi.y, d);
        lo.y = e4m3x4(32.0f * (x[4] - d[0]), 32.0f * (x[5] - d[1]), 32.0f * (x[6] - d[2]), 32.0f * (x[7] - d[3]));
        const uint32_t at = sw128_offset(n, lane16 >> 1) + 8 * (lane16 & 1);
        *reinterpret_cast<uint2 *>(img + at) = hi;
        *reinterpret_cast<uint2 *>(img + Image<N>::lo + at) = lo;
        if ((lane16 & 3) == 0) {
            const int byte = 127 + e;       // 27 .. 247
            uint8_t *q = sf + (n & 31) * 16 + (n >> 5) * 4 + (lane16 >> 2);
            q[0] = static_cast<uint8_t>(byte);
            q[N == 16 ? 256 : 512] = static_cast<uint8_t>(byte - 5);
        }
        if (lane16 == 0) {
            // a row that sees nothing adds nothing: 2^(S c - inf)
            reinterpret_cast<float *>(img + Image<N>::consts)[n] =
                seen > 0 ? -1.4426950408889634f * wp.lse[out_row(p, s, h, r)] : __int_as_float(0xff800000);
            reinterpret_cast<int *>(img + Image<N>::seen)[n] = seen;
        }
    }
}

// ---------------------------------------------------------------------------
// The sums
// ---------------------------------------------------------------------------
// Instruction descriptor of the block-scaled FP8 MMA, B's factor byte `sf` of its word, A's byte 0.
__host__ __device__ constexpr uint32_t make_idesc_mxf8_b(int M, int N, uint32_t sf) {
    return (sf << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void mma_mxf8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}
// A plain matrix of 16-byte rows one after another, 32 rows into TMEM columns
// taddr .. taddr + 3 of every lane quarter, before the MMAs issued after it.
__device__ __forceinline__ void copy_factors(uint32_t taddr, uint32_t saddr) {
    uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (1ull << 16) | (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// The sum of 2^(S c + (-lse)) over kCols rows of S^T, S, none of them larger than
// `top`, capped first where there is a cap; `lse` their -lse as pairs.
template <int kCols, bool kCap, bool kEdge>
__device__ __forceinline__ uint64_t sum_cols(uint32_t (&X)[kCols], float c, const uint64_t *lse, const int *seen, int key,
                                             float cap_out, float top, uint64_t sum2) {
    if constexpr (kCap) cap_scores(X, c, cap_out, __all_sync(0xffffffffu, top * c <= kTanhNear), [&](int k) { return lse[k / 2]; });
    const uint64_t c2 = pk2(__float_as_uint(c), __float_as_uint(c));
#pragma unroll
    for (int k = 0; k < kCols / 2; ++k) {
        float a = __uint_as_float(X[2 * k]), b = __uint_as_float(X[2 * k + 1]);
        if constexpr (!kCap) upk2(fma2(pk2(X[2 * k], X[2 * k + 1]), c2, lse[k]), a, b);
        a = ex2_approx(a);
        b = ex2_approx(b);
        if constexpr (kEdge) {
            if (key >= seen[2 * k]) a = 0.0f;
            if (key >= seen[2 * k + 1]) b = 0.0f;
        }
        sum2 = add2(sum2, pk2(__float_as_uint(a), __float_as_uint(b)));
    }
    return sum2;
}

// A key's sum over the rows whose -lse this thread holds, S^T's first of them at tS.
template <int N, bool kCap, bool kEdge>
__device__ __forceinline__ float sum_row(uint32_t tS, float c, const uint64_t *lse, const int *seen, int key, float cap_out) {
    uint32_t X0[32];
    uint64_t sum2 = 0;
    float top = 0.0f;
    if constexpr (kCap)
        VCA_TMEM_LDTOP32(tS, X0, top);
    else
        VCA_TMEM_LD32(tS, X0);
    if constexpr (N == 16) {
        tmem_ld_wait();
        uint32_t X[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) X[k] = __float_as_uint(__fadd_rn(__uint_as_float(X0[k]), __uint_as_float(X0[16 + k])));
        sum2 = sum_cols<16, kCap, kEdge>(X, c, lse, seen, key, cap_out, 2.0f * top, sum2);
    } else {
        uint32_t X1[32];
        tmem_ld_wait();
        if constexpr (!kCap) VCA_TMEM_LD32(tS + 32, X1);      // (a cap has no registers left for it)
        sum2 = sum_cols<32, kCap, kEdge>(X0, c, lse, seen, key, cap_out, top, sum2);
        if constexpr (kCap) VCA_TMEM_LDTOP32(tS + 32, X1, top);
        tmem_ld_wait();
        sum2 = sum_cols<32, kCap, kEdge>(X1, c, lse + 16, seen + 32, key, cap_out, top, sum2);
    }
    float a, b;
    upk2(sum2, a, b);
    return a + b;
}

template <int N, bool kCap>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_kernel(const __grid_constant__ CUtensorMap tmK, const WeighParams wp) {
    using L = Layout<N>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L::offBar), *k_empty = k_full + kKStages;
    uint64_t *q_full = k_empty + kKStages, *q_empty = q_full + L::qstages;
    uint64_t *s_full = q_empty + L::qstages, *s_empty = s_full + L::sbufs, *drain = s_empty + L::sbufs;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::offMisc);
    int *abort_flag = reinterpret_cast<int *>(smem + L::offMisc + 4);
    float2 *sSlot = reinterpret_cast<float2 *>(smem + L::offSlot);      // page (bits), its scale
    const AttnParams &p = wp.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int64_t all = all_work<N>(p), share = (all + gridDim.x - 1) / gridDim.x;
    // whoever returns here waits too: the call's end is the end of both kernels
    if (share * blockIdx.x >= all) return wait_for_results();
    const Place from = find_place<N>(p, share * blockIdx.x);
    const Place to = find_place<N>(p, min(all, share * (blockIdx.x + 1)));
    if (to.linear <= from.linear) return wait_for_results();
    Walk<N> wk;
    wk.begin(p, from, to.linear - from.linear);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(k_full + s, 1);
            mbar_init(k_empty + s, 1);
        }
        for (int s = 0; s < L::qstages; ++s) {
            mbar_init(q_full + s, 1);
            mbar_init(q_empty + s, kIssuers + 4 * kSets);       // the MMAs' commits, the sum warps
        }
        for (int s = 0; s < L::sbufs; ++s) {
            mbar_init(s_full + s, 2);            // the MMA's commit, the issuer itself
            mbar_init(s_empty + s, N == 128 ? 4 * kSets : 4);
        }
        for (int i = 0; i < kIssuers; ++i) mbar_init(drain + i, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, L::tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // A's factors are 1 everywhere
    if (warp > kIssuers && warp <= kIssuers + 4) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                         tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + L::tmem_sfa), "r"(0x7f7f7f7fu) : "memory");
        tmem_st_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_for_results();

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        bool ok = true;
        int kn = 0, qn = 0;      // pages and tiles issued
        // pages and scales come 32 at a time, one per lane, two batches ahead: a
        // load under full traffic takes longer than a unit's pages
        Feed<N> feed;
        feed.begin(p, wk);
        while (ok && wk.left > 0) {
            const int kp = wk.count();
            for (int j = 0; ok && j < kp; ++j) {
                int pg;
                float ks;
                feed.take(p, pg, ks);
                const int st = kn % kKStages;
                if (kn >= kKStages) ok = mbar_wait(k_empty + st, (kn / kKStages - 1) & 1, abort_flag, p.limit_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    sSlot[kn % kSlots] = make_float2(__int_as_float(pg), ks);
                    if (pg >= 0) {
                        mbar_expect_tx(k_full + st, kTile);
                        tma_load_2d(smem + st * kTile, &tmK, k_full + st, 0, (pg * p.c.H + wk.h) * kBlk);
                    } else {
                        mbar_arrive(k_full + st);
                    }
                }
                ++kn;
            }
            for (int t = first_tile<N>(p, wk.w.s, wk.page); ok && t < wk.w.tiles; ++t) {
                const int st = qn % L::qstages;
                if (qn >= L::qstages) ok = mbar_wait(q_empty + st, (qn / L::qstages - 1) & 1, abort_flag, p.limit_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    mbar_expect_tx(q_full + st, Image<N>::bytes);
                    bulk_load(smem + L::offQ + st * Image<N>::stride,
                              wp.images + (static_cast<int64_t>(wk.h) * wp.tiles + wk.tile0 + t) * Image<N>::stride,
                              Image<N>::bytes, q_full + st);
                }
                ++qn;
            }
            if (ok) wk.next(p, kp);
        }
        // every copy issued has landed before the CTA can exit
        if (lane == 0) {
            for (int k = max(0, kn - kKStages); k < kn; ++k) drain_wait(k_full + k % kKStages, (k / kKStages) & 1, p.limit_ns);
            for (int k = max(0, qn - L::qstages); k < qn; ++k)
                drain_wait(q_full + k % L::qstages, (k / L::qstages) & 1, p.limit_ns);
        }
    } else if (warp <= kIssuers) {
        // ------------------------------------------------------------ MMA issuers
        // one thread each: issuing costs more than the tensor core takes
        if (lane == 0) {
            const int odd = warp - 1, sb0 = N == 128 ? 0 : odd * L::ring;
            const uint32_t sbase = smem_u32(smem), tsfa = tmem + L::tmem_sfa;
            bool ok = true;
            int kn = 0, qs = 0, sb = 0;
            uint32_t qphase = 0, sphase = 1;       // a buffer's first use waits for nothing
            while (ok && wk.left > 0) {
                const int kp = wk.count();
                int landed = 0;
                for (int t = first_tile<N>(p, wk.w.s, wk.page); ok && t < wk.w.tiles; ++t) {
                    const int np = pages_seen<N>(p, wk.w.s, t, wk.page, kp);
                    ok = mbar_wait_spin(q_full + qs, qphase, abort_flag, p.limit_ns);
                    if (!ok) break;
                    const uint32_t img = sbase + L::offQ + qs * Image<N>::stride, tsf = tmem + L::tmem_sfb + 8 * (2 * qs + odd);
                    copy_factors(tsf, img + Image<N>::sf);
                    if constexpr (N == 128) copy_factors(tsf + 4, img + Image<N>::sf + 512);
                    const uint64_t dh = sdesc_k_sw128(img), dl = sdesc_k_sw128(img + Image<N>::lo);
                    for (int j = 0; j < np; ++j) {
                        const bool mine = (j & 1) == odd;
                        if (mine) {
                            const int st = (kn + j) % kKStages;
                            if (j >= landed) {
                                ok = mbar_wait_spin(k_full + st, ((kn + j) / kKStages) & 1, abort_flag, p.limit_ns);
                                landed = j + 1;
                            }
                            ok = ok && mbar_wait_spin(s_empty + sb0 + sb, sphase, abort_flag, p.limit_ns);
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t dk = sdesc_k_sw128(sbase + st * kTile);
                            const uint32_t d = tmem + (sb0 + sb) * L::cols;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_mxf8_ss(d, dk + 2 * i, dh + 2 * i, make_idesc_mxf8_b(128, L::cols, i), tsfa, tsf, i > 0);
                            if constexpr (N == 128) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    mma_mxf8_ss(d, dk + 2 * i, dl + 2 * i, make_idesc_mxf8_b(128, L::cols, i), tsfa, tsf + 4, 1u);
                            }
                            tc_commit(s_full + sb0 + sb);
                            mbar_arrive(s_full + sb0 + sb);
                            if (t + 1 == wk.w.tiles) tc_commit(k_empty + st);
                        }
                        if ((N == 128 || mine) && ++sb == L::ring) {
                            sb = 0;
                            sphase ^= 1;
                        }
                    }
                    if (ok) tc_commit(q_empty + qs);
                    if (++qs == L::qstages) {
                        qs = 0;
                        qphase ^= 1;
                    }
                }
                kn += kp;
                if (ok) wk.next(p, kp);
            }
            tc_commit(drain + odd);
            drain_wait(drain + odd, 0, p.limit_ns);
        }
    } else {
        // ------------------------------------------------------------ sums
        // 128 rows: each set takes half of every page's rows, whose -lse it keeps in
        // registers for the unit's pages (read from shared memory by every page they
        // take more of its bandwidth than the products do); 16 rows: every other page
        const int set = (warp - 1 - kIssuers) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        constexpr int kCols = N == 128 ? 64 : 16;
        const int col0 = N == 128 ? 64 * set : 0, sb0 = N == 128 ? 0 : set * L::ring;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + col0;
        const float c0 = kCap ? p.cap_in : p.scale_log2;
        float *sSum = reinterpret_cast<float *>(smem + L::offSum);
        bool ok = true;
        int kn = 0, qn = 0, un = 0, next_sb = 0;
        uint32_t next_phase = 0;
        while (ok && wk.left > 0) {
            const int kp = wk.count();
            float acc[kKP] = {};
            int page[kKP] = {-1, -1, -1, -1};
            for (int t = first_tile<N>(p, wk.w.s, wk.page); ok && t < wk.w.tiles; ++t, ++qn) {
                const int qs = qn % L::qstages;
                ok = __all_sync(0xffffffffu, mbar_wait(q_full + qs, (qn / L::qstages) & 1, abort_flag, p.limit_ns));
                if (!ok) break;
                const unsigned char *img = smem + L::offQ + qs * Image<N>::stride;
                const int *seen = reinterpret_cast<const int *>(img + Image<N>::seen) + col0;
                const int all_see = seen_by_row(p, wk.w.s, t * N), np = pages_seen<N>(p, wk.w.s, t, wk.page, kp);
                uint64_t lse[kCols / 2];
#pragma unroll
                for (int k = 0; k < kCols / 4; ++k) {
                    const ulonglong2 x = reinterpret_cast<const ulonglong2 *>(img + Image<N>::consts)[col0 / 4 + k];
                    lse[2 * k] = x.x;
                    lse[2 * k + 1] = x.y;
                }
#pragma unroll
                for (int j = 0; j < kKP; ++j) {
                    if (!ok || j >= np) break;
                    if (N == 16 && (j & 1) != set) continue;
                    const int sb = sb0 + next_sb;
                    const uint32_t phase = next_phase;
                    if (++next_sb == L::ring) {
                        next_sb = 0;
                        next_phase ^= 1;
                    }
                    ok = __all_sync(0xffffffffu, mbar_wait(s_full + sb, phase, abort_flag, p.limit_ns));
                    if (!ok) break;
                    tc_fence_after();
                    const float2 slot = sSlot[(kn + j) % kSlots];      // rewritten once its page's S is given back
                    page[j] = __float_as_int(slot.x);
                    const int key = (wk.page + j) * kBlk + row;
                    const uint32_t tS = tl + sb * L::cols;
                    acc[j] += (wk.page + j + 1) * kBlk > all_see
                                  ? sum_row<N, kCap, true>(tS, c0 * slot.y, lse, seen, key, p.cap_out)
                                  : sum_row<N, kCap, false>(tS, c0 * slot.y, lse, seen, key, p.cap_out);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty + sb);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(q_empty + qs);
            }
            if constexpr (N == 128) {
                // the second set's sums to the first, in buffers by turns: a buffer is
                // written again only behind the barrier after the one its reads precede
                float *buf = sSum + (un & 1) * kKP * kBlk;
                if (set == 1)
#pragma unroll
                    for (int j = 0; j < kKP; ++j) buf[j * kBlk + row] = acc[j];
                ok = bar_and(ok, kBarSums, 32 * 4 * kSets);
                if (set == 0)
#pragma unroll
                    for (int j = 0; j < kKP; ++j) acc[j] += buf[j * kBlk + row];
                ++un;
            }
            if (!ok) break;
            if (N == 16 || set == 0) {
#pragma unroll
                for (int j = 0; j < kKP; ++j)
                    if (page[j] >= 0 && (wk.page + j) * kBlk + row < wk.w.s.len)
                        atomicAdd(wp.weight + (static_cast<int64_t>(page[j]) * p.c.H + wk.h) * kBlk + row, acc[j]);
            }
            kn += kp;
            wk.next(p, kp);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::tmem_cols);
    }
    if (threadIdx.x == 0 && *reinterpret_cast<volatile int *>(abort_flag)) report(p.dev_status, kErrTimeout);
}

// Tiles of 16 rows where a sequence and KV head have at most 32 on average: a
// tile of 128 takes the products of 128 rows however many it has.  16 x 8 heads of
// 8,000 tokens, 16 rows each: 34 us against 56; 32 rows 54 against 57; 48 rows
// 73 against 58.
bool few_rows(int T, int Hq, int H, int B) { return static_cast<int64_t>(T) * (Hq / H) <= 32ll * B; }
int64_t tiles_at_most(int T, int Hq, int H, int B) {
    return static_cast<int64_t>(T) * (Hq / H) / (few_rows(T, Hq, H, B) ? 16 : 128) + (B < T ? B : T);
}

template <int N>
cudaError_t launch(const CacheWeighArgs &a, const WeighParams &wp, cudaStream_t st) {
    CUtensorMap mk;
    if (!make_tile_map(&mk, a.c.k8, static_cast<uint64_t>(a.c.pages) * a.c.H * kBlk)) return cudaErrorInvalidValue;
    const auto kernel = a.softcap > 0.0f ? weigh_kernel<N, true> : weigh_kernel<N, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<N>::smem);
    if (e != cudaSuccess) return e;
    image_kernel<N><<<dim3(wp.tiles, a.c.H), 256, 0, st>>>(wp);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t pages = static_cast<int64_t>(a.c.cols) * a.c.B * a.c.H;
    return launch_after(kernel, dim3(static_cast<unsigned>(pages < 152 ? pages : 152)), kThreads, Layout<N>::smem, st, mk, wp);
}

}  // namespace

size_t cache_weigh_workspace(int T, int Hq, int H, int B, int cols) {
    (void)cols;
    return static_cast<size_t>(tiles_at_most(T, Hq, H, B)) * H *
           (few_rows(T, Hq, H, B) ? Image<16>::stride : Image<128>::stride);
}

cudaError_t launch_cache_weigh(const CacheWeighArgs &a, cudaStream_t st) {
    WeighParams wp;
    wp.a = attn_params(a.c, a.q, a.start, a.T, a.Hq, a.causal, a.scale, a.softcap, a.dev_status, a.wait_limit_ns);
    wp.lse = a.lse;
    wp.weight = a.weight;
    wp.images = static_cast<uint8_t *>(a.ws);
    wp.tiles = static_cast<int>(tiles_at_most(a.T, a.Hq, a.c.H, a.c.B));
    return few_rows(a.T, a.Hq, a.c.H, a.c.B) ? launch<16>(a, wp, st) : launch<128>(a, wp, st);
}

}  // namespace vca
