// vca_cache_attention.cu -- attention over the 8-bit cache for few query rows
// (a token or a few of every sequence), bound by reading the codes once.
//
//   s_j = c (q . k_j), c = softmax_scale log2(e) sk(page);  with a cap
//   s_j = cap tanh(softmax_scale sk (q . k_j) / cap) log2(e);
//   O = sum_j 2^(s_j - m) sv(page) v_j / l,  l = sum_j 2^(s_j - m),
//   lse = ln 2 (m + log2 l), m the running maximum.
//
// The query rows of one (sequence, KV head) -- its new tokens times the G query
// heads that share the KV head -- are cut into tiles of 8.  The work is the
// list of all (sequence, KV head, tile, page) units in that order; each CTA
// takes an equal share of consecutive units, whatever the sequences' lengths,
// and writes an (O, m, l) partial where a tile's pages are shared between CTAs;
// a second kernel joins those.  The order of the sums is fixed, so equal calls
// give equal bits.  Short caches of few tiles are not cut: a CTA for each tile
// is done before a second kernel would be.
//
// One producer warp keeps a ring of pages (K and V tile, 16 KB each, one TMA
// load per tile) full across tile borders; their table entries and scales are
// loaded two batches ahead, since a load under full traffic takes longer than a
// page.  Eight consumer warps take 16 keys of every page each, with a running
// maximum, sum and O of their own, which they merge at a tile's end: no barrier
// but the ring's in between.
//
// Both products are m16n8k16 MMAs on fp16 with the long side as rows, so that
// eight query rows fill a tile: S^T = K Q^T (16 keys x 8 rows), then O^T = V^T P^T
// (16 channels x 8 rows), P^T being S^T's registers after an 8 x 8 transpose.  The
// codes are the A operands: an E4M3 code is exact in fp16, and so is a bf16
// query row after a power-of-two scaling that puts its largest element at 2^13
// (elements below 2^-30 of it lose bits); P is rounded to fp16 (2^-12
// relative), while l sums the unrounded values.
//
// One token for each of 32 sequences of up to 32,768 tokens, 40 heads over 8: 190
// us, 6.4 TB/s (0.94 of a copy); for one of 131,072 tokens with 40 KV heads 207 us,
// 6.5 TB/s.  A tile's issue slots are 37 % used, so that capped scores cost
// 9 us of the 190 more.
#include "vca_attention_common.cuh"
#include "vca_cache.cuh"

namespace vca {

namespace {

using namespace cache;

constexpr int kWarps = 8;                       // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr uint32_t kTile = kBlk * kD;           // bytes of one K or V tile
constexpr int kSmallest = 2;                    // units a CTA takes at least

constexpr int kRows = 8;                        // query rows of a tile
constexpr int kKeys = kBlk / kWarps;            // keys of a page per warp
constexpr int kStages = 5;
constexpr int kPartFloats = kRows * kD + 2 * kRows;      // O, m and l of a part of a tile

// Shared memory: the ring, the warps' O, m and l, the pages' scales, barriers.
constexpr uint32_t kOffMerge = kStages * 2 * kTile;                  // fp32 [8][8][128]
constexpr uint32_t kOffML = kOffMerge + kWarps * kRows * kD * 4;     // fp32 [8][8] m, [8][8] l
constexpr uint32_t kOffScale = kOffML + 2 * kWarps * kRows * 4;      // fp32 [stages][2]
constexpr uint32_t kOffBar = kOffScale + kStages * 8;
constexpr uint32_t kSmem = kOffBar + 2 * kStages * 8 + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

// ---------------------------------------------------------------------------
// The list of units
// ---------------------------------------------------------------------------
// Tiles and pages of a sequence; a sequence with rows but no tokens has one
// (empty) page so that its rows are written.
struct Shape {
    Seq s;
    int tiles, pages;
};
__device__ __forceinline__ Shape shape_of(const AttnParams &p, const Seq &s) {
    Shape x;
    x.s = s;
    x.tiles = static_cast<int>((static_cast<int64_t>(x.s.n) * p.G + kRows - 1) / kRows);
    x.pages = x.s.bad ? 0 : max(1, (x.s.len + kBlk - 1) / kBlk);
    return x;
}
__device__ __forceinline__ int64_t units_of(const AttnParams &p, const Shape &x) {
    return static_cast<int64_t>(x.tiles) * (p.whole ? min(x.pages, 1) : x.pages) * p.c.H;
}

__device__ __forceinline__ int64_t warp_incl_scan(int64_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// Units of all sequences (a warp's work).
__device__ int64_t count_units(const AttnParams &p) {
    int64_t all = 0;
    bool more = true;
    for (int b0 = 0; more; b0 += 32) {
        Seq s;
        more = load_seqs(p.c, p.start, p.T, b0, s);
        all += __shfl_sync(0xffffffffu, warp_incl_scan(units_of(p, shape_of(p, s))), 31);
    }
    return all;
}

// The share of every CTA.
__device__ __forceinline__ int64_t share_of(const AttnParams &p, int64_t all, int ctas) {
    const int64_t s = (all + ctas - 1) / ctas;
    return p.whole ? 1 : s < kSmallest ? kSmallest : s;
}

// Where unit u lies: sequence, and the unit's place among the sequence's.
__device__ void find_unit(const AttnParams &p, int64_t u, int &b_out, int64_t &local) {
    int64_t before = 0;
    bool more = true;
    for (int b0 = 0; more; b0 += 32) {
        Seq s;
        more = load_seqs(p.c, p.start, p.T, b0, s);
        const int64_t v = units_of(p, shape_of(p, s));
        const int64_t incl = warp_incl_scan(v) + before;
        const uint32_t hit = __ballot_sync(0xffffffffu, u < incl);
        if (hit) {
            const int l = __ffs(hit) - 1;
            b_out = b0 + l;
            local = u - __shfl_sync(0xffffffffu, incl - v, l);
            return;
        }
        before = __shfl_sync(0xffffffffu, incl, 31);
    }
    b_out = p.c.B;
    local = 0;
}

// A CTA's walk over its units, one (sequence, head, tile) at a time.
struct Walk {
    int b, h, tile, page;      // the next unit
    int64_t left;              // units left in the share
    Shape x;
    __device__ void begin(const AttnParams &p, int b_, int64_t local, int64_t units) {
        b = b_;
        left = units;
        if (b < p.c.B) {
            x = shape_of(p, load_seq(p.c, p.start, p.T, b));
            if (p.whole) {
                h = static_cast<int>(local / x.tiles);
                tile = static_cast<int>(local - static_cast<int64_t>(h) * x.tiles);
                page = 0;
                left = x.pages;
                return;
            }
            h = static_cast<int>(local / (static_cast<int64_t>(x.tiles) * x.pages));
            const int64_t r = local - static_cast<int64_t>(h) * x.tiles * x.pages;
            tile = static_cast<int>(r / x.pages);
            page = static_cast<int>(r - static_cast<int64_t>(tile) * x.pages);
        }
    }
    // Pages of the current tile in this share.
    __device__ int run() const { return static_cast<int>(left < x.pages - page ? left : x.pages - page); }
    __device__ void next(const AttnParams &p, int done) {
        left -= done;
        page += done;
        if (page < x.pages) return;
        page = 0;
        if (++tile < x.tiles) return;
        tile = 0;
        if (++h < p.c.H) return;
        h = 0;
        do {
            ++b;
            if (b >= p.c.B) return;
            x = shape_of(p, load_seq(p.c, p.start, p.T, b));
        } while (x.tiles == 0 || x.pages == 0);
    }
};

// ---------------------------------------------------------------------------
// The products
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The low and the high pair of four codes as fp16 pairs.
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint4 lds128(const unsigned char *p) { return *reinterpret_cast<const uint4 *>(p); }

// 8 x 8 transpose of 16-bit elements held as an MMA fragment.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
    return d;
}

// The 32 channels t * 32 .. t * 32 + 31 of one query row as fp16 pairs, scaled
// by a power of two; returns the factor's inverse.  All four threads of a quad
// hold a quarter of the same row.
__device__ __forceinline__ float load_q(const AttnParams &p, const Seq &s, int h, int r, int t, uint32_t (&q)[16]) {
    uint4 v[4];
    const bool real = r < s.n * p.G;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_uint4(0, 0, 0, 0);
    if (real) {
        const uint4 *at = reinterpret_cast<const uint4 *>(query_row(p, s, h, r) + t * 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = at[i];
    }
    uint32_t m = 0;
    bool odd = false;      // an infinity or NaN is one in fp16 too
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, amax_bf16x8(v[i], odd));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // 2^(13 - e), e the largest element's exponent, kept where both it and its inverse are normal
    const int e = max(static_cast<int>(m >> 23) - 127, -100);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 13 - e) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            q[4 * i + k] = pack_half2(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xffff0000u) * up);
    }
    return __uint_as_float(static_cast<uint32_t>(127 - 13 + e) << 23);
}

// The pages of a share and their scales, in order, for a whole warp: three
// batches of up to 32 pages of one tile, one page per lane -- the one being
// used, one whose scales are being loaded, one whose table entries are.
struct Feed {
    Walk ahead;
    int page[3], count[3], head[3], used;
    bool real[3];
    float sk[2], sv[2];
    __device__ void begin(const AttnParams &p, const Walk &w) {
        ahead = w;
        used = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) fetch(p, i);
        scales(p, 0);
        scales(p, 1);
    }
    __device__ void fetch(const AttnParams &p, int i) {
        page[i] = -1;
        count[i] = head[i] = 0;
        real[i] = false;
        if (ahead.left <= 0) return;
        count[i] = min(32, ahead.run());
        head[i] = ahead.h;
        const int lane = threadIdx.x & 31;
        // checked when its scales are fetched: the load is not waited for here
        if (lane < count[i] && ahead.x.s.len > 0)
            page[i] = p.c.table[static_cast<int64_t>(ahead.b) * p.c.cols + ahead.page + lane];
        real[i] = lane < count[i] && ahead.x.s.len > 0;
        ahead.next(p, count[i]);
    }
    __device__ void scales(const AttnParams &p, int i) {
        if (page[i] < 0 || page[i] >= p.c.pages) {
            if (real[i]) report(p.dev_status, kErrInvalid);
            page[i] = -1;
        }
        const int64_t at = static_cast<int64_t>(page[i]) * p.c.H + head[i];
        sk[i] = page[i] >= 0 ? p.c.sk[at] : -1.0f;      // -1: no page
        sv[i] = page[i] >= 0 ? p.c.sv[at] : 0.0f;
    }
    // The next page: its tile's first row of codes (negative: no page) and its scales.
    __device__ void take(const AttnParams &p, int &y, float &ks, float &vs) {
        if (used == count[0]) {
            used = 0;
            page[0] = page[1];
            count[0] = count[1];
            head[0] = head[1];
            sk[0] = sk[1];
            sv[0] = sv[1];
            page[1] = page[2];
            count[1] = count[2];
            head[1] = head[2];
            real[1] = real[2];
            scales(p, 1);
            fetch(p, 2);
        }
        const int pg = __shfl_sync(0xffffffffu, page[0], used);
        y = pg < 0 ? -1 : (pg * p.c.H + head[0]) * kBlk;
        ks = __shfl_sync(0xffffffffu, sk[0], used);
        vs = __shfl_sync(0xffffffffu, sv[0], used);
        ++used;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBar), *empty = full + kStages;
    int *abort_flag = reinterpret_cast<int *>(empty + kStages);
    float *sScale = reinterpret_cast<float *>(smem + kOffScale);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, kWarps);
        }
        *abort_flag = 0;
        mbar_fence_init();
    }
    __syncthreads();
    let_next_start();
    const int64_t all = count_units(p), share = share_of(p, all, gridDim.x);
    const int64_t u0 = share * blockIdx.x, u1 = min(all, u0 + share);
    if (blockIdx.x == 0 && warp == 0)
        for (int b = lane; b < p.c.B; b += 32)
            if (load_seq(p.c, p.start, p.T, b).bad) report(p.dev_status, kErrInvalid);
    if (u0 >= u1) return;
    int b0;
    int64_t local;
    find_unit(p, u0, b0, local);
    Walk w;
    w.begin(p, b0, local, u1 - u0);

    if (warp == kWarps) {
        // ------------------------------------------------------------ producer
        int stage = 0, round = 0;
        const int64_t units = w.left;
        int armed = 0;
        bool ok = true;
        Feed feed;
        feed.begin(p, w);
        for (int64_t i = 0; i < units; ++i) {
            int y;
            float ks, vs;
            feed.take(p, y, ks, vs);
            if (round > 0) ok = mbar_wait(empty + stage, (round - 1) & 1, abort_flag, p.limit_ns);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) {
                sScale[2 * stage] = ks;
                sScale[2 * stage + 1] = vs;
                if (y >= 0) {
                    unsigned char *at = smem + stage * 2 * kTile;
                    mbar_expect_tx(full + stage, 2 * kTile);
                    tma_load_2d(at, &tmK, full + stage, 0, y);
                    tma_load_2d(at + kTile, &tmV, full + stage, 0, y);
                } else {
                    mbar_arrive(full + stage);
                }
            }
            ++armed;
            if (++stage == kStages) {
                stage = 0;
                ++round;
            }
        }
        // every copy issued has landed before the CTA can exit
        if (lane == 0)
            for (int k = max(0, armed - kStages); k < armed; ++k)
                attn::drain_wait(full + k % kStages, (k / kStages) & 1, p.limit_ns);
    } else {
        // ------------------------------------------------------------ consumers
        // fragments: g and t are the row (key, channel or query row) and the pair of a quad
        const int g = lane >> 2, t = lane & 3;
        float *sMerge = reinterpret_cast<float *>(smem + kOffMerge);
        float *sM = reinterpret_cast<float *>(smem + kOffML), *sL = sM + kWarps * kRows;
        const int64_t u_left = w.left;
        int stage = 0, round = 0;
        bool ok = true;
        const float kNegInf = __int_as_float(0xff800000);
        while (w.left > 0) {
            const int run = w.run();
            const Seq s = w.x.s;
            const int R = s.n * p.G, r0 = w.tile * kRows;
            // Q: the B operand, row g; this thread's scores are of the rows 2 t and 2 t + 1
            uint32_t q[16];
            float f[2], m[2], l[2];
            int seen[2];
            const float down = load_q(p, s, w.h, r0 + g, t, q);
            const float fg = __fmul_rn(p.cap_out != 0.0f ? p.cap_in : p.scale_log2, down);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = r0 + 2 * t + e;
                f[e] = __shfl_sync(0xffffffffu, fg, (2 * t + e) * 4);
                seen[e] = r < R ? seen_by_row(p, s, r) : 0;
                m[e] = kNegInf;
                l[e] = 0.0f;
            }
            const int all_see = seen_by_row(p, s, r0);      // keys below this are seen by every row of the tile
            // O^T: channel 16 g + 2 j (elements 0, 1) and 16 g + 2 j + 1 (2, 3) of the rows 2 t, 2 t + 1
            float o[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;

            for (int i = 0; i < run; ++i) {
                if (ok) ok = mbar_wait(full + stage, round & 1, abort_flag, p.limit_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const float sk = sScale[2 * stage], sv = sScale[2 * stage + 1];
                const int key0 = (w.page + i) * kBlk + kKeys * warp;
                if (sk >= 0.0f && key0 < s.len) {
                    const unsigned char *sK = smem + stage * 2 * kTile, *sV = sK + kTile;
                    float S[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    // K: keys g and g + 8; the four codes of a word are channels 32 t + 4 k .. + 3
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t ka[4], kb[4];
                        *reinterpret_cast<uint4 *>(ka) = lds128(sK + sw128_offset(kKeys * warp + g, 2 * t + half));
                        *reinterpret_cast<uint4 *>(kb) = lds128(sK + sw128_offset(kKeys * warp + 8 + g, 2 * t + half));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t a[4];
                            codes_to_half(ka[k], a[0], a[2]);
                            codes_to_half(kb[k], a[1], a[3]);
                            mma16816(S, a, q[8 * half + 2 * k], q[8 * half + 2 * k + 1]);
                        }
                    }
                    uint32_t vw[4][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint4 *>(vw[k]) =
                            lds128(sV + sw128_offset(kKeys * warp + 2 * t + (k & 1) + 8 * (k >> 1), g));
                    // the last page's slots behind the last token may hold anything
                    if (key0 + kKeys > s.len) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (key0 + 2 * t + (k & 1) + 8 * (k >> 1) >= s.len)
                                vw[k][0] = vw[k][1] = vw[k][2] = vw[k][3] = 0u;
                    }
                    // scores in log2 units, the running maximum, P; element e: key g + 8 (e >> 1), row 2 t + (e & 1)
                    const bool edge = key0 + kKeys > all_see;
                    float alpha[2], mx[2] = {m[0], m[1]};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = scored(S[e], f[e & 1] * sk, p.cap_out);
                        if (edge && key0 + g + 8 * (e >> 1) >= seen[e & 1]) x = kNegInf;
                        S[e] = x;
                        mx[e & 1] = fmaxf(mx[e & 1], x);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 4));
                        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 8));
                        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 16));
                        const float mu = mx[e] == kNegInf ? 0.0f : mx[e];      // a row that sees nothing yet
                        alpha[e] = ex2_approx(m[e] - mu);
                        m[e] = mx[e];
                        S[e] = ex2_approx(S[e] - mu);
                        S[e + 2] = ex2_approx(S[e + 2] - mu);
                        l[e] = fmaf(l[e], alpha[e], S[e] + S[e + 2]);
                    }
                    const uint32_t p0 = transpose8x8(pack_half2(S[0], S[1])), p1 = transpose8x8(pack_half2(S[2], S[3]));
                    // this page's P V in the codes' units, then O = O alpha + sv (P V): the page
                    // scales may differ by any power of two
                    const uint64_t sv2 = pk2(__float_as_uint(sv), __float_as_uint(sv));
                    const uint64_t al = pk2(__float_as_uint(alpha[0]), __float_as_uint(alpha[1]));
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
                        uint32_t a[4];
                        codes_to_half(prmt(vw[0][j >> 1], vw[1][j >> 1], sel), a[0], a[1]);
                        codes_to_half(prmt(vw[2][j >> 1], vw[3][j >> 1], sel), a[2], a[3]);
                        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma16816(d, a, p0, p1);
#pragma unroll
                        for (int e = 0; e < 4; e += 2)
                            upk2(fma2(pk2(__float_as_uint(d[e]), __float_as_uint(d[e + 1])), sv2,
                                      mul2(pk2(__float_as_uint(o[j][e]), __float_as_uint(o[j][e + 1])), al)),
                                 o[j][e], o[j][e + 1]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + stage);
                if (++stage == kStages) {
                    stage = 0;
                    ++round;
                }
            }
            // ---- the warps' (O, m, l) merged: each writes its own, all add them up
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
                const int r = 2 * t + e;
                if (g == 0) {
                    sM[warp * kRows + r] = m[e];
                    sL[warp * kRows + r] = l[e];
                }
                float4 *at = reinterpret_cast<float4 *>(sMerge + (warp * kRows + r) * kD + 16 * g);
#pragma unroll
                for (int j = 0; j < 8; j += 2) at[j / 2] = make_float4(o[j][e], o[j][e + 2], o[j + 1][e], o[j + 1][e + 2]);
            }
            ok = attn::bar_and(ok, 1, 32 * kWarps);
            if (!ok) break;
            {
                const int r = threadIdx.x >> 5, ch = lane * 4;      // row, four channels
                float M = kNegInf;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sM[i * kRows + r]);
                const float Mu = M == kNegInf ? 0.0f : M;
                float sum = 0.0f, acc[4] = {};
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    const float k = ex2_approx(sM[i * kRows + r] - Mu);
                    sum = fmaf(sL[i * kRows + r], k, sum);
                    const float4 x = *reinterpret_cast<const float4 *>(sMerge + (i * kRows + r) * kD + ch);
                    acc[0] = fmaf(x.x, k, acc[0]);
                    acc[1] = fmaf(x.y, k, acc[1]);
                    acc[2] = fmaf(x.z, k, acc[2]);
                    acc[3] = fmaf(x.w, k, acc[3]);
                }
                const int row = r0 + r;
                if (run == w.x.pages) {
                    // the whole tile: the output itself
                    if (row < R) {
                        const int64_t at = out_row(p, s, w.h, row);
                        const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
                        *reinterpret_cast<uint2 *>(p.O + at * kD + ch) =
                            make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
                        if (p.lse && ch == 0) p.lse[at] = Mu * 0.6931471805599453f + logf(sum);
                    }
                } else {
                    // a share of it: slot 0 where the CTA's share begins in this tile, else slot 1
                    float *part = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + (w.left == u_left ? 0 : 1)) * kPartFloats;
                    *reinterpret_cast<float4 *>(part + r * kD + ch) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (ch == 0) {
                        part[kRows * kD + r] = M;
                        part[kRows * kD + kRows + r] = sum;
                    }
                }
            }
            w.next(p, run);
            // the merge buffers are free again once every warp has read them
            attn::bar_sync(1, 32 * kWarps);
        }
        if (!ok && lane == 0) report(p.dev_status, kErrTimeout);
    }
}

// Joins the partials of the tile that straddles the end of CTA blockIdx.x's
// share and begins in it.  One thread per (row, eight channels).
__global__ void __launch_bounds__(16 * kRows) combine_kernel(const AttnParams p, int ctas) {
    const int64_t all = count_units(p), share = share_of(p, all, ctas);
    const int64_t u0 = share * blockIdx.x, u1 = u0 + share;
    // whoever returns here waits too: the call's end is the end of all its kernels
    if (u1 >= all) return wait_for_results();                   // nothing behind this share
    int b;
    int64_t local;
    find_unit(p, u1 - 1, b, local);
    Walk w;
    w.begin(p, b, local, 1);
    if (w.page + 1 == w.x.pages) return wait_for_results();     // its tile ends with the share
    const int64_t begin = u1 - 1 - w.page, end = begin + w.x.pages;
    if (begin < u0) return wait_for_results();                  // it began in an earlier share
    const int r = threadIdx.x >> 4, ch = (threadIdx.x & 15) * 8, row = w.tile * kRows + r;
    const Seq s = w.x.s;
    if (row >= s.n * p.G) return wait_for_results();
    const int last = static_cast<int>((end - 1) / share);
    const float kNegInf = __int_as_float(0xff800000);
    wait_for_results();
    auto part_of = [&](int c) {
        return p.part + (static_cast<int64_t>(c) * 2 + (c == static_cast<int>(blockIdx.x) && begin > u0 ? 1 : 0)) * kPartFloats;
    };
    float M = kNegInf;
#pragma unroll 4
    for (int c = blockIdx.x; c <= last; ++c) M = fmaxf(M, part_of(c)[kRows * kD + r]);
    const float Mu = M == kNegInf ? 0.0f : M;
    float L = 0.0f, acc[8] = {};
#pragma unroll 4
    for (int c = blockIdx.x; c <= last; ++c) {
        const float *part = part_of(c);
        const float k = ex2_approx(part[kRows * kD + r] - Mu);
        L = fmaf(part[kRows * kD + kRows + r], k, L);
        const float4 *at = reinterpret_cast<const float4 *>(part + r * kD + ch);
        const float4 x = at[0], y = at[1];
        acc[0] = fmaf(x.x, k, acc[0]);
        acc[1] = fmaf(x.y, k, acc[1]);
        acc[2] = fmaf(x.z, k, acc[2]);
        acc[3] = fmaf(x.w, k, acc[3]);
        acc[4] = fmaf(y.x, k, acc[4]);
        acc[5] = fmaf(y.y, k, acc[5]);
        acc[6] = fmaf(y.z, k, acc[6]);
        acc[7] = fmaf(y.w, k, acc[7]);
    }
    const int64_t at = out_row(p, s, w.h, row);
    const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;
    uint4 y;
    y.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    y.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    y.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
    y.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
    *reinterpret_cast<uint4 *>(p.O + at * kD + ch) = y;
    if (p.lse && ch == 0) p.lse[at] = Mu * 0.6931471805599453f + logf(L);
}

// CTAs of the decode kernel: one per SM, fewer where there cannot be work for
// all; or one for each tile where caches are of at most kWholePages pages and
// tiles few.  8 heads of one sequence: 500 tokens 7.3 us whole, 7.9 cut; 1,000
// tokens 9.5 whole, 8.5 cut; of eight sequences 7.3 and 8.7, 9.7 and 9.8.
constexpr int kWholePages = 6;
struct Grid {
    int ctas;
    bool whole;
};
Grid grid_of(int T, int Hq, int H, int B, int cols) {
    const int64_t G = Hq / H;
    const int64_t tiles = (static_cast<int64_t>(T) * G / kRows + (B < T ? B : T)) * H;   // at most
    if (cols <= kWholePages && tiles <= 2 * 152) return {static_cast<int>(tiles), true};
    const int64_t most = (tiles * cols + kSmallest - 1) / kSmallest;
    return {static_cast<int>(most < 152 ? most : 152), false};
}

// More than a tile of rows a sequence and KV head on average: the tensor core
// kernel.  16 x 8 heads of 8,000 tokens: 8 rows 50 us here, 66 there; 16 rows 88
// here, 67 there; 32 rows 159 and 68.  (Tiles of 16 rows, by two MMAs a fragment,
// took 1.6 times as long as tiles of eight.)
bool many_rows(int T, int Hq, int H, int B) { return static_cast<int64_t>(T) * (Hq / H) > static_cast<int64_t>(kRows) * B; }

}  // namespace

size_t cache_attention_workspace(int T, int Hq, int H, int B, int cols) {
    if (many_rows(T, Hq, H, B)) return cache_chunk_workspace(T, Hq, H, B, cols);
    const Grid g = grid_of(T, Hq, H, B, cols);
    return static_cast<size_t>(g.ctas) * 2 * kPartFloats * sizeof(float);
}

cudaError_t launch_cache_attention(const CacheAttnArgs &a, cudaStream_t st) {
    if (many_rows(a.T, a.Hq, a.c.H, a.c.B)) return launch_cache_chunk(a, st);
    CUtensorMap mk, mv;
    const uint64_t rows = static_cast<uint64_t>(a.c.pages) * a.c.H * kBlk;
    if (!attn::make_tile_map(&mk, a.c.k8, rows) || !attn::make_tile_map(&mv, a.c.v8, rows)) return cudaErrorInvalidValue;
    AttnParams p = attn_params(a.c, a.q, a.start, a.T, a.Hq, a.causal, a.scale, a.softcap, a.dev_status, a.wait_limit_ns);
    p.O = a.O;
    p.lse = a.lse;
    p.part = static_cast<float *>(a.ws);
    const Grid g = grid_of(a.T, a.Hq, a.c.H, a.c.B, a.c.cols);
    p.whole = g.whole;
    cudaError_t e = cudaFuncSetAttribute(decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    decode_kernel<<<g.ctas, kThreads, kSmem, st>>>(mk, mv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.whole) return e;
    return launch_after(combine_kernel, dim3(g.ctas), 16 * kRows, 0, st, p, g.ctas);
}

}  // namespace vca
