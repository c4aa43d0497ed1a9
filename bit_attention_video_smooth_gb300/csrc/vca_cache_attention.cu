// vca_cache_attention.cu -- attention over the 8-bit cache for few query rows
// (a token or a few of every sequence), bound by reading the codes once.
//
//   s_j = c (q . k_j), c = softmax_scale log2(e) sk(page);  with a cap
//   s_j = cap tanh(softmax_scale sk (q . k_j) / cap) log2(e);
//   O = sum_j 2^(s_j - m) sv(page) v_j / l,  l = sum_j 2^(s_j - m),
//   lse = ln 2 (m + log2 l), m the running maximum.
//
// The query rows of one (sequence, KV head) -- its new tokens times the G query
// heads that share the KV head -- are cut into tiles of 16.  The work is the
// list of all (sequence, KV head, tile, page) units in that order; each CTA
// takes an equal share of consecutive units, whatever the sequences' lengths,
// and writes an (O, m, l) partial where a tile's pages are shared between CTAs;
// a second kernel joins those.  The order of the sums is fixed, so equal calls
// give equal bits.
//
// One producer warp keeps a ring of pages (K and V tile, 16 KB each, one TMA
// load per tile) full across tile borders.  Eight consumer warps take 16 keys of
// every page each, with a running maximum, sum and O of their own, which they
// merge at a tile's end: no barrier but the ring's in between.  Both products
// are m16n8k16 MMAs on fp16: an E4M3 code is exact in fp16, and so is a bf16
// query row after a power-of-two scaling that puts its largest element at 2^13
// (elements below 2^-30 of it lose bits); P is rounded to fp16 (2^-12
// relative), while l sums the unrounded values.
#include "vca_attention_common.cuh"
#include "vca_cache.cuh"

namespace vca {

namespace {

using namespace cache;

constexpr int kRows = 16;                       // query rows of a tile
constexpr int kWarps = 8;                       // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kKeys = kBlk / kWarps;            // keys of a page per warp
constexpr int kStages = 4;
constexpr uint32_t kTile = kBlk * kD;           // bytes of one K or V tile
constexpr int kSmallest = 2;                    // units a CTA takes at least

// One partial: O [16][128], m [16], l [16].
constexpr int kPartFloats = kRows * kD + 2 * kRows;

constexpr uint32_t kOffRing = 0;
constexpr uint32_t kOffMerge = kOffRing + kStages * 2 * kTile;       // fp32 [8][16][128]
constexpr uint32_t kOffML = kOffMerge + kWarps * kRows * kD * 4;     // fp32 [8][16] m, [8][16] l
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
__device__ __forceinline__ Shape shape_of(const AttnParams &p, int b) {
    Shape x;
    x.s = load_seq(p.c, p.start, p.T, b);
    x.tiles = static_cast<int>((static_cast<int64_t>(x.s.n) * p.G + kRows - 1) / kRows);
    x.pages = x.s.bad ? 0 : max(1, (x.s.len + kBlk - 1) / kBlk);
    return x;
}
__device__ __forceinline__ int64_t units_of(const AttnParams &p, const Shape &x) {
    return static_cast<int64_t>(x.tiles) * x.pages * p.c.H;
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
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        const int b = b0 + static_cast<int>(threadIdx.x & 31);
        int64_t v = b < p.c.B ? units_of(p, shape_of(p, b)) : 0;
        all += __shfl_sync(0xffffffffu, warp_incl_scan(v), 31);
    }
    return all;
}

// The share of every CTA.
__device__ __forceinline__ int64_t share_of(int64_t all, int ctas) {
    const int64_t s = (all + ctas - 1) / ctas;
    return s < kSmallest ? kSmallest : s;
}

// Where unit u lies: sequence, and the unit's place among the sequence's.
__device__ void find_unit(const AttnParams &p, int64_t u, int &b_out, int64_t &local) {
    int64_t before = 0;
    const int lane = threadIdx.x & 31;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        const int b = b0 + lane;
        const int64_t v = b < p.c.B ? units_of(p, shape_of(p, b)) : 0;
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
            x = shape_of(p, b);
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
            x = shape_of(p, b);
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

// The 32 channels t * 32 .. t * 32 + 31 of one query row as fp16 pairs, scaled
// by a power of two; returns the factor's inverse.  All four threads of a quad
// hold a quarter of the same row.
__device__ __forceinline__ float load_q(const AttnParams &p, const Seq &s, int h, int r, int t, uint32_t (&q)[16]) {
    uint4 v[4];
    const bool real = r < s.n * p.G;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_uint4(0, 0, 0, 0);
    if (real) {
        const uint16_t *at = p.q.p + (s.row0 + r / p.G) * p.q.tok + (h * p.G + r % p.G) * p.q.head + t * 32;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const uint4 *>(at)[i];
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, amax_bf16x8(v[i]));
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
    const int64_t all = count_units(p), share = share_of(all, gridDim.x);
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
        int stage = 0, round = 0, armed = 0;
        bool ok = true;
        while (ok && w.left > 0) {
            const int run = w.run();
            for (int i0 = 0; ok && i0 < run; i0 += 32) {
                // the next 32 pages and their scales, one per lane
                int page = -1;
                float sk = 0.0f, sv = 0.0f;
                if (i0 + lane < run && w.x.s.len > 0) {
                    page = load_page(p.c, w.b, w.page + i0 + lane, p.dev_status);
                    if (page >= 0) {
                        sk = p.c.sk[static_cast<int64_t>(page) * p.c.H + w.h];
                        sv = p.c.sv[static_cast<int64_t>(page) * p.c.H + w.h];
                    }
                }
                for (int i = 0; i < 32 && i0 + i < run; ++i) {
                    const int pg = __shfl_sync(0xffffffffu, page, i);
                    const float ks = __shfl_sync(0xffffffffu, sk, i), vs = __shfl_sync(0xffffffffu, sv, i);
                    if (round > 0) ok = mbar_wait(empty + stage, (round - 1) & 1, abort_flag, p.limit_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        sScale[2 * stage] = pg >= 0 ? ks : -1.0f;     // -1: no page
                        sScale[2 * stage + 1] = vs;
                        if (pg >= 0) {
                            unsigned char *at = smem + kOffRing + stage * 2 * kTile;
                            const int y = (pg * p.c.H + w.h) * kBlk;
                            mbar_expect_tx(full + stage, 2 * kTile);
                            tma_load_2d(at, &tmK, full + stage, 0, y);
                            tma_load_2d(at + kTile, &tmV, full + stage, 0, y);
                        } else {
                            mbar_arrive(full + stage);
                        }
                    }
                    armed = round * kStages + stage + 1;
                    if (++stage == kStages) {
                        stage = 0;
                        ++round;
                    }
                }
            }
            if (ok) w.next(p, run);
        }
        // every copy issued has landed before the CTA can exit
        if (lane == 0)
            for (int k = max(0, armed - kStages); k < armed; ++k)
                attn::drain_wait(full + k % kStages, (k / kStages) & 1, p.limit_ns);
    } else {
        // ------------------------------------------------------------ consumers
        const int g = lane >> 2, t = lane & 3;
        float *sMerge = reinterpret_cast<float *>(smem + kOffMerge);
        float *sM = reinterpret_cast<float *>(smem + kOffML), *sL = sM + kWarps * kRows;
        int stage = 0, round = 0;
        bool ok = true;
        const float kNegInf = __int_as_float(0xff800000);
        while (w.left > 0) {
            const int run = w.run();
            const Seq s = w.x.s;
            const int R = s.n * p.G, r0 = w.tile * kRows;
            uint32_t q[2][16];
            float f[2];
            int seen[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = r0 + g + 8 * i;
                const float down = load_q(p, s, w.h, r, t, q[i]);
                f[i] = __fmul_rn(p.cap_out != 0.0f ? p.cap_in : p.scale_log2, down);
                seen[i] = r < R ? seen_by_row(p, s, r) : 0;
            }
            const int all_see = seen_by_row(p, s, r0);      // keys below this are seen by every row of the tile
            float m[2] = {kNegInf, kNegInf}, l[2] = {0.0f, 0.0f};
            float o[16][4];
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;

            for (int i = 0; i < run; ++i) {
                if (ok) ok = mbar_wait(full + stage, round & 1, abort_flag, p.limit_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const float sk = sScale[2 * stage], sv = sScale[2 * stage + 1];
                const int key0 = (w.page + i) * kBlk + kKeys * warp;
                const bool edge = key0 + kKeys > all_see;
                // the last page's slots behind the last token may hold anything
                const bool tail = key0 + kKeys > s.len;
                if (sk >= 0.0f && key0 < s.len) {
                    const unsigned char *sK = smem + kOffRing + stage * 2 * kTile, *sV = sK + kTile;
                    float S[2][4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int key = kKeys * warp + 8 * j + g;
                        uint32_t kw[8];
                        *reinterpret_cast<uint4 *>(kw) = lds128(sK + sw128_offset(key, 2 * t));
                        *reinterpret_cast<uint4 *>(kw + 4) = lds128(sK + sw128_offset(key, 2 * t + 1));
#pragma unroll
                        for (int e = 0; e < 4; ++e) S[j][e] = 0.0f;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            uint32_t lo, hi;
                            codes_to_half(kw[k], lo, hi);
                            const uint32_t a[4] = {q[0][2 * k], q[1][2 * k], q[0][2 * k + 1], q[1][2 * k + 1]};
                            mma16816(S[j], a, lo, hi);
                        }
                    }
                    uint32_t vw[4][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tok = kKeys * warp + 2 * t + (k & 1) + 8 * (k >> 1);
                        uint4 x = lds128(sV + sw128_offset(tok, g));
                        if (tail && (w.page + i) * kBlk + tok >= s.len) x = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(vw[k]) = x;
                    }
                    // scores in log2 units, the running maximum, P
                    float mx[2] = {m[0], m[1]};
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float x = scored(S[j][e], f[e >> 1] * sk, p.cap_out);
                            if (edge && key0 + 8 * j + 2 * t + (e & 1) >= seen[e >> 1]) x = kNegInf;
                            S[j][e] = x;
                            mx[e >> 1] = fmaxf(mx[e >> 1], x);
                        }
                    float alpha[2], mu[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                        mu[e] = mx[e] == kNegInf ? 0.0f : mx[e];      // a row that sees nothing yet
                        alpha[e] = ex2_approx(m[e] - mu[e]);
                        l[e] *= alpha[e];
                        m[e] = mx[e];
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            S[j][e] = ex2_approx(S[j][e] - mu[e >> 1]);
                            l[e >> 1] += S[j][e];
                        }
                    const uint32_t a[4] = {pack_half2(S[0][0], S[0][1]), pack_half2(S[0][2], S[0][3]),
                                           pack_half2(S[1][0], S[1][1]), pack_half2(S[1][2], S[1][3])};
                    // this page's P V in the codes' units, then O = O alpha + sv (P V): the page
                    // scales may differ by any power of two
#pragma unroll
                    for (int n = 0; n < 16; n += 2) {
                        const uint32_t sel = (n & 2) ? 0x7362u : 0x5140u;
                        const uint32_t b01 = prmt(vw[0][n >> 2], vw[1][n >> 2], sel);
                        const uint32_t b89 = prmt(vw[2][n >> 2], vw[3][n >> 2], sel);
                        uint32_t x0, x1, y0, y1;
                        codes_to_half(b01, x0, x1);
                        codes_to_half(b89, y0, y1);
                        float d0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, d1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma16816(d0, a, x0, y0);
                        mma16816(d1, a, x1, y1);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            o[n][e] = fmaf(d0[e], sv, o[n][e] * alpha[e >> 1]);
                            o[n + 1][e] = fmaf(d1[e], sv, o[n + 1][e] * alpha[e >> 1]);
                        }
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
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
                if (t == 0) {
                    sM[warp * kRows + g + 8 * e] = m[e];
                    sL[warp * kRows + g + 8 * e] = l[e];
                }
            }
            // column 16 g' + n of the row: the n-th tile's column g', here g' = 2 t + (e & 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float *at = sMerge + (warp * kRows + g + 8 * (e >> 1)) * kD + 16 * (2 * t + (e & 1));
#pragma unroll
                for (int n = 0; n < 16; n += 4)
                    *reinterpret_cast<float4 *>(at + n) = make_float4(o[n][e], o[n + 1][e], o[n + 2][e], o[n + 3][e]);
            }
            ok = attn::bar_and(ok, 1, 32 * kWarps);
            if (!ok) break;
            {
                const int r = threadIdx.x >> 4, ch = (threadIdx.x & 15) * 8;     // row, eight channels
                float M = kNegInf;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sM[i * kRows + r]);
                const float Mu = M == kNegInf ? 0.0f : M;
                float L = 0.0f, acc[8] = {};
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    const float k = ex2_approx(sM[i * kRows + r] - Mu);
                    L = fmaf(sL[i * kRows + r], k, L);
                    const float4 *at = reinterpret_cast<const float4 *>(sMerge + (i * kRows + r) * kD + ch);
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
                const int row = r0 + r;
                if (run == w.x.pages) {
                    // the whole tile: the output itself
                    if (row < R) {
                        const int64_t at = static_cast<int64_t>(s.row0 + row / p.G) * p.Hq + w.h * p.G + row % p.G;
                        const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;
                        uint4 y;
                        y.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
                        y.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
                        y.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
                        y.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
                        *reinterpret_cast<uint4 *>(p.O + at * kD + ch) = y;
                        if (p.lse && ch == 0) p.lse[at] = Mu * 0.6931471805599453f + logf(L);
                    }
                } else {
                    // a share of it: slot 0 where the CTA's share begins in this tile, else slot 1
                    float *part = p.part + (static_cast<int64_t>(blockIdx.x) * 2 + (w.left == u1 - u0 ? 0 : 1)) * kPartFloats;
                    float4 *at = reinterpret_cast<float4 *>(part + r * kD + ch);
                    at[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    at[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
                    if (ch == 0) {
                        part[kRows * kD + r] = M;
                        part[kRows * kD + kRows + r] = L;
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
__global__ void __launch_bounds__(256) combine_kernel(const AttnParams p, int ctas) {
    const int64_t all = count_units(p), share = share_of(all, ctas);
    const int64_t u0 = share * blockIdx.x, u1 = u0 + share;
    if (u1 >= all) return;                   // nothing behind this share
    int b;
    int64_t local;
    find_unit(p, u1 - 1, b, local);
    Walk w;
    w.begin(p, b, local, 1);
    if (w.page + 1 == w.x.pages) return;     // its tile ends with the share
    const int64_t begin = u1 - 1 - w.page, end = begin + w.x.pages;
    if (begin < u0) return;                  // it began in an earlier share
    const int r = threadIdx.x >> 4, ch = (threadIdx.x & 15) * 8, row = w.tile * kRows + r;
    const Seq s = w.x.s;
    if (row >= s.n * p.G) return;
    const int last = static_cast<int>((end - 1) / share);
    const float kNegInf = __int_as_float(0xff800000);
    auto part_of = [&](int c) {
        return p.part + (static_cast<int64_t>(c) * 2 + (c == static_cast<int>(blockIdx.x) && begin > u0 ? 1 : 0)) * kPartFloats;
    };
    float M = kNegInf;
    for (int c = blockIdx.x; c <= last; ++c) M = fmaxf(M, part_of(c)[kRows * kD + r]);
    const float Mu = M == kNegInf ? 0.0f : M;
    float L = 0.0f, acc[8] = {};
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
    const int64_t at = static_cast<int64_t>(s.row0 + row / p.G) * p.Hq + w.h * p.G + row % p.G;
    const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;
    uint4 y;
    y.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    y.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    y.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
    y.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
    *reinterpret_cast<uint4 *>(p.O + at * kD + ch) = y;
    if (p.lse && ch == 0) p.lse[at] = Mu * 0.6931471805599453f + logf(L);
}

// CTAs of the decode kernel: one per SM, fewer where there cannot be work for all.
int decode_ctas(int T, int Hq, int H, int B, int cols) {
    const int64_t G = Hq / H;
    const int64_t tiles = static_cast<int64_t>(T) * G / kRows + (B < T ? B : T);   // of one head, at most
    const int64_t units = tiles * H * (cols > 0 ? cols : 1);
    const int64_t most = (units + kSmallest - 1) / kSmallest;
    return static_cast<int>(most < 152 ? (most < 1 ? 1 : most) : 152);
}

// More than one tile of 16 rows a sequence and KV head on average: the tensor
// core kernel's tiles of 128 rows.
bool many_rows(int T, int Hq, int H, int B) { return static_cast<int64_t>(T) * (Hq / H) > static_cast<int64_t>(kRows) * B; }

}  // namespace

size_t cache_attention_workspace(int T, int Hq, int H, int B, int cols) {
    if (many_rows(T, Hq, H, B)) return cache_chunk_workspace(T, Hq, H, B, cols);
    return static_cast<size_t>(decode_ctas(T, Hq, H, B, cols)) * 2 * kPartFloats * sizeof(float);
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
    const int ctas = decode_ctas(a.T, a.Hq, a.c.H, a.c.B, a.c.cols);
    cudaError_t e = cudaFuncSetAttribute(decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    decode_kernel<<<ctas, kThreads, kSmem, st>>>(mk, mv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    combine_kernel<<<ctas, 256, 0, st>>>(p, ctas);
    return cudaGetLastError();
}

}  // namespace vca
