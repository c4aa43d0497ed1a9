// vca_cache_chunk.cu -- attention over the 8-bit cache for many query rows (a
// chunk of frames, a prompt), bound by the tensor cores: 4 rows keys d flops.
// The mathematics is vca_cache_attention.cu's.
//
// One CTA takes 128 query rows of a (sequence, KV head) -- rows i G + g: the G
// query heads that share the KV head are rows of one tile, so its codes are
// read once for all of them -- and a run of the pages they see: all of them, or
// an even part where there are too few tiles to fill the GPU (then a second
// kernel joins the parts).  Warps:
//   0       TMA producer: K and V tiles into rings of three, each page's scales
//           into a ring of slots
//   1, 2    MMA issuers, one thread each, QK and PV: issuing an MMA costs more than
//           the tensor core takes for it.  QK(b+2) waits for PV(b), which reads
//           P(b), lying over S(b) in TMEM; PV(b+1) fills that wait
//   4-7     V codes -> fp16 in shared memory, a page ahead of PV (two buffers)
//   8-15    softmax, two threads per row, 64 scores of every page each, which stay in
//           registers from the maximum to the probabilities; warps w and w + 4
//           share a TMEM lane quarter and tell each other their half's maximum.
//           The reference maximum moves only when a page's exceeds it by 8 (then O
//           is rescaled in TMEM)
// QK: E4M3 codes of K straight from TMA.  A bf16 query element has 8 significant
// bits and an E4M3 code 4, so q = hi + lo: per 32 channels a power of two puts
// the largest element in [2^7, 2^8), hi = E4M3(q), lo = E4M3(32 (q - hi)), and
// the block-scaled MMA (kind::mxf8f6f4, one power-of-two factor per 32 channels)
// brings the factors back: exact for elements above 2^-15 of the largest of
// their 32, off by less than 2^-23 of it below.  Two FP8 products cost what one
// 16-bit product does, and K needs no conversion.
// PV: P as fp16 (TMEM) times V as fp16: exact codes times a power of two, the
// page's scale relative to a reference scale that moves, with O, only when a
// page's lies outside [2^-15, 2^7] of it.
// Every wait is bounded, as in vca_attention.cu.
#include "vca_attention_common.cuh"
#include "vca_cache.cuh"

namespace vca {

namespace {

using namespace attn;
using namespace cache;

constexpr int kRows = 128;
constexpr int kKStages = 3, kVStages = 3, kWStages = 2, kSlots = 16;
constexpr int kConvWarps = 4, kConvWarp0 = 4, kSoftWarp0 = 8;
constexpr int kThreads = 32 * (kSoftWarp0 + kSoftmaxWarps);
constexpr uint32_t kTile = kBlk * kD;            // E4M3 tile
constexpr uint32_t kWTile = 2 * kTile;           // fp16 tile, two panels of 64 channels
constexpr uint32_t kPanel = kTile;

constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemQ = 384, kTmemSFA = 448, kTmemSFB = 456, kTmemCols = 512;

constexpr uint32_t kOffK = 0;
constexpr uint32_t kOffV = kOffK + kKStages * kTile;
constexpr uint32_t kOffW = kOffV + kVStages * kTile;
constexpr uint32_t kOffSlot = kOffW + kWStages * kWTile;         // float4 [kSlots]: sk, V factor, O factor, reference scale
constexpr uint32_t kOffMX = kOffSlot + kSlots * 16;              // fp32 [2][2][128] the halves' maxima, by turns
constexpr uint32_t kOffL = kOffMX + 4 * kRows * 4;               // fp32 [2][128] the halves' l
constexpr uint32_t kOffF = kOffL + 2 * kRows * 4;                // fp32 [128] the rows' factors
constexpr uint32_t kOffBar = kOffF + kRows * 4;
constexpr uint32_t kBarPair = 2;                                 // + quarter: the two warps of a row's halves
constexpr int kNumBars = 1 + 2 * kKStages + 2 * kVStages + 2 * kWStages + 2 + 2 + 2 + 2;
constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
constexpr uint32_t kSmem = kOffMisc + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

constexpr int kPartFloats = kRows * kD + 2 * kRows;   // O, m, l of a part
constexpr int kSmallest = 4;                          // pages of a part at least

struct ChunkParams {
    AttnParams a;
    int split;         // 0: a CTA takes all pages of a tile; otherwise how many CTAs the pages should keep busy
};

// ---------------------------------------------------------------------------
// Tiles and their parts
// ---------------------------------------------------------------------------
__device__ __forceinline__ int tiles_of(const AttnParams &p, const Seq &s) {
    return static_cast<int>((static_cast<int64_t>(s.n) * p.G + kRows - 1) / kRows);
}
// Pages that the rows of a tile see; a tile that sees nothing has one, so that its rows are written.
__device__ __forceinline__ int pages_of(const AttnParams &p, const Seq &s, int tile) {
    const int last = min(static_cast<int64_t>(s.n) * p.G, (static_cast<int64_t>(tile) + 1) * kRows) - 1;
    return max(1, (min(seen_by_row(p, s, last), s.len) + kBlk - 1) / kBlk);
}
__device__ __forceinline__ int parts_of(int pages, int share) { return share > 0 ? (pages + share - 1) / share : 1; }

__device__ __forceinline__ int warp_scan(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// Pages of a part: an even share of all the tiles' pages of all heads (a warp's work).
__device__ int share_of(const ChunkParams &cp) {
    if (cp.split == 0) return 0;
    const AttnParams &p = cp.a;
    int64_t all = 0;
    for (int b = threadIdx.x & 31; b < p.c.B; b += 32) {
        const Seq s = load_seq(p.c, p.start, p.T, b);
        const int tiles = tiles_of(p, s);
        for (int t = 0; t < tiles; ++t) all += pages_of(p, s, t);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    return max(kSmallest, static_cast<int>((all * p.c.H + cp.split - 1) / cp.split));
}

// A tile, and one of its parts: pages [page0, page0 + pages).
struct Item {
    int b, tile, part, parts, page0, pages, slot;   // slot: the part's place among all parts of its head
    Seq s;
};

// The index-th part of a head (by_tile: the index-th tile, its part 0); false behind the last one.
__device__ bool find_item(const ChunkParams &cp, int share, int index, bool by_tile, Item &it) {
    const AttnParams &p = cp.a;
    const int lane = threadIdx.x & 31;
    int before = 0, slots = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        Seq mine{0, 0, 0, false};
        int cnt = 0, parts = 0;
        if (b0 + lane < p.c.B) {
            mine = load_seq(p.c, p.start, p.T, b0 + lane);
            const int tiles = tiles_of(p, mine);
            if (share == 0) {
                parts = tiles;
            } else {
                for (int t = 0; t < tiles; ++t) parts += parts_of(pages_of(p, mine, t), share);
            }
            cnt = by_tile ? tiles : parts;
        }
        const int incl = warp_scan(cnt) + before;
        const int pincl = warp_scan(parts) + slots;
        const uint32_t hit = __ballot_sync(0xffffffffu, index < incl);
        if (hit) {
            const int l = __ffs(hit) - 1;
            it.b = b0 + l;
            int rest = index - __shfl_sync(0xffffffffu, incl - cnt, l);
            it.slot = __shfl_sync(0xffffffffu, pincl - parts, l);
            it.s = load_seq(p.c, p.start, p.T, it.b);
            for (int t = 0;; ++t) {
                int q;
                if (share == 0 && !by_tile) {
                    t = rest;      // one part each: straight to the tile
                    it.slot += rest;
                    rest = 0;
                }
                it.tile = t;
                it.pages = pages_of(p, it.s, t);
                q = it.parts = parts_of(it.pages, share);
                if (by_tile ? rest == 0 : rest < q) break;
                rest -= by_tile ? 1 : q;
                it.slot += q;
            }
            it.part = by_tile ? 0 : rest;
            it.slot += it.part;
            const int all = it.pages;
            it.page0 = static_cast<int>(static_cast<int64_t>(all) * it.part / it.parts);
            it.pages = static_cast<int>(static_cast<int64_t>(all) * (it.part + 1) / it.parts) - it.page0;
            return true;
        }
        before = __shfl_sync(0xffffffffu, incl, 31);
        slots = __shfl_sync(0xffffffffu, pincl, 31);
    }
    return false;
}

// ---------------------------------------------------------------------------
// The products
// ---------------------------------------------------------------------------
// Instruction descriptor of the block-scaled FP8 MMA: A and B E4M3, UE8M0 scale
// factors, one per 32 elements of K; A's factor is byte `sf` of its word, B's byte 0.
__host__ __device__ constexpr uint32_t make_idesc_mxf8(int M, int N, uint32_t sf) {
    return (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24) | (sf << 29);
}
__device__ __forceinline__ void mma_mxf8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], [%1], %2, %3, [%4], [%5], p;\n\t}\n"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// One query row split as hi + lo into TMEM with its factors; returns 2^E, the
// row's largest group factor, which the scores are multiplied by.
__device__ __forceinline__ float store_query(uint32_t tl, int quarter, const uint16_t *row) {
    uint32_t sfh = 0, sfl = 0;
    int e[4], E = -100;
    uint4 v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = row ? reinterpret_cast<const uint4 *>(row)[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, amax_bf16x8(v[4 * g + i]));
        e[g] = max(static_cast<int>(m >> 23) - 127 - 7, -100);    // q 2^-e in [2^7, 2^8)
        E = max(E, e[g]);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e[g]) << 23);
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {v[4 * g + i].x, v[4 * g + i].y, v[4 * g + i].z, v[4 * g + i].w};
            float x[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[2 * k] = __uint_as_float(w[k] << 16) * down;
                x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u) * down;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float d[4];
                hi[2 * i + k] = e4m3x4(scaled_or_nan(x[4 * k], 1.0f), scaled_or_nan(x[4 * k + 1], 1.0f),
                                       scaled_or_nan(x[4 * k + 2], 1.0f), scaled_or_nan(x[4 * k + 3], 1.0f));
                e4m3x4_decode(hi[2 * i + k], d);
                lo[2 * i + k] = e4m3x4(32.0f * (x[4 * k] - d[0]), 32.0f * (x[4 * k + 1] - d[1]),
                                       32.0f * (x[4 * k + 2] - d[2]), 32.0f * (x[4 * k + 3] - d[3]));
            }
        }
        VCA_TMEM_ST8(tl + kTmemQ + 8 * g, hi);
        VCA_TMEM_ST8(tl + kTmemQ + 32 + 8 * g, lo);
        sfh |= static_cast<uint32_t>(max(127 + e[g] - E, 6)) << (8 * g);
        sfl |= static_cast<uint32_t>(max(127 + e[g] - E, 6) - 5) << (8 * g);
    }
    // row m's factor words lie in lane m, column m / 32; B's factors are 1 everywhere
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(tl + kTmemSFA + quarter), "r"(sfh) : "memory");
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(tl + kTmemSFA + 4 + quarter), "r"(sfl) : "memory");
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%1,%1,%1};" ::"r"(tl + kTmemSFB), "r"(0x7f7f7f7fu) : "memory");
    return __uint_as_float(static_cast<uint32_t>(127 + E) << 23);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a softmax thread needs for one page's probabilities.
struct PageScore {
    float c, bias;       // no cap: p = 2^(S c + bias); cap: p = 2^(r t + bias), r = 1 / (1 + 2^(S c))
    float t;             // -2 cap log2(e)
    int lim;             // how many of the thread's 64 columns the row sees
    bool edge;           // some row of the warp does not see all
};

// 32 raw scores -> 16 words of fp16 pairs; the unrounded probabilities add to l2.
template <bool kCap>
__device__ __forceinline__ void probabilities(const uint32_t (&X)[32], const PageScore &s, int col0, uint64_t &l2,
                                              uint32_t (&W)[16]) {
    const uint64_t c2 = pk2(__float_as_uint(s.c), __float_as_uint(s.c));
    const uint64_t b2 = pk2(__float_as_uint(s.bias), __float_as_uint(s.bias));
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float a, b;
        if constexpr (kCap) {
            upk2(mul2(pk2(X[2 * k], X[2 * k + 1]), c2), a, b);
            a = rcp_approx(1.0f + ex2_approx(a));
            b = rcp_approx(1.0f + ex2_approx(b));
            const uint64_t t2 = pk2(__float_as_uint(s.t), __float_as_uint(s.t));
            upk2(fma2(pk2(__float_as_uint(a), __float_as_uint(b)), t2, b2), a, b);
        } else {
            upk2(fma2(pk2(X[2 * k], X[2 * k + 1]), c2, b2), a, b);
        }
        a = ex2_approx(a);
        b = ex2_approx(b);
        if constexpr (kCap) {
            if (s.edge) {
                if (col0 + 2 * k >= s.lim) a = 0.0f;
                if (col0 + 2 * k + 1 >= s.lim) b = 0.0f;
            }
        }
        l2 = add2(l2, pk2(__float_as_uint(a), __float_as_uint(b)));
        W[k] = pack_half2(a, b);
    }
}

// A warp's 32 rows of V codes as fp16 times a power of two, rows from `live` on
// as zeros.  A lane takes a 16-byte chunk of codes to two 16-byte chunks of fp16,
// lanes 0-3 of eight the lower 64 channels of one row, lanes 4-7 the upper ones of
// its neighbour: by the swizzle a quarter warp's accesses then fall into
// different banks.
template <bool kPlain>
__device__ __forceinline__ void convert_rows(const unsigned char *src, unsigned char *dst, int part, float factor, int live) {
    const int lane = threadIdx.x & 31, c = lane & 7, up = c >> 2, oc = 2 * (c & 3);
    const __half2 f = __float2half2_rn(factor);
    dst += up * kPanel;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = part * 32 + 8 * (i >> 1) + 2 * (lane >> 3) + ((i & 1) ? 1 - up : up);
        const uint4 v = *reinterpret_cast<const uint4 *>(src + sw128_offset(r, c));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
                "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(o[2 * k]), "=r"(o[2 * k + 1]) : "r"(w[k]));
            if constexpr (!kPlain) {
                const __half2 x = __hmul2(*reinterpret_cast<__half2 *>(&o[2 * k]), f);
                const __half2 y = __hmul2(*reinterpret_cast<__half2 *>(&o[2 * k + 1]), f);
                o[2 * k] = r < live ? *reinterpret_cast<const uint32_t *>(&x) : 0u;
                o[2 * k + 1] = r < live ? *reinterpret_cast<const uint32_t *>(&y) : 0u;
            }
        }
        *reinterpret_cast<uint4 *>(dst + sw128_offset(r, oc)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(dst + sw128_offset(r, oc + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// Scores of keys that the row does not see, columns col0 + lim and up, become
// -inf; returns the largest of the others.
__device__ __forceinline__ float mask_scores(uint32_t (&X)[32], int col0, int lim) {
    float m = __int_as_float(0xff800000);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        if (col0 + e >= lim) X[e] = 0xff800000u;
        m = fmaxf(m, __uint_as_float(X[e]));
    }
    return m;
}

template <bool kCap>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const ChunkParams cp) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + kOffBar);
    uint64_t *k_full = q_full + 1, *k_empty = k_full + kKStages;
    uint64_t *v_full = k_empty + kKStages, *v_empty = v_full + kVStages;
    uint64_t *w_full = v_empty + kVStages, *w_empty = w_full + kWStages;
    uint64_t *s_full = w_empty + kWStages, *p_full = s_full + 2, *pv_done = p_full + 2, *drain = pv_done + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    int *abort_flag = reinterpret_cast<int *>(smem + kOffMisc + 4);
    float4 *sSlot = reinterpret_cast<float4 *>(smem + kOffSlot);
    float *sMX = reinterpret_cast<float *>(smem + kOffMX);
    float *sL = reinterpret_cast<float *>(smem + kOffL);
    float *sF = reinterpret_cast<float *>(smem + kOffF);

    const AttnParams &p = cp.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y;
    if (blockIdx.x == 0 && h == 0 && warp == 0)
        for (int b = lane; b < p.c.B; b += 32)
            if (load_seq(p.c, p.start, p.T, b).bad) report(p.dev_status, kErrInvalid);
    Item it;
    // the last tiles of a causal sequence see the most pages: they go first
    const int share = share_of(cp);
    if (!find_item(cp, share, static_cast<int>(gridDim.x - 1 - blockIdx.x), false, it)) return;
    const int nb = it.pages, r0 = it.tile * kRows, R = it.s.n * p.G;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 4);
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(k_full + s, 1);
            mbar_init(k_empty + s, 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(v_full + s, 1);
            mbar_init(v_empty + s, kConvWarps);
        }
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(w_full + s, kConvWarps);
            mbar_init(w_empty + s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 2);      // the MMA's commit and the issuer itself
            mbar_init(p_full + i, kSoftmaxWarps);
            mbar_init(pv_done + i, 1);
        }
        mbar_init(drain, 1);
        mbar_init(drain + 1, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        bool ok = true;
        int kk = 0, vk = 0;      // copies issued
        int ref = -1;            // the reference scale's biased exponent
        for (int j0 = 0; ok && j0 < nb; j0 += 32) {
            int page = -1;
            float sk = 0.0f, sv = 0.0f;
            if (j0 + lane < nb && it.s.len > 0) {
                page = load_page(p.c, it.b, it.page0 + j0 + lane, p.dev_status);
                if (page >= 0) {
                    sk = p.c.sk[static_cast<int64_t>(page) * p.c.H + h];
                    sv = p.c.sv[static_cast<int64_t>(page) * p.c.H + h];
                }
            }
            for (int i = 0; ok && i < 32 && j0 + i < nb; ++i) {
                const int j = j0 + i, st = j % kKStages, vt = j % kVStages;
                const int pg = __shfl_sync(0xffffffffu, page, i);
                const float ks = __shfl_sync(0xffffffffu, sk, i), vs = __shfl_sync(0xffffffffu, sv, i);
                float4 slot = make_float4(-1.0f, 0.0f, 1.0f, 1.0f);      // no page
                if (pg >= 0) {
                    const int e = static_cast<int>((__float_as_uint(vs) >> 23) & 255u);
                    int shift = 0;
                    if (ref < 0) ref = e;
                    if (e - ref > 7) {
                        shift = ref - e;
                        ref = e;
                    } else if (e - ref < -15) {
                        const int to = max(e, ref - 80);     // O, at most 2^41 references, stays finite
                        shift = ref - to;
                        ref = to;
                    }
                    slot.x = ks;
                    slot.y = __uint_as_float(static_cast<uint32_t>(127 + max(e - ref, -126)) << 23);
                    slot.z = __uint_as_float(static_cast<uint32_t>(127 + max(shift, -126)) << 23);
                }
                slot.w = __uint_as_float(static_cast<uint32_t>(max(ref, 0)) << 23);
                if (j >= kKStages) ok = mbar_wait(k_empty + st, (j / kKStages - 1) & 1, abort_flag, p.limit_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const int y = (pg * p.c.H + h) * kBlk;
                if (lane == 0) {
                    sSlot[j % kSlots] = slot;
                    if (pg >= 0) {
                        mbar_expect_tx(k_full + st, kTile);
                        tma_load_2d(smem + kOffK + st * kTile, &tmK, k_full + st, 0, y);
                    } else {
                        mbar_arrive(k_full + st);
                    }
                }
                kk = j + 1;
                if (j >= kVStages) ok = mbar_wait(v_empty + vt, (j / kVStages - 1) & 1, abort_flag, p.limit_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    if (pg >= 0) {
                        mbar_expect_tx(v_full + vt, kTile);
                        tma_load_2d(smem + kOffV + vt * kTile, &tmV, v_full + vt, 0, y);
                    } else {
                        mbar_arrive(v_full + vt);
                    }
                }
                vk = j + 1;
            }
        }
        // every copy issued has landed before the CTA can exit
        if (lane == 0) {
            for (int j = max(0, kk - kKStages); j < kk; ++j) drain_wait(k_full + j % kKStages, (j / kKStages) & 1, p.limit_ns);
            for (int j = max(0, vk - kVStages); j < vk; ++j) drain_wait(v_full + j % kVStages, (j / kVStages) & 1, p.limit_ns);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ QK issuer
        if (lane == 0) {
            const uint32_t tq = tmem + kTmemQ, sfa = tmem + kTmemSFA, sfb = tmem + kTmemSFB;
            const uint64_t dk0 = sdesc_k_sw128(smem_u32(smem) + kOffK);
            int st = 0;
            uint32_t kphase = 0, pphase = 0;
            bool ok = mbar_wait(q_full, 0, abort_flag, p.limit_ns);
            for (int b = 0; ok && b < nb; ++b) {
                const int sb = b & 1;
                ok = mbar_wait_spin(k_full + st, kphase, abort_flag, p.limit_ns);
                if (ok && b >= 2) ok = mbar_wait_spin(pv_done + sb, pphase, abort_flag, p.limit_ns);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dk = dk0 + static_cast<uint32_t>(st) * (kTile >> 4);
                const uint32_t d = tmem + kTmemS + 128 * sb;
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_mxf8_ts(d, tq + 8 * i, dk + 2 * i, make_idesc_mxf8(128, 128, i), sfa, sfb, i > 0);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_mxf8_ts(d, tq + 32 + 8 * i, dk + 2 * i, make_idesc_mxf8(128, 128, i), sfa + 4, sfb, 1u);
                tc_commit(s_full + sb);
                mbar_arrive(s_full + sb);
                tc_commit(k_empty + st);
                if (++st == kKStages) {
                    st = 0;
                    kphase ^= 1;
                }
                if (b >= 2) pphase ^= sb;
            }
            tc_commit(drain);
            drain_wait(drain, 0, p.limit_ns);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ PV issuer
        if (lane == 0) {
            constexpr uint32_t idesc = make_idesc(128, 128, 0, 0, 0, 1);
            const uint64_t dv0 = sdesc_mn_sw128(smem_u32(smem) + kOffW, kPanel);
            bool ok = true;
            for (int b = 0; b < nb; ++b) {
                const int wt = b % kWStages, sb = b & 1;
                ok = mbar_wait_spin(w_full + wt, (b / kWStages) & 1, abort_flag, p.limit_ns) &&
                     mbar_wait_spin(p_full + sb, (b >> 1) & 1, abort_flag, p.limit_ns);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dv = dv0 + static_cast<uint32_t>(wt) * (kWTile >> 4);
                const uint32_t a = tmem + kTmemS + 128 * sb;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mma_f16_ts(tmem + kTmemO, a + 8 * i, dv + (2048 >> 4) * i, idesc, (b > 0 || i > 0) ? 1u : 0u);
                tc_commit(pv_done + sb);
                tc_commit(w_empty + wt);
            }
            tc_commit(drain + 1);
            drain_wait(drain + 1, 0, p.limit_ns);
        }
    } else if (warp >= kConvWarp0 && warp < kConvWarp0 + kConvWarps) {
        // ------------------------------------------------------------ V codes -> fp16
        for (int j = 0; j < nb; ++j) {
            const int vt = j % kVStages, wt = j % kWStages;
            bool ok = mbar_wait(v_full + vt, (j / kVStages) & 1, abort_flag, p.limit_ns);
            if (ok && j >= kWStages) ok = mbar_wait(w_empty + wt, (j / kWStages - 1) & 1, abort_flag, p.limit_ns);
            if (!__all_sync(0xffffffffu, ok)) break;
            const float4 slot = sSlot[j % kSlots];
            const unsigned char *src = smem + kOffV + vt * kTile;
            unsigned char *dst = smem + kOffW + wt * kWTile;
            const int live = slot.x < 0.0f ? 0 : it.s.len - (it.page0 + j) * kBlk;    // rows behind the last token hold anything
            if (slot.y == 1.0f && live >= kBlk)
                convert_rows<true>(src, dst, warp - kConvWarp0, 1.0f, kBlk);
            else
                convert_rows<false>(src, dst, warp - kConvWarp0, slot.y, live);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(v_empty + vt);
                mbar_arrive(w_full + wt);
            }
        }
    } else if (warp >= kSoftWarp0) {
        // ------------------------------------------------------------ softmax
        const int quarter = warp & 3, half = (warp - kSoftWarp0) >> 2, row = quarter * 32 + lane;
        const uint32_t bar_pair = kBarPair + quarter;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const float kNegInf = __int_as_float(0xff800000);
        const int r = r0 + row;
        const bool real = r < R;
        float f;      // raw score -> log2 units (or the cap's inner argument), but for the page's scale
        if (half == 0) {
            f = store_query(tl, quarter, real ? query_row(p, it.s, h, r) : nullptr);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            sF[row] = f;
        }
        bar_sync(bar_pair, 64);
        if (half == 1) f = sF[row];
        f *= kCap ? p.cap_in : p.scale_log2;
        const int seen = (real ? min(seen_by_row(p, it.s, r), it.s.len) : it.s.len) - it.page0 * kBlk - 64 * half;
        PageScore s;
        s.t = -2.0f * p.cap_out;
        float m = kNegInf, l = 0.0f;
        bool ok = true;
        for (int b = 0; b < nb; ++b) {
            const int sb = b & 1;
            float *mx = sMX + sb * 2 * kRows;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(s_full + sb, (b >> 1) & 1, abort_flag, p.limit_ns));
            if (!ok) {
                // the other half learns of it where they meet
                mx[half * kRows + row] = __int_as_float(0x7fc00000);
                bar_sync(bar_pair, 64);
                break;
            }
            const uint32_t tS = tl + kTmemS + 128 * sb;
            uint32_t X0[32], X1[32];
            float bm = kNegInf;
            tc_fence_after();
            float m0, m1;
            VCA_TMEM_LDMAX32(tS + 64 * half, X0, m0);
            VCA_TMEM_LDMAX32(tS + 64 * half + 32, X1, m1);
            const float4 slot = sSlot[b % kSlots];
            s.lim = slot.x < 0.0f ? 0 : seen - b * kBlk;
            s.edge = __any_sync(0xffffffffu, s.lim < 64);
            s.c = fmaxf(__fmul_rn(f, slot.x), 0x1p-126f);      // above 0, so that -inf stays -inf
            tmem_ld_wait();
            if (s.edge) {
                m0 = mask_scores(X0, 0, s.lim);
                m1 = mask_scores(X1, 32, s.lim);
            }
            const float pm = fmaxf(m0, m1);
            if (pm != kNegInf)
                bm = kCap ? fmaf(rcp_approx(1.0f + ex2_approx(pm * s.c)), s.t, p.cap_out) : __fmul_rn(pm, s.c);
            // the row's maximum over both halves; NaN: the other half gave up.  Both
            // halves have read their scores when they meet, so P may be written over
            // them.  Buffers by turns: the next page's barrier separates this read
            // from the write after it
            mx[half * kRows + row] = bm;
            bar_sync(bar_pair, 64);
            const float other = mx[(half ^ 1) * kRows + row];
            if (__any_sync(0xffffffffu, other != other)) {
                ok = false;
                break;
            }
            const float top = fmaxf(bm, other);
            const bool moved = top > __fadd_rn(m, kLazyTau);
            const float m_in = m;
            if (moved) {
                l = __fmul_rn(l, ex2_approx(__fsub_rn(m, top)));
                m = top;
            }
            const float mu = m == kNegInf ? 0.0f : m;      // a row that sees nothing yet
            s.bias = kCap ? p.cap_out - mu : -mu;
            uint64_t l2 = pk2(__float_as_uint(l), 0u);
            uint32_t W[16];
            probabilities<kCap>(X0, s, 0, l2, W);
            VCA_TMEM_ST16(tS + 32 * half, W);
            probabilities<kCap>(X1, s, 32, l2, W);
            VCA_TMEM_ST16(tS + 32 * half + 16, W);
            {
                float a, c;
                upk2(l2, a, c);
                l = __fadd_rn(a, c);
            }
            // this half's channels of O after PV(b - 1) to the new reference maximum and scale
            const float alpha = b > 0 ? (moved ? ex2_approx(__fsub_rn(m_in, m)) : 1.0f) * slot.z : 1.0f;
            if (__any_sync(0xffffffffu, alpha != 1.0f)) {
                ok = __all_sync(0xffffffffu, mbar_wait(pv_done + (sb ^ 1), ((b - 1) >> 1) & 1, abort_flag, p.limit_ns));
                if (ok) {
                    tc_fence_after();
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        uint32_t o[32];
                        VCA_TMEM_LD32(tl + kTmemO + 64 * half + 32 * i, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), alpha));
                        VCA_TMEM_ST32(tl + kTmemO + 64 * half + 32 * i, o);
                    }
                }
            }
            // a thread that gave up here tells the other half at the next page
            if (ok) {
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + sb);
            }
        }
        // ------------------------------------------------------------ epilogue
        // PV(nb - 1) complete (PV(nb - 3) was when S(nb - 1) came)
        if (ok)
            ok = __all_sync(0xffffffffu, mbar_wait(pv_done + ((nb - 1) & 1), ((nb - 1) >> 1) & 1, abort_flag, p.limit_ns));
        sL[half * kRows + row] = l;
        ok = bar_and(ok, kBarSoftmax, 32 * kSoftmaxWarps);
        if (ok) {
            tc_fence_after();
            const float M = m, Mu = M == kNegInf ? 0.0f : M, L = __fadd_rn(sL[row], sL[kRows + row]);
            const float ref = sSlot[(nb - 1) % kSlots].w;
            if (it.parts == 1) {
                const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;
                uint16_t *orow = real ? p.O + out_row(p, it.s, h, r) * kD + 64 * half : nullptr;
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    uint32_t o[32], w[16];
                    VCA_TMEM_LD32(tl + kTmemO + 64 * half + 32 * i, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv * ref, __uint_as_float(o[2 * e + 1]) * inv * ref);
                    if (real) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<uint4 *>(orow + 32 * i)[e] =
                                make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                    }
                }
                if (real && half == 0 && p.lse) p.lse[out_row(p, it.s, h, r)] = Mu * 0.6931471805599453f + logf(L);
            } else {
                float *part = p.part + (static_cast<int64_t>(h) * gridDim.x + it.slot) * kPartFloats;
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    uint32_t o[32];
                    VCA_TMEM_LD32(tl + kTmemO + 64 * half + 32 * i, o);
                    tmem_ld_wait();
                    if (real) {
                        float4 *at = reinterpret_cast<float4 *>(part + row * kD + 64 * half + 32 * i);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            at[e] = make_float4(__uint_as_float(o[4 * e]) * ref, __uint_as_float(o[4 * e + 1]) * ref,
                                                __uint_as_float(o[4 * e + 2]) * ref, __uint_as_float(o[4 * e + 3]) * ref);
                    }
                }
                if (half == 0) {
                    part[kRows * kD + row] = M;
                    part[kRows * kD + kRows + row] = L;
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (threadIdx.x == 0 && *reinterpret_cast<volatile int *>(abort_flag)) report(p.dev_status, kErrTimeout);
}

// Joins the parts of a tile: one CTA per (tile, head, 16 rows).
__global__ void __launch_bounds__(256) join_kernel(const ChunkParams cp, int slots) {
    const AttnParams &p = cp.a;
    Item it;
    if (!find_item(cp, share_of(cp), blockIdx.x, true, it) || it.parts == 1) return;
    const int h = blockIdx.y, row = 16 * blockIdx.z + (threadIdx.x >> 4), ch = (threadIdx.x & 15) * 8, r = it.tile * kRows + row;
    if (r >= it.s.n * p.G) return;
    const float *part = p.part + (static_cast<int64_t>(h) * slots + it.slot) * kPartFloats;
    float M = __int_as_float(0xff800000);
    for (int c = 0; c < it.parts; ++c) M = fmaxf(M, part[c * static_cast<int64_t>(kPartFloats) + kRows * kD + row]);
    const float Mu = M == __int_as_float(0xff800000) ? 0.0f : M;
    float L = 0.0f, acc[8] = {};
    for (int c = 0; c < it.parts; ++c) {
        const float *q = part + c * static_cast<int64_t>(kPartFloats);
        const float k = ex2_approx(q[kRows * kD + row] - Mu);
        L = fmaf(q[kRows * kD + kRows + row], k, L);
        const float4 *at = reinterpret_cast<const float4 *>(q + row * kD + ch);
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
    const int64_t at = out_row(p, it.s, h, r);
    const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;
    uint4 y;
    y.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    y.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    y.z = pack_bf16x2(acc[4] * inv, acc[5] * inv);
    y.w = pack_bf16x2(acc[6] * inv, acc[7] * inv);
    *reinterpret_cast<uint4 *>(p.O + at * kD + ch) = y;
    if (p.lse && ch == 0) p.lse[at] = Mu * 0.6931471805599453f + logf(L);
}

// Tiles of one head at most, and whether their pages are cut into parts: with
// two tiles for every SM the last wave costs little.
struct Plan {
    int64_t tiles;
    int split, grid;
};
Plan plan_of(int T, int Hq, int H, int B, int cols) {
    Plan q;
    q.tiles = static_cast<int64_t>(T) * (Hq / H) / kRows + (B < T ? B : T);
    q.split = q.tiles * H < 2 * 152 && cols > kSmallest ? 152 : 0;
    q.grid = static_cast<int>(q.tiles + (q.split ? q.split / H + 1 : 0));
    return q;
}

}  // namespace

size_t cache_chunk_workspace(int T, int Hq, int H, int B, int cols) {
    const Plan q = plan_of(T, Hq, H, B, cols);
    return q.split ? static_cast<size_t>(q.grid) * H * kPartFloats * sizeof(float) : 0;
}

cudaError_t launch_cache_chunk(const CacheAttnArgs &a, cudaStream_t st) {
    CUtensorMap mk, mv;
    const uint64_t rows = static_cast<uint64_t>(a.c.pages) * a.c.H * kBlk;
    if (!make_tile_map(&mk, a.c.k8, rows) || !make_tile_map(&mv, a.c.v8, rows)) return cudaErrorInvalidValue;
    const Plan q = plan_of(a.T, a.Hq, a.c.H, a.c.B, a.c.cols);
    ChunkParams cp;
    cp.a = attn_params(a.c, a.q, a.start, a.T, a.Hq, a.causal, a.scale, a.softcap, a.dev_status, a.wait_limit_ns);
    cp.a.O = a.O;
    cp.a.lse = a.lse;
    cp.a.part = static_cast<float *>(a.ws);
    cp.split = q.split;
    const auto kernel = a.softcap > 0.0f ? chunk_kernel<true> : chunk_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    kernel<<<dim3(q.grid, a.c.H), kThreads, kSmem, st>>>(mk, mv, cp);
    e = cudaGetLastError();
    if (e != cudaSuccess || !q.split) return e;
    join_kernel<<<dim3(static_cast<unsigned>(q.tiles), a.c.H, kRows / 16), 256, 0, st>>>(cp, q.grid);
    return cudaGetLastError();
}

}  // namespace vca
