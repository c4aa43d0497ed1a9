// vca_cache_chunk.cu -- attention over the 8-bit cache for many query rows (a
// chunk of frames, a prompt), bound by the tensor cores: 4 rows keys d flops.
// The mathematics is vca_cache_attention.cu's.
//
// One CTA takes a tile of 128 query rows of a (sequence, KV head) -- rows i G + g:
// the G query heads that share the KV head are rows of one tile, so its codes are
// read once for all of them -- and a run of the pages they see: all of them, or
// an even part where there are too few tiles to fill the GPU (then a last
// kernel joins the parts).  A first kernel lays out every tile's queries as the
// product wants them, so that a CTA only copies them, and lists the CTAs' work.
// Warps:
//   0       TMA producer: K and V tiles into rings of three, each page's scales
//           into a ring of slots
//   1, 2    MMA issuers, one thread each, QK and PV: issuing an MMA costs more than
//           the tensor core takes for it.  QK(b+2) waits for PV(b), which reads
//           P(b), lying over S(b) in TMEM; PV(b+1) fills that wait
//   4-7     the queries into TMEM, then V codes -> fp16 in shared memory, a page
//           ahead of PV (two buffers)
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
// their 32, off by less than 2^-22 of it below.  Two FP8 products cost what one
// 16-bit product does, and K needs no conversion (V's is 10 % of the time).
// Few rows (tiles of N = 32): the 128 rows of the product are four copies of the
// tile's, and each copy takes the probabilities of a quarter of every page's
// keys, the other keys' being zeros to it: its warps then have 16 scores a thread
// instead of 64, and none of them idles.  The copies have statistics and O of
// their own, which are put together at the end like parts of a tile.
// PV: P as fp16 (TMEM) times V as fp16: exact codes times a power of two, the
// page's scale relative to a reference scale that moves, with O, only when a
// page's lies outside [2^-15, 2^7] of it, and never further down than 2^-80 of the
// largest so far: values whose page's scale is below 2^-95 of that lose bits.
// Every wait is bounded, as in vca_attention.cu.
//
// 4,416 rows over 70,656 tokens, 8 heads: 979 us, 1,305 TFLOP/s (957 us in a loop of
// nothing else), the tensor pipe 56 % busy: 280 tiles on 152 SMs keep 8 % of them
// idle, and in a page's 1,650 cycles (1,056 in the pipe) QK(b + 2) waits for PV(b)
// and that for the softmax.
// Prompts of 2,900 rows behind short prefixes, causal, 32 heads over 8: 270 us, 850
// TFLOP/s: a tile has 17 pages on average and 7,500 cycles of its own.  A cap
// costs the softmax warps seven multiply-adds a score: 957 -> 1,823 us.
// Measured and not kept: P in columns of its own, with Q's lo in shared memory
// (1,030 us); one persistent CTA per SM with equal runs of pages (1,016; prompts
// 513); probabilities before the halves' maxima meet (1,236); one issuer (1,066
// against 988 at the time).  Few rows: 8 sequences of up to 16,383 tokens, 5 rows
// each, 40 heads over 8, capped: 62 us (92 in tiles of 128), 2.7 TB/s.
#include "vca_attention_common.cuh"
#include "vca_cache.cuh"

namespace vca {

namespace {

using namespace attn;
using namespace cache;

constexpr int kLanes = 128;                      // rows of an MMA
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
constexpr uint32_t kOffL = kOffMX + 4 * kLanes * 4;              // fp32 [2][128] the halves' l
constexpr uint32_t kOffBar = kOffL + 2 * kLanes * 4;
constexpr uint32_t kBarPair = 2;                                 // + quarter: the two warps of a row's halves
constexpr int kNumBars = 1 + 2 * kKStages + 2 * kVStages + 2 * kWStages + 2 + 2 + 2 + 2;
constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
constexpr uint32_t kSmem = kOffMisc + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

// Of N rows: O, m, l of a part
template <int N>
constexpr int kPartFloats = N * kD + 2 * N;
constexpr int kSmallest = 4;                          // pages of a part at least

// What one CTA does: pages [page0, page0 + pages) of a tile, as one of `parts`
// parts, `slot` its place among the parts of its head, `image` its tile's among
// the tiles.  pages = 0: nothing.
struct alignas(16) Item {
    int b, tile, page0, pages, parts, slot, image;
    Seq s;
};

struct ChunkParams {
    AttnParams a;
    Item *items;         // [items] of every head alike
    int *first;          // [tiles] a tile's first item, where tiles are cut
    uint8_t *images;     // [heads of a launch][tiles][kImage]
    int h0;              // the launch's first head
    int tiles, grid;     // tiles and items of a head at most
    int split;           // CTAs that parts of tiles should fill; 0: tiles are not cut
};

// A tile's queries: hi, then lo codes, each as eight 16-byte columns of N rows,
// then the words of their factors.
template <int N>
constexpr int kImage = 2 * N * kD + 2 * N * 4;

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
template <int N>
__device__ __forceinline__ int tiles_of(const AttnParams &p, const Seq &s) {
    return static_cast<int>((static_cast<int64_t>(s.n) * p.G + N - 1) / N);
}
// Pages that the rows of a tile see; a tile that sees nothing has one, so that its rows are written.
template <int N>
__device__ __forceinline__ int pages_of(const AttnParams &p, const Seq &s, int tile) {
    const int last = min(static_cast<int64_t>(s.n) * p.G, (static_cast<int64_t>(tile) + 1) * N) - 1;
    return max(1, (min(seen_by_row(p, s, last), s.len) + kBlk - 1) / kBlk);
}
__device__ __forceinline__ int warp_scan(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}
// The index-th tile of a head: its sequence and place there (a warp's work).
template <int N>
__device__ bool find_tile(const AttnParams &p, int index, int &b, int &tile, Seq &s) {
    int before = 0;
    bool more = true;
    for (int b0 = 0; more; b0 += 32) {
        Seq mine;
        more = load_seqs(p.c, p.start, p.T, b0, mine);
        const int t = tiles_of<N>(p, mine), incl = warp_scan(t) + before;
        const uint32_t hit = __ballot_sync(0xffffffffu, index < incl);
        if (hit) {
            const int l = __ffs(hit) - 1;
            b = b0 + l;
            s.row0 = __shfl_sync(0xffffffffu, mine.row0, l);
            s.n = __shfl_sync(0xffffffffu, mine.n, l);
            s.len = __shfl_sync(0xffffffffu, mine.len, l);
            tile = index - __shfl_sync(0xffffffffu, incl - t, l);
            return true;
        }
        before = __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}

// The list of work where tiles are cut (fewer than kCutMost of them in all
// heads): into parts of at most `share` pages, the least for which all heads'
// parts fit cp.split CTAs.
constexpr int kCutMost = 2 * 152, kPlanThreads = 512;
template <int N>
__device__ void plan_parts(const ChunkParams &cp) {
    __shared__ int sB[kCutMost], sTile[kCutMost], sParts[kCutMost], sSum[kPlanThreads / 32], sTiles;
    const AttnParams &p = cp.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == 0) {
        int before = 0;
        bool more = true;
        for (int b0 = 0; more; b0 += 32) {
            Seq s;
            more = load_seqs(p.c, p.start, p.T, b0, s);
            const int n = tiles_of<N>(p, s);
            const int incl = warp_scan(n) + before;
            for (int t = 0; t < n; ++t) {
                sB[incl - n + t] = b0 + lane;
                sTile[incl - n + t] = t;
            }
            before = __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) sTiles = before;
    }
    __syncthreads();
    const int tiles = sTiles;
    Seq s{0, 0, 0, false, false};
    int pages = 0;
    if (tid < tiles) {
        s = load_seq(p.c, p.start, p.T, sB[tid]);
        pages = pages_of<N>(p, s, sTile[tid]);
    }
    auto block_sum = [&](int v) {
        v = __reduce_add_sync(0xffffffffu, v);
        __syncthreads();
        if (lane == 0) sSum[warp] = v;
        __syncthreads();
        int sum = 0;
        for (int i = 0; i < kPlanThreads / 32; ++i) sum += sSum[i];
        return sum;
    };
    // with W pages in all, sum ceil(pages / share) lies between W / share and W / share + tiles
    const int slots = max(1, cp.split / p.c.H);
    const int64_t W = 256ll * block_sum(pages >> 8) + block_sum(pages & 255);      // 2^24 pages a tile at most
    int lo = max(kSmallest, static_cast<int>((W + slots - 1) / slots));
    int hi = slots > tiles ? max(lo, static_cast<int>((W + slots - tiles - 1) / (slots - tiles))) : max(lo, p.c.cols);
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (block_sum((pages + mid - 1) / mid) <= slots)
            hi = mid;
        else
            lo = mid + 1;
    }
    const int parts = (pages + lo - 1) / lo;
    if (tid < tiles) sParts[tid] = parts;
    __syncthreads();
    int slot = 0, total = 0;
    for (int t = 0; t < tiles; ++t) {
        if (t < tid) slot += sParts[t];
        total += sParts[t];
    }
    if (tid < tiles) {
        cp.first[tid] = slot;
        for (int i = 0; i < parts; ++i) {
            const int from = static_cast<int>(static_cast<int64_t>(pages) * i / parts);
            const int to = static_cast<int>(static_cast<int64_t>(pages) * (i + 1) / parts);
            cp.items[slot + i] = Item{sB[tid], sTile[tid], from, to - from, parts, slot + i, tid, s};
        }
    }
    for (int i = total + tid; i < cp.grid; i += kPlanThreads) cp.items[i].pages = 0;
    for (int i = tiles + tid; i < cp.tiles; i += kPlanThreads) cp.first[i] = -1;
}

// One CTA per (tile, head), 16 threads per row, 8 channels each (a warp then reads
// two whole rows and writes whole sectors of the image): a query row split as hi +
// lo, with factors that carry the whole power of two, so that a score is the
// product times softmax_scale alone; and the list of work.
template <int N>
__global__ void __launch_bounds__(kPlanThreads, 3) queries_kernel(const ChunkParams cp) {
    let_next_start();
    const AttnParams &p = cp.a;
    const int h = cp.h0 + blockIdx.y;
    if (blockIdx.x == 0 && h == 0)
        for (int b = threadIdx.x; b < p.c.B; b += kPlanThreads)
            if (load_seq(p.c, p.start, p.T, b).bad) report(p.dev_status, kErrInvalid);
    int b = 0, tile = 0;
    Seq s{0, 0, 0, false, false};
    const bool found = find_tile<N>(p, blockIdx.x, b, tile, s);
    if (cp.split == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
        const int i = static_cast<int>(blockIdx.x);
        cp.items[i] = Item{b, tile, 0, found ? pages_of<N>(p, s, tile) : 0, 1, i, i, s};
    }
    if (found) {
        uint8_t *img = cp.images + (static_cast<int64_t>(blockIdx.y) * cp.tiles + blockIdx.x) * kImage<N>;
        const int lane16 = threadIdx.x & 15, row0 = threadIdx.x >> 4;
        constexpr int kStep = kPlanThreads / 16;
        uint4 v[N / kStep];
#pragma unroll
        for (int i = 0; i < N / kStep; ++i) {
            const int r = tile * N + row0 + i * kStep;
            v[i] = make_uint4(0, 0, 0, 0);
            if (r < s.n * p.G) v[i] = reinterpret_cast<const uint4 *>(query_row(p, s, h, r))[lane16];
        }
#pragma unroll
        for (int i = 0; i < N / kStep; ++i) {
            const int row = row0 + i * kStep;
            bool odd = false;
            uint32_t m = amax_bf16x8(v[i], odd);      // of the four threads that share 32 channels
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const int e = max(static_cast<int>(m >> 23) - 127 - 7, -100);      // q 2^-e in [2^7, 2^8)
            const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            float x[8], d[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[2 * k] = __uint_as_float(w[k] << 16) * down;
                x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u) * down;
            }
            if (odd) {      // the conversion would turn an infinity into a number
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = scaled_or_nan(x[k], 1.0f);
            }
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                hi[k] = e4m3x4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                e4m3x4_decode(hi[k], d);
#pragma unroll
                for (int q = 0; q < 4; ++q) d[q] = 32.0f * (x[4 * k + q] - d[q]);
                lo[k] = e4m3x4(d[0], d[1], d[2], d[3]);
            }
            uint2 *to = reinterpret_cast<uint2 *>(img + ((lane16 >> 1) * N + row) * 16 + (lane16 & 1) * 8);
            to[0] = make_uint2(hi[0], hi[1]);
            to[N * kD / 8] = make_uint2(lo[0], lo[1]);
            if ((lane16 & 3) == 0) {
                uint8_t *sf = img + 2 * N * kD + 4 * row + (lane16 >> 2);
                sf[0] = static_cast<uint8_t>(127 + e);          // 27 .. 247
                sf[4 * N] = static_cast<uint8_t>(127 + e - 5);
            }
        }
    }
    if (cp.split && blockIdx.x == 0 && h == 0) plan_parts<N>(cp);
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

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Contiguous shared -> global copy of `bytes` (a multiple of 16, both addresses
// 16-byte aligned), and the wait for this thread's.
__device__ __forceinline__ void bulk_store(void *gmem, const void *smem, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(gmem)),
                 "r"(smem_u32(smem)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_store_wait() {
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

// What a softmax thread needs for one page's probabilities.
struct PageScore {
    float c, bias;       // no cap: p = 2^(S c + bias); cap: p = 2^(cap tanh_half(S c) + bias)
    float cap;           // cap log2(e)
    bool near;           // the polynomial of the cap's tanh will do for the warp
    int lim;             // how many of the thread's columns the row sees
    bool edge;           // some row of the warp does not see all
};

// kN raw scores -> words of fp16 pairs; the unrounded probabilities add to l2.
template <bool kCap, int kN>
__device__ __forceinline__ void probabilities(uint32_t (&X)[kN], const PageScore &s, int col0, uint64_t &l2,
                                              uint32_t (&W)[kN / 2]) {
    const uint64_t c2 = pk2(__float_as_uint(s.c), __float_as_uint(s.c));
    const uint64_t b2 = pk2(__float_as_uint(s.bias), __float_as_uint(s.bias));
    if constexpr (kCap) cap_scores(X, s.c, s.cap, s.near, [&](int) { return b2; });
#pragma unroll
    for (int k = 0; k < kN / 2; ++k) {
        float a = __uint_as_float(X[2 * k]), b = __uint_as_float(X[2 * k + 1]);
        if constexpr (!kCap) upk2(fma2(pk2(X[2 * k], X[2 * k + 1]), c2, b2), a, b);
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
// -inf (0 where a cap follows); returns the largest of the others.
template <bool kCap, int kN>
__device__ __forceinline__ float mask_scores(uint32_t (&X)[kN], int col0, int lim) {
    float m = __int_as_float(0xff800000);
#pragma unroll
    for (int e = 0; e < kN; ++e) {
        if (col0 + e < lim) m = fmaxf(m, __uint_as_float(X[e]));
        else X[e] = kCap ? 0u : 0xff800000u;
    }
    return m;
}

// kN raw scores and the largest of them, or with kTop the largest magnitude.
template <bool kTop, int kN>
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t (&X)[kN], float &m) {
    if constexpr (kN == 32 && kTop)
        VCA_TMEM_LDTOP32(taddr, X, m);
    else if constexpr (kN == 32)
        VCA_TMEM_LDMAX32(taddr, X, m);
    else if constexpr (kTop)
        VCA_TMEM_LDTOP16(taddr, X, m);
    else
        VCA_TMEM_LDMAX16(taddr, X, m);
}

template <int N, bool kCap>
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

    const AttnParams &p = cp.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = cp.h0 + blockIdx.y;
    let_next_start();
    wait_for_results();
    // the last tiles of a causal sequence see the most pages: they go first
    const Item it = cp.items[gridDim.x - 1 - blockIdx.x];
    if (it.pages == 0) return;
    const int nb = it.pages, r0 = it.tile * N, R = it.s.n * p.G;

    if (threadIdx.x == 0) {
        mbar_init(q_full, kConvWarps);
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
        int ref = -1, top = 0;   // biased exponents: the reference scale's, the largest page scale's
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
                    top = max(top, e);
                    if (e - ref > 7) {
                        shift = ref - e;
                        ref = e;
                    } else if (e - ref < -15) {
                        // a token adds at most 2^8 448 of its page's scale to O, so that 2^31 of
                        // them, in units of 2^-80 of the largest scale, stay below 2^128
                        const int to = max(e, top - 80);
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
                ok = mbar_wait(k_full + st, kphase, abort_flag, p.limit_ns);
                if (ok && b >= 2) ok = mbar_wait(pv_done + sb, pphase, abort_flag, p.limit_ns);
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
                ok = mbar_wait(w_full + wt, (b / kWStages) & 1, abort_flag, p.limit_ns) &&
                     mbar_wait(p_full + sb, (b >> 1) & 1, abort_flag, p.limit_ns);
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
        // ------------------------------------------------------------ queries, V codes -> fp16
        {
            const int quarter = warp & 3, row = N == 128 ? quarter * 32 + lane : lane;
            const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
            const uint8_t *img = cp.images + (static_cast<int64_t>(blockIdx.y) * cp.tiles + it.image) * kImage<N>;
            const uint32_t *sf = reinterpret_cast<const uint32_t *>(img + 2 * N * kD) + row;
            const uint32_t sfh = sf[0], sfl = sf[N];
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4 *>(w + 4 * i) = reinterpret_cast<const uint4 *>(img)[(8 * part + i) * N + row];
                VCA_TMEM_ST32(tl + kTmemQ + 32 * part, w);
            }
            // row m's factor words lie in lane m, column m / 32; B's factors are 1 everywhere
            asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(tl + kTmemSFA + quarter), "r"(sfh) : "memory");
            asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(tl + kTmemSFA + 4 + quarter), "r"(sfl) : "memory");
            asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%1,%1,%1};" ::"r"(tl + kTmemSFB), "r"(0x7f7f7f7fu) : "memory");
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
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
        const int quarter = warp & 3, half = (warp - kSoftWarp0) >> 2, at_lane = quarter * 32 + lane;
        const int row = N == 128 ? at_lane : lane, col0 = N == 128 ? 64 * half : 32 * quarter + 16 * half;
        constexpr int kCols = N == 128 ? 64 : 16, kLoad = N == 128 ? 32 : 16;      // a thread's columns, at a time
        const uint32_t bar_pair = kBarPair + quarter;
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const float kNegInf = __int_as_float(0xff800000);
        const int r = r0 + row;
        const bool real = r < R;
        // raw score -> log2 units (or the cap's inner argument), but for the page's scale
        const float f = kCap ? p.cap_in : p.scale_log2;
        const int seen = (real ? min(seen_by_row(p, it.s, r), it.s.len) : it.s.len) - it.page0 * kBlk - col0;
        // the warp's columns of pages before this one every row sees
        const int full = (__reduce_min_sync(0xffffffffu, seen) + kBlk - kCols) >> 7;
        PageScore s;
        s.cap = p.cap_out;
        s.bias = 0.0f;
        float m = kNegInf;
        uint64_t l2 = 0;
        bool ok = true;
        for (int b = 0; b < nb; ++b) {
            const int sb = b & 1;
            float *mx = sMX + sb * 2 * kLanes;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(s_full + sb, (b >> 1) & 1, abort_flag, p.limit_ns));
            if (!ok) {
                // the other half learns of it where they meet
                mx[half * kLanes + at_lane] = __int_as_float(0x7fc00000);
                bar_sync(bar_pair, 64);
                break;
            }
            const uint32_t tS = tl + kTmemS + 128 * sb;
            uint32_t X0[kLoad], X1[kLoad];      // X1: of 128 rows
            tc_fence_after();
            float m0, m1 = kNegInf;
            const float4 slot = sSlot[b % kSlots];
            s.edge = b >= full || slot.x < 0.0f;
            s.c = fmaxf(__fmul_rn(f, slot.x), 0x1p-149f);      // above 0, so that -inf stays -inf
            if constexpr (kCap) {
                // loaded twice: the load's own maximum is cheaper than the thread's
                load_scores<true>(tS + col0, X0, m0);
                if constexpr (N == 128) load_scores<true>(tS + col0 + 32, X1, m1);
                tmem_ld_wait();
                s.near = __all_sync(0xffffffffu, fmaxf(m0, m1) * s.c <= kTanhNear);
            }
            load_scores<false>(tS + col0, X0, m0);
            if constexpr (N == 128) load_scores<false>(tS + col0 + 32, X1, m1);
            tmem_ld_wait();
            if (s.edge) {
                s.lim = slot.x < 0.0f ? 0 : seen - b * kBlk;
                m0 = mask_scores<kCap>(X0, 0, s.lim);
                if constexpr (N == 128) m1 = mask_scores<kCap>(X1, 32, s.lim);
            }
            const float pm = fmaxf(m0, m1) * s.c;
            const float pc = kCap ? capped(pm, p.cap_out) : pm;
            const float bm = pc != pc ? kNegInf : pc;      // NaN scores reach O by their probabilities
            // the row's maximum over both halves; NaN: the other half gave up.  Both
            // halves have read their scores when they meet, so P may be written over
            // them.  Buffers by turns: the next page's barrier separates this read
            // from the write after it
            mx[half * kLanes + at_lane] = bm;
            bar_sync(bar_pair, 64);
            const float other = mx[(half ^ 1) * kLanes + at_lane], most = __fadd_rn(m, kLazyTau);
            // mostly neither the reference maximum nor the reference scale moves
            if (__any_sync(0xffffffffu, !(bm <= most) || !(other <= most) || slot.z != 1.0f)) {
                if (__any_sync(0xffffffffu, other != other)) {
                    ok = false;
                    break;
                }
                const float top = fmaxf(bm, other);
                float alpha = slot.z;
                if (top > most) {
                    const float down = ex2_approx(__fsub_rn(m, top));
                    l2 = mul2(l2, pk2(__float_as_uint(down), __float_as_uint(down)));
                    alpha *= down;
                    m = top;
                    s.bias = -m;
                }
                if (b > 0) {
                    // this half's channels of O, after PV(b - 1), to the new references
                    ok = __all_sync(0xffffffffu, mbar_wait(pv_done + (sb ^ 1), ((b - 1) >> 1) & 1, abort_flag, p.limit_ns));
                    if (!ok) continue;      // the other half learns of it where they meet next
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
            uint32_t W[kLoad / 2];
            probabilities<kCap>(X0, s, 0, l2, W);
            if constexpr (N == 128) {
                VCA_TMEM_ST16(tS + 32 * half, W);
                probabilities<kCap>(X1, s, 32, l2, W);
                VCA_TMEM_ST16(tS + 32 * half + 16, W);
            } else {
                // the lane quarter's own keys; the other quarters' are not this copy's
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t Y[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) Y[k] = q == quarter ? W[k] : 0u;
                    VCA_TMEM_ST8(tS + 16 * q + 8 * half, Y);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + sb);
        }
        float l;
        {
            float a, c;
            upk2(l2, a, c);
            l = __fadd_rn(a, c);
        }
        // ------------------------------------------------------------ epilogue
        // PV(nb - 1) complete (PV(nb - 3) was when S(nb - 1) came)
        if (ok)
            ok = __all_sync(0xffffffffu, mbar_wait(pv_done + ((nb - 1) & 1), ((nb - 1) >> 1) & 1, abort_flag, p.limit_ns));
        sL[half * kLanes + at_lane] = l;
        ok = bar_and(ok, kBarSoftmax, 32 * kSoftmaxWarps);
        if (ok) {
            tc_fence_after();
            const float M = m, Mu = M == kNegInf ? 0.0f : M, L = __fadd_rn(sL[at_lane], sL[kLanes + at_lane]);
            const float ref = sSlot[(nb - 1) % kSlots].w;
            // rows to shared memory (the K and V rings, free by now), then one bulk copy a
            // row: a thread's own stores, a row each, would take a cycle for every sector
            const bool final = N == 128 && it.parts == 1;
            const uint32_t pitch = final ? kD * 2 + 16 : kD * 4 + 16;      // 16 more: the rows' banks differ
            unsigned char *line = smem + at_lane * pitch;
            const float inv = !final ? 1.0f : L > 0.0f || L != L ? 1.0f / L : 0.0f;
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                uint32_t o[32];
                VCA_TMEM_LD32(tl + kTmemO + 64 * half + 32 * i, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv * ref);   // inv ref may be subnormal
                if (final) {
                    uint4 *to = reinterpret_cast<uint4 *>(line + 2 * (64 * half + 32 * i));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * k]), __uint_as_float(o[8 * e + 2 * k + 1]));
                        to[e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    uint4 *to = reinterpret_cast<uint4 *>(line + 4 * (64 * half + 32 * i));
#pragma unroll
                    for (int e = 0; e < 8; ++e) to[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            }
            float *part = p.part + (static_cast<int64_t>(h) * cp.grid + it.slot) * kPartFloats<N>;
            if constexpr (N == 32) {
                // the four copies of a row, each over its quarter of the keys, put together
                if (half == 0) sMX[at_lane] = M;
                bar_sync(kBarSoftmax, 32 * kSoftmaxWarps);
                const int i = (threadIdx.x - 32 * kSoftWarp0) >> 3, ch = (threadIdx.x & 7) * 16, ri = r0 + i;
                float top = kNegInf;
#pragma unroll
                for (int q = 0; q < 4; ++q) top = fmaxf(top, sMX[32 * q + i]);
                const float tu = top == kNegInf ? 0.0f : top;
                float sum = 0.0f, acc[16] = {};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int from = 32 * q + i;
                    const float k = ex2_approx(sMX[from] - tu);
                    sum = fmaf(__fadd_rn(sL[from], sL[kLanes + from]), k, sum);
                    const float4 *o = reinterpret_cast<const float4 *>(smem + from * pitch + 4 * ch);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 x = o[e];
                        acc[4 * e] = fmaf(x.x, k, acc[4 * e]);
                        acc[4 * e + 1] = fmaf(x.y, k, acc[4 * e + 1]);
                        acc[4 * e + 2] = fmaf(x.z, k, acc[4 * e + 2]);
                        acc[4 * e + 3] = fmaf(x.w, k, acc[4 * e + 3]);
                    }
                }
                if (it.parts > 1) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        reinterpret_cast<float4 *>(part + i * kD + ch)[e] =
                            make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]);
                    if (ch == 0) {
                        part[N * kD + i] = top;
                        part[N * kD + N + i] = sum;
                    }
                } else if (ri < R) {
                    const int64_t at = out_row(p, it.s, h, ri);
                    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(acc[8 * e + 2 * k] * inv, acc[8 * e + 2 * k + 1] * inv);
                        reinterpret_cast<uint4 *>(p.O + at * kD + ch)[e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (p.lse && ch == 0) p.lse[at] = tu * 0.6931471805599453f + logf(sum);
                }
            } else {
                fence_proxy_async_smem();
                bar_sync(bar_pair, 64);      // both halves of the row are there
                if (half == 0) {
                    if (it.parts == 1) {
                        if (real) {
                            const int64_t at = out_row(p, it.s, h, r);
                            bulk_store(p.O + at * kD, line, kD * 2);
                            if (p.lse) p.lse[at] = Mu * 0.6931471805599453f + logf(L);
                        }
                    } else {
                        if (real) bulk_store(part + row * kD, line, kD * 4);
                        part[N * kD + row] = M;
                        part[N * kD + N + row] = L;
                    }
                    bulk_store_wait();
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
template <int N>
__global__ void __launch_bounds__(256) join_kernel(const ChunkParams cp) {
    const AttnParams &p = cp.a;
    wait_for_results();
    const int first = cp.first[blockIdx.x];
    if (first < 0) return;
    const Item it = cp.items[first];
    if (it.parts == 1) return;
    const int h = blockIdx.y, row = 16 * blockIdx.z + (threadIdx.x >> 4), ch = (threadIdx.x & 15) * 8, r = it.tile * N + row;
    if (r >= it.s.n * p.G) return;
    const float *part = p.part + (static_cast<int64_t>(h) * cp.grid + it.slot) * kPartFloats<N>;
    float M = __int_as_float(0xff800000);
    for (int c = 0; c < it.parts; ++c) M = fmaxf(M, part[c * static_cast<int64_t>(kPartFloats<N>) + N * kD + row]);
    const float Mu = M == __int_as_float(0xff800000) ? 0.0f : M;
    float L = 0.0f, acc[8] = {};
    for (int c = 0; c < it.parts; ++c) {
        const float *q = part + c * static_cast<int64_t>(kPartFloats<N>);
        const float k = ex2_approx(q[N * kD + row] - Mu);
        L = fmaf(q[N * kD + N + row], k, L);
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

// Sizes of a call, and whether tiles are cut: where there can be fewer than two
// for every SM (the sequences' own number is known on the device alone, which
// cuts none if they fill the SMs).  64 tiles of 25 rows over 16,383 tokens, in
// tiles of 128: 92 us cut, 218 whole.
struct Plan {
    int64_t tiles;
    int split, grid, heads;      // heads: of one launch
    size_t off_first, off_images, off_parts, bytes;
};
template <int N>
Plan plan_of(int T, int Hq, int H, int B, int cols) {
    Plan q;
    q.tiles = static_cast<int64_t>(T) * (Hq / H) / N + (B < T ? B : T);
    q.split = q.tiles * H < kCutMost && cols > kSmallest ? 152 : 0;
    // cut tiles number at most one CTA's parts each, or what fits the CTAs
    q.grid = static_cast<int>(q.split && q.tiles < q.split / H ? q.split / H : q.tiles);
    q.off_first = sizeof(Item) * q.grid;
    q.off_images = (q.off_first + 4 * static_cast<size_t>(q.tiles) + 1023) / 1024 * 1024;
    // images of some heads at a time: enough tiles for many waves, and a bound on the workspace
    const int64_t fit = (64ll << 20) / (q.tiles * kImage<N>);
    q.heads = static_cast<int>(fit < 1 ? 1 : fit < H ? fit : H);
    q.off_parts = q.off_images + static_cast<size_t>(q.tiles) * q.heads * kImage<N>;
    q.bytes = q.off_parts + (q.split ? static_cast<size_t>(q.grid) * H * kPartFloats<N> * sizeof(float) : 0);
    return q;
}

// Tiles of 32 rows where a sequence and KV head have no more than that on average.
// 16 x 8 heads of 8,000 tokens: 16 rows 67 us in tiles of 32, 70 in tiles of 128; 32
// rows 68 and 72, with a cap 77 and 124; 40 rows 119 and 72, with a cap 136 and 123.
bool few_rows(int T, int Hq, int H, int B) { return static_cast<int64_t>(T) * (Hq / H) <= 32ll * B; }

template <int N>
cudaError_t launch(const CacheAttnArgs &a, cudaStream_t st) {
    CUtensorMap mk, mv;
    const uint64_t rows = static_cast<uint64_t>(a.c.pages) * a.c.H * kBlk;
    if (!make_tile_map(&mk, a.c.k8, rows) || !make_tile_map(&mv, a.c.v8, rows)) return cudaErrorInvalidValue;
    const Plan q = plan_of<N>(a.T, a.Hq, a.c.H, a.c.B, a.c.cols);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    ChunkParams cp;
    cp.a = attn_params(a.c, a.q, a.start, a.T, a.Hq, a.causal, a.scale, a.softcap, a.dev_status, a.wait_limit_ns);
    cp.a.O = a.O;
    cp.a.lse = a.lse;
    cp.a.part = reinterpret_cast<float *>(ws + q.off_parts);
    cp.items = reinterpret_cast<Item *>(ws);
    cp.first = reinterpret_cast<int *>(ws + q.off_first);
    cp.images = ws + q.off_images;
    cp.tiles = static_cast<int>(q.tiles);
    cp.grid = q.grid;
    cp.split = q.split;
    const auto kernel = a.softcap > 0.0f ? chunk_kernel<N, true> : chunk_kernel<N, false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    for (cp.h0 = 0; cp.h0 < a.c.H; cp.h0 += q.heads) {
        const int heads = a.c.H - cp.h0 < q.heads ? a.c.H - cp.h0 : q.heads;
        queries_kernel<N><<<dim3(cp.tiles, heads), kPlanThreads, 0, st>>>(cp);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        e = launch_after(kernel, dim3(q.grid, heads), kThreads, kSmem, st, mk, mv, cp);
        if (e != cudaSuccess) return e;
    }
    if (!q.split) return cudaSuccess;      // cut tiles are few: one launch had all heads
    return launch_after(join_kernel<N>, dim3(cp.tiles, a.c.H, N / 16), 256, 0, st, cp);
}

}  // namespace

size_t cache_chunk_workspace(int T, int Hq, int H, int B, int cols) {
    return few_rows(T, Hq, H, B) ? plan_of<32>(T, Hq, H, B, cols).bytes : plan_of<128>(T, Hq, H, B, cols).bytes;
}

cudaError_t launch_cache_chunk(const CacheAttnArgs &a, cudaStream_t st) {
    return few_rows(a.T, a.Hq, a.c.H, a.c.B) ? launch<32>(a, st) : launch<128>(a, st);
}

}  // namespace vca
