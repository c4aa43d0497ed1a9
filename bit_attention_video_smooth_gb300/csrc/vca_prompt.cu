// vca_prompt.cu -- attention of packed prompts over their own keys and values
// (bf16), bound by the tensor cores: 4 d flops for every visible pair.
//
// One CTA an SM takes works in turn: 256 query rows of a (sequence, KV head), two tiles
// of 128: G query heads of whole tokens, so that heads that share a KV head share its
// keys and values, which pass through shared memory once for both tiles.  Per block of 128
// keys and tile: S = Q K^T (smem x smem -> TMEM), the softmax takes S to P in its
// place (bf16, the values' type, as the MMA wants it: 2^-8 relative a probability,
// while the row sums take the unrounded ones in fp32), O += P V (TMEM x smem).  While
// one tile's softmax runs the tensor core works for the other.  TMEM: S0, S1, O0, O1, all of it.
// Warps:
//   0      TMA producer: K and V blocks alternate in a ring of four
//   1      MMA issuer: PV of a block and QK of the next, tile by tile.  QK writes the scores
//          over the probabilities that the PV before it reads.  That this needs no wait
//          between them is observed, not guaranteed: PTX promises the order of issue for
//          MMAs of one accumulator and shape, and these have two accumulators.  One thread's
//          MMAs have run in their order in all that was measured (300,000 launches of random
//          shapes, three of each, gave equal bits), and TMEM has no columns left for P.
//          The whole warp waits and one thread of it, elected, issues: then the operands
//          are in uniform registers, and an MMA takes 10.5 cycles to issue with A in TMEM
//          and 40 with A in shared memory (46 from a branch on the lane, which the
//          softmax's warps beside it make 95: 1,389 TFLOP/s against 1,605)
//   2      loads the queries; zeroes the rows of V behind the sequence's last token (they
//          are another sequence's, and may hold NaN) and only then reports that block as full
//   3      finds the CTA's works, some ahead of the others
//   4-11   softmax, four warps a tile, a thread a row.  P goes over in two parts.
//          The reference lies 8 (log2 units) above the maximum when it is set, and moves only
//          when a block's maximum exceeds it; O is rescaled in TMEM then: S(j) full
//          means that PV(j - 1) is done too.  So no probability is above 1, and O
//          is finite where the sums of a sequence's values' magnitudes are
//   12-15  epilogue: O / sum, joined with what came before, while the tiles go on to
//          their next work
// Every wait is bounded, as in vca_attention.cu; those that last as long as a work by as
// many times the limit as it can have blocks, and a tile's first one, which may
// come after works without that tile, by as many as the works at hand can.  Where one gives
// up all others do.
//
// What bounds it.  A block of both tiles is 2,048 cycles of the tensor core; it takes
// 2,670, since a tile's chain (scores -> softmax 1,150 -> PV -> QK) is longer than the other
// tile's 1,024 cycles of MMAs.  One prompt of 32,768 tokens, causal, 40 heads over 8, other
// inputs in every call: 6.5 ms, 1,690 TFLOP/s, 0.90 of cuBLAS's burst rate; 17,664 tokens
// both ways, 8 heads: 800 us, 1,590 TFLOP/s (552 works on 152 SMs).  Short prompts are
// bound by what a work costs beside its blocks, about 6,000 cycles: 32 of up to 1,000
// tokens, 40 heads over 8, 147 us, 870 TFLOP/s.  The code's size counts: all roles share
// the instruction caches, and a loop that no longer fits costs 5 to 15 %.
// The figures from here on are of loops over equal inputs, which are 3 to 5 % faster
// (6.3 ms, 770 us, 139 us).  Measured and not kept: an issuer for each tile (both
// tiles' MMAs then mix and their softmaxes fall together: 8.7 ms), a ring of three
// (7.2) or of five, which leaves no room for the statistics (6.24 against 6.39 at the
// time), O read into registers at once before its stores (162 us for the 32 prompts
// against 155 at the time), the queries prefetched into L2 (no change), a CTA for each
// work (886 us for 32 prompts of 1,000 tokens, 315 now).
#include <type_traits>

#include "vca_attention_common.cuh"
#include "vca_cache.cuh"

namespace vca {

namespace {

using namespace attn;
using namespace cache;

constexpr int kTiles = 2;
constexpr int kStages = 4;      // a power of two: copies are counted modulo 2^32
constexpr int kSoftWarp0 = 4, kOutWarp0 = kSoftWarp0 + 4 * kTiles, kThreads = 32 * (kOutWarp0 + 4);
constexpr uint32_t kPanel = kBlk * 128;              // 128 rows of 64 bf16 channels
constexpr uint32_t kBlock = 2 * kPanel;              // Q, K or V: two panels
constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemCols = 512;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffKV = kOffQ + kTiles * kBlock;
constexpr uint32_t kOffStat = kOffKV + kStages * kBlock;                  // fp32 [2][tile][max, sum][128], by turns
constexpr uint32_t kOffSort = kOffStat + 2 * kTiles * 2 * kBlk * 4;           // Sorted, of at most 256 sequences
constexpr uint32_t kOffBar = kOffSort + 3 * 256 * 4;
constexpr float kAbove = 256.0f;                     // 2^kLazyTau
constexpr int kWorks = 3;                            // slots for what the CTA does now and next
constexpr int kTurns = 2;                            // o_full barriers a tile, by turns of its works
constexpr int kNumBars = 3 * kStages + (6 + kTurns) * kTiles + 2 * kWorks + 1;
constexpr uint32_t kOffWork = (kOffBar + kNumBars * 8 + 15) / 16 * 16;
constexpr uint32_t kOffMisc = kOffWork + kWorks * 16;
constexpr uint32_t kSmem = kOffMisc + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

struct PromptParams {
    const int32_t *start;
    int B, T, Hq, causal;
    int G, tokens;                          // a tile: G query heads (of one KV head) of so many tokens
    int groups, per_head;                   // of G query heads, and of those to a KV head
    int64_t items;                          // (two tiles, group) at most
    float scale_log2, cap_in, cap_out;      // as in AttnParams
    bool k_tokens, v_tokens;                // the tensor map's middle dimension: tokens, else heads
    int k_heads, v_heads;                   // 1, or 0: all heads are the same
    const uint16_t *prior;
    const float *prior_lse;
    uint16_t *O;
    bool wide;                              // O is 32-byte aligned
    float *lse;
    int32_t *dev_status;
    uint64_t limit_ns, work_limit_ns;       // of a wait for a block, and of one for a whole work
    uint64_t works_limit_ns;                // of one for the works that a CTA has at hand
    uint64_t drain_ns;                      // of the last wait for copies and MMAs under way, which outlive no CTA
};

__device__ __forceinline__ void tma_load_3d(void *smem_dst, const void *tmap, uint64_t *bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

#define VCA_TMEM_LD16(taddr, r)                                                                                   \
    asm volatile(                                                                                                 \
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"  \
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),         \
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])    \
        : "r"(taddr))

// mbar_wait in less code: the kernel's loops have to fit the instruction caches, and
// a test suspends the thread for up to 7,760 cycles (3.9 us, measured) anyway.  So a wait
// gives up after two tests at the earliest, whatever its limit.
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, int *abort, uint64_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    do {
        if (mbar_try_wait(bar, parity)) return true;
        if (*reinterpret_cast<volatile int *>(abort)) return false;
    } while (globaltimer_ns() - t0 <= limit_ns);
    *reinterpret_cast<volatile int *>(abort) = 1;
    return false;
}

// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r != 0;
}

// ---------------------------------------------------------------------------
// Which tiles a CTA takes
// ---------------------------------------------------------------------------
// Two tiles of a (sequence, group of query heads): its tokens [row0, row0 + n), and
// which pair; n = 0: there is no more work.
struct Work {
    int row0, n, tile, group;
};
__device__ __forceinline__ int tiles_of(const PromptParams &p, int n) { return (n + 2 * p.tokens - 1) / (2 * p.tokens); }

// Up to kSortable sequences: the tiles by their number of key blocks, most first.  A
// causal tile's number grows with its place in the sequence, another's is the
// sequence's.  The CTAs then take turns, there and back, and have done about the same at the
// end.  A warp's work; the sequences' first tokens, tokens and tiles in shared memory.
// Many short sequences are slower so than searched: 256 of 100 tokens, 40 heads over 8, take
// 130 us, 257 of them, which are searched, 105.
constexpr int kSortable = 256;
struct Sorted {
    int lo[kSortable], n[kSortable], q[kSortable];
};
// Returns the most tiles of a sequence.
__device__ __forceinline__ int load_sorted(const PromptParams &p, Sorted &s) {
    const int lane = threadIdx.x & 31;
    bool fell = false;
    int most = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        int lo = 0, hi = 0;
        if (b < p.B) {
            lo = p.start[b];
            hi = p.start[b + 1];
        }
        const uint32_t falls = __ballot_sync(0xffffffffu, lo < 0 || hi < lo || hi > p.T);
        const int n = fell || (falls & ((2u << lane) - 1u)) ? 0 : hi - lo;
        fell = fell || falls != 0;
        s.lo[b] = lo;
        s.n[b] = n;
        s.q[b] = tiles_of(p, n);
        most = max(most, s.q[b]);
    }
    if (blockIdx.x == 0 && lane == 0 && fell) report(p.dev_status, kErrInvalid);
    __syncwarp();
    return __reduce_max_sync(0xffffffffu, most);
}
__device__ __forceinline__ bool find_sorted(const PromptParams &p, const Sorted &s, int most, int rank, Work &w) {
    const int lane = threadIdx.x & 31;
    auto above = [&](int c) {      // tiles of a cost above c
        int f = 0;
        for (int b = lane; b < p.B; b += 32) f += p.causal ? max(0, s.q[b] - c) : s.q[b] > c ? s.q[b] : 0;
        return static_cast<int>(__reduce_add_sync(0xffffffffu, f));
    };
    if (above(0) <= rank) return false;
    int a = 0, z = most;      // above(a) > rank >= above(z)
    while (z - a > 1) {
        const int mid = a + (z - a) / 2;
        if (above(mid) > rank)
            a = mid;
        else
            z = mid;
    }
    int left = rank - above(z);      // among the tiles of cost a + 1, in the sequences' order
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int q = b0 + lane < p.B ? s.q[b0 + lane] : 0, has = p.causal ? (q > a) : q == a + 1 ? q : 0;
        int incl = has;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, left < incl);
        if (hit) {
            const int l = __ffs(hit) - 1;
            w.row0 = s.lo[b0 + l];
            w.n = s.n[b0 + l];
            w.tile = p.causal ? a : left - __shfl_sync(0xffffffffu, incl - has, l);
            return true;
        }
        left -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}

// More sequences: sequence b's tiles are those from floor(start / tokens) + b on, which
// leaves room for each sequence's and is found by search among the `rise` sequences
// before the first whose start falls.  A warp's work; false where no tile is.
__device__ __forceinline__ bool find_searched(const PromptParams &p, int rise, int index, Work &w) {
    const int lane = threadIdx.x & 31;
    auto base = [&](int b) { return static_cast<int64_t>(p.start[b] / (2 * p.tokens)) + b; };
    int a = 0, z = rise;      // base(a) <= index < base(z), or z = rise
    while (z - a > 1) {
        const int step = (z - a + 31) / 32, at = a + lane * step;
        const int hits = __popc(__ballot_sync(0xffffffffu, at < z && base(at) <= index));
        if (hits == 0) return false;
        a += (hits - 1) * step;
        z = min(z, a + step);
    }
    if (rise == 0 || base(a) > index) return false;
    w.row0 = p.start[a];
    w.n = p.start[a + 1] - w.row0;
    w.tile = static_cast<int>(index - base(a));
    return w.tile < tiles_of(p, w.n);
}

// Keys that the rows of tile t see, and blocks of them; 0: it has no rows.
__device__ __forceinline__ int seen_by(const PromptParams &p, const Work &w, int t) {
    const int first = (2 * w.tile + t) * p.tokens;
    return first >= w.n ? 0 : p.causal ? min(w.n, first + p.tokens) : w.n;
}
__device__ __forceinline__ int blocks_of(const PromptParams &p, const Work &w, int t) { return (seen_by(p, w, t) + kBlk - 1) / kBlk; }
// The block that ends behind the sequence's last token, if it is among the first nbs; else -1.
__device__ __forceinline__ int tail_of(const Work &w, int nbs) {
    return w.n % kBlk && nbs == (w.n + kBlk - 1) / kBlk ? nbs - 1 : -1;
}

// ---------------------------------------------------------------------------
// Softmax pieces
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t both(float x) { return pk2(__float_as_uint(x), __float_as_uint(x)); }
__device__ __forceinline__ uint64_t pk2f(float lo, float hi) { return pk2(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 32 raw scores -> words of bf16 pairs, p = 2^(S c + bias); the unrounded ones add to l2.
__device__ __forceinline__ void probabilities(const uint32_t (&X)[32], float c, float bias, uint64_t &l2, uint32_t (&W)[16]) {
    const uint64_t c2 = both(c), b2 = both(bias);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float a, b;
        upk2(fma2(pk2(X[2 * k], X[2 * k + 1]), c2, b2), a, b);
        a = ex2_approx(a);
        b = ex2_approx(b);
        l2 = add2(l2, pk2f(a, b));
        W[k] = pack_bf16x2(a, b);
    }
}

// The same of capped scores, p = 2^(cap tanh_half(S c) + bias), and 0 from column `lim`
// on.  tanh_half(u) = 1 - 2 / (1 + 2^u) has an absolute error, and with its roundings a
// score is off by up to 2^-20 of the cap, however small the score is itself: 6e-5 at
// kSmallCap, up to which this is all (kCap = 1).  For larger ones (kCap = 2) it is
// taken from |u| = kTanhNear on and the polynomial, with its relative error, below, as
// in tanh_half; alone where all lanes are `near`. 4 prompts of up to 2,900 tokens, 32
// heads over 8, cap 30: 189 us, by kCap = 2 322.
constexpr float kSmallCap = 64.0f;
template <int kCap>
__device__ __forceinline__ void capped_probabilities(const uint32_t (&X)[32], float c, float cap, float bias, bool near, int lim,
                                                     uint64_t &l2, uint32_t (&W)[16]) {
    const uint64_t c2 = both(c), b2 = both(bias), one = both(1.0f), far_m = both(-2.0f * cap), far_b = both(__fadd_rn(cap, bias));
    const uint64_t t0 = both(cap * kT0), t1 = both(cap * kT1), t2 = both(cap * kT2), t3 = both(cap * kT3), t4 = both(cap * kT4);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const uint64_t u = mul2(pk2(X[2 * k], X[2 * k + 1]), c2), w = mul2(u, u);
        float a = 0.0f, b = 0.0f;
        if constexpr (kCap == 2) upk2(fma2(u, fma2(fma2(fma2(fma2(t4, w, t3), w, t2), w, t1), w, t0), b2), a, b);
        if (kCap == 1 || !near) {
            float ua, ub, ra, rb;
            upk2(u, ua, ub);
            upk2(add2(pk2f(ex2_approx(ua), ex2_approx(ub)), one), ra, rb);
            upk2(fma2(pk2f(rcp_approx(ra), rcp_approx(rb)), far_m, far_b), ra, rb);
            a = kCap == 2 && fabsf(ua) <= kTanhNear ? a : ra;
            b = kCap == 2 && fabsf(ub) <= kTanhNear ? b : rb;
        }
        a = 2 * k < lim ? ex2_approx(a) : 0.0f;
        b = 2 * k + 1 < lim ? ex2_approx(b) : 0.0f;
        l2 = add2(l2, pk2f(a, b));
        W[k] = pack_bf16x2(a, b);
    }
}

// Scores of keys that the row does not see, from column `lim` on, become -inf;
// returns the largest of the others.
__device__ __forceinline__ float mask_scores(uint32_t (&X)[32], int lim) {
    float m = __int_as_float(0xff800000);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        if (e < lim) m = fmaxf(m, __uint_as_float(X[e]));
        else X[e] = 0xff800000u;
    }
    return m;
}

// A row's 32 bytes (kWide: 32-byte aligned).
template <bool kWide>
__device__ __forceinline__ void store32(uint16_t *to, const uint32_t *w) {
    if constexpr (kWide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(reinterpret_cast<uint64_t>(to)), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// kCap: 0 no cap, 1 a small one, 2 any.  kShort: the MMA issuer's code once for both
// tiles, not twice, and P handed over in 96 and 32 keys, not 64 and 64.  The code has to
// fit the instruction caches beside the softmax's, and a miss leaves the tensor core idle;
// in long loops the addresses that are known then count more, and the larger first part
// costs what the smaller second one brings.  Without a cap (us, kShort and not; 40 heads over 8
// causal, 8 heads both ways): 32 prompts of 1,000 tokens 315 and 335, 16 of 1,500 295 and
// 308, 12 of 2,000 363 and 368, 8 of 2,500 355 and 355, one of 32,768 6,400 and 6,280; both ways 64
// of 256 93 and 111, 32 of 1,200 147 and 145, one of 17,664 781 and 767.  With one kShort
// is the faster or the same: 8,192 tokens, 32 heads over 8, cap 30, 596 and 622.
constexpr int kShortKeys = 1024;      // that a work sees on average
template <int kCap, bool kShort>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const PromptParams p) {
    constexpr int kCopies = kShort ? 1 : kTiles, kFirst = kShort ? 3 : 2;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = smem_raw + (0u - smem_u32(smem_raw)) % 1024u;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBar), *empty = full + kStages, *raw = empty + kStages;
    uint64_t *q_full = raw + kStages, *q_free = q_full + kTiles, *s_full = q_free + kTiles, *p_full = s_full + kTiles;
    uint64_t *o_full = p_full + 2 * kTiles, *o_free = o_full + kTurns * kTiles, *w_full = o_free + kTiles, *w_free = w_full + kWorks;
    uint64_t *drain = w_free + kWorks;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    int *abort_flag = reinterpret_cast<int *>(smem + kOffMisc + 4);
    int *first_fall = reinterpret_cast<int *>(smem + kOffMisc + 8);
    Work *works = reinterpret_cast<Work *>(smem + kOffWork);
    float *stats = reinterpret_cast<float *>(smem + kOffStat);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
            mbar_init(raw + s, 1);
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(q_full + t, 1);
            mbar_init(q_free + t, 1);
            mbar_init(s_full + t, 1);
            mbar_init(p_full + 2 * t, 4);
            mbar_init(p_full + 2 * t + 1, 4);
            for (int i = 0; i < kTurns; ++i) mbar_init(o_full + kTurns * t + i, 1 + 4);      // the last MMAs, and the softmax warps' statistics
            mbar_init(o_free + t, 4);
        }
        for (int i = 0; i < kWorks; ++i) {
            mbar_init(w_full + i, 1);
            mbar_init(w_free + i, 3 + 4 * kTiles + 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        *first_fall = p.B;
        mbar_fence_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    if (p.B > kSortable) {
        __syncthreads();
        for (int b = threadIdx.x; b < p.B; b += kThreads) {
            const int lo = p.start[b], hi = p.start[b + 1];
            if (lo < 0 || hi < lo || hi > p.T) atomicMin(first_fall, b);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // The k-th work of this CTA, from its slot; false at the end, or where a wait gave up.
    auto next_work = [&](int k, Work &w) {
        const int i = k % kWorks;
        if (!__all_sync(0xffffffffu, wait_phase(w_full + i, (k / kWorks) & 1, abort_flag, p.work_limit_ns))) return false;
        w = works[i];
        return w.n > 0;
    };
    auto work_done = [&](int k) {      // a warp's
        __syncwarp();
        if (lane == 0) mbar_arrive(w_free + k % kWorks);
    };

    // registers: 128 x 72 + 256 x 168 + 128 x 104 = 512 x 128, those at launch
    if (warp < kSoftWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0) {
            // -------------------------------------------------------- producer of K and V
            Work w;
            uint32_t i = 0;             // the next copy: K(0), V(0), K(1), V(1), ... of one work after the other, modulo 2^32
            int issued = 0;             // copies, kStages at most
            uint32_t tails = 0;         // stages whose last copy `raw` counts,
            uint32_t turns = 0;         // and the next phase of each stage's
            bool ok = true;
            for (int k = 0; ok && next_work(k, w); ++k) {
                const int nbs = max(blocks_of(p, w, 0), blocks_of(p, w, 1)), tail = tail_of(w, nbs), kv_head = w.group / p.per_head;
                for (int j = 0; ok && j < 2 * nbs; ++j, ++i) {
                    const uint32_t st = i % kStages;
                    // of a new barrier the phase before the first counts as complete
                    ok = __all_sync(0xffffffffu, wait_phase(empty + st, (i / kStages - 1) & 1, abort_flag, p.limit_ns));
                    if (!ok) break;
                    issued = min(issued + 1, kStages);
                    const bool is_v = j & 1, is_tail = j == 2 * tail + 1;
                    tails = is_tail ? tails | (1u << st) : tails & ~(1u << st);
                    turns ^= is_tail ? 1u << st : 0u;
                    if (lane == 0) {
                        const int token = w.row0 + (j >> 1) * kBlk, head = kv_head * (is_v ? p.v_heads : p.k_heads);
                        const bool tokens = is_v ? p.v_tokens : p.k_tokens;
                        unsigned char *to = smem + kOffKV + st * kBlock;
                        uint64_t *landed = is_tail ? raw + st : full + st;
                        mbar_expect_tx(landed, kBlock);
                        for (int c = 0; c < 2; ++c)
                            tma_load_3d(to + c * kPanel, is_v ? &tmV : &tmK, landed, 64 * c, tokens ? token : head, tokens ? head : token);
                    }
                }
                work_done(k);
            }
            // every copy issued has landed before the CTA can exit
            if (lane == 0) {
                for (uint32_t j = i - issued; j != i; ++j) {
                    const uint32_t st = j % kStages;
                    if ((tails >> st) & 1u)
                        drain_wait(raw + st, ((turns >> st) & 1u) ^ 1u, p.drain_ns);
                    else
                        drain_wait(full + st, (j / kStages) & 1, p.drain_ns);
                }
            }
        } else if (warp == 1) {
            // -------------------------------------------------------- MMA issuer
            const uint32_t base = smem_u32(smem);
            const bool one = elect_one();
            auto wait = [&](uint64_t *bar, int parity) {
                const bool ok = __all_sync(0xffffffffu, wait_phase(bar, parity, abort_flag, p.limit_ns));
                tc_fence_after();
                return ok;
            };
            // a block of which the tile sees 64 keys or fewer is half a block
            auto qk = [&](int t, uint32_t st, bool half) {
                const uint64_t dq = sdesc_k_sw128(base + kOffQ + t * kBlock), dk = sdesc_k_sw128(base + kOffKV + st * kBlock);
                const uint32_t idesc = half ? make_idesc(128, 64, 1, 1) : make_idesc(128, 128, 1, 1);
                if (one) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t step = (i >> 2) * (kPanel >> 4) + 2 * (i & 3);
                        mma_f16(tmem + kTmemS + 128 * t, dq + step, dk + step, idesc, i > 0);
                    }
                    tc_commit(s_full + t);
                }
            };
            auto pv = [&](int t, uint32_t st, auto from, auto to, bool first) {      // of keys 16 from .. 16 to - 1
                const uint64_t dv = sdesc_mn_sw128(base + kOffKV + st * kBlock, kPanel);
                if (one) {
#pragma unroll
                    for (int i = decltype(from)::value; i < decltype(to)::value; ++i)
                        mma_f16_ts(tmem + kTmemO + 128 * t, tmem + kTmemS + 128 * t + 8 * i, dv + (2048 >> 4) * i,
                                   make_idesc(128, 128, 1, 1, 0, 1), !first || i > 0);
                }
            };
            using std::integral_constant;
            auto commit = [&](uint64_t *bar) {
                if (one) tc_commit(bar);
            };
            Work w;
            uint32_t i0 = 0;                    // the ring's copies before this work's, modulo 2^32
            uint32_t blocks[kTiles] = {0, 0};   // of each tile so far
            uint32_t had[kTiles] = {0, 0};      // works that had the tile, the current one not among them
            auto of = [](const auto (&x)[kTiles], int t) { return t ? x[1] : x[0]; };
            // a work's first QK, of tile t; its first block is in the ring's copy `at`
            auto begin = [&](int t, int seen, uint32_t at) {
                if (seen == 0) return true;
                if (!wait(full + at % kStages, (at / kStages) & 1) || !wait(q_full + t, of(had, t) & 1)) return false;
                qk(t, at % kStages, seen <= 64);
                if (seen <= kBlk) commit(q_free + t);
                return true;
            };
            bool ok = next_work(0, w);
            int seen[kTiles] = {0, 0};
            if (ok) {
                seen[0] = seen_by(p, w, 0);
                seen[1] = seen_by(p, w, 1);
#pragma unroll 1
                for (int t = 0; t < kTiles; ++t) ok = ok && begin(t, of(seen, t), 0);
                commit(empty);
            }
            for (int k = 0; ok; ++k) {
                const int nbs = (max(seen[0], seen[1]) + kBlk - 1) / kBlk;
                const uint32_t i1 = i0 + 2 * nbs;
                // Barriers are tested before they are needed, several at once, and V's and K's of the
                // next block while the tensor core has the second tile's scores to do: a test takes 100
                // cycles, and one after the other left it idle
                auto landed = [&](int j) {      // V of block j, and K of the next
                    const uint32_t iv = i0 + 2 * j + 1, ik = iv + 1;
                    return mbar_test_wait(full + iv % kStages, (iv / kStages) & 1) &
                           (j + 1 >= nbs || mbar_test_wait(full + ik % kStages, (ik / kStages) & 1));
                };
                bool there = landed(0);
                // A block of tile t: its PV and, unless it is the work's last block, the next QK.
                auto block = [&](int t, int j, bool last) {
                    const int left = of(seen, t) - j * kBlk;      // keys of this block and behind
                    if (left <= 0) return true;
                    const uint32_t iv = i0 + 2 * j + 1, ik = iv + 1, sv = iv % kStages, sk = ik % kStages;
                    const int turn = static_cast<int>(of(blocks, t)) & 1;
                    blocks[0] += t == 0;
                    blocks[1] += t == 1;
                    uint64_t *parts = p_full + 2 * t;
                    const bool first = mbar_test_wait(parts, turn), second = mbar_test_wait(parts + 1, turn);
                    if (!__all_sync(0xffffffffu, there)) {
                        if (!wait(full + sv, (iv / kStages) & 1)) return false;
                        if (!last && !wait(full + sk, (ik / kStages) & 1)) return false;
                        there = true;
                    }
                    // O's first product waits until the epilogue before has read it
                    if (j == 0 && of(had, t) > 0 && !wait(o_free + t, (of(had, t) - 1) & 1)) return false;
                    if (!__all_sync(0xffffffffu, first) && !wait(parts, turn)) return false;
                    tc_fence_after();
                    pv(t, sv, integral_constant<int, 0>{}, integral_constant<int, 4>{}, j == 0);
                    if (kFirst > 2 && left > 64) pv(t, sv, integral_constant<int, 4>{}, integral_constant<int, 2 * kFirst>{}, false);
                    if (!__all_sync(0xffffffffu, second) && !wait(parts + 1, turn)) return false;
                    tc_fence_after();
                    if (left > 64) pv(t, sv, integral_constant<int, 2 * kFirst>{}, integral_constant<int, 8>{}, false);
                    if (t == 1 || j * kBlk >= seen[1]) {
                        commit(empty + sv);
                        there = last || landed(j + 1);
                    }
                    if (left > kBlk) {
                        qk(t, sk, left <= kBlk + 64);
                        if (left <= 2 * kBlk) commit(q_free + t);
                    } else {
                        commit(o_full + kTurns * t + (of(had, t) & 1));
                    }
                    return true;
                };
                for (int j = 0; ok && j + 1 < nbs; ++j) {
#pragma unroll kCopies
                    for (int t = 0; t < kTiles; ++t) ok = ok && block(t, j, false);
                    if (ok) commit(empty + (i0 + 2 * j + 2) % kStages);
                }
                // the last one, after which each tile goes on to its next work's first scores
                Work next;
                const bool more = ok && next_work(k + 1, next);
                const int sees[kTiles] = {more ? seen_by(p, next, 0) : 0, more ? seen_by(p, next, 1) : 0};
                int begun = 0;
#pragma unroll kCopies
                for (int t = 0; t < kTiles; ++t) {
                    ok = ok && block(t, nbs - 1, true);
                    had[0] += t == 0;
                    had[1] += t == 1 && seen[1] > 0;
                    // tile 0 not where tile 1's block would wait for what this needs
                    const bool now = t == 1 || __all_sync(0xffffffffu, mbar_test_wait(q_full, had[0] & 1) &
                                                                           mbar_test_wait(full + i1 % kStages, (i1 / kStages) & 1));
                    for (; now && begun <= t; ++begun) ok = ok && begin(begun, of(sees, begun), i1);
                }
                if (!ok) break;
                work_done(k);
                if (!more) break;
                commit(empty + i1 % kStages);
                w = next;
                i0 = i1;
                seen[0] = sees[0];
                seen[1] = sees[1];
            }
            commit(drain);
            if (one) drain_wait(drain, 0, p.drain_ns);
            __syncwarp();
        } else if (warp == 2) {
            // -------------------------------------------------------- queries, and rows of V behind a sequence
            Work w;
            uint32_t i0 = 0;
            uint32_t turns = 0;                  // the phase of each stage's `raw`
            uint32_t had1 = 0;                   // works that had a second tile
            int queries0 = -1, queries1 = -1;    // the last copy of each tile's
            bool ok = true;
            for (int k = 0; ok && next_work(k, w); ++k) {
#pragma unroll 1
                for (int t = 0; ok && t < kTiles; ++t) {
                    const int token = (2 * w.tile + t) * p.tokens, earlier = t ? static_cast<int>(had1) : k;
                    if (token >= w.n) break;
                    if (earlier > 0) ok = __all_sync(0xffffffffu, wait_phase(q_free + t, (earlier - 1) & 1, abort_flag, p.work_limit_ns));
                    if (!ok) break;
                    if (lane == 0) {
                        unsigned char *sQ = smem + kOffQ + t * kBlock;
                        mbar_expect_tx(q_full + t, 2 * 128 * p.G * p.tokens);
                        for (int c = 0; c < 2; ++c) tma_load_3d(sQ + c * kPanel, &tmQ, q_full + t, 64 * c, w.group * p.G, w.row0 + token);
                    }
                    had1 += t;
                    if (t == 0)
                        queries0 = earlier;
                    else
                        queries1 = earlier;
                }
                const int nbs = max(blocks_of(p, w, 0), blocks_of(p, w, 1)), tail = tail_of(w, nbs);
                if (ok && tail >= 0) {
                    const uint32_t st = (i0 + 2 * tail + 1) % kStages;
                    const int live = w.n - tail * kBlk;
                    ok = __all_sync(0xffffffffu, wait_phase(raw + st, (turns >> st) & 1, abort_flag, p.work_limit_ns));
                    if (!ok) break;
                    turns ^= 1u << st;
                    uint4 *to = reinterpret_cast<uint4 *>(smem + kOffKV + st * kBlock);
                    for (int e = 8 * live + lane; e < 8 * kBlk; e += 32) to[e] = to[e + kPanel / 16] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full + st);
                }
                i0 += 2 * nbs;
                work_done(k);
            }
            // the last queries have landed before the CTA can exit
            if (lane == 0) {
                if (queries0 >= 0) drain_wait(q_full, queries0 & 1, p.drain_ns);
                if (queries1 >= 0) drain_wait(q_full + 1, queries1 & 1, p.drain_ns);
            }
        } else {
            // -------------------------------------------------------- the CTA's works, ahead of all others
            Sorted &s = *reinterpret_cast<Sorted *>(smem + kOffSort);
            const int rise = *first_fall;
            int most = 0;
            if (p.B <= kSortable)
                most = load_sorted(p, s);
            else if (blockIdx.x == 0 && lane == 0 && rise < p.B)
                report(p.dev_status, kErrInvalid);
            const int ctas = static_cast<int>(gridDim.x), me = static_cast<int>(blockIdx.x);
            int k = 0;
            bool ok = true;
            for (int64_t turn = 0; ok; ++turn) {
                const int64_t index = turn * ctas + (turn & 1 ? ctas - 1 - me : me);
                Work w{0, 0, 0, 0};
                const bool end = index >= p.items;
                if (!end) {
                    const int rank = static_cast<int>(index / p.groups);
                    w.group = static_cast<int>(index % p.groups);
                    if (!(p.B <= kSortable ? find_sorted(p, s, most, rank, w) : find_searched(p, rise, rank, w))) continue;
                }
                if (k >= kWorks) ok = __all_sync(0xffffffffu, wait_phase(w_free + k % kWorks, (k / kWorks - 1) & 1, abort_flag, p.work_limit_ns));
                if (!ok) break;
                __syncwarp();
                if (lane == 0) {
                    if (end) w.n = 0;
                    works[k % kWorks] = w;
                    mbar_arrive(w_full + k % kWorks);
                }
                if (end) break;
                ++k;
            }
        }
    } else if (warp < kOutWarp0) {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        const int t = (warp - kSoftWarp0) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const float kNegInf = __int_as_float(0xff800000);
        const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16), tS = tl + kTmemS + 128 * t,
                       tO = tl + kTmemO + 128 * t;
        const int row_token = row / p.G;
        Work w;
        uint32_t blocks = 0, had = 0;      // of this tile so far, and works that had it
        bool ok = true;
        for (int k = 0; ok && next_work(k, w); ++k) {
            const int tile_sees = seen_by(p, w, t), n_blocks = (tile_sees + kBlk - 1) / kBlk;
            work_done(k);
            if (n_blocks == 0) continue;
            const int token = (2 * w.tile + t) * p.tokens + row_token;
            const bool real = row_token < p.tokens && token < w.n;
            const int seen = real && p.causal ? token + 1 : w.n;
            const int whole = __reduce_min_sync(0xffffffffu, seen) / kBlk;      // blocks that every row of the warp sees all of
            const float c = fmaxf(kCap ? p.cap_in : p.scale_log2, 0x1p-149f);      // above 0, so that -inf stays -inf
            float bias = 0.0f;
            float m = kNegInf;      // the reference
            uint64_t l2 = 0;
            for (int b = 0; b < n_blocks; ++b) {
                // where the works before have no such tile, their other one's blocks come first
                ok = __all_sync(0xffffffffu, wait_phase(s_full + t, blocks++ & 1, abort_flag, b == 0 ? p.works_limit_ns : p.limit_ns));
                if (!ok) break;
                tc_fence_after();
                const bool edge = b >= whole, half_block = tile_sees - b * kBlk <= 64;
                const int lim = seen - b * kBlk;      // columns of the block that the row sees
                // 32 columns at a time: mostly all rows of the warp see them
                const int least = edge ? __reduce_min_sync(0xffffffffu, lim) : kBlk;
                uint32_t X[kCap == 2 ? 1 : 4][32];
                float bm = kNegInf;
                uint32_t near = 0;
                if constexpr (kCap == 2) {
                    // scores are loaded again where they are needed: the code of 32 columns fits the
                    // instruction caches, that of 128 does not
#pragma unroll 1
                    for (int i = 0; i < (half_block ? 2 : 4); ++i) {
                        float top, mx;
                        VCA_TMEM_LDTOP32(tS + 32 * i, X[0], top);
                        tmem_ld_wait();
                        VCA_TMEM_LDMAX32(tS + 32 * i, X[0], mx);
                        tmem_ld_wait();
                        near |= __all_sync(0xffffffffu, top * c <= kTanhNear) ? 1u << i : 0u;
                        if (least < 32 * (i + 1)) mx = mask_scores(X[0], lim - 32 * i);
                        bm = fmaxf(bm, mx);
                    }
                    bm = capped(bm * c, p.cap_out);
                } else {
                    float mx[4];
                    mx[2] = mx[3] = kNegInf;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < 2 || !half_block) VCA_TMEM_LDMAX32(tS + 32 * i, X[i], mx[i]);
                    tmem_ld_wait();
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (least < 32 * (i + 1) && (i < 2 || !half_block)) mx[i] = mask_scores(X[i], lim - 32 * i);
                    }
                    bm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                    if constexpr (kCap == 1) bm = capped(bm, p.cap_out);
                }
                const bool rises = real && bm > m;      // a row that is none may hold anything
                if (__any_sync(0xffffffffu, rises)) {
                    float alpha = 1.0f;
                    if (rises) {
                        bias = -__fadd_rn(bm, kLazyTau);
                        alpha = ex2_approx(__fadd_rn(m, bias));
                        l2 = mul2(l2, pk2(__float_as_uint(alpha), __float_as_uint(alpha)));
                        m = -bias;
                    }
                    if (b > 0) {
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {
                            uint32_t o[16];
                            VCA_TMEM_LD16(tO + 16 * i, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), alpha));
                            VCA_TMEM_ST16(tO + 16 * i, o);
                        }
                    }
                }
                // P of the first kFirst times 32 keys, and of the others
                auto hand_over = [&](int part) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + 2 * t + part);
                };
                if constexpr (kCap == 2) {
#pragma unroll 1
                    for (int i = 0; i < (half_block ? 2 : 4); ++i) {
                        uint32_t W[16];
                        VCA_TMEM_LD32(tS + 32 * i, X[0]);
                        tmem_ld_wait();
                        capped_probabilities<2>(X[0], c, p.cap_out, bias, (near >> i) & 1u, least < 32 * (i + 1) ? lim - 32 * i : 32, l2, W);
                        VCA_TMEM_ST16(tS + 16 * i, W);      // over scores already read
                        tmem_st_wait();
                        if (i == kFirst - 1) hand_over(0);
                        if (i == 3) hand_over(1);
                    }
                    if (half_block) {
                        if (kFirst > 2) hand_over(0);
                        hand_over(1);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i < 2 || !half_block) {
                            uint32_t W[16];
                            if constexpr (kCap == 1)
                                capped_probabilities<1>(X[i], c, p.cap_out, bias, false, least < 32 * (i + 1) ? lim - 32 * i : 32, l2, W);
                            else
                                probabilities(X[i], c, bias, l2, W);
                            VCA_TMEM_ST16(tS + 16 * i, W);
                        }
                        if (i == kFirst - 1 || i == 3) {
                            tmem_st_wait();
                            hand_over(i == 3);
                        }
                    }
                }
            }
            if (!ok) break;
            // The row's maximum and sum go to the epilogue, by turns: before the scores of
            // the work after next come, the epilogue has read O and these.  The barrier takes turns
            // too: the next work's scores wait for this one's probabilities of all four warps,
            // but not for their statistics, and a warp that is a work ahead must not arrive in
            // a slower one's place.  The scores of the work after next wait for probabilities
            // that each warp hands over behind this arrival.
            float even, odd;
            upk2(l2, even, odd);
            const uint32_t turn = had++ & 1;
            float *mine = stats + (turn * kTiles + t) * 2 * kBlk + row;
            mine[0] = __fsub_rn(m, kLazyTau);      // as if the reference were the maximum that set it,
            mine[kBlk] = __fmul_rn(__fadd_rn(even, odd), kAbove);      // which keeps the sum near 1 and lse its bits
            __syncwarp();
            if (lane == 0) mbar_arrive(o_full + kTurns * t + turn);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        const int quarter = warp & 3, row = quarter * 32 + lane, row_token = row / p.G, row_head = row % p.G;
        const float kNegInf = __int_as_float(0xff800000);
        Work w;
        uint32_t had[kTiles] = {0, 0};
        bool ok = true;
        for (int k = 0; ok && next_work(k, w); ++k) {
#pragma unroll 1
            for (int t = 0; ok && t < kTiles; ++t) {
                if (seen_by(p, w, t) == 0) break;
                const int token = (2 * w.tile + t) * p.tokens + row_token;
                const bool real = row_token < p.tokens && token < w.n;
                const int64_t at = static_cast<int64_t>(w.row0 + token) * p.Hq + w.group * p.G + row_head;
                float before = kNegInf, keep = 1.0f, add = 0.0f;
                if (p.prior && real) before = p.prior_lse[at] * 1.4426950408889634f;
                const bool joins = before != kNegInf;
                // the prior's row, 32 channels ahead: from here on the tile's next products wait for O
                const uint4 *prior = reinterpret_cast<const uint4 *>(p.prior + at * kD);
                uint4 ahead[4] = {};
                if (joins) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) ahead[e] = prior[e];
                }
                const uint32_t turn = t == 0 ? had[0]++ : had[1]++;
                ok = __all_sync(0xffffffffu, wait_phase(o_full + kTurns * t + (turn & 1), (turn >> 1) & 1, abort_flag, p.work_limit_ns));
                if (!ok) break;
                tc_fence_after();
                const float *stat = stats + ((turn & 1) * kTiles + t) * 2 * kBlk + row;
                float M = stat[0], l = stat[kBlk];
                // joined with what came before: both sums to the larger maximum
                if (joins) {
                    const float m = M;
                    M = before != before ? before : fmaxf(m, before);
                    keep = m == kNegInf ? 0.0f : ex2_approx(__fsub_rn(m, M));
                    add = ex2_approx(__fsub_rn(before, M));
                    l = __fadd_rn(__fmul_rn(l, keep), add);
                }
                const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
                keep *= inv * kAbove;
                add *= inv;
                const uint32_t tO = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kTmemO + 128 * t;
                uint16_t *to = p.O + at * kD;
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    uint32_t o[32];
                    VCA_TMEM_LD32(tO + 32 * i, o);
                    tmem_ld_wait();
                    if (i == 3) {      // O is read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_free + t);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), keep));
                    if (joins) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint4 x = ahead[e];
                            if (i < 3) ahead[e] = prior[4 * i + 4 + e];
                            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                uint32_t &lo = o[8 * e + 2 * q], &hi = o[8 * e + 2 * q + 1];
                                lo = __float_as_uint(fmaf(__uint_as_float(xs[q] << 16), add, __uint_as_float(lo)));
                                hi = __float_as_uint(fmaf(__uint_as_float(xs[q] & 0xffff0000u), add, __uint_as_float(hi)));
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                    if (real) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (p.wide)
                                store32<true>(to + 32 * i + 16 * e, o + 8 * e);
                            else
                                store32<false>(to + 32 * i + 16 * e, o + 8 * e);
                        }
                    }
                }
                if (p.lse && real) p.lse[at] = (M == kNegInf ? 0.0f : M) * 0.6931471805599453f + logf(l);
            }
            work_done(k);
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

// bf16 rows as a 3-D matrix [z][y][128] and boxes of 64 channels.
bool make_rows_map(CUtensorMap *map, const uint16_t *base, cuuint64_t y, cuuint64_t y_stride, cuuint64_t z, cuuint64_t z_stride,
                   uint32_t box_y, uint32_t box_z) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {kD, y, z};
    cuuint64_t strides[2] = {2 * y_stride, 2 * z_stride};
    cuuint32_t box[3] = {64, box_y, box_z};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Of K or V: 128 tokens of a head, dimensions in the order of their strides.  A
// dimension of one entry has no stride, and heads with stride 0 are one.
bool make_kv_map(CUtensorMap *map, const CacheRows &x, int T, int H, bool *tokens_first, int *heads) {
    *heads = H > 1 && x.head != 0 ? 1 : 0;
    const cuuint64_t tok = T > 1 ? x.tok : kD, head = *heads ? x.head : kD, n = *heads ? H : 1;
    *tokens_first = tok < head;
    return tok < head ? make_rows_map(map, x.p, T, tok, n, head, kBlk, 1) : make_rows_map(map, x.p, n, head, T, tok, 1, kBlk);
}

// The limit of a wait for so many whole works, of T / 128 + 2 blocks each at most.
constexpr uint64_t work_limit(uint64_t limit_ns, int T, int works = 1) {
    const uint64_t blocks = works * (static_cast<uint64_t>(T) / kBlk + 2);
    return limit_ns > ~0ull / blocks ? ~0ull : limit_ns * blocks;
}
static_assert(work_limit(2000000000ull, 1000) == 18000000000ull && work_limit(2000000000ull, 1000, 3) == 54000000000ull &&
                  work_limit(1ull << 63, 256) == ~0ull && work_limit(~0ull, 1) == ~0ull && work_limit(0, 0x7fffffff) == 0,
              "a limit of any length");

// Query heads of a tile: a divisor of G (they share a KV head).  More heads mean
// fewer tokens, so fewer keys that only some rows see, and more of a short prompt's
// rows in a tile; but whole tokens may not fill the tile's 128 rows.  The
// least work by the average prompt's length is taken.
int heads_of(int G, int causal, double length) {
    int best = 1;
    double least = 0.0;
    for (int g = 1; g <= kBlk && g <= G; ++g) {
        if (G % g) continue;
        const double tokens = kBlk / g, work = kBlk / (g * tokens) * (1.0 + (causal ? 2.0 * tokens + kBlk : tokens) / length);
        if (g == 1 || work <= least) {
            best = g;
            least = work;
        }
    }
    return best;
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs &a, cudaStream_t st) {
    CUtensorMap mq, mk, mv;
    PromptParams p{};
    const int G = a.Hq / a.H;
    p.G = heads_of(G, a.causal, static_cast<double>(a.T) / a.B);
    p.tokens = kBlk / p.G;
    p.groups = a.Hq / p.G;
    p.per_head = G / p.G;
    if (!make_rows_map(&mq, a.q.p, a.Hq, a.Hq > 1 ? a.q.head : kD, a.T, a.T > 1 ? a.q.tok : kD, p.G, p.tokens) ||
        !make_kv_map(&mk, a.k, a.T, a.H, &p.k_tokens, &p.k_heads) || !make_kv_map(&mv, a.v, a.T, a.H, &p.v_tokens, &p.v_heads))
        return cudaErrorInvalidValue;
    p.start = a.start;
    p.B = a.B;
    p.T = a.T;
    p.Hq = a.Hq;
    p.causal = a.causal;
    CacheView heads{};
    heads.H = a.H;
    const AttnParams f = attn_params(heads, a.q, a.start, a.T, a.Hq, a.causal, a.scale, a.softcap, nullptr, 0);
    p.scale_log2 = f.scale_log2;
    p.cap_in = f.cap_in;
    p.cap_out = f.cap_out;
    p.prior = a.prior;
    p.prior_lse = a.prior_lse;
    p.O = a.O;
    p.lse = a.lse;
    p.dev_status = a.dev_status;
    p.limit_ns = a.wait_limit_ns;
    p.drain_ns = a.wait_limit_ns > 100000000u ? a.wait_limit_ns : 100000000u;
    p.work_limit_ns = work_limit(a.wait_limit_ns, a.T);
    p.works_limit_ns = work_limit(a.wait_limit_ns, a.T, kWorks);
    const bool few = a.T <= static_cast<int64_t>(a.causal ? 2 * kShortKeys : kShortKeys) * a.B;
    const auto kernel = a.softcap == 0.0f        ? (few ? prompt_kernel<0, true> : prompt_kernel<0, false>)
                        : a.softcap <= kSmallCap ? prompt_kernel<1, true>
                                                 : prompt_kernel<2, true>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = a.T / (2 * p.tokens) + (a.B <= kSortable && a.T < a.B ? a.T : a.B);
    p.items = tiles * p.groups;
    p.wide = (reinterpret_cast<uintptr_t>(a.O) & 31u) == 0;
    int device = 0, sms = 0;
    if ((e = cudaGetDevice(&device)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device)) != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(p.items < sms ? p.items : sms), kThreads, kSmem, st>>>(mq, mk, mv, p);
    return cudaGetLastError();
}

}  // namespace vca
