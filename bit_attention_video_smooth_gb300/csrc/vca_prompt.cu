// vca_prompt.cu -- attention of packed prompts over their own keys and values
// (bf16), bound by the tensor cores: 4 d flops for every visible pair.
//
// One CTA takes 256 query rows of a (sequence, KV head), two tiles of 128: rows
// i G + g, so that the G query heads that share the KV head share its keys and
// values, which pass through shared memory once for both tiles.  Per block of 128
// keys and tile: S = Q K^T (smem x smem -> TMEM), the softmax takes S to P in its
// place (bf16, the values' type, as the MMA wants it: 2^-9 relative a
// probability, while the row sums take the unrounded ones in fp32), O += P V (TMEM x
// smem).  While one tile's softmax runs the tensor core works for the other.
// Warps:
//   0      TMA producer: K and V blocks alternate in a ring of five
//   1      MMA issuer: PV of a block and QK of the next, tile by tile.  MMAs of one
//          thread and shape run in order, so QK may write the scores over the
//          probabilities that the PV before it reads.  The whole warp waits and one
//          thread of it, elected, issues: then the operands are in uniform registers,
//          and an MMA takes 10 to 20 cycles to issue (46 from a branch on the lane)
//   2      zeroes the rows of V behind the sequence's last token (they are another
//          sequence's, and may hold NaN) and only then reports that block as full
//   4-11   softmax, four warps a tile, a thread a row.  The reference maximum moves
//          only when a block's exceeds it by 8 (log2 units); O is rescaled in TMEM
//          then: S(j) full means that PV(j - 1) is done too
// Every wait is bounded, as in vca_attention.cu.
#include "vca_attention_common.cuh"
#include "vca_cache.cuh"

namespace vca {

namespace {

using namespace attn;
using namespace cache;

constexpr int kTiles = 2, kTileRows = kTiles * kBlk;
constexpr int kStages = 5, kSoftWarp0 = 4, kThreads = 32 * (kSoftWarp0 + 4 * kTiles);
constexpr uint32_t kPanel = kBlk * 128;              // 128 rows of 64 bf16 channels
constexpr uint32_t kBlock = 2 * kPanel;              // Q, K or V: two panels
constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemCols = 512;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffKV = kOffQ + kTiles * kBlock;
constexpr uint32_t kOffBar = kOffKV + kStages * kBlock;
constexpr int kNumBars = 2 * kStages + 5 * kTiles + 2;
constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
constexpr uint32_t kSmem = kOffMisc + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

struct PromptParams {
    CacheRows q;
    const int32_t *start;
    int B, T, Hq, H, G, causal;
    float scale_log2, cap_in, cap_out;      // as in AttnParams
    bool k_tokens, v_tokens;                // the tensor map's middle dimension: tokens, else heads
    int k_heads, v_heads;                   // 1, or 0: all heads are the same
    const uint16_t *prior;
    const float *prior_lse;
    uint16_t *O;
    float *lse;
    int32_t *dev_status;
    uint64_t limit_ns;
};

__device__ __forceinline__ void tma_load_3d(void *smem_dst, const void *tmap, uint64_t *bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r != 0;
}

// ---------------------------------------------------------------------------
// Which tile a CTA takes
// ---------------------------------------------------------------------------
// Rows [row0, row0 + n) of a sequence, and which 256 of its n G.
struct Work {
    int row0, n, tile;
};
__device__ __forceinline__ int tiles_of(int n, int G) {
    return static_cast<int>((static_cast<int64_t>(n) * G + kTileRows - 1) / kTileRows);
}

// Up to kSortable sequences: the tiles by their number of key blocks, most first,
// so that the last wave's are short.  A causal tile's number grows with its
// place in the sequence, another's is the sequence's.  F(c) tiles have a cost
// above c; a warp evaluates it over sequences that it holds in registers.
constexpr int kHeld = 8, kSortable = 32 * kHeld;
__device__ bool find_sorted(const PromptParams &p, int rank, Work &w) {
    const int lane = threadIdx.x & 31;
    int q[kHeld], lo[kHeld], hi[kHeld], most = 0;
    bool fell = false;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        const int b = 32 * k + lane;
        lo[k] = hi[k] = 0;
        if (b < p.B) {
            lo[k] = p.start[b];
            hi[k] = p.start[b + 1];
        }
    }
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        const uint32_t falls = __ballot_sync(0xffffffffu, lo[k] < 0 || hi[k] < lo[k] || hi[k] > p.T);
        if (fell || (falls & ((2u << lane) - 1u))) hi[k] = lo[k];
        fell = fell || falls != 0;
        q[k] = tiles_of(hi[k] - lo[k], p.G);
        most = max(most, q[k]);
    }
    if (rank == 0 && blockIdx.x == 0 && lane == 0 && fell) report(p.dev_status, kErrInvalid);
    most = __reduce_max_sync(0xffffffffu, most);
    auto above = [&](int c) {
        int f = 0;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) f += p.causal ? max(0, q[k] - c) : q[k] > c ? q[k] : 0;
        return static_cast<int>(__reduce_add_sync(0xffffffffu, f));
    };
    if (above(0) <= rank) return false;
    int a = 0, z = most;      // F(a) > rank >= F(z)
    while (z - a > 1) {
        const int mid = a + (z - a) / 2;
        if (above(mid) > rank)
            a = mid;
        else
            z = mid;
    }
    int left = rank - above(z);      // among the tiles of cost a, in the sequences' order
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        const int has = p.causal ? (q[k] > a) : q[k] == a + 1 ? q[k] : 0;
        int incl = has;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, left < incl);
        if (hit) {
            const int l = __ffs(hit) - 1;
            w.row0 = __shfl_sync(0xffffffffu, lo[k], l);
            w.n = __shfl_sync(0xffffffffu, hi[k], l) - w.row0;
            w.tile = p.causal ? a : left - __shfl_sync(0xffffffffu, incl - has, l);
            return true;
        }
        left -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}

// More sequences: sequence b's tiles are those from floor(start G / 256) + b on, which
// leaves room for each sequence's and is found by search.  All threads; first checks
// that start rises up to there, since nothing behind a fall has rows.
__device__ bool find_searched(const PromptParams &p, int index, int *first_fall, Work &w) {
    if (threadIdx.x == 0) *first_fall = p.B;
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const int lo = p.start[b], hi = p.start[b + 1];
        if (lo < 0 || hi < lo || hi > p.T) atomicMin(first_fall, b);
    }
    __syncthreads();
    const int rise = *first_fall;      // sequences 0 .. rise - 1 are right
    if (index == 0 && blockIdx.x == 0 && threadIdx.x == 0 && rise < p.B) report(p.dev_status, kErrInvalid);
    auto base = [&](int b) { return static_cast<int64_t>(p.start[b]) * p.G / kTileRows + b; };
    if (rise == 0 || base(0) > index) return false;
    int a = 0, z = rise;      // base(a) <= index < base(z), or z = rise
    while (z - a > 1) {
        const int mid = a + (z - a) / 2;
        if (base(mid) <= index)
            a = mid;
        else
            z = mid;
    }
    w.row0 = p.start[a];
    w.n = p.start[a + 1] - w.row0;
    w.tile = static_cast<int>(index - base(a));
    return w.tile < tiles_of(w.n, p.G);
}

// ---------------------------------------------------------------------------
// Softmax pieces
// ---------------------------------------------------------------------------
struct BlockScore {
    float c, bias;       // no cap: p = 2^(S c + bias); cap: p = 2^(cap tanh_half(S c) + bias)
    float cap;
    bool near;           // the polynomial of the cap's tanh will do for the warp
    int lim;             // columns of the block that the row sees
    bool edge;           // some row of the warp does not see all
};

// 32 raw scores -> words of bf16 pairs; the unrounded probabilities add to l2.
template <bool kCap>
__device__ __forceinline__ void probabilities(uint32_t (&X)[32], const BlockScore &s, int col0, uint64_t &l2,
                                              uint32_t *W) {
    const uint64_t c2 = pk2(__float_as_uint(s.c), __float_as_uint(s.c));
    const uint64_t b2 = pk2(__float_as_uint(s.bias), __float_as_uint(s.bias));
    if constexpr (kCap) cap_scores(X, s.c, s.cap, s.near, [&](int) { return b2; });
#pragma unroll
    for (int k = 0; k < 16; ++k) {
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
        W[k] = pack_bf16x2(a, b);
    }
}

// Scores of keys that the row does not see become -inf (0 where a cap follows);
// returns the largest of the others.
template <bool kCap>
__device__ __forceinline__ float mask_scores(uint32_t (&X)[32], int col0, int lim) {
    float m = __int_as_float(0xff800000);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        if (col0 + e < lim) m = fmaxf(m, __uint_as_float(X[e]));
        else X[e] = kCap ? 0u : 0xff800000u;
    }
    return m;
}

template <bool kCap>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const PromptParams p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem =
        reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBar), *empty = full + kStages;
    uint64_t *q_full = empty + kStages, *s_full = q_full + kTiles, *p_full = s_full + kTiles, *o_full = p_full + 2 * kTiles;
    uint64_t *raw = o_full + kTiles, *drain = raw + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffMisc);
    int *abort_flag = reinterpret_cast<int *>(smem + kOffMisc + 4);
    int *first_fall = reinterpret_cast<int *>(smem + kOffMisc + 8);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x / p.H), h = static_cast<int>(blockIdx.x % p.H);
    Work w;
    // every warp finds the CTA's tile for itself
    if (!(p.B <= kSortable ? find_sorted(p, rank, w) : find_searched(p, rank, first_fall, w))) return;

    const int R = w.n * p.G, r0 = w.tile * kTileRows;
    // key blocks that each tile's rows see; none: the tile has no rows
    auto blocks_of = [&](int t) {
        if (r0 + t * kBlk >= R) return 0;
        const int last = min(R, r0 + (t + 1) * kBlk) - 1;
        return ((p.causal ? last / p.G + 1 : w.n) + kBlk - 1) / kBlk;
    };
    const int nb0 = blocks_of(0), nb1 = blocks_of(1), nbs = max(nb0, nb1);
    const int tail = w.n % kBlk && nbs == (w.n + kBlk - 1) / kBlk ? nbs - 1 : -1;      // the block that ends behind the sequence

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(q_full + t, 4);
            mbar_init(s_full + t, 1);
            mbar_init(p_full + 2 * t, 4);
            mbar_init(p_full + 2 * t + 1, 4);
            mbar_init(o_full + t, 1);
        }
        mbar_init(raw, 1);
        mbar_init(drain, 1);
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

    // registers: 128 x 80 + 256 x 208 of the 384 x 168 at launch
    if (warp < kSoftWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == 0) {
            // -------------------------------------------------------- producer
            if (lane == 0) {
                bool ok = true;
                int i = 0;
                for (; i < 2 * nbs; ++i) {      // K(0), V(0), K(1), V(1), ...
                    const int st = i % kStages;
                    if (i >= kStages) ok = mbar_wait(empty + st, (i / kStages - 1) & 1, abort_flag, p.limit_ns);
                    if (!ok) break;
                    const void *map = i & 1 ? &tmV : &tmK;
                    const int token = w.row0 + (i >> 1) * kBlk, head = h * (i & 1 ? p.v_heads : p.k_heads);
                    const bool tokens = i & 1 ? p.v_tokens : p.k_tokens;
                    unsigned char *to = smem + kOffKV + st * kBlock;
                    uint64_t *landed = i == 2 * tail + 1 ? raw : full + st;
                    mbar_expect_tx(landed, kBlock);
                    for (int c = 0; c < 2; ++c)
                        tma_load_3d(to + c * kPanel, map, landed, 64 * c, tokens ? token : head, tokens ? head : token);
                }
                // every copy issued has landed before the CTA can exit
                for (int j = max(0, i - kStages); j < i; ++j) {
                    if (j == 2 * tail + 1)
                        drain_wait(raw, 0, p.limit_ns);
                    else
                        drain_wait(full + j % kStages, (j / kStages) & 1, p.limit_ns);
                }
            }
        } else if (warp == 1) {
            // -------------------------------------------------------- MMA issuer
            constexpr uint32_t idesc_qk = make_idesc(128, 128, 1, 1), idesc_pv = make_idesc(128, 128, 1, 1, 0, 1);
            const uint32_t base = smem_u32(smem);
            const bool one = elect_one();
            auto wait = [&](uint64_t *bar, int parity) {
                const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.limit_ns));
                tc_fence_after();
                return ok;
            };
            auto qk = [&](int t, int st) {
                const uint64_t dq = sdesc_k_sw128(base + kOffQ + t * kBlock), dk = sdesc_k_sw128(base + kOffKV + st * kBlock);
                if (one) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t step = (i >> 2) * (kPanel >> 4) + 2 * (i & 3);
                        mma_f16(tmem + kTmemS + 128 * t, dq + step, dk + step, idesc_qk, i > 0);
                    }
                    tc_commit(s_full + t);
                }
            };
            auto pv = [&](int t, int st, int half, bool first) {      // of 64 keys
                const uint64_t dv = sdesc_mn_sw128(base + kOffKV + st * kBlock, kPanel);
                if (one) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_f16_ts(tmem + kTmemO + 128 * t, tmem + kTmemS + 128 * t + 32 * half + 8 * i,
                                   dv + (2048 >> 4) * (4 * half + i), idesc_pv, !first || i > 0);
                }
            };
            auto commit = [&](uint64_t *bar) {
                if (one) tc_commit(bar);
            };
            bool ok = wait(full, 0);
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                if (!ok || (t == 1 && nb1 == 0)) break;
                ok = wait(q_full + t, 0);
                if (ok) qk(t, 0);
            }
            commit(empty);
            for (int j = 0; ok && j < nbs; ++j) {
                const int iv = 2 * j + 1, ik = 2 * j + 2, sv = iv % kStages, sk = ik % kStages;
                ok = wait(full + sv, (iv / kStages) & 1);
                if (ok && j + 1 < nbs) ok = wait(full + sk, (ik / kStages) & 1);
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    const int last = t ? nb1 : nb0;
                    if (!ok || j >= last) continue;
                    ok = wait(p_full + 2 * t, j & 1);
                    if (!ok) break;
                    pv(t, sv, 0, j == 0);
                    ok = wait(p_full + 2 * t + 1, j & 1);
                    if (!ok) break;
                    pv(t, sv, 1, false);
                    if (t == 1 || j >= nb1) commit(empty + sv);
                    if (j + 1 < last)
                        qk(t, sk);
                    else
                        commit(o_full + t);
                }
                if (ok && j + 1 < nbs) commit(empty + sk);
            }
            commit(drain);
            if (one) drain_wait(drain, 0, p.limit_ns);
            __syncwarp();
        } else if (warp == 2 && tail >= 0) {
            // -------------------------------------------------------- rows of V behind the sequence
            const int st = (2 * tail + 1) % kStages, live = w.n - tail * kBlk;
            if (__all_sync(0xffffffffu, mbar_wait(raw, 0, abort_flag, p.limit_ns))) {
                uint4 *to = reinterpret_cast<uint4 *>(smem + kOffKV + st * kBlock);
                for (int e = 8 * live + lane; e < 8 * kBlk; e += 32) to[e] = to[e + kPanel / 16] = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + st);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = (warp - kSoftWarp0) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const int n_blocks = t ? nb1 : nb0, rt = r0 + t * kBlk;
        unsigned char *sQ = smem + kOffQ + t * kBlock;
        if (n_blocks > 0) {
            // the warp's rows of Q, half a warp a row
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
                const int mine = quarter * 32 + 2 * i + (lane >> 4), r = rt + mine, c = lane & 15;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < R)
                    v = reinterpret_cast<const uint4 *>(p.q.p + (w.row0 + r / p.G) * p.q.tok + (h * p.G + r % p.G) * p.q.head)[c];
                *reinterpret_cast<uint4 *>(sQ + (c >> 3) * kPanel + sw128_offset(mine, c & 7)) = v;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full + t);

            const float kNegInf = __int_as_float(0xff800000);
            const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16), tS = tl + kTmemS + 128 * t,
                           tO = tl + kTmemO + 128 * t;
            const int r = rt + row;
            const bool real = r < R;
            const int seen = real && p.causal ? r / p.G + 1 : w.n;
            const int whole = __reduce_min_sync(0xffffffffu, seen) / kBlk;      // blocks that every row of the warp sees all of
            BlockScore s;
            s.c = fmaxf(kCap ? p.cap_in : p.scale_log2, 0x1p-149f);
            s.cap = p.cap_out;
            s.bias = 0.0f;
            float m = kNegInf;
            uint64_t l2 = 0;
            bool ok = true;
            for (int b = 0; b < n_blocks; ++b) {
                ok = __all_sync(0xffffffffu, mbar_wait(s_full + t, b & 1, abort_flag, p.limit_ns));
                if (!ok) break;
                tc_fence_after();
                uint32_t X[4][32];
                float mx[4];
                s.edge = b >= whole;
                if constexpr (kCap) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) VCA_TMEM_LDTOP32(tS + 32 * i, X[i], mx[i]);
                    tmem_ld_wait();
                    s.near = __all_sync(0xffffffffu, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * s.c <= kTanhNear);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) VCA_TMEM_LDMAX32(tS + 32 * i, X[i], mx[i]);
                tmem_ld_wait();
                if (s.edge) {
                    s.lim = seen - b * kBlk;
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx[i] = mask_scores<kCap>(X[i], 32 * i, s.lim);
                }
                const float pm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * s.c;
                const float bm = kCap ? capped(pm, p.cap_out) : pm;
                if (__any_sync(0xffffffffu, bm > __fadd_rn(m, kLazyTau))) {
                    float alpha = 1.0f;
                    if (bm > __fadd_rn(m, kLazyTau)) {
                        alpha = ex2_approx(__fsub_rn(m, bm));
                        l2 = mul2(l2, pk2(__float_as_uint(alpha), __float_as_uint(alpha)));
                        m = bm;
                        s.bias = -m;
                    }
                    if (b > 0) {
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {
                            uint32_t o[16];
                            asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                                         : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]),
                                           "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
                                         : "r"(tO + 16 * i));
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), alpha));
                            VCA_TMEM_ST16(tO + 16 * i, o);
                        }
                    }
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int i = 2 * half; i < 2 * half + 2; ++i) {
                        uint32_t W[16];
                        probabilities<kCap>(X[i], s, 32 * i, l2, W);
                        VCA_TMEM_ST16(tS + 16 * i, W);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + 2 * t + half);
                }
            }
            // -------------------------------------------------------- epilogue
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait(o_full + t, 0, abort_flag, p.limit_ns));
            if (ok) {
                tc_fence_after();
                float l;
                {
                    float a, c;
                    upk2(l2, a, c);
                    l = __fadd_rn(a, c);
                }
                const int64_t at = static_cast<int64_t>(w.row0 + r / p.G) * p.Hq + h * p.G + r % p.G;
                // joined with what came before: both sums to the larger maximum
                float before = kNegInf, keep = 1.0f, add = 0.0f;
                if (p.prior && real) before = p.prior_lse[at] * 1.4426950408889634f;
                float M = m;
                if (before != kNegInf) {
                    M = m == kNegInf ? before : before != before ? before : fmaxf(m, before);
                    keep = m == kNegInf ? 0.0f : ex2_approx(__fsub_rn(m, M));
                    add = ex2_approx(__fsub_rn(before, M));
                    l = __fadd_rn(__fmul_rn(l, keep), add);
                }
                const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
                keep *= inv;
                add *= inv;
                const bool joins = before != kNegInf;
                const uint4 *prior = reinterpret_cast<const uint4 *>(p.prior + at * kD);
                // Q's place is free: rows of O through shared memory, half a warp a row to memory
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    uint32_t o[32];
                    VCA_TMEM_LD32(tO + 32 * i, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), keep));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (joins) {
                            const uint4 x = prior[4 * i + e];
                            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                o[8 * e + 2 * k] = __float_as_uint(fmaf(__uint_as_float(xs[k] << 16), add, __uint_as_float(o[8 * e + 2 * k])));
                                o[8 * e + 2 * k + 1] =
                                    __float_as_uint(fmaf(__uint_as_float(xs[k] & 0xffff0000u), add, __uint_as_float(o[8 * e + 2 * k + 1])));
                            }
                        }
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            y[k] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * k]), __uint_as_float(o[8 * e + 2 * k + 1]));
                        *reinterpret_cast<uint4 *>(sQ + row * 256 + (((4 * i + e) ^ (row & 15)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                if (p.lse && real) p.lse[at] = (M == kNegInf ? 0.0f : M) * 0.6931471805599453f + logf(l);
                __syncwarp();
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    const int mine = quarter * 32 + 2 * i + (lane >> 4), ri = rt + mine, c = lane & 15;
                    if (ri < R) {
                        const int64_t to = static_cast<int64_t>(w.row0 + ri / p.G) * p.Hq + h * p.G + ri % p.G;
                        reinterpret_cast<uint4 *>(p.O + to * kD)[c] =
                            *reinterpret_cast<const uint4 *>(sQ + mine * 256 + ((c ^ (mine & 15)) << 4));
                    }
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

// bf16 rows [T][heads][128] as a 3-D matrix, its dimensions in the order of their
// strides.  A dimension of one entry has no stride, and heads with stride 0 are one.
bool make_rows_map(CUtensorMap *map, const CacheRows &x, int T, int H, bool *tokens_first, int *heads) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    *heads = H > 1 && x.head != 0 ? 1 : 0;
    const cuuint64_t entries[2] = {static_cast<cuuint64_t>(T), *heads ? static_cast<cuuint64_t>(H) : 1u};
    const cuuint64_t bytes[2] = {T > 1 ? static_cast<cuuint64_t>(x.tok) * 2 : 2u * kD, *heads ? static_cast<cuuint64_t>(x.head) * 2 : 2u * kD};
    const int mid = bytes[0] < bytes[1] ? 0 : 1;
    *tokens_first = mid == 0;
    cuuint64_t dims[3] = {kD, entries[mid], entries[1 - mid]};
    cuuint64_t strides[2] = {bytes[mid], bytes[1 - mid]};
    cuuint32_t box[3] = {64, mid == 0 ? 128u : 1u, mid == 0 ? 1u : 128u};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(x.p), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs &a, cudaStream_t st) {
    CUtensorMap mk, mv;
    PromptParams p{};
    if (!make_rows_map(&mk, a.k, a.T, a.H, &p.k_tokens, &p.k_heads) || !make_rows_map(&mv, a.v, a.T, a.H, &p.v_tokens, &p.v_heads))
        return cudaErrorInvalidValue;
    p.q = a.q;
    p.start = a.start;
    p.B = a.B;
    p.T = a.T;
    p.Hq = a.Hq;
    p.H = a.H;
    p.G = a.Hq / a.H;
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
    const auto kernel = a.softcap > 0.0f ? prompt_kernel<true> : prompt_kernel<false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = static_cast<int64_t>(a.T) * p.G / kTileRows + (a.B <= kSortable && a.T < a.B ? a.T : a.B);
    kernel<<<static_cast<unsigned>(tiles * a.H), kThreads, kSmem, st>>>(mk, mv, p);
    return cudaGetLastError();
}

}  // namespace vca
