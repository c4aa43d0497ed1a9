// vca_cache.cuh -- what the kernels of the 8-bit cache share: the view of the
// cache, the place of a sequence's new rows, and the page scales.
//
// Cache: E4M3 codes [pages][H][128][128] with one fp32 scale per (page, head),
// a power of two; table[b][j] names the page of tokens 128 j .. 128 j + 127 of
// sequence b, len[b] counts its tokens, the current call's new ones included.
// Device-side values are never trusted: every index read from table, len or
// start is checked before it is used, and a bad one is reported in dev_status.
#pragma once

#include <cuda_fp16.h>

#include "vca_device.cuh"
#include "vca_internal.h"

namespace vca {
namespace cache {

constexpr int kErrInvalid = 1;       // mirrors VCA_ERR_INVALID_ARG
constexpr uint32_t kScaleExpMin = 127 - 120;   // biased exponent of the smallest page scale, 2^-120

__device__ __forceinline__ void report(int32_t *dev_status, int code) {
    if (dev_status) atomicExch(dev_status, code);
}

// Rows and length of sequence b: its new rows are [row0, row0 + n) of the T
// rows of the call, `len` its tokens.  bad: start or len out of range (the
// sequence then counts as having no new rows); falls: start is.
struct Seq {
    int row0, n, len;
    bool bad, falls;
};
__device__ __forceinline__ Seq load_seq(const CacheView &c, const int32_t *start, int T, int b) {
    Seq s;
    const int lo = start[b], hi = start[b + 1];
    s.len = c.len[b];
    s.falls = lo < 0 || hi < lo || hi > T;
    s.bad = s.falls || s.len < 0 || s.len > static_cast<int64_t>(c.cols) * kBlk;
    s.row0 = lo;
    s.n = s.bad ? 0 : hi - lo;
    return s;
}
// The sequences b0 .. b0 + 31, one per lane of a warp; returns whether more
// follow.  Lists of work end at the first sequence whose start falls: the
// rows of those before it are disjoint, so that no list outgrows T rows.
__device__ __forceinline__ bool load_seqs(const CacheView &c, const int32_t *start, int T, int b0, Seq &s) {
    const int lane = threadIdx.x & 31;
    s = Seq{0, 0, 0, false, false};
    if (b0 + lane < c.B) s = load_seq(c, start, T, b0 + lane);
    const uint32_t falls = __ballot_sync(0xffffffffu, s.falls);
    if (falls & ((1u << lane) - 1u)) {
        s.n = 0;
        s.bad = true;
    }
    return falls == 0 && b0 + 32 < c.B;
}

// Page of tokens 128 col .. 128 col + 127 of sequence b, or -1 (reported).
__device__ __forceinline__ int load_page(const CacheView &c, int b, int col, int32_t *dev_status) {
    const int page = c.table[static_cast<int64_t>(b) * c.cols + col];
    if (page < 0 || page >= c.pages) {
        report(dev_status, kErrInvalid);
        return -1;
    }
    return page;
}

// fp32 bits of the smallest power of two s >= 2^-120 with amax <= 448 s; `bits`
// are amax's (finite, >= 0).  448 = 1.75 * 2^8, so the exponent is the amax's
// less 8, or less 7 where its mantissa is above 1.75.
__device__ __forceinline__ uint32_t scale_bits(uint32_t bits) {
    const int e = static_cast<int>(bits >> 23) - ((bits & 0x7fffffu) > 0x600000u ? 7 : 8);
    return static_cast<uint32_t>(max(e, static_cast<int>(kScaleExpMin))) << 23;
}
// 1 / s of a power of two s in [2^-120, 2^120].
__device__ __forceinline__ float pow2_inverse(uint32_t sbits) { return __uint_as_float((254u << 23) - sbits); }

// Four E4M3 codes -> fp32 (exact).
__device__ __forceinline__ void e4m3x4_decode(uint32_t w, float (&f)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    f[0] = x.x;
    f[1] = x.y;
    f[2] = y.x;
    f[3] = y.y;
}

// Largest finite magnitude among eight bf16 values (as fp32 bits); `odd` is set
// where some are not finite.
__device__ __forceinline__ uint32_t amax_bf16x8(const uint4 &v, bool &odd) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t a = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    a = max(a & 0xffffu, a >> 16) << 16;
    if (a < 0x7f800000u) return a;
    odd = true;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = (w[i] & 0x7fffu) << 16, hi = w[i] & 0x7fff0000u;
        if (lo < 0x7f800000u) m = max(m, lo);
        if (hi < 0x7f800000u) m = max(m, hi);
    }
    return m;
}

// x * inv with what is not finite turned into NaN (E4M3 has no infinity, and
// a conversion that saturates would hide one).
__device__ __forceinline__ float scaled_or_nan(float x, float inv) {
    return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fc00000u) : __fmul_rn(x, inv);
}

// Largest of `v` over a block of kThreads threads, in every thread; `red` holds
// kThreads / 32 words.
template <int kThreads>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *red) {
    v = __reduce_max_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t m = red[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) m = max(m, red[i]);
    return m;
}

// What the kernels that score query rows against cached keys get.
struct AttnParams {
    CacheView c;
    CacheRows q;
    const int32_t *start;
    int T, Hq, G, causal;
    float scale_log2;      // softmax_scale log2(e)
    float cap_in;          // 2 log2(e) softmax_scale / cap: tanh(x) = 1 - 2 / (1 + 2^(2 log2(e) x))
    float cap_out;         // cap log2(e), 0: no cap
    uint16_t *O;
    float *lse;
    float *part;
    int whole;             // decode kernel: every CTA takes one whole tile
    int32_t *dev_status;
    uint64_t limit_ns;
};

inline AttnParams attn_params(const CacheView &c, const CacheRows &q, const int32_t *start, int T, int Hq, int causal,
                              float scale, float softcap, int32_t *dev_status, uint64_t limit_ns) {
    AttnParams p{};
    p.c = c;
    p.q = q;
    p.start = start;
    p.T = T;
    p.Hq = Hq;
    p.G = Hq / c.H;
    p.causal = causal;
    const double log2e = 1.4426950408889634;
    p.scale_log2 = static_cast<float>(scale * log2e);
    p.cap_in = softcap > 0.0f ? static_cast<float>(2.0 * log2e * scale / softcap) : 0.0f;
    p.cap_out = softcap > 0.0f ? static_cast<float>(softcap * log2e) : 0.0f;
    p.dev_status = dev_status;
    p.limit_ns = limit_ns;
    return p;
}

// Query row r of a (sequence, KV head) is token r / G of the sequence's new
// ones in query head h G + r % G.  It sees the keys [0, seen_by_row).
__device__ __forceinline__ int seen_by_row(const AttnParams &p, const Seq &s, int r) {
    return p.causal ? max(0, s.len - s.n + r / p.G + 1) : s.len;
}
__device__ __forceinline__ const uint16_t *query_row(const AttnParams &p, const Seq &s, int h, int r) {
    return p.q.p + (s.row0 + r / p.G) * p.q.tok + (h * p.G + r % p.G) * p.q.head;
}
// Place of the row among the outputs [T][Hq].
__device__ __forceinline__ int64_t out_row(const AttnParams &p, const Seq &s, int h, int r) {
    return static_cast<int64_t>(s.row0 + r / p.G) * p.Hq + h * p.G + r % p.G;
}

// A kernel that follows another of the same call may start while that one runs
// (launch_after) and waits here for its results; the first lets it start.
__device__ __forceinline__ void wait_for_results() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, Params(args)...);
}

// tanh(u ln 2 / 2) = 1 - 2 / (1 + 2^u), which cancels where u is small; below
// |u| = 1.6 an odd polynomial in u instead, of the least relative error (3.5e-8,
// weighted least squares with the weights raised where the error is largest),
// 7.7e-8 with its constants in fp32 and 2^-22 with its own roundings.
constexpr float kTanhNear = 1.6f;
constexpr float kT0 = 3.4657359e-01f, kT1 = -1.3875789e-02f, kT2 = 6.6592207e-04f, kT3 = -3.1559721e-05f, kT4 = 1.1715225e-06f;
__device__ __forceinline__ float tanh_half(float u) {
    const float w = u * u;
    const float q = fmaf(fmaf(fmaf(fmaf(kT4, w, kT3), w, kT2), w, kT1), w, kT0);
    const float far = 1.0f - __fdividef(2.0f, 1.0f + ex2_approx(fabsf(u)));
    return fabsf(u) <= kTanhNear ? u * q : copysignf(far, u);
}
// The capped score in log2 units, cap_out tanh.
__device__ __forceinline__ float capped(float u, float cap_out) { return cap_out * tanh_half(u); }

// 32 (16) columns of TMEM and, in `m`, the largest magnitude among them, NaN apart.
#define VCA_TMEM_LDTOP32(taddr, r, m)                                                                             \
    asm volatile(                                                                                                 \
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.abs.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"  \
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"                       \
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),         \
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),   \
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), \
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), \
          "=f"(m)                                                                                                 \
        : "r"(taddr))

#define VCA_TMEM_LDTOP16(taddr, r, m)                                                                             \
    asm volatile(                                                                                                 \
        "tcgen05.ld.red.sync.aligned.32x32b.x16.max.abs.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"  \
        "%15}, %16, [%17];"                                                                                       \
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),         \
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),   \
          "=f"(m)                                                                                                 \
        : "r"(taddr))

// X = cap_out tanh_half(X c) + add in place for kN raw scores of every lane of a
// warp; add(k): the terms of X[k], X[k + 1].  Scores are mostly well below the cap
// (`near`: |X| c <= kTanhNear in all lanes): then the polynomial alone, in
// pairs, without reciprocals and powers of two.
template <int kN, typename Add>
__device__ __forceinline__ void cap_scores(uint32_t (&X)[kN], float c, float cap_out, bool near, const Add &add) {
    if (!near) {
#pragma unroll
        for (int k = 0; k < kN; k += 2) {
            float a, b;
            upk2(add(k), a, b);
            X[k] = __float_as_uint(fmaf(tanh_half(__uint_as_float(X[k]) * c), cap_out, a));
            X[k + 1] = __float_as_uint(fmaf(tanh_half(__uint_as_float(X[k + 1]) * c), cap_out, b));
        }
        return;
    }
    auto both = [](float x) { return pk2(__float_as_uint(x), __float_as_uint(x)); };
    const uint64_t t0 = both(cap_out * kT0), t1 = both(cap_out * kT1), t2 = both(cap_out * kT2), t3 = both(cap_out * kT3),
                   t4 = both(cap_out * kT4);
#pragma unroll
    for (int k = 0; k < kN; k += 2) {
        const uint64_t u = mul2(pk2(X[k], X[k + 1]), both(c)), w = mul2(u, u);
        float a, b;
        upk2(fma2(u, fma2(fma2(fma2(fma2(t4, w, t3), w, t2), w, t1), w, t0), add(k)), a, b);
        X[k] = __float_as_uint(a);
        X[k + 1] = __float_as_uint(b);
    }
}

// Score in log2 units from the raw product: x = S * f with f = c (no cap) or
// the cap's inner factor.
__device__ __forceinline__ float scored(float s, float f, float cap_out) {
    const float x = __fmul_rn(s, f);
    return cap_out == 0.0f ? x : capped(x, cap_out);
}

}  // namespace cache
}  // namespace vca
