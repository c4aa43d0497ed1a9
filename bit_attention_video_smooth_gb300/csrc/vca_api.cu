// vca_api.cu -- the C ABI declared in include/vca.h: argument validation,
// workspace sizing and kernel launches.  No device memory is allocated here.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/vca.h"
#include "vca_internal.h"

namespace {

uint64_t g_wait_limit_ns = 2000000000ull;   // 2 s

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool shape_ok(int B, int H, int N, int d) {
    if (B < 1 || H < 1 || N < 128 || d != 128 || (N % 128) != 0) return false;
    const int64_t BH = static_cast<int64_t>(B) * H;
    return BH <= 65535 && BH * N <= (static_cast<int64_t>(1) << 31) - 1;   // BH is a grid y extent
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The cache's sizes and pointers; `view` gets them in the kernels' form.
bool cache_ok(const vca_cache *c, vca::CacheView *view) {
    const int64_t most = (static_cast<int64_t>(1) << 31) - 1;
    if (!c || c->d != 128 || c->pages < 1 || c->H < 1 || c->B < 1 || c->cols < 1) return false;
    if (static_cast<int64_t>(c->B) * c->H > 65535 || static_cast<int64_t>(c->cols) * 128 > most) return false;
    if (static_cast<int64_t>(c->pages) * c->H > most / 128) return false;
    if (!c->k8 || !c->v8 || !aligned16(c->k8) || !aligned16(c->v8)) return false;
    const void *ptrs[] = {c->sk, c->sv, c->table, c->len};
    for (const void *p : ptrs)
        if (!p || !aligned4(p)) return false;
    *view = vca::CacheView{c->k8, c->v8, c->sk, c->sv, c->table, c->len, c->pages, c->H, c->B, c->cols};
    return true;
}
bool rows_ok(const uint16_t *p, int64_t tok, int64_t head) {
    return p && aligned16(p) && (tok & 7) == 0 && (head & 7) == 0;
}
bool query_sizes_ok(int T, int Hq, int H) {
    return T >= 0 && Hq >= 1 && H >= 1 && Hq % H == 0 && static_cast<int64_t>(T) * Hq <= (static_cast<int64_t>(1) << 31) - 1;
}
float scale_or_default(float softmax_scale) {
    return softmax_scale > 0.0f ? softmax_scale : static_cast<float>(1.0 / std::sqrt(128.0));
}
// The kernels scale by softmax_scale, softmax_scale / softcap and softcap, times 2 log2(e): a factor 4 to fp32's largest.
bool scores_ok(int causal, float softmax_scale, float softcap) {
    if ((causal != 0 && causal != 1) || !std::isfinite(softmax_scale) || !std::isfinite(softcap) || softcap < 0.0f) return false;
    const double most = 8.5e37, scale = scale_or_default(softmax_scale);
    return scale < most && (softcap == 0.0f || (softcap < most && scale / softcap < most));
}
// The cap that the kernels get.  softcap tanh(s / softcap) is s to (s / softcap)^2 / 3:
// from 2^40 on, to less than an fp32 rounding for scores below 2^28, and 0 (no cap)
// it is.  Below 2^-40 all scores are 0 to 2^-40, as they are with a cap of 2^-40.
// In between softmax_scale / softcap times a page scale above 2^-80 is a normal number.
float cap_used(float softcap) { return softcap >= 0x1p40f ? 0.0f : softcap > 0.0f ? std::fmax(softcap, 0x1p-40f) : 0.0f; }

int from_cuda(cudaError_t e) { return e == cudaSuccess ? VCA_OK : VCA_ERR_CUDA; }

}  // namespace

extern "C" {

const char *vca_status_string(int status) {
    switch (status) {
        case VCA_OK: return "ok";
        case VCA_ERR_INVALID_ARG: return "invalid argument";
        case VCA_ERR_UNSUPPORTED: return "unsupported combination";
        case VCA_ERR_CUDA: return "CUDA error";
        case VCA_ERR_TIMEOUT: return "device wait timed out";
        case VCA_ERR_WORKSPACE: return "workspace missing or too small";
        default: return "unknown status";
    }
}

int vca_version(void) { return 100; }

size_t vca_workspace_bytes(int op, int B, int H, int N, int d, int k, int vmode) {
    if (!shape_ok(B, H, N, d)) return 0;
    const int BH = B * H;
    switch (op) {
        case VCA_OP_GROUP:
            if (k < 1 || k > vca::kMaxK || k > N) return 0;
            return vca::group_workspace_layout(BH, N, k).bytes;
        case VCA_OP_PREP:
        case VCA_OP_PREP_KSMOOTH:
            if (vmode != VCA_V_E4M3 && vmode != VCA_V_NVFP4) return 0;
            return vca::prep_workspace_layout(BH, N, op == VCA_OP_PREP_KSMOOTH ? vca::kPrepKSmooth : 0u).bytes;
        default:
            return 0;
    }
}

int vca_group(const uint16_t *V, int B, int H, int N, int d, int k, int iters, int32_t *labels, int32_t *perm,
              int32_t *counts, float *centroids, void *ws, size_t ws_bytes, int32_t *dev_status, void *stream) {
    if (!shape_ok(B, H, N, d) || k < 1 || k > vca::kMaxK || k > N || iters < 1 || iters > 1000) return VCA_ERR_INVALID_ARG;
    if (!V || !labels || !perm || !aligned16(V) || !aligned16(labels) || !aligned16(perm)) return VCA_ERR_INVALID_ARG;
    if ((counts && !aligned16(counts)) || (centroids && !aligned16(centroids))) return VCA_ERR_INVALID_ARG;
    if (dev_status && (reinterpret_cast<uintptr_t>(dev_status) & 3u)) return VCA_ERR_INVALID_ARG;
    const size_t need = vca_workspace_bytes(VCA_OP_GROUP, B, H, N, d, k, 0);
    if (!ws || ws_bytes < need || !aligned16(ws)) return VCA_ERR_WORKSPACE;
    return from_cuda(vca::launch_group(V, B * H, N, k, iters, labels, perm, counts, centroids, ws, dev_status,
                                       g_wait_limit_ns, static_cast<cudaStream_t>(stream)));
}

int vca_prep_quant(const uint16_t *Q, const uint16_t *K, const uint16_t *V, const int32_t *perm, int B, int H, int N,
                   int d, int vmode, uint8_t *q8, float *sq, uint8_t *k8, float *sk, uint8_t *v_res, uint8_t *v_sf,
                   float *v_scale, uint16_t *v_mean, void *ws, size_t ws_bytes, void *stream) {
    return vca_prep_quant_ex(Q, K, V, perm, B, H, N, d, vmode, 0u, q8, sq, k8, sk, v_res, v_sf, v_scale, v_mean, ws,
                             ws_bytes, stream);
}

int vca_prep_quant_ex(const uint16_t *Q, const uint16_t *K, const uint16_t *V, const int32_t *perm, int B, int H,
                      int N, int d, int vmode, uint32_t flags, uint8_t *q8, float *sq, uint8_t *k8, float *sk,
                      uint8_t *v_res, uint8_t *v_sf, float *v_scale, uint16_t *v_mean, void *ws, size_t ws_bytes,
                      void *stream) {
    if (!shape_ok(B, H, N, d) || (vmode != VCA_V_E4M3 && vmode != VCA_V_NVFP4)) return VCA_ERR_INVALID_ARG;
    if (flags & ~(VCA_PREP_QK_HADAMARD | VCA_PREP_K_SMOOTH)) return VCA_ERR_INVALID_ARG;
    const void *ptrs[] = {Q, K, V, perm, q8, sq, k8, sk, v_res, v_scale, v_mean};
    for (const void *p : ptrs)
        if (!p || !aligned16(p)) return VCA_ERR_INVALID_ARG;
    if (vmode == VCA_V_NVFP4 && (!v_sf || !aligned16(v_sf))) return VCA_ERR_INVALID_ARG;
    const size_t need = vca_workspace_bytes((flags & VCA_PREP_K_SMOOTH) ? VCA_OP_PREP_KSMOOTH : VCA_OP_PREP, B, H, N, d, 1,
                                            vmode);
    if (!ws || ws_bytes < need || !aligned16(ws)) return VCA_ERR_WORKSPACE;
    return from_cuda(vca::launch_prep(Q, K, V, perm, B * H, N, vmode, flags, q8, sq, k8, sk, v_res, v_sf, v_scale,
                                      v_mean, ws, static_cast<cudaStream_t>(stream)));
}

int vca_attention(const uint8_t *q8, const float *sq, const uint8_t *k8, const float *sk, const uint8_t *v_res,
                  const uint8_t *v_sf, const float *v_scale, const uint16_t *v_mean, int B, int H, int N, int d,
                  float softmax_scale, int expcast, int vmode, uint16_t *O, int32_t *dev_status, void *stream) {
    if (!shape_ok(B, H, N, d) || (vmode != VCA_V_E4M3 && vmode != VCA_V_NVFP4) || (expcast != 0 && expcast != 1))
        return VCA_ERR_INVALID_ARG;
    if (!std::isfinite(softmax_scale)) return VCA_ERR_INVALID_ARG;
    const void *ptrs[] = {q8, sq, k8, sk, v_res, v_scale, v_mean, O};
    for (const void *p : ptrs)
        if (!p || !aligned16(p)) return VCA_ERR_INVALID_ARG;
    if (dev_status && (reinterpret_cast<uintptr_t>(dev_status) & 3u)) return VCA_ERR_INVALID_ARG;
    if (vmode == VCA_V_NVFP4) {
        if (expcast) return VCA_ERR_UNSUPPORTED;   // no single affine log -> E2M1 code map
        if (!v_sf || !aligned16(v_sf)) return VCA_ERR_INVALID_ARG;
    }
    if (softmax_scale <= 0.0f) softmax_scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    vca::AttentionArgs a;
    a.q8 = q8;
    a.k8 = k8;
    a.v_res = v_res;
    a.v_sf = v_sf;
    a.sq = sq;
    a.sk = sk;
    a.v_scale = v_scale;
    a.v_mean = v_mean;
    a.O = O;
    a.dev_status = dev_status;
    a.BH = B * H;
    a.N = N;
    a.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
    a.expcast = expcast;
    a.vmode = vmode;
    a.wait_limit_ns = g_wait_limit_ns;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return from_cuda(vmode == VCA_V_NVFP4 ? vca::launch_attention_nvfp4(a, st) : vca::launch_attention(a, st));
}

size_t vca_cache_workspace_bytes(int op, int T, int Hq, int H, int B, int cols) {
    if (!query_sizes_ok(T, Hq, H) || T < 1 || B < 1 || cols < 1 || static_cast<int64_t>(B) * H > 65535 ||
        static_cast<int64_t>(cols) * 128 > (static_cast<int64_t>(1) << 31) - 1)
        return 0;
    switch (op) {
        case VCA_OP_CACHE_ATTENTION: return vca::cache_attention_workspace(T, Hq, H, B, cols);
        case VCA_OP_CACHE_WEIGH: return vca::cache_weigh_workspace(T, Hq, H, B, cols);
        default: return 0;
    }
}

int vca_cache_append(const vca_cache *cache, const uint16_t *K, int64_t k_token, int64_t k_head, const uint16_t *V,
                     int64_t v_token, int64_t v_head, const int32_t *start, int T, int32_t *dev_status, void *stream) {
    return vca_cache_append_ex(cache, K, k_token, k_head, V, v_token, v_head, start, T, nullptr, dev_status, stream);
}

int vca_cache_append_ex(const vca_cache *cache, const uint16_t *K, int64_t k_token, int64_t k_head, const uint16_t *V,
                        int64_t v_token, int64_t v_head, const int32_t *start, int T, float *weight, int32_t *dev_status,
                        void *stream) {
    vca::CacheView c;
    if (!cache_ok(cache, &c) || T < 0 || !start || !aligned4(start) || !aligned16(weight) || !aligned4(dev_status))
        return VCA_ERR_INVALID_ARG;
    if (T == 0) return VCA_OK;
    if (!rows_ok(K, k_token, k_head) || !rows_ok(V, v_token, v_head)) return VCA_ERR_INVALID_ARG;
    return from_cuda(vca::launch_cache_append(c, vca::CacheRows{K, k_token, k_head}, vca::CacheRows{V, v_token, v_head},
                                              start, T, weight, dev_status, static_cast<cudaStream_t>(stream)));
}

int vca_cache_attention(const vca_cache *cache, const uint16_t *Q, int64_t q_token, int64_t q_head,
                        const int32_t *start, int T, int Hq, int causal, float softmax_scale, float softcap,
                        uint16_t *O, float *lse, void *ws, size_t ws_bytes, int32_t *dev_status, void *stream) {
    vca::CacheView c;
    if (!cache_ok(cache, &c) || !query_sizes_ok(T, Hq, c.H) || !scores_ok(causal, softmax_scale, softcap))
        return VCA_ERR_INVALID_ARG;
    if (!start || !aligned4(start) || !aligned4(lse) || !aligned4(dev_status)) return VCA_ERR_INVALID_ARG;
    if (T == 0) return VCA_OK;
    if (!rows_ok(Q, q_token, q_head) || !O || !aligned16(O)) return VCA_ERR_INVALID_ARG;
    const size_t need = vca::cache_attention_workspace(T, Hq, c.H, c.B, c.cols);
    if (need && (!ws || ws_bytes < need || !aligned16(ws))) return VCA_ERR_WORKSPACE;
    vca::CacheAttnArgs a{c, vca::CacheRows{Q, q_token, q_head}, start, T, Hq, causal, scale_or_default(softmax_scale),
                         cap_used(softcap), O, lse, ws, dev_status, g_wait_limit_ns};
    return from_cuda(vca::launch_cache_attention(a, static_cast<cudaStream_t>(stream)));
}

int vca_cache_weigh(const vca_cache *cache, const uint16_t *Q, int64_t q_token, int64_t q_head, const int32_t *start,
                    int T, int Hq, int causal, float softmax_scale, float softcap, const float *lse, float *weight,
                    void *ws, size_t ws_bytes, int32_t *dev_status, void *stream) {
    vca::CacheView c;
    if (!cache_ok(cache, &c) || !query_sizes_ok(T, Hq, c.H) || !scores_ok(causal, softmax_scale, softcap))
        return VCA_ERR_INVALID_ARG;
    if (!start || !aligned4(start) || !aligned4(dev_status)) return VCA_ERR_INVALID_ARG;
    if (T == 0) return VCA_OK;
    if (!rows_ok(Q, q_token, q_head) || !lse || !aligned4(lse) || !weight || !aligned16(weight)) return VCA_ERR_INVALID_ARG;
    const size_t need = vca::cache_weigh_workspace(T, Hq, c.H, c.B, c.cols);
    if (need && (!ws || ws_bytes < need || !aligned16(ws))) return VCA_ERR_WORKSPACE;
    vca::CacheWeighArgs a{c, vca::CacheRows{Q, q_token, q_head}, start, T, Hq, causal, scale_or_default(softmax_scale),
                          cap_used(softcap), lse, weight, ws, dev_status, g_wait_limit_ns};
    return from_cuda(vca::launch_cache_weigh(a, static_cast<cudaStream_t>(stream)));
}

int vca_cache_evict(const vca_cache *cache, float *weight, const int32_t *dst_table, int dst_cols, int budget,
                    int recent, int32_t *new_len, int32_t *kept, int32_t *dev_status, void *stream) {
    vca::CacheView c;
    if (!cache_ok(cache, &c) || budget < 1 || recent < 0 || recent > budget || dst_cols < 1 ||
        static_cast<int64_t>(dst_cols) * 128 < budget)
        return VCA_ERR_INVALID_ARG;
    if (!weight || !aligned16(weight) || !aligned4(dev_status)) return VCA_ERR_INVALID_ARG;
    const void *ptrs[] = {dst_table, new_len, kept};
    for (const void *p : ptrs)
        if (!p || !aligned4(p)) return VCA_ERR_INVALID_ARG;
    // read by other heads' CTAs while they are written
    if (new_len == c.len || dst_table == c.table) return VCA_ERR_INVALID_ARG;
    return from_cuda(vca::launch_cache_evict(c, weight, dst_table, dst_cols, budget, recent, new_len, kept, dev_status,
                                             static_cast<cudaStream_t>(stream)));
}

int vca_expcast_codes(const float *s_raw, const float *c, const float *m, int64_t n, uint8_t *out, void *stream) {
    if (n < 0 || (n > 0 && (!s_raw || !c || !m || !out))) return VCA_ERR_INVALID_ARG;
    if (n == 0) return VCA_OK;
    return from_cuda(vca::launch_expcast_codes(s_raw, c, m, n, out, static_cast<cudaStream_t>(stream)));
}

int vca_e4m3_encode_bits(uint32_t start, int64_t n, uint8_t *out, void *stream) {
    if (n < 0 || (n > 0 && !out) || static_cast<uint64_t>(start) + static_cast<uint64_t>(n) > (1ull << 32))
        return VCA_ERR_INVALID_ARG;
    if (n == 0) return VCA_OK;
    return from_cuda(vca::launch_e4m3_encode_bits(start, n, out, static_cast<cudaStream_t>(stream)));
}

int vca_selftest_timeout(int32_t *dev_status, uint64_t limit_ns, void *stream) {
    if (!dev_status || limit_ns < 1000ull || limit_ns > 10000000000ull) return VCA_ERR_INVALID_ARG;
    return from_cuda(vca::launch_selftest_timeout(dev_status, limit_ns, static_cast<cudaStream_t>(stream)));
}

void vca_set_wait_limit_ns(uint64_t limit_ns) {
    if (limit_ns < 1000ull) limit_ns = 1000ull;
    if (limit_ns > 10000000000ull) limit_ns = 10000000000ull;
    g_wait_limit_ns = limit_ns;
}

}  // extern "C"
