// api_kv.cu -- the C ABI of the query / key norm and rotation, the paged NVFP4 cache and the attention over it:
// host-side validation, status codes, launches on the caller's stream (include/qlin.h).
#include <math.h>

#include "qlin_common.cuh"

extern "C" cudaError_t qlin_launch_qk_rope(const qlin_kv_cache* cache, const void* x, int xdt, int64_t T, int64_t ldx,
                                           int Hq, int Hkv, int D, const qlin_qk_params* p, const int32_t* positions,
                                           const int32_t* slots, void* q, int64_t ldq, void* k, int64_t ldk, int ydt,
                                           void* ws, cudaStream_t s);
extern "C" cudaError_t qlin_launch_kv_gather(const qlin_kv_cache* cache, int64_t T, const int32_t* slots, void* k,
                                             void* v, int ydt, void* ws, cudaStream_t s);
extern "C" size_t qlin_attn_kv4_ws_bytes(const qlin_kv_cache* c, int B, int max_q, int Hq);
extern "C" cudaError_t qlin_launch_attn_kv4(const qlin_kv_cache* c, const void* q, int64_t ldq, const int32_t* table,
                                            int64_t ldb, int max_pages, const int32_t* lens, const int32_t* cu, int B,
                                            int max_q, int64_t total_q, int Hq, float scale, int window, void* out,
                                            int64_t ldo, void* ws, cudaStream_t s);

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 20;
constexpr int64_t kMaxLd = (int64_t)1 << 31;
constexpr int kMaxHeads = 1024;
constexpr int kMaxSeqs = 1024;
constexpr int64_t kMaxContext = (int64_t)1 << 26;  // a block table's tokens: tiles are counted in 32 bits
constexpr int kMaxGroup = 64;  // query heads a kv head

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

qlin_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? QLIN_OK : QLIN_ERR_CUDA; }

bool valid_dtype(int t) { return t == QLIN_F32 || t == QLIN_BF16; }

qlin_status_t check_geometry(int64_t n_pages, int page, int Hkv, int D) {
    if (n_pages < 1 || Hkv < 1 || Hkv > kMaxHeads || D < 1) return QLIN_ERR_INVALID_ARG;
    if (page != 16 && page != 32 && page != 64 && page != 128 && page != 256) return QLIN_ERR_INVALID_ARG;
    if (n_pages > (((int64_t)1 << 31) - 1) / page) return QLIN_ERR_INVALID_ARG;
    if (n_pages * (page / 16) * Hkv >= ((int64_t)1 << 32) - 1) return QLIN_ERR_UNSUPPORTED;  // groups are numbered in 32 bits
    return D == 64 || D == 128 ? QLIN_OK : QLIN_ERR_UNSUPPORTED;
}

qlin_status_t check_cache(const qlin_kv_cache* c) {
    if (!c || !c->data) return QLIN_ERR_INVALID_ARG;
    const qlin_status_t st = check_geometry(c->n_pages, c->page, c->Hkv, c->D);
    if (st != QLIN_OK) return st;
    if (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || !isfinite(c->k_scale) || !isfinite(c->v_scale))
        return QLIN_ERR_INVALID_ARG;
    return aligned(c->data, 256) ? QLIN_OK : QLIN_ERR_ALIGNMENT;
}

// Rows of `cols` values of type dt at p, `ld` elements apart, read or written 16 bytes at a time.
qlin_status_t check_rows(const void* p, int dt, int64_t ld, int64_t cols) {
    if (!p || ld < cols || ld >= kMaxLd) return QLIN_ERR_INVALID_ARG;
    return aligned(p, 16) && ld % (dt == QLIN_F32 ? 4 : 8) == 0 ? QLIN_OK : QLIN_ERR_ALIGNMENT;
}

qlin_status_t check_params(const qlin_qk_params* p, int D, const int32_t* positions) {
    if (!p) return QLIN_ERR_INVALID_ARG;
    if (p->flags != QLIN_ROPE_HALVES && p->flags != QLIN_ROPE_INTERLEAVED) return QLIN_ERR_INVALID_ARG;
    if (p->rot < 0 || p->rot > D || p->rot % 16) return QLIN_ERR_INVALID_ARG;
    if (p->rot > 0 && (!p->cos_sin || !positions || p->n_pos < 1)) return QLIN_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f) || !isfinite(p->eps)) return QLIN_ERR_INVALID_ARG;
    if (!aligned(p->cos_sin, 16) || !aligned(p->q_weight, 16) || !aligned(p->k_weight, 16) || !aligned(positions, 4))
        return QLIN_ERR_ALIGNMENT;
    return QLIN_OK;
}

qlin_status_t check_ws(const void* ws, size_t bytes, size_t need) {
    if (!ws || bytes < need) return QLIN_ERR_WORKSPACE;
    return aligned(ws, 256) ? QLIN_OK : QLIN_ERR_ALIGNMENT;
}

qlin_status_t check_attn(const qlin_kv_cache* c, int B, int max_q, int Hq) {
    const qlin_status_t st = check_cache(c);
    if (st != QLIN_OK) return st;
    if (B < 1 || B > kMaxSeqs || max_q < 1 || max_q > kMaxTokens) return QLIN_ERR_INVALID_ARG;
    if (Hq < 1 || Hq % c->Hkv) return QLIN_ERR_INVALID_ARG;
    return Hq / c->Hkv <= kMaxGroup ? QLIN_OK : QLIN_ERR_UNSUPPORTED;
}

}  // namespace

#define QLIN_CHECK(call)                            \
    do {                                            \
        const qlin_status_t st_ = (call);           \
        if (st_ != QLIN_OK) return st_;             \
    } while (0)

extern "C" {

size_t qlin_kv_cache_bytes(int64_t n_pages, int page, int Hkv, int D) {
    if (check_geometry(n_pages, page, Hkv, D) != QLIN_OK) return 0;
    return (size_t)n_pages * (size_t)Hkv * (size_t)(page / 16) * (size_t)(18 * D);
}

qlin_status_t qlin_qk_norm_rope(const void* x, qlin_dtype_t xdt, int64_t T, int64_t ldx, int Hq, int Hkv, int D,
                                const qlin_qk_params* params, const int32_t* positions, void* q, int64_t ldq, void* k,
                                int64_t ldk, qlin_dtype_t ydt, int flags, void* ws, size_t ws_bytes,
                                qlin_stream_t stream) {
    if (!valid_dtype(xdt) || !valid_dtype(ydt) || flags != 0) return QLIN_ERR_INVALID_ARG;
    if (T < 0 || T > kMaxTokens || Hq < 1 || Hq > kMaxHeads || Hkv < 1 || Hkv > kMaxHeads || D < 1)
        return QLIN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return QLIN_ERR_UNSUPPORTED;
    if (T == 0) return QLIN_OK;
    QLIN_CHECK(check_params(params, D, positions));
    QLIN_CHECK(check_rows(x, xdt, ldx, (int64_t)(Hq + Hkv) * D));
    QLIN_CHECK(check_rows(q, ydt, ldq, (int64_t)Hq * D));
    QLIN_CHECK(check_rows(k, ydt, ldk, (int64_t)Hkv * D));
    QLIN_CHECK(check_ws(ws, ws_bytes, 256));
    return cuda_status(qlin_launch_qk_rope(nullptr, x, xdt, T, ldx, Hq, Hkv, D, params, positions, nullptr, q, ldq, k,
                                           ldk, ydt, ws, (cudaStream_t)stream));
}

qlin_status_t qlin_kv_append(const qlin_kv_cache* cache, const void* x, qlin_dtype_t xdt, int64_t T, int64_t ldx,
                             int Hq, const qlin_qk_params* params, const int32_t* positions, const int32_t* slots,
                             void* q, int64_t ldq, int flags, void* ws, size_t ws_bytes, qlin_stream_t stream) {
    QLIN_CHECK(check_cache(cache));
    if (!valid_dtype(xdt) || flags != 0 || T < 0 || T > kMaxTokens || Hq < 0 || Hq > kMaxHeads)
        return QLIN_ERR_INVALID_ARG;
    if (T == 0) return QLIN_OK;
    QLIN_CHECK(check_params(params, cache->D, positions));
    QLIN_CHECK(check_rows(x, xdt, ldx, (int64_t)(Hq + 2 * cache->Hkv) * cache->D));
    if (q) QLIN_CHECK(check_rows(q, QLIN_BF16, ldq, (int64_t)Hq * cache->D));
    if (!slots) return QLIN_ERR_INVALID_ARG;
    if (!aligned(slots, 4)) return QLIN_ERR_ALIGNMENT;
    QLIN_CHECK(check_ws(ws, ws_bytes, 256));
    return cuda_status(qlin_launch_qk_rope(cache, x, xdt, T, ldx, Hq, cache->Hkv, cache->D, params, positions, slots,
                                           q, ldq, nullptr, 0, QLIN_BF16, ws, (cudaStream_t)stream));
}

qlin_status_t qlin_kv_gather(const qlin_kv_cache* cache, int64_t T, const int32_t* slots, void* k, void* v,
                             qlin_dtype_t ydt, void* ws, size_t ws_bytes, qlin_stream_t stream) {
    QLIN_CHECK(check_cache(cache));
    if (!valid_dtype(ydt) || T < 0 || T > kMaxTokens) return QLIN_ERR_INVALID_ARG;
    if (T == 0) return QLIN_OK;
    if (!slots || !k || !v) return QLIN_ERR_INVALID_ARG;
    if (!aligned(slots, 4) || !aligned(k, 16) || !aligned(v, 16)) return QLIN_ERR_ALIGNMENT;
    QLIN_CHECK(check_ws(ws, ws_bytes, 256));
    return cuda_status(qlin_launch_kv_gather(cache, T, slots, k, v, ydt, ws, (cudaStream_t)stream));
}

size_t qlin_attn_kv4_workspace_bytes(const qlin_kv_cache* cache, int B, int max_q, int Hq) {
    if (check_attn(cache, B, max_q, Hq) != QLIN_OK) return 0;
    return qlin_attn_kv4_ws_bytes(cache, B, max_q, Hq);
}

qlin_status_t qlin_attn_kv4(const qlin_kv_cache* cache, const void* q, int64_t ldq, const int32_t* block_table,
                            int64_t ldb, int max_pages, const int32_t* seq_lens, const int32_t* cu_q, int B,
                            int max_q, int64_t total_q, int Hq, float scale, int window, void* out, int64_t ldo,
                            int flags, void* ws, size_t ws_bytes, qlin_stream_t stream) {
    QLIN_CHECK(check_attn(cache, B, max_q, Hq));
    if (flags != 0 || window < 0 || !isfinite(scale * cache->k_scale * 2.0f)) return QLIN_ERR_INVALID_ARG;
    if (total_q < 0 || total_q > kMaxTokens || max_pages < 1 || ldb < max_pages || ldb >= kMaxLd)
        return QLIN_ERR_INVALID_ARG;
    if (max_pages > kMaxContext / cache->page) return QLIN_ERR_INVALID_ARG;
    if (total_q == 0) return QLIN_OK;
    if (!block_table || !seq_lens || !cu_q) return QLIN_ERR_INVALID_ARG;
    QLIN_CHECK(check_rows(q, QLIN_BF16, ldq, (int64_t)Hq * cache->D));
    QLIN_CHECK(check_rows(out, QLIN_BF16, ldo, (int64_t)Hq * cache->D));
    if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q, 4)) return QLIN_ERR_ALIGNMENT;
    QLIN_CHECK(check_ws(ws, ws_bytes, qlin_attn_kv4_ws_bytes(cache, B, max_q, Hq)));
    return cuda_status(qlin_launch_attn_kv4(cache, q, ldq, block_table, ldb, max_pages, seq_lens, cu_q, B, max_q,
                                            total_q, Hq, scale, window, out, ldo, ws, (cudaStream_t)stream));
}

}  // extern "C"
