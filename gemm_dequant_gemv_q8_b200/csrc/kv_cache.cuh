// kv_cache.cuh -- layout of the paged NVFP4 cache of keys and values and the helpers that its kernels
// share.  A group is 16 tokens of one kv head, 18 * D bytes (the layout is stated in include/qlin.h):
//   K codes token-major : a thread that multiplies 16-byte pieces of a token's row by a query needs no
//                         other layout, and a token's codes and scales are whole words;
//   V codes block-major : [16-value block][token][8 bytes], so that the codes which one thread of a
//                         matrix instruction needs of four tokens (the long axis of P V) are 32
//                         contiguous bytes, and its four scales one word.
// A (page, kv head) is page / 16 contiguous groups: one bulk copy.
#pragma once
#include "chunk_common.cuh"

namespace qlin {
namespace kv {

constexpr int kGroup = 16;  // tokens a group

__host__ __device__ constexpr int group_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int k_scale_off(int D) { return 8 * D; }
__host__ __device__ constexpr int v_code_off(int D) { return 9 * D; }
__host__ __device__ constexpr int v_scale_off(int D) { return 17 * D; }

// What the kernels need of a qlin_kv_cache.
struct Cache {
    uint8_t* data;
    int64_t n_pages;
    int32_t page_log;  // page = 1 << page_log tokens
    int32_t Hkv;
    float k_scale, v_scale;
};

// The group of token `off` of a page, for kv head h.
template <int D>
__device__ __forceinline__ uint8_t* group_ptr(const Cache& c, int64_t page, int h, int off) {
    const int per = 1 << (c.page_log - 4);
    return c.data + ((page * c.Hkv + h) * per + (off >> 4)) * group_bytes(D);
}

inline Cache make_cache(const qlin_kv_cache* c) {
    Cache r = {};
    r.data = (uint8_t*)c->data;
    r.n_pages = c->n_pages;
    r.page_log = 31 - __builtin_clz((unsigned)c->page);
    r.Hkv = c->Hkv;
    r.k_scale = c->k_scale;
    r.v_scale = c->v_scale;
    return r;
}

constexpr unsigned kStatusBad = 2u;  // status word: a bad index (read as QLIN_ERR_INVALID_ARG)

}  // namespace kv
}  // namespace qlin
