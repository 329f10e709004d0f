// attn_common.cuh -- what the two attention kernels over the NVFP4 cache share.
#pragma once
#include "kv_cache.cuh"

namespace qlin {
namespace kv {

struct AttnArgs {
    Cache cache;
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    const int32_t *table, *lens, *cu;
    int64_t ldq, ldo, ldb, total_q;
    int max_pages, B, max_q, Hq, G;
    uint32_t g_magic;  // ceil(2^32 / G), 0 for G = 1: rows to queries without a division (group_div)
    float scale_log2;  // scale * k_scale * log2(e)
    int window;        // 0: none; below 2^30
    unsigned* status;
    int RB;             // few rows: row blocks of a (sequence, head)
    int* tickets;       // in the workspace: kMaxParts, zero between calls
    float* parts;       // then the parts of what several CTAs share
};

// r / G and r % G of a query row r < 2^26 (2^20 queries, G <= 64): r * (ceil(2^32 / G) - 2^32 / G) < 2^26 <= 2^32 / G, so
// the high word of the product is the quotient.
__device__ __forceinline__ int group_div(const AttnArgs& a, int r) { return a.g_magic ? (int)__umulhi((uint32_t)r, a.g_magic) : r; }
__device__ __forceinline__ int group_mod(const AttnArgs& a, int r) { return r - group_div(a, r) * a.G; }
// a / b, in 32 bits where both fit (the usual case by far).
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b) {
    if (((uint64_t)(a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

constexpr int kMaxParts = 512;  // CTAs of a launch at most: tickets in the workspace

// The first place that the first of a sequence's n queries sees, and its tile.  Groups of the cache that lie before it are
// not looked at, nor their pages' numbers: a user may have given the pages away.
__device__ __forceinline__ int first_seen(const AttnArgs& a, int n, int L) {
    const int lo = a.window > 0 ? L - n + 1 - a.window : 0;
    return lo > 0 ? lo : 0;
}
template <int TILE>
__device__ __forceinline__ int first_tile(const AttnArgs& a, int n, int L) {
    return first_seen(a, n, L) / TILE;
}
// A sequence's queries and context; bad ones are skipped.
struct Seq {
    int64_t row0;
    int n, L;
    bool bad;
};
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
    Seq s;
    s.row0 = __ldg(a.cu + b);
    s.n = __ldg(a.cu + b + 1) - (int)s.row0;
    s.L = __ldg(a.lens + b);
    s.bad = s.n < 0 || s.n > a.max_q || s.row0 < 0 || s.row0 + s.n > a.total_q || s.L < 0 ||
            (int64_t)s.L > ((int64_t)a.max_pages << a.cache.page_log);
    return s;
}

// The four f16x2 values of a word's bytes (low half: the byte's low nibble).
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        " cvt.rn.f16x2.e2m1x2 %1, b1;\n cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What is taken off a row's scores (its reference) is set kBelow under the largest score seen, and set anew only when a score
// has come to lie more than kGrow above it: O is rarely rescaled.  A row's largest probability is then 2^7 to 2^15 (2^15.1
// with the rounding of a product below 2^20), which fp16 holds, and those that it rounds to 0 lie 2^32 and more below the
// largest: of 2^20 equal tokens under one large one, less than half a step of bf16 is lost.  The sum counts them all.
constexpr float kBelow = 7.f, kGrow = 15.f;

// Exponent of a query row's largest magnitude, kept where both 2^(14 - e) and 2^(e - 14) are normal numbers: the row
// times 2^(14 - e) (with the sign of the scale) is fp16 with its largest magnitude in [2^14, 2^15), exact but for
// values 2^28 below it, and |scale| 2^(e - 14) takes the scores to the exponents of 2.
__device__ __forceinline__ int row_exponent(float amax) {
    return max(min((int)(__float_as_uint(amax) >> 23) - 127, 126), -100);
}
__device__ __forceinline__ float row_up(int e, float scale_log2) {
    return copysignf(__uint_as_float((uint32_t)(14 - e + 127) << 23), scale_log2);
}
__device__ __forceinline__ float row_down(int e, float scale_log2) {
    return fabsf(scale_log2) * __uint_as_float((uint32_t)(e - 14 + 127) << 23);
}
__device__ __forceinline__ float amax_bf16x2(uint32_t w) {
    return fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u)));
}
__device__ __forceinline__ uint32_t scaled_f16x2(uint32_t w, float up) {
    return pack_f16x2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
}

// Two output values: sums of P V times the reciprocal of P's sum, then the cache's scale (over the sum it need not be a
// normal number).
__device__ __forceinline__ __nv_bfloat162 out_pair(const AttnArgs& a, float x, float y, float inv) {
    return __floats2bfloat162_rn(x * inv * a.cache.v_scale, y * inv * a.cache.v_scale);
}

}  // namespace kv
}  // namespace qlin
