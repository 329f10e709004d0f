// qk_rope.cu -- norm and rotation of queries and keys, the append of keys and values to the paged
// NVFP4 cache, and the read-back of slots.
//
// Per head: n = h * w / sqrt(mean(h^2) + eps), then the first rot values in pairs (a, b) ->
// (a c - b s, b c + a s).  A lane holds 8 values of a head (one or two 16-byte loads), D / 8 lanes a head;
// the mean is a shuffle sum, a pair of the half-split rotation is one shuffle away.  A warp works on one
// token and on several heads, so that the token's cosines, sines and the weights are loaded once.
#include "kv_cache.cuh"

namespace qlin {
namespace kv {

constexpr int kHeadsPerWarp = 8;
constexpr int kRopeWarps = 4;

struct RopeArgs {
    const void* x;
    int64_t T, ldx;
    int Hq, Hkv, heads;  // heads: those of x that are worked on
    const float *qw, *kw, *cs;
    int64_t n_pos;
    int rot;
    float eps;
    const int32_t *pos, *slots;
    void *q, *k;
    int64_t ldq, ldk;
    Cache cache;
    unsigned* status;
};

template <typename X>
__device__ __forceinline__ void load8(const X* p, float (&v)[8]) {
    if constexpr (sizeof(X) == 4) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
}

template <typename Y>
__device__ __forceinline__ void store8(Y* p, const float (&v)[8]) {
    if constexpr (sizeof(Y) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// The cosines and sines of this lane's 8 values.  HALVES: of pairs i .. i + 7 with i = value % (rot / 2);
// INTERLEAVED: of pairs value / 2 .. + 3.
template <bool INTER>
__device__ __forceinline__ void load_turn(const float* row, int rot, int d0, float (&c)[8], float (&s)[8]) {
    if constexpr (INTER) {
        const float4 a = *reinterpret_cast<const float4*>(row + d0 / 2);
        const float4 b = *reinterpret_cast<const float4*>(row + rot / 2 + d0 / 2);
        c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
        s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
    } else {
        const int i = d0 < rot / 2 ? d0 : d0 - rot / 2;
        load8(row + i, c);
        load8(row + rot / 2 + i, s);
    }
}

// Norm (where w is given) and rotation of one head in the arithmetic of R (float, or double for keys
// that are quantized).  Every lane of the D / 8 lanes of a head calls it; `w` and `turn` are uniform.
template <typename R, int D, bool INTER>
__device__ __forceinline__ void norm_rope(float (&v)[8], bool norm, const float (&w)[8], float eps, int rot, int d0,
                                          const float (&c)[8], const float (&s)[8]) {
    R n[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) n[j] = (R)v[j];
    if (norm) {
        R ss = (R)0;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += n[j] * n[j];
#pragma unroll
        for (int m = D / 16; m; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const R ms = ss * (R)(1.0 / D) + (R)eps;
        R r;
        if constexpr (sizeof(R) == 8)
            r = 1.0 / sqrt(ms);
        else
            r = 1.0f / sqrtf(ms);
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = n[j] * r * (R)w[j];
    }
    if (rot > 0) {
        if constexpr (INTER) {
            if (d0 < rot) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const R a = n[2 * j], b = n[2 * j + 1];
                    n[2 * j] = a * (R)c[j] - b * (R)s[j];
                    n[2 * j + 1] = b * (R)c[j] + a * (R)s[j];
                }
            }
        } else {
            const int lane = threadIdx.x & 31;
            const bool lo = d0 < rot / 2;
            const int other = d0 < rot ? (lo ? lane + rot / 16 : lane - rot / 16) : lane;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const R o = __shfl_sync(0xffffffffu, n[j], other);
                if (d0 < rot) n[j] = lo ? n[j] * (R)c[j] - o * (R)s[j] : n[j] * (R)c[j] + o * (R)s[j];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)n[j];
}

// Quantize this lane's 8 values (its neighbour lane ^ 1 holds the block's other 8) under scale g.
__device__ __forceinline__ uint8_t quant8(const float (&v)[8], float g, uint32_t& codes) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint8_t s = e4m3_rne_sat(__fdiv_rn(m, __fmul_rn(6.0f, g)));
    const float div = __fmul_rn(e4m3_to_f32(s), g);
    codes = 0u;
    if (div > 0.f) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            codes |= e2m1x2_rne_sat(__fdiv_rn(v[2 * j], div), __fdiv_rn(v[2 * j + 1], div)) << (8 * j);
    }
    return s;
}

// APPEND: heads are [q | k | v]; q to bf16 rows, k and v to the cache.  Otherwise [q | k] to rows of Y.
template <typename X, typename Y, int D, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kRopeWarps * 32) qk_rope_kernel(const RopeArgs a) {
    constexpr int LPH = D / 8, HPW = 32 / LPH;  // lanes a head, heads a warp at once
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks = (a.heads + kHeadsPerWarp - 1) / kHeadsPerWarp;
    const int64_t item = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t t = item / chunks;
    if (t >= a.T) return;
    const int h0 = (int)(item - t * chunks) * kHeadsPerWarp;
    const int sub = lane / LPH, d0 = (lane % LPH) * 8;
    int slot = 0;
    if constexpr (APPEND) {
        slot = a.slots[t];
        if (slot == -1) return;
    }
    const int64_t pos = a.rot > 0 ? a.pos[t] : 0;
    bool bad = a.rot > 0 && (pos < 0 || pos >= a.n_pos);
    if constexpr (APPEND) bad |= slot < 0 || ((int64_t)slot >> a.cache.page_log) >= a.cache.n_pages;
    if (bad) {
        if (lane == 0) atomicOr(a.status, kStatusBad);
        return;
    }
    float c[8], s[8], qw[8], kw[8];
    if (d0 < a.rot) load_turn<INTER>(a.cs + pos * a.rot, a.rot, d0, c, s);
    if (a.qw) load8(a.qw + d0, qw);
    if (a.kw) load8(a.kw + d0, kw);
    const X* row = reinterpret_cast<const X*>(a.x) + t * a.ldx + d0;
#pragma unroll 4
    for (int i = 0; i < kHeadsPerWarp; i += HPW) {
        const int h = h0 + i + sub;
        const bool in = h < a.heads;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (in) load8(row + (int64_t)h * D, v);
        const bool isq = h < a.Hq, isv = h >= a.Hq + a.Hkv;
        if (__any_sync(0xffffffffu, in && isq)) {
            float u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = v[j];
            norm_rope<float, D, INTER>(u, a.qw != nullptr, qw, a.eps, a.rot, d0, c, s);
            if (in && isq && a.q) store8(reinterpret_cast<Y*>(a.q) + t * a.ldq + (int64_t)h * D + d0, u);
        }
        if (__any_sync(0xffffffffu, in && !isq)) {
            if constexpr (!APPEND) {
                norm_rope<float, D, INTER>(v, a.kw != nullptr, kw, a.eps, a.rot, d0, c, s);
                if (in && !isq) store8(reinterpret_cast<Y*>(a.k) + t * a.ldk + (int64_t)(h - a.Hq) * D + d0, v);
            } else {
                if (__any_sync(0xffffffffu, in && !isq && !isv)) {
                    float u[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[j] = v[j];
                    norm_rope<double, D, INTER>(u, a.kw != nullptr, kw, a.eps, a.rot, d0, c, s);
                    if (!isv) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = u[j];
                    }
                }
                uint32_t codes;
                const uint8_t sc = quant8(v, isv ? a.cache.v_scale : a.cache.k_scale, codes);
                if (in && !isq) {
                    const int kvh = h - a.Hq - (isv ? a.Hkv : 0);
                    const int off = slot & ((1 << a.cache.page_log) - 1), r = off & 15;
                    uint8_t* g = group_ptr<D>(a.cache, slot >> a.cache.page_log, kvh, off);
                    const int code_at = isv ? v_code_off(D) + (d0 >> 4) * 128 + r * 8 + (d0 & 15) / 2 : r * (D / 2) + d0 / 2;
                    *reinterpret_cast<uint32_t*>(g + code_at) = codes;
                    if ((lane & 1) == 0)
                        g[isv ? v_scale_off(D) + (d0 >> 4) * 16 + r : k_scale_off(D) + r * (D / 16) + (d0 >> 4)] = sc;
                }
            }
        }
    }
}

template <typename Y, int D>
__global__ void __launch_bounds__(256) kv_gather_kernel(Cache cache, int64_t T, const int32_t* slots, Y* k, Y* v,
                                                        unsigned* status) {
    constexpr int LPH = D / 8;
    const int64_t per = (int64_t)cache.Hkv * LPH;  // lanes a token
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = i / per;
    if (t >= T) return;
    const int rem = (int)(i - t * per), h = rem / LPH, d0 = (rem % LPH) * 8;
    const int slot = slots[t];
    if (slot == -1) return;
    if (slot < 0 || ((int64_t)slot >> cache.page_log) >= cache.n_pages) {
        atomicOr(status, kStatusBad);
        return;
    }
    const int off = slot & ((1 << cache.page_log) - 1), r = off & 15;
    const uint8_t* g = group_ptr<D>(cache, slot >> cache.page_log, h, off);
    const uint32_t kc = *reinterpret_cast<const uint32_t*>(g + r * (D / 2) + d0 / 2);
    const uint32_t vc = *reinterpret_cast<const uint32_t*>(g + v_code_off(D) + (d0 >> 4) * 128 + r * 8 + (d0 & 15) / 2);
    const float ks = e4m3_to_f32(g[k_scale_off(D) + r * (D / 16) + (d0 >> 4)]);
    const float vs = e4m3_to_f32(g[v_scale_off(D) + (d0 >> 4) * 16 + r]);
    float a[8], b[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t x = e2m1x2_to_f16x2(kc >> (8 * j)), y = e2m1x2_to_f16x2(vc >> (8 * j));
        a[2 * j] = fp16_bits_to_f32(x & 0xffffu) * ks * cache.k_scale;  // code * scale is exact
        a[2 * j + 1] = fp16_bits_to_f32(x >> 16) * ks * cache.k_scale;
        b[2 * j] = fp16_bits_to_f32(y & 0xffffu) * vs * cache.v_scale;
        b[2 * j + 1] = fp16_bits_to_f32(y >> 16) * vs * cache.v_scale;
    }
    const int64_t at = (t * cache.Hkv + h) * D + d0;
    store8(k + at, a);
    store8(v + at, b);
}

}  // namespace kv
}  // namespace qlin

using namespace qlin;

template <typename X, typename Y, bool APPEND>
static cudaError_t launch_rope(const kv::RopeArgs& a, int D, bool inter, cudaStream_t s) {
    const int64_t chunks = (a.heads + kv::kHeadsPerWarp - 1) / kv::kHeadsPerWarp;
    const int64_t blocks = (a.T * chunks + kv::kRopeWarps - 1) / kv::kRopeWarps;
    const dim3 grid((unsigned)blocks), block(kv::kRopeWarps * 32);
    if (D == 128)
        inter ? kv::qk_rope_kernel<X, Y, 128, true, APPEND><<<grid, block, 0, s>>>(a)
              : kv::qk_rope_kernel<X, Y, 128, false, APPEND><<<grid, block, 0, s>>>(a);
    else
        inter ? kv::qk_rope_kernel<X, Y, 64, true, APPEND><<<grid, block, 0, s>>>(a)
              : kv::qk_rope_kernel<X, Y, 64, false, APPEND><<<grid, block, 0, s>>>(a);
    return cudaGetLastError();
}

// cache == NULL: norm and rotation only.
extern "C" cudaError_t qlin_launch_qk_rope(const qlin_kv_cache* cache, const void* x, int xdt, int64_t T, int64_t ldx,
                                           int Hq, int Hkv, int D, const qlin_qk_params* p, const int32_t* positions,
                                           const int32_t* slots, void* q, int64_t ldq, void* k, int64_t ldk, int ydt,
                                           void* ws, cudaStream_t s) {
    kv::RopeArgs a = {};
    a.x = x, a.T = T, a.ldx = ldx, a.Hq = Hq, a.Hkv = Hkv, a.heads = Hq + (cache ? 2 : 1) * Hkv;
    a.qw = p->q_weight, a.kw = p->k_weight, a.cs = p->cos_sin, a.n_pos = p->n_pos, a.rot = p->rot, a.eps = p->eps;
    a.pos = positions, a.slots = slots, a.q = q, a.ldq = ldq, a.k = k, a.ldk = ldk;
    a.status = (unsigned*)ws;
    const bool inter = p->flags == QLIN_ROPE_INTERLEAVED, xf = xdt == QLIN_F32;
    if (cache) {
        a.cache = kv::make_cache(cache);
        return xf ? launch_rope<float, __nv_bfloat16, true>(a, D, inter, s)
                  : launch_rope<__nv_bfloat16, __nv_bfloat16, true>(a, D, inter, s);
    }
    if (ydt == QLIN_F32)
        return xf ? launch_rope<float, float, false>(a, D, inter, s)
                  : launch_rope<__nv_bfloat16, float, false>(a, D, inter, s);
    return xf ? launch_rope<float, __nv_bfloat16, false>(a, D, inter, s)
              : launch_rope<__nv_bfloat16, __nv_bfloat16, false>(a, D, inter, s);
}

extern "C" cudaError_t qlin_launch_kv_gather(const qlin_kv_cache* cache, int64_t T, const int32_t* slots, void* k,
                                             void* v, int ydt, void* ws, cudaStream_t s) {
    const kv::Cache c = kv::make_cache(cache);
    const int64_t n = T * c.Hkv * (cache->D / 8);
    const dim3 grid((unsigned)((n + 255) / 256));
    unsigned* st = (unsigned*)ws;
    if (cache->D == 128)
        ydt == QLIN_F32 ? kv::kv_gather_kernel<float, 128><<<grid, 256, 0, s>>>(c, T, slots, (float*)k, (float*)v, st)
                        : kv::kv_gather_kernel<__nv_bfloat16, 128><<<grid, 256, 0, s>>>(c, T, slots, (__nv_bfloat16*)k, (__nv_bfloat16*)v, st);
    else
        ydt == QLIN_F32 ? kv::kv_gather_kernel<float, 64><<<grid, 256, 0, s>>>(c, T, slots, (float*)k, (float*)v, st)
                        : kv::kv_gather_kernel<__nv_bfloat16, 64><<<grid, 256, 0, s>>>(c, T, slots, (__nv_bfloat16*)k, (__nv_bfloat16*)v, st);
    return cudaGetLastError();
}
