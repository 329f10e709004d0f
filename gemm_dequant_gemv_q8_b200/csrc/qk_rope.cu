// qk_rope.cu -- norm and rotation of queries and keys, the append of keys and values to the paged
// NVFP4 cache, and the read-back of slots.
//
// Per head: n = h * w / sqrt(mean(h^2) + eps), then the first rot values in pairs (a, b) ->
// (a c - b s, b c + a s).  Bound by memory: every value is read and written once.  A lane holds 8 values of a head
// (one or two 16-byte loads), D / 8 lanes a head; the mean is a shuffle sum, a pair of the half-split rotation is one
// shuffle away.  A warp works on one token and on 8 heads of one kind (queries, keys, values): their loads are all in
// flight before the token's row of cosines and sines, which needs its position, is asked for.
#include "kv_cache.cuh"

namespace qlin {
namespace kv {

constexpr int kHeadsPerWarp = 8;
constexpr int kRopeWarps = 4;

struct RopeArgs {
    const void* x;
    int64_t T, ldx;
    int Hq, Hkv, chunks;  // chunks: warps a token
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

// 8 values as they lie in memory, and as fp32.
template <typename X>
struct Raw8 {
    uint4 u[sizeof(X) / 2];
    __device__ __forceinline__ void load(const X* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(X) / 2; ++i) u[i] = *(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(X) / 2; ++i) u[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (sizeof(X) == 4) {
            const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
        } else {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(w[j] << 16);
                v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    }
};
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    Raw8<float> r;
    r.load(p);
    r.get(v);
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
            r = rsqrt(ms);
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
        // The reciprocal and its corrections give the correctly rounded quotient where nothing over- or underflows
        // on the way (div_by_recip): ordinary scales, quotients below 2^60.
        const float y = __frcp_rn(div);
        if (div >= 0x1p-96f && div <= 0x1p96f && m * y <= 0x1p60f) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 qv = div_by_recip2(make_float2(v[2 * j], v[2 * j + 1]), div, y);
                codes |= e2m1x2_rne_sat(qv.x, qv.y) << (8 * j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                codes |= e2m1x2_rne_sat(__fdiv_rn(v[2 * j], div), __fdiv_rn(v[2 * j + 1], div)) << (8 * j);
        }
    }
    return s;
}

// APPEND: heads are [q | k | v]; q to bf16 rows, k and v to the cache.  Otherwise [q | k] to rows of Y.
template <typename X, typename Y, int D, bool INTER, bool APPEND>
__global__ void __launch_bounds__(kRopeWarps * 32) qk_rope_kernel(const RopeArgs a) {
    constexpr int LPH = D / 8, HPW = 32 / LPH;         // lanes a head, heads a warp at once
    constexpr int N = kHeadsPerWarp / HPW;             // heads a lane
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t t = item / a.chunks;
    if (t >= a.T) return;
    // this warp's heads: chunks of queries, then of keys, then of values
    int c = (int)(item - t * a.chunks);
    const int cq = APPEND && !a.q ? 0 : (a.Hq + kHeadsPerWarp - 1) / kHeadsPerWarp, ck = (a.Hkv + kHeadsPerWarp - 1) / kHeadsPerWarp;
    const int kind = c < cq ? 0 : c < cq + ck ? 1 : 2;
    c -= kind == 0 ? 0 : kind == 1 ? cq : cq + ck;
    const int heads = kind == 0 ? a.Hq : a.Hkv, base = kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + a.Hkv;
    const int sub = lane / LPH, d0 = (lane % LPH) * 8;
    const int h0 = c * kHeadsPerWarp + sub;            // heads h0, h0 + HPW, ..
    const X* row = reinterpret_cast<const X*>(a.x) + t * a.ldx + (int64_t)base * D + d0;
    Raw8<X> raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (h0 + i * HPW < heads)
            raw[i].load(row + (int64_t)(h0 + i * HPW) * D);
        else
            raw[i].zero();
    }
    int slot = 0;
    if constexpr (APPEND) slot = a.slots[t];
    const int64_t pos = a.rot > 0 ? a.pos[t] : 0;
    const float* wp = kind == 0 ? a.qw : a.kw;
    const bool norm = kind < 2 && wp != nullptr;
    float cs[8], sn[8], w[8];
    if (norm) load8(wp + d0, w);
    bool bad = a.rot > 0 && (pos < 0 || pos >= a.n_pos);
    if constexpr (APPEND) {
        if (slot == -1) return;
        bad |= slot < 0 || ((int64_t)slot >> a.cache.page_log) >= a.cache.n_pages;
    }
    if (bad) {
        if (lane == 0) atomicOr(a.status, kStatusBad);
        return;
    }
    if (kind < 2 && d0 < a.rot) load_turn<INTER>(a.cs + pos * a.rot, a.rot, d0, cs, sn);
    if (!APPEND || kind == 0) {
        Y* out = kind == 0 ? reinterpret_cast<Y*>(a.q) + t * a.ldq : reinterpret_cast<Y*>(a.k) + t * a.ldk;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[8];
            raw[i].get(v);
            norm_rope<float, D, INTER>(v, norm, w, a.eps, a.rot, d0, cs, sn);
            if (h0 + i * HPW < heads) store8(out + (int64_t)(h0 + i * HPW) * D + d0, v);
        }
    } else {
        const bool isv = kind == 2;
        const int off = slot & ((1 << a.cache.page_log) - 1), r = off & 15;
        const int code_at = isv ? v_code_off(D) + (d0 >> 4) * 128 + r * 8 + (d0 & 15) / 2 : r * (D / 2) + d0 / 2;
        const int scale_at = isv ? v_scale_off(D) + (d0 >> 4) * 16 + r : k_scale_off(D) + r * (D / 16) + (d0 >> 4);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[8];
            raw[i].get(v);
            if (!isv) norm_rope<double, D, INTER>(v, norm, w, a.eps, a.rot, d0, cs, sn);
            uint32_t codes;
            const uint8_t sc = quant8(v, isv ? a.cache.v_scale : a.cache.k_scale, codes);
            if (h0 + i * HPW < heads) {
                uint8_t* g = group_ptr<D>(a.cache, slot >> a.cache.page_log, h0 + i * HPW, off);
                *reinterpret_cast<uint32_t*>(g + code_at) = codes;
                if ((lane & 1) == 0) g[scale_at] = sc;
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
    const int64_t blocks = (a.T * a.chunks + kv::kRopeWarps - 1) / kv::kRopeWarps;
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
    a.x = x, a.T = T, a.ldx = ldx, a.Hq = Hq, a.Hkv = Hkv;
    const auto chunks = [](int heads) { return (heads + kv::kHeadsPerWarp - 1) / kv::kHeadsPerWarp; };
    a.chunks = (cache && !q ? 0 : chunks(Hq)) + (cache ? 2 : 1) * chunks(Hkv);
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
