// qk_rope.cu -- norm and rotation of queries and keys, the append of keys and values to the paged
// NVFP4 cache, and the read-back of slots.
//
// Per head: n = h * w / sqrt(mean(h^2) + eps), then the first rot values in pairs (a, b) ->
// (a c - b s, b c + a s).  Bound by memory: every value is read and written once.  A lane holds two runs of 4 values of a
// head, D / 8 lanes a head: in the half-split rotation values i .. i + 3 and i + rot / 2 .., so that it has both members
// of its pairs and needs no other lane; elsewhere 8 neighbours.  (Where keys are quantized and an odd multiple of 16
// values is rotated: 8 neighbours and a shuffle, for a block of 16 values would be torn between the runs.)  A warp
// works on one token and on some heads of one kind (queries, keys, values): their loads are all in flight before the
// token's row of cosines and sines, which needs its position, is asked for.
#include <cuda/std/type_traits>

#include "kv_cache.cuh"

namespace qlin {
namespace kv {

// Heads a warp.  What is only normed and rotated: 8, so that a token's row of the table and the weights are loaded once for
// many (2048 tokens: 8.6 us, 9.8 with 4).  What is quantized: 4, for the path is long and its code repeated for each
// (8192 tokens appended: 53 us, 73 with 8).
constexpr int kHeadsPerWarp = 8;
constexpr int kQuantHeadsPerWarp = 4;
constexpr int kRopeWarps = 2;

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

enum Turn { kInterleaved, kSplit, kShuffled };  // how a lane meets the other members of its pairs

// A lane's two runs of 4 values as they lie in memory, and as fp32.
template <typename X>
struct Raw8 {
    uint32_t u[2][sizeof(X)];
    __device__ __forceinline__ void load(const X* p, int d0, int d1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const X* src = p + (i ? d1 : d0);
            if constexpr (sizeof(X) == 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(src);
                u[i][0] = v.x, u[i][1] = v.y, u[i][2] = v.z, u[i][3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(src);
                u[i][0] = v.x, u[i][1] = v.y;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(X); ++i) u[0][i] = u[1][i] = 0u;
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(X) == 4)
                    v[4 * i + j] = __uint_as_float(u[i][j]);
                else
                    v[4 * i + j] = __uint_as_float(j & 1 ? u[i][j / 2] & 0xffff0000u : u[i][j / 2] << 16);
            }
    }
};

template <typename Y>
__device__ __forceinline__ void store4(Y* p, const float* v) {
    if constexpr (sizeof(Y) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
}
template <typename Y>
__device__ __forceinline__ void store8(Y* p, const float (&v)[8]) {
    store4(p, v);
    store4(p + 4, v + 4);
}

// The cosines and sines of a lane's four (eight) pairs.
template <int TURN>
__device__ __forceinline__ void load_turn(const float* row, int rot, int d0, float (&c)[8], float (&s)[8]) {
    const int i = TURN == kInterleaved ? d0 / 2 : TURN == kSplit || d0 < rot / 2 ? d0 : d0 - rot / 2;
    const float4 a = *reinterpret_cast<const float4*>(row + i), b = *reinterpret_cast<const float4*>(row + rot / 2 + i);
    c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
    s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
    if constexpr (TURN == kShuffled) {  // eight pairs, with one member each here
        const float4 e = *reinterpret_cast<const float4*>(row + i + 4), f = *reinterpret_cast<const float4*>(row + rot / 2 + i + 4);
        c[4] = e.x, c[5] = e.y, c[6] = e.z, c[7] = e.w;
        s[4] = f.x, s[5] = f.y, s[6] = f.z, s[7] = f.w;
    }
}

// Norm (where `norm` says so) and rotation (of the lanes that `turn`) of one head in the arithmetic of R: float, or
// double for keys that are quantized.  Every lane of the D / 8 lanes of a head calls it.  False for all of them where the
// squares leave the range of R.
template <typename R, int D, int TURN>
__device__ __forceinline__ bool norm_rope(float (&v)[8], bool norm, const float (&w)[8], float eps, bool turn, int rot, int d0,
                                          const float (&c)[8], const float (&s)[8]) {
    R n[8];
    bool in_range = true;
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
        if constexpr (sizeof(R) == 8) {
            r = rsqrt(ms);
        } else {
            r = rsqrtf(ms);  // within 2 ulp
            in_range = ms >= 0x1p-100f && ms <= 0x1p126f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = n[j] * r * (R)w[j];
    }
    if constexpr (TURN == kShuffled) {
        const int lane = threadIdx.x & 31;
        const bool lo = d0 < rot / 2;
        const int other = !turn ? lane : lo ? lane + rot / 16 : lane - rot / 16;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const R o = __shfl_sync(0xffffffffu, n[j], other);
            if (turn) n[j] = lo ? n[j] * (R)c[j] - o * (R)s[j] : n[j] * (R)c[j] + o * (R)s[j];
        }
    } else if (turn) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            R &a = n[TURN == kInterleaved ? 2 * j : j], &b = n[TURN == kInterleaved ? 2 * j + 1 : j + 4];
            const R x = a, y = b;
            a = x * (R)c[j] - y * (R)s[j];
            b = y * (R)c[j] + x * (R)s[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)n[j];
    return in_range;
}

__device__ __forceinline__ float amax4(const float* v) {
    return fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
}

// The scale byte of a block whose largest magnitude is m, under scale g: E4M3(m / (6 g)).  div_by_recip gives the correctly
// rounded quotient where nothing over- or underflows on the way; g6 = 6 g and its reciprocal y6 are the same for all.  m is
// NaN where a block holds nothing else: scale 0, for a NaN in the cache would reach the queries that do not see it.
__device__ __forceinline__ uint8_t block_scale(float m, float g6, float y6) {
    m = fmaxf(m, 0.f);
    const bool plain = g6 >= 0x1p-60f && g6 <= 0x1p60f && m <= 0x1p60f;
    return e4m3_rne_sat(plain ? div_by_recip(m, g6, y6) : __fdiv_rn(m, g6));
}
// E2M1 codes (2 bytes a run) of N runs of 4 values under one scale byte; m bounds their magnitudes.
template <int N>
__device__ __forceinline__ void block_codes(const float* v, float m, uint8_t s, float g, uint32_t* codes) {
    const float div = __fmul_rn(e4m3_to_f32(s), g);
#pragma unroll
    for (int i = 0; i < N; ++i) codes[i] = 0u;
    if (!(div > 0.f)) return;
    const float y = __frcp_rn(div);
    if (div >= 0x1p-96f && div <= 0x1p96f && m * y <= 0x1p60f) {
#pragma unroll
        for (int j = 0; j < 2 * N; ++j) {
            const float2 qv = div_by_recip2(make_float2(v[2 * j], v[2 * j + 1]), div, y);
            codes[j / 2] |= e2m1x2_rne_sat(qv.x, qv.y) << (8 * (j & 1));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2 * N; ++j)
            codes[j / 2] |= e2m1x2_rne_sat(__fdiv_rn(v[2 * j], div), __fdiv_rn(v[2 * j + 1], div)) << (8 * (j & 1));
    }
}

// APPEND: heads are [q | k | v]; q to bf16 rows, k and v to the cache.  Otherwise [q | k] to rows of Y.
template <typename X, typename Y, int D, int TURN, bool APPEND>
__global__ void __launch_bounds__(kRopeWarps * 32) qk_rope_kernel(const RopeArgs a) {
    constexpr int LPH = D / 8, HPW = 32 / LPH;         // lanes a head, heads a warp at once
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t item = blockIdx.x * kRopeWarps + warp;  // below 2^30: 2^20 tokens of 2 x 128 + 2 x 256 warps at most
    const int64_t t = item / (uint32_t)a.chunks;
    if (t >= a.T) return;
    // this warp's heads: chunks of queries, then of keys, then of values
    int c = (int)(item - (uint32_t)t * (uint32_t)a.chunks);
    constexpr int KVH = APPEND ? kQuantHeadsPerWarp : kHeadsPerWarp;
    const int cq = APPEND && !a.q ? 0 : (a.Hq + kHeadsPerWarp - 1) / kHeadsPerWarp, ck = (a.Hkv + KVH - 1) / KVH;
    const int kind = c < cq ? 0 : c < cq + ck ? 1 : 2;
    c -= kind == 0 ? 0 : kind == 1 ? cq : cq + ck;
    const int heads = kind == 0 ? a.Hq : a.Hkv, base = kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + a.Hkv;
    const int sub = lane / LPH, l = lane % LPH;
    const bool turn = kind < 2 && l < a.rot / 8;  // this lane's values are rotated
    const bool split = TURN == kSplit && turn;            // its two runs lie half the rotated part apart
    const int d0 = split ? 4 * l : 8 * l, d1 = split ? a.rot / 2 + 4 * l : 8 * l + 4;
    const int h0 = c * (kind == 0 ? kHeadsPerWarp : KVH) + sub;  // heads h0, h0 + HPW, ..
    const X* row = reinterpret_cast<const X*>(a.x) + t * a.ldx + (int64_t)base * D;
    constexpr int N = kHeadsPerWarp / HPW, NKV = KVH / HPW;  // heads a lane
    Raw8<X> raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (h0 + i * HPW < heads && (i < NKV || kind == 0))
            raw[i].load(row + (int64_t)(h0 + i * HPW) * D, d0, d1);
        else
            raw[i].zero();
    }
    int slot = 0;
    if constexpr (APPEND) slot = a.slots[t];
    const int64_t pos = a.rot > 0 ? a.pos[t] : 0;
    const float* wp = kind == 0 ? a.qw : a.kw;
    const bool norm = kind < 2 && wp != nullptr;
    float cs[8], sn[8], w[8];
    if (norm) {
        Raw8<float> rw;
        rw.load(wp, d0, d1);
        rw.get(w);
    }
    bool bad = a.rot > 0 && (pos < 0 || pos >= a.n_pos);
    if constexpr (APPEND) {
        if (slot == -1) return;
        bad |= slot < 0 || ((int64_t)slot >> a.cache.page_log) >= a.cache.n_pages;
    }
    if (bad) {
        if (lane == 0) atomicOr(a.status, kStatusBad);
        return;
    }
    if (turn) load_turn<TURN>(a.cs + pos * a.rot, a.rot, d0, cs, sn);
    if (!APPEND || kind == 0) {
        Y* out = kind == 0 ? reinterpret_cast<Y*>(a.q) + t * a.ldq : reinterpret_cast<Y*>(a.k) + t * a.ldk;
        unsigned again = 0;  // heads whose squares leave the range of 32 bits
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[8];
            raw[i].get(v);
            const bool good = norm_rope<float, D, TURN>(v, norm, w, a.eps, turn, a.rot, d0, cs, sn);
            if (h0 + i * HPW < heads) {
                if (good) {
                    Y* dst = out + (int64_t)(h0 + i * HPW) * D;
                    store4(dst + d0, v);
                    store4(dst + d1, v + 4);
                } else {
                    again |= 1u << i;
                }
            }
        }
        // Those once more, from memory (they have not been written, also where q and k are x's own heads): the head, and the
        // root of eps, times a power of two that brings the squares into the range; the norm is the same.
        if (__any_sync(0xffffffffu, again != 0)) {
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                const bool mine = (again >> i) & 1;
                Raw8<X> one;
                if (mine)
                    one.load(row + (int64_t)(h0 + i * HPW) * D, d0, d1);
                else
                    one.zero();
                float v[8];
                one.get(v);
                const bool large = fmaxf(fmaxf(amax4(v), amax4(v + 4)), a.eps) >= 1.f;
                const unsigned larges = __ballot_sync(0xffffffffu, large) >> (sub * LPH) & ((1u << LPH) - 1);
                const float s = larges ? 0x1p-70f : 0x1p90f;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= s;
                norm_rope<float, D, TURN>(v, norm, w, a.eps * s * s, turn, a.rot, d0, cs, sn);
                if (mine) {
                    Y* dst = out + (int64_t)(h0 + i * HPW) * D;
                    store4(dst + d0, v);
                    store4(dst + d1, v + 4);
                }
            }
        }
    } else {
        const bool isv = kind == 2;
        const float g = isv ? a.cache.v_scale : a.cache.k_scale, g6 = __fmul_rn(6.0f, g), y6 = __frcp_rn(g6);
        const int off = slot & ((1 << a.cache.page_log) - 1), r = off & 15;
        auto code_at = [&](int d) { return isv ? v_code_off(D) + (d >> 4) * 128 + r * 8 + (d & 15) / 2 : r * (D / 2) + d / 2; };
        auto scale_at = [&](int d) { return isv ? v_scale_off(D) + (d >> 4) * 16 + r : k_scale_off(D) + r * (D / 16) + (d >> 4); };
#pragma unroll
        for (int i = 0; i < NKV; ++i) {
            float v[8];
            raw[i].get(v);
            if (!isv) norm_rope<double, D, TURN>(v, norm, w, a.eps, turn, a.rot, d0, cs, sn);
            // a block of 16 values: both runs of two lanes, or one run of four (the same branch for all lanes but where a
            // head is rotated in part)
            float m0 = amax4(v), m1 = amax4(v + 4);
            if (!split) m0 = m1 = fmaxf(m0, m1);
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, 1));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, 1));
            const float o0 = __shfl_xor_sync(0xffffffffu, m0, 2), o1 = __shfl_xor_sync(0xffffffffu, m1, 2);
            uint32_t code[2];
            uint8_t s0, s1;
            if (split) {
                m0 = fmaxf(m0, o0), m1 = fmaxf(m1, o1);
                s0 = block_scale(m0, g6, y6), s1 = block_scale(m1, g6, y6);
                block_codes<1>(v, m0, s0, g, code);
                block_codes<1>(v + 4, m1, s1, g, code + 1);
            } else {
                s0 = s1 = block_scale(m0, g6, y6);
                block_codes<2>(v, m0, s0, g, code);
            }
            const uint32_t c0 = code[0], c1 = code[1];
            if (h0 + i * HPW < heads) {
                uint8_t* dst = group_ptr<D>(a.cache, slot >> a.cache.page_log, h0 + i * HPW, off);
                if (split) {
                    *reinterpret_cast<uint16_t*>(dst + code_at(d0)) = (uint16_t)c0;
                    *reinterpret_cast<uint16_t*>(dst + code_at(d1)) = (uint16_t)c1;
                    if ((l & 3) == 0) dst[scale_at(d0)] = s0, dst[scale_at(d1)] = s1;
                } else {
                    *reinterpret_cast<uint32_t*>(dst + code_at(d0)) = c0 | c1 << 16;
                    if ((l & 1) == 0) dst[scale_at(d0)] = s0;
                }
            }
        }
    }
}

template <typename Y, int D>
__global__ void __launch_bounds__(256) kv_gather_kernel(Cache cache, int64_t T, const int32_t* slots, Y* k, Y* v,
                                                        unsigned* status) {
    constexpr int LPH = D / 8;
    const int per = cache.Hkv * LPH;  // lanes a token
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = (i >> 32) == 0 ? (int64_t)((uint32_t)i / (uint32_t)per) : i / per;
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
    const auto with = [&](auto d) {
        constexpr int DD = decltype(d)::value;
        if (inter)
            kv::qk_rope_kernel<X, Y, DD, kv::kInterleaved, APPEND><<<grid, block, 0, s>>>(a);
        else if (!APPEND || a.rot % 32 == 0)
            kv::qk_rope_kernel<X, Y, DD, kv::kSplit, APPEND><<<grid, block, 0, s>>>(a);
        else if constexpr (APPEND)
            kv::qk_rope_kernel<X, Y, DD, kv::kShuffled, APPEND><<<grid, block, 0, s>>>(a);
    };
    if (D == 128)
        with(cuda::std::integral_constant<int, 128>());
    else
        with(cuda::std::integral_constant<int, 64>());
    return cudaGetLastError();
}

// cache == NULL: norm and rotation only.
extern "C" cudaError_t qlin_launch_qk_rope(const qlin_kv_cache* cache, const void* x, int xdt, int64_t T, int64_t ldx,
                                           int Hq, int Hkv, int D, const qlin_qk_params* p, const int32_t* positions,
                                           const int32_t* slots, void* q, int64_t ldq, void* k, int64_t ldk, int ydt,
                                           void* ws, cudaStream_t s) {
    kv::RopeArgs a = {};
    a.x = x, a.T = T, a.ldx = ldx, a.Hq = Hq, a.Hkv = Hkv;
    const auto chunks = [](int heads, int per) { return (heads + per - 1) / per; };
    a.chunks = cache ? (q ? chunks(Hq, kv::kHeadsPerWarp) : 0) + 2 * chunks(Hkv, kv::kQuantHeadsPerWarp)
                     : chunks(Hq, kv::kHeadsPerWarp) + chunks(Hkv, kv::kHeadsPerWarp);
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
