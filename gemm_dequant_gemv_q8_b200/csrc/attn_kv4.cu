// attn_kv4.cu -- attention of single tokens and prompt chunks over the paged NVFP4 cache:
// out = softmax(scale * q K^T) V with K and V dequantized in the kernel.
//
// A warp per (query, query head): 32 tokens at a time, a token a lane, with the running maximum and sum of the
// softmax; the probabilities then go round the warp while each lane sums its D / 32 values of V.
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
    float scale_log2;  // scale * k_scale * log2(e)
    int window;
    unsigned* status;
};

template <int D>
__global__ void __launch_bounds__(128) attn_simple_kernel(const AttnArgs a) {
    constexpr int V = D / 32;
    __shared__ float qs[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y * 4 + warp, b = blockIdx.z, i = blockIdx.x;
    if (h >= a.Hq) return;
    const int64_t r0 = a.cu[b];
    const int n = a.cu[b + 1] - a.cu[b], L = a.lens[b];
    if (n < 0 || n > a.max_q || r0 < 0 || r0 + n > a.total_q || L < 0 ||
        (int64_t)L > ((int64_t)a.max_pages << a.cache.page_log)) {
        if (lane == 0) atomicOr(a.status, kStatusBad);
        return;
    }
    if (i >= n) return;
    const int p = L - n + i, kvh = h / a.G;
    const __nv_bfloat16* qr = a.q + (r0 + i) * a.ldq + (int64_t)h * D;
    for (int d = lane; d < D; d += 32) qs[warp][d] = __bfloat162float(qr[d]) * a.scale_log2;
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = 0.f;
    const int first = a.window > 0 && p - a.window + 1 > 0 ? p - a.window + 1 : 0;
    for (int t0 = first & ~15; t0 <= p; t0 += 32) {
        const int t = t0 + lane;
        float s = -INFINITY;
        const uint8_t* g = nullptr;
        if (t >= first && t <= p) {
            const int page = a.table[b * a.ldb + (t >> a.cache.page_log)];
            if (page < 0 || page >= a.cache.n_pages) {
                atomicOr(a.status, kStatusBad);
            } else {
                g = group_ptr<D>(a.cache, page, kvh, t & ((1 << a.cache.page_log) - 1));
                const int r = t & 15;
                s = 0.f;
                for (int blk = 0; blk < D / 16; ++blk) {
                    const uint2 w = *reinterpret_cast<const uint2*>(g + r * (D / 2) + blk * 8);
                    float x = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t c = e2m1x2_to_f16x2((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
                        x += fp16_bits_to_f32(c & 0xffffu) * qs[warp][blk * 16 + 2 * j];
                        x += fp16_bits_to_f32(c >> 16) * qs[warp][blk * 16 + 2 * j + 1];
                    }
                    s += x * e4m3_to_f32(g[k_scale_off(D) + r * (D / 16) + blk]);
                }
            }
        }
        float mx = s;
#pragma unroll
        for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        const float mn = fmaxf(m, mx);
        if (mn == -INFINITY) continue;
        const float f = exp2f(m - mn), e = exp2f(s - mn);
        m = mn;
        l = l * f + e;
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] *= f;
        const unsigned long long gp = (unsigned long long)g;
        for (int k = 0; k < 32; ++k) {
            const float pe = __shfl_sync(0xffffffffu, e, k);
            const uint8_t* gk = (const uint8_t*)__shfl_sync(0xffffffffu, gp, k);
            if (gk == nullptr) continue;
            const int r = (t0 + k) & 15, d = lane * V;
            const float sc = pe * e4m3_to_f32(gk[v_scale_off(D) + (d >> 4) * 16 + r]);
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                const uint32_t c = e2m1x2_to_f16x2(gk[v_code_off(D) + (d >> 4) * 128 + r * 8 + ((d & 15) + j) / 2]);
                o[j] += sc * fp16_bits_to_f32(c & 0xffffu);
                o[j + 1] += sc * fp16_bits_to_f32(c >> 16);
            }
        }
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    const float inv = l > 0.f ? a.cache.v_scale / l : 0.f;
    __nv_bfloat16* orow = a.out + (r0 + i) * a.ldo + (int64_t)h * D + lane * V;
#pragma unroll
    for (int j = 0; j < V; ++j) orow[j] = __float2bfloat16_rn(o[j] * inv);
}

}  // namespace kv
}  // namespace qlin

using namespace qlin;

extern "C" size_t qlin_attn_kv4_ws_bytes(const qlin_kv_cache* c, int B, int max_q, int Hq) {
    (void)c, (void)B, (void)max_q, (void)Hq;
    return 256;
}

extern "C" cudaError_t qlin_launch_attn_kv4(const qlin_kv_cache* c, const void* q, int64_t ldq, const int32_t* table,
                                            int64_t ldb, int max_pages, const int32_t* lens, const int32_t* cu, int B,
                                            int max_q, int64_t total_q, int Hq, float scale, int window, void* out,
                                            int64_t ldo, void* ws, cudaStream_t s) {
    kv::AttnArgs a = {};
    a.cache = kv::make_cache(c);
    a.q = (const __nv_bfloat16*)q, a.out = (__nv_bfloat16*)out;
    a.table = table, a.lens = lens, a.cu = cu, a.ldq = ldq, a.ldo = ldo, a.ldb = ldb, a.total_q = total_q;
    a.max_pages = max_pages, a.B = B, a.max_q = max_q, a.Hq = Hq, a.G = Hq / c->Hkv;
    a.scale_log2 = scale * c->k_scale * 1.4426950408889634f;
    a.window = window;
    a.status = (unsigned*)ws;
    const dim3 grid((unsigned)max_q, (unsigned)((Hq + 3) / 4), (unsigned)B);
    if (c->D == 128)
        kv::attn_simple_kernel<128><<<grid, 128, 0, s>>>(a);
    else
        kv::attn_simple_kernel<64><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}
