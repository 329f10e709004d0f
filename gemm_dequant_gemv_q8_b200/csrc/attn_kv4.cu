// attn_kv4.cu -- attention of single tokens and prompt chunks over the paged NVFP4 cache:
// out = softmax(scale * q K^T) V with K and V dequantized in the kernel.
//
// Here: few query rows of a kv head (single tokens and a few more), and the choice between this kernel and the one for
// prompt chunks (attn_chunk.cu).
#include <cuda/std/type_traits>

#include "attn_common.cuh"

namespace qlin {
namespace kv {

// ------------------------------------------------------------------------------------- few rows, a long axis
//
// One persistent launch, one CTA an SM.  The work is a list of tiles (sequence, kv head, row block, 32 tokens), cut into
// one equal contiguous range a CTA, so that a batch of any lengths keeps every SM busy to the end.
// Within a CTA the tiles go round its warps; each warp has a ring of its own, filled by bulk copies of whole groups,
// and a running maximum, sum and P V of its own.  Where a (sequence, head, row block) ends, the warps' parts are
// joined in shared memory; where it is shared between CTAs, the last of them to finish joins their parts from the
// workspace, in the order of the CTAs.
//
// A tile is S^T = K q^T, then O^T = V^T P^T, both as m16n8k16: the tokens (then the values of V) fill the 16 rows and
// up to 8 * NT query rows of one kv head the columns, so that every code is dequantized once (to its exact fp16
// product of code and scale) whatever the group size.  The order of the inner axis is free as long as both
// operands share it: for S it is the order in which a lane's 16 (8) bytes of a token's row hold the values, for P V the
// lanes' tokens are four neighbours, whose codes of one block are 32 contiguous bytes.
//
// The cache has to be read once, and is for single tokens; a call's largest sequence gives the row blocks of all, and each
// reads the context, also one without rows (32 x 2000 tokens, single tokens 32 us; with one sequence of 8 queries of four
// heads 69).  No pipe is full (ALU 50%, tensor cores 23%, HBM 42%, an instruction issued in 56% of the active cycles): the
// kernel is bound by the dequantizing arithmetic's instructions and their latencies together (one conversion a byte and one
// product a pair of values), beside some 9 us of start and end (launch, lengths and pages, the joining).  64 sequences of
// up to 8192 tokens (8 kv heads of 128, 374 MB): 104 us, 3.6 TB/s; the copies alone 67, without V's arithmetic 80,
// without K's 89.  1 x 131071 40 us
// (3.8 TB/s); 16 x 4096 ragged (heads of 64, 24 MB) 20; 1 x 1000 9.5.  Warps: 16 give 102 / 41 / 20.1 us on the first
// three (before the shares), 12 105 / 44 / 20.8, 8 114 / 47 / 21.1.
template <int D, int NT>
struct Dec {
    static constexpr int kWarps = NT == 1 ? 16 : 8;
    static constexpr int kTile = 32;  // tokens a stage
    static constexpr int kGroups = kTile / kGroup;
    static constexpr int kStageBytes = kGroups * group_bytes(D);
    static constexpr int kStages = D == 128 ? (NT == 1 ? 3 : 5) : (NT == 1 ? 5 : 9);  // 147 KB in flight
    static constexpr int kRows = 8 * NT;
    static constexpr int kSteps = D / 16;  // k-steps of S, and 16-row tiles of O^T
    static constexpr int kPad = D + 8;     // floats a row of a warp's O in its stage buffer
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kBatch = 32 / kGroups;  // tiles whose sources a warp looks up at once
    static constexpr int kQBytes = kRows * (D * 2 + 4);  // a segment's queries as fp16, and their scales
    static constexpr int kFixed = kRing + kWarps * kStages * 16 + kWarps * 8 * 8 + kWarps * 32 * 4 + 2 * kQBytes + 16;
    static constexpr int smem(int B) { return kFixed + (3 * B + 2) * 4; }
};
constexpr int kMaxDecSeqs = 256;  // sequences of a launch
// Fewest tiles that another CTA is worth (1 x 1000 tokens: 2 9.7 us, 4 9.3, 8 9.2, 16 10.4).
constexpr int kMinTiles = 8;
static_assert(Dec<128, 1>::smem(kMaxDecSeqs) <= 232448 && Dec<64, 1>::smem(kMaxDecSeqs) <= 232448 &&
                  Dec<128, 2>::smem(kMaxDecSeqs) <= 232448 && Dec<64, 2>::smem(kMaxDecSeqs) <= 232448,
              "shared memory");
static_assert(8 * Dec<128, 1>::kPad * 4 <= Dec<128, 1>::kStageBytes && 8 * Dec<64, 1>::kPad * 4 <= Dec<64, 1>::kStageBytes,
              "a warp's O of 8 rows fits a stage");

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {  // C = 0
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// A place in the list of tiles: tile i of (sequence b, head and row block hr).
struct Cursor {
    int b, hr, i, per;
};

template <int D, int NT>
__global__ void __launch_bounds__(Dec<D, NT>::kWarps * 32, 1) attn_decode_kernel(const AttnArgs a) {
    using C = Dec<D, NT>;
    constexpr int W = C::kWarps, S = C::kStages, TILE = C::kTile, NG = C::kGroups, KS = C::kSteps;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kRing);
    uint32_t* bad_groups = reinterpret_cast<uint32_t*>(bars + W * S);
    float2* red = reinterpret_cast<float2*>(bad_groups + 2 * W * S);  // [warp][8 rows] {m, l}
    uint32_t* source = reinterpret_cast<uint32_t*>(red + W * 8);  // [warp][32] the cache's groups that its next tiles are
    uint8_t* qbuf = reinterpret_cast<uint8_t*>(source + W * 32);  // [2] this segment's queries and the next one's
    int* flag = reinterpret_cast<int*>(qbuf + 2 * C::kQBytes);
    int* longest = flag + 1;  // tiles of the longest sequence's segments
    int *share = flag + 2, *place = flag + 3;  // tiles of a CTA's share, 0: equal parts; this CTA's sequence and its first CTA
    int* prefix = flag + 4;  // [B + 1] tiles of one (head, row block) before sequence b
    int *row0 = prefix + a.B + 1, *length = row0 + a.B + 1;  // [B + 1] first rows of q, [B] contexts
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int HR = a.cache.Hkv * a.RB;

    if (lane < S) mbar_init(&bars[warp * S + lane], NG);
    if (warp == 0) {
        int run = 0, most = 0, some = 0;  // tiles, the most of a sequence, sequences with any
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            int v = 0;
            if (b < a.B) {
                const Seq s = seq_of(a, b);
                if (!s.bad && s.n > 0 && s.L > 0) v = (s.L + TILE - 1) / TILE - first_tile<TILE>(a, s.n, s.L);
                row0[b + 1] = (int)s.row0 + s.n, length[b] = s.L;
                if (s.bad && blockIdx.x == 0) atomicOr(a.status, kStatusBad);
            }
            most = max(most, v);
            some += __popc(__ballot_sync(0xffffffffu, v > 0));
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, k);
                if (lane >= k) v += u;
            }
            if (b < a.B) prefix[b + 1] = run + v;
            run += __shfl_sync(0xffffffffu, v, 31);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) prefix[0] = 0, row0[0] = __ldg(a.cu), *longest = most;
        // Equal parts of the list put two segments into most CTAs where these are few: a second joining.  There, whole
        // numbers of CTAs for each segment, if shares of the equal parts' rounds of the warps (and one more where they are
        // many) allow it (8 x 2048 16.7 -> 13.5 us, 1 x 131071 41.6 -> 39.4).  The search takes 0.9 us: not where
        // it seldom finds such shares, nor for parts of less than a round (16 x 4096, 1 x 1000).
        int tiles = 0, at = -1;
        const int grid = gridDim.x;
        if ((int64_t)some * HR * 2 <= grid && run * HR > grid * W) {
            __syncwarp();
            const int least = (run * HR + grid - 1) / grid, n = (least + W - 1) / W * W + (least > 4 * W ? W : 0);
            int before = 0;
            for (int b0 = 0; b0 < a.B; b0 += 32) {
                const int b = b0 + lane, ctas = b < a.B ? (prefix[b + 1] - (b ? prefix[b] : 0) + n - 1) / n * HR : 0;
                int v = ctas;
#pragma unroll
                for (int k = 1; k < 32; k <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, v, k);
                    if (lane >= k) v += u;
                }
                const int first = before + v - ctas, me = blockIdx.x;
                const unsigned here = __ballot_sync(0xffffffffu, me >= first && me < first + ctas);
                if (here) at = __shfl_sync(0xffffffffu, b << 16 | first, __ffs(here) - 1);
                before += __shfl_sync(0xffffffffu, v, 31);
            }
            if (before <= grid) tiles = n;
        }
        if (lane == 0) *share = tiles, *place = at;
    }
    fence_mbar_init();
    __syncthreads();

    // queries that see nothing at all: rows of zeros
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (prefix[b + 1] > prefix[b]) continue;
        const Seq s = seq_of(a, b);
        if (s.bad) continue;
        for (int64_t i = threadIdx.x; i < (int64_t)s.n * a.Hq * D / 8; i += W * 32) {
            const int64_t r = i / (a.Hq * D / 8), c = i % (a.Hq * D / 8);
            *reinterpret_cast<uint4*>(a.out + (s.row0 + r) * a.ldo + c * 8) = make_uint4(0, 0, 0, 0);
        }
    }

    auto locate = [&](int64_t tile) {
        Cursor c;
        int lo = 0, hi = a.B - 1;  // the last b with prefix[b] * HR <= tile (it has tiles)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)prefix[mid] * HR <= tile) lo = mid;
            else hi = mid - 1;
        }
        c.b = lo;
        c.per = prefix[lo + 1] - prefix[lo];
        const int64_t u = tile - (int64_t)prefix[lo] * HR;
        c.hr = (int)div_small(u, c.per);
        c.i = (int)(u - (int64_t)c.hr * c.per);
        return c;
    };
    // This CTA's range of tiles: a share of one segment, or an equal part of the list.  Where every segment is at most a
    // tile a warp, the parts end with segments: no parts to join between CTAs.
    const int64_t T = (int64_t)prefix[a.B] * HR;
    const bool whole_segs = *longest <= W;
    const int64_t want = whole_segs ? (int64_t)a.B * HR : div_small(T + kMinTiles - 1, kMinTiles);
    const int P = (int)(want < gridDim.x ? want : gridDim.x);
    if (*share ? *place < 0 : (int)blockIdx.x >= P || T == 0) return;
    int64_t t0 = div_small(T * blockIdx.x, P), t1 = div_small(T * (blockIdx.x + 1), P);
    if (whole_segs) {
        t0 -= t0 < T ? locate(t0).i : 0;
        t1 -= t1 < T ? locate(t1).i : 0;
        if (t0 >= t1) return;
    }
    if (*share) {
        const int b = *place >> 16, r = (int)blockIdx.x - (*place & 0xffff), per = prefix[b + 1] - prefix[b];
        const int n = (per + *share - 1) / *share, hr = r / n, j = r - hr * n;
        const int64_t start = (int64_t)prefix[b] * HR + (int64_t)hr * per;
        t0 = start + div_small((int64_t)per * j, n), t1 = start + div_small((int64_t)per * (j + 1), n);
    }

    auto queries = [&](int b) { return row0[b + 1] - row0[b]; };
    auto skip = [&](Cursor& c, int n) {  // n tiles on; the end of the list is not reached
        c.i += n;
        while (c.i >= c.per) {
            c.i -= c.per;
            if (++c.hr == HR) {
                c.hr = 0;
                do {
                    ++c.b;
                    c.per = prefix[c.b + 1] - prefix[c.b];
                } while (c.per == 0);
            }
        }
    };

    // this warp's tiles: t0 + warp, t0 + warp + W, ..
    int mine = t1 - t0 > warp ? (int)((t1 - t0 - warp + W - 1) / W) : 0;
    int issued = 0, istage = 0;
    uint8_t* ring = smem + warp * S * C::kStageBytes;
    const unsigned heads_groups = (unsigned)a.cache.Hkv << (a.cache.page_log - 4);
    auto issue = [&]() {  // lane j copies group j of the next tile
        const int s = istage, e = issued % C::kBatch;
        if (e == 0) {
            // where the next kBatch tiles lie, a group a lane: the searches and the page table's latency once for all
            uint32_t src = 0xffffffffu;  // not seen, or a bad page: not copied, and masked
            if (issued + lane / NG < mine) {
                const Cursor c = locate(t0 + warp + (int64_t)(issued + lane / NG) * W);
                const int tok = (first_tile<TILE>(a, queries(c.b), length[c.b]) + c.i) * TILE + (lane % NG) * kGroup;
                if (tok < length[c.b] && tok + kGroup > first_seen(a, queries(c.b), length[c.b])) {
                    const int page = __ldg(a.table + c.b * a.ldb + (tok >> a.cache.page_log));
                    if (page >= 0 && page < a.cache.n_pages)
                        src = (unsigned)page * heads_groups + ((unsigned)(c.hr / a.RB) << (a.cache.page_log - 4)) +
                              ((tok & ((1 << a.cache.page_log) - 1)) >> 4);
                    else
                        atomicOr(a.status, kStatusBad);
                }
            }
            source[warp * 32 + lane] = src;
            __syncwarp();
        }
        if (lane < NG) {
            const uint32_t src = source[warp * 32 + e * NG + lane];
            uint64_t* bar = &bars[warp * S + s];
            const unsigned ok = __ballot_sync((1u << NG) - 1, src != 0xffffffffu);
            if (lane == 0) bad_groups[warp * S + s] = ~ok & ((1u << NG) - 1);
            mbar_arrive_expect_tx(bar, src != 0xffffffffu ? group_bytes(D) : 0);
            if (src != 0xffffffffu)
                bulk_g2s(ring + s * C::kStageBytes + lane * group_bytes(D), a.cache.data + (uint64_t)src * group_bytes(D),
                         group_bytes(D), bar);
        }
        __syncwarp();
        ++issued;
        istage = istage == S - 1 ? 0 : istage + 1;
    };
    Cursor seg = locate(t0);
    int64_t s0 = t0 - seg.i;  // the first tile of this (sequence, head, row block)
    int done = 0, stage = 0, phase = 0;
    bool failed = false;
    // The queries of a segment go to shared memory as fp16 (row_exponent).  A row's D / 8 lanes hold 8 values each; lane
    // (g, t) of a product later reads its values (D / 4) t + 8 w .. + 7 of row g as one 16 bytes.
    constexpr int LPR = D / 8;
    const int qr = threadIdx.x / LPR, qd = threadIdx.x % LPR * 8;
    auto load_q = [&](const Cursor& c) {
        const int rr = c.hr % a.RB * C::kRows + qr;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (qr < C::kRows && rr < queries(c.b) * a.G)
            u = __ldg(reinterpret_cast<const uint4*>(a.q + ((int64_t)row0[c.b] + group_div(a, rr)) * a.ldq +
                                                     (int64_t)(c.hr / a.RB * a.G + group_mod(a, rr)) * D + qd));
        return u;
    };
    auto store_q = [&](const uint4& u, uint8_t* to) {
        if (threadIdx.x >= (C::kRows * LPR + 31) / 32 * 32) return;
        const uint32_t raw[4] = {u.x, u.y, u.z, u.w};
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) mx = fmaxf(mx, amax_bf16x2(raw[k]));
#pragma unroll
        for (int k = LPR / 2; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        const int e = row_exponent(mx);
        const float up = row_up(e, a.scale_log2);
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = scaled_f16x2(raw[k], up);
        const int at = ((qd % (D / 4) / 8 * C::kRows + qr) * 4 + qd / (D / 4)) * 16;
        *reinterpret_cast<uint4*>(to + at) = make_uint4(h[0], h[1], h[2], h[3]);
        if (qd == 0) reinterpret_cast<float*>(to + C::kRows * D * 2)[qr] = row_down(e, a.scale_log2);
    };
    uint4 qnext = load_q(seg);  // in flight with the first copies
    // one stage stays free: the last one read, which holds the warp's O while the warps' parts are joined
    for (int k = 0; k < S - 1 && k < mine; ++k) issue();
    store_q(qnext, qbuf);
    __syncthreads();

    for (int turn = 0;; turn ^= 1) {
        const int qn = queries(seg.b), qL = length[seg.b], tile0 = first_tile<TILE>(a, qn, qL);
        const int64_t qrow = row0[seg.b];
        const int h = seg.hr / a.RB, rb = seg.hr % a.RB;
        const int rows = min(C::kRows, qn * a.G - rb * C::kRows);  // may be <= 0
        const int64_t s1 = s0 + seg.per;
        const uint8_t* qs = qbuf + turn * C::kQBytes;
        float rs[NT][2], m[NT][2], l[NT][2];  // rs takes the scores to the exponents of 2
        int hi[NT][2];
        float o[KS][NT][4];
        // this warp's tiles of the segment: every W-th from `next`
        const int64_t next = t0 + warp + (int64_t)done * W, end = s1 < t1 ? s1 : t1;
        const int tiles = next < end ? (int)((end - next + W - 1) / W) : 0;
        const bool any = tiles > 0;
        float nref[NT][2];  // what is added to the exponents: -m (m the reference), 0 where nothing has been seen
        bool huge = false;  // some |m| of the warp is 2^20 or more
        if (any) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = nt * 8 + 2 * t + c;
                    rs[nt][c] = reinterpret_cast<const float*>(qs + C::kRows * D * 2)[r];
                    hi[nt][c] = qL - qn + group_div(a, rb * C::kRows + r);  // the last place that the column's query sees
                    m[nt][c] = -INFINITY;
                    l[nt][c] = nref[nt][c] = 0.f;
                }
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[i][nt][c] = 0.f;
        }
        int tok0 = (tile0 + (int)(next - s0)) * TILE;
        for (int j = 0; j < tiles; ++j, tok0 += W * TILE) {
            const int s = stage;
            if (failed && done >= issued) break;
            // the warp goes on, or gives up, as one
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&bars[warp * S + s], phase, failed ? 50000000ull : 2000000000ull))) {
                if (lane == 0) atomicOr(a.status, 1u);
                failed = true;
                mine = issued;  // nothing more is copied; what is in flight is waited for
            }
            const uint8_t* st = ring + s * C::kStageBytes;
            const uint32_t bad = bad_groups[warp * S + s];
            // every row sees all of the tile's tokens, unless the tile reaches past the first row's place or
            // before the last one's window: the common form has no masks at all
            auto step = [&](auto masked) {
                constexpr bool edge = decltype(masked)::value;
                // S^T: rows g and g + 8 of a group's 16 are its tokens ta and ta + 2
                const int ta = 4 * (g >> 1) + (g & 1);
                constexpr int WK = D / 32;  // words of codes a lane has of a token
                float sc[NG][NT][4];
                uint32_t w0[NG][WK], w1[NG][WK], f0[NG][D / 64], f1[NG][D / 64];
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    const uint8_t* gp = st + gr * group_bytes(D);
                    if constexpr (D == 128) {
                        const uint4 x = *reinterpret_cast<const uint4*>(gp + ta * 64 + t * 16);
                        const uint4 y = *reinterpret_cast<const uint4*>(gp + (ta + 2) * 64 + t * 16);
                        w0[gr][0] = x.x, w0[gr][1] = x.y, w0[gr][2] = x.z, w0[gr][3] = x.w;
                        w1[gr][0] = y.x, w1[gr][1] = y.y, w1[gr][2] = y.z, w1[gr][3] = y.w;
                        const uint32_t z0 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(gp + k_scale_off(D) + ta * 8 + t * 2));
                        const uint32_t z1 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(gp + k_scale_off(D) + (ta + 2) * 8 + t * 2));
                        f0[gr][0] = __byte_perm(z0, 0, 0x1010), f0[gr][1] = __byte_perm(z0, 0, 0x3232);
                        f1[gr][0] = __byte_perm(z1, 0, 0x1010), f1[gr][1] = __byte_perm(z1, 0, 0x3232);
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2*>(gp + ta * 32 + t * 8);
                        const uint2 y = *reinterpret_cast<const uint2*>(gp + (ta + 2) * 32 + t * 8);
                        w0[gr][0] = x.x, w0[gr][1] = x.y;
                        w1[gr][0] = y.x, w1[gr][1] = y.y;
                        const uint32_t z = e4m3x2_to_f16x2((uint32_t)gp[k_scale_off(D) + ta * 4 + t] |
                                                           (uint32_t)gp[k_scale_off(D) + (ta + 2) * 4 + t] << 8);
                        f0[gr][0] = __byte_perm(z, 0, 0x1010), f1[gr][0] = __byte_perm(z, 0, 0x3232);
                    }
                }
#pragma unroll
                for (int w = 0; w < WK; ++w) {  // a word of codes: two steps of the inner axis
                    uint4 qf[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) qf[nt] = *reinterpret_cast<const uint4*>(qs + ((w * C::kRows + nt * 8 + g) * 4 + t) * 16);
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) {
                        uint32_t h0[4], h1[4];
                        e2m1x8(w0[gr][w], h0);
                        e2m1x8(w1[gr][w], h1);
#pragma unroll
                        for (int c = 0; c < 4; ++c) h0[c] = hmul2(h0[c], f0[gr][w / 2]), h1[c] = hmul2(h1[c], f1[gr][w / 2]);
                        const uint32_t a0[4] = {h0[0], h1[0], h0[1], h1[1]}, a1[4] = {h0[2], h1[2], h0[3], h1[3]};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (w == 0)
                                mma16816_zero(sc[gr][nt], a0, qf[nt].x, qf[nt].y);
                            else
                                mma16816(sc[gr][nt], a0, qf[nt].x, qf[nt].y);
                            mma16816(sc[gr][nt], a1, qf[nt].z, qf[nt].w);
                        }
                    }
                }
                if constexpr (edge) {
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const int tok = tok0 + gr * kGroup + ta + (c & 2);
                                const bool sees = tok <= hi[nt][c & 1] && tok < qL && !((bad >> gr) & 1) &&
                                                  (a.window == 0 || tok > hi[nt][c & 1] - a.window);
                                sc[gr][nt][c] = sees ? sc[gr][nt][c] : -INFINITY;
                            }
                }
                // The maximum goes round the lanes, and O is rescaled, only where the reference has to follow it (kGrow).  The
                // growth is the difference, exact where it matters: a sum would be rounded up where scores are large.
                float mx[NT][2];
                bool grow = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v = fmaxf(sc[0][nt][c], sc[0][nt][2 + c]);
#pragma unroll
                        for (int gr = 1; gr < NG; ++gr) v = fmaxf(v, fmaxf(sc[gr][nt][c], sc[gr][nt][2 + c]));
                        mx[nt][c] = v;
                        grow |= __fsub_rn(__fmul_rn(v, rs[nt][c]), m[nt][c]) > kGrow;
                    }
                if (__any_sync(0xffffffffu, grow)) {
                    bool big = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float f[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float v = mx[nt][c];
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                            const float mn = fmaxf(m[nt][c], v == -INFINITY ? v : __fsub_rn(__fmul_rn(v, rs[nt][c]), kBelow));
                            f[c] = m[nt][c] == -INFINITY ? 0.f : ex2(m[nt][c] - mn);
                            m[nt][c] = mn;
                            nref[nt][c] = mn == -INFINITY ? 0.f : -mn;
                            big |= fabsf(nref[nt][c]) >= 0x1p20f;
                            l[nt][c] *= f[c];
                        }
#pragma unroll
                        for (int i = 0; i < KS; ++i)
#pragma unroll
                            for (int c = 0; c < 4; ++c) o[i][nt][c] *= f[c & 1];
                    }
                    huge = __any_sync(0xffffffffu, big);
                }
                // One rounding leaves up to half an ulp of the largest score on its exponent, at most 2^-4 below 2^20, the
                // same for the whole row; beyond that two, as the reference has, leave none.
                float p[NG][NT][4];
                if (edge || huge) {
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const float e = ex2(__fadd_rn(__fmul_rn(sc[gr][nt][c], rs[nt][c & 1]), nref[nt][c & 1]));
                                p[gr][nt][c] = sc[gr][nt][c] == -INFINITY ? 0.f : e;  // also where rs is 0
                            }
                } else {
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 4; ++c) p[gr][nt][c] = ex2(fmaf(sc[gr][nt][c], rs[nt][c & 1], nref[nt][c & 1]));
                }
                uint32_t pf[NG][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) {
                        const float* e = p[gr][nt];
                        l[nt][0] += e[0] + e[2];
                        l[nt][1] += e[1] + e[3];
                        // tokens to rows, heads to columns: the transpose is the operand that P V takes
                        pf[gr][nt][0] = transpose8x8(pack_f16x2(e[0], e[1]));
                        pf[gr][nt][1] = transpose8x8(pack_f16x2(e[2], e[3]));
                    }
                // O^T: this lane's tokens of a group are 4 t .. 4 t + 3; row g (g + 8) of tile i is its value 2 i (2 i + 1)
                // of D / 8 neighbouring values
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    const uint8_t* gp = st + gr * group_bytes(D);
                    constexpr int VW = D / 64;  // words of codes a token
                    const int blk = D == 128 ? g : g >> 1;
                    uint32_t v[4][VW];
                    if constexpr (D == 128) {
                        const uint4 x = *reinterpret_cast<const uint4*>(gp + v_code_off(D) + blk * 128 + t * 32);
                        const uint4 y = *reinterpret_cast<const uint4*>(gp + v_code_off(D) + blk * 128 + t * 32 + 16);
                        v[0][0] = x.x, v[0][1] = x.y, v[1][0] = x.z, v[1][1] = x.w;
                        v[2][0] = y.x, v[2][1] = y.y, v[3][0] = y.z, v[3][1] = y.w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[k][0] = *reinterpret_cast<const uint32_t*>(gp + v_code_off(D) + blk * 128 + t * 32 + k * 8 + (g & 1) * 4);
                    }
                    uint32_t vs = *reinterpret_cast<const uint32_t*>(gp + v_scale_off(D) + blk * 16 + t * 4);
                    if constexpr (edge) {  // places that no query sees hold anything: scale 0, so that 0 * value is 0
                        const int left = (bad >> gr) & 1 ? 0 : qL - (tok0 + gr * kGroup + 4 * t);
                        vs = left >= 4 ? vs : left <= 0 ? 0u : vs & ((1u << (8 * left)) - 1u);
                        const int before = first_seen(a, qn, qL) - (tok0 + gr * kGroup + 4 * t);
                        vs = before <= 0 ? vs : before >= 4 ? 0u : vs & ~((1u << (8 * before)) - 1u);
                    }
                    const uint32_t f01 = e4m3x2_to_f16x2(vs & 0xffffu), f23 = e4m3x2_to_f16x2(vs >> 16);
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        constexpr uint32_t lo = 0x0f0f0f0fu;
                        uint32_t x01[4], y01[4], x23[4], y23[4];
                        e2m1x8((v[0][w] & lo) | ((v[1][w] << 4) & ~lo), x01);
                        e2m1x8(((v[0][w] >> 4) & lo) | (v[1][w] & ~lo), y01);
                        e2m1x8((v[2][w] & lo) | ((v[3][w] << 4) & ~lo), x23);
                        e2m1x8(((v[2][w] >> 4) & lo) | (v[3][w] & ~lo), y23);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t af[4] = {hmul2(x01[i], f01), hmul2(y01[i], f01), hmul2(x23[i], f23), hmul2(y23[i], f23)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16816(o[4 * w + i][nt], af, pf[gr][nt][0], pf[gr][nt][1]);
                        }
                    }
                }
            };
            if (bad != 0 || tok0 + TILE - 1 > qL - qn || (a.window > 0 && tok0 <= qL - 1 - a.window))
                step(cuda::std::true_type());
            else
                step(cuda::std::false_type());
            ++done;
            if (++stage == S) stage = 0, phase ^= 1;
            __syncwarp();
            if (issued < mine) issue();  // into the stage that was read before this one
        }

        // the next segment's queries: in flight while this one's parts are joined
        const bool last = s1 >= t1;
        if (!last) {
            seg.i = 0;
            skip(seg, seg.per);
            qnext = load_q(seg);
        }
        // join the warps' parts, 8 rows at a time, in the order of the warps
        int c0 = 0, c1 = 0;  // the CTAs that have tiles of the segment
        if (*share) {
            const int n = (seg.per + *share - 1) / *share;
            c0 = (*place & 0xffff) + seg.hr * n, c1 = c0 + n - 1;
        } else if (!whole_segs) {
            c0 = (int)div_small((s0 + 1) * P - 1, T), c1 = (int)div_small(s1 * P - 1, T);
        }
        const bool whole = c0 == c1;
        float* part = a.parts + (int64_t)(2 * blockIdx.x + ((int)blockIdx.x == c0)) * C::kRows * (D + 2);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float* mo = reinterpret_cast<float*>(ring + (stage ? stage - 1 : S - 1) * C::kStageBytes);
            if (any) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = l[nt][c];
                    v += __shfl_xor_sync(0xffffffffu, v, 4);
                    v += __shfl_xor_sync(0xffffffffu, v, 8);
                    v += __shfl_xor_sync(0xffffffffu, v, 16);
                    if (g == 0) red[warp * 8 + 2 * t + c] = make_float2(m[nt][c], v);
#pragma unroll
                    for (int i = 0; i < KS; ++i) {  // the pair of values (KS g + i), its place among 8 (4) turned by g
                        const int at = KS * g + (i ^ (g & (KS - 1)));
                        *reinterpret_cast<float2*>(mo + (2 * t + c) * C::kPad + 2 * at) = make_float2(o[i][nt][c], o[i][nt][2 + c]);
                    }
                }
            } else if (lane < 8) {
                red[warp * 8 + lane] = make_float2(-INFINITY, 0.f);
            }
            // where each warp's buffer lies: a warp without a tile of its own is not read
            if (lane == 0) bad_groups[W * S + warp] = (uint32_t)(stage ? stage - 1 : S - 1);
            __syncthreads();
            for (int e = threadIdx.x; e < 8 * D / 2; e += W * 32) {
                const int r = e / (D / 2), pair = e % (D / 2);
                if (nt * 8 + r >= rows) break;
                const int pg = pair / KS, at = KS * pg + ((pair % KS) ^ (pg & (KS - 1)));
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < W; ++w) M = fmaxf(M, red[w * 8 + r].x);
                const float top = M == -INFINITY ? 0.f : M;
                float2 acc = make_float2(0.f, 0.f);
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float2 ml = red[w * 8 + r];
                    float2 v = *reinterpret_cast<const float2*>(
                        smem + (w * S + bad_groups[W * S + w]) * C::kStageBytes + (r * C::kPad + 2 * at) * 4);
                    const float f = ex2(ml.x - top);
                    if (f == 0.f) v = make_float2(0.f, 0.f);  // also a buffer that holds something else
                    acc.x += f * v.x, acc.y += f * v.y;
                    sum += f * ml.y;
                }
                if (whole) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    const int rr = rb * C::kRows + nt * 8 + r;
                    *reinterpret_cast<__nv_bfloat162*>(a.out + (qrow + group_div(a, rr)) * a.ldo +
                                                       (int64_t)(h * a.G + group_mod(a, rr)) * D + 2 * pair) =
                        out_pair(a, acc.x, acc.y, inv);
                } else {
                    __stcg(reinterpret_cast<float2*>(part + (nt * 8 + r) * D + 2 * pair), acc);
                    if (pair == 0) __stcg(reinterpret_cast<float2*>(part + C::kRows * D + 2 * (nt * 8 + r)), make_float2(M, sum));
                }
            }
            __syncthreads();
        }
        if (!whole) {
            // the last CTA of this (sequence, head, row block) to come here joins the CTAs' parts
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                const int before = atomicAdd(&a.tickets[c0], 1);
                *flag = before == c1 - c0;
                if (*flag) a.tickets[c0] = 0;  // everyone has come: zero for the next call
                __threadfence();
            }
            __syncthreads();
            if (*flag) {
                // a row a warp; where the rows are fewer than the warps, each takes every nsp-th part of its row
                constexpr int V = D / 32;  // values a lane
                const int64_t psz = (int64_t)C::kRows * (D + 2);
                int rp = 1;
                while (rp < rows && rp < W) rp *= 2;
                const int nsp = W / rp, sp = warp / rp;
                float* mo = reinterpret_cast<float*>(ring + (stage ? stage - 1 : S - 1) * C::kStageBytes);
                for (int r = warp % rp; r < C::kRows; r += rp) {
                    float M = -INFINITY, sum = 0.f, acc[V];
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[k] = 0.f;
                    if (r < rows) {
                        constexpr int U = 4;  // parts in flight
                        for (int c = c0 + sp; c <= c1; c += U * nsp) {
                            float2 ml[U], v[U][V / 2];
#pragma unroll
                            for (int u = 0; u < U; ++u) {
                                const int cu = c + u * nsp;
                                ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
                                for (int k = 0; k < V / 2; ++k) v[u][k] = make_float2(0.f, 0.f);
                                if (cu > c1) continue;
                                const float* p = a.parts + (2 * cu + (cu == c0)) * psz;
                                ml[u] = __ldcg(reinterpret_cast<const float2*>(p + C::kRows * D + 2 * r));
#pragma unroll
                                for (int k = 0; k < V / 2; ++k)
                                    v[u][k] = __ldcg(reinterpret_cast<const float2*>(p + r * D + lane * V + 2 * k));
                            }
                            float mn = M;
#pragma unroll
                            for (int u = 0; u < U; ++u) mn = fmaxf(mn, ml[u].x);
                            const float top = mn == -INFINITY ? 0.f : mn, f0 = ex2(M - top);
                            M = mn;
                            sum *= f0;
#pragma unroll
                            for (int k = 0; k < V; ++k) acc[k] *= f0;
#pragma unroll
                            for (int u = 0; u < U; ++u) {
                                const float f = ex2(ml[u].x - top);
                                sum += f * ml[u].y;
#pragma unroll
                                for (int k = 0; k < V / 2; ++k)
                                    acc[2 * k] += f * v[u][k].x, acc[2 * k + 1] += f * v[u][k].y;
                            }
                        }
                    }
                    if (nsp > 1) {
                        if (lane == 0) red[warp] = make_float2(M, sum);
#pragma unroll
                        for (int k = 0; k < V; ++k) mo[lane * V + k] = acc[k];
                        __syncthreads();
                        if (sp == 0 && r < rows) {
                            float mn = M;
                            for (int w = warp + rp; w < W; w += rp) mn = fmaxf(mn, red[w].x);
                            const float top = mn == -INFINITY ? 0.f : mn, f0 = ex2(M - top);
                            sum *= f0;
#pragma unroll
                            for (int k = 0; k < V; ++k) acc[k] *= f0;
                            for (int w = warp + rp; w < W; w += rp) {
                                const float f = ex2(red[w].x - top);
                                const float* p = reinterpret_cast<const float*>(smem + (w * S + bad_groups[W * S + w]) * C::kStageBytes);
                                sum += f * red[w].y;
#pragma unroll
                                for (int k = 0; k < V; ++k) acc[k] += f * p[lane * V + k];
                            }
                        }
                        __syncthreads();
                    }
                    if (sp == 0 && r < rows) {
                        const float inv = sum == 0.f ? 0.f : 1.f / sum;
                        const int rr = rb * C::kRows + r;
                        __nv_bfloat16* dst = a.out + (qrow + group_div(a, rr)) * a.ldo + (int64_t)(h * a.G + group_mod(a, rr)) * D + lane * V;
#pragma unroll
                        for (int k = 0; k < V; k += 2)
                            *reinterpret_cast<__nv_bfloat162*>(dst + k) = out_pair(a, acc[k], acc[k + 1], inv);
                    }
                }
            }
        }
        if (last) break;
        store_q(qnext, qbuf + (turn ^ 1) * C::kQBytes);
        // the joining wrote stages that bulk copies fill next
        fence_proxy_async_smem();
        __syncthreads();
        s0 = s1;
    }
}

}  // namespace kv
}  // namespace qlin

using namespace qlin;

extern "C" size_t qlin_attn_chunk_part_bytes(int D, int sms);
extern "C" cudaError_t qlin_launch_attn_chunk(const kv::AttnArgs* a, int D, int sms, cudaStream_t s);

static int kv_sm_count() {
    static int cached[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (cached[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cached[dev] = n < kv::kMaxParts ? n : kv::kMaxParts;
    }
    return cached[dev];
}

// Whether the kernel for few rows takes a call.  It goes over the cache once for every 16 query rows of a kv head, but
// spreads any context over all SMs; the one for chunks goes over it once for 256, in units of at least 128 rows.  us, few
// rows against chunks: 1 x 8000 tokens (8 kv heads) 64 rows 28 / 47, 128 rows 38 / 49; 8 x 2000 32 rows 27 / 34, 64 rows
// 41 / 34; 32 x 4000 32 rows 117 / 167, 64 rows 216 / 168.  max_q decides for the whole call: single tokens beside a prompt
// chunk go the chunks' way (31 of 4000 and a chunk of 512 153 us; in two calls 44 and 20).
static bool few_rows(int64_t rows, int B, int Hkv) {
    return rows <= 32 || (rows <= 128 && rows * B * Hkv <= 2048);
}

extern "C" size_t qlin_attn_kv4_ws_bytes(const qlin_kv_cache* c, int B, int max_q, int Hq) {
    const int64_t rows = (int64_t)max_q * (Hq / c->Hkv);
    const size_t fixed = 256 + kv::kMaxParts * 4;
    if (!few_rows(rows, B, c->Hkv)) return fixed + qlin_attn_chunk_part_bytes(c->D, kv_sm_count());
    return fixed + (size_t)2 * kv_sm_count() * (rows <= 8 ? 8 : 16) * (c->D + 2) * 4;
}

template <int D, int NT>
static cudaError_t launch_decode(kv::AttnArgs a, cudaStream_t s) {
    using C = kv::Dec<D, NT>;
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev]) {
        e = cudaFuncSetAttribute(kv::attn_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::smem(kv::kMaxDecSeqs));
        if (e != cudaSuccess) return e;
        set[dev] = true;
    }
    const int sms = kv_sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    for (int left = a.B; left > 0; left -= kv::kMaxDecSeqs) {
        a.B = left < kv::kMaxDecSeqs ? left : kv::kMaxDecSeqs;
        kv::attn_decode_kernel<D, NT><<<sms, C::kWarps * 32, C::smem(a.B), s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        a.table += a.B * a.ldb, a.lens += a.B, a.cu += a.B;
    }
    return cudaSuccess;
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
    a.g_magic = a.G == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + a.G - 1) / a.G);
    a.scale_log2 = scale * c->k_scale * 1.4426950408889634f;
    a.window = window < (1 << 30) ? window : 0;  // no context is longer
    a.status = (unsigned*)ws;
    a.tickets = (int*)((uint8_t*)ws + 256);
    a.parts = (float*)((uint8_t*)ws + 256 + kv::kMaxParts * 4);
    const int64_t rows = (int64_t)max_q * a.G;
    if (!few_rows(rows, B, c->Hkv)) return qlin_launch_attn_chunk(&a, c->D, kv_sm_count(), s);
    a.RB = rows <= 8 ? 1 : (int)((rows + 15) / 16);
    if (c->D == 128) return rows <= 8 ? launch_decode<128, 1>(a, s) : launch_decode<128, 2>(a, s);
    return rows <= 8 ? launch_decode<64, 1>(a, s) : launch_decode<64, 2>(a, s);
}
