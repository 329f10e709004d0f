// attn_chunk.cu -- attention of prompt chunks over the paged NVFP4 cache on the 5th-generation tensor cores.
//
// A unit is 256 query rows of one (sequence, kv head): row r is query r / G, head r % G of the group, so that every
// group size fills the tiles and K and V are dequantized once for all heads that share them.  A CTA (one an SM) works
// on a unit's two tiles of 128 rows against 128 tokens at a time, tcgen05.mma kind::f16 with fp32 accumulators in tensor
// memory:
//   warps 0-3, 4-7: softmax of tile A and of tile B, a row a thread: scores from tensor memory, once for their maximum
//                   and once for the exponentials, probabilities back as the fp16 A operand of P V (in the scores'
//                   columns); they also bring the queries in (fp16, row_exponent) and take O out;
//   warps 8-11    : dequantize K, a token a thread, and V, 16 values x 8 tokens a thread, into 128-byte-swizzled K-major
//                   tiles [token][value] and [value][token] in two stages each, with the next tile's codes on their way
//                   into registers and the pages after that looked up;
//   warp 12       : issues the products, S_A, S_B, then per tile of tokens P V of A, the next S_A, P V of B, the
//                   next S_B: the tensor cores work for one tile while the other's softmax runs;
//   warp 13       : deals out the units: a ring of descriptions in shared memory that the others read
//                   (warps 14 and 15 are idle: registers are dealt out by four warps).
// The exponents' reference follows the running maximum only when that has grown by 2^8 (kBelow, kGrow), so O is rarely
// rescaled.
//
// 2 x 2047 queries of 8189 tokens (32 heads of 128): 371 us, 886 TFLOP/s; 8192 of 8192: 594 us, 926 TFLOP/s.  The bound is
// the chain of a tile of rows: 1.55 us of softmax, then 0.8 us until its next scores are there (measured at 381 us),
// while the tensor cores have 1.1 us of work and the special function units as much for both tiles; two tiles (scores
// and O: 512 columns) fill tensor memory.  No unit is full (issue 48%, special functions 43%, tensor cores 43% of the
// cycles).  Two threads a row (493 us), scores in halves of 64 (485) and exponentials by polynomial for a part of the
// scores (384 to 410) were slower than 381.
// Units are dealt out there and back, sequences as they stand and in each the heaviest first (a long prompt behind a short
// one costs: 512 of 512, then 2047 of 8189 346 us, the other way round 283); those of the last, partial round are split
// along the tokens where that shortens it, and the last CTA of a unit to finish joins its parts in their order.
// Every wait is bounded; a timeout sets the status word and the CTA winds down.
#include <cuda/std/type_traits>

#include "attn_common.cuh"

namespace qlin {
namespace kv {

namespace ch {

constexpr int kRows = 256, kTok = 128;  // rows of a unit at most, tokens of a tile

constexpr int kSoftWarps = 8, kDqWarps = 4, kMmaWarp = kSoftWarps + kDqWarps;
constexpr int kThreads = (kMmaWarp + 4) * 32;
// Registers a thread: 128 at launch (512 threads), then by role.  The softmax warps wait for what the others give back, so
// every other role has its dec, and the shares add up to the launch's at most.
constexpr int kSoftRegs = 152, kDqRegs = 112, kMmaRegs = 96;
static_assert(kDqRegs < 128 && kMmaRegs < 128 && 256 * kSoftRegs + 128 * kDqRegs + 128 * kMmaRegs <= 512 * 128,
              "the launch's registers");
constexpr int kMaxSeqs = 1024;
// Descriptions in the ring.  The dequantizing warps take up to two tiles' pieces beyond the one that the softmax warps work
// on, and the empty ones between them, which is no more than the last round's two parts and the end mark: five in all.
constexpr int kItems = 8;
// What a unit costs beside its tiles, and what joining its parts does, in tiles (2.4 us): queries in and rows out; the parts'
// way through the workspace; reading one (131 KB at what an SM gets).
constexpr float kUnitCost = 2.f, kJoinCost = 1.5f, kPartCost = 0.3f;

template <int D>
struct Cfg {
    static constexpr int kQBytes = 128 * D * 2;  // one tile of queries
    static constexpr int kKBytes = kTok * D * 2, kVBytes = kTok * D * 2;
    static constexpr int kSmem = 1024 + 2 * kQBytes + 2 * kKBytes + 2 * kVBytes + 512 + kItems * 64;
    static constexpr int smem(int B) { return kSmem + (3 * B + 2) * 4; }
};
static_assert(Cfg<128>::smem(kMaxSeqs) <= 232448, "shared memory");

// The low word of a shared-memory descriptor (address, unused leading offset); the high word is the same for every
// operand here: 8-row groups 1024 bytes apart, the sm_100 version, 128-byte swizzle (K-major).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3fffu) | (1u << 16); }
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// One thread of the converged warp issues; the operands are the same in all of it, so they stay in uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 da, db;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
        " setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate),
        "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 db;\n mov.b64 db, {%2, %5};\n"
        " setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accumulate),
        "n"(kDescHi)
        : "memory");
}
// Commits the elected thread's products: elect.sync picks the same thread each time.
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* r) {  // complete after ld_wait
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// The wait names the registers, so that nothing reads them before it.
__device__ __forceinline__ void ld_wait(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
        "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A piece of work: 256 rows of one (sequence, kv head) from row `base`, tiles [t0, t1) of 128 tokens.
struct Item {
    int b, h, base, rows, n, L, t0, t1;
    int64_t row0;
    int first;        // the first place that its first row sees
    int part, parts;  // part of a unit that several CTAs share (parts > 1)
    int tail;         // its number among the shared ones
};
static_assert(sizeof(Item) <= 64, "an item's slot");

}  // namespace ch

template <int D>
__global__ void __launch_bounds__(ch::kThreads, 1) attn_chunk_kernel(const AttnArgs a) {
    using namespace ch;
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* qt = smem;
    uint8_t* kt = qt + 2 * C::kQBytes;
    uint8_t* vt = kt + 2 * C::kKBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(vt + 2 * C::kVBytes);
    uint64_t *qfull = bars, *kfull = bars + 2, *kfree = bars + 4, *vfull = bars + 6, *vfree = bars + 8, *sfull = bars + 10,
             *pfull = bars + 12, *ofull = bars + 14, *mma_done = bars + 16;
    uint8_t* bad = reinterpret_cast<uint8_t*>(bars + 17);  // [4][8]: groups of a tile that a bad page leaves out
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 21);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    int* last_flag = reinterpret_cast<int*>(tmem_holder + 2);
    int* unit_rows = last_flag + 1;
    uint64_t *itemfull = bars + 28, *itemfree = itemfull + kItems, *softbar = itemfree + kItems;
    Item* ring = reinterpret_cast<Item*>(bars + 64);
    int* prefix = reinterpret_cast<int*>(ring + kItems);  // [B + 1] units of one kv head before sequence b
    int *row0 = prefix + a.B + 1, *length = row0 + a.B + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qfull[i], 4);
            mbar_init(&kfull[i], kDqWarps * 32);
            mbar_init(&vfull[i], kDqWarps * 32);
            mbar_init(&kfree[i], 1);
            mbar_init(&vfree[i], 1);
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);
            mbar_init(&ofull[i], 1);
        }
        mbar_init(mma_done, 1);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&itemfull[i], 1);
            mbar_init(&itemfree[i], kSoftWarps + kDqWarps + 1);
        }
        mbar_init(softbar, kSoftWarps);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_holder)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (warp == 0) {
        // Where units of 256 rows would leave half of the SMs without one, units of one tile of rows.
        int big = 0;
        for (int b = lane; b < a.B; b += 32) {
            const Seq s = seq_of(a, b);
            if (!s.bad) big += (int)(((int64_t)s.n * a.G + kRows - 1) / kRows);
        }
        big = __reduce_add_sync(0xffffffffu, big);
        const int ur = (int64_t)big * a.cache.Hkv * 2 <= gridDim.x ? kRows / 2 : kRows;
        if (lane == 0) *unit_rows = ur;
        int run = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            int v = 0;
            if (b < a.B) {
                const Seq s = seq_of(a, b);
                if (!s.bad) v = (int)(((int64_t)s.n * a.G + ur - 1) / ur);
                row0[b + 1] = (int)s.row0 + s.n, length[b] = s.L;
                if (s.bad && blockIdx.x == 0) atomicOr(a.status, kStatusBad);
            }
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, k);
                if (lane >= k) v += u;
            }
            if (b < a.B) prefix[b + 1] = run + v;
            run += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) prefix[0] = 0, row0[0] = __ldg(a.cu);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_holder;

    auto wait = [&](uint64_t* bar, int parity) {  // false: gave up, or another warp has
        if (*abort_flag) return false;
        if (mbar_wait_bounded(bar, parity)) return true;
        atomicOr(a.status, 1u);
        *abort_flag = 1;
        return false;
    };
    auto warp_wait = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    auto warp_arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) arrive(bar);
    };
    // A role's k-th piece of work; false at the end.  done(k) gives its place in the ring back.
    auto take = [&](int k) { return warp_wait(&itemfull[k % kItems], (k / kItems) & 1) && ring[k % kItems].b >= 0; };
    auto done_with = [&](int k) { warp_arrive(&itemfree[k % kItems]); };

    if (warp < kSoftWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int x = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane, srow = x * 128 + row;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t ts = tmem + lanes + x * 128, to = tmem + lanes + 256 + x * D;
        uint8_t* qx = qt + x * C::kQBytes;
        int tiles = 0, its = 0;  // of this tile of rows so far: the barriers' phases
        int soft_syncs = 0;
        bool ok = true;          // after a wait that gave up: no more work
        int all_tiles = 0;       // of the CTA: the bad groups' ring
        auto soft_sync = [&]() {  // the eight warps
            warp_arrive(softbar);
            ok = warp_wait(softbar, soft_syncs & 1) && ok;
            ++soft_syncs;
        };
        for (int k = 0; ok && take(k); done_with(k), ++k) {
            const Item& it = ring[k % kItems];
            const int cnt = it.t1 - it.t0, first = it.t0;
            const int p = it.L - it.n + group_div(a, it.base + srow);  // the last place this row sees
            // of this warp's rows: the first one's and the last one's
            const int pw0 = it.L - it.n + group_div(a, it.base + x * 128 + quarter * 32);
            const int pw1 = it.L - it.n + group_div(a, it.base + x * 128 + quarter * 32 + 31);
            float rs = 0.f, m = -INFINITY, l = 0.f;
            const bool active = x * 128 < it.rows && cnt > 0;
            if (active) {
                // This warp's 32 rows of queries as fp16, 16-byte pieces of 128-byte rows turned by the row: D / 8 lanes a row,
                // so that a load is whole rows.
                constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes a row, rows a load
#pragma unroll 1
                for (int h0 = 0; h0 < 32; h0 += 8 * RPI) {
                    uint4 u[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int wr = quarter * 32 + h0 + i * RPI + lane / LPR, rr = it.base + x * 128 + wr;
                        u[i] = make_uint4(0, 0, 0, 0);
                        if (x * 128 + wr < it.rows)
                            u[i] = __ldg(reinterpret_cast<const uint4*>(a.q + (it.row0 + group_div(a, rr)) * a.ldq +
                                                                        (int64_t)(it.h * a.G + group_mod(a, rr)) * D) + lane % LPR);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int wr = quarter * 32 + h0 + i * RPI + lane / LPR, ci = lane % LPR;
                        float mx = fmaxf(fmaxf(amax_bf16x2(u[i].x), amax_bf16x2(u[i].y)), fmaxf(amax_bf16x2(u[i].z), amax_bf16x2(u[i].w)));
#pragma unroll
                        for (int k2 = LPR / 2; k2; k2 >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k2));
                        const int e = row_exponent(mx);
                        const float up = row_up(e, a.scale_log2);
                        *reinterpret_cast<uint4*>(qx + (ci >> 3) * (128 * 128) + wr * 128 + (((ci & 7) ^ (wr & 7)) << 4)) =
                            make_uint4(scaled_f16x2(u[i].x, up), scaled_f16x2(u[i].y, up), scaled_f16x2(u[i].z, up), scaled_f16x2(u[i].w, up));
                        // the row's own thread takes its factor
                        const float down = __shfl_sync(0xffffffffu, row_down(e, a.scale_log2), (lane % RPI) * LPR);
                        if ((lane - h0) / RPI == i && lane >= h0) rs = down;
                    }
                }
                fence_proxy_async_smem();
                warp_arrive(&qfull[x]);
                for (int j = 0; j < cnt; ++j) {
                    ok = warp_wait(&sfull[x], tiles & 1);
                    if (!ok) break;
                    ++tiles;
                    fence_after();
                    const int tok0 = (first + j) * kTok;
                    const uint64_t out = *reinterpret_cast<const volatile uint64_t*>(bad + ((all_tiles + j) & 3) * 8);
                    const bool edge = out != 0 || tok0 + kTok - 1 > pw0 || (a.window > 0 && tok0 <= pw1 - a.window);
                    auto seen = [&](int c) {  // which of tokens 32 c .. 32 c + 31 of the tile this row sees
                        const int last = p - tok0 - 32 * c, before = a.window > 0 ? last - a.window : -1;  // before < t <= last
                        uint32_t b = last >= 31 ? 0xffffffffu : last < 0 ? 0u : (2u << last) - 1u;
                        b &= before >= 31 ? 0u : before < 0 ? 0xffffffffu : ~((2u << before) - 1u);
                        if (out != 0) b &= ~(((out >> (16 * c)) & 1 ? 0xffffu : 0u) | ((out >> (16 * c + 8)) & 1 ? 0xffff0000u : 0u));
                        return b;
                    };
                    // 32 scores at a time, the next ones on their way while these are worked on.  (Loops of two such steps
                    // and not of all four: the roles' code shares the instruction cache.)
                    uint32_t u0[32], u1[32];
                    float top = -INFINITY;
                    if (edge) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            ld32(ts + 32 * c, u0);
                            ld_wait(u0);
                            const uint32_t b = seen(c);
#pragma unroll
                            for (int i = 0; i < 32; ++i) top = fmaxf(top, (b >> i) & 1 ? __uint_as_float(u0[i]) : -INFINITY);
                        }
                    } else {
                        ld32(ts, u0);
                        float t0 = -INFINITY, t1 = -INFINITY;
                        auto most = [&](const uint32_t* u) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                t0 = fmaxf(t0, fmaxf(__uint_as_float(u[i]), __uint_as_float(u[i + 1])));
                                t1 = fmaxf(t1, fmaxf(__uint_as_float(u[i + 2]), __uint_as_float(u[i + 3])));
                            }
                        };
#pragma unroll 1
                        for (int c = 0; c < 128; c += 64) {
                            ld_wait(u0);
                            ld32(ts + c + 32, u1);
                            most(u0);
                            ld_wait(u1);
                            ld32(ts + ((c + 64) & 127), u0);  // at the end the first ones again, for the exponentials
                            most(u1);
                        }
                        top = fmaxf(t0, t1);
                    }
                    top = top == -INFINITY ? top : __fmul_rn(top, rs);
                    if (__any_sync(0xffffffffu, __fsub_rn(top, m) > kGrow)) {  // the difference: a sum would be rounded up where m is large
                        const float mn = fmaxf(m, __fsub_rn(top, kBelow));
                        const float f = m == -INFINITY ? 0.f : ex2(m - mn);
                        m = mn;
                        l *= f;
                        if (j > 0) {  // the products before this tile are done: S of this tile came after them
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t u[32];
                                ld32(to + c, u);
                                ld_wait(u);
#pragma unroll
                                for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * f);
                                st32(to + c, u);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : m;
                    float2 sum = make_float2(0.f, 0.f);
                    // the probabilities go where scores have been read already
                    if (edge || __any_sync(0xffffffffu, fabsf(ref) >= 0x1p20f)) {
                        // The careful form rounds twice, as the reference does: no score's exponent is above kGrow whatever
                        // its size.  One rounding (below) leaves up to half an ulp of the score there, at most 2^-4 below
                        // 2^20, the same for the whole row.
                        if (!edge) ld_wait(u0);
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t pk[16];
                            ld32(ts + 32 * c, u0);
                            ld_wait(u0);
                            const uint32_t b = seen(c);
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                float2 e2 = make_float2(ex2(__fsub_rn(__fmul_rn(__uint_as_float(u0[i]), rs), ref)),
                                                        ex2(__fsub_rn(__fmul_rn(__uint_as_float(u0[i + 1]), rs), ref)));
                                e2.x = (b >> i) & 1 ? e2.x : 0.f;
                                e2.y = (b >> (i + 1)) & 1 ? e2.y : 0.f;
                                sum = __fadd2_rn(sum, e2);
                                pk[i / 2] = pack_f16x2(e2.x, e2.y);
                            }
                            st16(ts + 16 * c, pk);
                        }
                    } else {
                        const float2 rs2 = make_float2(rs, rs), ref2 = make_float2(-ref, -ref);
                        auto exponentials = [&](const uint32_t* u, uint32_t* pk) {
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float2 y = __ffma2_rn(make_float2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), rs2, ref2);
                                const float2 e2 = make_float2(ex2(y.x), ex2(y.y));
                                sum = __fadd2_rn(sum, e2);
                                pk[i / 2] = pack_f16x2(e2.x, e2.y);
                            }
                        };
#pragma unroll 1
                        for (int c = 0; c < 128; c += 64) {
                            uint32_t pk[16];
                            ld_wait(u0);
                            ld32(ts + c + 32, u1);
                            exponentials(u0, pk);
                            st16(ts + c / 2, pk);
                            ld_wait(u1);
                            if (c == 0) ld32(ts + 64, u0);
                            exponentials(u1, pk);
                            st16(ts + c / 2 + 16, pk);
                        }
                    }
                    l += sum.x + sum.y;
                    st_wait();
                    fence_before();
                    warp_arrive(&pfull[x]);
                }
                ok = ok && warp_wait(&ofull[x], its & 1);
                ++its;
                fence_after();
            }
            all_tiles += cnt;
            // O: to its rows, or as this part's sums
            const bool valid = srow < it.rows;
            const int r = it.base + srow;
            const int64_t slot = it.parts > 1 ? (int64_t)(it.tail * it.parts + it.part) : 0;
            float* part = a.parts + slot * kRows * (D + 2);  // [D / 4][256 rows] of four values, then [256] {m, l}
            const float inv = l == 0.f ? 0.f : 1.f / l;
            __nv_bfloat16* dst = a.out + (it.row0 + group_div(a, r)) * a.ldo + (int64_t)(it.h * a.G + group_mod(a, r)) * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float v[32];
                uint32_t raw[32];
                __syncwarp();
                if (active && ok) {
                    ld32(to + c, raw);
                    ld_wait(raw);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) raw[i] = 0u;
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[i]);
                if (!valid) continue;
                if (it.parts == 1) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t u[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const __nv_bfloat162 b2 = out_pair(a, v[i + 2 * q], v[i + 2 * q + 1], inv);
                            u[q] = *reinterpret_cast<const uint32_t*>(&b2);
                        }
                        *reinterpret_cast<uint4*>(dst + c + i) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        __stcg(reinterpret_cast<float4*>(part) + (c + i) / 4 * kRows + srow,
                               make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
                }
            }
            fence_before();  // O is read before the next unit's products (the queries' barrier)
            if (it.parts > 1) {
                if (valid) __stcg(reinterpret_cast<float2*>(part + (int64_t)kRows * D) + srow, make_float2(m, l));
                __threadfence();
                soft_sync();
                if (threadIdx.x == 0) {
                    const int before = atomicAdd(&a.tickets[it.tail], 1);
                    *last_flag = before == it.parts - 1;
                    if (*last_flag) a.tickets[it.tail] = 0;  // everyone has come: zero for the next call
                    __threadfence();
                }
                soft_sync();
                if (*last_flag && valid) {
                    // Each row its own thread.  The parts' factors wait in the queries' place, which nothing reads any
                    // more; the sums come four parts at a time.
                    const int64_t psz = (int64_t)kRows * (D + 2);
                    const float* base = a.parts + (int64_t)it.tail * it.parts * psz;
                    auto ml_of = [&](int s) { return __ldcg(reinterpret_cast<const float2*>(base + s * psz + (int64_t)kRows * D) + srow); };
                    float* factor = reinterpret_cast<float*>(qt) + srow;
                    float mj = -INFINITY, lj = 0.f;
#pragma unroll 8
                    for (int s = 0; s < it.parts; ++s) mj = fmaxf(mj, ml_of(s).x);
                    const float ref = mj == -INFINITY ? 0.f : mj;
#pragma unroll 8
                    for (int s = 0; s < it.parts; ++s) {
                        const float2 ml = ml_of(s);
                        const float f = ex2(ml.x - ref);
                        factor[s * kRows] = f;
                        lj += ml.y * f;
                    }
                    const float invj = lj == 0.f ? 0.f : 1.f / lj;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float4 acc[4] = {};
                        for (int s0 = 0; s0 < it.parts; s0 += 4) {
                            float4 v[4][4];
                            float f[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int s = s0 + u < it.parts ? s0 + u : it.parts - 1;
                                f[u] = s0 + u < it.parts ? factor[s * kRows] : 0.f;
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    v[u][i] = __ldcg(reinterpret_cast<const float4*>(base + s * psz) + (c / 4 + i) * kRows + srow);
                            }
#pragma unroll
                            for (int u = 0; u < 4; ++u)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    acc[i].x += f[u] * v[u][i].x, acc[i].y += f[u] * v[u][i].y, acc[i].z += f[u] * v[u][i].z,
                                        acc[i].w += f[u] * v[u][i].w;
                        }
                        uint32_t u[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __nv_bfloat162 lo = out_pair(a, acc[i].x, acc[i].y, invj);
                            const __nv_bfloat162 hi = out_pair(a, acc[i].z, acc[i].w, invj);
                            u[2 * i] = *reinterpret_cast<const uint32_t*>(&lo), u[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&hi);
                        }
                        *reinterpret_cast<uint4*>(dst + c) = make_uint4(u[0], u[1], u[2], u[3]);
                        *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(u[4], u[5], u[6], u[7]);
                    }
                }
                soft_sync();  // the flag is free
            }
        }
    } else if (warp < kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDqRegs));
        const int id = threadIdx.x - kSoftWarps * 32;  // 0 .. 127
        // K: token id of the tile.  V: 16 values, block id / 16, of 8 tokens from 8 (id % 16)
        const int vblk = id >> 4, vch = id & 15;
        const bool vuse = vblk < D / 16;
        constexpr int KW = D / 8, KS = D / 64;  // words of codes and of scales of a token's K
        int k = -1;
        auto next_item = [&]() {  // the next one that has tokens
            for (;;) {
                if (k >= 0) done_with(k);
                if (!take(++k)) return false;
                if (ring[k % kItems].t1 > ring[k % kItems].t0) return true;
            }
        };
        // a tile that this thread has looked up: the groups of its tokens, or NULL (behind the end, a bad page)
        struct Place {
            const uint8_t *k, *v;
            int span;  // of V's 8 tokens those that may be seen: from the high half word up to the low one
            bool bad, some;
        };
        bool more = next_item();
        int tile = more ? ring[k % kItems].t0 - 1 : 0;
        auto group = [&](int tok, bool& bad_page) -> const uint8_t* {
            const Item& it = ring[k % kItems];
            if (tok >= it.L || (tok | (kGroup - 1)) < it.first) return nullptr;
            const int page = __ldg(a.table + it.b * a.ldb + (tok >> a.cache.page_log));
            if (page < 0 || page >= a.cache.n_pages) {
                atomicOr(a.status, kStatusBad);
                bad_page = true;
                return nullptr;
            }
            return group_ptr<D>(a.cache, page, it.h, tok & ((1 << a.cache.page_log) - 1));
        };
        auto step = [&]() {  // on to the next tile
            Place pl = {nullptr, nullptr, 8, false, false};
            if (more && ++tile >= ring[k % kItems].t1) {
                more = next_item();
                tile = more ? ring[k % kItems].t0 : 0;
            }
            if (!more) return pl;
            bool ignored = false;
            pl.some = true;
            pl.k = group(tile * kTok + id, pl.bad);
            pl.v = vuse ? group(tile * kTok + vch * 8, ignored) : nullptr;
            const int tok = tile * kTok + vch * 8;
            pl.span = (int)((uint32_t)max(ring[k % kItems].first - tok, 0) << 16) | min(ring[k % kItems].L - tok, 8);  // read where v is
            return pl;
        };
        struct Codes {
            uint32_t k[KW], ks[KS], v[16], vs[2];
        };
        auto fetch = [&](const Place& pl, Codes& c) {
#pragma unroll
            for (int i = 0; i < KW; ++i) c.k[i] = 0u;
#pragma unroll
            for (int i = 0; i < KS; ++i) c.ks[i] = 0u;
#pragma unroll
            for (int i = 0; i < 16; ++i) c.v[i] = 0u;
            c.vs[0] = c.vs[1] = 0u;
            if (pl.k) {
                const int r = id & 15;
#pragma unroll
                for (int i = 0; i < KW / 4; ++i) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(pl.k + r * (D / 2)) + i);
                    c.k[4 * i] = u.x, c.k[4 * i + 1] = u.y, c.k[4 * i + 2] = u.z, c.k[4 * i + 3] = u.w;
                }
#pragma unroll
                for (int i = 0; i < KS; ++i) c.ks[i] = __ldg(reinterpret_cast<const uint32_t*>(pl.k + k_scale_off(D) + r * (D / 16)) + i);
            }
            if (pl.v) {
                const int r = (vch * 8) & 15;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4*>(pl.v + v_code_off(D) + vblk * 128 + r * 8) + i);
                    c.v[4 * i] = u.x, c.v[4 * i + 1] = u.y, c.v[4 * i + 2] = u.z, c.v[4 * i + 3] = u.w;
                }
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(pl.v + v_scale_off(D) + vblk * 16 + r));
                c.vs[0] = u.x, c.vs[1] = u.y;
                if (pl.span != 8) {  // places that no row sees hold anything: scale 0, so that 0 * value is 0
                    const int from = pl.span >> 16, to = pl.span & 0xffff;  // to > 0: some of the 8 are in the context
                    uint64_t keep = ~(uint64_t)0 >> (8 * (8 - to));
                    keep = from >= 8 ? 0 : keep & (~(uint64_t)0 << (8 * from));
                    c.vs[0] &= (uint32_t)keep, c.vs[1] &= (uint32_t)(keep >> 32);
                }
            }
        };
        Codes c;
        Place now = step();
        fetch(now, c);
        Place next = step();
        for (int tiles = 0; now.some; ++tiles) {
            const int s = tiles & 1;
            Codes nc;
            fetch(next, nc);
            const Place ahead = step();
            if (tiles >= 2 && !warp_wait(&kfree[s], ((tiles >> 1) - 1) & 1)) break;
            {
                uint8_t* dst = kt + s * C::kKBytes + id * 128;
#pragma unroll
                for (int w = 0; w < KW; w += 2) {  // 16 values under one scale
                    const uint32_t two = e4m3x2_to_f16x2((c.ks[w / 8] >> (8 * ((w / 2) & 3))) & 0xffu);
                    const uint32_t f = __byte_perm(two, 0, 0x1010);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t h[4];
                        e2m1x8(c.k[w + u], h);
                        const int piece = w + u;  // 8 values: 16 bytes
                        *reinterpret_cast<uint4*>(dst + (piece >> 3) * (kTok * 128) + (((piece & 7) ^ (id & 7)) << 4)) =
                            make_uint4(hmul2(h[0], f), hmul2(h[1], f), hmul2(h[2], f), hmul2(h[3], f));
                    }
                }
                if ((id & 15) == 0) bad[(tiles & 3) * 8 + (id >> 4)] = now.bad ? 1 : 0;
            }
            fence_proxy_async_smem();
            arrive(&kfull[s]);
            if (tiles >= 2 && !warp_wait(&vfree[s], ((tiles >> 1) - 1) & 1)) break;
            if (vuse) {
                uint8_t* dst = vt + s * C::kVBytes + (vch >> 3) * (D * 128);
                const uint32_t f[4] = {e4m3x2_to_f16x2(c.vs[0] & 0xffffu), e4m3x2_to_f16x2(c.vs[0] >> 16),
                                       e4m3x2_to_f16x2(c.vs[1] & 0xffffu), e4m3x2_to_f16x2(c.vs[1] >> 16)};
#pragma unroll
                for (int w = 0; w < 2; ++w) {  // a word of each token: 8 of the 16 values
                    constexpr uint32_t lo = 0x0f0f0f0fu;
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {  // the even values, then the odd ones
                        uint32_t x[4][4];                // [token pair][byte]
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t p0 = c.v[4 * i + w], p1 = c.v[4 * i + 2 + w];
                            e2m1x8(odd ? ((p0 >> 4) & lo) | (p1 & ~lo) : (p0 & lo) | ((p1 << 4) & ~lo), x[i]);
                        }
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const int d = vblk * 16 + w * 8 + 2 * b + odd;
                            *reinterpret_cast<uint4*>(dst + d * 128 + (((vch & 7) ^ (d & 7)) << 4)) =
                                make_uint4(hmul2(x[0][b], f[0]), hmul2(x[1][b], f[1]), hmul2(x[2][b], f[2]), hmul2(x[3][b], f[3]));
                        }
                    }
                }
            }
            fence_proxy_async_smem();
            arrive(&vfull[s]);
            c = nc;
            now = next, next = ahead;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
        if (warp == kMmaWarp) {
            const uint32_t idesc_s = (1u << 4) | ((uint32_t)(kTok >> 3) << 17) | ((128u >> 4) << 24);  // fp16 x fp16 -> fp32
            const uint32_t idesc_o = (1u << 4) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
            int tiles = 0, q_its[2] = {0, 0}, p_tiles[2] = {0, 0};
            bool ok = true;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t dq = desc_lo(smem_u32(qt)), dk = desc_lo(smem_u32(kt)), dv = desc_lo(smem_u32(vt));
            auto scores = [&](int x, int s) {
                const uint32_t qa = dq + x * (C::kQBytes >> 4), ka = dk + s * (C::kKBytes >> 4), d = tm + x * 128;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t at = ((i >> 2) * (128 * 128) + (i & 3) * 32) >> 4;
                    mma_ss(d, qa + at, ka + at, idesc_s, i > 0);
                }
                commit(&sfull[x]);
            };
            for (int k = 0; ok && take(k); ++k) {
                const int cnt = ring[k % kItems].t1 - ring[k % kItems].t0, two = ring[k % kItems].rows > 128 ? 2 : 1;
                done_with(k);
                if (cnt <= 0) continue;
                for (int x = 0; x < two && ok; ++x) {
                    ok = warp_wait(&qfull[x], q_its[x] & 1);
                    ++q_its[x];
                }
                ok = ok && warp_wait(&kfull[tiles & 1], (tiles >> 1) & 1);
                if (!ok) break;
                fence_after();
                for (int x = 0; x < two; ++x) scores(x, tiles & 1);
                commit(&kfree[tiles & 1]);
                for (int j = 0; j < cnt && ok; ++j, ++tiles) {
                    const int s = tiles & 1, sn = (tiles + 1) & 1;
                    ok = warp_wait(&vfull[s], (tiles >> 1) & 1);
                    for (int x = 0; x < two && ok; ++x) {
                        ok = warp_wait(&pfull[x], p_tiles[x] & 1);
                        ++p_tiles[x];
                        if (!ok) break;
                        fence_after();
                        const uint32_t d = tm + 256 + x * D, pa = tm + x * 128, va = dv + s * (C::kVBytes >> 4);
#pragma unroll
                        for (int i = 0; i < kTok / 16; ++i)
                            mma_ts(d, pa + i * 8, va + (((i >> 2) * (D * 128) + (i & 3) * 32) >> 4), idesc_o, j > 0 || i > 0);
                        if (x == two - 1) commit(&vfree[s]);
                        if (j + 1 < cnt) {
                            if (x == 0) {
                                ok = warp_wait(&kfull[sn], ((tiles + 1) >> 1) & 1);
                                if (!ok) break;
                                fence_after();
                            }
                            scores(x, sn);
                            if (x == two - 1) commit(&kfree[sn]);
                        } else {
                            commit(&ofull[x]);
                        }
                    }
                }
            }
            commit(mma_done);  // every tensor-core operation of this warp is done before the teardown
            if (!mbar_wait_bounded(mma_done, 0)) atomicOr(a.status, 1u);
        } else if (warp == kMmaWarp + 1) {
            // unit u: sequences in order; in each the last rows first (the most tokens), the kv heads of a block side by side
            auto unit = [&](int u) {
                Item it;
                int lo = 0, hi = a.B - 1;  // the last b with prefix[b] * a.cache.Hkv <= u (it has units)
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if ((int64_t)prefix[mid] * a.cache.Hkv <= u) lo = mid;
                    else hi = mid - 1;
                }
                const int k = u - prefix[lo] * a.cache.Hkv, blocks = prefix[lo + 1] - prefix[lo];
                it.b = lo;
                it.h = k % a.cache.Hkv;
                it.base = (blocks - 1 - k / a.cache.Hkv) * *unit_rows;
                it.n = row0[lo + 1] - row0[lo];
                it.L = length[lo];
                it.row0 = row0[lo];
                it.rows = min(*unit_rows, it.n * a.G - it.base);
                const int p0 = it.L - it.n + group_div(a, it.base), p1 = it.L - it.n + group_div(a, it.base + it.rows - 1);
                it.first = a.window > 0 && p0 - a.window + 1 > 0 ? p0 - a.window + 1 : 0;
                it.t0 = it.first / kTok;
                it.t1 = p1 < 0 ? it.t0 : p1 / kTok + 1;
                it.part = 0, it.parts = 1, it.tail = -1;
                return it;
            };
            // rows that sequences share (cu_q not rising) could number more units than an int holds
            const int64_t all_units = (int64_t)prefix[a.B] * a.cache.Hkv;
            const int units = all_units < (1 << 30) ? (int)all_units : 0;
            if (units != all_units && lane == 0) atomicOr(a.status, kStatusBad);
            const int grid = gridDim.x, whole = units / grid * grid, tails = units - whole;
            // splits of the last round's units: their rounds times a part's tiles and its fixed cost, the least of it
            int splits = 1;
            if (tails > 0) {
                int sum = 0;
                for (int i = lane; i < tails; i += 32) {
                    const Item it = unit(whole + i);
                    sum += it.t1 - it.t0;
                }
                sum = __reduce_add_sync(0xffffffffu, sum);
                const float avg = (float)sum / tails;
                float best = avg + kUnitCost;
                for (int s = 2; s <= 32 && tails * s <= 2 * grid; ++s) {
                    const float cost = (float)((tails * s + grid - 1) / grid) * (avg / s + kUnitCost) + kJoinCost + kPartCost * s;
                    if (cost < best && avg >= 2 * s) best = cost, splits = s;
                }
            }
            const int items = whole + tails * splits;
            int pushed = 0;
            for (int k = 0;; ++k) {
                // rounds go there and back
                const int i = k * grid + ((k & 1) ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x);
                Item it = {};
                it.b = -1;
                if (i < whole || (i < items && splits == 1)) {
                    it = unit(i);
                } else if (i < items) {
                    const int r = (i - whole) / splits, s = (i - whole) % splits;
                    it = unit(whole + r);
                    it.part = s, it.parts = splits, it.tail = r;
                }
                if (it.b >= 0 && it.t0 >= it.t1) {  // a unit that sees nothing: rows of zeros, no work for the others
                    for (int j = lane; it.part == 0 && j < it.rows * (D / 8); j += 32) {
                        const int row = it.base + j / (D / 8);
                        *(reinterpret_cast<uint4*>(a.out + (it.row0 + group_div(a, row)) * a.ldo +
                                                   (int64_t)(it.h * a.G + group_mod(a, row)) * D) + j % (D / 8)) = make_uint4(0, 0, 0, 0);
                    }
                    continue;
                }
                if (it.parts > 1) {
                    const int cnt = it.t1 - it.t0, first = it.t0;
                    it.t0 = first + (int)((int64_t)cnt * it.part / splits);
                    it.t1 = first + (int)((int64_t)cnt * (it.part + 1) / splits);
                }
                if (pushed >= kItems && !warp_wait(&itemfree[pushed % kItems], (pushed / kItems - 1) & 1)) break;
                if (lane == 0) ring[pushed % kItems] = it;
                warp_arrive(&itemfull[pushed % kItems]);
                ++pushed;
                if (it.b < 0) break;  // only the last round has places without work
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

}  // namespace kv
}  // namespace qlin

using namespace qlin;

// Bytes of the parts of shared units at most.
extern "C" size_t qlin_attn_chunk_part_bytes(int D, int sms) { return (size_t)2 * sms * kv::ch::kRows * (D + 2) * 4; }

template <int D>
static cudaError_t launch_chunk(kv::AttnArgs a, int sms, cudaStream_t s) {
    using C = kv::ch::Cfg<D>;
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev]) {
        e = cudaFuncSetAttribute(kv::attn_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 C::smem(kv::ch::kMaxSeqs));
        if (e != cudaSuccess) return e;
        set[dev] = true;
    }
    kv::attn_chunk_kernel<D><<<sms, kv::ch::kThreads, C::smem(a.B), s>>>(a);
    return cudaGetLastError();
}

extern "C" cudaError_t qlin_launch_attn_chunk(const kv::AttnArgs* a, int D, int sms, cudaStream_t s) {
    return D == 128 ? launch_chunk<128>(*a, sms, s) : launch_chunk<64>(*a, sms, s);
}
