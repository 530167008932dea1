// The products of a linear layer of any size (see linear.cu), on the tensor cores.
#include <cuda.h>

#include "linear_internal.cuh"

namespace pulsar {
namespace linear {
namespace {

// -------------------------------------------------------------- products --
// One kernel for the three products, a persistent CTA per SM, or a pair of them on
// a tile of twice the rows.  Roles: one thread keeps a ring of operand stages
// filled by TMA (out of range: zeros), one issues the MMAs into one of two
// accumulators in tensor memory, and the other warps finish the other (four per
// half or quarter of the tile's columns, a thread per row): bias, activation,
// residual, rounding; through a swizzled exchange in shared memory, so that a
// warp stores whole sectors.
//
// A stage of a 128 x 256 tile is 48 KB, and at the MMAs' rate the SMs would ask
// the L2 for more than it gives (the MMAs waited for operands half of the time).
// A pair of CTAs reads each half of B once for both: 32 KB a stage.  16381 x 1024
// -> 4096 in 16 bits: 83 us (101 by single CTAs), dx 82 (95), dW 79 (89); by the
// operations 73 at the rate of a library's product in a burst, 81 in a long run.
// dx and dW have 256 and 64 tiles for 76 pairs, which is 84 % of them busy; the
// MMAs of a 256 x 256 tile follow each other at 1.05 times their own time.  (The
// outputs' kernels that store parts spill some 200 bytes: 300 x 4096 -> 256 in 16
// bits 12 us with the join.  dW's drained ones spill up to 100: their times at
// kDrain.)
//
// In 32 bits the tensor cores' accumulation, which truncates, would be what
// limits the result (of K = 2048, some 2^-18.5 of it): hi hi and the other
// five products have accumulators of their own, and both are drained and
// summed in registers every kChunk panels (128 of K).  4001 x 1500 -> 509: 24
// panels of 24 MMAs of 256 x 128 at 78 cycles, some 30 us, after 8 us for the
// planes (dx 42 us of 45 by single CTAs; drained every 256 of K: 39, and twice as far
// off).  In 16 bits an instruction's truncation, of 16 of K, is at most 2^-23 of the
// sum: the outputs' and dx's K of 2^16 or less lose an eighth of half a step of the
// result and are not drained, dW's, whose K is the rows, is every kDrain panels (2^14
// rows: 2^-13, a thirtieth of half a step).
//
// Where a product has few tiles for the SMs and a long contraction (dW: one
// tile and a million rows), its parts are separate work items, whose sums
// k_linear_joins adds up in their order.
struct Product {
    CUtensorMap a, b;
    int tiles_m, tiles_n, panels;   // panels of the contraction
    Result out;
};

// warps: copies, MMAs, and of the epilogue eight, or for a layer's outputs in 16 bits, where it has
// every tile's activation to do within the MMAs' time, sixteen (16381 x 1024 -> 4096: 83 us, with
// eight 85; dx, which has none: 82 us with eight, with sixteen 85)
constexpr int epilogue_warps(int planes, bool outputs) { return planes == 1 && outputs ? 16 : 8; }
constexpr int kChunk = 2;              // panels per drained sum (32 bits)
// the same in 16 bits, where a part has more than one of them (262144 x 1024 -> 4096: dW 1178 us,
// undrained 1183; one of them has a kernel that keeps no sums: 16381 rows 77 us, else 79)
constexpr int kDrain = 256;
constexpr int kGroup = 4;              // row blocks whose tiles lie side by side in time (of 16: 1 us more)

template <int kPlanes, int kN, int kCtas, bool kOutputs>
struct ProductSmem {
    static constexpr int rows_b = kN / kCtas;   // of B, in each CTA of a pair
    static constexpr int a = kBlock * kPanel * 2, b = rows_b * kPanel * 2;
    static constexpr int stage = kPlanes * (a + b);
    static constexpr int epilogue = epilogue_warps(kPlanes, kOutputs), threads = 64 + 32 * epilogue;
    // a warp's exchange: 32 x 32 words, in 32 bits 32 x 8 for a third stage
    static constexpr int warp_exchange = 32 * (kPlanes == 3 ? 8 : 32) * 4;
    static constexpr int exchange_bytes = epilogue * warp_exchange;
    static constexpr int stages = (227 * 1024 - 1024 - exchange_bytes - 256) / stage;
    static constexpr int exchange = stages * stage;
    static constexpr int bars = exchange + exchange_bytes;
    static constexpr int bytes = bars + 256 + 1024;   // and the alignment to 1024
    static_assert(stages >= 2 && (2 * stages + 5) * 8 + 8 <= 256, "shared memory of a product");
};

// A box of a tensor map [planes][rows][cols] at (plane, row, col): col a multiple of 64.
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int col, int row,
                                         int plane, uint64_t* mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(col), "r"(row), "r"(plane), "r"(smem_u32(mbar))
        : "memory");
}
// ---- pairs of CTAs (cta_group::2) on one tile
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// the place of this CTA's shared address in the pair's first CTA
__device__ __forceinline__ uint32_t in_first(const void* p) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(smem_u32(p)));
    return at;
}
// (what it orders is the accumulator's loads, which are complete: a release to the whole cluster
// would wait for the stores of the results too)
__device__ __forceinline__ void arrive_at(uint32_t mbar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mbar) : "memory");
}
// into this CTA's shared memory, counted on the first one's barrier
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int col, int row,
                                              int plane, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
        "bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(col), "r"(row), "r"(plane), "r"(mbar)
        : "memory");
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a, uint64_t b,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// arrives at the barrier's place in both CTAs
__device__ __forceinline__ void mma_commit_pair(uint64_t* mbar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(mbar)),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* s_taddr, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(s_taddr)),
                 "r"(cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols));
}
// Whether any of the epilogue's kThreads has `v`: one decision for all.
template <int kThreads>
__device__ __forceinline__ bool epilogue_any(bool v) {
    uint32_t any;
    __syncwarp();
    asm volatile(
        "{\n.reg .pred p, r;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred r, 1, %2, p;\n"
        "selp.u32 %0, 1, 0, r;\n}\n"
        : "=r"(any)
        : "r"((uint32_t)v), "n"(kThreads)
        : "memory");
    return any != 0;
}

// T: the result's type (float for parts).  kAMn, kBMn: the operand's matrix has the contraction
// as its rows.  kCtas: 1, or a pair of CTAs on a tile of 256 rows, each with its 128 rows of A and
// of the sums, and half of B's; the first one issues the MMAs of both.  kLong: a part's contraction
// is more than kDrain panels, in 16 bits.
template <typename T, int kPlanes, int kN, bool kAMn, bool kBMn, int kCtas, bool kVec, bool kLong>
__global__ void __launch_bounds__(64 + 32 * epilogue_warps(kPlanes, !kAMn && !kBMn)) __cluster_dims__(kCtas, 1, 1)
k_linear_product(const __grid_constant__ Product q, LearnState* st) {
    using L = ProductSmem<kPlanes, kN, kCtas, !kAMn && !kBMn>;
    constexpr bool kPair = kCtas == 2;
    constexpr int kAcc = kPlanes == 3 ? 2 * kN : kN;   // columns of an accumulator
    constexpr int kHalf = kN / (L::epilogue / 4);      // columns of an epilogue thread
    constexpr bool kDrained = kPlanes == 3 || kLong;
    constexpr int kPiece = kPlanes == 3 ? kChunk : kDrain;   // panels of a drained sum
    static_assert(2 * kAcc <= 512, "tensor memory");
    extern __shared__ unsigned char raw[];
    unsigned char* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bars);
    uint64_t* empty = full + L::stages;
    uint64_t* acc_full = empty + L::stages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* s_taddr = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* s_fail = s_taddr + 1;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (known to be the same in a warp)
    if (tid == 0) {
        for (int s = 0; s < L::stages; ++s) {
            mbar_init(full + s);
            mbar_init(empty + s);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + s);
            mbar_init_n(acc_empty + s, L::epilogue * kCtas);
        }
        mbar_init(drain);
        *s_fail = 0u;
        fence_async_smem();
    }
    if (warp == 1) {
        if constexpr (kPair) tmem_alloc_pair(s_taddr, 2 * kAcc);
        else tmem_alloc(s_taddr, 2 * kAcc);
    }
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync();   // the barriers are there
    tc_fence_after();
    const uint32_t rank = kPair ? cluster_rank() : 0u;
    const int first = blockIdx.x / kCtas, step = gridDim.x / kCtas;
    const uint32_t tmem = *s_taddr;
    pdl_next();
    pdl_begin();
    const int tiles = q.tiles_m * q.tiles_n, total = tiles * q.out.splits;
    auto place = [&](int t, int* i, int* j, int* k0, int* k1, int* part) {
        *part = t / tiles;
        t -= *part * tiles;
        const int g = t / (kGroup * q.tiles_n), rows = min(kGroup, q.tiles_m - g * kGroup);
        t -= g * kGroup * q.tiles_n;
        *i = g * kGroup + t % rows;
        *j = t / rows;
        *k0 = (int)((int64_t)*part * q.panels / q.out.splits);
        *k1 = (int)((int64_t)(*part + 1) * q.panels / q.out.splits);
    };
    if (warp == 0) {
        if (elect_one()) {   // ---- copies
            int n = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += step) {
                int i, j, k0, k1, part;
                place(t, &i, &j, &k0, &k1, &part);
                for (int k = k0; k < k1; ++k, ++n) {
                    const int s = n % L::stages;
                    ok = mbar_wait(empty + s, ((n / L::stages) & 1) ^ 1) && !*s_fail;
                    if (!ok) break;
                    unsigned char* dst = smem + s * L::stage;
                    const uint32_t bar = kPair ? in_first(full + s) : 0u;
                    const auto load = [&](void* to, const CUtensorMap* map, int col, int row, int p) {
                        if constexpr (kPair) tma_load_pair(to, map, col, row, p, bar);
                        else tma_load(to, map, col, row, p, full + s);
                    };
                    if (rank == 0) expect_bytes(full + s, kCtas * L::stage);
                    const int row_a = (i * kCtas + (int)rank) * kBlock;
                    const int row_b = j * kN + (int)rank * L::rows_b;
#pragma unroll
                    for (int p = 0; p < kPlanes; ++p) {
                        if (kAMn) {
#pragma unroll
                            for (int c = 0; c < kBlock / kPanel; ++c)
                                load(dst + p * L::a + c * kPanel * kPanel * 2, &q.a,
                                     row_a + c * kPanel, k * kPanel, p);
                        } else {
                            load(dst + p * L::a, &q.a, k * kPanel, row_a, p);
                        }
                    }
                    dst += kPlanes * L::a;
#pragma unroll
                    for (int p = 0; p < kPlanes; ++p) {
                        if (kBMn) {
#pragma unroll
                            for (int c = 0; c < L::rows_b / kPanel; ++c)
                                load(dst + p * L::b + c * kPanel * kPanel * 2, &q.b,
                                     row_b + c * kPanel, k * kPanel, p);
                        } else {
                            load(dst + p * L::b, &q.b, k * kPanel, row_b, p);
                        }
                    }
                }
            }
            if (!ok) {   // give the copies in flight one more bounded wait
                // (the second CTA's are counted by the first, which it meets before it leaves)
                *s_fail = 1u;
                for (int k = n > L::stages ? n - L::stages : 0; k < n && rank == 0; ++k)
                    mbar_wait(full + k % L::stages, (k / L::stages) & 1);
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {   // ---- MMAs
            constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) |
                                       (kAMn ? 1u << 15 : 0u) | (kBMn ? 1u << 16 : 0u) |
                                       ((uint32_t)(kN >> 3) << 17) |
                                       ((uint32_t)(kCtas * kBlock >> 4) << 24);
            const auto mma = [&](uint32_t d, uint64_t a, uint64_t b, uint32_t more) {
                if constexpr (kPair) mma_f16_pair(d, a, b, idesc, more);
                else mma_f16(d, a, b, idesc, more);
            };
            const auto commit = [&](uint64_t* bar) {
                if constexpr (kPair) mma_commit_pair(bar);
                else mma_commit(bar);
            };
            const uint32_t base = smem_u32(smem);
            int n = 0, it = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += step) {
                int i, j, k0, k1, part;
                place(t, &i, &j, &k0, &k1, &part);
                const int chunk = kDrained ? kPiece : k1 - k0;
                for (int kc = k0; kc < k1 && ok; kc += chunk, ++it) {
                    const int buf = it & 1, ke = min(kc + chunk, k1);
                    const uint32_t d = tmem + buf * kAcc;
                    ok = mbar_wait(acc_empty + buf, ((it >> 1) & 1) ^ 1) && !*s_fail;
                    if (!ok) break;
                    tc_fence_after();
                    for (int k = kc; k < ke; ++k, ++n) {
                        const int s = n % L::stages;
                        ok = mbar_wait(full + s, (n / L::stages) & 1) && !*s_fail;
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t at = base + s * L::stage;
                        uint64_t a[kPlanes], b[kPlanes];
#pragma unroll
                        for (int p = 0; p < kPlanes; ++p) {
                            a[p] = desc_sw128(at + p * L::a, kAMn ? kPanel * kPanel * 2 : 16);
                            b[p] = desc_sw128(at + kPlanes * L::a + p * L::b,
                                              kBMn ? kPanel * kPanel * 2 : 16);
                        }
#pragma unroll
                        for (int e = 0; e < kPanel / 16; ++e) {
                            // 16 of K: 32 bytes along a K-major row, 16 rows of an MN-major operand
                            const uint32_t ea = (kAMn ? 2048u : 32u) * e >> 4;
                            const uint32_t eb = (kBMn ? 2048u : 32u) * e >> 4;
                            const uint32_t more = k > kc || e > 0;
                            mma(d, a[0] + ea, b[0] + eb, more);
                            if constexpr (kPlanes == 3) {
                                mma(d + kN, a[0] + ea, b[2] + eb, more);
                                mma(d + kN, a[1] + ea, b[1] + eb, 1);
                                mma(d + kN, a[2] + ea, b[0] + eb, 1);
                                mma(d + kN, a[0] + ea, b[1] + eb, 1);
                                mma(d + kN, a[1] + ea, b[0] + eb, 1);
                            }
                        }
                        commit(empty + s);
                    }
                    if (ok) commit(acc_full + buf);
                }
            }
            if (!ok) {
                *s_fail = 1u;
                commit(drain);
                mbar_wait(drain, 0);
            }
        }
    } else {   // ---- epilogue
        const int group = (warp - 2) >> 2, quarter = warp & 3;   // (from warp 2 on)
        float4* x = reinterpret_cast<float4*>(smem + L::exchange + (warp - 2) * L::warp_exchange);
        const auto release = [&](int buf) {
            if constexpr (kPair) arrive_at(in_first(acc_empty + buf));
            else mbar_arrive(acc_empty + buf);
        };
        int it = 0;
        for (int t = first; t < total; t += step) {
            int i, j, k0, k1, part;
            place(t, &i, &j, &k0, &k1, &part);
            const int64_t r0 = ((int64_t)i * kCtas + rank) * kBlock + quarter * 32;
            const int64_t base = part * q.out.part;
            // 32 columns from `col` of the tile, a row in each lane
            auto emit = [&](const float (&v)[32], int col) {
                const int64_t c0 = (int64_t)j * kN + col;
                if constexpr (kPlanes == 3) {
                    if (kAMn || kBMn)
                        finish_small<T, kActNone, true, kVec>(q.out, x, v, r0, c0, base, lane);
                    else if (q.out.act == kActNone)
                        finish_small<T, kActNone, false, kVec>(q.out, x, v, r0, c0, base, lane);
                    else if (q.out.act == kActSilu)
                        finish_small<T, kActSilu, false, kVec>(q.out, x, v, r0, c0, base, lane);
                    else
                        finish_small<T, kActRelu, false, kVec>(q.out, x, v, r0, c0, base, lane);
                } else {
                    const auto finish = [&](auto skip) {
                        Share<T, kVec, decltype(skip)::value> share;
                        share.begin(q.out, r0, c0, base, lane);
                        float bias[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            bias[e] = q.out.bias && e < share.n ? q.out.bias[share.c + e] : 0.0f;
                        if (kAMn || kBMn)
                            share.template end<kActNone>(q.out, x, v, bias, r0, c0, base, lane);
                        else
                            share.end(q.out, x, v, bias, r0, c0, base, lane);
                    };
                    if (kAMn || kBMn || !q.out.residual) finish(std::false_type());
                    else finish(std::true_type());
                }
            };
            bool ok = true;
            if constexpr (kDrained) {
                float v[kHalf];
#pragma unroll
                for (int e = 0; e < kHalf; ++e) v[e] = 0.0f;
                for (int kc = k0; kc < k1; kc += kPiece, ++it) {
                    const int buf = it & 1;
                    ok = mbar_wait(acc_full + buf, (it >> 1) & 1) && !*s_fail;
                    ok = !epilogue_any<32 * L::epilogue>(!ok);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t acc = tmem + buf * kAcc + ((uint32_t)(quarter * 32) << 16) +
                                         group * kHalf;
#pragma unroll
                    for (int h = 0; h < kHalf; h += 16) {
                        uint32_t u[16], w[16];
                        tmem_ld16(acc + h, u);
                        if (kPlanes == 3) tmem_ld16(acc + kN + h, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            v[h + e] += kPlanes == 3 ? __uint_as_float(u[e]) + __uint_as_float(w[e])
                                                     : __uint_as_float(u[e]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) release(buf);
                }
                if (ok) {
#pragma unroll
                    for (int h = 0; h < kHalf; h += 32) {
                        float w[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) w[e] = v[h + e];
                        emit(w, group * kHalf + h);
                    }
                }
            } else {
                const int buf = it & 1;
                ok = mbar_wait(acc_full + buf, (it >> 1) & 1) && !*s_fail;
                ok = !epilogue_any<32 * L::epilogue>(!ok);
                if (ok) {
                    tc_fence_after();
                    const uint32_t acc = tmem + buf * kAcc + ((uint32_t)(quarter * 32) << 16) +
                                         group * kHalf;
#pragma unroll 1
                    for (int h = 0; h < kHalf; h += 32) {
                        uint32_t u[32];
                        float v[32];
                        __syncwarp();
                        tmem_ld32(acc + h, u);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(u[e]);
                        if (h + 32 == kHalf) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) release(buf);
                        }
                        emit(v, group * kHalf + h);
                    }
                    ++it;
                }
            }
            if (!ok) {
                *s_fail = 1u;
                break;
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (kPair) cluster_sync();   // the pair's MMAs and arrivals reach into both
    tc_fence_after();
    if (tid == 0 && *s_fail) atomicOr(&st->error, kErrTimeout);
    if (warp == 1) {
        if constexpr (kPair) tmem_dealloc_pair(tmem, 2 * kAcc);
        else tmem_dealloc(tmem, 2 * kAcc);
    }
}

// ------------------------------------------------------------------ plans --
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;

// A map whose boxes are 64 columns of `box_rows` rows.
bool encode(CUtensorMap* map, const Matrix& m, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows, (cuuint64_t)m.planes};
    const cuuint64_t strides[2] = {(cuuint64_t)m.pitch * 2,
                                   (cuuint64_t)(m.planes > 1 ? m.plane : m.pitch) * 2};
    const cuuint32_t box[3] = {(cuuint32_t)kPanel, (cuuint32_t)box_rows, 1};
    const cuuint32_t steps[3] = {1, 1, 1};
    return g_encode &&
           g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                    const_cast<__nv_bfloat16*>(m.at), dims, strides, box, steps,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The parts of a product: as many as fill the SMs once, of kLeast panels or more.
constexpr int kLeast = 4;
int splits_of(int64_t tiles, int64_t panels, int n_sms) {
    const int64_t fit = n_sms / tiles, most = panels / kLeast;
    const int64_t s = fit < most ? fit : most;
    return s > 1 ? (int)s : 1;
}
// Pairs of CTAs where tiles of 256 rows are not half empty.
bool paired(int64_t m) { return m > kBlock; }
// Columns of a tile.  In 32 bits the accumulators of both kinds, twice, leave room for 128.  In 16
// bits tiles of 128 x 128 that fill the SMs once at most have the shorter way from the first operand
// to the last result (some 6 us: 960 x 512 -> 512 8 us for 11, 2000 x 1000 -> 1000 11 for 17), while
// a panel takes a CTA of them 0.24 us and a pair's, of four times the products, 0.36: dW of 20000 x
// 1000 -> 1000 takes the pairs (with its dx 112 us, else 144), of 20000 x 512 -> 512 it does not.
int tile_n(int planes, int64_t m, int64_t n, int64_t k) {
    if (planes == 3 || n <= 128) return 128;
    constexpr int kSms = 152;   // (a choice that does not depend on the device: it sizes workspace)
    const int64_t small = ceil_div(m, 128) * ceil_div(n, 128), panels = ceil_div(k, kPanel);
    if (small > kSms) return 256;
    const int ctas = paired(m) ? 2 : 1;
    const int64_t large = ceil_div(m, kBlock * ctas) * ceil_div(n, 256);
    const int64_t by_small = ceil_div(panels, splits_of(small, panels, kSms));
    const int64_t by_large = ceil_div(panels, splits_of(large, panels, kSms / ctas));
    return 2 * by_small <= 3 * by_large + 40 ? 128 : 256;
}

template <typename T, int kPlanes, int kN, bool kAMn, bool kBMn, int kCtas>
cudaError_t product_as(const Result& r, const Matrix& a, const Matrix& b, int64_t k, float* parts,
                       Result* pending, LearnState* st, int n_sms, cudaStream_t s) {
    using L = ProductSmem<kPlanes, kN, kCtas, !kAMn && !kBMn>;
    Product q{};
    q.out = r;
    q.tiles_m = (int)ceil_div(r.m, kBlock * kCtas);
    q.tiles_n = (int)ceil_div(r.n, kN);
    q.panels = (int)ceil_div(k, kPanel);
    const int64_t tiles = (int64_t)q.tiles_m * q.tiles_n;
    const int groups = n_sms / kCtas;   // of CTAs that share a tile
    q.out.splits = tiles <= groups ? splits_of(tiles, q.panels, groups) : 1;
    q.out.part = part_size(r.m, r.n);
    *pending = q.out;
    if (!encode(&q.a, a, kAMn ? kPanel : kBlock) || !encode(&q.b, b, kBMn ? kPanel : L::rows_b))
        return cudaErrorInvalidValue;
    if (q.out.splits > 1)
        q.out = Result{r.m, r.n, nullptr, nullptr, nullptr, parts, kActNone, r.n % 4 == 0,
                       q.out.splits, q.out.part};
    const auto launch = [&](auto type, auto is_long) {
        using R = decltype(type);
        constexpr bool kLong = decltype(is_long)::value;
        const int64_t total = tiles * q.out.splits;
        return launch_pdl(q.out.vec ? k_linear_product<R, kPlanes, kN, kAMn, kBMn, kCtas, true, kLong>
                                    : k_linear_product<R, kPlanes, kN, kAMn, kBMn, kCtas, false, kLong>,
                          dim3((unsigned)((total < groups ? total : groups) * kCtas)),
                          dim3(L::threads), L::bytes, s, q, st);
    };
    const auto typed = [&](auto is_long) {
        return q.out.splits > 1 ? launch(float(), is_long) : launch(T(), is_long);
    };
    if constexpr (kPlanes == 1 && kAMn) {
        if (ceil_div(q.panels, q.out.splits) > kDrain) return typed(std::true_type());
    }
    return typed(std::false_type());
}

template <typename T, bool kAMn, bool kBMn>
cudaError_t product(const Result& q, const Matrix& a, const Matrix& b, int64_t k, float* parts,
                    Result* pending, LearnState* st, int n_sms, cudaStream_t s) {
    if constexpr (sizeof(T) == 4)
        return paired(q.m) ? product_as<T, 3, 128, kAMn, kBMn, 2>(q, a, b, k, parts, pending, st, n_sms, s)
                           : product_as<T, 3, 128, kAMn, kBMn, 1>(q, a, b, k, parts, pending, st, n_sms, s);
    else if (tile_n(1, q.m, q.n, k) == 128)
        return product_as<T, 1, 128, kAMn, kBMn, 1>(q, a, b, k, parts, pending, st, n_sms, s);
    else if (paired(q.m))
        return product_as<T, 1, 256, kAMn, kBMn, 2>(q, a, b, k, parts, pending, st, n_sms, s);
    else
        return product_as<T, 1, 256, kAMn, kBMn, 1>(q, a, b, k, parts, pending, st, n_sms, s);
}

template <typename T, int kPlanes, int kN, int kCtas, bool kAMn, bool kBMn>
cudaError_t prepare_one() {
    cudaError_t e = cudaSuccess;
    const auto prepare = [&](auto* f) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     ProductSmem<kPlanes, kN, kCtas, !kAMn && !kBMn>::bytes);
    };
    const auto both = [&](auto type, auto is_long) {
        using R = decltype(type);
        constexpr bool kLong = decltype(is_long)::value;
        prepare(k_linear_product<R, kPlanes, kN, kAMn, kBMn, kCtas, true, kLong>);
        prepare(k_linear_product<R, kPlanes, kN, kAMn, kBMn, kCtas, false, kLong>);
    };
    both(T(), std::false_type());
    if constexpr (sizeof(T) == 2) {
        both(float(), std::false_type());
        if constexpr (kAMn) {
            both(T(), std::true_type());
            both(float(), std::true_type());
        }
    }
    return e;
}
template <typename T, int kPlanes, int kN, int kCtas>
cudaError_t prepare_three() {
    cudaError_t e = prepare_one<T, kPlanes, kN, kCtas, false, false>();
    if (e == cudaSuccess) e = prepare_one<T, kPlanes, kN, kCtas, false, true>();
    if (e == cudaSuccess) e = prepare_one<T, kPlanes, kN, kCtas, true, true>();
    return e;
}

}  // namespace

size_t product_parts(int planes, int64_t m, int64_t n, int64_t k) {
    const int kn = tile_n(planes, m, n, k), ctas = (planes == 3 || kn == 256) && paired(m) ? 2 : 1;
    const int64_t tiles = ceil_div(m, kBlock * ctas) * ceil_div(n, kn);
    if (tiles == 0 || tiles > kMostSms / ctas) return 0;
    const int s = splits_of(tiles, ceil_div(k, kPanel), kMostSms / ctas);
    return s > 1 ? (size_t)s * part_size(m, n) : 0;
}

template <typename T>
cudaError_t launch_product(const Result& q, const Matrix& a, bool a_mn, const Matrix& b, bool b_mn,
                           int64_t k, float* parts, Result* pending, LearnState* st, int n_sms,
                           cudaStream_t s) {
    if (a_mn) return product<T, true, true>(q, a, b, k, parts, pending, st, n_sms, s);
    return b_mn ? product<T, false, true>(q, a, b, k, parts, pending, st, n_sms, s)
                : product<T, false, false>(q, a, b, k, parts, pending, st, n_sms, s);
}
template cudaError_t launch_product<float>(const Result&, const Matrix&, bool, const Matrix&, bool,
                                           int64_t, float*, Result*, LearnState*, int,
                                           cudaStream_t);
template cudaError_t launch_product<__nv_bfloat16>(const Result&, const Matrix&, bool,
                                                   const Matrix&, bool, int64_t, float*, Result*,
                                                   LearnState*, int, cudaStream_t);

cudaError_t prepare_product() {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                     cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<EncodeTiled>(f);
    e = prepare_three<float, 3, 128, 1>();
    if (e == cudaSuccess) e = prepare_three<float, 3, 128, 2>();
    if (e == cudaSuccess) e = prepare_three<__nv_bfloat16, 1, 128, 1>();
    if (e == cudaSuccess) e = prepare_three<__nv_bfloat16, 1, 256, 1>();
    if (e == cudaSuccess) e = prepare_three<__nv_bfloat16, 1, 256, 2>();
    return e;
}

}  // namespace linear
}  // namespace pulsar
