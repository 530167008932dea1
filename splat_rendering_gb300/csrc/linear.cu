// A linear layer with its bias, activation and residual, and its gradients:
//
//   z = x W^T + b,   y = act(z) + residual            x [m, k], W [n, k]
//   dz = dy act'(z),   dx = dz W,   dW = dz^T x,   db = sum of dz's rows
//
// The three products run on the tensor cores (tcgen05, fp32 accumulation).  A
// product is D(i, j) = sum over c of A(i, c) B(j, c); an operand's matrix in
// memory has either its i (j) or its c as rows: x, W and dz are read as they
// lie by all three products (K-major or MN-major operands).
//
// bfloat16 operands are used as they are.  A float32 value is the sum of three
// bfloat16 ones, hi + mid + lo (8 + 8 + 8 bits, the whole float32 range up to
// bfloat16's largest value, and so no scales), and a product is the sum of six
// of theirs: hi hi, hi mid, mid hi, mid mid, hi lo, lo hi.  The other three are
// at most 2^-23 of it and, their signs being random, far below the rounding of
// a sum in 32 bits.
#include <cuda.h>

#include <type_traits>

#include "learn_internal.cuh"
#include "tensor_core.cuh"

namespace pulsar {
namespace {

constexpr int kPanel = 64;       // of the contraction, per stage: 128 bytes of a swizzled row
constexpr int kBlock = 128;      // rows of a tile
constexpr int kMaxPlanes = 3;

// ------------------------------------------------------------ activation --
// 1 / (1 + exp(-z)) by the PTX ISA's approximate base-2 exponential and reciprocal, with
// subnormals flushed: a few ulps, and below 2^-125 (z < -87) zero.  Five instructions; without the
// flush, and as a division, eleven.
__device__ __forceinline__ float sigmoid_of(float z) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
}
template <int kAct>
__device__ __forceinline__ float act_of(float z) {
    if (kAct == kActSilu) return z * sigmoid_of(z);
    if (kAct == kActRelu) return z > 0.0f ? z : 0.0f;
    return z;
}
template <int kAct>
__device__ __forceinline__ float act_slope(float z) {
    if (kAct == kActSilu) {
        const float s = sigmoid_of(z);
        return s * (1.0f + z * (1.0f - s));
    }
    if (kAct == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
    return 1.0f;
}
// ---------------------------------------------------------------- planes --
// Two floats as three words of two bfloat16 each, whose sums they are (an infinity, or what rounds
// to one, leaves NaNs over).
__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void split3(float a, float b, uint32_t (&w)[3]) {
    w[0] = pair_bf16(a, b);
    a -= low_of(w[0]);
    b -= high_of(w[0]);
    w[1] = pair_bf16(a, b);
    w[2] = pair_bf16(a - low_of(w[1]), b - high_of(w[1]));
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, float (&v)[8]) {
    constexpr int V = VecOf<T>::n;
    if (vec) {
#pragma unroll
        for (int h = 0; h < 8; h += V) {
            float u[V];
            Pack<T, V>::load(p + h, u);
#pragma unroll
            for (int e = 0; e < V; ++e) v[h + e] = u[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float u[1] = {0.0f};
            if (e < n) Pack<T, 1>::load(p + e, u);
            v[e] = u[0];
        }
    }
}

// kCount consecutive elements at any alignment, from the 16-byte vectors that they lie in.
template <typename T, int kCount>
struct Window {
    static constexpr int kSize = (int)sizeof(T), kVectors = kCount * kSize / 16 + 1;
    uint4 raw[kVectors];
    int shift;   // elements from the first vector's beginning

    __device__ __forceinline__ void load_shared(uint32_t at) {
        shift = (int)(at & 15u) / kSize;
        at &= ~15u;
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(raw[i].x), "=r"(raw[i].y), "=r"(raw[i].z), "=r"(raw[i].w)
                         : "r"(at + 16 * i));
    }
    // whether the vectors lie within [begin, end)
    __device__ __forceinline__ static bool within(const T* p, const T* begin, const T* end) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15;
        return at >= reinterpret_cast<uintptr_t>(begin) &&
               at + 16 * kVectors <= reinterpret_cast<uintptr_t>(end);
    }
    __device__ __forceinline__ void load(const T* p) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        shift = (int)(at & 15u) / kSize;
        const uint4* v = reinterpret_cast<const uint4*>(at & ~(uintptr_t)15);
#pragma unroll
        for (int i = 0; i < kVectors; ++i) raw[i] = v[i];
    }
    __device__ __forceinline__ void open(float (&v)[kCount]) const {
        constexpr int kWords = 4 * kVectors;
        uint32_t w[kWords];
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            w[4 * i] = raw[i].x;
            w[4 * i + 1] = raw[i].y;
            w[4 * i + 2] = raw[i].z;
            w[4 * i + 3] = raw[i].w;
        }
        if constexpr (kSize == 4) {
#pragma unroll
            for (int i = 0; i + 2 < kWords; ++i) w[i] = shift & 2 ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i < kCount; ++i) v[i] = __uint_as_float(shift & 1 ? w[i + 1] : w[i]);
        } else {
#pragma unroll
            for (int i = 0; i + 2 < kWords; ++i) w[i] = shift & 4 ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i + 3 < kWords; ++i) w[i] = shift & 2 ? w[i + 1] : w[i];
#pragma unroll
            for (int i = 0; i < kCount / 2; ++i) {
                const uint32_t u = shift & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
                v[2 * i] = low_of(u);
                v[2 * i + 1] = high_of(u);
            }
        }
    }
};

// Eight columns of a row as they were loaded: nothing waits for them before they are opened.
template <typename T>
struct Chunk {
    static constexpr int V = VecOf<T>::n;
    typename Pack<T, V>::Raw raw[8 / V];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int h = 0; h < 8 / V; ++h) raw[h] = Pack<T, V>::raw_last(p + h * V);
    }
    __device__ __forceinline__ void open(float (&v)[8]) const {
#pragma unroll
        for (int h = 0; h < 8 / V; ++h) {
            float u[V];
            Pack<T, V>::open(raw[h], u);
#pragma unroll
            for (int e = 0; e < V; ++e) v[h * V + e] = u[e];
        }
    }
};

// dy made dz = dy act'(z)
template <int kAct, int V>
__device__ __forceinline__ void to_dz(float (&v)[V], const float (&z)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (kAct == kActRelu) v[e] = z[e] > 0.0f ? v[e] : 0.0f;
        if (kAct == kActSilu) v[e] *= act_slope<kActSilu>(z[e]);
    }
}

// Eight columns, 16 bytes of bfloat16 in each plane.
template <int kPlanes>
__device__ __forceinline__ void put_chunk(void* at, size_t plane_bytes, const float (&v)[8]) {
    uint32_t w[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (kPlanes == 3)
            split3(v[2 * e], v[2 * e + 1], w[e]);
        else
            w[e][0] = pair_bf16(v[2 * e], v[2 * e + 1]);
    }
#pragma unroll
    for (int p = 0; p < kPlanes; ++p)
        *reinterpret_cast<uint4*>(static_cast<unsigned char*>(at) + p * plane_bytes) =
            make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
}

// A matrix [rows, cols] made into an operand: times the activation's slope at `pre` (the gradient
// dz from dy), split into planes [planes][rows][pitch] of bfloat16, and its column sums taken, a
// partial sum [cols] per block of rows.  A thread has eight columns of every (256 / tx)-th row.
struct Operand {
    const void* src;
    const void* pre;
    int64_t rows, cols;
    int64_t pitch;          // a multiple of 8
    __nv_bfloat16* planes;  // NULL: none are wanted
    size_t plane;           // elements from one plane to the next
    float* sums;            // NULL: none are wanted
    int tx;                 // threads along the columns: a power of two up to 32
    int64_t block_rows;
    unsigned blocks, col_blocks;
    bool vec;
};
struct Operands {   // of one call: the first may be a gradient with its activation
    Operand of[3];
};

template <typename T, int kPlanes, int kAct>
__device__ __forceinline__ void make_planes(const Operand& q, float* s_sums) {
    const int tx = threadIdx.x & (q.tx - 1), ty = threadIdx.x / q.tx, step = 256 / q.tx;
    const int64_t c = ((int64_t)blockIdx.y * q.tx + tx) * 8;
    const int n = (int)(q.cols - c < 8 ? q.cols - c : 8);
    const int64_t r0 = blockIdx.x * q.block_rows;
    const int64_t r1 = r0 + q.block_rows < q.rows ? r0 + q.block_rows : q.rows;
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
    const T* src = static_cast<const T*>(q.src) + c;
    const T* pre = static_cast<const T*>(q.pre) + c;
    const auto finish = [&](int64_t r, float (&v)[8], const float (&z)[8]) {
        to_dz<kAct>(v, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += e < n ? v[e] : 0.0f;
        if (q.planes) put_chunk<kPlanes>(q.planes + r * q.pitch + c, q.plane * 2, v);
    };
    if (q.vec && n == 8) {
        constexpr int kBatch = sizeof(T) == 4 ? 2 : 4;   // rows whose loads are in flight together
        for (int64_t r = r0 + ty; r < r1; r += kBatch * step) {
            Chunk<T> a[kBatch], b[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t at = (r + i * step) * q.cols;
                if (r + i * step < r1) {
                    a[i].load(src + at);
                    if (kAct != kActNone) b[i].load(pre + at);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float v[8], z[8];
                a[i].open(v);
                if (kAct != kActNone) b[i].open(z);
                if (r + i * step < r1) finish(r + i * step, v, z);
            }
        }
    } else if (n > 0) {
        const T* end = static_cast<const T*>(q.src) + q.rows * q.cols;
        const T* pre_end = static_cast<const T*>(q.pre) + q.rows * q.cols;
        const auto load = [&](const T* p, const T* begin, const T* stop, float (&v)[8]) {
            if (Window<T, 8>::within(p, begin, stop)) {
                Window<T, 8> w;
                w.load(p);
                w.open(v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = e < n ? v[e] : 0.0f;
            } else {
                load8(p, n, false, v);
            }
        };
#pragma unroll 2
        for (int64_t r = r0 + ty; r < r1; r += step) {
            float v[8], z[8];
            load(src + r * q.cols, static_cast<const T*>(q.src), end, v);
            if (kAct != kActNone)
                load(pre + r * q.cols, static_cast<const T*>(q.pre), pre_end, z);
            finish(r, v, z);
        }
    }
    if (!q.sums) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) s_sums[(ty * q.tx + tx) * 8 + e] = sum[e];
    __syncthreads();
    for (int half = step / 2; half > 0; half /= 2) {   // [step][8 tx] by halves
        for (int i = threadIdx.x; i < half * q.tx * 8; i += 256)
            s_sums[i] += s_sums[i + half * q.tx * 8];
        __syncthreads();
    }
    for (int i = threadIdx.x; i < q.tx * 8; i += 256) {
        const int64_t col = (int64_t)blockIdx.y * q.tx * 8 + i;
        if (col < q.cols) q.sums[(int64_t)blockIdx.x * q.cols + col] = s_sums[i];
    }
}

template <typename T, int kPlanes, int kAct>
__global__ void __launch_bounds__(256)
k_linear_operands(const __grid_constant__ Operands all) {
    __shared__ float s_sums[256 * 8];
    pdl_next();
    pdl_begin();
    const Operand& q = all.of[blockIdx.z];
    if (blockIdx.x >= q.blocks || blockIdx.y >= q.col_blocks) return;
    if (blockIdx.z == 0) make_planes<T, kPlanes, kAct>(q, s_sums);
    else make_planes<T, kPlanes, kActNone>(q, s_sums);
}

// The sums of `blocks` partial rows of `cols`: 32 columns a block, 32 rows of threads.
__global__ void __launch_bounds__(1024)
k_linear_sums(const float* __restrict__ part, int64_t blocks, int64_t cols,
              float* __restrict__ out) {
    __shared__ float s[32][33];
    pdl_begin();
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float v = 0.0f;
    if (col < cols)
        for (int64_t b = threadIdx.y; b < blocks; b += 32) v += part[b * cols + col];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = s[threadIdx.x][threadIdx.y];   // a warp per column
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
    const int64_t mine = (int64_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && mine < cols) out[mine] = v;
}

// -------------------------------------------------------------- products --
// One kernel for the three products, a persistent CTA per SM.  Roles: one
// thread keeps a ring of operand stages filled by TMA (out of range: zeros), one
// issues the MMAs into one of two accumulators in tensor memory, and the other
// warps finish the other (four per half or quarter of the tile's columns, a
// thread per row): bias, activation, residual, rounding; through a swizzled exchange in
// shared memory, so that a warp stores whole sectors.
//
// In 32 bits the tensor cores' accumulation, which truncates, would be what
// limits the result (of K = 2048, some 2^-18.5 of it): hi hi and the other
// five products have accumulators of their own, and both are drained and
// summed in registers every kChunk panels (128 of K).
//
// Where a product has few tiles for the SMs and a long contraction (dW: one
// tile and a million rows), its parts are separate work items, whose sums
// k_linear_join adds up in their order.
struct Product {
    CUtensorMap a, b;
    int tiles_m, tiles_n, splits, panels;   // panels of the contraction
    int64_t m, n;
    int64_t part;   // floats from one part's sums to the next
    // the finished result, or, where there are parts, their sums [splits][m][n]
    const float* bias;
    const void* residual;
    void* pre;
    void* out;
    int act;
    bool vec;   // four columns at a time
};

// warps: copies, MMAs, and of the epilogue eight, or in 16 bits, where it has every tile's
// activation to do within the MMAs' time, sixteen
constexpr int epilogue_warps(int planes) { return planes == 3 ? 8 : 16; }
constexpr int kChunk = 2;              // panels per drained sum (32 bits)
constexpr int kGroup = 16;             // row blocks whose tiles lie side by side in time

template <int kPlanes, int kN, int kCtas>
struct ProductSmem {
    static constexpr int rows_b = kN / kCtas;   // of B, in each CTA of a pair
    static constexpr int a = kBlock * kPanel * 2, b = rows_b * kPanel * 2;
    static constexpr int stage = kPlanes * (a + b);
    static constexpr int epilogue = epilogue_warps(kPlanes), threads = 64 + 32 * epilogue;
    // a warp's exchange: 32 x 32 words, in 32 bits 32 x 8 for a third stage
    static constexpr int warp_exchange = 32 * (kPlanes == 3 ? 8 : 32) * 4;
    static constexpr int exchange_bytes = epilogue * warp_exchange;
    static constexpr int stages = (227 * 1024 - 1024 - exchange_bytes - 256) / stage;
    static constexpr int exchange = stages * stage;
    static constexpr int bars = exchange + exchange_bytes;
    static constexpr int bytes = bars + 256 + 1024;   // and the alignment to 1024
    static_assert(stages >= 2 && (2 * stages + 5) * 8 + 8 <= 256, "shared memory of a product");
};

// Descriptor of a 128-byte-swizzled operand: `lbo` is the stride between
// 64-element groups along M/N of an MN-major operand (unused when K-major);
// groups of eight rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// One lane of a whole warp, the compiler knowing that it is one: MMAs issued by it follow each
// other at their own rate, while those of a lane that a comparison chose take 105 cycles each
// (measured: M = 128, N = 64: 76 cycles, with A in tensor memory 49; N = 16: 57 and 35).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void expect_bytes(uint64_t* mbar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(mbar)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_init_n(uint64_t* mbar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(mbar)), "r"(n));
}
__device__ __forceinline__ void mbar_arrive(uint64_t* mbar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(mbar)) : "memory");
}
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* mbar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(mbar))
        : "memory");
}
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
__device__ __forceinline__ void arrive_at(uint32_t mbar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(mbar)
                 : "memory");
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

// What the epilogue does with 32 columns of a warp's 32 rows, a row in each lane: through the
// warp's exchange in shared memory (float4 chunks, swizzled), after which a lane has four columns
// of every fourth row, and a warp reads the residual and writes whole sectors of eight rows' 32
// columns at a time.
// (The residual's sum is kept apart from the activation's last product: whether z is wanted too
// changes no bits.)
__device__ __forceinline__ float plus(float a, float b) { return __fadd_rn(a, b); }

template <typename T>
struct Four;
template <>
struct Four<float> {
    using Raw = float4;
    static __device__ __forceinline__ void add(const Raw& r, float (&y)[4]) {
        y[0] = plus(y[0], r.x); y[1] = plus(y[1], r.y);
        y[2] = plus(y[2], r.z); y[3] = plus(y[3], r.w);
    }
    static __device__ __forceinline__ Raw pack(const float (&y)[4]) {
        return make_float4(y[0], y[1], y[2], y[3]);
    }
};
template <>
struct Four<__nv_bfloat16> {
    using Raw = uint2;
    static __device__ __forceinline__ void add(const Raw& r, float (&y)[4]) {
        y[0] = plus(y[0], low_of(r.x)); y[1] = plus(y[1], high_of(r.x));
        y[2] = plus(y[2], low_of(r.y)); y[3] = plus(y[3], high_of(r.y));
    }
    static __device__ __forceinline__ Raw pack(const float (&y)[4]) {
        return make_uint2(pair_bf16(y[0], y[1]), pair_bf16(y[2], y[3]));
    }
};

// One element of a result: bias (already in z), pre-activation, activation, residual.
template <typename T, int kAct>
__device__ __forceinline__ void finish1(const Product& q, float z, int64_t at) {
    const float one[1] = {z};
    if (q.pre) Pack<T, 1>::store(static_cast<T*>(q.pre) + at, one);
    float y[1] = {act_of<kAct>(z)};
    if (q.residual) {
        float f[1];
        Pack<T, 1>::load(static_cast<const T*>(q.residual) + at, f);
        y[0] = plus(y[0], f[0]);
    }
    Pack<T, 1>::store(static_cast<T*>(q.out) + at, y);
}
template <typename T>
__device__ __forceinline__ void finish1(const Product& q, float z, int64_t at) {
    if (q.act == kActSilu) finish1<T, kActSilu>(q, z, at);
    else if (q.act == kActRelu) finish1<T, kActRelu>(q, z, at);
    else finish1<T, kActNone>(q, z, at);
}

// A block of 32 rows and 32 (or, kSmall, eight) columns whose sums are in the exchange, where rows
// are no whole vectors: as many lanes to a row as it has columns, so that a warp stores what is
// contiguous.  `first`: its first element, col0: its column.
template <typename T, int kAct, bool kSmall>
__device__ __forceinline__ void finish_scalar(const Product& q, const float4* x, int64_t col0,
                                           int64_t first, int64_t left_rows, int lane) {
    const int rows = (int)(left_rows < 32 ? left_rows : 32);
    const int64_t left = q.n - col0;
    const int cols = (int)(left < (kSmall ? 8 : 32) ? left : (kSmall ? 8 : 32));
    int log = 0;
    while (1 << log < cols) ++log;
    const int c = lane & ((1 << log) - 1);
    const float* word = reinterpret_cast<const float*>(x) + (c & 3);
    if (c >= cols) return;
    const float b = q.bias ? q.bias[col0 + c] : 0.0f;
#pragma unroll 1
    for (int r = lane >> log; r < rows; r += 32 >> log) {
        const int at = kSmall ? r * 2 + ((c >> 2) ^ (r >> 2 & 1)) : r * 8 + ((c >> 2) ^ (r & 7));
        finish1<T, kAct>(q, plus(word[at * 4], b), first + r * q.n + c);
    }
}

// A lane's share of the block of 32 rows from r0 and 32 columns from c0.  kVec: rows are whole
// vectors (four columns at a time), known when compiled: kernels that have the other case's
// instructions too were up to a tenth slower.  kSkip: there is a residual.
template <typename T, bool kVec, bool kSkip>
struct Share {
    using Raw = typename Four<T>::Raw;
    int64_t c, at;   // its first column, and its first element
    int n, rows;     // columns (of four), rows that there are from its first on
    Raw residual[kSkip ? 8 : 1];

    // (at: of the element (r0, c0) in a matrix of q.n columns)
    __device__ __forceinline__ void begin(const Product& q, int64_t r0, int64_t c0, int64_t base,
                                          int lane) {
        c = c0 + 4 * (lane & 7);
        n = (int)(q.n - c < 4 ? q.n - c : 4);
        at = base + (r0 + (lane >> 3)) * q.n + c;
        const int64_t left = q.m - r0 - (lane >> 3);
        rows = n <= 0 ? 0 : (int)(left < 32 ? left : 32);
        if (kSkip && kVec) {
#pragma unroll
            for (int h = 0; h < 8; ++h)
                if (4 * h < rows)
                    residual[kSkip ? h : 0] = __ldcs(reinterpret_cast<const Raw*>(
                        static_cast<const T*>(q.residual) + at + (int64_t)4 * h * q.n));
        }
    }

    __device__ __forceinline__ static void put(float4* x, const float (&v)[32], int lane) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[lane * 8 + (e ^ (lane & 7))] =
                make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        __syncwarp();
    }
    __device__ __forceinline__ static float4 get(const float4* x, int r, int lane) {
        return x[r * 8 + ((lane & 7) ^ (r & 7))];
    }

    // `bias`: of its four columns; r0, c0, base as in begin()
    template <int kAct>
    __device__ __forceinline__ void end(const Product& q, float4* x, const float (&v)[32],
                                        const float (&bias)[4], int64_t r0, int64_t c0,
                                        int64_t base, int lane) {
        T* out = static_cast<T*>(q.out) + at;
        T* pre = q.pre ? static_cast<T*>(q.pre) + at : nullptr;
        const int rq = lane >> 3;
        const int64_t step = 4 * q.n;
        if constexpr (kVec) {
            // (all loads, then all stores: the compiler keeps a load behind a store before it)
            float z[8][4];
            put(x, v, lane);
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const float4 u = get(x, 4 * h + rq, lane);
                z[h][0] = plus(u.x, bias[0]);
                z[h][1] = plus(u.y, bias[1]);
                z[h][2] = plus(u.z, bias[2]);
                z[h][3] = plus(u.w, bias[3]);
            }
            if (pre) {
#pragma unroll
                for (int h = 0; h < 8; ++h)
                    if (4 * h < rows) *reinterpret_cast<Raw*>(pre + h * step) = Four<T>::pack(z[h]);
            }
#pragma unroll
            for (int h = 0; h < 8; ++h) {
#pragma unroll
                for (int e = 0; e < 4; ++e) z[h][e] = act_of<kAct>(z[h][e]);
                if (kSkip) Four<T>::add(residual[kSkip ? h : 0], z[h]);
            }
#pragma unroll
            for (int h = 0; h < 8; ++h)
                if (4 * h < rows) *reinterpret_cast<Raw*>(out + h * step) = Four<T>::pack(z[h]);
        } else {
            put(x, v, lane);
            finish_scalar<T, kAct, false>(q, x, c0, base + r0 * q.n + c0, q.m - r0, lane);
        }
    }
    __device__ __forceinline__ void end(const Product& q, float4* x, const float (&v)[32],
                                        const float (&bias)[4], int64_t r0, int64_t c0,
                                        int64_t base, int lane) {
        if (q.act == kActSilu) end<kActSilu>(q, x, v, bias, r0, c0, base, lane);
        else if (q.act == kActRelu) end<kActRelu>(q, x, v, bias, r0, c0, base, lane);
        else end<kActNone>(q, x, v, bias, r0, c0, base, lane);
    }
};

// The same where there is room for an exchange of 32 x 8 words only: eight columns at a time, of
// which a lane has four of every 16th row; a warp stores sectors.  (kPlain: the sums are the result.)
template <typename T, int kAct, bool kPlain, bool kVec>
__device__ __forceinline__ void finish_small(const Product& q, float4* x, const float (&v)[32],
                                             int64_t r0, int64_t c0, int64_t base, int lane) {
    using Raw = typename Four<T>::Raw;
    const int j = lane & 1, rq = lane >> 1;
    const int64_t left = q.m - r0 - rq, at0 = base + (r0 + rq) * q.n + c0 + 4 * j;
    const int rows = (int)(left < 32 ? left : 32);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            x[lane * 2 + (i ^ (lane >> 2 & 1))] =
                make_float4(v[8 * m + 4 * i], v[8 * m + 4 * i + 1], v[8 * m + 4 * i + 2],
                            v[8 * m + 4 * i + 3]);
        __syncwarp();
        const int64_t c = c0 + 8 * m + 4 * j;
        const int n = (int)(q.n - c < 4 ? q.n - c : 4);
        float z[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 16 * h + rq;
            const float4 u = x[r * 2 + (j ^ (r >> 2 & 1))];
            z[h][0] = u.x;
            z[h][1] = u.y;
            z[h][2] = u.z;
            z[h][3] = u.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (kPlain) continue;
            const float bias = q.bias && e < n ? q.bias[c + e] : 0.0f;
            z[0][e] = plus(z[0][e], bias);
            z[1][e] = plus(z[1][e], bias);
        }
        if constexpr (!kVec) {
            finish_scalar<T, kAct, true>(q, x, c0 + 8 * m, base + r0 * q.n + c0 + 8 * m, q.m - r0,
                                         lane);
            continue;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (16 * h >= rows || n <= 0) continue;
            const int64_t at = at0 + 16 * h * q.n + 8 * m;
            if (!kPlain && q.pre)
                *reinterpret_cast<Raw*>(static_cast<T*>(q.pre) + at) = Four<T>::pack(z[h]);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[h][e] = act_of<kAct>(z[h][e]);
            if (!kPlain && q.residual)
                Four<T>::add(*reinterpret_cast<const Raw*>(static_cast<const T*>(q.residual) + at),
                             z[h]);
            *reinterpret_cast<Raw*>(static_cast<T*>(q.out) + at) = Four<T>::pack(z[h]);
        }
    }
}

// T: the result's type (float for parts).  kAMn, kBMn: the operand's matrix has the contraction
// as its rows.  kCtas: 1, or a pair of CTAs on a tile of 256 rows, each with its 128 rows of A and
// of the sums, and half of B's; the first one issues the MMAs of both.
template <typename T, int kPlanes, int kN, bool kAMn, bool kBMn, int kCtas, bool kVec>
__global__ void __launch_bounds__(64 + 32 * epilogue_warps(kPlanes)) __cluster_dims__(kCtas, 1, 1)
k_linear_product(const __grid_constant__ Product q, LearnState* st) {
    using L = ProductSmem<kPlanes, kN, kCtas>;
    constexpr bool kPair = kCtas == 2;
    constexpr int kAcc = kPlanes == 3 ? 2 * kN : kN;   // columns of an accumulator
    constexpr int kHalf = kN / (L::epilogue / 4);      // columns of an epilogue thread
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
    const int tiles = q.tiles_m * q.tiles_n, total = tiles * q.splits;
    auto place = [&](int t, int* i, int* j, int* k0, int* k1, int* part) {
        *part = t / tiles;
        t -= *part * tiles;
        const int g = t / (kGroup * q.tiles_n), rows = min(kGroup, q.tiles_m - g * kGroup);
        t -= g * kGroup * q.tiles_n;
        *i = g * kGroup + t % rows;
        *j = t / rows;
        *k0 = (int)((int64_t)*part * q.panels / q.splits);
        *k1 = (int)((int64_t)(*part + 1) * q.panels / q.splits);
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
                const int chunk = kPlanes == 3 ? kChunk : k1 - k0;
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
            const int64_t base = part * q.part;
            // 32 columns from `col` of the tile, a row in each lane
            auto emit = [&](const float (&v)[32], int col) {
                const int64_t c0 = (int64_t)j * kN + col;
                if constexpr (kPlanes == 3) {
                    if (kAMn || kBMn)
                        finish_small<T, kActNone, true, kVec>(q, x, v, r0, c0, base, lane);
                    else if (q.act == kActNone)
                        finish_small<T, kActNone, false, kVec>(q, x, v, r0, c0, base, lane);
                    else if (q.act == kActSilu)
                        finish_small<T, kActSilu, false, kVec>(q, x, v, r0, c0, base, lane);
                    else
                        finish_small<T, kActRelu, false, kVec>(q, x, v, r0, c0, base, lane);
                } else {
                    const auto finish = [&](auto skip) {
                        Share<T, kVec, decltype(skip)::value> share;
                        share.begin(q, r0, c0, base, lane);
                        float bias[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            bias[e] = q.bias && e < share.n ? q.bias[share.c + e] : 0.0f;
                        if (kAMn || kBMn)
                            share.template end<kActNone>(q, x, v, bias, r0, c0, base, lane);
                        else
                            share.end(q, x, v, bias, r0, c0, base, lane);
                    };
                    if (kAMn || kBMn || !q.residual) finish(std::false_type());
                    else finish(std::true_type());
                }
            };
            bool ok = true;
            if constexpr (kPlanes == 3) {
                float v[kHalf];
#pragma unroll
                for (int e = 0; e < kHalf; ++e) v[e] = 0.0f;
                for (int kc = k0; kc < k1; kc += kChunk, ++it) {
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
                        tmem_ld16(acc + kN + h, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            v[h + e] += __uint_as_float(u[e]) + __uint_as_float(w[e]);
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

// The parts of a product added in a fixed order, and finished: a thread has four columns, of few
// parts all of them, of many (kLanes = 64) every 64th, which the block then adds up.
template <typename T, int kLanes>
__global__ void __launch_bounds__(256)
k_linear_join(const __grid_constant__ Product q, const float* __restrict__ part) {
    constexpr int kPer = 256 / kLanes;   // groups of four columns of a block
    __shared__ float4 s_sum[8][kLanes > 1 ? kPer : 1];
    pdl_begin();
    const int64_t size = q.m * q.n, total = (size + 3) / 4;
    const int mine = threadIdx.x % kPer, from = threadIdx.x / kPer;
    for (int64_t g0 = (int64_t)blockIdx.x * kPer; g0 < total; g0 += (int64_t)gridDim.x * kPer) {
        const int64_t at = (g0 + mine) * 4;
        const int n = (int)(size - at < 4 ? size - at : 4);   // (a part ends on a whole vector)
        float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (n > 0) {
#pragma unroll 8
            for (int s = from; s < q.splits; s += kLanes) {
                const float4 u = __ldcs(reinterpret_cast<const float4*>(part + s * q.part + at));
                z[0] += u.x; z[1] += u.y; z[2] += u.z; z[3] += u.w;
            }
        }
        if (kLanes > 1) {   // the warp's (its lanes kPer apart), then the block's
#pragma unroll
            for (int d = kPer; d < 32; d *= 2)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] += __shfl_xor_sync(0xffffffffu, z[e], d);
            __syncthreads();
            if ((threadIdx.x & 31) < kPer)
                s_sum[threadIdx.x >> 5][kLanes > 1 ? mine : 0] = make_float4(z[0], z[1], z[2], z[3]);
            __syncthreads();
            if (from > 0) continue;
            for (int e = 0; e < 4; ++e) z[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const float4 u = s_sum[w][kLanes > 1 ? mine : 0];
                z[0] += u.x; z[1] += u.y; z[2] += u.z; z[3] += u.w;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) finish1<T>(q, plus(z[e], q.bias ? q.bias[(at + e) % q.n] : 0.0f), at + e);
    }
}

// -------------------------------------------------------------- few rows --
// Up to kFewRows rows are bound by reading the weights once: the products are
// taken in 32 bits, `per` warps to an output, their lanes along the inputs: so
// many that a lane has up to eight vectors of the weights to take, four of them
// in flight (a row of 4096 into 2048 outputs in 16 bits: 5.1 us in a chain of
// launches, 2.5 by the bytes; one warp to an output, which leaves the SMs one or
// two blocks each, 5.8, and with four rows 10.3 instead of 6.9).
constexpr int kFewRows = 8;

template <typename T, int V, int kRows>
__global__ void __launch_bounds__(256)
k_linear_rows(const T* __restrict__ x, const T* __restrict__ weight, int64_t k, int per,
              const __grid_constant__ Product q) {
    __shared__ float s_sum[8][kRows];
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp & (per - 1);
    const int64_t j = blockIdx.x * (int64_t)(8 / per) + warp / per;
    float sum[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) sum[r] = 0.0f;
    if (j < q.n) {
        const T* w = weight + j * k;
        const int64_t step = (int64_t)per * 32 * V;
        constexpr int kBatch = 4;
        for (int64_t c0 = (part * 32 + lane) * V; c0 < k; c0 += kBatch * step) {
            typename Pack<T, V>::Raw u[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (c0 + i * step < k) u[i] = Pack<T, V>::raw_last(w + c0 + i * step);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (c0 + i * step >= k) continue;
                float a[V];
                Pack<T, V>::open(u[i], a);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    float v[V];
                    Pack<T, V>::load(x + r * k + c0 + i * step, v);
#pragma unroll
                    for (int e = 0; e < V; ++e) sum[r] = fmaf(a[e], v[e], sum[r]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
        for (int d = 16; d > 0; d /= 2) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], d);
        if (lane == 0) s_sum[warp][r] = sum[r];
    }
    __syncthreads();
    if (part == 0 && lane < kRows && j < q.n) {
        float z = s_sum[warp][lane];
        for (int p = 1; p < per; ++p) z += s_sum[warp + p][lane];
        finish1<T>(q, plus(z, q.bias ? q.bias[j] : 0.0f), lane * q.n + j);
    }
}

// ---------------------------------------------------------- narrow layers --
// A layer of few inputs and outputs over many rows (a network's hidden layer
// over an image) is bound by its rows' way in and out.  One launch, a
// persistent CTA per SM, tiles of 128 rows, each read and written once.  Roles:
// one thread keeps a ring of raw tiles filled (128 rows are one contiguous bulk
// copy, whatever their width), eight warps make a tile's operand from it, 64
// columns of the contraction at a time (in 32 bits its three planes), one
// thread issues the MMAs, and eight warps finish the tile from tensor memory.
// The weights are made into operands by every CTA once, and stay.
//
// In 32 bits the weights' planes lie below one another, [hi; mid; lo], so that a
// plane of the rows takes one MMA against those that count: hi against all
// three, mid against hi and mid, lo against hi.  Their sums in three ranges of
// columns are hi hi, (hi mid + mid hi), (hi lo + mid mid + lo hi), so that what
// the tensor cores truncate is relative to each, of at most 128 of K, as there.
// (Six MMAs into one accumulator, hi hi last, are as exact; an MMA takes some
// 140 cycles whatever its columns, and 24 of them were 80 % of a tile's time.)
constexpr int kStreamThreads = 576;   // warps: copies, MMAs, eight of operands, eight of the epilogue
constexpr int kStreamMaxK = 128;
template <typename T>
constexpr int kStreamN = sizeof(T) == 4 ? 64 : 128;   // outputs of a CTA

struct Stream {
    const void* x;         // [m, k]
    const void* weight;    // [n, k]
    int64_t tiles;
    int k, panels;         // of the contraction
    int np, blocks;        // outputs of a block (a multiple of 16), blocks
    int raws, units;       // raw tiles, operand panels in flight
    bool vec;              // a row of x, and of the weight, is whole 16-byte vectors
    bool skip;             // there is a residual, on 16 bytes, and one block of outputs
    Product out;           // m, n, bias, ..., vec
};
struct StreamSmem {
    int raw, raw_bytes, unit, unit_bytes, weight, weight_panel, exchange, bars, bytes;
};
__host__ __device__ inline StreamSmem stream_smem(int planes, int size, int k, int panels, int np,
                                                  int raws, int units) {
    StreamSmem s;
    s.unit = 0;
    s.unit_bytes = planes * kBlock * kPanel * 2;
    s.weight = s.unit + units * s.unit_bytes;
    s.weight_panel = planes * np * kPanel * 2;
    s.exchange = s.weight + panels * s.weight_panel;
    s.raw = s.exchange + 8 * 32 * 32 * 4;
    s.raw_bytes = (kBlock * k * size + 127) / 128 * 128;
    s.bars = s.raw + raws * s.raw_bytes;
    s.bytes = s.bars + 256 + 1024;
    return s;
}
constexpr int kStreamSmemMax = 227 * 1024 - 512;   // (and the bias)

__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    if (bytes)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

// kVec: rows of x and of the result are whole vectors.  kSkip: there is a residual.
template <typename T, bool kVec, bool kSkip>
__global__ void __launch_bounds__(kStreamThreads, 1)
k_linear_stream(const __grid_constant__ Stream q, LearnState* st) {
    constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
    constexpr int kCols = sizeof(T) == 4 ? 512 : 256;   // tensor memory: two accumulators
    extern __shared__ unsigned char raw_smem[];
    __shared__ __align__(16) float s_bias[128];
    unsigned char* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
    const StreamSmem L = stream_smem(kPlanes, sizeof(T), q.k, q.panels, q.np, q.raws, q.units);
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + L.bars);
    uint64_t* raw_empty = raw_full + 4;
    uint64_t* unit_full = raw_empty + 4;
    uint64_t* unit_empty = unit_full + 4;
    uint64_t* acc_full = unit_empty + 4;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* s_taddr = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* s_fail = s_taddr + 1;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (known to be the same in a warp)
    const int block = blockIdx.x % q.blocks, first = blockIdx.x / q.blocks;
    const int step = gridDim.x / q.blocks;
    const int n0 = block * kStreamN<T>;
    const int steps16 = (q.k + 15) / 16;
    if (tid == 0) {
        for (int s = 0; s < 4; ++s) {
            mbar_init(raw_full + s);
            mbar_init_n(raw_empty + s, 8);
            mbar_init_n(unit_full + s, 8);
            mbar_init(unit_empty + s);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + s);
            mbar_init_n(acc_empty + s, 8);
        }
        mbar_init(drain);
        *s_fail = 0u;
    }
    if (warp == 1) tmem_alloc(s_taddr, kCols);
    pdl_next();
    pdl_begin();
    if (tid < 128)
        s_bias[tid] = q.out.bias && n0 + tid < q.out.n ? q.out.bias[n0 + tid] : 0.0f;
    {   // the weights, zeros below and behind them
        const int chunks = steps16 * 2, total = q.np * chunks;
        for (int t = tid; t < total; t += kStreamThreads) {
            const int r = t / chunks, c = t % chunks;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            const int n = q.k - c * 8 < 8 ? q.k - c * 8 : 8;
            if (n0 + r < q.out.n && n > 0)
                load8(static_cast<const T*>(q.weight) + (int64_t)(n0 + r) * q.k + c * 8, n,
                      q.vec && n == 8, v);
            put_chunk<kPlanes>(smem + L.weight + (c >> 3) * L.weight_panel + r * 128 +
                                   (((c & 7) ^ (r & 7)) << 4),
                               q.np * 128, v);
        }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_taddr;
    if (warp == 0) {
        if (elect_one()) {   // ---- raw tiles
            int n = 0;
            bool ok = true;
            for (int64_t t = first; t < q.tiles; t += step, ++n) {
                const int s = n % q.raws;
                ok = mbar_wait(raw_empty + s, ((n / q.raws) & 1) ^ 1) && !*s_fail;
                if (!ok) break;
                const int64_t left = q.out.m - t * kBlock;
                const uint32_t bytes =
                    (uint32_t)((left < kBlock ? left : kBlock) * q.k * (int)sizeof(T));
                const unsigned char* src =
                    static_cast<const unsigned char*>(q.x) + t * kBlock * q.k * (int64_t)sizeof(T);
                unsigned char* dst = smem + L.raw + s * L.raw_bytes;
                if (q.skip) {   // its residual is on its way to the L2 before the epilogue asks
                    const uint32_t row = (uint32_t)(q.out.n * (int)sizeof(T));
                    prefetch_l2(static_cast<const unsigned char*>(q.out.residual) +
                                    t * kBlock * (int64_t)row,
                                (uint32_t)(left < kBlock ? left : kBlock) * row & ~15u);
                }
                const uint32_t bulk = bytes & ~15u;   // the last rows need not end on 16 bytes
                for (uint32_t e = bulk / sizeof(T); e < bytes / sizeof(T); ++e)
                    reinterpret_cast<T*>(dst)[e] = reinterpret_cast<const T*>(src)[e];
                if (bulk)
                    bulk_load(dst, src, bulk, raw_full + s);
                else
                    mbar_arrive(raw_full + s);
            }
            if (!ok) {   // give the copies in flight one more bounded wait
                *s_fail = 1u;
                for (int k = n > q.raws ? n - q.raws : 0; k < n; ++k)
                    mbar_wait(raw_full + k % q.raws, (k / q.raws) & 1);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {   // ---- MMAs
            const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) |
                                    ((uint32_t)(kBlock >> 4) << 24);
            const uint32_t np = (uint32_t)q.np;
            uint32_t idesc[kPlanes];   // against the weights' first kPlanes - p planes
#pragma unroll
            for (int p = 0; p < kPlanes; ++p)
                idesc[p] = idesc0 | ((np * (uint32_t)(kPlanes - p) >> 3) << 17);
            const uint32_t base = smem_u32(smem);
            int u = 0, it = 0;
            bool ok = true;
            for (int64_t t = first; t < q.tiles && ok; t += step, ++it) {
                const int buf = it & 1;
                const uint32_t d = tmem + buf * (kCols / 2);
                ok = mbar_wait(acc_empty + buf, ((it >> 1) & 1) ^ 1) && !*s_fail;
                if (!ok) break;
                for (int h = 0; h < q.panels; ++h, ++u) {
                    const int s = u % q.units;
                    ok = mbar_wait(unit_full + s, (u / q.units) & 1) && !*s_fail;
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = base + L.unit + s * L.unit_bytes;
                    const uint64_t b = desc_sw128(base + L.weight + h * L.weight_panel, 16);
                    uint64_t a[kPlanes];
#pragma unroll
                    for (int p = 0; p < kPlanes; ++p)
                        a[p] = desc_sw128(at + p * kBlock * kPanel * 2, 16);
                    const int ends = min(4, steps16 - 4 * h);
                    for (int e = 0; e < ends; ++e) {
                        const uint32_t off = 32u * e >> 4;
                        mma_f16(d, a[0] + off, b + off, idesc[0], h > 0 || e > 0);
#pragma unroll
                        for (int p = 1; p < kPlanes; ++p)
                            mma_f16(d + p * np, a[p] + off, b + off, idesc[p], 1);
                    }
                    mma_commit(unit_empty + s);
                }
                if (ok) mma_commit(acc_full + buf);
            }
            if (!ok) {
                *s_fail = 1u;
                mma_commit(drain);
                mbar_wait(drain, 0);
            }
        }
    } else if (warp < 10) {   // ---- operands
        const int mine = tid - 64;
        int n = 0, u = 0;
        bool ok = true;
        for (int64_t t = first; t < q.tiles && ok; t += step, ++n) {
            const int s = n % q.raws;
            ok = warp_all(mbar_wait(raw_full + s, (n / q.raws) & 1) && !*s_fail);
            if (!ok) break;
            const T* tile = reinterpret_cast<const T*>(smem + L.raw + s * L.raw_bytes);
            const int64_t left = q.out.m - t * kBlock;
            const int rows = (int)(left < kBlock ? left : kBlock);
            for (int h = 0; h < q.panels; ++h, ++u) {
                const int a = u % q.units;
                ok = warp_all(mbar_wait(unit_empty + a, ((u / q.units) & 1) ^ 1) && !*s_fail);
                if (!ok) break;
                unsigned char* unit = smem + L.unit + a * L.unit_bytes;
                const int chunks = min(8, 2 * steps16 - 8 * h);
                // a thread has a chunk of every 32nd row (rows behind the last keep what they
                // held: their sums are not stored)
                const int c = mine & 7, r0 = mine >> 3, col = h * kPanel + c * 8;
                const T* src = tile + r0 * q.k + col;
                unsigned char* dst = unit + r0 * 128 + ((c ^ (r0 & 7)) << 4);
                if ((kVec || q.vec) && q.k - col >= 8) {
                    float v[4][8];   // (all loads, then all stores, as there)
#pragma unroll
                    for (int i = 0; i < 4; ++i) load8(src + 32 * i * q.k, 8, true, v[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        put_chunk<kPlanes>(dst + 32 * i * 128, kBlock * kPanel * 2, v[i]);
                } else if (c < chunks) {   // (what lies behind the last row is shared too)
                    const uint32_t at = smem_u32(src);
                    Window<T, 8> w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i].load_shared(at + (uint32_t)(32 * i * q.k * (int)sizeof(T)));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v[8];
                        w[i].open(v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = col + e < q.k ? v[e] : 0.0f;
                        put_chunk<kPlanes>(dst + 32 * i * 128, kBlock * kPanel * 2, v);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(unit_full + a);
            }
            if (lane == 0) mbar_arrive(raw_empty + s);   // (after the last __syncwarp)
        }
        if (!ok) *s_fail = 1u;
    } else {   // ---- epilogue
        const int e0 = warp - 10, quarter = warp & 3, group = e0 >> 2;
        float4* x = reinterpret_cast<float4*>(smem + L.exchange) + e0 * 256;
        int it = 0;
        for (int64_t t = first; t < q.tiles; t += step, ++it) {
            const int buf = it & 1;
            const int64_t r0 = t * kBlock + quarter * 32;
            Share<T, kVec, kSkip> share;
            if (group * 32 < q.np) share.begin(q.out, r0, n0 + group * 32, 0, lane);
            const bool ok = warp_all(mbar_wait(acc_full + buf, (it >> 1) & 1) && !*s_fail);
            if (!ok) {
                *s_fail = 1u;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + buf * (kCols / 2) + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
            for (int c = group * 32; c < q.np; c += 64) {
                float v[32];
#pragma unroll
                for (int p = 0; p < kPlanes; ++p) {
                    uint32_t w[32];
                    __syncwarp();
                    tmem_ld32(acc + p * q.np + c, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        v[e] = p ? v[e] + __uint_as_float(w[e]) : __uint_as_float(w[e]);
                }
                if (c + 64 >= q.np) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty + buf);
                }
                if (c != group * 32) share.begin(q.out, r0, n0 + c, 0, lane);
                const float4 b = *reinterpret_cast<const float4*>(s_bias + c + 4 * (lane & 7));
                const float bias[4] = {b.x, b.y, b.z, b.w};
                share.end(q.out, x, v, bias, r0, n0 + c, 0, lane);
            }
            if (group * 32 >= q.np && lane == 0) mbar_arrive(acc_empty + buf);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *s_fail) atomicOr(&st->error, kErrTimeout);
    if (warp == 1) tmem_dealloc(tmem, kCols);
}

// --------------------------------------------- narrow layers, gradients --
// All gradients of a narrow layer in one pass over dy, z and x: a persistent CTA
// per SM, tiles of 128 rows.  One thread keeps raw rows coming (contiguous bulk
// copies, in pieces of 16 or 32 KB: a whole tile at a time, its way in was 44 %
// of the time), eight warps make dz and x into operands (and add up dz's columns), one
// thread issues the MMAs, eight warps finish dx.  dz's tile, 128 rows of 128
// bytes a panel, is an MN-major left operand of dW = dz^T x (its rows are the
// contraction) and, the same bytes, a K-major one of dx = dz W (its rows are
// rows).  dW stays in the CTA; k_linear_join adds up the CTAs' sums in their
// order.
//
// In 32 bits the planes of dz are two groups of one left operand [hi; mid] of
// dW, those of x three of the right one, so that one MMA makes six products
// (mid lo among them, in columns that are not read); lo hi is a second one, into
// the columns of hi lo.  They are drained every tile (128 of K) into registers:
// the rows of hi, and those of mid, are parts of their own.  dx as in the
// forward kernel.  There is room for one tile's operands and its raw rows: x's
// are made while the MMAs of dx run, which do not need them.
constexpr int kBackThreads = 576;   // warps: MMAs, eight of operands, eight of the epilogue, copies
template <typename T>
constexpr int kBackSide = sizeof(T) == 4 ? 64 : 128;   // inputs and outputs of a layer

struct Narrow {
    const void *grad_y, *pre, *x, *weight;
    int64_t rows, tiles;
    int k, n;              // inputs, outputs
    bool raw;              // the tensors begin on 16 bytes: raw tiles by bulk copies
    bool vec_n, vec_k;     // ... and rows of n (k) elements are whole 16-byte vectors
    bool vec_w;            // rows of the weight are whole chunks of eight, on 16 bytes
    bool want_x, want_w;
    float* parts;          // [parts of all CTAs][n][k], `part` floats each
    int64_t part;
    float* sums;           // [CTA][n]; may be NULL
    Product out;           // of dx
};
template <typename T, int kPanels>
struct BackSmem {
    static constexpr int planes = sizeof(T) == 4 ? 3 : 1;
    static constexpr int side = kPanels * kPanel;
    static constexpr int panel = kBlock * kPanel * 2;          // of one plane
    static constexpr int operand = planes * kPanels * panel;   // [panel][plane]
    static constexpr int unit = 2 * operand;                   // dz, x
    static constexpr int units = planes == 1 && kPanels == 1 ? 2 : 1;
    static constexpr int weight_panel = side * kPanel * 2;
    static constexpr int weight = units * unit;                // [panel of inputs][plane]
    // a warp's exchange is 32 x 32 words; in 32 bits, for want of room, 32 x 8
    static constexpr int exchange = weight + planes * kPanels * weight_panel;
    static constexpr int exchange_bytes = planes == 3 ? 8 * 1024 : 8 * 4096;
    static constexpr int raw = exchange + exchange_bytes;
    // pieces of x's rows, or of dy's and z's: whole tiles of x in 32 bits
    static constexpr int piece = planes == 3 ? 32 * 1024 : 16 * 1024;
    static constexpr int pieces = 96 * 1024 / piece;
    static constexpr int rows_x = piece / (side * (int)sizeof(T));
    static constexpr int bars = raw + pieces * piece;
    static constexpr int bytes = bars + 256 + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory of a narrow layer's gradients");
};

// V columns (eight or sixteen bytes of bfloat16 in a plane).
template <int kPlanes, int V>
__device__ __forceinline__ void put_columns(unsigned char* at, uint32_t plane_bytes,
                                            const float (&v)[V]) {
    uint32_t w[V / 2][3];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
        if (kPlanes == 3)
            split3(v[2 * e], v[2 * e + 1], w[e]);
        else
            w[e][0] = pair_bf16(v[2 * e], v[2 * e + 1]);
    }
#pragma unroll
    for (int p = 0; p < kPlanes; ++p) {
        if constexpr (V == 8)
            *reinterpret_cast<uint4*>(at + p * plane_bytes) =
                make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
        else
            *reinterpret_cast<uint2*>(at + p * plane_bytes) = make_uint2(w[0][p], w[1][p]);
    }
}

// 16 bytes of shared memory, said to be that: a pointer that may also be global costs a generic
// load, whose latency is several times a shared one's.
template <typename T>
__device__ __forceinline__ typename Pack<T, VecOf<T>::n>::Raw lds16(uint32_t at) {
    typename Pack<T, VecOf<T>::n>::Raw r;
    if constexpr (sizeof(T) == 4)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(at));
    else
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at));
    return r;
}

// kRows rows of an operand, [rows, cols] at `src` (times the activation's slope at `pre`, its
// columns added to `sum`, where kDz), by a thread that has 16 bytes' columns of every kStep-th row:
// rows behind the last, and columns up to the next 16, are zeros.  `shared`: src is a raw piece in
// shared memory, `vec`: whose rows are whole 16-byte vectors.
template <typename T, int kAct, int kPanels, bool kDz, int kRows>
__device__ __forceinline__ void make_operand(unsigned char* operand, const T* src, const T* pre,
                                             int rows, int cols, bool shared, bool vec, int mine,
                                             float (&sum)[kPanels][VecOf<T>::n]) {
    using L = BackSmem<T, kPanels>;
    constexpr int V = VecOf<T>::n, kLanes = kPanel / V, kStep = 256 / kLanes;
    constexpr int kBatch = kRows / kStep < 4 ? kRows / kStep : 4;
    const int c = mine % kLanes * V, r0 = mine / kLanes, cols16 = (cols + 15) / 16 * 16;
#pragma unroll
    for (int h = 0; h < kPanels; ++h) {
        const int col = h * kPanel + c;
        if (col >= cols16) break;
        unsigned char* dst = operand + h * L::planes * L::panel + r0 * 128 +
                             (((c >> 3) ^ (r0 & 7)) << 4) + (c & 7) * 2;
        if (vec) {
            const uint32_t s = smem_u32(src + r0 * cols + col);
            const uint32_t z = smem_u32(pre + r0 * cols + col);
            const uint32_t pitch = (uint32_t)(kStep * cols) * (uint32_t)sizeof(T);
#pragma unroll
            for (int i0 = 0; i0 < kRows / kStep; i0 += kBatch) {
                typename Pack<T, V>::Raw a[kBatch], b[kBatch];   // (all loads, then all stores)
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {   // (what lies behind the last row is shared too)
                    a[i] = lds16<T>(s + (i0 + i) * pitch);
                    if (kAct != kActNone) b[i] = lds16<T>(z + (i0 + i) * pitch);
                }
                float v[kBatch][V], w[kBatch][V];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    Pack<T, V>::open(a[i], v[i]);
                    if (kAct != kActNone) Pack<T, V>::open(b[i], w[i]);
                    to_dz<kAct>(v[i], w[i]);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const bool in = r0 + (i0 + i) * kStep < rows && col < cols;
#pragma unroll
                    for (int e = 0; e < V; ++e) v[i][e] = in ? v[i][e] : 0.0f;
                    if (kDz)
#pragma unroll
                        for (int e = 0; e < V; ++e) sum[h][e] += v[i][e];
                    put_columns<L::planes>(dst + (i0 + i) * kStep * 128, L::panel, v[i]);
                }
            }
        } else if (shared) {
            const uint32_t s = smem_u32(src + r0 * cols + col), z = smem_u32(pre + r0 * cols + col);
            const uint32_t pitch = (uint32_t)(kStep * cols) * (uint32_t)sizeof(T);
#pragma unroll
            for (int i = 0; i < kRows / kStep; ++i) {   // (what lies behind the last is shared too)
                Window<T, V> a, b;
                a.load_shared(s + i * pitch);
                if (kAct != kActNone) b.load_shared(z + i * pitch);
                float v[V], w[V];
                a.open(v);
                if (kAct != kActNone) b.open(w);
                to_dz<kAct>(v, w);
                const bool row = r0 + i * kStep < rows;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    v[e] = row && col + e < cols ? v[e] : 0.0f;
                    if (kDz) sum[h][e] += v[e];
                }
                put_columns<L::planes>(dst + i * kStep * 128, L::panel, v);
            }
        } else {
#pragma unroll 1
            for (int r = r0; r < kRows; r += kStep) {
                float v[V], w[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float one[1] = {0.0f}, z[1] = {0.0f};
                    if (r < rows && col + e < cols) {
                        Pack<T, 1>::load(src + (int64_t)r * cols + col + e, one);
                        if (kAct != kActNone) Pack<T, 1>::load(pre + (int64_t)r * cols + col + e, z);
                    }
                    v[e] = one[0];
                    w[e] = z[0];
                }
                to_dz<kAct>(v, w);
                if (kDz)
#pragma unroll
                    for (int e = 0; e < V; ++e) sum[h][e] += v[e];
                put_columns<L::planes>(dst + (r - r0) * 128, L::panel, v);
            }
        }
    }
}

// kVec: rows of dy, z, x and dx are whole vectors, in raw pieces.
template <typename T, int kAct, int kPanels, bool kVec>
__global__ void __launch_bounds__(kBackThreads, 1)
k_linear_narrow(const __grid_constant__ Narrow q, LearnState* st) {
    using L = BackSmem<T, kPanels>;
    constexpr int kPlanes = L::planes, V = VecOf<T>::n;
    constexpr bool kSplit = kPlanes == 3;
    constexpr int kRowsX = L::rows_x, kRowsZ = kAct == kActNone ? L::rows_x : L::rows_x / 2;
    constexpr uint32_t kDw = kSplit ? 192 : 256;   // columns: dx below, dW from here
    extern __shared__ unsigned char raw_smem[];
    unsigned char* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + L::bars);
    uint64_t* raw_empty = raw_full + L::pieces;
    uint64_t* unit_full = raw_empty + L::pieces;
    uint64_t* dz_empty = unit_full + 2;
    uint64_t* x_empty = dz_empty + 2;
    uint64_t* dx_full = x_empty + 2;
    uint64_t* dx_empty = dx_full + 2;
    uint64_t* dw_full = dx_empty + 2;
    uint64_t* dw_empty = dw_full + 1;
    uint64_t* drain = dw_empty + 1;
    uint32_t* s_taddr = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* s_fail = s_taddr + 1;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (known to be the same in a warp)
    if (tid == 0) {
        for (int s = 0; s < L::pieces; ++s) {
            mbar_init(raw_full + s);
            mbar_init_n(raw_empty + s, 8);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init_n(unit_full + s, 8);
            mbar_init(dz_empty + s);
            mbar_init(x_empty + s);
            mbar_init(dx_full + s);
            mbar_init_n(dx_empty + s, 8);
        }
        mbar_init(dw_full);
        mbar_init_n(dw_empty, 8);
        mbar_init(drain);
        *s_fail = 0u;
    }
    if (warp == 0) tmem_alloc(s_taddr, 512);
    pdl_next();
    pdl_begin();
    if (q.want_x) {   // W, rows of outputs: an MN-major operand; zeros in the rows up to the next 16
        const int rows = (q.n + 15) / 16 * 16, chunks = (q.k + 7) / 8;
        for (int t = tid; t < rows * chunks; t += kBackThreads) {
            const int r = t / chunks, c = t % chunks, n = q.k - c * 8;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            if (r < q.n)
                load8(static_cast<const T*>(q.weight) + r * q.k + c * 8, n, q.vec_w && n >= 8, v);
            put_chunk<kPlanes>(smem + L::weight + (c >> 3) * kPlanes * L::weight_panel + r * 128 +
                                   (((c & 7) ^ (r & 7)) << 4),
                               L::weight_panel, v);
        }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_taddr;
    const int first = blockIdx.x, step = gridDim.x;
    if (warp == 17) {
        if (q.raw && elect_one()) {   // ---- raw pieces, in the order in which they are used
            int f = 0;
            bool ok = true;
            // `rows` rows of one tensor or two from row r on
            const auto piece = [&](const void* p, const void* p2, int64_t r, int rows, int cols) {
                const int s = f % L::pieces;
                ok = mbar_wait(raw_empty + s, ((f / L::pieces) & 1) ^ 1) && !*s_fail;
                if (!ok) return;
                ++f;
                const int64_t left = q.rows - r;
                if (left < rows) rows = left > 0 ? (int)left : 0;
                const uint32_t bytes = (uint32_t)rows * cols * (uint32_t)sizeof(T);
                const uint32_t bulk = bytes & ~15u;   // (the last rows need not end on 16 bytes)
                T* dst = reinterpret_cast<T*>(smem + L::raw + s * L::piece);
                T* dst2 = dst + L::piece / 2 / (int)sizeof(T);
                const T* src = static_cast<const T*>(p) + r * cols;
                const T* src2 = static_cast<const T*>(p2) + r * cols;
                for (uint32_t e = bulk / sizeof(T); e < bytes / sizeof(T); ++e) {
                    dst[e] = src[e];
                    if (p2) dst2[e] = src2[e];
                }
                expect_bytes(raw_full + s, p2 ? 2 * bulk : bulk);
                if (bulk) {
                    bulk_copy(dst, src, bulk, raw_full + s);
                    if (p2) bulk_copy(dst2, src2, bulk, raw_full + s);
                }
            };
            for (int64_t t = first; t < q.tiles && ok; t += step) {
                const int64_t r = t * kBlock;
                if (q.want_w)
                    for (int i = 0; i < kBlock && ok; i += kRowsX)
                        piece(q.x, nullptr, r + i, kRowsX, q.k);
                for (int i = 0; i < kBlock && ok; i += kRowsZ)
                    piece(q.grad_y, kAct != kActNone ? q.pre : nullptr, r + i, kRowsZ, q.n);
            }
            if (!ok) {   // give the copies in flight one more bounded wait
                *s_fail = 1u;
                for (int k = f > L::pieces ? f - L::pieces : 0; k < f; ++k)
                    mbar_wait(raw_full + k % L::pieces, (k / L::pieces) & 1);
            }
        }
    } else if (warp == 0) {
        if (elect_one()) {   // ---- MMAs
            constexpr uint32_t kBase = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                       ((uint32_t)(kBlock >> 4) << 24);   // B MN-major
            constexpr uint32_t kAMn = 1u << 15;
            const uint32_t base = smem_u32(smem);
            const uint32_t k16 = (uint32_t)(q.k + 15) / 16 * 16;
            const int steps_n = (q.n + 15) / 16;
            int u = 0;
            bool ok = true;
            for (int64_t t = first; t < q.tiles; t += step, ++u) {
                const int s = u % L::units;
                ok = mbar_wait(unit_full + s, (u / L::units) & 1) && !*s_fail;
                if (!ok) break;
                const uint32_t dz = base + s * L::unit, x = dz + L::operand;
                if (q.want_w) {
                    if (kSplit) {
                        ok = mbar_wait(dw_empty, (u & 1) ^ 1) && !*s_fail;
                        if (!ok) break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + kDw;
                    const uint64_t a = desc_sw128(dz, L::panel), b = desc_sw128(x, L::panel);
                    const uint64_t lo = desc_sw128(dz + 2 * L::panel, L::panel);
                    for (int e = 0; e < kBlock / 16; ++e) {
                        const uint32_t off = 2048u * e >> 4;
                        if constexpr (kSplit) {
                            mma_f16(d, a + off, b + off, kBase | kAMn | (192u >> 3 << 17), e > 0);
                            mma_f16(d + 128, lo + off, b + off, kBase | kAMn | (64u >> 3 << 17), 1);
                        } else {
                            mma_f16(d, a + off, b + off, kBase | kAMn | (k16 >> 3 << 17),
                                    u > 0 || e > 0);
                        }
                    }
                    if (kSplit || t + step >= q.tiles) mma_commit(dw_full);
                }
                mma_commit(x_empty + s);
                if (q.want_x) {
                    // (one accumulator in 32 bits, two in 16)
                    const int buf = kSplit ? 0 : u & 1, turn = kSplit ? u : u >> 1;
                    ok = mbar_wait(dx_empty + buf, (turn & 1) ^ 1) && !*s_fail;
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * 128;
                    const uint64_t b = desc_sw128(base + L::weight, L::weight_panel);
                    for (int e = 0; e < steps_n; ++e) {
                        const uint32_t at = dz + (e >> 2) * kPlanes * L::panel + (e & 3) * 32;
                        const uint64_t be = b + (2048u * e >> 4);
                        if constexpr (kSplit) {
                            mma_f16(d, desc_sw128(at, 16), be, kBase | (192u >> 3 << 17), e > 0);
                            mma_f16(d + 64, desc_sw128(at + L::panel, 16), be,
                                    kBase | (128u >> 3 << 17), 1);
                            mma_f16(d + 128, desc_sw128(at + 2 * L::panel, 16), be,
                                    kBase | (64u >> 3 << 17), 1);
                        } else {
                            mma_f16(d, desc_sw128(at, 16), be, kBase | (k16 >> 3 << 17), e > 0);
                        }
                    }
                    mma_commit(dx_full + buf);
                }
                mma_commit(dz_empty + s);
            }
            if (!ok) {
                *s_fail = 1u;
                mma_commit(drain);
                mbar_wait(drain, 0);
            }
        }
    } else if (warp < 9) {   // ---- operands
        const int mine = tid - 32;
        float sum[kPanels][V], none[kPanels][V];
#pragma unroll
        for (int h = 0; h < kPanels; ++h)
#pragma unroll
            for (int e = 0; e < V; ++e) sum[h][e] = none[h][e] = 0.0f;
        int u = 0, f = 0;
        bool ok = true;
        // the piece in turn, or the place of row r in the tensor
        const auto wait_piece = [&]() {
            if (kVec || q.raw)
                ok = warp_all(mbar_wait(raw_full + f % L::pieces, (f / L::pieces) & 1) && !*s_fail);
            return ok;
        };
        const auto done_piece = [&]() {
            __syncwarp();
            if ((kVec || q.raw) && lane == 0) mbar_arrive(raw_empty + f % L::pieces);
            ++f;
        };
        for (int64_t t = first; t < q.tiles; t += step, ++u) {
            const int s = u % L::units, turn = u / L::units;
            const int64_t row0 = t * kBlock, left = q.rows - row0;
            const int rows = (int)(left < kBlock ? left : kBlock);
            unsigned char* unit = smem + s * L::unit;
            if (q.want_w) {
                ok = warp_all(mbar_wait(x_empty + s, (turn & 1) ^ 1) && !*s_fail);
#pragma unroll 1
                for (int i = 0; i < kBlock && ok; i += kRowsX) {
                    if (!wait_piece()) break;
                    const T* raw =
                        reinterpret_cast<const T*>(smem + L::raw + f % L::pieces * L::piece);
                    unsigned char* to = unit + L::operand + i * 128;
                    if (kVec || q.vec_k)
                        make_operand<T, kActNone, kPanels, false, kRowsX>(to, raw, nullptr, rows - i,
                                                                          q.k, true, true, mine,
                                                                          none);
                    else
                        make_operand<T, kActNone, kPanels, false, kRowsX>(
                            to, q.raw ? raw : static_cast<const T*>(q.x) + (row0 + i) * q.k, nullptr,
                            rows - i, q.k, q.raw, false, mine, none);
                    done_piece();
                }
            }
            if (ok) ok = warp_all(mbar_wait(dz_empty + s, (turn & 1) ^ 1) && !*s_fail);
#pragma unroll 1
            for (int i = 0; i < kBlock && ok; i += kRowsZ) {
                if (!wait_piece()) break;
                const T* raw = reinterpret_cast<const T*>(smem + L::raw + f % L::pieces * L::piece);
                const T* z = raw + L::piece / 2 / (int)sizeof(T);
                unsigned char* to = unit + i * 128;
                if (kVec || q.vec_n) {
                    make_operand<T, kAct, kPanels, true, kRowsZ>(to, raw, z, rows - i, q.n, true,
                                                                 true, mine, sum);
                } else {
                    const int64_t at = (row0 + i) * q.n;
                    make_operand<T, kAct, kPanels, true, kRowsZ>(
                        to, q.raw ? raw : static_cast<const T*>(q.grad_y) + at,
                        q.raw ? z : static_cast<const T*>(q.pre) + at, rows - i, q.n, q.raw,
                        false, mine, sum);
                }
                done_piece();
            }
            if (!ok) break;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(unit_full + s);
        }
        if (!ok) *s_fail = 1u;
        if (q.sums) {   // the rows of threads: in a warp, then between the warps
            constexpr int kLanes = kPanel / V;
#pragma unroll
            for (int h = 0; h < kPanels; ++h)
#pragma unroll
                for (int e = 0; e < V; ++e)
#pragma unroll
                    for (int d = kLanes; d < 32; d *= 2)
                        sum[h][e] += __shfl_xor_sync(0xffffffffu, sum[h][e], d);
            // (every raw piece has been read by all of these warps)
            float* all = reinterpret_cast<float*>(smem + L::raw);
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (lane < kLanes)
#pragma unroll
                for (int h = 0; h < kPanels; ++h)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        all[(warp - 1) * L::side + h * kPanel + lane * V + e] = sum[h][e];
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (mine < q.n) {
                float v[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) v[w] = all[w * L::side + mine];
                q.sums[(int64_t)blockIdx.x * q.n + mine] =
                    ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            }
        }
    } else {   // ---- epilogue
        const int e0 = warp - 9, quarter = warp & 3, group = e0 >> 2;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        float dw[kSplit ? 32 : 1];
#pragma unroll
        for (int e = 0; e < (kSplit ? 32 : 1); ++e) dw[e] = 0.0f;
        float4* x = reinterpret_cast<float4*>(smem + L::exchange) + e0 * (kSplit ? 64 : 256);
        // 32 columns of dx, a row in each lane
        auto store_dx = [&](const float (&v)[32], int64_t t, int c0) {
            const int64_t r0 = t * kBlock + quarter * 32;
            if constexpr (kSplit) {
                finish_small<T, kActNone, true, kVec>(q.out, x, v, r0, c0, 0, lane);
            } else {
                Share<T, kVec, false> share;
                const float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                share.begin(q.out, r0, c0, 0, lane);
                share.template end<kActNone>(q.out, x, v, bias, r0, c0, 0, lane);
            }
        };
        bool ok = true;
        int u = 0;
        for (int64_t t = first; t < q.tiles; t += step, ++u) {
            if (q.want_x) {
                const int buf = kSplit ? 0 : u & 1, turn = kSplit ? u : u >> 1;
                ok = warp_all(mbar_wait(dx_full + buf, turn & 1) && !*s_fail);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = group * 32; c < (kSplit ? 64 : q.k); c += 64) {
                    float v[32];
#pragma unroll
                    for (int p = 0; p < kPlanes; ++p) {
                        uint32_t w[32];
                        __syncwarp();
                        tmem_ld32(tmem + buf * 128 + lanes + p * 64 + c, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[e] = p ? v[e] + __uint_as_float(w[e]) : __uint_as_float(w[e]);
                    }
                    if (c + 64 >= (kSplit ? 64 : q.k)) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(dx_empty + buf);
                    }
                    store_dx(v, t, c);
                }
                if (!kSplit && group * 32 >= q.k && lane == 0) mbar_arrive(dx_empty + buf);
            }
            if (kSplit && q.want_w) {
                ok = warp_all(mbar_wait(dw_full, u & 1) && !*s_fail);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    if (p == 2 && quarter >= 2) continue;   // lo mid, or what lies behind lo
                    uint32_t w[32];
                    __syncwarp();
                    tmem_ld32(tmem + kDw + lanes + p * 64 + group * 32, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) dw[kSplit ? e : 0] += __uint_as_float(w[e]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dw_empty);
            }
        }
        if (ok && q.want_w) {
            // a lane has a row of its part
            const int row = kSplit ? (quarter & 1) * 32 + lane : quarter * 32 + lane;
            float* part = q.parts + ((int64_t)blockIdx.x * (kSplit ? 2 : 1) +
                                     (kSplit ? quarter >> 1 : 0)) * q.part +
                          (int64_t)row * q.k;
            if constexpr (kSplit) {
                if (row < q.n)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (group * 32 + e < q.k) part[group * 32 + e] = dw[e];
            } else {
                ok = warp_all(mbar_wait(dw_full, 0) && !*s_fail);
                tc_fence_after();
#pragma unroll 1
                for (int c = group * 32; ok && c < q.k; c += 64) {
                    uint32_t w[32];
                    __syncwarp();
                    tmem_ld32(tmem + kDw + lanes + c, w);
                    tmem_wait_ld();
                    if (row < q.n)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c + e < q.k) part[c + e] = __uint_as_float(w[e]);
                }
            }
        }
        if (!ok) *s_fail = 1u;
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *s_fail) atomicOr(&st->error, kErrTimeout);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ plans --
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;

// An operand as the products read it: a bfloat16 matrix [planes][rows][pitch].
struct Matrix {
    const __nv_bfloat16* at;
    int64_t rows, cols, pitch;
    size_t plane;
    int planes;
};

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

int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }
size_t plane_size(int64_t rows, int64_t cols) { return (size_t)rows * round8(cols); }

// The sums' workspace of a product in parts: as many as fill the SMs once, of kLeast panels.
constexpr int kMostSms = 160;
constexpr int kLeast = 4;
int splits_of(int64_t tiles, int64_t panels, int n_sms) {
    const int64_t fit = n_sms / tiles, most = panels / kLeast;
    const int64_t s = fit < most ? fit : most;
    return s > 1 ? (int)s : 1;
}
// Columns of a tile: an MMA of N = 256 takes little longer than one of 128.
int tile_n(int planes, int64_t n) { return planes == 3 || n <= 128 ? 128 : 256; }
// Pairs of CTAs where tiles of 256 rows are not half empty.
bool paired(int64_t m) { return m > kBlock; }
int64_t part_size(int64_t m, int64_t n) { return (m * n + 3) / 4 * 4; }
size_t part_floats(int planes, int64_t m, int64_t n, int64_t k) {
    const int kn = tile_n(planes, n), ctas = (planes == 3 || kn == 256) && paired(m) ? 2 : 1;
    const int64_t tiles = ceil_div(m, kBlock * ctas) * ceil_div(n, kn);
    if (tiles == 0 || tiles > kMostSms / ctas) return 0;
    const int s = splits_of(tiles, ceil_div(k, kPanel), kMostSms / ctas);
    return s > 1 ? (size_t)s * part_size(m, n) : 0;
}

// Blocks of rows of k_linear_operand: about eight blocks per SM over the whole matrix.
struct OperandGrid {
    int tx;
    int64_t block_rows, blocks, col_blocks;
};
OperandGrid operand_grid(int64_t rows, int64_t cols) {
    OperandGrid g;
    const int64_t groups = ceil_div(cols, 8);
    g.tx = 1;
    while (g.tx < 32 && g.tx < groups) g.tx *= 2;
    g.col_blocks = ceil_div(groups, g.tx);
    const int64_t least = 256 / g.tx;   // a row per thread
    int64_t want = kMostSms * 8 / g.col_blocks;
    if (want < 1) want = 1;
    g.block_rows = ceil_div(ceil_div(rows, want), least) * least;
    if (g.block_rows < least) g.block_rows = least;
    g.blocks = ceil_div(rows, g.block_rows);
    return g;
}

struct Space {
    __nv_bfloat16 *x, *w, *dz;
    float *sums, *parts;
    size_t bytes;
};
Space carve(void* ws, int64_t m, int64_t k, int64_t n, int dtype) {
    const int planes = dtype == kF32 ? kMaxPlanes : 1;
    Carve c{static_cast<unsigned char*>(ws)};
    Space s;
    s.x = c.take<__nv_bfloat16>(planes * plane_size(m, k));
    s.w = c.take<__nv_bfloat16>(planes * plane_size(n, k));
    s.dz = c.take<__nv_bfloat16>(planes * plane_size(m, n));
    const int64_t blocks = operand_grid(m, n).blocks;
    s.sums = c.take<float>((size_t)(blocks > kMostSms ? blocks : kMostSms) * n);
    size_t parts = part_floats(planes, m, n, k);
    const size_t dx = part_floats(planes, m, k, n), dw = part_floats(planes, n, k, m);
    if (dx > parts) parts = dx;
    if (dw > parts) parts = dw;
    const int64_t side = dtype == kF32 ? kBackSide<float> : kBackSide<__nv_bfloat16>;
    if (k <= side && n <= side) {   // two parts of every CTA
        const size_t tiles = (size_t)ceil_div(m, kBlock);
        const size_t narrow = 2 * (tiles < kMostSms ? tiles : kMostSms) * (size_t)part_size(n, k);
        if (narrow > parts) parts = narrow;
    }
    s.parts = c.take<float>(parts);
    s.bytes = c.used;
    return s;
}

// A call's operands: those that have to be made are made by one launch.
template <typename T>
struct Maker {
    static constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
    Operands all{};
    int count = 0, act = kActNone;

    // `src` (in the first one times the activation's slope at `pre`) as an operand: its planes in
    // `planes` (NULL: not wanted), where it is not one as it lies, and its column sums
    Matrix add(const void* src, const void* pre, int slope, int64_t rows, int64_t cols,
               __nv_bfloat16* planes, float* sums) {
        if (!pre) slope = kActNone;
        const bool as_is =
            kPlanes == 1 && slope == kActNone && cols % 8 == 0 && aligned16(src);
        const int64_t pitch = round8(cols);
        if (!((as_is || !planes) && !sums)) {
            const OperandGrid g = operand_grid(rows, cols);
            if (count == 0) act = slope;
            all.of[count++] = Operand{src, pre, rows, cols, pitch, as_is ? nullptr : planes,
                                      (size_t)rows * pitch, sums, g.tx, g.block_rows,
                                      (unsigned)g.blocks, (unsigned)g.col_blocks,
                                      cols % VecOf<T>::n == 0 && aligned16(src) && aligned16(pre)};
        }
        return as_is ? Matrix{static_cast<const __nv_bfloat16*>(src), rows, cols, cols, 0, 1}
                     : Matrix{planes, rows, cols, pitch, (size_t)rows * pitch, kPlanes};
    }
    cudaError_t launch(cudaStream_t s) const {
        if (count == 0) return cudaSuccess;
        dim3 grid(1, 1, (unsigned)count);
        for (int i = 0; i < count; ++i) {
            if (all.of[i].blocks > grid.x) grid.x = all.of[i].blocks;
            if (all.of[i].col_blocks > grid.y) grid.y = all.of[i].col_blocks;
        }
        return launch_pdl(act == kActSilu   ? k_linear_operands<T, kPlanes, kActSilu>
                          : act == kActRelu ? k_linear_operands<T, kPlanes, kActRelu>
                                            : k_linear_operands<T, kPlanes, kActNone>,
                          grid, dim3(256), 0, s, all);
    }
};

// (16 parts or fewer: a thread per four columns, each part's load behind the one before)
template <typename T>
cudaError_t join(const Product& q, const float* parts, int n_sms, cudaStream_t s) {
    const bool many = q.splits > 16;
    const int64_t blocks = ceil_div(ceil_div(q.m * q.n, 4), many ? 4 : 256);
    return launch_pdl(many ? k_linear_join<T, 64> : k_linear_join<T, 1>,
                      dim3((unsigned)(blocks < n_sms * 8 ? blocks : n_sms * 8)), dim3(256), 0, s, q,
                      parts);
}

template <typename T, int kPlanes, int kN, bool kAMn, bool kBMn, int kCtas>
cudaError_t product_as(Product q, const Matrix& a, const Matrix& b, int64_t k, float* parts,
                       LearnState* st, int n_sms, cudaStream_t s) {
    using L = ProductSmem<kPlanes, kN, kCtas>;
    q.tiles_m = (int)ceil_div(q.m, kBlock * kCtas);
    q.tiles_n = (int)ceil_div(q.n, kN);
    q.panels = (int)ceil_div(k, kPanel);
    const int64_t tiles = (int64_t)q.tiles_m * q.tiles_n;
    const int groups = n_sms / kCtas;   // of CTAs that share a tile
    q.splits = tiles <= groups ? splits_of(tiles, q.panels, groups) : 1;
    q.part = part_size(q.m, q.n);
    if (!encode(&q.a, a, kAMn ? kPanel : kBlock) || !encode(&q.b, b, kBMn ? kPanel : L::rows_b))
        return cudaErrorInvalidValue;
    const auto launch = [&](auto kernel, const Product& p) {
        const int64_t total = tiles * p.splits;
        return launch_pdl(kernel, dim3((unsigned)((total < groups ? total : groups) * kCtas)),
                          dim3(L::threads), L::bytes, s, p, st);
    };
    if (q.splits == 1)
        return launch(q.vec ? k_linear_product<T, kPlanes, kN, kAMn, kBMn, kCtas, true>
                            : k_linear_product<T, kPlanes, kN, kAMn, kBMn, kCtas, false>, q);
    Product p = q;
    p.bias = nullptr;
    p.residual = p.pre = nullptr;
    p.out = parts;
    p.act = kActNone;
    p.vec = q.n % 4 == 0;
    cudaError_t e =
        launch(p.vec ? k_linear_product<float, kPlanes, kN, kAMn, kBMn, kCtas, true>
                     : k_linear_product<float, kPlanes, kN, kAMn, kBMn, kCtas, false>, p);
    if (e != cudaSuccess) return e;
    return join<T>(q, parts, n_sms, s);
}

template <typename T, bool kAMn, bool kBMn>
cudaError_t product(const Product& q, const Matrix& a, const Matrix& b, int64_t k, float* parts,
                    LearnState* st, int n_sms, cudaStream_t s) {
    if constexpr (sizeof(T) == 4)
        return paired(q.m) ? product_as<T, 3, 128, kAMn, kBMn, 2>(q, a, b, k, parts, st, n_sms, s)
                           : product_as<T, 3, 128, kAMn, kBMn, 1>(q, a, b, k, parts, st, n_sms, s);
    else if (tile_n(1, q.n) == 128)
        return product_as<T, 1, 128, kAMn, kBMn, 1>(q, a, b, k, parts, st, n_sms, s);
    else if (paired(q.m))
        return product_as<T, 1, 256, kAMn, kBMn, 2>(q, a, b, k, parts, st, n_sms, s);
    else
        return product_as<T, 1, 256, kAMn, kBMn, 1>(q, a, b, k, parts, st, n_sms, s);
}

bool aligned_to4(const void* p, int size) {
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(4 * size - 1)) == 0;
}
template <typename T>
bool vec4(const Product& q) {
    return q.n % 4 == 0 && aligned_to4(q.out, sizeof(T)) && aligned_to4(q.pre, sizeof(T)) &&
           aligned_to4(q.residual, sizeof(T));
}

template <typename T, int V>
cudaError_t few_rows(const LinearCall& c, const Product& q, cudaStream_t s) {
    int per = 1;
    while (per < 8 && (int64_t)per * 32 * V * 8 < c.inputs) per *= 2;
    const dim3 grid((unsigned)ceil_div(c.outputs, 8 / per)), block(256);
    auto* kernel = c.rows == 1   ? k_linear_rows<T, V, 1>
                   : c.rows == 2 ? k_linear_rows<T, V, 2>
                   : c.rows == 3 ? k_linear_rows<T, V, 3>
                   : c.rows == 4 ? k_linear_rows<T, V, 4>
                   : c.rows == 5 ? k_linear_rows<T, V, 5>
                   : c.rows == 6 ? k_linear_rows<T, V, 6>
                   : c.rows == 7 ? k_linear_rows<T, V, 7>
                                 : k_linear_rows<T, V, 8>;
    return launch_pdl(kernel, grid, block, 0, s, static_cast<const T*>(c.x),
                      static_cast<const T*>(c.weight), c.inputs, per, q);
}

// The plan of a narrow layer; false where it is none.
template <typename T>
bool stream_plan(const LinearCall& c, int n_sms, Stream* q, int* smem) {
    constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
    if (c.inputs > kStreamMaxK || c.outputs > 4 * kStreamN<T> || !aligned16(c.x)) return false;
    q->x = c.x;
    q->weight = c.weight;
    q->tiles = ceil_div(c.rows, kBlock);
    q->k = (int)c.inputs;
    q->panels = (int)ceil_div(c.inputs, kPanel);
    q->blocks = (int)ceil_div(c.outputs, kStreamN<T>);
    q->np = q->blocks > 1 ? kStreamN<T> : (int)ceil_div(c.outputs, 16) * 16;
    q->vec = c.inputs % VecOf<T>::n == 0 && aligned16(c.weight);
    // as many operands, then raw tiles in flight as fit
    const auto fits = [&](int raws, int units) {
        *smem = stream_smem(kPlanes, sizeof(T), q->k, q->panels, q->np, raws, units).bytes;
        return *smem <= kStreamSmemMax;
    };
    for (int units = 2; units >= 1; --units)
        for (int raws = 4; raws >= units; --raws)
            if (fits(raws, units)) {
                q->raws = raws;
                q->units = units;
                return true;
            }
    return false;
}

template <typename T>
cudaError_t forward(const LinearCall& c, LearnState* st, void* ws, int n_sms, cudaStream_t s) {
    const int64_t m = c.rows, k = c.inputs, n = c.outputs;
    if (m == 0) return cudaSuccess;
    Product q{};
    q.m = m;
    q.n = n;
    q.bias = c.bias;
    q.residual = c.residual;
    q.pre = c.pre;
    q.out = c.out;
    q.act = c.act;
    if (m <= kFewRows) {
        constexpr int V = VecOf<T>::n;
        return k % V == 0 && aligned16(c.x) && aligned16(c.weight) ? few_rows<T, V>(c, q, s)
                                                                   : few_rows<T, 1>(c, q, s);
    }
    q.vec = vec4<T>(q);
    Stream narrow{};
    int smem = 0;
    if (stream_plan<T>(c, n_sms, &narrow, &smem)) {
        narrow.out = q;
        narrow.skip = q.residual && aligned16(q.residual) && narrow.blocks == 1;
        const int64_t per = n_sms / narrow.blocks;
        const int64_t grid = narrow.blocks * (narrow.tiles < per ? narrow.tiles : per);
        auto* kernel = !(narrow.vec && q.vec) ? k_linear_stream<T, false, true>
                       : q.residual           ? k_linear_stream<T, true, true>
                                              : k_linear_stream<T, true, false>;
        return launch_pdl(kernel, dim3((unsigned)grid), dim3(kStreamThreads),
                          (size_t)smem, s, narrow, st);
    }
    const Space sp = carve(ws, m, k, n, c.dtype);
    Maker<T> make;
    const Matrix x = make.add(c.x, nullptr, kActNone, m, k, sp.x, nullptr);
    const Matrix w = make.add(c.weight, nullptr, kActNone, n, k, sp.w, nullptr);
    const cudaError_t e = make.launch(s);
    if (e != cudaSuccess) return e;
    return product<T, false, false>(q, x, w, k, sp.parts, st, n_sms, s);
}

template <typename T>
cudaError_t narrow(const LinearCall& c, const Space& sp, LearnState* st, int n_sms,
                   cudaStream_t s) {
    const int64_t m = c.rows, k = c.inputs, n = c.outputs;
    Narrow q{};
    q.grad_y = c.grad_y;
    q.pre = c.pre;
    q.x = c.x;
    q.weight = c.weight;
    q.rows = m;
    q.tiles = ceil_div(m, kBlock);
    q.k = (int)k;
    q.n = (int)n;
    const bool act = c.act != kActNone;
    q.raw = aligned16(c.grad_y) && (!act || aligned16(c.pre)) && aligned16(c.x);
    q.vec_n = q.raw && n % VecOf<T>::n == 0;
    q.vec_k = q.raw && k % VecOf<T>::n == 0;
    q.vec_w = aligned16(c.weight) && k % 8 == 0;
    q.want_x = c.grad_x != nullptr;
    q.want_w = c.grad_weight != nullptr;
    q.parts = sp.parts;
    q.part = part_size(n, k);
    q.sums = c.grad_bias ? sp.sums : nullptr;
    q.out.m = m;
    q.out.n = k;
    q.out.out = c.grad_x;
    q.out.vec = vec4<T>(q.out);
    const unsigned ctas = (unsigned)(q.tiles < n_sms ? q.tiles : n_sms);
    const auto run = [&](auto panels) {
        constexpr int kPanels = decltype(panels)::value;
        const auto pick = [&](auto vec) {
            constexpr bool kVec = decltype(vec)::value;
            return c.act == kActSilu   ? k_linear_narrow<T, kActSilu, kPanels, kVec>
                   : c.act == kActRelu ? k_linear_narrow<T, kActRelu, kPanels, kVec>
                                       : k_linear_narrow<T, kActNone, kPanels, kVec>;
        };
        auto* kernel = q.vec_n && q.vec_k && q.out.vec ? pick(std::true_type()) : pick(std::false_type());
        return launch_pdl(kernel, dim3(ctas), dim3(kBackThreads), BackSmem<T, kPanels>::bytes, s, q,
                          st);
    };
    cudaError_t e = k <= kPanel && n <= kPanel
                        ? run(std::integral_constant<int, 1>())
                        : run(std::integral_constant<int, kBackSide<T> / kPanel>());
    if (e == cudaSuccess && c.grad_bias)
        e = launch_pdl(k_linear_sums, dim3((unsigned)ceil_div(n, 32)), dim3(32, 32), 0, s,
                       (const float*)sp.sums, (int64_t)ctas, n, c.grad_bias);
    if (e == cudaSuccess && c.grad_weight) {
        Product p{};
        p.m = n;
        p.n = k;
        p.out = c.grad_weight;
        p.splits = (int)ctas * (sizeof(T) == 4 ? 2 : 1);
        p.part = q.part;
        e = join<T>(p, sp.parts, n_sms, s);
    }
    return e;
}

template <typename T>
cudaError_t backward(const LinearCall& c, LearnState* st, void* ws, int n_sms, cudaStream_t s) {
    const int64_t m = c.rows, k = c.inputs, n = c.outputs;
    if (m == 0) {
        cudaError_t e = cudaSuccess;
        if (c.grad_weight) e = cudaMemsetAsync(c.grad_weight, 0, sizeof(T) * n * k, s);
        if (e == cudaSuccess && c.grad_bias) e = cudaMemsetAsync(c.grad_bias, 0, 4 * n, s);
        return e;
    }
    const Space sp = carve(ws, m, k, n, c.dtype);
    if (k <= kBackSide<T> && n <= kBackSide<T>) return narrow<T>(c, sp, st, n_sms, s);
    Maker<T> make;
    const Matrix dz = make.add(c.grad_y, c.act == kActNone ? nullptr : c.pre, c.act, m, n,
                               c.grad_x || c.grad_weight ? sp.dz : nullptr,
                               c.grad_bias ? sp.sums : nullptr);
    const Matrix w = make.add(c.weight, nullptr, kActNone, n, k, c.grad_x ? sp.w : nullptr, nullptr);
    const Matrix x = make.add(c.x, nullptr, kActNone, m, k, c.grad_weight ? sp.x : nullptr, nullptr);
    cudaError_t e = make.launch(s);
    if (e == cudaSuccess && c.grad_bias)
        e = launch_pdl(k_linear_sums, dim3((unsigned)ceil_div(n, 32)), dim3(32, 32), 0, s,
                       (const float*)sp.sums, operand_grid(m, n).blocks, n, c.grad_bias);
    if (e == cudaSuccess && c.grad_x) {
        Product q{};
        q.m = m;
        q.n = k;
        q.out = c.grad_x;
        q.vec = vec4<T>(q);
        e = product<T, false, true>(q, dz, w, n, sp.parts, st, n_sms, s);
    }
    if (e == cudaSuccess && c.grad_weight) {
        Product q{};
        q.m = n;
        q.n = k;
        q.out = c.grad_weight;
        q.vec = vec4<T>(q);
        e = product<T, true, true>(q, dz, x, m, sp.parts, st, n_sms, s);
    }
    return e;
}

template <typename T, int kPlanes, int kN, int kCtas, bool kAMn, bool kBMn>
cudaError_t prepare_one() {
    cudaError_t e = cudaSuccess;
    const auto prepare = [&](auto* f) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     ProductSmem<kPlanes, kN, kCtas>::bytes);
    };
    prepare(k_linear_product<T, kPlanes, kN, kAMn, kBMn, kCtas, true>);
    prepare(k_linear_product<T, kPlanes, kN, kAMn, kBMn, kCtas, false>);
    if constexpr (sizeof(T) == 2) {
        prepare(k_linear_product<float, kPlanes, kN, kAMn, kBMn, kCtas, true>);
        prepare(k_linear_product<float, kPlanes, kN, kAMn, kBMn, kCtas, false>);
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

template <typename T, int kPanels>
cudaError_t prepare_narrow() {
    cudaError_t e = cudaSuccess;
    for (auto* f : {k_linear_narrow<T, kActNone, kPanels, true>,
                    k_linear_narrow<T, kActSilu, kPanels, true>,
                    k_linear_narrow<T, kActRelu, kPanels, true>,
                    k_linear_narrow<T, kActNone, kPanels, false>,
                    k_linear_narrow<T, kActSilu, kPanels, false>,
                    k_linear_narrow<T, kActRelu, kPanels, false>})
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     BackSmem<T, kPanels>::bytes);
    return e;
}

}  // namespace

size_t linear_workspace(int64_t rows, int64_t inputs, int64_t outputs, int dtype) {
    return carve(nullptr, rows, inputs, outputs, dtype).bytes;
}

cudaError_t prepare_linear() {
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
    if (e == cudaSuccess) e = prepare_narrow<float, 1>();
    if (e == cudaSuccess) e = prepare_narrow<__nv_bfloat16, 1>();
    if (e == cudaSuccess) e = prepare_narrow<__nv_bfloat16, 2>();
    for (auto* f : {k_linear_stream<float, true, true>, k_linear_stream<float, true, false>,
                    k_linear_stream<float, false, true>, k_linear_stream<__nv_bfloat16, true, true>,
                    k_linear_stream<__nv_bfloat16, true, false>,
                    k_linear_stream<__nv_bfloat16, false, true>})
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kStreamSmemMax);
    return e;
}

cudaError_t launch_linear_forward(const LinearCall& c, LearnState* st, void* ws, int n_sms,
                                  cudaStream_t stream) {
    return c.dtype == kF32 ? forward<float>(c, st, ws, n_sms, stream)
                           : forward<__nv_bfloat16>(c, st, ws, n_sms, stream);
}
cudaError_t launch_linear_backward(const LinearCall& c, LearnState* st, void* ws, int n_sms,
                                   cudaStream_t stream) {
    return c.dtype == kF32 ? backward<float>(c, st, ws, n_sms, stream)
                           : backward<__nv_bfloat16>(c, st, ws, n_sms, stream);
}

}  // namespace pulsar
