// Orthogonalisation of an update by Newton-Schulz products:
//
//   X_0 = G / (|G|_F + eps),   X' = P X,   P = a I + b A + c A^2,   A = X X^T
//
// for every matrix of a batch, on the orientation with the fewer rows (the
// result of the transpose is the transpose of the result).  r rows, c columns.
//
// The products run on the tensor cores (tcgen05, fp32 accumulation) on
// operands in half precision: 11 significant bits, eight times closer than
// bfloat16 at the same rate, and its narrow range is no limit because the
// iterates are bounded: |X_0|_F <= 1 and the polynomial keeps the singular
// values near 1, so powers of two (kScale*) place X, A and P inside it.  For
// float32 tensors every operand is a pair hi + lo of halves (22 bits) and a
// product is hi hi + hi lo + lo hi.  aI is folded into P, so that the last
// product needs nothing but P and X.  A and P are symmetric: only the 128 x
// 128 tiles on and below the diagonal are computed, each written twice.
//
// Matrices lie in panels of 64 columns, a row of a panel being the 128 bytes
// of one swizzled shared-memory row: any run of rows of a panel is one
// contiguous bulk copy, and the same bytes serve as a K-major operand (rows
// are M or N) and as an MN-major one (rows are K).
#include "learn_internal.cuh"
#include "tensor_core.cuh"

#include <cuda_fp16.h>

namespace pulsar {
namespace {

constexpr int kThreads = 256;
constexpr int kPanel = 64;      // columns of a panel: 128 bytes of halves
constexpr int kBlock = 128;     // rows are padded to it
// stored value = value times this: |X|, |A| < 1.6 and |P| < 4 for the usual
// coefficients, far inside 65504; typical entries (1/sqrt(rc) and above) stay
// above the smallest normal half
constexpr float kScaleX = 1024.0f, kScaleA = 4096.0f, kScaleP = 1024.0f;

// Element (row, col) of a matrix of `rows` padded rows, in halves.
__host__ __device__ __forceinline__ size_t panel_at(int64_t row, int64_t col, int64_t rows) {
    const int64_t chunk = (col & (kPanel - 1)) >> 3;
    return (size_t)(((col / kPanel) * rows + row) * kPanel + ((chunk ^ (row & 7)) << 3) + (col & 7));
}

// ------------------------------------------------------------------ norm --
// Sums of squares, a block per chunk of a matrix.  The second sum is of the
// values times 2^-64, and is taken where the first overflows.
constexpr float kDown = 5.421010862427522e-20f;   // 2^-64
constexpr int kNormBlocks = 128;                  // at most, per matrix

__device__ __forceinline__ float2 block_sum(float2 v) {
    __shared__ float2 s[kThreads / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        t.x += s[w].x;
        t.y += s[w].y;
    }
    __syncthreads();
    return t;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
k_orth_norm(const T* __restrict__ g, int64_t elems, float2* __restrict__ part) {
    pdl_begin();
    const T* m = g + (size_t)blockIdx.y * elems;
    float2 s = make_float2(0.0f, 0.0f);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < elems;
         i += (int64_t)gridDim.x * kThreads) {
        float v[1];
        Pack<T, 1>::load(m + i, v);
        s.x = fmaf(v[0], v[0], s.x);
        s.y = fmaf(v[0] * kDown, v[0] * kDown, s.y);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// 1 / (|G|_F + eps) from a matrix's parts (every thread of the block calls).
__device__ __forceinline__ float inv_norm(const float2* part, int blocks, float eps) {
    float2 s = make_float2(0.0f, 0.0f);
    for (int i = threadIdx.x; i < blocks; i += kThreads) {
        s.x += part[i].x;
        s.y += part[i].y;
    }
    s = block_sum(s);
    const float norm = isinf(s.x) ? sqrtf(s.y) * 18446744073709551616.0f : sqrtf(s.x);
    return 1.0f / (norm + eps);
}

// Eight values as halves, and what their rounding left (kParts 2).
template <int kParts>
__device__ __forceinline__ void halves(const float (&v)[8], uint4 (&h)[kParts]) {
    uint32_t w[kParts][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 p = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        w[0][j] = *reinterpret_cast<const uint32_t*>(&p);
        if (kParts == 2) {
            const float2 f = __half22float2(p);
            const __half2 q = __floats2half2_rn(v[2 * j] - f.x, v[2 * j + 1] - f.y);
            w[kParts - 1][j] = *reinterpret_cast<const uint32_t*>(&q);
        }
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k) h[k] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
}

// X_0 in panels, g [m, n] transposed where it is tall; the padding is zero.
// A thread takes eight columns of a row; consecutive threads lie along what
// is contiguous in g.
template <typename T, int kParts>
__global__ void __launch_bounds__(kThreads)
k_orth_start(const T* __restrict__ g, int64_t r, int64_t c, int64_t rp, int64_t cp, bool tall,
             const float2* __restrict__ part, int parts, float eps, __half* __restrict__ x,
             size_t lo) {
    pdl_begin();
    const float inv = inv_norm(part + (size_t)blockIdx.y * parts, parts, eps);
    const T* m = g + (size_t)blockIdx.y * r * c;
    __half* o = x + (size_t)blockIdx.y * rp * cp;
    const int64_t chunks = cp / 8;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < rp * chunks;
         i += (int64_t)gridDim.x * kThreads) {
        const int64_t row = tall ? i % rp : i / chunks, c0 = (tall ? i / rp : i % chunks) * 8;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float u[1] = {0.0f};
            if (row < r && c0 + j < c)
                Pack<T, 1>::load(m + (tall ? (c0 + j) * r + row : row * c + c0 + j), u);
            v[j] = u[0] * inv * kScaleX;
        }
        uint4 h[kParts];
        halves<kParts>(v, h);
        const size_t at = panel_at(row, c0, rp);
#pragma unroll
        for (int k = 0; k < kParts; ++k) *reinterpret_cast<uint4*>(o + k * lo + at) = h[k];
    }
}

// No step at all: out = g / (|g| + eps).
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_orth_scale(const T* __restrict__ g, int64_t elems, const float2* __restrict__ part, int parts,
             float eps, T* __restrict__ out) {
    pdl_begin();
    const float inv = inv_norm(part + (size_t)blockIdx.y * parts, parts, eps);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < elems;
         i += (int64_t)gridDim.x * kThreads) {
        float v[1];
        Pack<T, 1>::load(g + (size_t)blockIdx.y * elems + i, v);
        v[0] *= inv;
        Pack<T, 1>::store(out + (size_t)blockIdx.y * elems + i, v);
    }
}

// -------------------------------------------------------------- products --
// One kernel for the three products, a persistent CTA per SM.  Roles: one
// thread keeps a ring of operand stages filled with bulk copies, one issues
// the MMAs into one of two accumulators in tensor memory, and four warps
// drain the other: scale, round, and write the tile back in panels through
// shared memory (bulk stores), or in the last step as the result.
struct Product {
    const __half *l, *r;      // left and right operands, hi parts
    size_t l_lo, r_lo;        // halves from a hi part to its lo part
    size_t l_size, r_size;    // halves per matrix of the batch
    int64_t l_rows, r_rows;   // padded rows
    int k_panels;
    int tiles_m, tiles_n;     // of the product (kGram: tiles_m^2 / 2 are computed)
    int tiles;                // per matrix
    int batch;
    // D = alpha (accumulator) + beta C + gamma I, C and D in panels
    const __half* c;
    __half* d;
    size_t d_lo, d_size;      // also C's
    int64_t d_rows;
    float alpha, beta, gamma;
    // the result, where `out` is given: [r, c] or its transpose, unpadded
    void* out;
    int64_t out_r, out_c;
    bool tall;
    int dtype;
};

constexpr int kProductThreads = 192;   // warps: copies, MMAs, four of the epilogue
constexpr int kEpilogue = 128;
constexpr int kStaging = kBlock * kPanel * 2;   // one panel of a tile: 16 KB

template <bool kSplit, int kN>
struct ProductSmem {
    static constexpr int parts = kSplit ? 2 : 1;
    static constexpr int a = kBlock * kPanel * 2, b = kN * kPanel * 2;
    static constexpr int stage = parts * (a + b);
    static constexpr int stages = (227 * 1024 - 1024 - 2 * kStaging - 256) / stage;
    static constexpr int staging = stages * stage;
    static constexpr int bars = staging + 2 * kStaging;
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

__device__ __forceinline__ void expect_bytes(uint64_t* mbar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(mbar)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* mbar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(mbar))
        : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void bulk_store_read() {   // all but kLeft stores have been read
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void epilogue_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(kEpilogue) : "memory");
}
// The same, and whether any thread has `v`: one decision for all.
__device__ __forceinline__ bool epilogue_any(bool v) {
    uint32_t any;
    __syncwarp();
    asm volatile(
        "{\n.reg .pred p, r;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred r, 1, %2, p;\n"
        "selp.u32 %0, 1, 0, r;\n}\n"
        : "=r"(any)
        : "r"((uint32_t)v), "n"(kEpilogue)
        : "memory");
    return any != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* mbar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(mbar)) : "memory");
}

// Tile t of a symmetric product, row blocks i >= j.
__device__ __forceinline__ void lower_tile(int t, int* i, int* j) {
    int row = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while ((row + 1) * (row + 2) / 2 <= t) ++row;
    while (row * (row + 1) / 2 > t) --row;
    *i = row;
    *j = t - row * (row + 1) / 2;
}

template <bool kSplit, int kN, bool kGram>
__global__ void __launch_bounds__(kProductThreads)
k_orth_product(const __grid_constant__ Product q, LearnState* st) {
    using L = ProductSmem<kSplit, kN>;
    constexpr int kParts = L::parts;
    constexpr int kPanels = kN / kPanel;   // of a tile
    static_assert(!kGram || kN == kBlock, "symmetric products have square tiles");
    extern __shared__ unsigned char raw[];
    unsigned char* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bars);
    uint64_t* empty = full + L::stages;
    uint64_t* acc_full = empty + L::stages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* s_taddr = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* s_fail = s_taddr + 1;
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < L::stages; ++s) {
            mbar_init(full + s);
            mbar_init(empty + s);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + s);
            mbar_init(acc_empty + s);
        }
        mbar_init(drain);
        *s_fail = 0u;
        fence_async_smem();
    }
    if (warp == 1) tmem_alloc(s_taddr, 2 * kN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_taddr;
    pdl_begin();
    const int total = q.tiles * q.batch;
    auto place = [&](int t, int* z, int* i, int* j) {
        *z = t / q.tiles;
        t -= *z * q.tiles;
        if (kGram) {
            lower_tile(t, i, j);
        } else {
            *i = t % q.tiles_m;   // neighbours share the columns of X
            *j = t / q.tiles_m;
        }
    };

    if (warp == 0) {
        if (tid == 0) {   // ---- copies
            int n = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                int z, i, j;
                place(t, &z, &i, &j);
                const __half* l = q.l + z * q.l_size + (size_t)i * kBlock * kPanel;
                const __half* r = q.r + z * q.r_size +
                                  (kGram ? (size_t)j * kN * kPanel
                                         : (size_t)j * kPanels * q.r_rows * kPanel);
                for (int k = 0; k < q.k_panels; ++k, ++n) {
                    const int s = n % L::stages;
                    ok = mbar_wait(empty + s, ((n / L::stages) & 1) ^ 1) && !*s_fail;
                    if (!ok) break;
                    unsigned char* dst = smem + s * L::stage;
                    expect_bytes(full + s, L::stage);
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
                        bulk_copy(dst + p * L::a, l + p * q.l_lo + (size_t)k * q.l_rows * kPanel,
                                  L::a, full + s);
                    dst += kParts * L::a;
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        const __half* b = r + p * q.r_lo;
                        if (kGram) {
                            bulk_copy(dst + p * L::b, b + (size_t)k * q.r_rows * kPanel, L::b,
                                      full + s);
                        } else {   // 64 rows of each of the tile's panels
#pragma unroll
                            for (int c = 0; c < kPanels; ++c)
                                bulk_copy(dst + p * L::b + c * kPanel * kPanel * 2,
                                          b + ((size_t)c * q.r_rows + (size_t)k * kPanel) * kPanel,
                                          kPanel * kPanel * 2, full + s);
                        }
                    }
                }
            }
            if (!ok) {   // give the copies in flight one more bounded wait
                *s_fail = 1u;
                for (int k = n > L::stages ? n - L::stages : 0; k < n; ++k)
                    mbar_wait(full + k % L::stages, (k / L::stages) & 1);
            }
        }
    } else if (warp == 1) {
        if (tid == 32) {   // ---- MMAs
            constexpr uint32_t idesc = (1u << 4) | (kGram ? 0u : 1u << 16) |
                                       ((uint32_t)(kN >> 3) << 17) |
                                       ((uint32_t)(kBlock >> 4) << 24);
            const uint32_t base = smem_u32(smem);
            int n = 0, it = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x, ++it) {
                const int buf = it & 1;
                const uint32_t d = tmem + buf * kN;
                ok = mbar_wait(acc_empty + buf, ((it >> 1) & 1) ^ 1) && !*s_fail;
                if (!ok) break;
                tc_fence_after();
                for (int k = 0; k < q.k_panels; ++k, ++n) {
                    const int s = n % L::stages;
                    ok = mbar_wait(full + s, (n / L::stages) & 1) && !*s_fail;
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = base + s * L::stage;
                    uint64_t a[kParts], b[kParts];
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        a[p] = desc_sw128(at + p * L::a, 16);
                        b[p] = desc_sw128(at + kParts * L::a + p * L::b,
                                          kGram ? 16 : kPanel * kPanel * 2);
                    }
#pragma unroll
                    for (int e = 0; e < kPanel / 16; ++e) {
                        // 16 of K: 32 bytes along a K-major row, 16 rows of an MN-major operand
                        const uint32_t ea = 32u * e >> 4, eb = kGram ? ea : (2048u * e >> 4);
                        mma_f16(d, a[0] + ea, b[0] + eb, idesc, (k | e) != 0);
                        if (kSplit) {
                            mma_f16(d, a[0] + ea, b[kParts - 1] + eb, idesc, 1);
                            mma_f16(d, a[kParts - 1] + ea, b[0] + eb, idesc, 1);
                        }
                    }
                    mma_commit(empty + s);
                }
                if (ok) mma_commit(acc_full + buf);
            }
            if (!ok) {
                *s_fail = 1u;
                mma_commit(drain);
                mbar_wait(drain, 0);
            }
        }
    } else {   // ---- epilogue
        const int quarter = warp & 3, lane = tid & 31;
        const int row = quarter * 32 + lane;   // of the tile: its lane in tensor memory
        const bool lead = tid == 64;
        unsigned char* stage = smem + L::staging;
        int it = 0;
        for (int t = blockIdx.x; t < total; t += gridDim.x, ++it) {
            const int buf = it & 1;
            int z, i, j;
            place(t, &z, &i, &j);
            const bool ok = mbar_wait(acc_full + buf, (it >> 1) & 1) && !*s_fail;
            if (epilogue_any(!ok)) {
                *s_fail = 1u;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + buf * kN + ((uint32_t)(quarter * 32) << 16);
            const int64_t grow = (int64_t)i * kBlock + row;
            // 32 columns of this row of D
            auto values = [&](int col, float (&v)[32]) {
                uint32_t u[32];
                __syncwarp();
                tmem_ld32(acc + col, u);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = q.alpha * __uint_as_float(u[e]);
                if (q.c) {
                    const __half* c = q.c + z * q.d_size;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int64_t gcol = (int64_t)j * kN + col + 8 * h;
                        const size_t at = panel_at(grow, gcol, q.d_rows);
#pragma unroll
                        for (int p = 0; p < kParts; ++p) {
                            const uint4 w = *reinterpret_cast<const uint4*>(c + p * q.d_lo + at);
                            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 f =
                                    __half22float2(*reinterpret_cast<const __half2*>(&ws[e]));
                                v[8 * h + 2 * e] = fmaf(q.beta, f.x, v[8 * h + 2 * e]);
                                v[8 * h + 2 * e + 1] = fmaf(q.beta, f.y, v[8 * h + 2 * e + 1]);
                            }
                        }
                    }
                    const int64_t on = grow - ((int64_t)j * kN + col);   // the diagonal
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] += e == on ? q.gamma : 0.0f;
                }
            };
            if (q.out) {
                for (int col = 0; col < kN; col += 32) {
                    float v[32];
                    values(col, v);
                    const int64_t gcol = (int64_t)j * kN + col;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        if (grow >= q.out_r || gcol + e >= q.out_c) continue;
                        const size_t at = (size_t)z * q.out_r * q.out_c +
                                          (q.tall ? (gcol + e) * q.out_r + grow
                                                  : grow * q.out_c + gcol + e);
                        if (q.dtype == kF32)
                            static_cast<float*>(q.out)[at] = v[e];
                        else
                            static_cast<__nv_bfloat16*>(q.out)[at] = __float2bfloat16_rn(v[e]);
                    }
                }
            } else {
                __half* d = q.d + z * q.d_size;
                for (int c = 0; c < kPanels; ++c) {
                    uint4 h[8][kParts];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float v[32];
                        values(c * kPanel + 32 * half, v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float w[8];
#pragma unroll
                            for (int b = 0; b < 8; ++b) w[b] = v[8 * e + b];
                            halves<kParts>(w, h[4 * half + e]);
                        }
                    }
                    __half* dst = d + ((size_t)(j * kPanels + c) * q.d_rows + (size_t)i * kBlock) *
                                          kPanel;
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        unsigned char* b = stage + ((c * kParts + p) & 1) * kStaging;
                        if (lead) bulk_store_read<1>();
                        epilogue_sync();
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<uint4*>(b + row * 128 + ((e ^ (row & 7)) << 4)) =
                                h[e][p];
                        fence_async_smem();
                        epilogue_sync();
                        if (lead) bulk_store(dst + p * q.d_lo, b, kStaging);
                    }
                }
                if (kGram && i != j) {   // the mirrored tile: its panels are halves of our rows
#pragma unroll 1
                    for (int p = 0; p < kParts; ++p) {
                        if (lead) bulk_store_read<0>();
                        epilogue_sync();
                        unsigned char* b = stage + (row >> 6) * kStaging + (row & 7) * 2;
                        const int chunk = (row & 63) >> 3;
                        for (int col = 0; col < kN; col += 32) {
                            float v[32];
                            values(col, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                __half h = __float2half_rn(v[e]);
                                if (p == 1) h = __float2half_rn(v[e] - __half2float(h));
                                *reinterpret_cast<__half*>(b + (col + e) * 128 +
                                                           ((chunk ^ (e & 7)) << 4)) = h;
                            }
                        }
                        fence_async_smem();
                        epilogue_sync();
                        if (lead) {
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                bulk_store(d + p * q.d_lo + ((size_t)(2 * i + c) * q.d_rows +
                                                             (size_t)j * kBlock) * kPanel,
                                           stage + c * kStaging, kStaging);
                        }
                    }
                }
            }
            tc_fence_before();
            epilogue_sync();
            if (lead) mbar_arrive(acc_empty + buf);
        }
        if (lead) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *s_fail) atomicOr(&st->error, kErrTimeout);
    if (warp == 1) tmem_dealloc(tmem, 2 * kN);
}

// ----------------------------------------------------------------- plans --
struct Plan {
    int64_t r, c, rp, cp;   // padded
    bool tall;
    int parts;
};
Plan plan_of(int64_t m, int64_t n, int dtype) {
    Plan p;
    p.tall = m > n;
    p.r = p.tall ? n : m;
    p.c = p.tall ? m : n;
    p.rp = ceil_div(p.r, kBlock) * kBlock;
    const int64_t to = p.c > 1024 ? 256 : 128;   // two widths of a tile of the last product
    p.cp = ceil_div(p.c, to) * to;
    p.parts = dtype == kF32 ? 2 : 1;
    return p;
}

struct Space {
    __half *x[2], *a, *p;
    size_t x_lo, a_lo;
    float2* part;
};
Space carve(Carve& w, int64_t batch, const Plan& p) {
    Space s;
    s.x_lo = (size_t)batch * p.rp * p.cp;
    s.a_lo = (size_t)batch * p.rp * p.rp;
    for (int k = 0; k < 2; ++k) s.x[k] = w.take<__half>(s.x_lo * p.parts);
    s.a = w.take<__half>(s.a_lo * p.parts);
    s.p = w.take<__half>(s.a_lo * p.parts);
    s.part = w.take<float2>((size_t)batch * kNormBlocks);
    return s;
}

template <bool kSplit, int kN, bool kGram>
cudaError_t product(const Product& q, LearnState* st, int n_sms, cudaStream_t s) {
    const int64_t total = (int64_t)q.tiles * q.batch;
    return launch_pdl(k_orth_product<kSplit, kN, kGram>,
                      dim3((unsigned)(total < n_sms ? total : n_sms)), dim3(kProductThreads),
                      ProductSmem<kSplit, kN>::bytes, s, q, st);
}

template <typename T, bool kSplit>
cudaError_t run(const OrthCall& o, LearnState* st, void* ws, int n_sms, cudaStream_t s) {
    constexpr int kParts = kSplit ? 2 : 1;
    const Plan p = plan_of(o.m, o.n, o.dtype);
    Carve cv{static_cast<unsigned char*>(ws)};
    const Space w = carve(cv, o.batch, p);
    const unsigned B = (unsigned)o.batch;
    const int64_t elems = p.r * p.c;
    const int64_t want = ceil_div(elems, kThreads * 16);
    const int parts = (int)(want < kNormBlocks ? want : kNormBlocks);
    const auto flat = [&](int64_t items) {
        const int64_t b = ceil_div(items, kThreads);
        return dim3((unsigned)(b < 2048 ? b : 2048), B);
    };
    cudaError_t e = launch_pdl(k_orth_norm<T>, dim3(parts, B), dim3(kThreads), 0, s,
                               (const T*)o.grad, elems, w.part);
    if (e != cudaSuccess) return e;
    if (o.steps == 0)
        return launch_pdl(k_orth_scale<T>, flat(elems), dim3(kThreads), 0, s, (const T*)o.grad,
                          elems, (const float2*)w.part, parts, o.eps, (T*)o.out);
    e = launch_pdl(k_orth_start<T, kParts>, flat(p.rp * p.cp / 8), dim3(kThreads), 0, s,
                   (const T*)o.grad, p.r, p.c, p.rp, p.cp, p.tall, (const float2*)w.part, parts,
                   o.eps, w.x[0], w.x_lo);
    const int tm = (int)(p.rp / kBlock);
    for (int k = 0; k < o.steps && e == cudaSuccess; ++k) {
        const __half* x = w.x[k & 1];
        Product g{};   // A = X X^T
        g.l = g.r = x;
        g.l_lo = g.r_lo = w.x_lo;
        g.l_size = g.r_size = (size_t)p.rp * p.cp;
        g.l_rows = g.r_rows = p.rp;
        g.k_panels = (int)(p.cp / kPanel);
        g.tiles_m = g.tiles_n = tm;
        g.tiles = tm * (tm + 1) / 2;
        g.batch = (int)o.batch;
        g.d = w.a;
        g.d_lo = w.a_lo;
        g.d_size = (size_t)p.rp * p.rp;
        g.d_rows = p.rp;
        g.alpha = kScaleA / (kScaleX * kScaleX);
        e = product<kSplit, kBlock, true>(g, st, n_sms, s);
        if (e != cudaSuccess) return e;
        Product h = g;   // P = a I + b A + c A A
        h.l = h.r = h.c = w.a;
        h.l_lo = h.r_lo = w.a_lo;
        h.l_size = h.r_size = (size_t)p.rp * p.rp;
        h.k_panels = (int)(p.rp / kPanel);
        h.d = w.p;
        h.alpha = o.c * (kScaleP / (kScaleA * kScaleA));
        h.beta = o.b * (kScaleP / kScaleA);
        h.gamma = o.a * kScaleP;
        e = product<kSplit, kBlock, true>(h, st, n_sms, s);
        if (e != cudaSuccess) return e;
        Product f = g;   // X' = P X
        f.l = w.p;
        f.l_lo = w.a_lo;
        f.l_size = (size_t)p.rp * p.rp;
        f.k_panels = (int)(p.rp / kPanel);
        f.d = w.x[(k + 1) & 1];
        f.d_lo = w.x_lo;
        f.d_size = (size_t)p.rp * p.cp;
        f.alpha = 1.0f / kScaleP;
        if (k + 1 == o.steps) {
            f.out = o.out;
            f.out_r = p.r;
            f.out_c = p.c;
            f.tall = p.tall;
            f.dtype = o.dtype;
            f.alpha = 1.0f / (kScaleP * kScaleX);
        }
        // 256 columns a tile move fewer operand bytes per product; 128 give twice the tiles
        const bool wide = !kSplit && p.cp % 256 == 0 &&
                          (int64_t)tm * (p.cp / 256) * o.batch >= n_sms;
        f.tiles_n = (int)(p.cp / (wide ? 256 : 128));
        f.tiles = tm * f.tiles_n;
        if (wide)
            e = product<kSplit, kSplit ? 128 : 256, false>(f, st, n_sms, s);
        else
            e = product<kSplit, 128, false>(f, st, n_sms, s);
    }
    return e;
}

template <bool kSplit, int kN, bool kGram>
cudaError_t prepare_one() {
    return cudaFuncSetAttribute(k_orth_product<kSplit, kN, kGram>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                ProductSmem<kSplit, kN>::bytes);
}

}  // namespace

size_t orth_workspace(int64_t batch, int64_t m, int64_t n, int dtype) {
    if (batch == 0 || m == 0 || n == 0) return 0;
    Carve cv{nullptr};
    carve(cv, batch, plan_of(m, n, dtype));
    return cv.used;
}

cudaError_t prepare_orth() {
    cudaError_t e = prepare_one<false, 128, true>();
    if (e == cudaSuccess) e = prepare_one<false, 128, false>();
    if (e == cudaSuccess) e = prepare_one<false, 256, false>();
    if (e == cudaSuccess) e = prepare_one<true, 128, true>();
    if (e == cudaSuccess) e = prepare_one<true, 128, false>();
    return e;
}

cudaError_t launch_orth(const OrthCall& q, LearnState* st, void* ws, int n_sms, cudaStream_t s) {
    if (q.batch == 0 || q.m == 0 || q.n == 0) return cudaSuccess;
    return q.dtype == kF32 ? run<float, true>(q, st, ws, n_sms, s)
                           : run<__nv_bfloat16, false>(q, st, ws, n_sms, s);
}

}  // namespace pulsar
