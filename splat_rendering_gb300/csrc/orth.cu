// Orthogonalisation of an update by Newton-Schulz products:
//
//   X_0 = G / (|G|_F + eps),   X' = a X + (b A + c A^2) X,   A = X X^T
//
// for every matrix of a batch, on the orientation with the fewer rows (the
// result of the transpose is the transpose of the result).
#include "learn_internal.cuh"

namespace pulsar {
namespace {

constexpr int kThreads = 256;

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

// x [r, c] = g / (|g| + eps), g [m, n] transposed where it is tall.
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_orth_start(const T* __restrict__ g, int64_t r, int64_t c, bool tall,
             const float2* __restrict__ part, int parts, float eps, float* __restrict__ x) {
    pdl_begin();
    const float inv = inv_norm(part + (size_t)blockIdx.y * parts, parts, eps);
    const T* m = g + (size_t)blockIdx.y * r * c;
    float* o = x + (size_t)blockIdx.y * r * c;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < r * c;
         i += (int64_t)gridDim.x * kThreads) {
        float v[1];
        Pack<T, 1>::load(m + (tall ? (i % c) * r + i / c : i), v);
        o[i] = v[0] * inv;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
k_orth_finish(const float* __restrict__ x, int64_t r, int64_t c, bool tall, T* __restrict__ out) {
    pdl_begin();
    const float* m = x + (size_t)blockIdx.y * r * c;
    T* o = out + (size_t)blockIdx.y * r * c;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < r * c;
         i += (int64_t)gridDim.x * kThreads) {
        const float v[1] = {m[i]};
        Pack<T, 1>::store(o + (tall ? (i % c) * r + i / c : i), v);
    }
}

// -------------------------------------------------------------- products --
// D = alpha L R + beta C + gamma I, a 64 x 64 tile per block in 32 bits; R is
// [n, k] row-major (kNt, the product with a transpose) or [k, n].
constexpr int kTileG = 64, kStepG = 16;

template <bool kNt>
__global__ void __launch_bounds__(kThreads)
k_orth_product(const float* __restrict__ l, const float* __restrict__ r,
               const float* __restrict__ c, int64_t m, int64_t n, int64_t k, float alpha,
               float beta, float gamma, float* __restrict__ d) {
    pdl_begin();
    __shared__ float sl[kStepG][kTileG + 4], sr[kStepG][kTileG + 4];
    const size_t z = blockIdx.z;
    l += z * m * k;
    r += z * n * k;
    d += z * m * n;
    if (c) c += z * m * n;
    const int64_t m0 = (int64_t)blockIdx.y * kTileG, n0 = (int64_t)blockIdx.x * kTileG;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < k; k0 += kStepG) {
        for (int e = threadIdx.x; e < kTileG * kStepG; e += kThreads) {
            const int row = e / kStepG, kk = e % kStepG;
            sl[kk][row] = m0 + row < m && k0 + kk < k ? l[(m0 + row) * k + k0 + kk] : 0.0f;
            if (kNt) {
                sr[kk][row] = n0 + row < n && k0 + kk < k ? r[(n0 + row) * k + k0 + kk] : 0.0f;
            } else {
                const int col = e % kTileG, kr = e / kTileG;
                sr[kr][col] = n0 + col < n && k0 + kr < k ? r[(k0 + kr) * n + n0 + col] : 0.0f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kStepG; ++kk) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = sl[kk][ty * 4 + i];
                b[i] = sr[kk][tx * 4 + i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t row = m0 + ty * 4 + i, col = n0 + tx * 4 + j;
            if (row >= m || col >= n) continue;
            float v = alpha * acc[i][j];
            if (c) v = fmaf(beta, c[row * n + col], v);
            if (row == col) v += gamma;
            d[row * n + col] = v;
        }
}

struct Space {
    float *x[2], *a, *p;
    float2* part;
};
Space carve(Carve& w, int64_t batch, int64_t r, int64_t c) {
    Space s;
    for (int k = 0; k < 2; ++k) s.x[k] = w.take<float>((size_t)batch * r * c);
    s.a = w.take<float>((size_t)batch * r * r);
    s.p = w.take<float>((size_t)batch * r * r);
    s.part = w.take<float2>((size_t)batch * kNormBlocks);
    return s;
}

template <typename T>
cudaError_t run(const OrthCall& q, void* ws, cudaStream_t s) {
    const bool tall = q.m > q.n;
    const int64_t r = tall ? q.n : q.m, c = tall ? q.m : q.n, elems = r * c;
    Carve cv{static_cast<unsigned char*>(ws)};
    const Space w = carve(cv, q.batch, r, c);
    const unsigned B = (unsigned)q.batch;
    const int64_t want = ceil_div(elems, kThreads * 16);
    const int parts = (int)(want < kNormBlocks ? want : kNormBlocks);
    const int64_t wide = ceil_div(elems, kThreads * 4);
    const dim3 flat((unsigned)(wide < 4096 ? wide : 4096), B);
    cudaError_t e = launch_pdl(k_orth_norm<T>, dim3(parts, B), dim3(kThreads), 0, s,
                               (const T*)q.grad, elems, w.part);
    if (e == cudaSuccess)
        e = launch_pdl(k_orth_start<T>, flat, dim3(kThreads), 0, s, (const T*)q.grad, r, c, tall,
                       (const float2*)w.part, parts, q.eps, w.x[0]);
    const dim3 gr((unsigned)ceil_div(r, kTileG), (unsigned)ceil_div(r, kTileG), B);
    const dim3 gx((unsigned)ceil_div(c, kTileG), (unsigned)ceil_div(r, kTileG), B);
    for (int k = 0; k < q.steps && e == cudaSuccess; ++k) {
        const float* x = w.x[k & 1];
        e = launch_pdl(k_orth_product<true>, gr, dim3(kThreads), 0, s, x, x, (const float*)nullptr,
                       r, r, c, 1.0f, 0.0f, 0.0f, w.a);
        if (e == cudaSuccess)
            e = launch_pdl(k_orth_product<true>, gr, dim3(kThreads), 0, s, (const float*)w.a,
                           (const float*)w.a, (const float*)w.a, r, r, r, q.c, q.b, q.a, w.p);
        if (e == cudaSuccess)
            e = launch_pdl(k_orth_product<false>, gx, dim3(kThreads), 0, s, (const float*)w.p, x,
                           (const float*)nullptr, r, c, r, 1.0f, 0.0f, 0.0f, w.x[(k + 1) & 1]);
    }
    if (e == cudaSuccess)
        e = launch_pdl(k_orth_finish<T>, flat, dim3(kThreads), 0, s,
                       (const float*)w.x[q.steps & 1], r, c, tall, (T*)q.out);
    return e;
}

}  // namespace

size_t orth_workspace(int64_t batch, int64_t m, int64_t n, int dtype) {
    (void)dtype;
    if (batch == 0 || m == 0 || n == 0) return 0;
    Carve cv{nullptr};
    carve(cv, batch, m < n ? m : n, m < n ? n : m);
    return cv.used;
}

cudaError_t prepare_orth() { return cudaSuccess; }

cudaError_t launch_orth(const OrthCall& q, LearnState* st, void* ws, int n_sms, cudaStream_t s) {
    (void)st;
    (void)n_sms;
    if (q.batch == 0 || q.m == 0 || q.n == 0) return cudaSuccess;
    return q.dtype == kF32 ? run<float>(q, ws, s) : run<__nv_bfloat16>(q, ws, s);
}

}  // namespace pulsar
