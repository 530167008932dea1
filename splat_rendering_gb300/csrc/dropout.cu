// Dropout without a stored mask:
//
//   y_i = [w_i >= p 2^32] x_i / (1 - p) + residual_i
//
// w_i is word i mod 4 of Philox4x32 (Salmon, Moraes, Dror, Shaw: Parallel
// random numbers: as easy as 1, 2, 3, SC 2011) with seven rounds, the fewest
// that pass the paper's tests, of the counter offset + i / 4 under the key
// `seed`.  So the gradient is the same call on dy.
//
// Bound by DRAM in 32 bits (16M values with a residual: 27 us, 7.4 TB/s in a run
// of calls on the same tensors, some of them still in the L2).  In 16 bits the
// generator, two wide multiplications a round for four values, costs 3 us of 36
// for 50M values (199 MB; one round instead of seven: 33), as its instructions
// keep warps from issuing loads.  The rounds' keys are arguments: worked out by
// every thread they cost another 2 us.
#include "learn_internal.cuh"

namespace pulsar {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;   // vectors a thread has in flight

constexpr int kRounds = 7;

struct Draw {
    uint32_t key[kRounds][2];   // of each round
    uint64_t offset;
    const int64_t* counter;     // added to the offset; may be NULL
    uint32_t least;             // the smallest word that keeps an element
    float scale;
};

__device__ __forceinline__ uint4 philox(uint64_t counter, const Draw& d) {
    uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c2 = 0, c3 = 0;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ d.key[r][0];
        c2 = (uint32_t)(a >> 32) ^ c3 ^ d.key[r][1];
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Four elements from their words.
template <bool kSkip>
__device__ __forceinline__ void keep4(const Draw& d, uint64_t block, const float* x, const float* r,
                                      float* y) {
    const uint4 u = philox(block, d);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float skip = kSkip ? r[e] : 0.0f;
        y[e] = w[e] >= d.least ? fmaf(x[e], d.scale, skip) : skip;
    }
}

// V elements at a time (a multiple of four), and the rest by one thread.  (out may be x or
// residual: a thread writes what it alone has read.)
template <typename T, int V, bool kSkip>
__global__ void __launch_bounds__(kThreads)
k_dropout(const T* x, const T* residual, int64_t n, const __grid_constant__ Draw d, T* out) {
    pdl_begin();
    const uint64_t first = d.offset + (d.counter ? (uint64_t)*d.counter : 0u);
    const int64_t vectors = n / V, step = (int64_t)gridDim.x * kThreads;
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    for (int64_t i0 = t; i0 < vectors; i0 += step * kAhead) {
        typename Pack<T, V>::Raw a[kAhead], b[kAhead];
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
            const int64_t i = i0 + h * step;
            if (i < vectors) {
                a[h] = Pack<T, V>::raw_last(x + i * V);
                if (kSkip) b[h] = Pack<T, V>::raw_last(residual + i * V);
            }
        }
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
            const int64_t i = i0 + h * step;
            if (i < vectors) {
                float u[V], r[V], y[V];
                Pack<T, V>::open(a[h], u);
                if (kSkip) Pack<T, V>::open(b[h], r);
#pragma unroll
                for (int e = 0; e < V; e += 4)
                    keep4<kSkip>(d, first + (uint64_t)(i * V + e) / 4, u + e, r + e, y + e);
                Pack<T, V>::store_through(out + i * V, y);
            }
        }
    }
    if (t == 0) {
        for (int64_t i = vectors * V; i < n; i += 4) {
            float u[4], r[4], y[4];
            const int m = (int)(n - i < 4 ? n - i : 4);
            for (int e = 0; e < 4; ++e) {
                float one[1] = {0.0f};
                if (e < m) Pack<T, 1>::load(x + i + e, one);
                u[e] = one[0];
                if (kSkip && e < m) Pack<T, 1>::load(residual + i + e, one);
                r[e] = one[0];
            }
            keep4<kSkip>(d, first + (uint64_t)i / 4, u, r, y);
            for (int e = 0; e < m; ++e) {
                const float one[1] = {y[e]};
                Pack<T, 1>::store(out + i + e, one);
            }
        }
    }
}

// Tensors at any element alignment: four elements a thread, one at a time.
template <typename T, bool kSkip>
__global__ void __launch_bounds__(kThreads)
k_dropout_any(const T* x, const T* residual, int64_t n, const __grid_constant__ Draw d, T* out) {
    pdl_begin();
    const uint64_t first = d.offset + (d.counter ? (uint64_t)*d.counter : 0u);
    const int64_t blocks = (n + 3) / 4, step = (int64_t)gridDim.x * kThreads;
    for (int64_t b = (int64_t)blockIdx.x * kThreads + threadIdx.x; b < blocks; b += step) {
        float u[4], r[4], y[4];
        const int64_t i = b * 4;
        const int m = (int)(n - i < 4 ? n - i : 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float one[1] = {0.0f};
            if (e < m) Pack<T, 1>::load(x + i + e, one);
            u[e] = one[0];
            if (kSkip && e < m) Pack<T, 1>::load(residual + i + e, one);
            r[e] = one[0];
        }
        keep4<kSkip>(d, first + (uint64_t)b, u, r, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float one[1] = {y[e]};
            if (e < m) Pack<T, 1>::store(out + i + e, one);
        }
    }
}

template <typename T, bool kSkip>
cudaError_t run(const DropoutCall& c, int n_sms, cudaStream_t s) {
    constexpr int V = VecOf<T>::n;
    Draw d{{}, (uint64_t)c.offset, c.counter, c.least, c.scale};
    for (uint32_t r = 0; r < kRounds; ++r) {
        d.key[r][0] = (uint32_t)c.seed + r * 0x9E3779B9u;
        d.key[r][1] = (uint32_t)(c.seed >> 32) + r * 0xBB67AE85u;
    }
    const T *x = static_cast<const T*>(c.x), *r = static_cast<const T*>(c.residual);
    T* out = static_cast<T*>(c.out);
    const bool vec = aligned16(x) && aligned16(r) && aligned16(out);
    const int64_t threads = vec ? ceil_div(c.n, (int64_t)V * kAhead) : ceil_div(c.n, 4);
    int64_t blocks = ceil_div(threads, kThreads);
    if (blocks > n_sms * 16) blocks = n_sms * 16;
    return launch_pdl(vec ? k_dropout<T, V, kSkip> : k_dropout_any<T, kSkip>,
                      dim3((unsigned)blocks), dim3(kThreads), 0, s, x, r, c.n, d, out);
}

}  // namespace

cudaError_t launch_dropout(const DropoutCall& c, int n_sms, cudaStream_t stream) {
    if (c.n == 0) return cudaSuccess;
    if (c.dtype == kF32)
        return c.residual ? run<float, true>(c, n_sms, stream) : run<float, false>(c, n_sms, stream);
    return c.residual ? run<__nv_bfloat16, true>(c, n_sms, stream)
                      : run<__nv_bfloat16, false>(c, n_sms, stream);
}

}  // namespace pulsar
