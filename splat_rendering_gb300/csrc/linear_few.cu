// Linear layers of a few outputs (heads: a density, a colour), which are bound by reading x: sums in
// 32 bits, no operands to make.  A tile of the tensor cores would hold one to four useful columns
// of 64 or more, and its epilogue stores them two bytes at a time.
#include "linear_internal.cuh"

namespace pulsar {
namespace linear {
namespace {

// As many elements of a row as one load takes.
template <typename T, int V>
struct Some : Pack<T, V> {};
template <>
struct Some<__nv_bfloat16, 2> {
    using Raw = uint32_t;
    static __device__ __forceinline__ Raw raw(const __nv_bfloat16* p) {
        return *reinterpret_cast<const uint32_t*>(p);
    }
    static __device__ __forceinline__ void open(const Raw& u, float (&v)[2]) {
        v[0] = low_of(u);
        v[1] = high_of(u);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[2]) {
        *reinterpret_cast<uint32_t*>(p) = pair_bf16(v[0], v[1]);
    }
};

template <>
struct Some<__nv_bfloat16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ Raw raw(const __nv_bfloat16* p) {
        return *reinterpret_cast<const uint2*>(p);
    }
    static __device__ __forceinline__ void open(const Raw& u, float (&v)[4]) {
        v[0] = low_of(u.x);
        v[1] = high_of(u.x);
        v[2] = low_of(u.y);
        v[3] = high_of(u.y);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[4]) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pair_bf16(v[0], v[1]), pair_bf16(v[2], v[3]));
    }
};

constexpr int kBatch = 4;    // rows of a thread in flight
constexpr int kChunk = 1024;   // rows whose dz a block has at a time
constexpr int kBlocks = 4;     // of an SM, of the backward call, at most

// The outputs: 1 << log_g lanes to a row, each with every so many'th V of its inputs, the weights
// in shared memory in 32 bits.  590465 x 96 -> 1 in 16 bits: 20 us for 115 MB, 84 % of the copy rate
// (the narrow layers' kernel 39), 874606 x 4 -> 1 4.8 (45); it waits for its loads.
template <typename T, int V, int kN>
__global__ void __launch_bounds__(256)
k_linear_few(const T* __restrict__ x, const T* __restrict__ weight, int k, int log_g,
             const __grid_constant__ Result q) {
    extern __shared__ float w[];   // [kN][k]
    pdl_next();
    pdl_begin();
    for (int i = threadIdx.x; i < kN * k; i += 256) {
        float v[1];
        Pack<T, 1>::load(weight + i, v);
        w[i] = v[0];
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, g = lane & ((1 << log_g) - 1), rows = 32 >> log_g;
    const int64_t step = (int64_t)gridDim.x * 8 * kBatch * rows;
    for (int64_t first = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kBatch * rows; first < q.m;
         first += step) {
        const int64_t row = first + (lane >> log_g);
        const T* at = x + row * k;
        float sum[kBatch][kN];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int j = 0; j < kN; ++j) sum[i][j] = 0.0f;
#pragma unroll 2
        for (int c = g * V; c < k; c += V << log_g) {
            typename Some<T, V>::Raw u[kBatch] = {};
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (row + i * rows < q.m) u[i] = Some<T, V>::raw(at + (int64_t)i * rows * k + c);
            float b[kN][V];
#pragma unroll
            for (int j = 0; j < kN; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) b[j][e] = w[j * k + c + e];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float a[V];
                Some<T, V>::open(u[i], a);
#pragma unroll
                for (int j = 0; j < kN; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) sum[i][j] = fmaf(a[e], b[j][e], sum[i][j]);
            }
        }
        for (int d = 1; d < 1 << log_g; d *= 2)
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    sum[i][j] += __shfl_xor_sync(0xffffffffu, sum[i][j], d);
        // a row's results by one of its lanes
        for (int h = 0; h < kBatch; h += 1 << log_g) {
            const int i = h + g;
            if (i >= kBatch || row + i * rows >= q.m) continue;
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                float z = sum[0][j];
#pragma unroll
                for (int e = 1; e < kBatch; ++e) z = i == e ? sum[e][j] : z;
                finish1<T>(q, plus(z, q.bias ? q.bias[j] : 0.0f), (row + i * rows) * kN + j);
            }
        }
    }
}

// The gradients in one pass: a thread has V columns of every (256 >> log_tx)-th row, its sums of dW
// in registers and added up over the block; dz, in shared memory, stays in 32 bits.  590465 x 96 -> 1 in 16 bits with SiLU:
// 45 us for 229 MB, with the join (the narrow layers' kernel 112).
struct Few {
    const void *dy, *pre, *x, *weight;   // pre, x, weight: NULL where not read
    void* dx;                            // NULL: not wanted
    float *parts, *sums;                 // of dW [blocks][part], of the bias [blocks][kN]; NULL
    int64_t m, block_rows, part;
    int k, act, log_tx;
};
template <typename T, int V, int kN>
__global__ void __launch_bounds__(256, 2)
k_linear_few_back(const __grid_constant__ Few q) {
    __shared__ float s[256 * V], s_dz[kChunk * kN];
    pdl_next();
    pdl_begin();
    const int tid = threadIdx.x, tx = 1 << q.log_tx, step = 256 >> q.log_tx;
    const int c = ((int)blockIdx.y * tx + (tid & (tx - 1))) * V;
    const bool mine = c < q.k;
    const int64_t r0 = blockIdx.x * q.block_rows;
    const int64_t r1 = r0 + q.block_rows < q.m ? r0 + q.block_rows : q.m;
    const T* dy = static_cast<const T*>(q.dy);
    const T* pre = static_cast<const T*>(q.pre);
    const T* x = static_cast<const T*>(q.x) + c;
    T* dx = static_cast<T*>(q.dx) + c;
    float w[kN][V], sum[kN][V], bias[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        bias[j] = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            sum[j][e] = 0.0f;
            float u[1] = {0.0f};
            if (q.dx && mine) Pack<T, 1>::load(static_cast<const T*>(q.weight) + j * q.k + c + e, u);
            w[j][e] = u[0];
        }
    }
    for (int64_t first = r0; first < r1; first += kChunk) {
        const int rows = (int)(r1 - first < kChunk ? r1 - first : kChunk);
        __syncthreads();
        for (int i = tid; i < rows * kN; i += 256) {
            float v[1], z[1] = {0.0f};
            Pack<T, 1>::load(dy + first * kN + i, v);
            if (q.act != kActNone) Pack<T, 1>::load(pre + first * kN + i, z);
            if (q.act == kActSilu) to_dz<kActSilu>(v, z);
            else if (q.act == kActRelu) to_dz<kActRelu>(v, z);
            s_dz[i] = v[0];
        }
        __syncthreads();
        for (int r = tid >> q.log_tx; r < rows; r += kBatch * step) {
            typename Some<T, V>::Raw u[kBatch] = {};
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (q.parts && mine && r + i * step < rows)
                    u[i] = Some<T, V>::raw(x + (first + r + i * step) * q.k);
            // in 32 bits a batch's sums are apart: a quarter as many roundings in a row
            float more[sizeof(T) == 4 ? kN : 1][V];
            if (sizeof(T) == 4) {
#pragma unroll
                for (int j = 0; j < kN; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) more[sizeof(T) == 4 ? j : 0][e] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (r + i * step >= rows) continue;
                float a[V], y[V];
                Some<T, V>::open(u[i], a);
#pragma unroll
                for (int e = 0; e < V; ++e) y[e] = 0.0f;
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    const float dz = s_dz[(r + i * step) * kN + j];
                    float(&to)[V] = sizeof(T) == 4 ? more[sizeof(T) == 4 ? j : 0] : sum[j];
                    bias[j] += dz;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        to[e] = fmaf(dz, a[e], to[e]);
                        y[e] = fmaf(dz, w[j][e], y[e]);
                    }
                }
                if (q.dx && mine) Some<T, V>::store(dx + (first + r + i * step) * q.k, y);
            }
            if (sizeof(T) == 4) {
#pragma unroll
                for (int j = 0; j < kN; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) sum[j][e] += more[sizeof(T) == 4 ? j : 0][e];
            }
        }
    }
    __syncthreads();
    // the block's sums: [step][tx V] by halves
    const int width = tx * V;
    if (q.parts) {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
#pragma unroll
            for (int e = 0; e < V; ++e) s[tid * V + e] = sum[j][e];
            __syncthreads();
            for (int half = step / 2; half > 0; half /= 2) {
                for (int i = tid; i < half * width; i += 256) s[i] += s[i + half * width];
                __syncthreads();
            }
            for (int i = tid; i < width; i += 256) {
                const int col = (int)blockIdx.y * width + i;
                if (col < q.k) q.parts[blockIdx.x * q.part + (int64_t)j * q.k + col] = s[i];
            }
            __syncthreads();
        }
    }
    if (q.sums && blockIdx.y == 0) {   // of the first columns' threads
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            if ((tid & (tx - 1)) == 0) s[tid >> q.log_tx] = bias[j];
            __syncthreads();
            for (int half = step / 2; half > 0; half /= 2) {
                if (tid < half) s[tid] += s[tid + half];
                __syncthreads();
            }
            if (tid == 0) q.sums[blockIdx.x * kN + j] = s[0];
            __syncthreads();
        }
    }
}

int log2_up(int64_t n, int most) {
    int log = 0;
    while (log < most && (int64_t)1 << log < n) ++log;
    return log;
}

// The widest load that rows of k elements allow which begin at all of `ps`.
template <typename T>
int width_of(int64_t k, const void* a, const void* b) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b);
    if (k % VecOf<T>::n == 0 && at % 16 == 0) return VecOf<T>::n;
    if (sizeof(T) == 4) return 1;
    return k % 4 == 0 && at % 8 == 0 ? 4 : k % 2 == 0 && at % 4 == 0 ? 2 : 1;
}
// kernel<V, kN> of a call: f is called with both as constants
template <typename T, typename F>
cudaError_t with_sizes(int width, int64_t n, F f) {
    const auto outputs = [&](auto v) {
        return n == 1   ? f(v, std::integral_constant<int, 1>())
               : n == 2 ? f(v, std::integral_constant<int, 2>())
               : n == 3 ? f(v, std::integral_constant<int, 3>())
                        : f(v, std::integral_constant<int, 4>());
    };
    if (width == VecOf<T>::n) return outputs(std::integral_constant<int, VecOf<T>::n>());
    if constexpr (sizeof(T) == 2) {
        if (width == 4) return outputs(std::integral_constant<int, 4>());
        if (width == 2) return outputs(std::integral_constant<int, 2>());
    }
    return outputs(std::integral_constant<int, 1>());
}

// Blocks of rows: as many for an SM, over all columns, as it holds at once by their registers (`held`
// floats of a thread: 590465 x 64 -> 4 in 32 bits 70 us by two, 75 by four; 952959 x 52 -> 3 in 16
// bits 80 and 60), of kBatch rows for each thread or more.
struct FewGrid {
    int log_tx;
    int64_t block_rows, blocks, col_blocks;
};
FewGrid few_grid(int64_t rows, int64_t k, int width, int held, int n_sms) {
    FewGrid g;
    const int64_t groups = ceil_div(k, width);
    g.log_tx = log2_up(groups, 5);
    g.col_blocks = ceil_div(groups, 1 << g.log_tx);
    const int64_t least = kBatch * (256 >> g.log_tx);
    int64_t want = (held < 32 ? kBlocks : 2) * n_sms / g.col_blocks;
    if (want < 1) want = 1;
    g.block_rows = ceil_div(ceil_div(rows, want), least) * least;
    g.blocks = ceil_div(rows, g.block_rows);
    return g;
}

}  // namespace

bool is_few(int64_t inputs, int64_t outputs) {
    return outputs <= kFewOutputs && inputs <= kFewInputs;
}
int64_t few_parts(int64_t rows, int n_sms) {
    const int64_t least = ceil_div(rows, kBatch * 8);
    return least < kBlocks * n_sms ? least : kBlocks * n_sms;
}

// The other forms keep what they are faster at: up to 128 inputs the narrow one, but for 32 inputs or
// fewer and loads of 8 bytes or more (1176470 x 51 -> 4 in 16 bits 67 us, here 111; 967741 x 31 54,
// here 42; 590465 x 96 42, here 30); above 128 the products of 16 bits, where they need no copy of x
// (58593 x 1024 -> 4 32 us, here 55; to one output 32, here 25; 119521 x 502 -> 4 96, here 58).
template <typename T>
bool launch_few(const LinearCall& c, const Result& q, int n_sms, cudaStream_t s, cudaError_t* result) {
    if (!is_few(c.inputs, c.outputs)) return false;
    const int width = width_of<T>(c.inputs, c.x, nullptr);
    if (c.inputs > 32 && c.inputs <= 128 && width * sizeof(T) < 8) return false;
    if (c.inputs > 128 && sizeof(T) == 2 && width == VecOf<T>::n && c.outputs > 1 &&
        c.inputs * c.outputs > 1024)
        return false;
    *result = with_sizes<T>(width, c.outputs, [&](auto v, auto n) {
        constexpr int V = decltype(v)::value, kN = decltype(n)::value;
        const int log_g = log2_up(ceil_div(c.inputs / V, 4), 5);   // (up to four loads to a lane)
        const int64_t blocks = ceil_div(c.rows, 8 * kBatch * (32 >> log_g));
        const int64_t most = n_sms * (sizeof(T) == 2 ? 6 : 4);   // (in 32 bits 4 are up to a tenth faster)
        return launch_pdl(k_linear_few<T, V, kN>,
                          dim3((unsigned)(blocks < most ? blocks : most)), dim3(256),
                          (size_t)(kN * c.inputs * 4), s, static_cast<const T*>(c.x),
                          static_cast<const T*>(c.weight), (int)c.inputs, log_g, q);
    });
    return true;
}
template bool launch_few<float>(const LinearCall&, const Result&, int, cudaStream_t, cudaError_t*);
template bool launch_few<__nv_bfloat16>(const LinearCall&, const Result&, int, cudaStream_t,
                                        cudaError_t*);

template <typename T>
cudaError_t launch_few_back(const LinearCall& c, float* parts, float* sums, int n_sms, cudaStream_t s,
                            int64_t* blocks) {
    const int width = width_of<T>(c.inputs, c.grad_weight ? c.x : nullptr, c.grad_x);
    const int held = (int)c.outputs * width * (sizeof(T) == 4 ? 3 : 2);
    const FewGrid g = few_grid(c.rows, c.inputs, width, held, n_sms);
    *blocks = g.blocks;
    const Few q{c.grad_y, c.pre, c.x, c.weight, c.grad_x, parts, sums, c.rows, g.block_rows,
                part_size(c.outputs, c.inputs), (int)c.inputs, c.act, g.log_tx};
    return with_sizes<T>(width, c.outputs, [&](auto v, auto n) {
        return launch_pdl(k_linear_few_back<T, decltype(v)::value, decltype(n)::value>,
                          dim3((unsigned)g.blocks, (unsigned)(c.grad_x || parts ? g.col_blocks : 1)),
                          dim3(256), 0, s, q);
    });
}
template cudaError_t launch_few_back<float>(const LinearCall&, float*, float*, int, cudaStream_t,
                                            int64_t*);
template cudaError_t launch_few_back<__nv_bfloat16>(const LinearCall&, float*, float*, int,
                                                    cudaStream_t, int64_t*);

}  // namespace linear
}  // namespace pulsar
