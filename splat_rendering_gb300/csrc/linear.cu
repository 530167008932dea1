// A linear layer with its bias, activation and residual, and its gradients:
//
//   z = x W^T + b,   y = act(z) + residual            x [m, k], W [n, k]
//   dz = dy act'(z),   dx = dz W,   dW = dz^T x,   db = sum of dz's rows
//
// The three products run on the tensor cores (tcgen05, fp32 accumulation), but
// for few rows (below) or outputs (linear_few.cu).  A product is D(i, j) = sum over c of A(i, c) B(j, c); an operand's matrix in
// memory has either its i (j) or its c as rows: x, W and dz are read as they
// lie by all three products (K-major or MN-major operands).
//
// bfloat16 operands are used as they are.  A float32 value is the sum of three
// bfloat16 ones, hi + mid + lo (8 + 8 + 8 bits, the whole float32 range up to
// bfloat16's largest value, and so no scales), and a product is the sum of six
// of theirs: hi hi, hi mid, mid hi, mid mid, hi lo, lo hi.  The other three are
// at most 2^-23 of it and, their signs being random, far below the rounding of
// a sum in 32 bits.
//
// This file has the calls' plans and their small kernels: operands, joins, few rows.
#include "linear_internal.cuh"

namespace pulsar {
using namespace linear;
namespace {

// A matrix [rows, cols] made into an operand: times the activation's slope at `pre` (the gradient
// dz from dy), split into planes [planes][rows][pitch] of bfloat16, and its column sums taken, a
// partial sum [cols] per block of rows.  A thread has eight columns of every (256 / tx)-th row, and
// the loads of two or four rows in flight.  16381 x 4096 with SiLU in 16 bits: 72 us for 403 MB.
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

// kWindows: rows may be no whole vectors, and are read by windows of whole ones.  (A kernel of its
// own: its registers would cost the other a sixth, 60 us for 51 of a bias' gradient of 16381 x 4096
// with SiLU.  Four windows in flight, not one by one: the gradients of 57072 x 27 -> 782 169 -> 146.)
template <typename T, int kPlanes, int kAct, bool kWindows>
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
        for (int e = 0; e < 8; ++e) {
            v[e] = e < n ? v[e] : 0.0f;   // (what a window has behind the row)
            sum[e] += v[e];
        }
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
        const auto alone = [&](int64_t r) {
            float v[8], z[8];
            load8(src + r * q.cols, n, false, v);
            if (kAct != kActNone) load8(pre + r * q.cols, n, false, z);
            finish(r, v, z);
        };
        if constexpr (!kWindows) {   // (of 32 bits: the last four columns)
#pragma unroll 2
            for (int64_t r = r0 + ty; r < r1; r += step) alone(r);
        } else {
            constexpr int kBatch = sizeof(T) == 4 ? 2 : 4;
            const int64_t total = q.rows * q.cols;
            for (int64_t r = r0 + ty; r < r1; r += kBatch * step) {
                const int64_t last = r + (kBatch - 1) * step;
                // (a window may reach eight elements out of its own to the left, 16 to the right)
                if (last < r1 && r * q.cols + c >= 8 && last * q.cols + c + 24 <= total) {
                    Window<T, 8> a[kBatch], b[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        a[i].load(src + (r + i * step) * q.cols);
                        if (kAct != kActNone) b[i].load(pre + (r + i * step) * q.cols);
                    }
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        float v[8], z[8];
                        a[i].open(v);
                        if (kAct != kActNone) b[i].open(z);
                        finish(r + i * step, v, z);
                    }
                } else {
#pragma unroll 1
                    for (int64_t row = r; row <= last && row < r1; row += step) alone(row);
                }
            }
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

template <typename T, int kPlanes, int kAct, bool kWindows>
__global__ void __launch_bounds__(256)
k_linear_operands(const __grid_constant__ Operands all) {
    __shared__ float s_sums[256 * 8];
    pdl_next();
    pdl_begin();
    const Operand& q = all.of[blockIdx.z];
    if (blockIdx.x >= q.blocks || blockIdx.y >= q.col_blocks) return;
    if (blockIdx.z == 0) make_planes<T, kPlanes, kAct, kWindows>(q, s_sums);
    else make_planes<T, kPlanes, kActNone, kWindows>(q, s_sums);
}

// The last launch of a call: the parts of its products added in a fixed order, and finished, and
// the partial column sums [blocks][cols] of a bias' gradient.
struct Joins {
    Result of[2];
    const float* parts[2];   // NULL: there are none
    const float* sums;       // NULL: none
    int64_t sum_blocks, cols;
    float* sum_out;
};

// A thread has four elements, of up to 16 parts all of them, of more every kLanes-th (8, or of more
// than 128 parts 64), which the block then adds up.  (Of 16 parts a thread's loads may follow one
// another; 304 parts of 64 x 64 would take some 20 us so, and take 4 by 64 threads.)
template <typename T, int kLanes>
__device__ __forceinline__ void join_parts(const Result& q, const float* __restrict__ part,
                                           float4* s_sum) {
    constexpr int kPer = 256 / kLanes;   // fours of elements of a block
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
                s_sum[(threadIdx.x >> 5) * kPer + mine] = make_float4(z[0], z[1], z[2], z[3]);
            __syncthreads();
            if (from > 0) continue;
            for (int e = 0; e < 4; ++e) z[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const float4 u = s_sum[w * kPer + mine];
                z[0] += u.x; z[1] += u.y; z[2] += u.z; z[3] += u.w;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) finish1<T>(q, plus(z[e], q.bias ? q.bias[(at + e) % q.n] : 0.0f), at + e);
    }
}

// Eight columns of sums a block, 32 threads to each.
__device__ __forceinline__ void join_sums(const Joins& q, float (*s)[33]) {
    const int c = threadIdx.x & 7, from = threadIdx.x >> 3;
    for (int64_t c0 = (int64_t)blockIdx.x * 8; c0 < q.cols; c0 += (int64_t)gridDim.x * 8) {
        float v = 0.0f;
        if (c0 + c < q.cols)
#pragma unroll 4
            for (int64_t b = from; b < q.sum_blocks; b += 32) v += q.sums[b * q.cols + c0 + c];
        __syncthreads();
        s[c][from] = v;
        __syncthreads();
        v = s[threadIdx.x >> 5][threadIdx.x & 31];   // a warp per column
#pragma unroll
        for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
        const int64_t col = c0 + (threadIdx.x >> 5);
        if ((threadIdx.x & 31) == 0 && col < q.cols) q.sum_out[col] = v;
    }
}

__host__ __device__ inline int lanes_of(int splits) { return splits <= 16 ? 1 : splits <= 128 ? 8 : 64; }

template <typename T>
__global__ void __launch_bounds__(256)
k_linear_joins(const __grid_constant__ Joins q) {
    __shared__ float4 s_sum[8 * 32];
    __shared__ float s_cols[8][33];
    pdl_begin();
    if (blockIdx.y == 2) {
        if (q.sums) join_sums(q, s_cols);
    } else if (q.parts[blockIdx.y]) {
        const Result& r = q.of[blockIdx.y];
        const int lanes = lanes_of(r.splits);
        if (lanes == 64) join_parts<T, 64>(r, q.parts[blockIdx.y], s_sum);
        else if (lanes == 8) join_parts<T, 8>(r, q.parts[blockIdx.y], s_sum);
        else join_parts<T, 1>(r, q.parts[blockIdx.y], s_sum);
    }
}

// -------------------------------------------------------------- few rows --
// Up to kFewRows rows are bound by reading the weights once: the products are
// taken in 32 bits, `per` warps to an output, their lanes along the inputs: so
// many that a lane has up to eight vectors of the weights to take, four of them
// in flight (a row of 4096 into 2048 outputs in 16 bits: 5.1 us in a chain of
// launches, 2.5 by the bytes; one warp to an output, which leaves the SMs one or
// two blocks each, 5.8, and with four rows 10.3 instead of 6.9).

template <typename T, int V, int kRows>
__global__ void __launch_bounds__(256)
k_linear_rows(const T* __restrict__ x, const T* __restrict__ weight, int64_t k, int per,
              const __grid_constant__ Result q) {
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

// ------------------------------------------------------------------ plans --
size_t plane_size(int64_t rows, int64_t cols) { return (size_t)rows * round8(cols); }

// Blocks of rows of k_linear_operands: about eight blocks per SM over the whole matrix.
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

// The workspace of both calls of a layer of these sizes, whatever its tensors' alignment: operands
// only where a call may take the products, whose own matrices are operands as they lie in 16 bits
// where that allows it.  (The forms for few rows and narrow layers, forward, have none, those for
// few outputs and narrow layers, backward, the parts of their sums.)
struct Space {
    __nv_bfloat16 *x, *w, *dz;
    float *sums, *parts, *parts_w;   // parts: of the outputs or dx, of dW
    size_t bytes;
};
template <typename T>
Space carve(void* ws, int64_t m, int64_t k, int64_t n) {
    constexpr int kPlanes = sizeof(T) == 4 ? kMaxPlanes : 1;
    const bool few = is_few(k, n), narrow = is_narrow<T>(k, n);
    const bool back = !few && !narrow;
    // (of few outputs the products take x as it lies)
    const bool products = m > kFewRows && !is_stream<T>(k, n);   // of the forward call
    const bool wide_few = products && few && sizeof(T) == 2, wide = products && !few;
    const auto larger = [](size_t a, size_t b) { return a > b ? a : b; };
    Carve c{static_cast<unsigned char*>(ws)};
    Space s;
    s.x = c.take<__nv_bfloat16>(back || wide ? kPlanes * plane_size(m, k) : 0);
    s.w = c.take<__nv_bfloat16>(back || wide || wide_few ? kPlanes * plane_size(n, k) : 0);
    s.dz = c.take<__nv_bfloat16>(back ? kPlanes * plane_size(m, n) : 0);
    const int64_t blocks = few ? few_parts(m, kMostSms)
                           : narrow ? kMostSms : operand_grid(m, n).blocks;
    s.sums = c.take<float>((size_t)blocks * n);
    size_t parts = wide || wide_few ? product_parts(kPlanes, m, n, k) : 0, parts_w;
    if (back) {
        parts = larger(parts, product_parts(kPlanes, m, k, n));
        parts_w = product_parts(kPlanes, n, k, m);
    } else {
        parts_w = (size_t)(few ? few_parts(m, kMostSms) : narrow_parts<T>(m, kMostSms)) *
                  part_size(n, k);
    }
    s.parts = c.take<float>(parts);
    s.parts_w = c.take<float>(parts_w);
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
        bool vec = true;
        for (int i = 0; i < count; ++i) vec &= all.of[i].vec;
        const auto pick = [&](auto windows) {
            constexpr bool kWindows = decltype(windows)::value;
            return act == kActSilu   ? k_linear_operands<T, kPlanes, kActSilu, kWindows>
                   : act == kActRelu ? k_linear_operands<T, kPlanes, kActRelu, kWindows>
                                     : k_linear_operands<T, kPlanes, kActNone, kWindows>;
        };
        return launch_pdl(vec ? pick(std::false_type()) : pick(std::true_type()), grid, dim3(256),
                          0, s, all);
    }
};

template <typename T>
cudaError_t launch_joins(const Joins& q, int n_sms, cudaStream_t s) {
    int64_t blocks = 0;
    for (int i = 0; i < 2; ++i) {
        if (!q.parts[i]) continue;
        const Result& r = q.of[i];
        const int64_t b = ceil_div(ceil_div(r.m * r.n, 4), 256 / lanes_of(r.splits));
        if (b > blocks) blocks = b;
    }
    if (q.sums && ceil_div(q.cols, 8) > blocks) blocks = ceil_div(q.cols, 8);
    if (blocks == 0) return cudaSuccess;
    return launch_pdl(k_linear_joins<T>,
                      dim3((unsigned)(blocks < n_sms * 8 ? blocks : n_sms * 8), q.sums ? 3 : 2),
                      dim3(256), 0, s, q);
}

template <typename T, int V>
cudaError_t few_rows(const LinearCall& c, const Result& q, cudaStream_t s) {
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

template <typename T>
cudaError_t forward(const LinearCall& c, LearnState* st, void* ws, int n_sms, cudaStream_t s) {
    const int64_t m = c.rows, k = c.inputs, n = c.outputs;
    if (m == 0) return cudaSuccess;
    Result q{};
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
    cudaError_t e = cudaSuccess;
    if (launch_few<T>(c, q, n_sms, s, &e)) return e;
    if (launch_stream<T>(c, q, st, n_sms, s, &e)) return e;
    const Space sp = carve<T>(ws, m, k, n);
    Maker<T> make;
    const Matrix x = make.add(c.x, nullptr, kActNone, m, k, sp.x, nullptr);
    const Matrix w = make.add(c.weight, nullptr, kActNone, n, k, sp.w, nullptr);
    e = make.launch(s);
    if (e != cudaSuccess) return e;
    Joins joins{};
    e = launch_product<T>(q, x, false, w, false, k, sp.parts, &joins.of[0], st, n_sms, s);
    if (e != cudaSuccess || joins.of[0].splits <= 1) return e;
    joins.parts[0] = sp.parts;
    return launch_joins<T>(joins, n_sms, s);
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
    const Space sp = carve<T>(ws, m, k, n);
    Joins joins{};
    joins.sums = c.grad_bias ? sp.sums : nullptr;
    joins.sum_blocks = operand_grid(m, n).blocks;
    joins.cols = n;
    joins.sum_out = c.grad_bias;
    Result dx{}, dw{};
    dx.m = m;
    dw.m = n;
    dx.n = dw.n = k;
    dx.out = c.grad_x;
    dw.out = c.grad_weight;
    dx.vec = vec4<T>(dx);
    dw.vec = vec4<T>(dw);
    if (is_few(k, n)) {
        int64_t blocks = 0;
        const cudaError_t e = launch_few_back<T>(c, c.grad_weight ? sp.parts_w : nullptr,
                                                 c.grad_bias ? sp.sums : nullptr, n_sms, s, &blocks);
        if (e != cudaSuccess) return e;
        joins.sum_blocks = blocks;
        if (c.grad_weight) {
            joins.of[1] = dw;
            joins.of[1].splits = (int)blocks;
            joins.of[1].part = part_size(n, k);
            joins.parts[1] = sp.parts_w;
        }
        return launch_joins<T>(joins, n_sms, s);
    }
    if (is_narrow<T>(k, n)) {
        const cudaError_t e = launch_narrow<T>(c, sp.parts_w, c.grad_bias ? sp.sums : nullptr, st,
                                               n_sms, s);
        if (e != cudaSuccess) return e;
        const int64_t tiles = ceil_div(m, kBlock);
        joins.sum_blocks = tiles < n_sms ? tiles : n_sms;
        if (c.grad_weight) {
            joins.of[1] = dw;
            joins.of[1].splits = narrow_parts<T>(m, n_sms);
            joins.of[1].part = part_size(n, k);
            joins.parts[1] = sp.parts_w;
        }
        return launch_joins<T>(joins, n_sms, s);
    }
    Maker<T> make;
    const Matrix dz = make.add(c.grad_y, c.act == kActNone ? nullptr : c.pre, c.act, m, n,
                               c.grad_x || c.grad_weight ? sp.dz : nullptr,
                               c.grad_bias ? sp.sums : nullptr);
    const Matrix w = make.add(c.weight, nullptr, kActNone, n, k, c.grad_x ? sp.w : nullptr, nullptr);
    const Matrix x = make.add(c.x, nullptr, kActNone, m, k, c.grad_weight ? sp.x : nullptr, nullptr);
    cudaError_t e = make.launch(s);
    if (e == cudaSuccess && c.grad_x)
        e = launch_product<T>(dx, dz, false, w, true, n, sp.parts, &joins.of[0], st, n_sms, s);
    if (e == cudaSuccess && c.grad_weight)
        e = launch_product<T>(dw, dz, true, x, true, m, sp.parts_w, &joins.of[1], st, n_sms, s);
    if (e != cudaSuccess) return e;
    joins.parts[0] = joins.of[0].splits > 1 ? sp.parts : nullptr;
    joins.parts[1] = joins.of[1].splits > 1 ? sp.parts_w : nullptr;
    return launch_joins<T>(joins, n_sms, s);
}

}  // namespace

size_t linear_forward_workspace(int64_t rows, int64_t inputs, int64_t outputs, int dtype) {
    return rows <= linear::kFewRows ? 0 : linear_workspace(rows, inputs, outputs, dtype);
}
size_t linear_workspace(int64_t rows, int64_t inputs, int64_t outputs, int dtype) {
    return dtype == kF32 ? carve<float>(nullptr, rows, inputs, outputs).bytes
                         : carve<__nv_bfloat16>(nullptr, rows, inputs, outputs).bytes;
}

cudaError_t prepare_linear() {
    const cudaError_t e = linear::prepare_product();
    return e == cudaSuccess ? linear::prepare_narrow() : e;
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
