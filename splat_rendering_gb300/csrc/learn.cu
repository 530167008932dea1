// C ABI of the learned parts around the renderer: a handle with one block of
// workspace and a latched device error, and the embedding, group-norm, linear,
// dropout and orthogonalisation calls on it.  As with the renderer's calls, arguments are
// checked on the host before anything is enqueued, and nothing synchronises
// but pulsar_learn_status.
#include <cmath>
#include <new>

#include "../../include/pulsar.h"
#include "learn_internal.cuh"
#include "host_util.cuh"

using namespace pulsar;

struct pulsar_learn {
    int device = 0, n_sms = 1;
    int64_t bytes = 0;
    unsigned char* ws = nullptr;
    LearnState* state = nullptr;        // device
    LearnState* host_state = nullptr;   // pinned mirror for pulsar_learn_status
};

namespace {

constexpr int64_t kMaxIndex = 0x7fff0000LL;   // positions and rows are 32-bit on the device
constexpr int kMaxSms = 160;                  // of an sm_103a part (launches size workspace by it)
constexpr int64_t kMaxDim = 65536;
constexpr int64_t kMaxSide = 65536;           // of a matrix
constexpr int64_t kMaxElements = 1LL << 38;   // of a matrix of rows: strides of its maps, tiles
constexpr int64_t kMaxBatch = 65535;          // a launch's grid

bool valid_type(int t) { return t == PULSAR_F32 || t == PULSAR_BF16; }
bool aligned_to(const void* p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == PULSAR_BF16 ? 1u : 3u)) == 0;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool finite(float v) { return v - v == 0.0f; }

bool embed_sizes(int64_t n, int64_t rows, int64_t dim) {
    return n >= 0 && n <= kMaxIndex && rows >= 1 && rows <= kMaxIndex && dim >= 1 && dim <= kMaxDim;
}
bool norm_sizes(int64_t images, int64_t pixels, int32_t channels, int32_t groups) {
    return images >= 0 && images <= kMaxBatch && pixels >= 0 && pixels <= (1LL << 40) &&
           channels >= 1 && channels <= 4096 && groups >= 1 && channels % groups == 0;
}
bool orth_sizes(int64_t batch, int64_t m, int64_t n) {
    return batch >= 0 && batch <= kMaxBatch && m >= 0 && m <= kMaxSide && n >= 0 && n <= kMaxSide;
}
bool linear_sizes(int64_t rows, int64_t inputs, int64_t outputs) {
    return rows >= 0 && rows <= kMaxIndex && inputs >= 1 && inputs <= kMaxSide && outputs >= 1 &&
           outputs <= kMaxSide && rows * inputs <= kMaxElements && rows * outputs <= kMaxElements;
}
bool valid_act(int a) { return a == PULSAR_ACT_NONE || a == PULSAR_ACT_SILU || a == PULSAR_ACT_RELU; }
// Tensors as ranges of bytes, and whether two of them share some.
struct Range {
    const void* p;
    int64_t bytes;
};
bool overlap(const Range& a, const Range& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x && y && a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes &&
           y < x + (uintptr_t)a.bytes;
}
int64_t bytes_of(int64_t count, int dtype) { return count * (dtype == PULSAR_BF16 ? 2 : 4); }

bool embed_args(const void* src, const void* tokens, int64_t n, float scale, int dtype, int index,
                const void* dst) {
    if (!valid_type(dtype) || (index != PULSAR_I32 && index != PULSAR_I64) || !finite(scale))
        return false;
    return aligned_to(src, dtype) && aligned_to(dst, dtype) &&
           (reinterpret_cast<uintptr_t>(tokens) & (index == PULSAR_I64 ? 7u : 3u)) == 0 &&
           (n == 0 || (src && tokens));
}

}  // namespace

extern "C" {

int pulsar_learn_create(pulsar_learn_t* out, int device, int64_t workspace_bytes) {
    PULSAR_TRACE("pulsar_learn_create");
    if (!out) return PULSAR_ERR_ARG;
    *out = nullptr;
    if (workspace_bytes < 0) return PULSAR_ERR_ARG;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess) return PULSAR_ERR_CUDA;
    if (device < 0 || device >= ndev) return PULSAR_ERR_ARG;
    DeviceGuard guard(device);
    pulsar_learn* h = new (std::nothrow) pulsar_learn();
    if (!h) return PULSAR_ERR_NOMEM;
    h->device = device;
    h->bytes = workspace_bytes;
    bool ok = cudaMalloc(reinterpret_cast<void**>(&h->ws),
                         workspace_bytes > 0 ? (size_t)workspace_bytes : 256) == cudaSuccess;
    if (ok) ok = cudaMalloc(reinterpret_cast<void**>(&h->state), sizeof(LearnState)) == cudaSuccess;
    if (ok)
        ok = cudaMallocHost(reinterpret_cast<void**>(&h->host_state), sizeof(LearnState)) ==
             cudaSuccess;
    if (ok)
        ok = cudaDeviceGetAttribute(&h->n_sms, cudaDevAttrMultiProcessorCount, device) ==
                 cudaSuccess &&
             h->n_sms <= kMaxSms && prepare_orth() == cudaSuccess &&
             prepare_group_norm() == cudaSuccess && prepare_embed() == cudaSuccess &&
             prepare_linear() == cudaSuccess && cudaMemset(h->state, 0, sizeof(LearnState)) == cudaSuccess &&
             cudaDeviceSynchronize() == cudaSuccess;
    if (!ok) {
        cudaFree(h->ws);
        cudaFree(h->state);
        if (h->host_state) cudaFreeHost(h->host_state);
        delete h;
        cudaGetLastError();
        return PULSAR_ERR_NOMEM;
    }
    *out = h;
    return PULSAR_OK;
}

int pulsar_learn_destroy(pulsar_learn_t h) {
    PULSAR_TRACE("pulsar_learn_destroy");
    if (!h) return PULSAR_ERR_ARG;
    DeviceGuard guard(h->device);
    cudaDeviceSynchronize();
    cudaFree(h->ws);
    cudaFree(h->state);
    cudaFreeHost(h->host_state);
    delete h;
    return PULSAR_OK;
}

int pulsar_learn_status(pulsar_learn_t h, void* stream) {
    PULSAR_TRACE("pulsar_learn_status");
    if (!h) return PULSAR_ERR_ARG;
    DeviceGuard guard(h->device);
    cudaStream_t s = as_stream(stream);
    if (cudaMemcpyAsync(h->host_state, h->state, sizeof(LearnState), cudaMemcpyDeviceToHost, s) !=
            cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return PULSAR_ERR_CUDA;
    const uint32_t error = h->host_state->error;
    if (!error) return PULSAR_OK;
    if (cudaMemsetAsync(h->state, 0, sizeof(LearnState), s) != cudaSuccess) return PULSAR_ERR_CUDA;
    return error & kErrTimeout ? PULSAR_ERR_TIMEOUT : PULSAR_ERR_INDEX;
}

// -------------------------------------------------------------- embedding --
int64_t pulsar_embed_workspace(int64_t n, int64_t rows, int64_t dim) {
    if (!embed_sizes(n, rows, dim)) return PULSAR_ERR_ARG;
    return (int64_t)embed_workspace(n, rows, dim);
}

int pulsar_embed_forward(pulsar_learn_t h, const void* table, const void* tokens, int64_t n,
                         int64_t rows, int64_t dim, float scale, int dtype, int index, void* out,
                         void* stream) {
    PULSAR_TRACE("pulsar_embed_forward");
    if (!h || !embed_sizes(n, rows, dim) ||
        !embed_args(table, tokens, n, scale, dtype, index, out) || (n > 0 && !out))
        return PULSAR_ERR_ARG;
    DeviceGuard guard(h->device);
    const EmbedCall c{table, tokens, n, rows, dim, scale, dtype, index, out};
    return cuda_err(launch_embed_forward(c, h->state, as_stream(stream)));
}

int pulsar_embed_backward(pulsar_learn_t h, const void* grad_out, const void* tokens, int64_t n,
                          int64_t rows, int64_t dim, float scale, int dtype, int index,
                          void* grad_table, void* stream) {
    PULSAR_TRACE("pulsar_embed_backward");
    if (!h || !embed_sizes(n, rows, dim) ||
        !embed_args(grad_out, tokens, n, scale, dtype, index, grad_table) || !grad_table)
        return PULSAR_ERR_ARG;
    if ((int64_t)embed_workspace(n, rows, dim) > h->bytes) return PULSAR_ERR_WORKSPACE;
    DeviceGuard guard(h->device);
    const EmbedCall c{grad_out, tokens, n, rows, dim, scale, dtype, index, grad_table};
    return cuda_err(launch_embed_backward(c, h->state, h->ws, h->n_sms, as_stream(stream)));
}

// ------------------------------------------------------------- group norm --
int64_t pulsar_group_norm_workspace(int64_t images, int64_t pixels, int32_t channels,
                                    int32_t groups) {
    if (!norm_sizes(images, pixels, channels, groups)) return PULSAR_ERR_ARG;
    return (int64_t)group_norm_workspace(images, pixels, channels, groups);
}

static bool norm_args(const NormCall& c) {
    if (!norm_sizes(c.images, c.pixels, c.channels, c.groups) || !valid_type(c.dtype) ||
        (c.act != PULSAR_ACT_NONE && c.act != PULSAR_ACT_SILU && c.act != PULSAR_ACT_RELU))
        return false;
    if (c.images > 0 && !c.stats) return false;
    for (const void* p : {(const void*)c.weight, (const void*)c.bias, (const void*)c.grad_weight,
                          (const void*)c.grad_bias})
        if (!aligned4(p)) return false;
    if ((reinterpret_cast<uintptr_t>(c.stats) & 7u) != 0) return false;   // pairs
    return aligned_to(c.x, c.dtype) && aligned_to(c.grad_y, c.dtype) && aligned_to(c.out, c.dtype) &&
           (c.images == 0 || c.pixels == 0 || c.x);
}

int pulsar_group_norm_forward(pulsar_learn_t h, const void* x, int64_t images, int64_t pixels,
                              int32_t channels, int32_t groups, const float* weight,
                              const float* bias, float eps, int act, int dtype, void* y,
                              float* stats, void* stream) {
    PULSAR_TRACE("pulsar_group_norm_forward");
    const NormCall c{x, nullptr, weight, bias, images, pixels, channels, groups,
                     eps, act, dtype, y, stats, nullptr, nullptr};
    if (!h || !norm_args(c) || !(eps >= 0.0f) || !finite(eps) ||
        (images > 0 && pixels > 0 && !y))
        return PULSAR_ERR_ARG;
    if ((int64_t)group_norm_workspace(images, pixels, channels, groups) > h->bytes)
        return PULSAR_ERR_WORKSPACE;
    DeviceGuard guard(h->device);
    return cuda_err(launch_group_norm_forward(c, h->ws, h->n_sms, as_stream(stream)));
}

int pulsar_group_norm_backward(pulsar_learn_t h, const void* grad_y, const void* x,
                               const float* stats, int64_t images, int64_t pixels,
                               int32_t channels, int32_t groups, const float* weight,
                               const float* bias, int act, int dtype, void* grad_x,
                               float* grad_weight, float* grad_bias, void* stream) {
    PULSAR_TRACE("pulsar_group_norm_backward");
    const NormCall c{x, grad_y, weight, bias, images, pixels, channels, groups,
                     0.0f, act, dtype, grad_x, const_cast<float*>(stats), grad_weight, grad_bias};
    if (!h || !norm_args(c) || (images > 0 && pixels > 0 && !grad_y)) return PULSAR_ERR_ARG;
    if (!grad_x && !grad_weight && !grad_bias) return PULSAR_OK;   // nothing requested
    if ((int64_t)group_norm_workspace(images, pixels, channels, groups) > h->bytes)
        return PULSAR_ERR_WORKSPACE;
    DeviceGuard guard(h->device);
    return cuda_err(launch_group_norm_backward(c, h->ws, h->n_sms, as_stream(stream)));
}

// ------------------------------------------------------ orthogonalisation --
int64_t pulsar_orthogonalize_workspace(int64_t batch, int64_t m, int64_t n, int dtype) {
    if (!orth_sizes(batch, m, n) || !valid_type(dtype)) return PULSAR_ERR_ARG;
    return (int64_t)orth_workspace(batch, m, n, dtype);
}

int pulsar_orthogonalize(pulsar_learn_t h, const void* grad, int64_t batch, int64_t m, int64_t n,
                         int steps, const float* coeffs, float eps, int dtype, void* out,
                         void* stream) {
    PULSAR_TRACE("pulsar_orthogonalize");
    if (!h || !orth_sizes(batch, m, n) || !valid_type(dtype) || !coeffs || steps < 0 ||
        steps > 100 || !(eps >= 0.0f) || !finite(eps) || !finite(coeffs[0]) ||
        !finite(coeffs[1]) || !finite(coeffs[2]) || !aligned_to(grad, dtype) ||
        !aligned_to(out, dtype) || !orth_in_range(steps, coeffs[0], coeffs[1], coeffs[2]))
        return PULSAR_ERR_ARG;
    if (batch > 0 && m > 0 && n > 0 && (!grad || !out)) return PULSAR_ERR_ARG;
    if ((int64_t)orth_workspace(batch, m, n, dtype) > h->bytes) return PULSAR_ERR_WORKSPACE;
    DeviceGuard guard(h->device);
    const OrthCall c{grad, batch, m, n, steps, coeffs[0], coeffs[1], coeffs[2], eps, dtype, out};
    return cuda_err(launch_orth(c, h->state, h->ws, h->n_sms, as_stream(stream)));
}

// ------------------------------------------------------------ linear layer --
int64_t pulsar_linear_workspace(int64_t rows, int64_t inputs, int64_t outputs, int dtype) {
    if (!linear_sizes(rows, inputs, outputs) || !valid_type(dtype)) return PULSAR_ERR_ARG;
    return (int64_t)linear_workspace(rows, inputs, outputs, dtype);
}

static bool linear_args(const LinearCall& c) {
    if (!linear_sizes(c.rows, c.inputs, c.outputs) || !valid_type(c.dtype) || !valid_act(c.act))
        return false;
    // no output may share memory with an input that is still read, or with another output
    const int64_t x_bytes = bytes_of(c.rows * c.inputs, c.dtype);
    const int64_t y_bytes = bytes_of(c.rows * c.outputs, c.dtype);
    const int64_t w_bytes = bytes_of(c.outputs * c.inputs, c.dtype), b_bytes = 4 * c.outputs;
    const Range in[] = {{c.x, x_bytes},        {c.weight, w_bytes}, {c.bias, b_bytes},
                        {c.residual, y_bytes}, {c.grad_y, y_bytes}, {c.grad_y ? c.pre : nullptr, y_bytes}};
    const Range out[] = {{c.out, y_bytes},    {c.grad_y ? nullptr : c.pre, y_bytes},
                         {c.grad_x, x_bytes}, {c.grad_weight, w_bytes},
                         {c.grad_bias, b_bytes}};
    for (const Range& o : out) {
        for (const Range& i : in)
            if (overlap(o, i) && !(&o == &out[0] && &i == &in[3] && o.p == i.p)) return false;
        for (const Range& other : out)
            if (&other != &o && overlap(o, other)) return false;
    }
    for (const void* p : {c.x, c.weight, (const void*)c.pre, (const void*)c.out, c.residual,
                          c.grad_y, (const void*)c.grad_x, (const void*)c.grad_weight})
        if (!aligned_to(p, c.dtype)) return false;
    return aligned4(c.bias) && aligned4(c.grad_bias);
}

int pulsar_linear_forward(pulsar_learn_t h, const void* x, const void* weight, int64_t rows,
                          int64_t inputs, int64_t outputs, const float* bias,
                          const void* residual, int act, int dtype, void* y, void* pre,
                          void* stream) {
    PULSAR_TRACE("pulsar_linear_forward");
    const LinearCall c{x, weight, rows, inputs, outputs, act, dtype, pre, y, bias, residual,
                       nullptr, nullptr, nullptr, nullptr};
    if (!h || !linear_args(c) || (rows > 0 && (!x || !weight || !y))) return PULSAR_ERR_ARG;
    if ((int64_t)linear_forward_workspace(rows, inputs, outputs, dtype) > h->bytes)
        return PULSAR_ERR_WORKSPACE;
    DeviceGuard guard(h->device);
    return cuda_err(launch_linear_forward(c, h->state, h->ws, h->n_sms, as_stream(stream)));
}

int pulsar_linear_backward(pulsar_learn_t h, const void* grad_y, const void* x,
                           const void* weight, const void* pre, int64_t rows, int64_t inputs,
                           int64_t outputs, int act, int dtype, void* grad_x, void* grad_weight,
                           float* grad_bias, void* stream) {
    PULSAR_TRACE("pulsar_linear_backward");
    const LinearCall c{x, weight, rows, inputs, outputs, act, dtype, const_cast<void*>(pre),
                       nullptr, nullptr, nullptr, grad_y, grad_x, grad_weight, grad_bias};
    if (!h || !linear_args(c)) return PULSAR_ERR_ARG;
    if (!grad_x && !grad_weight && !grad_bias) return PULSAR_OK;   // nothing requested
    if (rows > 0 && (!grad_y || (act != PULSAR_ACT_NONE && !pre) || (grad_x && !weight) ||
                     (grad_weight && !x)))
        return PULSAR_ERR_ARG;
    if ((int64_t)linear_workspace(rows, inputs, outputs, dtype) > h->bytes)
        return PULSAR_ERR_WORKSPACE;
    DeviceGuard guard(h->device);
    return cuda_err(launch_linear_backward(c, h->state, h->ws, h->n_sms, as_stream(stream)));
}

// ---------------------------------------------------------------- dropout --
int pulsar_dropout(pulsar_learn_t h, const void* x, const void* residual, int64_t n, double p,
                   uint64_t seed, int64_t offset, const int64_t* counter, int dtype, void* out,
                   void* stream) {
    PULSAR_TRACE("pulsar_dropout");
    if (!h || n < 0 || n > kMaxElements || !valid_type(dtype) || !(p >= 0.0 && p < 1.0) ||
        offset < 0 || !aligned_to(x, dtype) || !aligned_to(residual, dtype) ||
        !aligned_to(out, dtype) || (reinterpret_cast<uintptr_t>(counter) & 7u) != 0 ||
        (n > 0 && (!x || !out)))
        return PULSAR_ERR_ARG;
    const Range result{out, bytes_of(n, dtype)};
    if ((out != x && overlap(result, Range{x, result.bytes})) ||
        (out != residual && overlap(result, Range{residual, result.bytes})) ||
        overlap(result, Range{counter, 8}))
        return PULSAR_ERR_ARG;
    const double least = std::nearbyint(p * 4294967296.0);
    if (least > 4294967295.0) return PULSAR_ERR_ARG;   // nothing would be kept
    DeviceGuard guard(h->device);
    const DropoutCall c{x, residual, n, seed, offset, counter, (uint32_t)least,
                        (float)(1.0 / (1.0 - p)), dtype, out};
    return cuda_err(launch_dropout(c, h->n_sms, as_stream(stream)));
}

}  // extern "C"
