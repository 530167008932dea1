// C ABI of the learned parts around the renderer: a handle with one block of
// workspace and a latched device error, and the embedding, group-norm and
// orthogonalisation calls on it.  As with the renderer's calls, arguments are
// checked on the host before anything is enqueued, and nothing synchronises
// but pulsar_learn_status.
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
             cudaMemset(h->state, 0, sizeof(LearnState)) == cudaSuccess &&
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

}  // extern "C"
