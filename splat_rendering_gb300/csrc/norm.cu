// Group normalisation of channels-last feature images with an activation,
// forward and backward.  x is [images, pixels, C], a group is C / G adjacent
// channels of one image:
//
//   h = (x - mean_g) rstd_g,  z = w_c h + b_c,  y = act(z)
//   dz = dy act'(z),  db_c = sum dz,  dw_c = sum dz h,  dh = w_c dz,
//   dx = rstd_g (dh - mean_g(dh) - h mean_g(dh h))
//
// A block owns a run of pixels of one image; its threads lie along the
// channels in 16-byte vectors and walk the pixels, so every access is
// coalesced and a thread's channels (its weights, its sums) never change.
//
// Statistics: a thread sums x - k and (x - k)^2 with k its own first value,
// which bounds the cancellation of the second moment by the number of its
// pixels whatever the mean, and turns them into (mean, M2); parts are joined
// by sum(M2) + sum(n (mean - common mean)^2), in 32 bits and a fixed order.
#include "learn_internal.cuh"

namespace pulsar {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxNormChannels = 4096;
constexpr int kMaxChunks = 1024;   // pixel chunks per image

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// How the threads lie on an image's rows of C channels.
struct Shape {
    int64_t pixels;
    int channels, groups, cpg;   // cpg = channels / groups
    int cols;                    // vectors per pixel
    int rpb;                     // pixels a block covers at once (cols <= kThreads), else 1
    int chunks;                  // blocks per image
    int64_t chunk;               // pixels per block
};

__device__ __forceinline__ int rows_of(int64_t len, int row, int rpb) {
    return len > row ? (int)((len - row + rpb - 1) / rpb) : 0;
}

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

__device__ __forceinline__ float activate(float z, int act) {
    if (act == kActSilu) return z * sigmoid(z);
    if (act == kActRelu) return z > 0.0f || z != z ? z : 0.0f;   // NaN stays NaN
    return z;
}
__device__ __forceinline__ float activate_grad(float z, float dy, int act) {
    if (act == kActSilu) {
        const float s = sigmoid(z);
        return dy * (s * fmaf(z, 1.0f - s, 1.0f));
    }
    if (act == kActRelu) return z > 0.0f ? dy : 0.0f;
    return dy;
}

// ------------------------------------------------------------ statistics --
// part[image][chunk][group] = (mean, M2) of the chunk's values.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
k_norm_stats(const T* __restrict__ x, Shape sh, float2* __restrict__ part) {
    pdl_begin();
    // one entry per thread and channel (or per vector, where a vector stays in a group)
    __shared__ float s_mean[kMaxNormChannels], s_m2[kMaxNormChannels];
    const bool whole = sh.cpg % V == 0;
    const int sub = whole ? 1 : V;               // entries per vector
    const int epr = sh.cols * sub, eg = epr / sh.groups;
    const int64_t p0 = blockIdx.x * sh.chunk;
    const int64_t len = min(sh.chunk, sh.pixels - p0);
    const T* base = x + ((int64_t)blockIdx.y * sh.pixels + p0) * sh.channels;
    const int row = sh.rpb > 1 ? (int)threadIdx.x / sh.cols : 0;
    const int cnt = rows_of(len, row, sh.rpb);
    for (int col = threadIdx.x - row * sh.cols; col < sh.cols && row < sh.rpb; col += kThreads) {
        float k[V], s[V], q[V];
        if (cnt > 0) Pack<T, V>::load(base + (int64_t)row * sh.channels + col * V, k);
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = q[j] = 0.0f;
#pragma unroll 4
        for (int i = 0; i < cnt; ++i) {
            float v[V];
            Pack<T, V>::load(base + (row + (int64_t)i * sh.rpb) * sh.channels + col * V, v);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = v[j] - k[j];
                s[j] += d;
                q[j] = fmaf(d, d, q[j]);
            }
        }
        const float inv = cnt > 0 ? 1.0f / (float)cnt : 0.0f;
        float mean[V], m2[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            mean[j] = cnt > 0 ? fmaf(s[j], inv, k[j]) : 0.0f;
            m2[j] = fmaxf(fmaf(-s[j] * inv, s[j], q[j]), 0.0f);
            if (q[j] != q[j]) m2[j] = q[j];   // fmaxf drops a NaN
        }
        const int e = row * epr + col * sub;
        if (whole) {
            float m = 0.0f, t = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) m += mean[j];
            m *= 1.0f / V;
#pragma unroll
            for (int j = 0; j < V; ++j) t += fmaf((float)cnt * (mean[j] - m), mean[j] - m, m2[j]);
            s_mean[e] = m;
            s_m2[e] = t;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s_mean[e + j] = mean[j];
                s_m2[e + j] = m2[j];
            }
        }
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const float per = (float)(V / sub);   // channels per entry
    const float inv_all = 1.0f / ((float)len * (float)sh.cpg);
    for (int g = threadIdx.x >> 5; g < sh.groups; g += kThreads / 32) {
        const int n_e = sh.rpb * eg;
        float m = 0.0f;
        for (int e = lane; e < n_e; e += 32) {
            const int r = e / eg, at = r * epr + g * eg + (e - r * eg);
            const int c = rows_of(len, r, sh.rpb);
            if (c > 0) m = fmaf((float)c * per, s_mean[at], m);
        }
        m = warp_sum(m) * inv_all;
        float t = 0.0f;
        for (int e = lane; e < n_e; e += 32) {
            const int r = e / eg, at = r * epr + g * eg + (e - r * eg);
            const int c = rows_of(len, r, sh.rpb);
            const float d = s_mean[at] - m;
            if (c > 0) t += fmaf((float)c * per * d, d, s_m2[at]);
        }
        t = warp_sum(t);
        if (lane == 0)
            part[((size_t)blockIdx.y * sh.chunks + blockIdx.x) * sh.groups + g] = make_float2(m, t);
    }
}

// stats[image][group] = (mean, rstd) from the chunks: a warp per group.
__global__ void __launch_bounds__(kThreads)
k_norm_finish(const float2* __restrict__ part, Shape sh, float eps, float2* __restrict__ stats) {
    pdl_begin();
    const int lane = threadIdx.x & 31;
    const int g = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (g >= sh.groups) return;
    const float2* p = part + (size_t)blockIdx.y * sh.chunks * sh.groups + g;
    const float inv_pix = 1.0f / (float)sh.pixels;   // (no chunk reads it where there is no pixel)
    float m = 0.0f;
    for (int c = lane; c < sh.chunks; c += 32) {
        const float len = (float)min(sh.chunk, sh.pixels - c * sh.chunk);
        m = fmaf(len * inv_pix, p[(size_t)c * sh.groups].x, m);
    }
    m = warp_sum(m);
    float t = 0.0f;
    for (int c = lane; c < sh.chunks; c += 32) {
        const float len = (float)min(sh.chunk, sh.pixels - c * sh.chunk);
        const float2 u = p[(size_t)c * sh.groups];
        const float d = u.x - m;
        t += fmaf(len * (float)sh.cpg * d, d, u.y);
    }
    t = warp_sum(t);
    if (lane == 0) {
        const float var = sh.pixels > 0 ? t / ((float)sh.pixels * (float)sh.cpg) : 0.0f;
        stats[(size_t)blockIdx.y * sh.groups + g] = make_float2(m, 1.0f / sqrtf(var + eps));
    }
}

// ----------------------------------------------------------------- apply --
// What a thread's V channels need: the mean, rstd w and b.
template <int V>
struct Affine {
    float mean[V], rstd[V], w[V], b[V];
    __device__ __forceinline__ void load(const float2* stats, const float* weight,
                                         const float* bias, int c0, int cpg) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 s = stats[(c0 + j) / cpg];
            mean[j] = s.x;
            rstd[j] = s.y;
            w[j] = weight ? weight[c0 + j] : 1.0f;
            b[j] = bias ? bias[c0 + j] : 0.0f;
        }
    }
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
k_norm_apply(const T* __restrict__ x, Shape sh, const float2* __restrict__ stats,
             const float* __restrict__ weight, const float* __restrict__ bias, int act,
             T* __restrict__ y) {
    pdl_begin();
    const int64_t p0 = blockIdx.x * sh.chunk;
    const int64_t len = min(sh.chunk, sh.pixels - p0);
    const int64_t off = ((int64_t)blockIdx.y * sh.pixels + p0) * sh.channels;
    const int row = sh.rpb > 1 ? (int)threadIdx.x / sh.cols : 0;
    const int cnt = rows_of(len, row, sh.rpb);
    for (int col = threadIdx.x - row * sh.cols; col < sh.cols && row < sh.rpb; col += kThreads) {
        Affine<V> f;
        f.load(stats + (size_t)blockIdx.y * sh.groups, weight, bias, col * V, sh.cpg);
#pragma unroll
        for (int j = 0; j < V; ++j) f.rstd[j] *= f.w[j];
#pragma unroll 4
        for (int i = 0; i < cnt; ++i) {
            const int64_t at = off + (row + (int64_t)i * sh.rpb) * sh.channels + col * V;
            float v[V];
            Pack<T, V>::load(x + at, v);
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[j] = activate(fmaf(v[j] - f.mean[j], f.rstd[j], f.b[j]), act);
            Pack<T, V>::store(y + at, v);
        }
    }
}

// -------------------------------------------------------------- backward --
// part[image][chunk][channel] = (sum dz, sum dz h) over the chunk's pixels.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
k_norm_back_sums(const T* __restrict__ x, const T* __restrict__ dy, Shape sh,
                 const float2* __restrict__ stats, const float* __restrict__ weight,
                 const float* __restrict__ bias, int act, float2* __restrict__ part) {
    pdl_begin();
    __shared__ float s1[kThreads * V], s2[kThreads * V];
    const int64_t p0 = blockIdx.x * sh.chunk;
    const int64_t len = min(sh.chunk, sh.pixels - p0);
    const int64_t off = ((int64_t)blockIdx.y * sh.pixels + p0) * sh.channels;
    const int row = sh.rpb > 1 ? (int)threadIdx.x / sh.cols : 0;
    const int cnt = rows_of(len, row, sh.rpb);
    float2* out = part + ((size_t)blockIdx.y * sh.chunks + blockIdx.x) * sh.channels;
    for (int col = threadIdx.x - row * sh.cols; col < sh.cols && row < sh.rpb; col += kThreads) {
        Affine<V> f;
        f.load(stats + (size_t)blockIdx.y * sh.groups, weight, bias, col * V, sh.cpg);
        float a[V], q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = q[j] = 0.0f;
#pragma unroll 2
        for (int i = 0; i < cnt; ++i) {
            const int64_t at = off + (row + (int64_t)i * sh.rpb) * sh.channels + col * V;
            float v[V], g[V];
            Pack<T, V>::load(x + at, v);
            Pack<T, V>::load(dy + at, g);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float h = (v[j] - f.mean[j]) * f.rstd[j];
                const float dz = activate_grad(fmaf(h, f.w[j], f.b[j]), g[j], act);
                a[j] += dz;
                q[j] = fmaf(dz, h, q[j]);
            }
        }
        if (sh.rpb == 1) {
#pragma unroll
            for (int j = 0; j < V; ++j) out[col * V + j] = make_float2(a[j], q[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s1[row * sh.channels + col * V + j] = a[j];
                s2[row * sh.channels + col * V + j] = q[j];
            }
        }
    }
    if (sh.rpb == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < sh.channels; c += kThreads) {
        float a = 0.0f, q = 0.0f;
        for (int r = 0; r < sh.rpb; ++r) {
            a += s1[r * sh.channels + c];
            q += s2[r * sh.channels + c];
        }
        out[c] = make_float2(a, q);
    }
}

// sums[image][channel] over the chunks: a warp per channel.
__global__ void __launch_bounds__(kThreads)
k_norm_back_chunks(const float2* __restrict__ part, Shape sh, float2* __restrict__ sums) {
    pdl_begin();
    const int lane = threadIdx.x & 31;
    const int c = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (c >= sh.channels) return;
    const float2* p = part + (size_t)blockIdx.y * sh.chunks * sh.channels + c;
    float a = 0.0f, q = 0.0f;
    for (int k = lane; k < sh.chunks; k += 32) {
        const float2 u = p[(size_t)k * sh.channels];
        a += u.x;
        q += u.y;
    }
    a = warp_sum(a);
    q = warp_sum(q);
    if (lane == 0) sums[(size_t)blockIdx.y * sh.channels + c] = make_float2(a, q);
}

// The parameters' gradients (sums over the images), and
// means[image][group] = (mean dh, mean dh h).
__global__ void __launch_bounds__(kThreads)
k_norm_back_finish(const float2* __restrict__ sums, Shape sh, int images,
                   const float* __restrict__ weight, float* __restrict__ grad_weight,
                   float* __restrict__ grad_bias, float2* __restrict__ means) {
    pdl_begin();
    const int64_t stride = (int64_t)gridDim.x * kThreads;
    for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
         e < sh.channels + (int64_t)images * sh.groups; e += stride) {
        if (e < sh.channels) {
            float a = 0.0f, q = 0.0f;
            for (int i = 0; i < images; ++i) {
                const float2 u = sums[(size_t)i * sh.channels + e];
                a += u.x;
                q += u.y;
            }
            if (grad_bias) grad_bias[e] = a;
            if (grad_weight) grad_weight[e] = q;
        } else {
            const int64_t ig = e - sh.channels;
            const int64_t image = ig / sh.groups;
            const int c0 = (int)(ig % sh.groups) * sh.cpg;
            float a = 0.0f, q = 0.0f;
            for (int c = c0; c < c0 + sh.cpg; ++c) {
                const float2 u = sums[(size_t)image * sh.channels + c];
                const float wc = weight ? weight[c] : 1.0f;
                a = fmaf(wc, u.x, a);
                q = fmaf(wc, u.y, q);
            }
            const float inv = 1.0f / ((float)sh.pixels * (float)sh.cpg);
            means[ig] = make_float2(a * inv, q * inv);
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
k_norm_back_apply(const T* __restrict__ x, const T* __restrict__ dy, Shape sh,
                  const float2* __restrict__ stats, const float2* __restrict__ means,
                  const float* __restrict__ weight, const float* __restrict__ bias, int act,
                  T* __restrict__ dx) {
    pdl_begin();
    const int64_t p0 = blockIdx.x * sh.chunk;
    const int64_t len = min(sh.chunk, sh.pixels - p0);
    const int64_t off = ((int64_t)blockIdx.y * sh.pixels + p0) * sh.channels;
    const int row = sh.rpb > 1 ? (int)threadIdx.x / sh.cols : 0;
    const int cnt = rows_of(len, row, sh.rpb);
    for (int col = threadIdx.x - row * sh.cols; col < sh.cols && row < sh.rpb; col += kThreads) {
        Affine<V> f;
        f.load(stats + (size_t)blockIdx.y * sh.groups, weight, bias, col * V, sh.cpg);
        float m1[V], m2[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 u = means[(size_t)blockIdx.y * sh.groups + (col * V + j) / sh.cpg];
            m1[j] = u.x;
            m2[j] = u.y;
        }
#pragma unroll 2
        for (int i = 0; i < cnt; ++i) {
            const int64_t at = off + (row + (int64_t)i * sh.rpb) * sh.channels + col * V;
            float v[V], g[V];
            Pack<T, V>::load(x + at, v);
            Pack<T, V>::load(dy + at, g);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float h = (v[j] - f.mean[j]) * f.rstd[j];
                const float dz = activate_grad(fmaf(h, f.w[j], f.b[j]), g[j], act);
                v[j] = f.rstd[j] * (fmaf(dz, f.w[j], -m1[j]) - h * m2[j]);
            }
            Pack<T, V>::store(dx + at, v);
        }
    }
}

// ----------------------------------------------------------------- plans --
Shape shape_of(int64_t images, int64_t pixels, int channels, int groups, int v) {
    Shape s;
    s.pixels = pixels;
    s.channels = channels;
    s.groups = groups;
    s.cpg = channels / groups;
    s.cols = channels / v;
    s.rpb = s.cols < kThreads ? kThreads / s.cols : 1;
    // about 1216 blocks (eight per SM) over the images, none with less than
    // eight pixels per thread
    int64_t per = ceil_div(images * pixels, 1216);
    const int64_t least = (int64_t)s.rpb * 8;
    per = ceil_div(per < least ? least : per, s.rpb) * s.rpb;
    if (ceil_div(pixels, per) > kMaxChunks) per = ceil_div(ceil_div(pixels, kMaxChunks), s.rpb) * s.rpb;
    s.chunk = per;
    s.chunks = (int)ceil_div(pixels, per);
    return s;
}

struct Space {
    float2 *part, *sums, *means;
};
Space carve(Carve& w, int64_t images, int chunks, int channels, int groups) {
    Space s;
    s.part = w.take<float2>((size_t)images * chunks * channels);
    s.sums = w.take<float2>((size_t)images * channels);
    s.means = w.take<float2>((size_t)images * groups);
    return s;
}

template <typename T, int V>
cudaError_t forward(const NormCall& c, const Shape& sh, const Space& w, cudaStream_t s) {
    const dim3 grid(sh.chunks, (unsigned)c.images);
    cudaError_t e = launch_pdl(k_norm_stats<T, V>, grid, dim3(kThreads), 0, s, (const T*)c.x, sh,
                               w.part);
    if (e == cudaSuccess)
        e = launch_pdl(k_norm_finish, dim3((unsigned)ceil_div(sh.groups, kThreads / 32),
                                           (unsigned)c.images),
                       dim3(kThreads), 0, s, (const float2*)w.part, sh, c.eps, (float2*)c.stats);
    if (e == cudaSuccess)
        e = launch_pdl(k_norm_apply<T, V>, grid, dim3(kThreads), 0, s, (const T*)c.x, sh,
                       (const float2*)c.stats, c.weight, c.bias, c.act, (T*)c.out);
    return e;
}

template <typename T, int V>
cudaError_t backward(const NormCall& c, const Shape& sh, const Space& w, cudaStream_t s) {
    const dim3 grid(sh.chunks, (unsigned)c.images);
    cudaError_t e = launch_pdl(k_norm_back_sums<T, V>, grid, dim3(kThreads), 0, s, (const T*)c.x,
                               (const T*)c.grad_y, sh, (const float2*)c.stats, c.weight, c.bias,
                               c.act, w.part);
    if (e == cudaSuccess)
        e = launch_pdl(k_norm_back_chunks, dim3((unsigned)ceil_div(sh.channels, kThreads / 32),
                                                (unsigned)c.images),
                       dim3(kThreads), 0, s, (const float2*)w.part, sh, w.sums);
    if (e == cudaSuccess) {
        const int64_t work = sh.channels + c.images * sh.groups;
        e = launch_pdl(k_norm_back_finish, dim3((unsigned)ceil_div(work, kThreads)), dim3(kThreads),
                       0, s, (const float2*)w.sums, sh, (int)c.images, c.weight, c.grad_weight,
                       c.grad_bias, w.means);
    }
    if (e == cudaSuccess && c.out)
        e = launch_pdl(k_norm_back_apply<T, V>, grid, dim3(kThreads), 0, s, (const T*)c.x,
                       (const T*)c.grad_y, sh, (const float2*)c.stats, (const float2*)w.means,
                       c.weight, c.bias, c.act, (T*)c.out);
    return e;
}

template <typename T>
cudaError_t run(const NormCall& c, void* ws, bool back, cudaStream_t s) {
    constexpr int V = VecOf<T>::n;
    const bool wide = c.channels % V == 0 && aligned16(c.x) && aligned16(c.out) &&
                      aligned16(c.grad_y);
    const Shape sh = shape_of(c.images, c.pixels, c.channels, c.groups, wide ? V : 1);
    Carve cv{static_cast<unsigned char*>(ws)};
    const Space w = carve(cv, c.images, sh.chunks, c.channels, c.groups);
    if (wide) return back ? backward<T, V>(c, sh, w, s) : forward<T, V>(c, sh, w, s);
    return back ? backward<T, 1>(c, sh, w, s) : forward<T, 1>(c, sh, w, s);
}

}  // namespace

size_t group_norm_workspace(int64_t images, int64_t pixels, int32_t channels, int32_t groups) {
    if (images == 0 || pixels == 0) return 0;
    int chunks = 0;
    for (int v : {1, 4, 8})
        if (channels % v == 0) {
            const int k = shape_of(images, pixels, channels, groups, v).chunks;
            chunks = k > chunks ? k : chunks;
        }
    Carve cv{nullptr};
    carve(cv, images, chunks, channels, groups);
    return cv.used;
}

cudaError_t launch_group_norm_forward(const NormCall& c, void* ws, int, cudaStream_t s) {
    if (c.images == 0) return cudaSuccess;
    if (c.pixels == 0) {   // the statistics of nothing: mean 0, variance 0
        Shape sh = shape_of(1, 1, c.channels, c.groups, 1);
        sh.pixels = sh.chunks = 0;
        return launch_pdl(k_norm_finish, dim3((unsigned)ceil_div(sh.groups, kThreads / 32),
                                              (unsigned)c.images),
                          dim3(kThreads), 0, s, (const float2*)nullptr, sh, c.eps,
                          (float2*)c.stats);
    }
    return c.dtype == kF32 ? run<float>(c, ws, false, s) : run<__nv_bfloat16>(c, ws, false, s);
}

cudaError_t launch_group_norm_backward(const NormCall& c, void* ws, int, cudaStream_t s) {
    if (c.images == 0 || c.pixels == 0) {
        for (float* g : {c.grad_weight, c.grad_bias})
            if (g) {
                const cudaError_t e = cudaMemsetAsync(g, 0, (size_t)c.channels * 4, s);
                if (e != cudaSuccess) return e;
            }
        return cudaSuccess;
    }
    return c.dtype == kF32 ? run<float>(c, ws, true, s) : run<__nv_bfloat16>(c, ws, true, s);
}

}  // namespace pulsar
