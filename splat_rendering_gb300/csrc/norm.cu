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
// A small image is one cluster's: its blocks keep their pixels in registers
// between the reduction and its use and join through distributed shared
// memory, one launch that reads and writes everything once.  A larger one
// takes two launches, each one wave of resident blocks: the second joins the
// parts of the first and reads the image again, from the end, where the L2
// still holds it; of a batch that the L2 does not hold, as many images at a
// time as it does.
//
// Statistics: a thread sums x - k and (x - k)^2 over up to 64 pixels with k
// the first of them, which bounds the cancellation of the second moment by
// that number whatever the mean, and turns them into (mean, M2); parts are
// joined by sum(M2) + sum(n (mean - common mean)^2), in 32 bits and a fixed
// order.
#include "learn_internal.cuh"

namespace pulsar {
namespace {

constexpr int kThreads = 256;
constexpr int kSegment = 64;   // pixels a thread sums about one value
constexpr int kAhead = 8;      // 16-byte loads a thread has in flight
constexpr int kAheadApply = 6; // (beside what the forward's output needs in registers)

// Resident blocks per SM: registers for kAhead loads in flight come first (one
// more block with spilled ones is 5 to 40 percent slower).
constexpr int blocks_per_sm(int v) { return v == 8 ? 2 : 3; }
constexpr int kMostBlocks = 3 * 160;   // of a wave, on the largest part

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// How an image lies on its blocks.
struct Shape {
    int64_t pixels;
    int channels, groups, cpg;   // cpg = channels / groups
    int cols;                    // vectors per pixel
    int rpb;                     // pixels a block covers at once (cols <= kThreads), else 1
    int blocks;                  // per image
    int64_t chunk;               // pixels per block
};

__device__ __forceinline__ int rows_of(int64_t len, int row, int rpb) {
    return len > row ? (int)((len - row + rpb - 1) / rpb) : 0;
}

// ------------------------------------------------------------- activation --
// The fast exponential and division: with the exact ones the gradients of a 1024 x 1024 x 16 image
// take 60 us instead of 53, and are no nearer (dx 7.1e-8 of its norm off either way, plain 32-bit
// operations 7.6e-8; dw and db are as far off as their sums' roundings).
template <int kAct>
__device__ __forceinline__ float activate(float z) {
    if (kAct == kActSilu) return __fdividef(z, 1.0f + __expf(-z));
    if (kAct == kActRelu) return z > 0.0f || z != z ? z : 0.0f;   // NaN stays NaN
    return z;
}
template <int kAct>
__device__ __forceinline__ float activate_grad(float z, float dy) {
    if (kAct == kActSilu) {
        const float s = __fdividef(1.0f, 1.0f + __expf(-z));
        return dy * (s * fmaf(z, 1.0f - s, 1.0f));
    }
    if (kAct == kActRelu) return z > 0.0f ? dy : 0.0f;
    return dy;
}

// What a thread's V channels need: the mean, rstd, w and b.
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

// ------------------------------------------------------------------ joins --
// The image's statistics from its blocks' parts, a warp per group, in two passes: the mean, about
// the first part's, and then the shares of (part's mean - mean)^2, whose sum nothing is taken from
// but the square of what the mean was off by.  (About the first part's mean in one pass, the two
// sums cancel by the number of blocks where it is far from the others': a border of 8 above 0 in
// 1024 x 1024 pixels, 37 times float32's rounding.)
// kMost bounds the parts; a lane keeps its own of them in registers.
template <int kMost, typename Part>
__device__ __forceinline__ void join_stats(const Part& part, const Shape& sh, float eps,
                                           float2* s_stats) {
    constexpr int kPer = (kMost + 31) / 32;
    const int lane = threadIdx.x & 31;
    const float inv_pix = 1.0f / (float)sh.pixels;
    const float full = (float)sh.chunk * inv_pix;
    const float last = (float)(sh.pixels - (sh.blocks - 1) * sh.chunk) * inv_pix;
    const auto share = [&](int b) { return b + 1 < sh.blocks ? full : last; };
    for (int g = threadIdx.x >> 5; g < sh.groups; g += kThreads / 32) {
        const float k = part(0, g).x;
        float2 u[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (lane + 32 * j < sh.blocks) u[j] = part(lane + 32 * j, g);
        float s = 0.0f, t = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (lane + 32 * j >= sh.blocks) continue;
            s = fmaf(share(lane + 32 * j), u[j].x - k, s);
            t += u[j].y;
        }
        const float near = k + warp_sum(s);
        t = warp_sum(t);
        float off = 0.0f, q = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (lane + 32 * j >= sh.blocks) continue;
            const float f = share(lane + 32 * j), d = u[j].x - near;
            off = fmaf(f, d, off);
            q = fmaf(f * d, d, q);
        }
        off = warp_sum(off);
        q = warp_sum(q);
        if (lane == 0) {
            float between = fmaxf(fmaf(-off, off, q), 0.0f);
            if (q != q) between = q;   // fmaxf drops a NaN
            const float var = t / ((float)sh.pixels * (float)sh.cpg) + between;
            s_stats[g] = make_float2(near + off, 1.0f / sqrtf(var + eps));
        }
    }
    __syncthreads();
}

// s_means[g] = (mean dh, mean dh h) from the blocks' parts.
template <typename Part>
__device__ __forceinline__ void join_means(const Part& part, const Shape& sh, float2* s_means) {
    const int lane = threadIdx.x & 31;
    const float inv = 1.0f / ((float)sh.pixels * (float)sh.cpg);
    for (int g = threadIdx.x >> 5; g < sh.groups; g += kThreads / 32) {
        float a = 0.0f, q = 0.0f;
        for (int b = lane; b < sh.blocks; b += 32) {
            const float2 u = part(b, g);
            a += u.x;
            q += u.y;
        }
        a = warp_sum(a);
        q = warp_sum(q);
        if (lane == 0) s_means[g] = make_float2(a * inv, q * inv);
    }
    __syncthreads();
}

// -------------------------------------------------- reductions over a run --
// s_mean, s_m2 hold one entry per thread and channel (or per vector, where a
// vector stays in a group).
__device__ __forceinline__ bool whole_vectors(const Shape& sh, int v) { return sh.cpg % v == 0; }

// A thread's (mean, M2) of cnt pixels of its V channels, as its entries.
template <int V>
__device__ __forceinline__ void put_entries(const Shape& sh, int row, int col, int cnt,
                                            const float (&mean)[V], const float (&m2)[V],
                                            float* s_mean, float* s_m2) {
    if (whole_vectors(sh, V)) {
        const int e = row * sh.cols + col;
        float m = 0.0f, t = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) m += mean[j];
        m *= 1.0f / V;
#pragma unroll
        for (int j = 0; j < V; ++j) t += fmaf((float)cnt * (mean[j] - m), mean[j] - m, m2[j]);
        s_mean[e] = m;
        s_m2[e] = t;
    } else {
        const int e = (row * sh.cols + col) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s_mean[e + j] = mean[j];
            s_m2[e + j] = m2[j];
        }
    }
}

// (mean, M2) of the run per group from the entries: a warp per group.
template <int V>
__device__ __forceinline__ void group_entries(const Shape& sh, int64_t len, const float* s_mean,
                                              const float* s_m2, float2* part) {
    const int sub = whole_vectors(sh, V) ? 1 : V;
    const int epr = sh.cols * sub, eg = epr / sh.groups;
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
        if (lane == 0) part[g] = make_float2(m, t);
    }
}

// (mean, M2) of n values about k, one of them, from s = sum(x - k), q = sum(x - k)^2.
__device__ __forceinline__ void settle(float k, float s, float q, float inv_n, float* mean,
                                       float* m2) {
    *mean = fmaf(s, inv_n, k);
    const float t = fmaxf(fmaf(-s * inv_n, s, q), 0.0f);
    *m2 = q != q ? q : t;
}

template <typename T, int V>
__device__ __forceinline__ void run_stats(const T* __restrict__ base, int64_t len, const Shape& sh,
                                          float* s_mean, float* s_m2, float2* __restrict__ part) {
    const int row = sh.rpb > 1 ? (int)threadIdx.x / sh.cols : 0;
    const int cnt = rows_of(len, row, sh.rpb);
    const int64_t pitch = (int64_t)sh.rpb * sh.channels;
    for (int col = threadIdx.x - row * sh.cols; col < sh.cols && row < sh.rpb; col += kThreads) {
        const T* at = base + (int64_t)row * sh.channels + col * V;
        float mean[V], m2[V];
#pragma unroll
        for (int j = 0; j < V; ++j) mean[j] = m2[j] = 0.0f;
        for (int i0 = 0; i0 < cnt; i0 += kSegment) {
            const int n = min(kSegment, cnt - i0);
            float k[V], s[V], q[V];
            Pack<T, V>::load(at, k);   // (kAhead divides kSegment: `at` is at pixel i0)
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = q[j] = 0.0f;
            for (int i = 0; i < n; i += kAhead, at += kAhead * pitch) {
                typename Pack<T, V>::Raw r[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (i + u < n) r[u] = Pack<T, V>::raw(at + u * pitch);
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    float v[V];
                    Pack<T, V>::open(r[u], v);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float d = i + u < n ? v[j] - k[j] : 0.0f;
                        s[j] += d;
                        q[j] = fmaf(d, d, q[j]);
                    }
                }
            }
            // this segment joins the ones before
            const float f = (float)n / (float)(i0 + n);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float m, t;
                settle(k[j], s[j], q[j], 1.0f / (float)n, &m, &t);
                const float d = m - mean[j];
                m2[j] = i0 ? m2[j] + fmaf(d * d, f * (float)i0, t) : t;
                mean[j] = i0 ? fmaf(d, f, mean[j]) : m;
            }
        }
        put_entries<V>(sh, row, col, cnt, mean, m2, s_mean, s_m2);
    }
    __syncthreads();
    group_entries<V>(sh, len, s_mean, s_m2, part);
}

// Rows of s_sum added by halves until kFewRows are left, zeros in the others: one after the other,
// the 256 rows of a single channel left its sums 2.5 times as far off as plain 32-bit ones (now
// nearer than those; 0.3 of 53 us at 1024 x 1024 x 16 floats).  Out of line, and nothing else
// changed by it: in the kernel, or with fewer rows for the loop after it, six images of 480 x 270
// x 64 in 16 bits took 91 us instead of 84.
constexpr int kFewRows = 32;
__device__ __noinline__ void fold_rows(int rows, int channels, float2* s_sum) {
    while (rows > kFewRows) {
        const int half = (rows + 1) / 2;
        for (int e = threadIdx.x; e < (rows - half) * channels; e += kThreads) {
            const float2 u = s_sum[e], v = s_sum[half * channels + e];
            s_sum[e] = make_float2(u.x + v.x, u.y + v.y);
            s_sum[half * channels + e] = make_float2(0.0f, 0.0f);
        }
        rows = half;
        __syncthreads();
    }
}

// s_sum holds (sum dz, sum dz h) per thread and channel: per channel into row
// 0 (and `total`), and per group, weighted by w, into `part`.  (One after the
// other, the 256 rows of a single channel left its sums 2.5 times as far off
// as plain 32-bit ones.)
__device__ __forceinline__ void channel_sums(const Shape& sh, const float* __restrict__ weight,
                                             float2* s_sum, float2* total, float2* part) {
    __syncthreads();
    if (sh.rpb > kFewRows) fold_rows(sh.rpb, sh.channels, s_sum);
    for (int c = threadIdx.x; c < sh.channels; c += kThreads) {
        float a = 0.0f, q = 0.0f;
#pragma unroll 4
        for (int r = 0; r < sh.rpb; ++r) {
            const float2 u = s_sum[r * sh.channels + c];
            a += u.x;
            q += u.y;
        }
        s_sum[c] = make_float2(a, q);   // (row 0's own entry: nobody else reads it)
        if (total) total[c] = make_float2(a, q);
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int g = threadIdx.x >> 5; g < sh.groups; g += kThreads / 32) {
        float a = 0.0f, q = 0.0f;
        for (int c = g * sh.cpg + lane; c < (g + 1) * sh.cpg; c += 32) {
            const float wc = weight ? weight[c] : 1.0f;
            a = fmaf(wc, s_sum[c].x, a);
            q = fmaf(wc, s_sum[c].y, q);
        }
        a = warp_sum(a);
        q = warp_sum(q);
        if (lane == 0) part[g] = make_float2(a, q);
    }
}

// One value's share of the sums, and its gradient.
template <int kAct>
__device__ __forceinline__ float grad_h(float x, float dy, float mean, float rstd, float w, float b,
                                        float* h) {
    *h = (x - mean) * rstd;
    return activate_grad<kAct>(fmaf(*h, w, b), dy);
}

// ----------------------------------------------------------- two launches --
// (y may be x, dx may be dy or x: they are not restrict)
template <typename T, int V, int kAct>
__device__ __forceinline__ void run_apply(const T* x, T* y, int64_t off, int64_t len,
                                          const Shape& sh, const float2* stats,
                                          const float* __restrict__ weight,
                                          const float* __restrict__ bias) {
    const int row = sh.rpb > 1 ? (int)threadIdx.x / sh.cols : 0;
    const int cnt = rows_of(len, row, sh.rpb);
    const int64_t pitch = (int64_t)sh.rpb * sh.channels;
    for (int col = threadIdx.x - row * sh.cols; col < sh.cols && row < sh.rpb; col += kThreads) {
        Affine<V> f;
        f.load(stats, weight, bias, col * V, sh.cpg);
#pragma unroll
        for (int j = 0; j < V; ++j) f.rstd[j] *= f.w[j];
        // from the end: what was read last is nearest
        int64_t at = off + (row + (int64_t)(cnt - 1) * sh.rpb) * sh.channels + col * V;
        for (int i = 0; i < cnt; i += kAheadApply, at -= kAheadApply * pitch) {
            typename Pack<T, V>::Raw r[kAheadApply];
#pragma unroll
            for (int u = 0; u < kAheadApply; ++u)
                if (i + u < cnt) r[u] = Pack<T, V>::raw_last(x + at - u * pitch);
#pragma unroll
            for (int u = 0; u < kAheadApply; ++u) {
                if (i + u >= cnt) break;
                float v[V];
                Pack<T, V>::open(r[u], v);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[j] = activate<kAct>(fmaf(v[j] - f.mean[j], f.rstd[j], f.b[j]));
                Pack<T, V>::store_through(y + at - u * pitch, v);
            }
        }
    }
}

struct Place {
    int64_t off, len;   // first element of the block's run, pixels
};
__device__ __forceinline__ Place place(const Shape& sh, int64_t image) {
    const int64_t p0 = (int64_t)blockIdx.x * sh.chunk;
    return {(image * sh.pixels + p0) * sh.channels, min(sh.chunk, sh.pixels - p0)};
}

// part[image of the launch][block][group] = (mean, M2).  Bound by the reads and
// a fixed 6 us of launch, first loads and the block's reduction: 14 us for
// 1024 x 1024 x 16 floats (64 MB, 4.8 TB/s), 25 us for 100 MB in 16 bits.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(V))
k_norm_stats(const T* __restrict__ x, const __grid_constant__ Shape sh, int64_t image0,
             float2* __restrict__ part) {
    pdl_begin();
    extern __shared__ float smem[];
    const Place p = place(sh, image0 + blockIdx.y);
    const int entries = sh.rpb * sh.cols * V;
    run_stats<T, V>(x + p.off, p.len, sh, smem, smem + entries,
                    part + ((size_t)blockIdx.y * sh.blocks + blockIdx.x) * sh.groups);
}

// Joins the parts (every block for itself: 300 to 450 of them, a warp per
// group) and writes the output: 18 us for 1024 x 1024 x 16 floats, 8 MB of the
// image coming from DRAM again, 34 us for 100 MB in 16 bits.
template <typename T, int V, int kAct>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(V))
k_norm_apply(const T* x, const __grid_constant__ Shape sh, int64_t image0,
             const float2* __restrict__ part, const float* __restrict__ weight,
             const float* __restrict__ bias, float eps, T* y,
             float2* __restrict__ stats) {
    pdl_begin();
    extern __shared__ float smem[];
    float2* s_stats = reinterpret_cast<float2*>(smem);
    const int64_t image = image0 + blockIdx.y;
    const Place p = place(sh, image);
    const float2* mine = part + (size_t)blockIdx.y * sh.blocks * sh.groups;
    join_stats<kMostBlocks>([&](int b, int g) { return mine[(size_t)b * sh.groups + g]; }, sh, eps,
                            s_stats);
    if (blockIdx.x == 0)
        for (int g = threadIdx.x; g < sh.groups; g += kThreads)
            stats[(size_t)image * sh.groups + g] = s_stats[g];
    run_apply<T, V, kAct>(x, y, p.off, p.len, sh, s_stats, weight, bias);
}

// part[image of the launch][block][group], total[..][block][channel].  31 us
// for an image and a gradient of 1024 x 1024 x 16 floats (128 MB: more than the
// L2 keeps).
template <typename T, int V, int kAct>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(V))
k_norm_back_sums(const T* __restrict__ x, const T* __restrict__ dy, const __grid_constant__ Shape sh,
                 int64_t image0, const float2* __restrict__ stats,
                 const float* __restrict__ weight, const float* __restrict__ bias,
                 float2* __restrict__ part, float2* __restrict__ total) {
    pdl_begin();
    extern __shared__ float smem[];
    float2* s_sum = reinterpret_cast<float2*>(smem);
    const int64_t image = image0 + blockIdx.y;
    const Place p = place(sh, image);
    const int row = sh.rpb > 1 ? (int)threadIdx.x / sh.cols : 0;
    const int cnt = rows_of(p.len, row, sh.rpb);
    const int64_t pitch = (int64_t)sh.rpb * sh.channels;
    for (int col = threadIdx.x - row * sh.cols; col < sh.cols && row < sh.rpb; col += kThreads) {
        Affine<V> f;
        f.load(stats + (size_t)image * sh.groups, weight, bias, col * V, sh.cpg);
        float a[V], q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = q[j] = 0.0f;
        int64_t at = p.off + (int64_t)row * sh.channels + col * V;
        for (int i = 0; i < cnt; i += kAhead / 2, at += kAhead / 2 * pitch) {
            typename Pack<T, V>::Raw rx[kAhead / 2], ry[kAhead / 2];
#pragma unroll
            for (int u = 0; u < kAhead / 2; ++u) {
                if (i + u < cnt) {
                    rx[u] = Pack<T, V>::raw(x + at + u * pitch);
                    ry[u] = Pack<T, V>::raw(dy + at + u * pitch);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead / 2; ++u) {
                if (i + u >= cnt) break;
                float v[V], g[V];
                Pack<T, V>::open(rx[u], v);
                Pack<T, V>::open(ry[u], g);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float h;
                    const float dz =
                        grad_h<kAct>(v[j], g[j], f.mean[j], f.rstd[j], f.w[j], f.b[j], &h);
                    a[j] += dz;
                    q[j] = fmaf(dz, h, q[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            s_sum[row * sh.channels + col * V + j] = make_float2(a[j], q[j]);
    }
    const size_t blk = (size_t)blockIdx.y * sh.blocks + blockIdx.x;
    channel_sums(sh, weight, s_sum,
                 total + blk * sh.channels,
                 part + blk * sh.groups);
}

template <typename T, int V, int kAct>
__device__ __forceinline__ void run_back(const T* x, const T* dy, T* dx, int64_t off,
                                         int64_t len, const Shape& sh, const float2* __restrict__ stats,
                                         const float2* means, const float* __restrict__ weight,
                                         const float* __restrict__ bias) {
    const int row = sh.rpb > 1 ? (int)threadIdx.x / sh.cols : 0;
    const int cnt = rows_of(len, row, sh.rpb);
    const int64_t pitch = (int64_t)sh.rpb * sh.channels;
    for (int col = threadIdx.x - row * sh.cols; col < sh.cols && row < sh.rpb; col += kThreads) {
        Affine<V> f;
        f.load(stats, weight, bias, col * V, sh.cpg);
        float m1[V], m2[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 u = means[(col * V + j) / sh.cpg];
            m1[j] = u.x;
            m2[j] = u.y;
        }
        int64_t at = off + (row + (int64_t)(cnt - 1) * sh.rpb) * sh.channels + col * V;
        for (int i = 0; i < cnt; i += kAhead / 2, at -= kAhead / 2 * pitch) {
            typename Pack<T, V>::Raw rx[kAhead / 2], ry[kAhead / 2];
#pragma unroll
            for (int u = 0; u < kAhead / 2; ++u) {
                if (i + u < cnt) {
                    rx[u] = Pack<T, V>::raw_last(x + at - u * pitch);
                    ry[u] = Pack<T, V>::raw_last(dy + at - u * pitch);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead / 2; ++u) {
                if (i + u >= cnt) break;
                float v[V], g[V];
                Pack<T, V>::open(rx[u], v);
                Pack<T, V>::open(ry[u], g);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float h;
                    const float dz =
                        grad_h<kAct>(v[j], g[j], f.mean[j], f.rstd[j], f.w[j], f.b[j], &h);
                    v[j] = f.rstd[j] * (fmaf(dz, f.w[j], -m1[j]) - h * m2[j]);
                }
                Pack<T, V>::store_through(dx + at - u * pitch, v);
            }
        }
    }
}

// 25 us for the same, 59 MB of 128 coming from DRAM again.
template <typename T, int V, int kAct>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(V))
k_norm_back_apply(const T* x, const T* dy, const __grid_constant__ Shape sh, int64_t image0,
                  const float2* __restrict__ stats, const float2* __restrict__ part,
                  const float* __restrict__ weight, const float* __restrict__ bias,
                  T* dx, const float2* __restrict__ total, int images,
                  float2* __restrict__ image_total, float* __restrict__ grad_weight,
                  float* __restrict__ grad_bias) {
    pdl_begin();
    extern __shared__ float smem[];
    float2* s_means = reinterpret_cast<float2*>(smem);
    const int64_t image = image0 + blockIdx.y;
    const Place p = place(sh, image);
    if (dx) {
        const float2* mine = part + (size_t)blockIdx.y * sh.blocks * sh.groups;
        join_means([&](int b, int g) { return mine[(size_t)b * sh.groups + g]; }, sh, s_means);
        run_back<T, V, kAct>(x, dy, dx, p.off, p.len, sh, stats + (size_t)image * sh.groups,
                             s_means, weight, bias);
    }
    // the image's channel sums, a warp per channel; of one image, the gradients themselves
    const float2* t = total + (size_t)blockIdx.y * sh.blocks * sh.channels;
    const int lane = threadIdx.x & 31;
    for (int c = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); c < sh.channels;
         c += gridDim.x * (kThreads / 32)) {
        float a = 0.0f, q = 0.0f;
#pragma unroll 4
        for (int b = lane; b < sh.blocks; b += 32) {
            const float2 u = t[(size_t)b * sh.channels + c];
            a += u.x;
            q += u.y;
        }
        a = warp_sum(a);
        q = warp_sum(q);
        if (lane == 0) {
            if (images > 1) {
                image_total[(size_t)image * sh.channels + c] = make_float2(a, q);
            } else {
                if (grad_bias) grad_bias[c] = a;
                if (grad_weight) grad_weight[c] = q;
            }
        }
    }
}

// The parameters' gradients from the images' totals [n][channels].
__global__ void __launch_bounds__(kThreads)
k_norm_back_params(const float2* __restrict__ total, int64_t n, int channels,
                   float* __restrict__ grad_weight, float* __restrict__ grad_bias) {
    pdl_begin();
    const int lane = threadIdx.x & 31, c = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (c >= channels) return;
    float a = 0.0f, q = 0.0f;
#pragma unroll 4
    for (int64_t r = lane; r < n; r += 32) {
        const float2 u = total[r * channels + c];
        a += u.x;
        q += u.y;
    }
    a = warp_sum(a);
    q = warp_sum(q);
    if (lane == 0) {
        if (grad_bias) grad_bias[c] = a;
        if (grad_weight) grad_weight[c] = q;
    }
}

// The statistics of nothing: mean 0, variance 0.
__global__ void k_norm_empty(float2* stats, int64_t n, float eps) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) stats[i] = make_float2(0.0f, 1.0f / sqrtf(eps));
}

// ---------------------------------------------------------- small images --
// A cluster of sh.blocks blocks (1 to 8) has an image; a thread keeps its
// pixels, at most kHeld, as they were loaded.  Bound by the chain of latencies
// (launch, load, block, cluster, store): 6.7 us for 40 x 24 x 16 floats either
// way, 7.3 us for eight images of 1000 x 64.
constexpr int kHeld = 8;
constexpr int kMaxCluster = 8;

// (every thread of the block calls; the barrier wants each warp whole, and the work before it
// may have split one)
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// *p in the shared memory of the cluster's block `rank`
__device__ __forceinline__ float2 of_block(const float2* p, int rank) {
    uint32_t at;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(at)
                 : "memory");
    return v;
}

template <typename T, int V, int kAct>
__global__ void __launch_bounds__(kThreads)
k_norm_small(const T* x, const __grid_constant__ Shape sh,
             const float* __restrict__ weight, const float* __restrict__ bias, float eps,
             T* y, float2* __restrict__ stats) {
    using P = Pack<T, V>;
    pdl_begin();
    extern __shared__ float smem[];
    const int entries = sh.rpb * sh.cols * V;
    float* s_mean = smem;
    float* s_m2 = smem + entries;
    float2* s_part = reinterpret_cast<float2*>(smem + 2 * entries);
    float2* s_stats = s_part + sh.groups;
    const Place p = place(sh, blockIdx.y);
    const int row = (int)threadIdx.x / sh.cols, col = (int)threadIdx.x - row * sh.cols;
    const int cnt = row < sh.rpb ? rows_of(p.len, row, sh.rpb) : 0;
    const int64_t at = p.off + (int64_t)row * sh.channels + col * V;
    const int64_t pitch = (int64_t)sh.rpb * sh.channels;
    typename P::Raw held[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (i < cnt) held[i] = P::raw(x + at + i * pitch);
    if (row < sh.rpb) {
        float k[V], mean[V], m2[V], s[V], q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) k[j] = mean[j] = m2[j] = s[j] = q[j] = 0.0f;
        if (cnt > 0) P::open(held[0], k);
#pragma unroll
        for (int i = 1; i < kHeld; ++i) {
            if (i < cnt) {
                float v[V];
                P::open(held[i], v);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = v[j] - k[j];
                    s[j] += d;
                    q[j] = fmaf(d, d, q[j]);
                }
            }
        }
        if (cnt > 0) {
            const float inv = 1.0f / (float)cnt;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                // (an infinite k leaves no difference to itself where it is alone)
                if (!(k[j] - k[j] == 0.0f)) q[j] = k[j] - k[j];
                settle(k[j], s[j], q[j], inv, &mean[j], &m2[j]);
            }
        }
        put_entries<V>(sh, row, col, cnt, mean, m2, s_mean, s_m2);
    }
    __syncthreads();
    group_entries<V>(sh, p.len, s_mean, s_m2, s_part);
    cluster_meet();
    join_stats<kMaxCluster>([&](int b, int g) { return of_block(s_part + g, b); }, sh, eps, s_stats);
    if (blockIdx.x == 0)
        for (int g = threadIdx.x; g < sh.groups; g += kThreads)
            stats[(size_t)blockIdx.y * sh.groups + g] = s_stats[g];
    if (row < sh.rpb) {
        Affine<V> f;
        f.load(s_stats, weight, bias, col * V, sh.cpg);
#pragma unroll
        for (int j = 0; j < V; ++j) f.rstd[j] *= f.w[j];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            if (i < cnt) {
                float v[V];
                P::open(held[i], v);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    v[j] = activate<kAct>(fmaf(v[j] - f.mean[j], f.rstd[j], f.b[j]));
                P::store(y + at + i * pitch, v);
            }
        }
    }
    cluster_meet();   // the others may still read this block's parts
}

// total[image][channel]; where there is one image, its gradients themselves.
template <typename T, int V, int kAct>
__global__ void __launch_bounds__(kThreads)
k_norm_small_back(const T* x, const T* dy,
                  const __grid_constant__ Shape sh, const float2* __restrict__ stats,
                  const float* __restrict__ weight, const float* __restrict__ bias,
                  T* dx, float* __restrict__ grad_weight,
                  float* __restrict__ grad_bias, float2* __restrict__ total) {
    using P = Pack<T, V>;
    pdl_begin();
    extern __shared__ float smem[];
    float2* s_sum = reinterpret_cast<float2*>(smem);
    float2* s_part = s_sum + sh.rpb * sh.cols * V;
    float2* s_means = s_part + sh.groups;
    const Place p = place(sh, blockIdx.y);
    const int row = (int)threadIdx.x / sh.cols, col = (int)threadIdx.x - row * sh.cols;
    const int cnt = row < sh.rpb ? rows_of(p.len, row, sh.rpb) : 0;
    const int64_t at = p.off + (int64_t)row * sh.channels + col * V;
    const int64_t pitch = (int64_t)sh.rpb * sh.channels;
    typename P::Raw hx[kHeld], hy[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        if (i < cnt) {
            hx[i] = P::raw(x + at + i * pitch);
            hy[i] = P::raw(dy + at + i * pitch);
        }
    }
    Affine<V> f;
    if (row < sh.rpb) {
        f.load(stats + (size_t)blockIdx.y * sh.groups, weight, bias, col * V, sh.cpg);
        float a[V], q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = q[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            if (i < cnt) {
                float v[V], g[V];
                P::open(hx[i], v);
                P::open(hy[i], g);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float h;
                    const float dz =
                        grad_h<kAct>(v[j], g[j], f.mean[j], f.rstd[j], f.w[j], f.b[j], &h);
                    a[j] += dz;
                    q[j] = fmaf(dz, h, q[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            s_sum[row * sh.channels + col * V + j] = make_float2(a[j], q[j]);
    }
    channel_sums(sh, weight, s_sum, nullptr, s_part);
    cluster_meet();
    join_means([&](int b, int g) { return of_block(s_part + g, b); }, sh, s_means);
    // the channels' sums over the cluster: each block takes a share of them
    for (int c = blockIdx.x * kThreads + threadIdx.x; c < sh.channels; c += sh.blocks * kThreads) {
        float a = 0.0f, q = 0.0f;
        for (int b = 0; b < sh.blocks; ++b) {
            const float2 u = of_block(s_sum + c, b);
            a += u.x;
            q += u.y;
        }
        if (gridDim.y > 1) {
            total[(size_t)blockIdx.y * sh.channels + c] = make_float2(a, q);
        } else {
            if (grad_bias) grad_bias[c] = a;
            if (grad_weight) grad_weight[c] = q;
        }
    }
    if (row < sh.rpb && dx) {
        float m1[V], m2[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 u = s_means[(col * V + j) / sh.cpg];
            m1[j] = u.x;
            m2[j] = u.y;
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            if (i < cnt) {
                float v[V], g[V];
                P::open(hx[i], v);
                P::open(hy[i], g);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float h;
                    const float dz =
                        grad_h<kAct>(v[j], g[j], f.mean[j], f.rstd[j], f.w[j], f.b[j], &h);
                    v[j] = f.rstd[j] * (fmaf(dz, f.w[j], -m1[j]) - h * m2[j]);
                }
                P::store(dx + at + i * pitch, v);
            }
        }
    }
    cluster_meet();
}

// ----------------------------------------------------------------- plans --
// Shared memory of the reductions: an entry of two floats per thread and
// channel of a vector, and the per-group values.
size_t smem_bytes(const Shape& s, int v) { return (size_t)8 * (s.rpb * s.cols * v + 2 * s.groups); }
constexpr size_t kSmemMost = 8 * 3 * 4096;   // 4096 channels in as many groups
constexpr int64_t kL2Share = 128 << 20;      // bytes of images in flight that the L2 keeps (in part)

Shape shape_of(int64_t pixels, int channels, int groups, int v) {
    Shape s{};
    s.pixels = pixels;
    s.channels = channels;
    s.groups = groups;
    s.cpg = channels / groups;
    s.cols = channels / v;
    s.rpb = s.cols < kThreads ? kThreads / s.cols : 1;
    return s;
}

// Whether a cluster holds an image, and its blocks: the fewest pixels per
// thread that eight blocks give.
bool small_shape(Shape* s) {
    if (s->cols > kThreads || s->pixels > (int64_t)kMaxCluster * s->rpb * kHeld) return false;
    int n = 1;
    while (n < kMaxCluster && (int64_t)n * s->rpb < s->pixels) n *= 2;
    while ((n - 1) * ceil_div(s->pixels, n) >= s->pixels) n /= 2;   // no block without a pixel
    s->blocks = n;
    s->chunk = ceil_div(s->pixels, n);
    return s->chunk <= (int64_t)s->rpb * kHeld;
}

// Two launches: as many images a round as the L2 keeps, in equal rounds ...
int64_t images_at_once(int64_t images, int64_t pixels, int channels, int elem, bool back) {
    const int64_t fit = kL2Share / (pixels * channels * elem * (back ? 2 : 1));
    return ceil_div(images, ceil_div(images, fit < 1 ? 1 : fit < images ? fit : images));
}
// ... over which one wave of resident blocks lies, none with less than four
// pixels per thread.
void large_shape(Shape* s, int64_t at_once, int v, int n_sms) {
    int per_sm = (int)(220 * 1024 / (smem_bytes(*s, v) + 1024));
    per_sm = per_sm < blocks_per_sm(v) ? per_sm : blocks_per_sm(v);
    const int64_t blocks = (int64_t)n_sms * per_sm;
    const int64_t each = blocks / at_once > 0 ? blocks / at_once : 1;
    int64_t per = ceil_div(s->pixels, each);
    const int64_t least = (int64_t)s->rpb * 4;
    per = ceil_div(per < least ? least : per, s->rpb) * s->rpb;
    s->chunk = per;
    s->blocks = (int)ceil_div(s->pixels, per);
}

struct Space {
    float2 *part, *total, *image_total;
};
// `at_once` images of `blocks` blocks each
Space carve(Carve& w, int64_t images, int64_t at_once, int64_t blocks, int channels, int groups) {
    Space p;
    p.part = w.take<float2>((size_t)at_once * blocks * groups);
    p.total = w.take<float2>((size_t)at_once * blocks * channels);
    p.image_total = w.take<float2>((size_t)images * channels);
    return p;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), const Shape& sh, int64_t images, size_t smem,
                           cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sh.blocks, (unsigned)images);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)sh.blocks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

template <typename T, int V, int kAct>
cudaError_t forward(const NormCall& c, void* ws, int n_sms, cudaStream_t s) {
    Shape sh = shape_of(c.pixels, c.channels, c.groups, V);
    if (small_shape(&sh))
        return launch_cluster(k_norm_small<T, V, kAct>, sh, c.images, smem_bytes(sh, V), s,
                              (const T*)c.x, sh, c.weight, c.bias, c.eps, (T*)c.out,
                              (float2*)c.stats);
    const int64_t at_once = images_at_once(c.images, c.pixels, c.channels, sizeof(T), false);
    large_shape(&sh, at_once, V, n_sms);
    Carve cv{static_cast<unsigned char*>(ws)};
    const Space w = carve(cv, c.images, at_once, sh.blocks, c.channels, c.groups);
    cudaError_t e = cudaSuccess;
    for (int64_t i = 0; i < c.images && e == cudaSuccess; i += at_once) {
        const int64_t n = c.images - i < at_once ? c.images - i : at_once;
        const dim3 grid((unsigned)sh.blocks, (unsigned)n);
        e = launch_pdl(k_norm_stats<T, V>, grid, dim3(kThreads), smem_bytes(sh, V), s,
                       (const T*)c.x, sh, i, w.part);
        if (e == cudaSuccess)
            e = launch_pdl(k_norm_apply<T, V, kAct>, grid, dim3(kThreads), (size_t)8 * sh.groups,
                           s, (const T*)c.x, sh, i, (const float2*)w.part, c.weight, c.bias, c.eps,
                           (T*)c.out, (float2*)c.stats);
    }
    return e;
}

cudaError_t params(const NormCall& c, const float2* total, int64_t rows, cudaStream_t s) {
    if (!c.grad_weight && !c.grad_bias) return cudaSuccess;
    return launch_pdl(k_norm_back_params, dim3((unsigned)ceil_div(c.channels, kThreads / 32)),
                      dim3(kThreads), 0, s, total, rows, c.channels, c.grad_weight, c.grad_bias);
}

template <typename T, int V, int kAct>
cudaError_t backward(const NormCall& c, void* ws, int n_sms, cudaStream_t s) {
    Shape sh = shape_of(c.pixels, c.channels, c.groups, V);
    Carve cv{static_cast<unsigned char*>(ws)};
    if (small_shape(&sh)) {
        const Space w = carve(cv, c.images, 0, 0, c.channels, c.groups);
        const cudaError_t e = launch_cluster(
            k_norm_small_back<T, V, kAct>, sh, c.images, smem_bytes(sh, V), s, (const T*)c.x,
            (const T*)c.grad_y, sh, (const float2*)c.stats, c.weight, c.bias, (T*)c.out,
            c.grad_weight, c.grad_bias, w.image_total);
        return e != cudaSuccess || c.images == 1 ? e : params(c, w.image_total, c.images, s);
    }
    const int64_t at_once = images_at_once(c.images, c.pixels, c.channels, sizeof(T), true);
    large_shape(&sh, at_once, V, n_sms);
    const Space w = carve(cv, c.images, at_once, sh.blocks, c.channels, c.groups);
    cudaError_t e = cudaSuccess;
    for (int64_t i = 0; i < c.images && e == cudaSuccess; i += at_once) {
        const int64_t n = c.images - i < at_once ? c.images - i : at_once;
        const dim3 grid((unsigned)sh.blocks, (unsigned)n);
        e = launch_pdl(k_norm_back_sums<T, V, kAct>, grid, dim3(kThreads), smem_bytes(sh, V), s,
                       (const T*)c.x, (const T*)c.grad_y, sh, i, (const float2*)c.stats, c.weight,
                       c.bias, w.part, w.total);
        if (e == cudaSuccess)
            e = launch_pdl(k_norm_back_apply<T, V, kAct>, grid, dim3(kThreads),
                           (size_t)8 * sh.groups, s, (const T*)c.x, (const T*)c.grad_y, sh, i,
                           (const float2*)c.stats, (const float2*)w.part, c.weight, c.bias,
                           (T*)c.out, (const float2*)w.total, (int)c.images, w.image_total,
                           c.grad_weight, c.grad_bias);
    }
    return e != cudaSuccess || c.images == 1 ? e : params(c, w.image_total, c.images, s);
}

template <typename T, int V>
cudaError_t by_act(const NormCall& c, bool back, void* ws, int n_sms, cudaStream_t s) {
    switch (c.act) {
        case kActSilu:
            return back ? backward<T, V, kActSilu>(c, ws, n_sms, s)
                        : forward<T, V, kActSilu>(c, ws, n_sms, s);
        case kActRelu:
            return back ? backward<T, V, kActRelu>(c, ws, n_sms, s)
                        : forward<T, V, kActRelu>(c, ws, n_sms, s);
        default:
            return back ? backward<T, V, kActNone>(c, ws, n_sms, s)
                        : forward<T, V, kActNone>(c, ws, n_sms, s);
    }
}

cudaError_t run(const NormCall& c, bool back, void* ws, int n_sms, cudaStream_t s) {
    const int v = c.dtype == kF32 ? 4 : 8;
    const bool wide = c.channels % v == 0 && aligned16(c.x) && aligned16(c.out) &&
                      aligned16(c.grad_y);
    if (c.dtype == kF32)
        return wide ? by_act<float, 4>(c, back, ws, n_sms, s)
                    : by_act<float, 1>(c, back, ws, n_sms, s);
    return wide ? by_act<__nv_bfloat16, 8>(c, back, ws, n_sms, s)
                : by_act<__nv_bfloat16, 1>(c, back, ws, n_sms, s);
}

template <typename T, int V, int kAct>
cudaError_t prepare_one() {
    const auto most = [](const void* k) {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
    };
    cudaError_t e = most((const void*)k_norm_stats<T, V>);
    if (e == cudaSuccess) e = most((const void*)k_norm_apply<T, V, kAct>);
    if (e == cudaSuccess) e = most((const void*)k_norm_back_sums<T, V, kAct>);
    if (e == cudaSuccess) e = most((const void*)k_norm_back_apply<T, V, kAct>);
    if (e == cudaSuccess) e = most((const void*)k_norm_small<T, V, kAct>);
    if (e == cudaSuccess) e = most((const void*)k_norm_small_back<T, V, kAct>);
    return e;
}
template <typename T, int V>
cudaError_t prepare_acts() {
    cudaError_t e = prepare_one<T, V, kActNone>();
    if (e == cudaSuccess) e = prepare_one<T, V, kActSilu>();
    if (e == cudaSuccess) e = prepare_one<T, V, kActRelu>();
    return e;
}

}  // namespace

size_t group_norm_workspace(int64_t images, int64_t pixels, int32_t channels, int32_t groups) {
    if (images == 0 || pixels == 0) return 0;
    // the most blocks of a round in any form: one wave of the largest part, or
    // one per image; and no more than the pixels
    int64_t blocks = 0;
    for (int elem : {2, 4})
        for (bool back : {false, true}) {
            const int64_t n = images_at_once(images, pixels, channels, elem, back);
            const int64_t each = kMostBlocks / n > 0 ? kMostBlocks / n : 1;
            const int64_t all = n * (each < pixels ? each : pixels);
            blocks = all > blocks ? all : blocks;
        }
    Carve cv{nullptr};
    carve(cv, images, 1, blocks, channels, groups);
    return cv.used;
}

cudaError_t prepare_group_norm() {
    cudaError_t e = prepare_acts<float, 4>();
    if (e == cudaSuccess) e = prepare_acts<float, 1>();
    if (e == cudaSuccess) e = prepare_acts<__nv_bfloat16, 8>();
    if (e == cudaSuccess) e = prepare_acts<__nv_bfloat16, 1>();
    return e;
}

cudaError_t launch_group_norm_forward(const NormCall& c, void* ws, int n_sms, cudaStream_t s) {
    const int64_t n = c.images * c.groups;
    if (c.images == 0) return cudaSuccess;
    if (c.pixels == 0) {
        k_norm_empty<<<(unsigned)ceil_div(n, kThreads), kThreads, 0, s>>>((float2*)c.stats, n, c.eps);
        return cudaGetLastError();
    }
    return run(c, false, ws, n_sms, s);
}

cudaError_t launch_group_norm_backward(const NormCall& c, void* ws, int n_sms, cudaStream_t s) {
    if (c.images == 0 || c.pixels == 0) {
        for (float* g : {c.grad_weight, c.grad_bias})
            if (g) {
                const cudaError_t e = cudaMemsetAsync(g, 0, (size_t)c.channels * 4, s);
                if (e != cudaSuccess) return e;
            }
        return cudaSuccess;
    }
    return run(c, true, ws, n_sms, s);
}

}  // namespace pulsar
