// Internal definitions shared by the kernels of the learned parts around the
// renderer: the codebook embedding, the group normalisation of feature images
// and the orthogonalisation of an update.  Their entry points work on a
// handle that owns one block of device workspace and a latched error word;
// every launcher below carves what it needs out of that block.
#pragma once

#include <cuda_bf16.h>

#include "pulsar_internal.cuh"

namespace pulsar {

constexpr uint32_t kErrIndex = 8u;   // a token at or above the table's rows

// Small device-resident state of a learn handle.
struct LearnState {
    uint32_t error;   // latched kErr* bits
};

enum ElemType { kF32 = 0, kBf16 = 1 };
enum IndexType { kI32 = 0, kI64 = 1 };
enum Activation { kActNone = 0, kActSilu = 1, kActRelu = 2 };

// The launches of a call form a chain in which each needs all of the one
// before: a kernel of long-lived blocks lets the next one's blocks take SMs
// as they fall free and set up, and those wait in pdl_begin() for its results.
__device__ __forceinline__ void pdl_next() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Piece by piece carve-up of the workspace, every piece 256-byte aligned; run
// over a null base it counts the bytes a call needs.
struct Carve {
    unsigned char* base;
    size_t used = 0;
    template <typename T>
    T* take(size_t count) {
        T* p = reinterpret_cast<T*>(base + used);
        used += (count * sizeof(T) + 255) / 256 * 256;
        return p;
    }
};

// ------------------------------------------------------- 16-byte vectors --
// V consecutive elements of type T: 16 bytes of them (V = 4 or 8), or one.
template <typename T, int V>
struct Pack;
template <>
struct Pack<float, 4> {
    using Raw = float4;   // as it was loaded
    static __device__ __forceinline__ Raw raw(const float* p) {
        return *reinterpret_cast<const float4*>(p);
    }
    static __device__ __forceinline__ void open(const Raw& u, float (&v)[4]) {
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
    static __device__ __forceinline__ void load(const float* p, float (&v)[4]) {
        const float4 u = *reinterpret_cast<const float4*>(p);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
    static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
    // read for the last time; written, not to be read soon
    static __device__ __forceinline__ Raw raw_last(const float* p) {
        return __ldcs(reinterpret_cast<const float4*>(p));
    }
    static __device__ __forceinline__ void store_through(float* p, const float (&v)[4]) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    }
};
template <>
struct Pack<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ Raw raw(const __nv_bfloat16* p) {
        return *reinterpret_cast<const uint4*>(p);
    }
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[8]) {
        open(*reinterpret_cast<const uint4*>(p), v);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(p) = round8(v);
    }
    static __device__ __forceinline__ Raw raw_last(const __nv_bfloat16* p) {
        return __ldcs(reinterpret_cast<const uint4*>(p));
    }
    static __device__ __forceinline__ void store_through(__nv_bfloat16* p, const float (&v)[8]) {
        __stcs(reinterpret_cast<uint4*>(p), round8(v));
    }
    static __device__ __forceinline__ void open(const uint4& u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 round8(const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Pack<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ Raw raw(const float* p) { return *p; }
    static __device__ __forceinline__ void open(const Raw& u, float (&v)[1]) { v[0] = u; }
    static __device__ __forceinline__ void load(const float* p, float (&v)[1]) { v[0] = *p; }
    static __device__ __forceinline__ void store(float* p, const float (&v)[1]) { *p = v[0]; }
    static __device__ __forceinline__ Raw raw_last(const float* p) { return *p; }
    static __device__ __forceinline__ void store_through(float* p, const float (&v)[1]) {
        store(p, v);
    }
};
template <>
struct Pack<__nv_bfloat16, 1> {
    using Raw = __nv_bfloat16;
    static __device__ __forceinline__ Raw raw(const __nv_bfloat16* p) { return *p; }
    static __device__ __forceinline__ void open(const Raw& u, float (&v)[1]) {
        v[0] = __bfloat162float(u);
    }
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[1]) {
        v[0] = __bfloat162float(*p);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[1]) {
        *p = __float2bfloat16_rn(v[0]);
    }
    static __device__ __forceinline__ Raw raw_last(const __nv_bfloat16* p) { return *p; }
    static __device__ __forceinline__ void store_through(__nv_bfloat16* p, const float (&v)[1]) {
        store(p, v);
    }
};

template <typename T>
struct VecOf;   // elements in 16 bytes
template <>
struct VecOf<float> { static constexpr int n = 4; };
template <>
struct VecOf<__nv_bfloat16> { static constexpr int n = 8; };

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---------------------------------------------------------- launchers --
struct EmbedCall {
    const void* src;      // table (forward) or grad_out (backward)
    const void* tokens;
    int64_t n, rows, dim;
    float scale;
    int dtype, index;
    void* dst;            // out (forward) or grad_table (backward)
};
size_t embed_workspace(int64_t n, int64_t rows, int64_t dim);
cudaError_t prepare_embed();
cudaError_t launch_embed_forward(const EmbedCall& c, LearnState* st, cudaStream_t stream);
cudaError_t launch_embed_backward(const EmbedCall& c, LearnState* st, void* ws, int n_sms,
                                  cudaStream_t stream);

struct NormCall {
    const void* x;
    const void* grad_y;       // backward
    const float* weight;      // may be NULL: ones
    const float* bias;        // may be NULL: zeros
    int64_t images, pixels;
    int32_t channels, groups;
    float eps;
    int act, dtype;
    void* out;                // y or grad_x
    float* stats;             // [images, groups, 2]: written by the forward, read by the backward
    float* grad_weight;       // may be NULL
    float* grad_bias;         // may be NULL
};
size_t group_norm_workspace(int64_t images, int64_t pixels, int32_t channels, int32_t groups);
cudaError_t prepare_group_norm();
cudaError_t launch_group_norm_forward(const NormCall& c, void* ws, int n_sms, cudaStream_t stream);
cudaError_t launch_group_norm_backward(const NormCall& c, void* ws, int n_sms,
                                       cudaStream_t stream);

struct OrthCall {
    const void* grad;
    int64_t batch, m, n;
    int steps;
    float a, b, c, eps;
    int dtype;
    void* out;
};
// Whether the iterates and the polynomial's values stay inside what the products can hold.
bool orth_in_range(int steps, float a, float b, float c);
size_t orth_workspace(int64_t batch, int64_t m, int64_t n, int dtype);
cudaError_t prepare_orth();
cudaError_t launch_orth(const OrthCall& c, LearnState* st, void* ws, int n_sms,
                        cudaStream_t stream);

}  // namespace pulsar
