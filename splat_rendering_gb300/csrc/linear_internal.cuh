// What the kernels of a linear layer share: activations, the planes of a float32 operand, rows of
// any length, the tensor cores' descriptors and barriers, and the epilogue; and what its parts
// offer one another.
#pragma once

#include <type_traits>

#include "learn_internal.cuh"
#include "tensor_core.cuh"

namespace pulsar {
namespace linear {

constexpr int kPanel = 64;       // of the contraction, per stage: 128 bytes of a swizzled row
constexpr int kBlock = 128;      // rows of a tile
constexpr int kMaxPlanes = 3;

// ------------------------------------------------------------ activation --
// 1 / (1 + exp(-z)) by the PTX ISA's approximate base-2 exponential and reciprocal, with
// subnormals flushed (below 2^-125, z < -87, zero).  The exponent's product is rounded once, so that
// it is off by (8 + 2 |z|) 2^-24 at most for negative z: z * it was seen to be off by 3 x 2^-24 above
// -1, 5 down to -5, 18 down to -20, 64 at -80, of values that are themselves exp(z).  Five
// instructions; with the product's lower part, 5 x 2^-24 everywhere, seven (1M x 64 -> 64 in 32 bits
// 97 us for 94, its gradients 208 for 204, of an error that is the same in all); as expf() and a
// division 171 and 305.
__device__ __forceinline__ float sigmoid_of(float z) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return s;
}
template <int kAct>
__device__ __forceinline__ float act_of(float z) {
    if (kAct == kActSilu) return z * sigmoid_of(z);
    if (kAct == kActRelu) {   // NaN stays NaN
        float y;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(z), "f"(0.0f));
        return y;
    }
    return z;
}
__device__ __forceinline__ float silu_slope(float z) {
    const float s = sigmoid_of(z);
    return s * (1.0f + z * (1.0f - s));
}
// ---------------------------------------------------------------- planes --
// Two floats as three words of two bfloat16 each, whose sums they are (an infinity, or what rounds
// to one, leaves NaNs over).
__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void split3(float a, float b, uint32_t (&w)[3]) {
    w[0] = pair_bf16(a, b);
    a -= low_of(w[0]);
    b -= high_of(w[0]);
    w[1] = pair_bf16(a, b);
    w[2] = pair_bf16(a - low_of(w[1]), b - high_of(w[1]));
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, float (&v)[8]) {
    constexpr int V = VecOf<T>::n;
    if (vec) {
#pragma unroll
        for (int h = 0; h < 8; h += V) {
            float u[V];
            Pack<T, V>::load(p + h, u);
#pragma unroll
            for (int e = 0; e < V; ++e) v[h + e] = u[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float u[1] = {0.0f};
            if (e < n) Pack<T, 1>::load(p + e, u);
            v[e] = u[0];
        }
    }
}

// kCount consecutive elements at any alignment, from the 16-byte vectors that they lie in.
template <typename T, int kCount>
struct Window {
    static constexpr int kSize = (int)sizeof(T), kVectors = kCount * kSize / 16 + 1;
    uint4 raw[kVectors];
    int shift;   // elements from the first vector's beginning

    __device__ __forceinline__ void load_shared(uint32_t at) {
        shift = (int)(at & 15u) / kSize;
        at &= ~15u;
#pragma unroll
        for (int i = 0; i < kVectors; ++i)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(raw[i].x), "=r"(raw[i].y), "=r"(raw[i].z), "=r"(raw[i].w)
                         : "r"(at + 16 * i));
    }
    // (up to seven elements before p and 16 behind it are read)
    __device__ __forceinline__ void load(const T* p) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        shift = (int)(at & 15u) / kSize;
        const uint4* v = reinterpret_cast<const uint4*>(at & ~(uintptr_t)15);
#pragma unroll
        for (int i = 0; i < kVectors; ++i) raw[i] = v[i];
    }
    __device__ __forceinline__ void open(float (&v)[kCount]) const {
        constexpr int kWords = 4 * kVectors;
        uint32_t w[kWords];
#pragma unroll
        for (int i = 0; i < kVectors; ++i) {
            w[4 * i] = raw[i].x;
            w[4 * i + 1] = raw[i].y;
            w[4 * i + 2] = raw[i].z;
            w[4 * i + 3] = raw[i].w;
        }
        if constexpr (kSize == 4) {
#pragma unroll
            for (int i = 0; i + 2 < kWords; ++i) w[i] = shift & 2 ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i < kCount; ++i) v[i] = __uint_as_float(shift & 1 ? w[i + 1] : w[i]);
        } else {
#pragma unroll
            for (int i = 0; i + 2 < kWords; ++i) w[i] = shift & 4 ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i + 3 < kWords; ++i) w[i] = shift & 2 ? w[i + 1] : w[i];
#pragma unroll
            for (int i = 0; i < kCount / 2; ++i) {
                const uint32_t u = shift & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
                v[2 * i] = low_of(u);
                v[2 * i + 1] = high_of(u);
            }
        }
    }
};

// Eight columns of a row as they were loaded: nothing waits for them before they are opened.
template <typename T>
struct Chunk {
    static constexpr int V = VecOf<T>::n;
    typename Pack<T, V>::Raw raw[8 / V];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int h = 0; h < 8 / V; ++h) raw[h] = Pack<T, V>::raw_last(p + h * V);
    }
    __device__ __forceinline__ void open(float (&v)[8]) const {
#pragma unroll
        for (int h = 0; h < 8 / V; ++h) {
            float u[V];
            Pack<T, V>::open(raw[h], u);
#pragma unroll
            for (int e = 0; e < V; ++e) v[h * V + e] = u[e];
        }
    }
};

// dy made dz = dy act'(z).  (Through ReLU dy passes where z is a NaN: a float32 sum with an
// infinity, whose parts cancel to one, may be that infinity.)
template <int kAct, int V>
__device__ __forceinline__ void to_dz(float (&v)[V], const float (&z)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (kAct == kActRelu) v[e] = z[e] <= 0.0f ? 0.0f : v[e];
        if (kAct == kActSilu) v[e] *= silu_slope(z[e]);
    }
}

// Eight columns, 16 bytes of bfloat16 in each plane.
template <int kPlanes>
__device__ __forceinline__ void put_chunk(void* at, size_t plane_bytes, const float (&v)[8]) {
    uint32_t w[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (kPlanes == 3)
            split3(v[2 * e], v[2 * e + 1], w[e]);
        else
            w[e][0] = pair_bf16(v[2 * e], v[2 * e + 1]);
    }
#pragma unroll
    for (int p = 0; p < kPlanes; ++p)
        *reinterpret_cast<uint4*>(static_cast<unsigned char*>(at) + p * plane_bytes) =
            make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
}

// -------------------------------------------------------- barriers, copies --
// Descriptor of a 128-byte-swizzled operand: `lbo` is the stride between
// 64-element groups along M/N of an MN-major operand (unused when K-major);
// groups of eight rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// One lane of a whole warp, the compiler knowing that it is one: MMAs issued by it follow each
// other at their own rate, while those of a lane that a comparison chose take 105 cycles each
// (measured: M = 128, N = 64: 76 cycles, with A in tensor memory 49; N = 16: 57 and 35).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void expect_bytes(uint64_t* mbar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(mbar)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_init_n(uint64_t* mbar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(mbar)), "r"(n));
}
__device__ __forceinline__ void mbar_arrive(uint64_t* mbar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(mbar)) : "memory");
}
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* mbar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(mbar))
        : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    if (bytes)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool warp_all(bool v) { return __all_sync(0xffffffffu, v); }

// ---------------------------------------------------------------- epilogue --
// What becomes of a product's sums [m, n].
struct Result {
    int64_t m, n;
    // the finished result, or, where there are parts, their sums [splits][m][n]
    const float* bias;
    const void* residual;
    void* pre;
    void* out;
    int act;
    bool vec;       // rows are whole vectors of four, on their alignment
    int splits;     // parts of the contraction
    int64_t part;   // floats from one part's sums to the next
};

// What the epilogue does with 32 columns of a warp's 32 rows, a row in each lane: through the
// warp's exchange in shared memory (float4 chunks, swizzled), after which a lane has four columns
// of every fourth row, and a warp reads the residual and writes whole sectors of eight rows' 32
// columns at a time.
// (The residual's sum is kept apart from the activation's last product: whether z is wanted too
// changes no bits.)
__device__ __forceinline__ float plus(float a, float b) { return __fadd_rn(a, b); }

template <typename T>
struct Four;
template <>
struct Four<float> {
    using Raw = float4;
    static __device__ __forceinline__ void add(const Raw& r, float (&y)[4]) {
        y[0] = plus(y[0], r.x); y[1] = plus(y[1], r.y);
        y[2] = plus(y[2], r.z); y[3] = plus(y[3], r.w);
    }
    static __device__ __forceinline__ Raw pack(const float (&y)[4]) {
        return make_float4(y[0], y[1], y[2], y[3]);
    }
};
template <>
struct Four<__nv_bfloat16> {
    using Raw = uint2;
    static __device__ __forceinline__ void add(const Raw& r, float (&y)[4]) {
        y[0] = plus(y[0], low_of(r.x)); y[1] = plus(y[1], high_of(r.x));
        y[2] = plus(y[2], low_of(r.y)); y[3] = plus(y[3], high_of(r.y));
    }
    static __device__ __forceinline__ Raw pack(const float (&y)[4]) {
        return make_uint2(pair_bf16(y[0], y[1]), pair_bf16(y[2], y[3]));
    }
};

// One element of a result: bias (already in z), pre-activation, activation, residual.
template <typename T, int kAct>
__device__ __forceinline__ void finish1(const Result& q, float z, int64_t at) {
    const float one[1] = {z};
    if (q.pre) Pack<T, 1>::store(static_cast<T*>(q.pre) + at, one);
    float y[1] = {act_of<kAct>(z)};
    if (q.residual) {
        float f[1];
        Pack<T, 1>::load(static_cast<const T*>(q.residual) + at, f);
        y[0] = plus(y[0], f[0]);
    }
    Pack<T, 1>::store(static_cast<T*>(q.out) + at, y);
}
template <typename T>
__device__ __forceinline__ void finish1(const Result& q, float z, int64_t at) {
    if (q.act == kActSilu) finish1<T, kActSilu>(q, z, at);
    else if (q.act == kActRelu) finish1<T, kActRelu>(q, z, at);
    else finish1<T, kActNone>(q, z, at);
}

// A block of 32 rows and 32 (or, kSmall, eight) columns whose sums are in the exchange, where rows
// are no whole vectors: as many lanes to a row as it has columns, so that a warp stores what is
// contiguous.  `first`: its first element, col0: its column.  (kPlain: the sums are the result.)
template <typename T, int kAct, bool kPlain, bool kSmall>
__device__ __forceinline__ void finish_scalar(const Result& q, const float4* x, int64_t col0,
                                              int64_t first, int64_t left_rows, int lane) {
    const int rows = (int)(left_rows < 32 ? left_rows : 32);
    const int64_t left = q.n - col0;
    const int cols = (int)(left < (kSmall ? 8 : 32) ? left : (kSmall ? 8 : 32));
    int log = 0;
    while (1 << log < cols) ++log;
    const int c = lane & ((1 << log) - 1);
    const float* word = reinterpret_cast<const float*>(x) + (c & 3);
    if (c >= cols) return;
    const float b = q.bias ? q.bias[col0 + c] : 0.0f;
    // all loads, then all stores: 25778 x 21 -> 351 in 16 bits 17 us, one by one 32
    constexpr int kBatch = kSmall ? 4 : 8;
    const int step = 32 >> log;
    const int64_t ahead = step * q.n, from = first + (lane >> log) * q.n + c;
    const auto all = [&](auto skip) {
        constexpr bool kSkip = decltype(skip)::value;
        T* out = static_cast<T*>(q.out) + from;
        T* pre = static_cast<T*>(q.pre) + from;
        const T* residual = static_cast<const T*>(q.residual) + from;
#pragma unroll 1
        for (int r0 = lane >> log; r0 < rows; r0 += kBatch * step) {
            float z[kBatch][1], more[kSkip ? kBatch : 1][1];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (kSkip) {
                    more[kSkip ? i : 0][0] = 0.0f;
                    if (r0 + i * step < rows) Pack<T, 1>::load(residual, more[kSkip ? i : 0]);
                    residual += ahead;
                }
                const int r = (r0 + i * step) & 31;
                z[i][0] = plus(word[4 * (kSmall ? r * 2 + ((c >> 2) ^ (r >> 2 & 1))
                                                : r * 8 + ((c >> 2) ^ (r & 7)))], b);
            }
            if (!kPlain && q.pre) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    if (r0 + i * step < rows) Pack<T, 1>::store(pre, z[i]);
                    pre += ahead;
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float y[1] = {act_of<kAct>(z[i][0])};
                if (kSkip) y[0] = plus(y[0], more[kSkip ? i : 0][0]);
                if (r0 + i * step < rows) Pack<T, 1>::store(out, y);
                out += ahead;
            }
        }
    };
    if (!kPlain && q.residual) all(std::true_type());
    else all(std::false_type());
}

// A lane's share of the block of 32 rows from r0 and 32 columns from c0.  kVec: rows are whole
// vectors (four columns at a time), known when compiled: kernels that have the other case's
// instructions too were up to a tenth slower.  kSkip: there is a residual.
template <typename T, bool kVec, bool kSkip>
struct Share {
    using Raw = typename Four<T>::Raw;
    int64_t c, at;   // its first column, and its first element
    int n, rows;     // columns (of four), rows that there are from its first on
    Raw residual[kSkip ? 8 : 1];

    // (at: of the element (r0, c0) in a matrix of q.n columns)
    __device__ __forceinline__ void begin(const Result& q, int64_t r0, int64_t c0, int64_t base,
                                          int lane) {
        c = c0 + 4 * (lane & 7);
        n = (int)(q.n - c < 4 ? q.n - c : 4);
        at = base + (r0 + (lane >> 3)) * q.n + c;
        const int64_t left = q.m - r0 - (lane >> 3);
        rows = n <= 0 ? 0 : (int)(left < 32 ? left : 32);
        if (kSkip && kVec) {
#pragma unroll
            for (int h = 0; h < 8; ++h)
                if (4 * h < rows)
                    residual[kSkip ? h : 0] = __ldcs(reinterpret_cast<const Raw*>(
                        static_cast<const T*>(q.residual) + at + (int64_t)4 * h * q.n));
        }
    }

    __device__ __forceinline__ static void put(float4* x, const float (&v)[32], int lane) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[lane * 8 + (e ^ (lane & 7))] =
                make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        __syncwarp();
    }
    __device__ __forceinline__ static float4 get(const float4* x, int r, int lane) {
        return x[r * 8 + ((lane & 7) ^ (r & 7))];
    }

    // `bias`: of its four columns; r0, c0, base as in begin()
    template <int kAct>
    __device__ __forceinline__ void end(const Result& q, float4* x, const float (&v)[32],
                                        const float (&bias)[4], int64_t r0, int64_t c0,
                                        int64_t base, int lane) {
        T* out = static_cast<T*>(q.out) + at;
        T* pre = q.pre ? static_cast<T*>(q.pre) + at : nullptr;
        const int rq = lane >> 3;
        const int64_t step = 4 * q.n;
        if constexpr (kVec) {
            // (all loads, then all stores: the compiler keeps a load behind a store before it)
            float z[8][4];
            put(x, v, lane);
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const float4 u = get(x, 4 * h + rq, lane);
                z[h][0] = plus(u.x, bias[0]);
                z[h][1] = plus(u.y, bias[1]);
                z[h][2] = plus(u.z, bias[2]);
                z[h][3] = plus(u.w, bias[3]);
            }
            if (pre) {
#pragma unroll
                for (int h = 0; h < 8; ++h)
                    if (4 * h < rows) *reinterpret_cast<Raw*>(pre + h * step) = Four<T>::pack(z[h]);
            }
#pragma unroll
            for (int h = 0; h < 8; ++h) {
#pragma unroll
                for (int e = 0; e < 4; ++e) z[h][e] = act_of<kAct>(z[h][e]);
                if (kSkip) Four<T>::add(residual[kSkip ? h : 0], z[h]);
            }
#pragma unroll
            for (int h = 0; h < 8; ++h)
                if (4 * h < rows) *reinterpret_cast<Raw*>(out + h * step) = Four<T>::pack(z[h]);
        } else {
            put(x, v, lane);
            finish_scalar<T, kAct, false, false>(q, x, c0, base + r0 * q.n + c0, q.m - r0, lane);
        }
    }
    __device__ __forceinline__ void end(const Result& q, float4* x, const float (&v)[32],
                                        const float (&bias)[4], int64_t r0, int64_t c0,
                                        int64_t base, int lane) {
        if (q.act == kActSilu) end<kActSilu>(q, x, v, bias, r0, c0, base, lane);
        else if (q.act == kActRelu) end<kActRelu>(q, x, v, bias, r0, c0, base, lane);
        else end<kActNone>(q, x, v, bias, r0, c0, base, lane);
    }
};

// The same where there is room for an exchange of 32 x 8 words only: eight columns at a time, of
// which a lane has four of every 16th row; a warp stores sectors.  (kPlain: the sums are the result.)
template <typename T, int kAct, bool kPlain, bool kVec>
__device__ __forceinline__ void finish_small(const Result& q, float4* x, const float (&v)[32],
                                             int64_t r0, int64_t c0, int64_t base, int lane) {
    using Raw = typename Four<T>::Raw;
    const int j = lane & 1, rq = lane >> 1;
    const int64_t left = q.m - r0 - rq, at0 = base + (r0 + rq) * q.n + c0 + 4 * j;
    const int rows = (int)(left < 32 ? left : 32);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            x[lane * 2 + (i ^ (lane >> 2 & 1))] =
                make_float4(v[8 * m + 4 * i], v[8 * m + 4 * i + 1], v[8 * m + 4 * i + 2],
                            v[8 * m + 4 * i + 3]);
        __syncwarp();
        const int64_t c = c0 + 8 * m + 4 * j;
        const int n = (int)(q.n - c < 4 ? q.n - c : 4);
        float z[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 16 * h + rq;
            const float4 u = x[r * 2 + (j ^ (r >> 2 & 1))];
            z[h][0] = u.x;
            z[h][1] = u.y;
            z[h][2] = u.z;
            z[h][3] = u.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (kPlain) continue;
            const float bias = q.bias && e < n ? q.bias[c + e] : 0.0f;
            z[0][e] = plus(z[0][e], bias);
            z[1][e] = plus(z[1][e], bias);
        }
        if constexpr (!kVec) {
            finish_scalar<T, kAct, kPlain, true>(q, x, c0 + 8 * m, base + r0 * q.n + c0 + 8 * m,
                                                 q.m - r0, lane);
            continue;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (16 * h >= rows || n <= 0) continue;
            const int64_t at = at0 + 16 * h * q.n + 8 * m;
            if (!kPlain && q.pre)
                *reinterpret_cast<Raw*>(static_cast<T*>(q.pre) + at) = Four<T>::pack(z[h]);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[h][e] = act_of<kAct>(z[h][e]);
            if (!kPlain && q.residual)
                Four<T>::add(*reinterpret_cast<const Raw*>(static_cast<const T*>(q.residual) + at),
                             z[h]);
            *reinterpret_cast<Raw*>(static_cast<T*>(q.out) + at) = Four<T>::pack(z[h]);
        }
    }
}

// ------------------------------------------------------------------- parts --
constexpr int kMostSms = 160;   // of a part: workspaces are sized by it
inline int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }
inline int64_t part_size(int64_t m, int64_t n) { return (m * n + 3) / 4 * 4; }
template <typename T>
bool vec4(const Result& q) {
    const auto aligned = [](const void* p) {
        return (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(T) - 1)) == 0;
    };
    return q.n % 4 == 0 && aligned(q.out) && aligned(q.pre) && aligned(q.residual);
}

// An operand as the products read it: a bfloat16 matrix [planes][rows][pitch].
struct Matrix {
    const __nv_bfloat16* at;
    int64_t rows, cols, pitch;
    size_t plane;
    int planes;
};

// Wide layers (linear_product.cu): a product of any size, q's sums of a(i, c) b(j, c) over k
// values of c; x_mn: the operand's matrix has c as its rows.  Where *pending has more than one part
// they are in `parts` and still to be joined.
size_t product_parts(int planes, int64_t m, int64_t n, int64_t k);   // floats of workspace
cudaError_t prepare_product();
template <typename T>
cudaError_t launch_product(const Result& q, const Matrix& a, bool a_mn, const Matrix& b, bool b_mn,
                           int64_t k, float* parts, Result* pending, LearnState* st, int n_sms,
                           cudaStream_t s);

// Narrow layers (linear_narrow.cu).  The forward call: false where the layer is none.
cudaError_t prepare_narrow();
template <typename T>
bool is_stream(int64_t inputs, int64_t outputs);   // of the forward call
template <typename T>
bool launch_stream(const LinearCall& c, const Result& q, LearnState* st, int n_sms, cudaStream_t s,
                   cudaError_t* e);
template <typename T>
bool is_narrow(int64_t inputs, int64_t outputs);   // of the backward call
template <typename T>
int narrow_parts(int64_t rows, int n_sms);         // sums of dW, [outputs][inputs] each
template <typename T>
cudaError_t launch_narrow(const LinearCall& c, float* parts, float* sums, LearnState* st, int n_sms,
                          cudaStream_t s);

constexpr int64_t kFewRows = 8;   // of the forward call that the products have no part in (linear.cu)

// Layers of a few outputs (linear_few.cu).  The forward call: false where another form is faster.
constexpr int64_t kFewOutputs = 4, kFewInputs = 2048;
bool is_few(int64_t inputs, int64_t outputs);   // of the backward call
int64_t few_parts(int64_t rows, int n_sms);   // at most; sums of dW as above, and of the bias
template <typename T>
bool launch_few(const LinearCall& c, const Result& q, int n_sms, cudaStream_t s,
                cudaError_t* result);
template <typename T>
cudaError_t launch_few_back(const LinearCall& c, float* parts, float* sums, int n_sms, cudaStream_t s,
                            int64_t* blocks);   // how many there are

}  // namespace linear
}  // namespace pulsar
