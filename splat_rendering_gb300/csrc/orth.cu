// Orthogonalisation of an update by Newton-Schulz products:
//
//   X_0 = G / (|G|_F + eps),   X' = P X,   P = a I + b A + c A^2,   A = X X^T
//
// for every matrix of a batch, on the orientation with the fewer rows (the
// result of the transpose is the transpose of the result).  r rows, c columns.
//
// The products run on the tensor cores (tcgen05, fp32 accumulation) on
// operands in half precision: 11 significant bits, eight times closer than
// bfloat16 at the same rate, and powers of two place X, A and P inside its
// narrow range: what the polynomial can make of the largest singular value at
// most is known from step to step (see Scales).  For
// float32 tensors, and tiny ones in 16 bits, every operand is a pair hi + lo of
// halves (22 bits) and a product is hi hi + hi lo + lo hi.  aI is folded into P, so that the last
// product needs nothing but P and X.  A and P are symmetric: only the 128 x
// 128 tiles on and below the diagonal are computed, each written twice.
//
// Matrices lie in panels of 64 columns, a row of a panel being the 128 bytes
// of one swizzled shared-memory row: any run of rows of a panel is one
// contiguous bulk copy, and the same bytes serve as a K-major operand (rows
// are M or N) and as an MN-major one (rows are K).
#include "learn_internal.cuh"
#include "tensor_core.cuh"

#include <cuda_fp16.h>

#include <cmath>
#include <cstring>

namespace pulsar {
namespace {

constexpr int kThreads = 256;
constexpr int kPanel = 64;      // columns of a panel: 128 bytes of halves
constexpr int kBlock = 128;     // rows are padded to it

// ---------------------------------------------------------------- scales --
// No element of a matrix is larger than its largest singular value.  X_0's are at most |X_0|_F;
// from the bound m of X's, A's are at most m^2, P's the largest |q(u)| over 0 <= u <= m^2,
// q(u) = a + b u + c u^2, and those of X' the largest |s q(s^2)| over 0 <= s <= m.  A polynomial
// that grows or shrinks by orders of magnitude would lose sight of the matrix in a few steps: for
// such a one m is lowered to |X|_F, the root of A's trace, once A is known.
// Stored value = value times a power of two that puts its bound into [2^12, 2^13) (X: twice
// that), four times below half's largest and 2^36 above its smallest.
constexpr int kMaxSteps = 100;
constexpr int kMostX = 30, kMostP = 96;   // log2 of the largest bounds that are taken

struct Polynomial {
    float a, b, c;
    // where |q| and |s q(s^2)| have extrema (u; beyond every bound where they have none) and
    // their values
    float u_q, q, u_s[2], s[2];
    bool wild;   // A's traces are needed (0.5 of 24 us at eight 64 x 64)
    __host__ __device__ float at(float u) const { return fabsf(a + u * (b + u * c)); }
    // for the bound u of A's singular values
    __host__ __device__ float most_q(float u) const {
        const float v = fmaxf(fabsf(a), at(u));
        return u_q < u ? fmaxf(v, q) : v;
    }
    __host__ __device__ float most_s(float u) const {
        float v = sqrtf(u) * at(u);
        if (u_s[0] < u) v = fmaxf(v, s[0]);
        return u_s[1] < u ? fmaxf(v, s[1]) : v;
    }
};

Polynomial polynomial(float fa, float fb, float fc, int steps) {
    const double a = fa, b = fb, c = fc;
    const auto value = [&](double u) { return fabs(a + u * (b + u * c)); };
    const auto place = [](double u) { return u > 0.0 && u < 0x1p62 ? (float)u : INFINITY; };
    Polynomial p{fa, fb, fc};
    const double u = -b / (2.0 * c);
    // 5 c u^2 + 3 b u + a = 0 by the form that does not cancel
    const double t = -0.5 * (3.0 * b + copysign(sqrt(9.0 * b * b - 20.0 * a * c), b));
    const double us[2] = {t / (5.0 * c), a / t};
    p.u_q = place(u);
    p.q = p.u_q < INFINITY ? (float)value(u) : 0.0f;
    for (int k = 0; k < 2; ++k) {
        p.u_s[k] = place(us[k]);
        p.s[k] = p.u_s[k] < INFINITY ? (float)(sqrt(us[k]) * value(us[k])) : 0.0f;
    }
    // (where |a| >= 1, small singular values do not shrink)
    p.wild = !(fabs(a) >= 1.0);
    float m = 1.0f;
    for (int k = 0; k < steps && !p.wild; ++k) {
        m = p.most_s(m * m);
        p.wild = !(m <= 2.0f);
    }
    return p;
}

// The smallest e, within the limits, with v < 2^e.
__host__ __device__ __forceinline__ int above(float v, int lo, int hi) {
    int bits;
    memcpy(&bits, &v, 4);
    const int e = (bits >> 23 & 255) - 126;   // (below the limits where v is subnormal)
    return e < lo ? lo : e > hi ? hi : e;
}
__host__ __device__ __forceinline__ float pow2(int e) {   // zero below the normal ones
    const int b = e + 127, bits = (b < 0 ? 0 : b > 254 ? 254 : b) << 23;
    float v;
    memcpy(&v, &bits, 4);
    return v;
}
__host__ __device__ __forceinline__ float times_pow2(float v, int e) {   // (|e| below 252)
    return v * pow2(e >> 1) * pow2(e - (e >> 1));
}
// log2 of the scales for the bounds of X, of X in A = X X^T, and of P
__host__ __device__ __forceinline__ int scale_x(float m) { return 14 - above(m, -112, kMostX + 1); }
__host__ __device__ __forceinline__ int scale_a(float m) {
    return 13 - above(m * m, -126, 2 * kMostX + 2);
}
__host__ __device__ __forceinline__ int scale_p(float q) { return 13 - above(q, -60, kMostP + 1); }

// A trace's part in whole numbers of 2^-10 stored units, rounded up: their sum has no order (and
// that of 128 rows, each below 2^13, no overflow).
__device__ __forceinline__ uint32_t trace_units(float stored) {
    return stored > 0.0f ? __float2uint_ru(stored * 1024.0f) : 0u;
}
// The bound of A, where X's was `m` before A was known, with A's trace.
__device__ __forceinline__ float known_bound(const Polynomial& p, float m, float trace) {
    if (!p.wild || !(m > 0x1p-30f)) return m * m;   // (tiny ones are far from any overflow)
    return fminf(m * m, trace * (1.001f / 1024.0f) * pow2(-scale_a(m)));
}
// The factors of P = p2 (A A) + p1 A + p0 I of stored values, for X's bound m and A's bound u.
struct Factors {
    float p2, p1, p0;
};
__host__ __device__ __forceinline__ Factors factors_p(const Polynomial& p, float m, float u) {
    const int sa = scale_a(m), sp = scale_p(p.most_q(u));
    const int sc = sp - 2 * sa;
    return {times_pow2(p.c, sc < -250 ? -250 : sc), times_pow2(p.b, sp - sa), times_pow2(p.a, sp)};
}
// X's next bound.  (sqrt(u) loses a bound below 2^-63, whose steps are all a X)
__host__ __device__ __forceinline__ float next_bound(const Polynomial& p, float m, float u) {
    return m > 0x1p-30f ? p.most_s(u) : fmaxf(p.most_s(u), m * fabsf(p.a));
}
// The factor of X' = x (P X), whose bound is `next`; the last X' is the result itself.
__host__ __device__ __forceinline__ float factor_x(const Polynomial& p, float m, float u, float next,
                                                   bool last) {
    return times_pow2(1.0f, (last ? 0 : scale_x(next)) - scale_p(p.most_q(u)) - scale_x(m));
}
// The factor of A = X X^T
__host__ __device__ __forceinline__ float factor_a(float m) {
    return pow2(scale_a(m) - 2 * scale_x(m));
}

// Element (row, col) of a matrix of `rows` padded rows, in halves.
__host__ __device__ __forceinline__ size_t panel_at(int64_t row, int64_t col, int64_t rows) {
    const int64_t chunk = (col & (kPanel - 1)) >> 3;
    return (size_t)(((col / kPanel) * rows + row) * kPanel + ((chunk ^ (row & 7)) << 3) + (col & 7));
}

// ------------------------------------------------------------------ norm --
// Sums of squares, a block per chunk of a matrix: of the values, and of the
// values times 2^-80 and 2^80, which are taken where the first overflows or
// is so small that squares were lost below float32's range.
constexpr float kDown = 8.271806125530277e-25f;   // 2^-80
constexpr float kUp = 1.2089258196146292e24f;     // 2^80
constexpr int kNormBlocks = 608;                  // at most, per matrix
constexpr int kNormAhead = 4;                     // vectors a thread has in flight

struct __align__(16) Squares {
    float plain, down, up, pad;
    __device__ __forceinline__ void add(const Squares& s) {
        plain += s.plain;
        down += s.down;
        up += s.up;
    }
};

// What is seldom needed is kept out of line: a launch on chip waits for its instructions, and
// those that it does not run cost it up to 2 us of 16 where they stand between the others.
template <int kN>
__device__ __forceinline__ float sum_of_warps(float v, float* s) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    return v;
}
template <int kN>
__device__ __forceinline__ float sum_of_block(const float* s) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kN / 32; ++w) t += s[w];
    return t;
}
template <int kN>
__device__ __noinline__ void sum_ends(Squares* v, float* s) {
    for (float* f : {&v->down, &v->up}) {
        sum_of_warps<kN>(*f, s);
        __syncthreads();
        *f = sum_of_block<kN>(s);
        __syncthreads();
    }
}
template <int kN = kThreads>
__device__ __forceinline__ Squares block_sum(Squares v) {
    __shared__ float s[kN / 32];
    sum_of_warps<kN>(v.plain, s);
    const bool ends = __syncthreads_or(v.down != 0.0f || v.up != 0.0f);
    Squares t{};
    t.plain = sum_of_block<kN>(s);
    __syncthreads();
    if (ends) {
        t.down = v.down;
        t.up = v.up;
        sum_ends<kN>(&t, s);
    }
    return t;
}

// The scaled sums of a thread's next kNormAhead vectors.
template <typename T, int V>
__device__ __noinline__ Squares squares_ends(const T* __restrict__ m, int64_t vectors, int64_t i,
                                             int64_t step) {
    Squares s{};
    for (int k = 0; k < kNormAhead && i < vectors; ++k, i += step) {
        float v[V], d = 0.0f, u = 0.0f;
        Pack<T, V>::load(m + i * V, v);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            d = fmaf(v[j] * kDown, v[j] * kDown, d);
            u = fmaf(v[j] * kUp, v[j] * kUp, u);
        }
        s.down += d;
        s.up += u;
    }
    return s;
}

// The squares of a matrix's vectors i0, i0 + step, ...  The scaled sums count where the total is
// beyond 2^128 or below 2^-80: a vector of 2^-60 to 2^60 is nothing to the first and cannot be in
// the second, so that theirs are seldom taken.
template <typename T, int V>
__device__ __forceinline__ Squares sum_squares(const T* __restrict__ m, int64_t vectors, int64_t i0,
                                               int64_t step) {
    Squares s{};
    for (int64_t i = i0; i < vectors; i += kNormAhead * step) {
        typename Pack<T, V>::Raw r[kNormAhead];
#pragma unroll
        for (int k = 0; k < kNormAhead; ++k)
            if (i + k * step < vectors) r[k] = Pack<T, V>::raw(m + (i + k * step) * V);
        bool ends = false;
#pragma unroll
        for (int k = 0; k < kNormAhead; ++k) {
            if (i + k * step >= vectors) break;
            float v[V], p = 0.0f;
            Pack<T, V>::open(r[k], v);
#pragma unroll
            for (int j = 0; j < V; ++j) p = fmaf(v[j], v[j], p);
            s.plain += p;
            ends |= !(p >= 0x1p-60f && p <= 0x1p60f);
        }
        if (ends) s.add(squares_ends<T, V>(m, vectors, i, step));
    }
    return s;
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
k_orth_norm(const T* __restrict__ g, int64_t elems, Squares* __restrict__ part) {
    pdl_begin();
    const Squares s = block_sum(
        sum_squares<T, V>(g + (size_t)blockIdx.y * elems, elems / V,
                          (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads));
    if (threadIdx.x == 0) part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// g / (|G|_F + eps) is (g * pre) * inv: pre, a power of two, keeps the norm inside float32's range.
struct Inverse {
    float pre, inv, norm;   // norm: |X_0|_F, or 1 where that is zero or no number
};
__device__ __forceinline__ Inverse norm_inverse(const Squares& s, float eps) {
    const bool down = isinf(s.plain), up = s.plain < kDown;
    // (an eps that would leave the range times 2^80 is all there is beside a norm below 2^-40)
    const float pre = down ? kDown : up && eps < 0x1p40f ? kUp : 1.0f;
    const float unit = up && pre == 1.0f ? kDown : 1.0f;
    const float norm = sqrtf(down ? s.down : up ? s.up : s.plain), sum = norm * unit + eps * pre;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // (zero stays zero without an eps)
    const float bound = norm * inv * unit;
    return {pre, inv, bound > 0.0f ? bound : 1.0f};
}

// The same from a matrix's parts (every thread of the block calls).
__device__ __forceinline__ Inverse inv_norm(const Squares* part, int blocks, float eps) {
    Squares s{};
    for (int i = threadIdx.x; i < blocks; i += kThreads) s.add(part[i]);
    return norm_inverse(block_sum(s), eps);
}

// Eight values as halves, and what their rounding left (kParts 2).
template <int kParts>
__device__ __forceinline__ void halves(const float (&v)[8], uint4 (&h)[kParts]) {
    uint32_t w[kParts][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 p = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        w[0][j] = *reinterpret_cast<const uint32_t*>(&p);
        if (kParts == 2) {
            const float2 f = __half22float2(p);
            const __half2 q = __floats2half2_rn(v[2 * j] - f.x, v[2 * j + 1] - f.y);
            w[kParts - 1][j] = *reinterpret_cast<const uint32_t*>(&q);
        }
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k) h[k] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
}

// X_0 in panels, g [m, n] transposed where it is tall; the padding is zero.
// 2048 x 4096 in 16 bits (16 MB in, 16 MB out): 10.8 us, the norm before it 7.4.
// A thread takes eight columns of a row (V at a time); consecutive threads
// lie along what is contiguous in g.
template <typename T, int kParts, int V>
__global__ void __launch_bounds__(kThreads)
k_orth_start(const T* __restrict__ g, int64_t r, int64_t c, int64_t rp, int64_t cp, bool tall,
             const Squares* __restrict__ part, int parts, float eps, float* __restrict__ bound,
             unsigned long long* __restrict__ trace, __half* __restrict__ x, size_t lo) {
    pdl_begin();
    const Inverse by = inv_norm(part + (size_t)blockIdx.y * parts, parts, eps);
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) bound[(size_t)blockIdx.y * kMaxSteps] = by.norm;
        if (threadIdx.x < kMaxSteps) trace[(size_t)blockIdx.y * kMaxSteps + threadIdx.x] = 0;
    }
    const float inv = by.inv * pow2(scale_x(by.norm));
    const T* m = g + (size_t)blockIdx.y * r * c;
    __half* o = x + (size_t)blockIdx.y * rp * cp;
    // a block takes 128 of what is contiguous in g, four a thread, of eight lines of it
    const int inner = (int)(tall ? rp : cp / 8), lines = (int)(tall ? cp / 8 : rp);
    const int across = (inner + 127) / 128, pieces = across * ((lines + 7) / 8);
    for (int piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
        const int line = piece / across * 8 + (threadIdx.x >> 5);
        const int i0 = piece % across * 128 + (threadIdx.x & 31);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = i0 + 32 * q;
            if (i >= inner || line >= lines) continue;
            const int64_t row = tall ? i : line, c0 = 8 * (int64_t)(tall ? line : i);
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; j += V) {
                float u[V] = {};
                if (row < r && c0 + j < c)
                    Pack<T, V>::load(m + (tall ? (c0 + j) * r + row : row * c + c0 + j), u);
#pragma unroll
                for (int e = 0; e < V; ++e) v[j + e] = u[e] * by.pre * inv;
            }
            uint4 h[kParts];
            halves<kParts>(v, h);
            const size_t at = panel_at(row, c0, rp);
#pragma unroll
            for (int k = 0; k < kParts; ++k) *reinterpret_cast<uint4*>(o + k * lo + at) = h[k];
        }
    }
}

// No step at all: out = g / (|g| + eps).  (`out` may be g.)
template <typename T>
__global__ void __launch_bounds__(kThreads)
k_orth_scale(const T* g, int64_t elems, const Squares* __restrict__ part, int parts, float eps,
             T* out) {
    pdl_begin();
    const Inverse by = inv_norm(part + (size_t)blockIdx.y * parts, parts, eps);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < elems;
         i += (int64_t)gridDim.x * kThreads) {
        float v[1];
        Pack<T, 1>::load(g + (size_t)blockIdx.y * elems + i, v);
        v[0] = v[0] * by.pre * by.inv;
        Pack<T, 1>::store(out + (size_t)blockIdx.y * elems + i, v);
    }
}

// -------------------------------------------------------------- products --
// One kernel for the three products, a persistent CTA per SM.  Roles: one
// thread keeps a ring of operand stages filled with bulk copies, one issues
// the MMAs into one of two accumulators in tensor memory, and eight warps
// drain the other (four per half of the tile's columns, a thread per row):
// sum, scale, round, and store, into panels or, in the last step, as the
// result.
//
// Per 64 of K a tile of 128 x 128 takes 0.30 us, of 128 x 256 0.39 us (86 % of
// the MMAs' rate at the clock of a long run): the width of an MMA counts more
// than the operands' way in (pairs of CTAs on one MMA, with half the operand
// bytes each, took 0.36 us for 256 x 256 and gained nothing overall).  2048 x
// 4096 in 16 bits: A 21 us, P 17, X' 34, of each some 8 us outside the MMAs:
// launch, first operands, the cluster's exchange, stores.
//
// In 32 bits the tensor cores' accumulation, which truncates, would be what
// limits the result: hi hi and the cross terms have accumulators of their
// own, and both are drained and summed in registers every kChunk panels (two;
// of four, 683 x 2967 was 2.0 times as far off as plain 32-bit products, now 1.3
// times, and 1024 x 1024 1.65, now 0.9; 1500 x 509: 142 us, now 147; of one: 152).
//
// Diagonals.  In single halves the roundings of A and P average out but for
// those of their diagonals: where the rows are nearly orthogonal, as they are in
// an oblong matrix, each diagonal's elements are nearly equal, are rounded alike,
// and move every singular value the same way (512 x 8192: the result 1.5 times as
// far off as its own rounding to 16 bits, now 1.06).  So A's diagonal keeps what
// its rounding left (`rest`) for P's, and P's is made exact by a factor per row
// of X' (`rows`, within 2^-11 of 1), for which a row of P counts as scaled: its
// other elements move by less than their own rounding.  It costs 3 of 351 us at
// 2048 x 4096.
//
// Where a product has too few tiles for the SMs (the symmetric ones of a
// small or oblong matrix), a cluster of kCluster CTAs shares a tile: each
// takes a part of K, leaves its sums in shared memory, and finishes a part of
// the columns from all of them, in the order of the CTAs.
struct Product {
    const __half *l, *r;      // left and right operands, hi parts
    size_t l_lo, r_lo;        // halves from a hi part to its lo part
    size_t l_size, r_size;    // halves per matrix of the batch
    int64_t l_rows, r_rows;   // padded rows
    int k_panels;
    int tiles_m;              // row blocks of the product
    int tiles;                // per matrix
    int batch;
    Polynomial poly;
    float* bound;             // [batch][kMaxSteps] X's, of this step and (from X') the next
    unsigned long long* trace;   // [batch][kMaxSteps] A's, of this step (from A)
    bool last;
    // A, P (where there is a C, which is A) or X', C and D in panels
    const __half* c;
    __half* d;
    size_t d_lo, d_size;      // also C's
    int64_t d_rows;
    float *rest, *rows;       // [batch][rows], single halves (see Diagonals)
    // the result, where `out` is given: [r, c] or its transpose, unpadded
    void* out;
    int64_t out_r, out_c;
    bool tall;
    int dtype;
};

constexpr int kProductThreads = 320;   // warps: copies, MMAs, eight of the epilogue
constexpr int kChunk = 2;              // panels of K per drained sum (32 bits)
constexpr int kRowPitch = 33;          // words of a row of a warp's 32 x 32 word exchange

template <bool kSplit, int kN>
struct ProductSmem {
    static constexpr int parts = kSplit ? 2 : 1;
    static constexpr int a = kBlock * kPanel * 2, b = kN * kPanel * 2;
    static constexpr int stage = parts * (a + b);
    static constexpr int exchange_bytes = 8 * 32 * kRowPitch * 4;
    static constexpr int stages = (227 * 1024 - 1024 - exchange_bytes - 256) / stage;
    static constexpr int exchange = stages * stage;
    static constexpr int bars = exchange + exchange_bytes;
    static constexpr int bytes = bars + 256 + 1024;   // and the alignment to 1024
    static_assert(stages >= 2 && (2 * stages + 5) * 8 + 8 <= 256, "shared memory of a product");
    static_assert(stages * stage >= kBlock * kN * 4, "a tile of sums fits the stages");
};

// Descriptor of a 128-byte-swizzled operand: `lbo` is the stride between
// 64-element groups along M/N of an MN-major operand (unused when K-major);
// groups of eight rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void expect_bytes(uint64_t* mbar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(mbar)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* mbar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(mbar))
        : "memory");
}
// Whether any of the epilogue's threads has `v`: one decision for all.
__device__ __forceinline__ bool epilogue_any(bool v) {
    uint32_t any;
    __syncwarp();
    asm volatile(
        "{\n.reg .pred p, r;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred r, 1, 256, p;\n"
        "selp.u32 %0, 1, 0, r;\n}\n"
        : "=r"(any)
        : "r"((uint32_t)v)
        : "memory");
    return any != 0;
}
__device__ __forceinline__ void mbar_init_n(uint64_t* mbar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(mbar)), "r"(n));
}
__device__ __forceinline__ void mbar_arrive(uint64_t* mbar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(mbar)) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t saddr, uint32_t rank) {
    uint32_t at;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(saddr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_cluster(uint32_t saddr, uint32_t rank, const float4& v) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(saddr), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y),
                 "f"(v.z), "f"(v.w)
                 : "memory");
}
// Tile t of a symmetric product in tiles of 128 x 256: row blocks of 128, the
// column blocks up to the diagonal, i / 2 + 1 of them in row block i.
__device__ __forceinline__ void lower_wide(int t, int* i, int* j) {
    // rows 2 a and 2 a + 1 have a + 1 tiles each; a (a + 1) lie before row 2 a
    int a = (int)((sqrtf(4.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while ((a + 1) * (a + 2) <= t) ++a;
    while (a * (a + 1) > t) --a;
    const int rest = t - a * (a + 1);
    *i = 2 * a + (rest > a ? 1 : 0);
    *j = rest > a ? rest - a - 1 : rest;
}

// Tile t of a symmetric product, row blocks i >= j.
__device__ __forceinline__ void lower_tile(int t, int* i, int* j) {
    int row = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while ((row + 1) * (row + 2) / 2 <= t) ++row;
    while (row * (row + 1) / 2 > t) --row;
    *i = row;
    *j = t - row * (row + 1) / 2;
}

// What a row of X' is scaled with for P's diagonal: its value over its rounded one.
// (Not where that is subnormal, whose rounding may be large, or infinite.)
__device__ __forceinline__ float row_factor(float v, float rounded) {
    const float m = fabsf(rounded);
    return m >= 6.103515625e-5f && m <= 65504.0f ? __fdividef(v, rounded) : 1.0f;
}

// C's halves of eight columns added to v.
__device__ __forceinline__ void add_halves(float (&v)[8], const uint4& w, float beta) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[e]));
        v[2 * e] = fmaf(beta, f.x, v[2 * e]);
        v[2 * e + 1] = fmaf(beta, f.y, v[2 * e + 1]);
    }
}

template <bool kSplit, int kN, bool kGram, int kCluster>
__global__ void __launch_bounds__(kProductThreads) __cluster_dims__(kCluster, 1, 1)
k_orth_product(const __grid_constant__ Product q, LearnState* st) {
    using L = ProductSmem<kSplit, kN>;
    constexpr int kParts = L::parts;
    constexpr int kPanels = kN / kPanel;          // of a tile
    constexpr int kMine = kPanels / 2;            // panels of an epilogue thread
    constexpr int kCols = kPanel / kCluster;      // columns of a panel it finishes
    constexpr int kAcc = kSplit ? 2 * kN : kN;    // columns of an accumulator
    static_assert(2 * kAcc <= 512, "tensor memory");
    extern __shared__ unsigned char raw[];
    unsigned char* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bars);
    uint64_t* empty = full + L::stages;
    uint64_t* acc_full = empty + L::stages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* s_taddr = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* s_fail = s_taddr + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < L::stages; ++s) {
            mbar_init(full + s);
            mbar_init(empty + s);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + s);
            mbar_init_n(acc_empty + s, 8);
        }
        mbar_init(drain);
        *s_fail = 0u;
        fence_async_smem();
    }
    if (warp == 1) tmem_alloc(s_taddr, 2 * kAcc);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_taddr;
    pdl_next();
    pdl_begin();
    const int total = q.tiles * q.batch;
    const uint32_t rank = kCluster > 1 ? cluster_rank() : 0u;
    const int first = blockIdx.x / kCluster, step = gridDim.x / kCluster;
    const int k0 = (int)(rank * (uint32_t)q.k_panels / kCluster);
    const int k1 = (int)((rank + 1) * (uint32_t)q.k_panels / kCluster);
    const int chunk = kSplit ? kChunk : k1 - k0;
    auto place = [&](int t, int* z, int* i, int* j) {
        *z = t / q.tiles;
        t -= *z * q.tiles;
        if (kGram) {
            if (kN == kBlock)
                lower_tile(t, i, j);
            else
                lower_wide(t, i, j);
        } else {
            *i = t % q.tiles_m;   // neighbours share the columns of X
            *j = t / q.tiles_m;
        }
    };
    bool met = false;   // this thread was at the cluster's first meeting: all sums are written
    // ---- what an epilogue thread owns: a row of the tile, the columns of its panels
    const int group = (warp - 2) >> 2, quarter = warp & 3;   // (epilogue warps are 2 .. 9)
    const int row = quarter * 32 + lane;
    // columns col .. col + kCols - 1 of the tile from their finished sums
    using CHalves = uint4[kCols / 8][kParts];
    auto finish = [&](int z, int i, int j, int col, const CHalves& c, float alpha, float beta,
                      float gamma, float rest, float (&v)[kCols]) {
        const int64_t grow = (int64_t)i * kBlock + row, gcol = (int64_t)j * kN + col;
        const int jb = j * (kN / kBlock) + col / kBlock;   // the columns' block of 128
        if (kGram && jb > i) return;   // above the diagonal: the mirrored block's
        __half* d = q.d + z * q.d_size;
        // col begins a run of kCols inside one panel: its row of 64 halves, and mirrored
        // the run's rows in the panel of this thread's column (the warp's are adjacent)
        __half* line = d + ((gcol / kPanel) * q.d_rows + grow) * kPanel;
        __half* column = d + ((grow / kPanel) * q.d_rows + gcol) * kPanel + (row & 7);
        const int chunk0 = (int)(gcol & (kPanel - 1)) >> 3, rchunk = (row & (kPanel - 1)) >> 3;
        const int on = i == jb ? row - col % kBlock : -1;   // the diagonal's place in them
        float exact = 0.0f, rounded = 0.0f;                 // its value, where it is here
#pragma unroll
        for (int b = 0; b < kCols / 8; ++b) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = alpha * v[8 * b + e];
            if (kGram && q.c) {
#pragma unroll
                for (int p = 0; p < kParts; ++p) add_halves(w, c[b][p], beta);
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] += 8 * b + e == on ? gamma : 0.0f;
                if (!kSplit && i == jb) {
                    const __half* e16 = reinterpret_cast<const __half*>(&c[b][0]);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[e] += 8 * b + e == on
                                    ? rest * (beta + 2.0f * alpha * __half2float(e16[e]))
                                    : 0.0f;
                }
            }
            uint4 h[kParts];
            halves<kParts>(w, h);
            if (kGram && i == jb) {
                const __half* e16 = reinterpret_cast<const __half*>(&h[0]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    exact = 8 * b + e == on ? w[e] : exact;
                    if (!kSplit) rounded = 8 * b + e == on ? __half2float(e16[e]) : rounded;
                }
            }
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                *reinterpret_cast<uint4*>(line + p * q.d_lo + (((chunk0 + b) ^ (row & 7)) << 3)) =
                    h[p];
                if (kGram && i != jb) {
                    const __half* e16 = reinterpret_cast<const __half*>(&h[p]);
                    __half* m = column + p * q.d_lo + 8 * b * kPanel;
#pragma unroll
                    for (int e = 0; e < 8; ++e) m[e * kPanel + ((rchunk ^ e) << 3)] = e16[e];
                }
            }
        }
        if (kGram && !kSplit && on >= 0 && on < kCols)
            (q.c ? q.rows : q.rest)[z * q.d_rows + grow] =
                q.c ? row_factor(exact, rounded) : exact - rounded;
        if (kGram && !q.c && q.poly.wild && i == jb) {   // (`exact` is zero off the diagonal)
            const uint32_t t = __reduce_add_sync(0xffffffffu, trace_units(exact));
            if (lane == 0 && t) atomicAdd(q.trace + (size_t)z * kMaxSteps, (unsigned long long)t);
        }
    };

    // a panel of the result from its sums: through the warp's exchange, so that
    // a warp writes whole rows (of the transpose, whole columns as they are)
    auto store_result = [&](int z, int i, int j, int col, float alpha, const float (&v)[kPanel]) {
        const int64_t r0 = (int64_t)i * kBlock + quarter * 32, c0 = (int64_t)j * kN + col;
        const size_t base = (size_t)z * q.out_r * q.out_c;
        if (q.tall) {
            if (r0 + lane >= q.out_r) return;
            const size_t at = base + c0 * q.out_r + r0 + lane;
            const int n = (int)min((int64_t)kPanel, q.out_c - c0);
#pragma unroll
            for (int e = 0; e < kPanel; ++e) {
                if (e >= n) continue;
                const float y = alpha * v[e];
                if (q.dtype == kF32)
                    static_cast<float*>(q.out)[at + e * q.out_r] = y;
                else
                    static_cast<__nv_bfloat16*>(q.out)[at + e * q.out_r] = __float2bfloat16_rn(y);
            }
            return;
        }
        uint32_t* x = reinterpret_cast<uint32_t*>(smem + L::exchange) + (warp - 2) * 32 * kRowPitch;
        const int rows = (int)min((int64_t)32, q.out_r - r0);
        if (q.dtype == kF32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    x[lane * kRowPitch + e] = __float_as_uint(alpha * v[32 * h + e]);
                __syncwarp();
                if (c0 + 32 * h + lane < q.out_c) {
                    float* o = static_cast<float*>(q.out) + base + r0 * q.out_c + c0 + 32 * h + lane;
                    for (int e = 0; e < rows; ++e, o += q.out_c)
                        *o = __uint_as_float(x[e * kRowPitch + lane]);
                }
            }
        } else {   // two columns a word
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const __nv_bfloat162 h =
                    __floats2bfloat162_rn(alpha * v[2 * e], alpha * v[2 * e + 1]);
                x[lane * kRowPitch + e] = *reinterpret_cast<const uint32_t*>(&h);
            }
            __syncwarp();
            const int64_t c = c0 + 2 * lane;
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(q.out) + base + r0 * q.out_c + c;
            const bool words = q.out_c % 2 == 0 && (reinterpret_cast<uintptr_t>(q.out) & 3u) == 0;
            for (int e = 0; e < rows; ++e, o += q.out_c) {
                const uint32_t u = x[e * kRowPitch + lane];
                const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&u);
                if (words) {
                    if (c < q.out_c) *reinterpret_cast<uint32_t*>(o) = u;
                } else {
                    if (c < q.out_c) o[0] = h.x;
                    if (c + 1 < q.out_c) o[1] = h.y;
                }
            }
        }
    };

    if (warp == 0) {
        if (lane == 0) {   // ---- copies
            int n = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += step) {
                int z, i, j;
                place(t, &z, &i, &j);
                const __half* l = q.l + z * q.l_size + (size_t)i * kBlock * kPanel;
                const __half* r = q.r + z * q.r_size +
                                  (kGram ? (size_t)j * kN * kPanel
                                         : (size_t)j * kPanels * q.r_rows * kPanel);
                for (int k = k0; k < k1; ++k, ++n) {
                    const int s = n % L::stages;
                    ok = mbar_wait(empty + s, ((n / L::stages) & 1) ^ 1) && !*s_fail;
                    if (!ok) break;
                    unsigned char* dst = smem + s * L::stage;
                    expect_bytes(full + s, L::stage);
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
                        bulk_copy(dst + p * L::a, l + p * q.l_lo + (size_t)k * q.l_rows * kPanel,
                                  L::a, full + s);
                    dst += kParts * L::a;
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        const __half* b = r + p * q.r_lo;
                        if (kGram) {
                            bulk_copy(dst + p * L::b, b + (size_t)k * q.r_rows * kPanel, L::b,
                                      full + s);
                        } else {   // 64 rows of each of the tile's panels
#pragma unroll
                            for (int c = 0; c < kPanels; ++c)
                                bulk_copy(dst + p * L::b + c * kPanel * kPanel * 2,
                                          b + ((size_t)c * q.r_rows + (size_t)k * kPanel) * kPanel,
                                          kPanel * kPanel * 2, full + s);
                        }
                    }
                }
            }
            if (!ok) {   // give the copies in flight one more bounded wait
                *s_fail = 1u;
                for (int k = n > L::stages ? n - L::stages : 0; k < n; ++k)
                    mbar_wait(full + k % L::stages, (k / L::stages) & 1);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {   // ---- MMAs
            constexpr uint32_t idesc = (1u << 4) | (kGram ? 0u : 1u << 16) |
                                       ((uint32_t)(kN >> 3) << 17) |
                                       ((uint32_t)(kBlock >> 4) << 24);
            const uint32_t base = smem_u32(smem);
            int n = 0, it = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += step) {
                for (int kc = k0; kc < k1 && ok; kc += chunk, ++it) {
                    const int buf = it & 1, ke = min(kc + chunk, k1);
                    const uint32_t d = tmem + buf * kAcc;
                    ok = mbar_wait(acc_empty + buf, ((it >> 1) & 1) ^ 1) && !*s_fail;
                    if (!ok) break;
                    tc_fence_after();
                    for (int k = kc; k < ke; ++k, ++n) {
                        const int s = n % L::stages;
                        ok = mbar_wait(full + s, (n / L::stages) & 1) && !*s_fail;
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t at = base + s * L::stage;
                        uint64_t a[kParts], b[kParts];
#pragma unroll
                        for (int p = 0; p < kParts; ++p) {
                            a[p] = desc_sw128(at + p * L::a, 16);
                            b[p] = desc_sw128(at + kParts * L::a + p * L::b,
                                              kGram ? 16 : kPanel * kPanel * 2);
                        }
#pragma unroll
                        for (int e = 0; e < kPanel / 16; ++e) {
                            // 16 of K: 32 bytes along a K-major row, 16 rows of an MN-major operand
                            const uint32_t ea = 32u * e >> 4, eb = kGram ? ea : (2048u * e >> 4);
                            const uint32_t more = k > kc || e > 0;
                            mma_f16(d, a[0] + ea, b[0] + eb, idesc, more);
                            if (kSplit) {
                                mma_f16(d + kN, a[0] + ea, b[kParts - 1] + eb, idesc, more);
                                mma_f16(d + kN, a[kParts - 1] + ea, b[0] + eb, idesc, 1);
                            }
                        }
                        mma_commit(empty + s);
                    }
                    if (ok) mma_commit(acc_full + buf);
                }
            }
            if (!ok) {
                *s_fail = 1u;
                mma_commit(drain);
                mbar_wait(drain, 0);
            }
        }
    } else {   // ---- epilogue
        int it = 0;
        for (int t = first; t < total; t += step) {   // (once, where a cluster shares the tile)
            int z, i, j;
            place(t, &z, &i, &j);
            CHalves c[kGram ? kMine : 1];   // C of the columns this thread finishes, loaded early
            if (kGram && q.c) {
                const __half* cz = q.c + z * q.d_size;
#pragma unroll
                for (int m = 0; m < kMine; ++m)
#pragma unroll
                    for (int b = 0; b < kCols / 8; ++b)
#pragma unroll
                        for (int p = 0; p < kParts; ++p)
                            c[kGram ? m : 0][b][p] = *reinterpret_cast<const uint4*>(
                                cz + p * q.d_lo +
                                panel_at((int64_t)i * kBlock + row,
                                         (int64_t)j * kN + (group * kMine + m) * kPanel +
                                             rank * kCols + 8 * b,
                                         q.d_rows));
            }
            float* const bound = q.bound + (size_t)z * kMaxSteps;
            float alpha, beta = 0.0f, gamma = 0.0f;
            if (kGram && !q.c) {
                alpha = factor_a(*bound);
            } else {
                const float m = *bound;
                const float u =
                    known_bound(q.poly, m, __ull2float_ru(q.trace[(size_t)z * kMaxSteps]));
                if (kGram) {
                    const Factors f = factors_p(q.poly, m, u);
                    alpha = f.p2;
                    beta = f.p1;
                    gamma = f.p0;
                } else {
                    const float next = next_bound(q.poly, m, u);
                    alpha = factor_x(q.poly, m, u, next, q.last);
                    if (!q.last && i == 0 && j == 0 && tid == 64) bound[1] = next;
                }
            }
            if (!kSplit && !kGram) alpha *= q.rows[z * q.d_rows + (int64_t)i * kBlock + row];
            const float rest = kGram && !kSplit && q.c
                                   ? q.rest[z * q.d_rows + (int64_t)i * kBlock + row] : 0.0f;
            float v[kPanel];
            bool ok = true;
            if (kSplit) {
#pragma unroll
                for (int e = 0; e < kPanel; ++e) v[e] = 0.0f;
                for (int kc = k0; kc < k1; kc += chunk, ++it) {
                    const int buf = it & 1;
                    ok = mbar_wait(acc_full + buf, (it >> 1) & 1) && !*s_fail;
                    ok = !epilogue_any(!ok);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t acc = tmem + buf * kAcc + ((uint32_t)(quarter * 32) << 16) +
                                         group * kPanel;
#pragma unroll
                    for (int h = 0; h < kPanel; h += 16) {
                        uint32_t u[16], w[16];
                        tmem_ld16(acc + h, u);
                        tmem_ld16(acc + kN + h, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            v[h + e] += __uint_as_float(u[e]) + __uint_as_float(w[e]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty + buf);
                }
            } else {
                ok = mbar_wait(acc_full + (it & 1), (it >> 1) & 1) && !*s_fail;
                ok = !epilogue_any(!ok);
                tc_fence_after();
            }
            if (!ok) {
                *s_fail = 1u;
                break;
            }
#pragma unroll 1
            for (int m = 0; m < kMine; ++m) {
                const int col = (group * kMine + m) * kPanel;
                if (!kSplit) {
                    const uint32_t acc = tmem + (it & 1) * kAcc +
                                         ((uint32_t)(quarter * 32) << 16) + col;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t u[32];
                        __syncwarp();
                        tmem_ld32(acc + 32 * h, u);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[32 * h + e] = __uint_as_float(u[e]);
                    }
                    if (m + 1 == kMine) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(acc_empty + (it & 1));
                        ++it;
                    }
                }
                if (kCluster > 1) {   // the stages are free: every MMA of this CTA is complete
                    float4* sums = reinterpret_cast<float4*>(smem);   // [column / 4][row]
#pragma unroll
                    for (int e = 0; e < kPanel; e += 4)
                        sums[(col + e) / 4 * kBlock + row] =
                            make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                } else if (kGram || !q.out) {
                    float w[kCols];
#pragma unroll
                    for (int e = 0; e < kCols; ++e) w[e] = v[e % kPanel];
                    // (one panel where there is a C)
                    finish(z, i, j, col, c[0], alpha, beta, gamma, rest, w);
                } else {   // the result
                    store_result(z, i, j, col, alpha, v);
                }
            }
            if (kCluster > 1) {
                __syncwarp();
                cluster_sync();
                met = true;
#pragma unroll
                for (int m = 0; m < kMine; ++m) {
                    float w[kCols];
#pragma unroll
                    for (int e = 0; e < kCols; ++e) w[e] = 0.0f;
                    const int col = (group * kMine + m) * kPanel + (int)rank * kCols;
                    const uint32_t at = smem_u32(smem) + (uint32_t)((col / 4 * kBlock + row) * 16);
#pragma unroll
                    for (int s = 0; s < kCluster; ++s)
#pragma unroll
                        for (int e = 0; e < kCols; e += 4) {
                            const float4 u = ld_cluster(at + e / 4 * kBlock * 16, s);
                            w[e] += u.x;
                            w[e + 1] += u.y;
                            w[e + 2] += u.z;
                            w[e + 3] += u.w;
                        }
                    finish(z, i, j, col, c[kGram ? m : 0], alpha, beta, gamma, rest, w);
                }
            }
        }
    }
    __syncwarp();
    // the other CTAs of the cluster still read this one's sums
    if (kCluster > 1) {
        if (!met) cluster_sync();
        __syncwarp();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *s_fail) atomicOr(&st->error, kErrTimeout);
    if (warp == 1) tmem_dealloc(tmem, 2 * kAcc);
}

// ----------------------------------------------------------- small matrices --
// A matrix of up to 128 rows whose X and A fit the shared memory of one SM, or
// of the SMs of a cluster: one launch takes it through all steps, X, A and P
// never leaving the SMs (P overwrites A, X' overwrites X: a product is
// complete before its epilogue writes, and an epilogue thread reads no row but
// its own).  The CTAs of a cluster have the columns of X in equal shares of
// whole panels; each makes its share of A = X X^T, adds up a part of all
// shares, in the order of the CTAs, for everybody, and goes on with the same A
// and its own columns.  Bound by latency: a step of a 64 x 64 matrix takes 4.2
// us (MMAs 1.7, epilogues and their barriers 2.5), eight of them 24 us in 32
// bits; 10 x 3000 on eight CTAs 59 us, 128 x 2000 88 us (by separate products:
// 117).
//
// The diagonals D_A of A and D_P of P stay in 32 bits and out of the operands:
// with O = A - D_A, A^2 = O^2 + D_A O + O D_A + D_A^2, and X' = D_P X + (P - D_P) X.
// What the tensor cores truncate and the operands round is then relative to the
// rest: 35 x 1330 in 32 bits 4.9e-6 -> 0.7e-6 from the exact result, 64 x 64
// 1.9e-6 -> 0.5e-6 (32-bit library products: 1.8e-6 and 1.2e-6), for 2 of 24 us.
//
// Panels hold rn rows, a panel's lo part behind its hi part: as a K-major right
// operand the two are one of 2 rn rows, and the product of a hi panel with
// both is one MMA (an MMA takes 50 ns here whatever its N).  An MMA's 128 rows
// reach past a panel into what follows, which only makes rows of the product
// that nobody reads.  Sixteen warps share an epilogue: a thread has a row and
// every fourth 16 of the columns.
constexpr int kSmallThreads = 512;
constexpr int kSmallGroups = kSmallThreads / 128;
constexpr int kKnownSteps = 16;

struct StepFactors {
    Factors p;
    float a, x;   // of A and of X'
};
struct Held {   // in shared memory
    float m, u;   // bounds of X and A, where they have to be worked out
    StepFactors of[kMaxSteps];
};

struct Small {
    int r, c, rn;          // rn: padded to 16
    int xp, ap;            // panels of a CTA's share of X, and of A
    int ctas;              // of the cluster
    bool tall;
    int steps;
    Polynomial poly;
    float eps;
    // the factors where |X_0|_F is 1 or little less and the traces are not needed, as nearly always
    bool known;
    StepFactors of[kKnownSteps];
};
constexpr int kMaxShares = 8;
// K of a sum in tensor memory (as kChunk).  Pairs: of 256, 128 x 2000 was 1.25
// times as far off as plain 32-bit products, now 0.5 (85 us, now 87).
constexpr int small_chunk(bool split) { return split ? 128 : 256; }

// A and P; before them, where there is a cluster, a CTA's share of A in 32 bits.
__host__ __device__ inline uint32_t small_a_bytes(int parts, int rn, int ap, int ctas) {
    const uint32_t a = (uint32_t)(parts * ap * rn * 128), sums = (uint32_t)(rn * rn * 4);
    return ctas > 1 && sums > a ? (sums + 1023) / 1024 * 1024 : a;
}
size_t small_bytes(int parts, int rn, int xp, int ap, int ctas) {
    return (size_t)parts * xp * rn * 128 + small_a_bytes(parts, rn, ap, ctas) +
           (kBlock - 16) * 128 + 64 + 1024;
}

constexpr int kScaler = kSmallThreads / 32 - 1;   // the warp that works out factors
// Those of every step, a lane a step, where no trace is needed but |X_0|_F is small.
__device__ __noinline__ void scale_steps(const Polynomial& p, float m, int steps, StepFactors* of) {
    for (int at = 0, k = threadIdx.x & 31; k < steps; k += 32) {
        for (; at < k; ++at) m = next_bound(p, m, m * m);
        const float u = m * m;
        of[k] = {factors_p(p, m, u), factor_a(m),
                 factor_x(p, m, u, next_bound(p, m, u), k + 1 == steps)};
    }
}
// A step's of P, by a warp while the others wait for A A, and of X' and the next A, by a thread
// while they wait for P X.
__device__ __noinline__ void scale_p_step(const Polynomial& p, const float* a_diag, int rn, int step,
                                          Held* held) {
    uint32_t t = 0u;
    for (int i = threadIdx.x & 31; i < rn; i += 32) t += trace_units(a_diag[i]);
    const float m = held->m, u = known_bound(p, m, (float)__reduce_add_sync(0xffffffffu, t));
    if ((threadIdx.x & 31) == 0) {
        held->of[step].p = factors_p(p, m, u);
        held->u = u;
    }
}
__device__ __noinline__ void scale_x_step(const Polynomial& p, int step, int steps, Held* held) {
    const float m = held->m, u = held->u, next = next_bound(p, m, u);
    held->of[step].x = factor_x(p, m, u, next, step + 1 == steps);
    if (step + 1 < steps) held->of[step + 1].a = factor_a(next);
    held->m = next;
}

// kWild: poly.wild.
template <typename T, bool kSplit, int V, bool kWild>
__global__ void __launch_bounds__(kSmallThreads, 1)
k_orth_small(const T* grad, const __grid_constant__ Small q, T* out, LearnState* st) {
    constexpr int kParts = kSplit ? 2 : 1;
    extern __shared__ unsigned char raw[];
    __shared__ Squares s_norm;
    unsigned char* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t pb = (uint32_t)q.rn * 128u;   // bytes of a part of a panel
    unsigned char* xs = smem;
    unsigned char* as = smem + kParts * q.xp * pb;
    // the diagonals of A and P, in the room that the MMAs' unused rows reach into
    float* a_diag = reinterpret_cast<float*>(as + small_a_bytes(kParts, q.rn, q.ap, q.ctas));
    float* p_diag = a_diag + kBlock;
    Held* held = reinterpret_cast<Held*>(p_diag + kBlock);
    static_assert(2 * kBlock * 4 + sizeof(Held) <= (kBlock - 16) * 128, "room for the factors");
    uint64_t* mbar = reinterpret_cast<uint64_t*>(as + small_a_bytes(kParts, q.rn, q.ap, q.ctas) +
                                                 (kBlock - 16) * 128);
    uint32_t* s_taddr = reinterpret_cast<uint32_t*>(mbar + 2);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int quarter = warp & 3, group = warp >> 2;
    const int row = quarter * 32 + lane;
    const bool shared = q.ctas > 1;
    const int rank = (int)blockIdx.x % q.ctas;
    if (tid == 0) {
        mbar_init(mbar);
        mbar_init(mbar + 1);
        fence_async_smem();
    }
    if (warp == 0) tmem_alloc(s_taddr, 512);
    pdl_begin();
    const size_t elems = (size_t)q.r * q.c;
    const T* g = grad + blockIdx.x / q.ctas * elems;
    // this CTA's columns of X, and of those that the matrix has, padded to 16
    const int col0 = rank * q.xp * kPanel;
    const int mine = max(0, min(q.xp * kPanel, q.c - col0)), cn = (mine + 15) / 16 * 16;
    {   // (any share of the elements serves the norm)
        const Squares sq = block_sum<kSmallThreads>(
            sum_squares<T, V>(g, (int64_t)(elems / V), rank * kSmallThreads + tid,
                              kSmallThreads * q.ctas));
        if (tid == 0) s_norm = sq;
    }
    Squares sq{};
    if (shared) {
        __syncwarp();
        cluster_sync();
        for (int k = 0; k < q.ctas; ++k) {
            const float4 u = ld_cluster(smem_u32(&s_norm), k);
            sq.add(Squares{u.x, u.y, u.z, 0.0f});
        }
    } else {
        __syncthreads();
        sq = s_norm;
    }
    const Inverse by = norm_inverse(sq, q.eps);
    const bool known = !kWild && q.known && by.norm >= 0.5f;
    const float inv = by.inv * pow2(scale_x(known ? 1.0f : by.norm));
    if (known) {
        constexpr int kEach = sizeof(StepFactors) / 4;
        if (tid < q.steps * kEach)
            reinterpret_cast<float*>(held->of)[tid] = reinterpret_cast<const float*>(q.of)[tid];
    } else if (kWild && tid == 0) {
        held->m = by.norm;
        held->of[0].a = factor_a(by.norm);
    } else if (!kWild && warp == kScaler) {
        scale_steps(q.poly, by.norm, q.steps, held->of);
    }
#pragma unroll 4
    for (int i = tid; i < q.rn * q.xp * 8; i += kSmallThreads) {
        const int xr = q.tall ? i % q.rn : i / (q.xp * 8);
        const int l0 = (q.tall ? i / q.rn : i % (q.xp * 8)) * 8, c0 = col0 + l0;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; j += V) {
            float u[V] = {};
            if (xr < q.r && c0 + j < q.c)
                Pack<T, V>::load(g + (q.tall ? (size_t)(c0 + j) * q.r + xr
                                             : (size_t)xr * q.c + c0 + j), u);
#pragma unroll
            for (int e = 0; e < V; ++e) v[j + e] = u[e] * by.pre * inv;
        }
        uint4 h[kParts];
        halves<kParts>(v, h);
#pragma unroll
        for (int p = 0; p < kParts; ++p)
            *reinterpret_cast<uint4*>(xs + l0 / kPanel * kParts * pb + p * pb +
                                      panel_at(xr, l0 % kPanel, q.rn) * 2) = h[p];
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_taddr;
    const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t x0 = smem_u32(xs), a0 = smem_u32(as);
    const bool busy = quarter * 32 < q.rn;   // this warp has rows
    uint32_t ph[2] = {0u, 0u};
    bool ok = true;
    // D = the rows of the panels at l times the operand at r, K = 16 ks: hi times hi in the
    // columns at d, the cross terms in those at x.  mn: r's rows are K (X), not columns of D.
    auto issue = [&](int buf, uint32_t d, uint32_t x, uint32_t l, uint32_t r, int n, int k_begin,
                     int k_end, bool mn) {
        const auto idesc = [&](int columns) {
            return (1u << 4) | (mn ? 1u << 16 : 0u) | ((uint32_t)(columns >> 3) << 17) |
                   ((uint32_t)(kBlock >> 4) << 24);
        };
        const uint32_t lbo = mn ? kParts * pb : 16;
        for (int k = k_begin; k < k_end; ++k) {
            const uint32_t ka = (uint32_t)(k >> 2) * kParts * pb + (uint32_t)(k & 3) * 32u;
            const uint32_t kb = mn ? (uint32_t)k * 2048u : ka;
            const uint64_t hi = desc_sw128(l + ka, 16), rhi = desc_sw128(r + kb, lbo);
            const uint32_t more = k > k_begin;
            if (!kSplit) {
                mma_f16(tmem + d, hi, rhi, idesc(n), more);
                continue;
            }
            if (mn) {
                mma_f16(tmem + d, hi, rhi, idesc(n), more);
                mma_f16(tmem + x, hi, desc_sw128(r + pb + kb, lbo), idesc(n), more);
            } else {   // (x is d + n)
                mma_f16(tmem + d, hi, rhi, idesc(2 * n), more);
            }
            mma_f16(tmem + x, desc_sw128(l + pb + ka, 16), rhi, idesc(n), 1);
        }
        mma_commit(mbar + buf);
    };
    auto await = [&](int buf) {   // one decision for all
        ok = __syncthreads_and(mbar_wait(mbar + buf, ph[buf] & 1));
        ++ph[buf];
        tc_fence_after();
        return ok;
    };
    // sixteen columns of this row of D
    auto sums = [&](uint32_t d, uint32_t x, float (&v)[16]) {
        uint32_t u[16], w[16];
        __syncwarp();
        tmem_ld16(trow + d, u);
        if (kSplit) tmem_ld16(trow + x, w);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
            v[e] = kSplit ? __uint_as_float(u[e]) + __uint_as_float(w[e]) : __uint_as_float(u[e]);
    };
    auto put = [&](unsigned char* m, int col, const float (&v)[16]) {
        if (row >= q.rn) return;
        m += col / kPanel * kParts * pb;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = v[8 * b + e];
            uint4 h[kParts];
            halves<kParts>(w, h);
#pragma unroll
            for (int p = 0; p < kParts; ++p)
                *reinterpret_cast<uint4*>(m + p * pb + panel_at(row, col % kPanel + 8 * b, q.rn) * 2) =
                    h[p];
        }
    };
    // sixteen columns of this row without the diagonal's element, which goes to `diag`
    auto off_diagonal = [&](float* diag, int col, float (&v)[16]) {
        float d = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            d = col + e == row ? v[e] : d;
            v[e] = col + e == row ? 0.0f : v[e];
        }
        if (row >= col && row < min(col + 16, q.rn)) diag[row] = d;
    };
    auto ready = [&]() {   // what the threads wrote is ready for the next product
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    // the result's element (r, c): in the bytes that were X's there, a float in those of a pair
    const auto staged = [&](int r, int c) {
        const int part = sizeof(T) == 4 ? c >> 2 & 1 : 0, in = sizeof(T) == 4 ? c & 3 : c & 7;
        return reinterpret_cast<T*>(xs + (c / kPanel * kParts + part) * pb +
                                    panel_at(r, c % kPanel & ~7, q.rn) * 2) + in;
    };
    // a thread's units of 16 columns of A: group, group + 4
    const int r_units = q.rn / 16, r_mine = (r_units + kSmallGroups - 1 - group) / kSmallGroups;
    constexpr int kMost = 128 / 16 / kSmallGroups;
    // (a CTA that gave up skips the work but not the cluster's meetings)
    for (int step = 0; step < q.steps && (ok || shared); ++step) {
        // ---- A = X X^T, in chunks of K through two accumulators
        float acc[kMost][16];
#pragma unroll
        for (int m = 0; m < kMost; ++m)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[m][e] = 0.0f;
        const int ks = cn / 16, per = small_chunk(kSplit) / 16, chunks = (ks + per - 1) / per;
        if (ok && tid == 0 && chunks > 0)
            issue(0, 0, q.rn, x0, x0, q.rn, 0, min(per, ks), false);
        for (int ch = 0; ch < chunks && ok; ++ch) {
            if (tid == 0 && ch + 1 < chunks)
                issue((ch + 1) & 1, 256 * ((ch + 1) & 1), 256 * ((ch + 1) & 1) + q.rn, x0, x0, q.rn,
                      (ch + 1) * per, min((ch + 2) * per, ks), false);
            if (!await(ch & 1)) break;
            if (busy) {
#pragma unroll
                for (int m = 0; m < kMost; ++m) {
                    if (m < r_mine) {
                        float v[16];
                        const uint32_t at = 256 * (ch & 1) + 16 * (group + kSmallGroups * m);
                        sums(at, at + q.rn, v);
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[m][e] += v[e];
                    }
                }
            }
            tc_fence_before();
            if (ch + 2 < chunks) __syncthreads();   // its accumulator is refilled next
            tc_fence_after();
        }
        if (shared) {   // the sum of the cluster's shares: [column / 4][row]
            float4* mine4 = reinterpret_cast<float4*>(as);
            if (row < q.rn) {
#pragma unroll
                for (int m = 0; m < kMost; ++m)
                    if (m < r_mine)
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            mine4[(4 * (group + kSmallGroups * m) + e / 4) * q.rn + row] = make_float4(
                                acc[m][e], acc[m][e + 1], acc[m][e + 2], acc[m][e + 3]);
            }
            __syncwarp();
            cluster_sync();
            // each CTA adds up a part of them and leaves the sum with all
            // (at most four places a thread: 128 x 128 over two CTAs; all loads before the stores)
            constexpr int kPlaces = 128 * 128 / 4 / (2 * kSmallThreads);
            float4 t[kPlaces];
            const auto at_of = [&](int j) { return (j * q.ctas + rank) * kSmallThreads + tid; };
#pragma unroll
            for (int j = 0; j < kPlaces; ++j) {
                t[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (at_of(j) >= q.rn * q.rn / 4) continue;
#pragma unroll 8
                for (int k = 0; k < q.ctas; ++k) {
                    const float4 u = ld_cluster(a0 + (uint32_t)at_of(j) * 16, k);
                    t[j].x += u.x;
                    t[j].y += u.y;
                    t[j].z += u.z;
                    t[j].w += u.w;
                }
            }
#pragma unroll
            for (int j = 0; j < kPlaces; ++j) {
                if (at_of(j) >= q.rn * q.rn / 4) continue;
                for (int k = 0; k < q.ctas; ++k)
                    st_cluster(a0 + (uint32_t)at_of(j) * 16, k, t[j]);
            }
            __syncwarp();
            cluster_sync();
            if (row < q.rn) {
#pragma unroll
                for (int m = 0; m < kMost; ++m)
                    if (m < r_mine)
#pragma unroll
                        for (int e = 0; e < 16; e += 4) {
                            const float4 u = mine4[(4 * (group + kSmallGroups * m) + e / 4) * q.rn + row];
                            acc[m][e] = u.x;
                            acc[m][e + 1] = u.y;
                            acc[m][e + 2] = u.z;
                            acc[m][e + 3] = u.w;
                        }
            }
            __syncthreads();   // A takes the place of the shares
        }
        if (!ok) continue;
        if (busy) {
            const float fa = held->of[step].a;
#pragma unroll
            for (int m = 0; m < kMost; ++m) {
                if (m < r_mine) {
                    const int col = 16 * (group + kSmallGroups * m);
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[m][e] *= fa;
                    if (col / 32 == quarter) off_diagonal(a_diag, col, acc[m]);
                    put(as, col, acc[m]);
                }
            }
        }
        ready();
        // ---- P = a I + b A + c A A
        if (tid == 0) issue(0, 0, q.rn, a0, a0, q.rn, 0, r_units, false);
        const bool last = step + 1 == q.steps;
        if (kWild && warp == kScaler) scale_p_step(q.poly, a_diag, q.rn, step, held);
        if (!await(0)) continue;
        if (busy) {
            const float d = a_diag[row];
            const Factors f = held->of[step].p;
#pragma unroll
            for (int m = 0; m < kMost; ++m) {
                if (m >= r_mine) continue;
                const int col = 16 * (group + kSmallGroups * m);
                float v[16];
                sums(col, col + q.rn, v);
                if (row < q.rn) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {   // (acc is O here)
                        const float beta = fmaf(f.p2, d + a_diag[col + e], f.p1);
                        v[e] = fmaf(beta, acc[m][e], v[e] * f.p2);
                    }
                    if (col / 32 == quarter) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)   // (O is zero there)
                            v[e] += col + e == row ? fmaf(d, fmaf(f.p2, d, f.p1), f.p0) : 0.0f;
                    }
                }
                if (col / 32 == quarter) off_diagonal(p_diag, col, v);
                put(as, col, v);
            }
        }
        ready();
        const float d = busy ? p_diag[row] : 0.0f;
        // ---- X' = P X, 256 columns at a time; the last one is the result
        for (int c0 = 0; c0 < cn; c0 += 256) {
            const int n = min(256, cn - c0);
            if (tid == 0)
                issue(0, 0, 256, a0, x0 + (uint32_t)(c0 / kPanel) * kParts * pb, n, 0, r_units, true);
            if (kWild && c0 == 0 && tid == kScaler * 32) scale_x_step(q.poly, step, q.steps, held);
            uint4 x[2][kParts];   // this row's halves of X in the next unit
            const auto fetch = [&](int u) {
                if (row >= q.rn || u >= n / 16) return;
                const int col = c0 + 16 * u;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int p = 0; p < kParts; ++p)
                        x[b][p] = *reinterpret_cast<const uint4*>(
                            xs + (col / kPanel * kParts + p) * pb +
                            panel_at(row, col % kPanel + 8 * b, q.rn) * 2);
            };
            fetch(group);
            if (!await(0)) break;
            if (busy) {
                const float unit = held->of[step].x;
#pragma unroll 1
                for (int u = group; u < n / 16; u += kSmallGroups) {
                    float v[16];
                    sums(16 * u, 256 + 16 * u, v);
                    if (row >= q.rn) continue;
                    const int col = c0 + 16 * u;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = v[8 * b + e];
#pragma unroll
                        for (int p = 0; p < kParts; ++p) add_halves(w, x[b][p], d);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[8 * b + e] = w[e] * unit;
                    }
                    fetch(u + kSmallGroups);
                    if (!last) {
                        put(xs, col, v);
                    } else if (q.tall) {   // (the warp's rows are adjacent there)
                        T* o = out + blockIdx.x / q.ctas * elems;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float y[1] = {v[e]};
                            const int oc = col0 + col + e;
                            if (row < q.r && oc < q.c)
                                Pack<T, 1>::store(o + (size_t)oc * q.r + row, y);
                        }
                    } else {
                        constexpr int kChunk16 = VecOf<T>::n;
#pragma unroll
                        for (int e = 0; e < 16; e += kChunk16) {
                            float y[kChunk16];
#pragma unroll
                            for (int b = 0; b < kChunk16; ++b) y[b] = v[e + b];
                            Pack<T, kChunk16>::store(staged(row, col + e), y);
                        }
                    }
                }
            }
            if (last && !q.tall) {   // whole rows of the block's columns
                __syncthreads();
                T* o = out + blockIdx.x / q.ctas * elems + col0 + c0;
                const int width = min(n, mine - c0) / V;
                for (int e = tid; e < q.r * width; e += kSmallThreads) {
                    const int orow = e / width, oc = (e - orow * width) * V;
                    float y[V];
                    Pack<T, V>::load(staged(orow, c0 + oc), y);
                    Pack<T, V>::store(o + (size_t)orow * q.c + oc, y);
                }
            }
            ready();
        }
    }
    if (!ok) {
        // an MMA did not complete in time: report it, give what was awaited and
        // what may still be in flight one more bounded wait each, then release
        // the tensor memory
        if (tid == 0) atomicOr(&st->error, kErrTimeout);
        for (int k = 0; k < 2; ++k) {
            mbar_wait(mbar + k, (ph[k] - 1) & 1);
            mbar_wait(mbar + k, ph[k] & 1);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
    if (shared) {   // (the others may still read this CTA's norm where there was no step)
        __syncwarp();
        cluster_sync();
    }
}

// ----------------------------------------------------------------- plans --
constexpr size_t kSmemMax = 227 * 1024 - 512;   // (the norm has a little of its own)

constexpr size_t kSmemHalf = 120 * 1024;

struct Plan {
    int64_t r, c, rp, cp;   // padded
    bool tall;
    int parts;
    int ctas;               // on chip: a cluster of them takes a matrix through all steps; else 0
    int norm_blocks;        // per matrix, of the norm by a launch of its own
};
Plan plan_of(int64_t batch, int64_t m, int64_t n, int dtype) {
    Plan p;
    p.tall = m > n;
    p.r = p.tall ? n : m;
    p.c = p.tall ? m : n;
    // (of 1024 rows and more in pairs of blocks, for the wide symmetric tiles)
    p.rp = p.r > 1024 ? ceil_div(p.r, 2 * kBlock) * 2 * kBlock : ceil_div(p.r, kBlock) * kBlock;
    const int64_t to = p.c > 1024 ? 256 : 128;   // two widths of a tile of the last product
    p.cp = ceil_div(p.c, to) * to;
    const int64_t chunks = ceil_div(p.r * p.c, kThreads * 16);
    p.norm_blocks = (int)(chunks < kNormBlocks ? chunks : kNormBlocks);
    // pairs in 16 bits too where there are too few elements for the roundings of single halves to
    // average out (5 x 6: the result up to 2.4 times as far off as its own rounding; with pairs 1.0;
    // 16 x 16: 1.7 us more)
    p.parts = dtype == kF32 || (p.r <= 32 && p.c <= 256) ? 2 : 1;
    // on chip: shares of about 256 columns, more where memory or the SMs ask for it
    p.ctas = 0;
    const int rn = (int)ceil_div(p.r, 16) * 16, ap = (int)ceil_div(p.r, kPanel);
    if (rn <= kBlock && p.c <= 65536) {
        const auto fits = [&](int n) {
            return small_bytes(p.parts, rn, (int)ceil_div(ceil_div(p.c, kPanel), n), ap, n) <= kSmemMax;
        };
        int n = 1;
        while (n < kMaxShares && (!fits(n) || (n * 256 < p.c && batch * n * 2 <= 152))) n *= 2;
        if (fits(n)) p.ctas = n;
    }
    return p;
}

struct Space {
    __half *x[2], *a, *p;
    size_t x_lo, a_lo;
    Squares* part;
    float* bound;
    unsigned long long* trace;
    float *rest, *rows;
};
Space carve(Carve& w, int64_t batch, const Plan& p) {
    Space s{};
    s.part = w.take<Squares>((size_t)batch * p.norm_blocks);
    if (p.ctas > 0) return s;   // on chip, all but the norm where no step follows it
    s.x_lo = (size_t)batch * p.rp * p.cp;
    s.a_lo = (size_t)batch * p.rp * p.rp;
    for (int k = 0; k < 2; ++k) s.x[k] = w.take<__half>(s.x_lo * p.parts);
    s.a = w.take<__half>(s.a_lo * p.parts);
    s.p = w.take<__half>(s.a_lo * p.parts);
    s.bound = w.take<float>((size_t)batch * kMaxSteps);
    s.trace = w.take<unsigned long long>((size_t)batch * kMaxSteps);
    s.rest = w.take<float>(p.parts == 1 ? (size_t)batch * p.rp : 0);
    s.rows = w.take<float>(p.parts == 1 ? (size_t)batch * p.rp : 0);
    return s;
}

template <bool kSplit, int kN, bool kGram, int kCluster = 1>
cudaError_t product(const Product& q, LearnState* st, int n_sms, cudaStream_t s) {
    const int64_t total = (int64_t)q.tiles * q.batch * kCluster;
    return launch_pdl(k_orth_product<kSplit, kN, kGram, kCluster>,
                      dim3((unsigned)(total < n_sms || kCluster > 1 ? total : n_sms)),
                      dim3(kProductThreads), ProductSmem<kSplit, kN>::bytes, s, q, st);
}

// A symmetric product: as many CTAs share a tile as there are SMs (and panels)
// for; clusters do not fill every SM of a GPC, hence seven eighths of them.
template <bool kSplit>
cudaError_t symmetric(const Product& q, LearnState* st, int n_sms, cudaStream_t s) {
    const int64_t total = (int64_t)q.tiles * q.batch;
    const auto fits = [&](int n) { return total * n * 8 <= n_sms * 7 && q.k_panels >= n; };
    if (fits(8)) return product<kSplit, kBlock, true, 8>(q, st, n_sms, s);
    if (fits(4)) return product<kSplit, kBlock, true, 4>(q, st, n_sms, s);
    if (fits(2)) return product<kSplit, kBlock, true, 2>(q, st, n_sms, s);
    if constexpr (!kSplit) {
        // An MMA of N = 256 takes little longer than one of 128: tiles twice as wide, shared by
        // two CTAs, take two thirds of the time (2048 rows: 72 tiles instead of 136).  A cluster
        // takes one tile, so that this is for calls of up to 76 of them (one matrix of 1281 to
        // 2048 rows, two of 1025 to 1280); larger ones have tiles of 128 x 128 again.
        const int64_t half = (q.tiles_m + 1) / 2, wide = half * (half + 1) * q.batch;
        if (q.tiles_m % 2 == 0 && q.k_panels >= 2 && wide * 2 <= n_sms) {
            Product w = q;
            w.tiles = (int)(half * (half + 1));
            return product<kSplit, 256, true, 2>(w, st, n_sms, s);
        }
    }
    return product<kSplit, kBlock, true>(q, st, n_sms, s);
}

template <typename T, bool kSplit>
cudaError_t run(const OrthCall& o, LearnState* st, void* ws, int n_sms, cudaStream_t s) {
    constexpr int kParts = kSplit ? 2 : 1;
    const Plan p = plan_of(o.batch, o.m, o.n, o.dtype);
    if (o.steps > 0 && p.ctas > 0) {
        constexpr int V = VecOf<T>::n;
        Small q{(int)p.r, (int)p.c, (int)ceil_div(p.r, 16) * 16,
                (int)ceil_div(ceil_div(p.c, kPanel), p.ctas), (int)ceil_div(p.r, kPanel),
                p.ctas, p.tall, o.steps, polynomial(o.a, o.b, o.c, o.steps), o.eps};
        q.known = !q.poly.wild && o.steps <= kKnownSteps;
        float m = 1.0f;
        for (int k = 0; q.known && k < o.steps; ++k) {
            const float u = m * m, next = next_bound(q.poly, m, u);
            q.of[k] = {factors_p(q.poly, m, u), factor_a(m),
                       factor_x(q.poly, m, u, next, k + 1 == o.steps)};
            m = next;
        }
        // (the loads of `grad` and the stores to `out` are of one width)
        const bool vec = !p.tall && p.c % V == 0 && aligned16(o.grad) && aligned16(o.out);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(o.batch * p.ctas));
        cfg.blockDim = dim3(kSmallThreads);
        cfg.dynamicSmemBytes = small_bytes(kParts, q.rn, q.xp, q.ap, q.ctas);
        // CTAs of a cluster wait for one another holding all of their SM's tensor memory: more
        // than half of its shared memory keeps a second one from waiting for that
        if (p.ctas > 1 && cfg.dynamicSmemBytes < kSmemHalf) cfg.dynamicSmemBytes = kSmemHalf;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)p.ctas;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        // (a wild polynomial has one form: nothing waits for it)
        return cudaLaunchKernelEx(&cfg, q.poly.wild ? k_orth_small<T, kSplit, 1, true>
                                        : vec       ? k_orth_small<T, kSplit, V, false>
                                                    : k_orth_small<T, kSplit, 1, false>,
                                  (const T*)o.grad, q, (T*)o.out, st);
    }
    Carve cv{static_cast<unsigned char*>(ws)};
    const Space w = carve(cv, o.batch, p);
    const unsigned B = (unsigned)o.batch;
    const int64_t elems = p.r * p.c;
    const int parts = p.norm_blocks;
    const auto flat = [&](int64_t items) {
        const int64_t b = ceil_div(items, kThreads);
        return dim3((unsigned)(b < 2048 ? b : 2048), B);
    };
    constexpr int V = VecOf<T>::n;
    const bool vec = aligned16(o.grad) && elems % V == 0;   // every matrix of the batch
    cudaError_t e = vec ? launch_pdl(k_orth_norm<T, V>, dim3(parts, B), dim3(kThreads), 0, s,
                                     (const T*)o.grad, elems, w.part)
                        : launch_pdl(k_orth_norm<T, 1>, dim3(parts, B), dim3(kThreads), 0, s,
                                     (const T*)o.grad, elems, w.part);
    if (e != cudaSuccess) return e;
    if (o.steps == 0)
        return launch_pdl(k_orth_scale<T>, flat(elems), dim3(kThreads), 0, s, (const T*)o.grad,
                          elems, (const Squares*)w.part, parts, o.eps, (T*)o.out);
    const auto start = !p.tall && vec && p.c % V == 0 ? k_orth_start<T, kParts, V>
                                                      : k_orth_start<T, kParts, 1>;
    const int64_t inner = p.tall ? p.rp : p.cp / 8, lines = p.tall ? p.cp / 8 : p.rp;
    const int64_t pieces = ceil_div(inner, 128) * ceil_div(lines, 8);
    const dim3 grid((unsigned)(pieces < 2432 ? pieces : 2432), B);
    e = launch_pdl(start, grid, dim3(kThreads), 0, s, (const T*)o.grad, p.r, p.c,
                   p.rp, p.cp, p.tall, (const Squares*)w.part, parts, o.eps, w.bound, w.trace, w.x[0],
                   w.x_lo);
    const int tm = (int)(p.rp / kBlock);
    const Polynomial poly = polynomial(o.a, o.b, o.c, o.steps);
    for (int k = 0; k < o.steps && e == cudaSuccess; ++k) {
        const __half* x = w.x[k & 1];
        Product g{};   // A = X X^T
        g.l = g.r = x;
        g.l_lo = g.r_lo = w.x_lo;
        g.l_size = g.r_size = (size_t)p.rp * p.cp;
        g.l_rows = g.r_rows = p.rp;
        g.k_panels = (int)(p.cp / kPanel);
        g.tiles_m = tm;
        g.tiles = tm * (tm + 1) / 2;
        g.batch = (int)o.batch;
        g.d = w.a;
        g.d_lo = w.a_lo;
        g.d_size = (size_t)p.rp * p.rp;
        g.d_rows = p.rp;
        g.poly = poly;
        g.bound = w.bound + k;
        g.trace = w.trace + k;
        g.last = k + 1 == o.steps;
        g.rest = w.rest;
        g.rows = w.rows;
        e = symmetric<kSplit>(g, st, n_sms, s);
        if (e != cudaSuccess) return e;
        Product h = g;   // P = a I + b A + c A A
        h.l = h.r = h.c = w.a;
        h.l_lo = h.r_lo = w.a_lo;
        h.l_size = h.r_size = (size_t)p.rp * p.rp;
        h.k_panels = (int)(p.rp / kPanel);
        h.d = w.p;
        e = symmetric<kSplit>(h, st, n_sms, s);
        if (e != cudaSuccess) return e;
        Product f = g;   // X' = P X
        f.l = w.p;
        f.l_lo = w.a_lo;
        f.l_size = (size_t)p.rp * p.rp;
        f.k_panels = (int)(p.rp / kPanel);
        f.d = w.x[(k + 1) & 1];
        f.d_lo = w.x_lo;
        f.d_size = (size_t)p.rp * p.cp;
        if (k + 1 == o.steps) {
            f.out = o.out;
            f.out_r = p.r;
            f.out_c = p.c;
            f.tall = p.tall;
            f.dtype = o.dtype;
        }
        // 256 columns a tile move fewer operand bytes per product; 128 give twice the tiles
        const bool wide = !kSplit && p.cp % 256 == 0 &&
                          (int64_t)tm * (p.cp / 256) * o.batch >= n_sms;
        f.tiles = tm * (int)(p.cp / (wide ? 256 : 128));
        if (wide)
            e = product<kSplit, kSplit ? 128 : 256, false>(f, st, n_sms, s);
        else
            e = product<kSplit, 128, false>(f, st, n_sms, s);
    }
    return e;
}

template <bool kSplit, int kN, bool kGram, int kCluster = 1>
cudaError_t prepare_one() {
    return cudaFuncSetAttribute(k_orth_product<kSplit, kN, kGram, kCluster>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                ProductSmem<kSplit, kN>::bytes);
}
template <bool kSplit>
cudaError_t prepare_type() {
    cudaError_t e = prepare_one<kSplit, 128, true>();
    if (e == cudaSuccess) e = prepare_one<kSplit, 128, true, 2>();
    if (e == cudaSuccess) e = prepare_one<kSplit, 128, true, 4>();
    if (e == cudaSuccess) e = prepare_one<kSplit, 128, true, 8>();
    if (e == cudaSuccess) e = prepare_one<kSplit, 128, false>();
    return e;
}

}  // namespace

size_t orth_workspace(int64_t batch, int64_t m, int64_t n, int dtype) {
    if (batch == 0 || m == 0 || n == 0) return 0;
    Carve cv{nullptr};
    carve(cv, batch, plan_of(batch, m, n, dtype));
    return cv.used;
}

bool orth_in_range(int steps, float a, float b, float c) {
    const Polynomial p = polynomial(a, b, c, 0);
    float m = 1.0f;
    for (int k = 0; k < steps; ++k) {
        // (in this form a NaN is refused too)
        if (!(m < ldexpf(1.0f, kMostX) && p.at(m * m) < ldexpf(1.0f, kMostP) &&
              p.most_q(m * m) < ldexpf(1.0f, kMostP)))
            return false;
        m = p.most_s(m * m);
    }
    return true;
}

cudaError_t prepare_orth() {
    cudaError_t e = prepare_type<false>();
    if (e == cudaSuccess) e = prepare_type<true>();
    if (e == cudaSuccess) e = prepare_one<false, 256, false>();
    if (e == cudaSuccess) e = prepare_one<false, 256, true, 2>();
    using B = __nv_bfloat16;
    for (const void* k : {(const void*)k_orth_small<float, true, 1, false>,
                          (const void*)k_orth_small<float, true, 4, false>,
                          (const void*)k_orth_small<float, true, 1, true>,
                          (const void*)k_orth_small<B, true, 1, false>,
                          (const void*)k_orth_small<B, true, 8, false>,
                          (const void*)k_orth_small<B, true, 1, true>,
                          (const void*)k_orth_small<B, false, 1, false>,
                          (const void*)k_orth_small<B, false, 8, false>,
                          (const void*)k_orth_small<B, false, 1, true>})
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
    return e;
}

cudaError_t launch_orth(const OrthCall& q, LearnState* st, void* ws, int n_sms, cudaStream_t s) {
    if (q.batch == 0 || q.m == 0 || q.n == 0) return cudaSuccess;
    if (q.dtype == kF32) return run<float, true>(q, st, ws, n_sms, s);
    return plan_of(q.batch, q.m, q.n, q.dtype).parts == 2
               ? run<__nv_bfloat16, true>(q, st, ws, n_sms, s)
               : run<__nv_bfloat16, false>(q, st, ws, n_sms, s);
}

}  // namespace pulsar
