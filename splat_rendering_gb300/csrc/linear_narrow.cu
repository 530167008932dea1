// Narrow linear layers (see linear.cu): few inputs and outputs, many rows.
#include <type_traits>

#include "linear_internal.cuh"

namespace pulsar {
namespace linear {
namespace {

// ---------------------------------------------------------- narrow layers --
// A layer of few inputs and outputs over many rows (a network's hidden layer
// over an image) is bound by its rows' way in and out.  One launch, a
// persistent CTA per SM, tiles of 128 rows, each read and written once.  Roles:
// one thread keeps a ring of raw tiles filled (128 rows are one contiguous bulk
// copy, whatever their width, but for what lies before x's first 16-byte boundary
// in a tile and behind its last), eight warps make a tile's operand from it, 64
// columns of the contraction at a time (in 32 bits its three planes), one
// thread issues the MMAs, and eight warps finish the tile from tensor memory.
// The weights are made into operands by every CTA once, and stay.
//
// In 32 bits the weights' planes lie below one another, [hi; mid; lo], so that a
// plane of the rows takes one MMA against those that count: hi against all
// three, mid against hi and mid, lo against hi.  Their sums in three ranges of
// columns are hi hi, (hi mid + mid hi), (hi lo + mid mid + lo hi), so that what
// the tensor cores truncate is relative to each, of at most 128 of K, as there.
// (Six MMAs of 64 columns into one accumulator, hi hi last, are as exact and take
// half as long again: an MMA reads 128 rows of A whatever its columns.)
//
// 1M x 64 -> 64 with SiLU in 32 bits: 94 us, 5.7 TB/s of measured 6.8 (its bytes
// take 79), storing z too 125 (118); 777600 x 64 -> 64 in 16 bits with ReLU 45 us,
// storing z too 48, with a residual 64 (29, 44 and 44).  In 32 bits a residual, eight
// vectors of it in flight, does not fit the registers (336 bytes of spills are read
// again): 1M x 64 -> 64 with SiLU and a residual 171 us, storing z too 214 (118, 158).
// Bound by the warps' work on a tile, not by its bytes: operands (LDS, three
// conversions, STS), the exchange and the activation, whose exponential and
// reciprocal are half of the bfloat16 tile's time on their pipe.
constexpr int kStreamThreads = 576;   // warps: copies, MMAs, eight of operands, eight of the epilogue
constexpr int kStreamMaxK = 128;
template <typename T>
constexpr int kStreamN = sizeof(T) == 4 ? 64 : 128;   // outputs of a CTA
// Up to eight blocks of them read the same rows side by side: 200000 x 64 -> 512 in 32 bits takes 125
// us, by the wide products 262, 128 -> 512 291 and 300 (but 128 -> 1024 in sixteen blocks, per 100000
// rows, 302 and 274); in 16 bits 200000 x 64 -> 64 17 and 28, 100000 x 128 -> 1024 92 and 104.
constexpr int kStreamBlocks = 8;

struct Stream {
    const void* x;         // [m, k]
    const void* weight;    // [n, k]
    int64_t tiles;
    int k, panels;         // of the contraction
    int np, blocks;        // outputs of a block (a multiple of 16), blocks
    int raws, units;       // raw tiles, operand panels in flight
    int shift;             // bytes from a 16-byte boundary to x, as to every tile of it
    bool vec, vec_w;       // rows of x (the weight) are whole 16-byte vectors
    bool skip;             // there is a residual, on 16 bytes, and one block of outputs
    Result out;
};
struct StreamSmem {
    int raw, raw_bytes, unit, unit_bytes, weight, weight_panel, exchange, bars, bytes;
};
__host__ __device__ inline StreamSmem stream_smem(int planes, int size, int k, int panels, int np,
                                                  int raws, int units, int shift) {
    StreamSmem s;
    s.unit = 0;
    s.unit_bytes = planes * kBlock * kPanel * 2;
    s.weight = s.unit + units * s.unit_bytes;
    s.weight_panel = planes * np * kPanel * 2;
    s.exchange = s.weight + panels * s.weight_panel;
    s.raw = s.exchange + 8 * 32 * 32 * 4;
    s.raw_bytes = (kBlock * k * size + shift + 127) / 128 * 128;
    s.bars = s.raw + raws * s.raw_bytes;
    s.bytes = s.bars + 256 + 1024;
    return s;
}
constexpr int kStreamSmemMax = 227 * 1024 - 512;   // (and the bias)

// kVec: rows of the result are whole vectors.  kSkip: there is a residual.
template <typename T, bool kVec, bool kSkip>
__global__ void __launch_bounds__(kStreamThreads, 1)
k_linear_stream(const __grid_constant__ Stream q, LearnState* st) {
    constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
    constexpr int kCols = sizeof(T) == 4 ? 512 : 256;   // tensor memory: two accumulators
    extern __shared__ unsigned char raw_smem[];
    __shared__ __align__(16) float s_bias[128];
    unsigned char* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
    const StreamSmem L = stream_smem(kPlanes, sizeof(T), q.k, q.panels, q.np, q.raws, q.units,
                                     q.shift);
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + L.bars);
    uint64_t* raw_empty = raw_full + 4;
    uint64_t* unit_full = raw_empty + 4;
    uint64_t* unit_empty = unit_full + 4;
    uint64_t* acc_full = unit_empty + 4;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* s_taddr = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* s_fail = s_taddr + 1;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (known to be the same in a warp)
    const int block = blockIdx.x % q.blocks, first = blockIdx.x / q.blocks;
    const int step = gridDim.x / q.blocks;
    const int n0 = block * kStreamN<T>;
    const int steps16 = (q.k + 15) / 16;
    if (tid == 0) {
        for (int s = 0; s < 4; ++s) {
            mbar_init(raw_full + s);
            mbar_init_n(raw_empty + s, 8);
            mbar_init_n(unit_full + s, 8);
            mbar_init(unit_empty + s);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + s);
            mbar_init_n(acc_empty + s, 8);
        }
        mbar_init(drain);
        *s_fail = 0u;
    }
    if (warp == 1) tmem_alloc(s_taddr, kCols);
    pdl_begin();
    if (tid < 128)
        s_bias[tid] = q.out.bias && n0 + tid < q.out.n ? q.out.bias[n0 + tid] : 0.0f;
    {   // the weights, zeros below and behind them
        const int chunks = steps16 * 2, total = q.np * chunks;
        for (int t = tid; t < total; t += kStreamThreads) {
            const int r = t / chunks, c = t % chunks;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            const int n = q.k - c * 8 < 8 ? q.k - c * 8 : 8;
            if (n0 + r < q.out.n && n > 0)
                load8(static_cast<const T*>(q.weight) + (int64_t)(n0 + r) * q.k + c * 8, n,
                      q.vec_w && n == 8, v);
            put_chunk<kPlanes>(smem + L.weight + (c >> 3) * L.weight_panel + r * 128 +
                                   (((c & 7) ^ (r & 7)) << 4),
                               q.np * 128, v);
        }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_taddr;
    pdl_next();   // (not before this block has its tensor memory: the next one's would wait with it)
    if (warp == 0) {
        if (elect_one()) {   // ---- raw tiles
            int n = 0;
            bool ok = true;
            for (int64_t t = first; t < q.tiles; t += step, ++n) {
                const int s = n % q.raws;
                ok = mbar_wait(raw_empty + s, ((n / q.raws) & 1) ^ 1) && !*s_fail;
                if (!ok) break;
                const int64_t left = q.out.m - t * kBlock;
                const uint32_t bytes =
                    (uint32_t)((left < kBlock ? left : kBlock) * q.k * (int)sizeof(T));
                const unsigned char* src =
                    static_cast<const unsigned char*>(q.x) + t * kBlock * q.k * (int64_t)sizeof(T);
                unsigned char* dst = smem + L.raw + s * L.raw_bytes + q.shift;
                if (q.skip) {   // its residual is on its way to the L2 before the epilogue asks
                    const uint32_t row = (uint32_t)(q.out.n * (int)sizeof(T));
                    prefetch_l2(static_cast<const unsigned char*>(q.out.residual) +
                                    t * kBlock * (int64_t)row,
                                (uint32_t)(left < kBlock ? left : kBlock) * row & ~15u);
                }
                // (neither the first rows need begin on 16 bytes nor the last ones end there)
                const auto alone = [&](uint32_t from, uint32_t to) {
                    for (uint32_t e = from / sizeof(T); e < to / sizeof(T); ++e)
                        reinterpret_cast<T*>(dst)[e] = reinterpret_cast<const T*>(src)[e];
                };
                const uint32_t head = min((16u - q.shift) & 15u, bytes), bulk = (bytes - head) & ~15u;
                alone(0, head);
                alone(head + bulk, bytes);
                if (bulk)
                    bulk_load(dst + head, src + head, bulk, raw_full + s);
                else
                    mbar_arrive(raw_full + s);
            }
            if (!ok) {   // give the copies in flight one more bounded wait
                *s_fail = 1u;
                for (int k = n > q.raws ? n - q.raws : 0; k < n; ++k)
                    mbar_wait(raw_full + k % q.raws, (k / q.raws) & 1);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {   // ---- MMAs
            const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) |
                                    ((uint32_t)(kBlock >> 4) << 24);
            const uint32_t np = (uint32_t)q.np;
            uint32_t idesc[kPlanes];   // against the weights' first kPlanes - p planes
#pragma unroll
            for (int p = 0; p < kPlanes; ++p)
                idesc[p] = idesc0 | ((np * (uint32_t)(kPlanes - p) >> 3) << 17);
            const uint32_t base = smem_u32(smem);
            int u = 0, it = 0;
            bool ok = true;
            for (int64_t t = first; t < q.tiles && ok; t += step, ++it) {
                const int buf = it & 1;
                const uint32_t d = tmem + buf * (kCols / 2);
                ok = mbar_wait(acc_empty + buf, ((it >> 1) & 1) ^ 1) && !*s_fail;
                if (!ok) break;
                for (int h = 0; h < q.panels; ++h, ++u) {
                    const int s = u % q.units;
                    ok = mbar_wait(unit_full + s, (u / q.units) & 1) && !*s_fail;
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = base + L.unit + s * L.unit_bytes;
                    const uint64_t b = desc_sw128(base + L.weight + h * L.weight_panel, 16);
                    uint64_t a[kPlanes];
#pragma unroll
                    for (int p = 0; p < kPlanes; ++p)
                        a[p] = desc_sw128(at + p * kBlock * kPanel * 2, 16);
                    const int ends = min(4, steps16 - 4 * h);
                    for (int e = 0; e < ends; ++e) {
                        const uint32_t off = 32u * e >> 4;
                        mma_f16(d, a[0] + off, b + off, idesc[0], h > 0 || e > 0);
#pragma unroll
                        for (int p = 1; p < kPlanes; ++p)
                            mma_f16(d + p * np, a[p] + off, b + off, idesc[p], 1);
                    }
                    mma_commit(unit_empty + s);
                }
                if (ok) mma_commit(acc_full + buf);
            }
            if (!ok) {
                *s_fail = 1u;
                mma_commit(drain);
                mbar_wait(drain, 0);
            }
        }
    } else if (warp < 10) {   // ---- operands
        const int mine = tid - 64;
        int n = 0, u = 0;
        bool ok = true;
        for (int64_t t = first; t < q.tiles && ok; t += step, ++n) {
            const int s = n % q.raws;
            ok = warp_all(mbar_wait(raw_full + s, (n / q.raws) & 1) && !*s_fail);
            if (!ok) break;
            const T* tile = reinterpret_cast<const T*>(smem + L.raw + s * L.raw_bytes + q.shift);
            const int64_t left = q.out.m - t * kBlock;
            const int rows = (int)(left < kBlock ? left : kBlock);
            for (int h = 0; h < q.panels; ++h, ++u) {
                const int a = u % q.units;
                ok = warp_all(mbar_wait(unit_empty + a, ((u / q.units) & 1) ^ 1) && !*s_fail);
                if (!ok) break;
                unsigned char* unit = smem + L.unit + a * L.unit_bytes;
                const int chunks = min(8, 2 * steps16 - 8 * h);
                // a thread has a chunk of every 32nd row (rows behind the last keep what they
                // held: their sums are not stored)
                const int c = mine & 7, r0 = mine >> 3, col = h * kPanel + c * 8;
                const T* src = tile + r0 * q.k + col;
                unsigned char* dst = unit + r0 * 128 + ((c ^ (r0 & 7)) << 4);
                if (q.vec && q.k - col >= 8) {
                    float v[4][8];   // (all loads, then all stores, as there)
#pragma unroll
                    for (int i = 0; i < 4; ++i) load8(src + 32 * i * q.k, 8, true, v[i]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        put_chunk<kPlanes>(dst + 32 * i * 128, kBlock * kPanel * 2, v[i]);
                } else if (c < chunks) {   // (what lies behind the last row is shared too)
                    const uint32_t at = smem_u32(src);
                    Window<T, 8> w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i].load_shared(at + (uint32_t)(32 * i * q.k * (int)sizeof(T)));
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v[8];
                        w[i].open(v);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = col + e < q.k ? v[e] : 0.0f;
                        put_chunk<kPlanes>(dst + 32 * i * 128, kBlock * kPanel * 2, v);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(unit_full + a);
            }
            if (lane == 0) mbar_arrive(raw_empty + s);   // (after the last __syncwarp)
        }
        if (!ok) *s_fail = 1u;
    } else {   // ---- epilogue
        const int e0 = warp - 10, quarter = warp & 3, group = e0 >> 2;
        float4* x = reinterpret_cast<float4*>(smem + L.exchange) + e0 * 256;
        int it = 0;
        for (int64_t t = first; t < q.tiles; t += step, ++it) {
            const int buf = it & 1;
            const int64_t r0 = t * kBlock + quarter * 32;
            Share<T, kVec, kSkip> share;
            if (group * 32 < q.np) share.begin(q.out, r0, n0 + group * 32, 0, lane);
            const bool ok = warp_all(mbar_wait(acc_full + buf, (it >> 1) & 1) && !*s_fail);
            if (!ok) {
                *s_fail = 1u;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + buf * (kCols / 2) + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
            for (int c = group * 32; c < q.np; c += 64) {
                float v[32];
#pragma unroll
                for (int p = 0; p < kPlanes; ++p) {
                    uint32_t w[32];
                    __syncwarp();
                    tmem_ld32(acc + p * q.np + c, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        v[e] = p ? v[e] + __uint_as_float(w[e]) : __uint_as_float(w[e]);
                }
                if (c + 64 >= q.np) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty + buf);
                }
                if (c != group * 32) share.begin(q.out, r0, n0 + c, 0, lane);
                const float4 b = *reinterpret_cast<const float4*>(s_bias + c + 4 * (lane & 7));
                const float bias[4] = {b.x, b.y, b.z, b.w};
                share.end(q.out, x, v, bias, r0, n0 + c, 0, lane);
            }
            if (group * 32 >= q.np && lane == 0) mbar_arrive(acc_empty + buf);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *s_fail) atomicOr(&st->error, kErrTimeout);
    if (warp == 1) tmem_dealloc(tmem, kCols);
}

// --------------------------------------------- narrow layers, gradients --
// All gradients of a narrow layer in one pass over dy, z and x: a persistent CTA
// per SM, tiles of 128 rows.  One thread keeps raw rows coming (contiguous bulk
// copies, in pieces of 16 or 32 KB: with a whole tile at a time their way in was
// 44 % of the time), eight warps make dz and x into operands (and add up dz's
// columns), one thread issues the MMAs, eight warps finish dx.  dz's tile, 128
// rows of 128 bytes a panel, is a K-major left operand of dx = dz W (its rows are
// rows) and, the same bytes, an MN-major one of dW = dz^T x (its rows are the
// contraction).  dW stays in the CTA; k_linear_joins adds up the CTAs' sums in
// their order.
//
// In 32 bits the planes of dz are two groups of one left operand [hi; mid] of
// dW, those of x three of the right one, so that one MMA makes six products
// (mid lo among them, in columns that are not read); lo hi is a second one, into
// the columns of hi lo.  They are drained every tile (128 of K) into registers:
// the rows of hi, and those of mid, are parts of their own.  dx as in the
// forward kernel.  x's operand is made while the MMAs of dx run, which do not
// need it, and where there is room dz's next one during those of dW.
//
// In 16 bits dW's accumulator, whose sums the tensor cores truncate, is added to
// the CTA's part in memory every kPieceTiles tiles (2^14 rows), while the next
// ones go to another: what is lost of terms of one sign is 2^-13 of a sum at
// most, and no wait lasts for more than that many tiles.  (16M x 64 -> 64 takes
// 1091 us, without it 1043.)
//
// 1M x 64 -> 64 in 32 bits: 169 us, with SiLU 205 (118 and 158 by the bytes); 777600
// x 64 -> 64 in 16 bits 61 us, with ReLU 72, with SiLU 80 (44 and 59).  Bound by the
// eight warps that make operands; loads straight to registers, kept ahead of their
// use, were slower (their fence awaits every load).
constexpr int kBackThreads = 576;   // warps: MMAs, eight of operands, eight of the epilogue, copies
// Inputs and outputs of a layer, as many as there is room for (200000 x 64 -> 64 with SiLU in 32
// bits: 55 us, by the wide products 130; 128 -> 128 in 16 bits 66 and 81).
template <typename T>
constexpr int kBackSide = sizeof(T) == 4 ? 64 : 128;
constexpr int kPieceTiles = 128;   // (no layer of a million rows has more for a CTA)

struct Narrow {
    const void *grad_y, *pre, *x, *weight;
    int64_t rows, tiles;
    int k, n;              // inputs, outputs
    bool raw;              // the tensors begin on 16 bytes: raw tiles by bulk copies
    bool vec_n, vec_k;     // ... and rows of n (k) elements are whole 16-byte vectors
    bool vec_w;            // rows of the weight are whole chunks of eight, on 16 bytes
    bool want_x, want_w;
    float* parts;          // [parts of all CTAs][n][k], `part` floats each
    int64_t part;
    float* sums;           // [CTA][n]; may be NULL
    Result out;            // of dx
};
template <typename T, int kPanels, bool kAct>
struct BackSmem {
    static constexpr int planes = sizeof(T) == 4 ? 3 : 1;
    static constexpr int side = kPanels * kPanel;
    static constexpr int panel = kBlock * kPanel * 2;          // of one plane
    static constexpr int operand = planes * kPanels * panel;   // [panel][plane]
    // dz's operands, x's: in 32 bits with an activation, whose raw rows are half as many again, the
    // room is theirs (1M x 64 -> 64 with SiLU: 210 us, with two operands of dz and half the raw rows
    // 230; without an activation 195 and 169)
    static constexpr int dzs = planes == 3 && kAct ? 1 : 2;
    static constexpr int xs = planes == 1 && kPanels == 1 ? 2 : 1;
    static constexpr int x = dzs * operand;                    // dz's come first
    static constexpr int weight_panel = side * kPanel * 2;
    static constexpr int weight = x + xs * operand;            // [panel of inputs][plane]
    // a warp's exchange is 32 x 32 words; in 32 bits, for want of room, 32 x 8
    static constexpr int exchange = weight + planes * kPanels * weight_panel;
    static constexpr int exchange_bytes = planes == 3 ? 8 * 1024 : 8 * 4096;
    static constexpr int raw = exchange + exchange_bytes;
    // pieces of x's rows, or of dy's and z's
    static constexpr int piece = dzs == 1 ? 32 * 1024 : 16 * 1024;
    static constexpr int room = (227 * 1024 - 1280 - raw) / piece;
    static constexpr int pieces = room < 6 ? room : 6;
    static constexpr int rows_x = piece / (side * (int)sizeof(T));
    static constexpr int bars = raw + pieces * piece;
    static constexpr int bytes = bars + 256 + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory of a narrow layer's gradients");
};

// V columns (eight or sixteen bytes of bfloat16 in a plane).
template <int kPlanes, int V>
__device__ __forceinline__ void put_columns(unsigned char* at, uint32_t plane_bytes,
                                            const float (&v)[V]) {
    uint32_t w[V / 2][3];
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
        if (kPlanes == 3)
            split3(v[2 * e], v[2 * e + 1], w[e]);
        else
            w[e][0] = pair_bf16(v[2 * e], v[2 * e + 1]);
    }
#pragma unroll
    for (int p = 0; p < kPlanes; ++p) {
        if constexpr (V == 8)
            *reinterpret_cast<uint4*>(at + p * plane_bytes) =
                make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
        else
            *reinterpret_cast<uint2*>(at + p * plane_bytes) = make_uint2(w[0][p], w[1][p]);
    }
}

// 16 bytes of shared memory, said to be that: a pointer that may also be global costs a generic
// load, whose latency is several times a shared one's.
template <typename T>
__device__ __forceinline__ typename Pack<T, VecOf<T>::n>::Raw lds16(uint32_t at) {
    typename Pack<T, VecOf<T>::n>::Raw r;
    if constexpr (sizeof(T) == 4)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(at));
    else
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at));
    return r;
}

// kRows rows of an operand, [rows, cols] at `src` (times the activation's slope at `pre`, its
// columns added to `sum`, where kDz), by a thread that has 16 bytes' columns of every kStep-th row:
// rows behind the last, and columns up to the next 16, are zeros.  `shared`: src is a raw piece in
// shared memory, `vec`: whose rows are whole 16-byte vectors.
template <typename T, int kAct, int kPanels, bool kDz, int kRows>
__device__ __forceinline__ void make_operand(unsigned char* operand, const T* src, const T* pre,
                                             int rows, int cols, bool shared, bool vec, int mine,
                                             float (&sum)[kPanels][VecOf<T>::n]) {
    using L = BackSmem<T, kPanels, false>;   // (its planes and panels)
    constexpr int V = VecOf<T>::n, kLanes = kPanel / V, kStep = 256 / kLanes;
    constexpr int kBatch = kRows / kStep < 4 ? kRows / kStep : 4;
    const int c = mine % kLanes * V, r0 = mine / kLanes, cols16 = (cols + 15) / 16 * 16;
#pragma unroll
    for (int h = 0; h < kPanels; ++h) {
        const int col = h * kPanel + c;
        if (col >= cols16) break;
        float more[V];   // these rows' sum: a quarter as many roundings in a row
        if (kDz)
#pragma unroll
            for (int e = 0; e < V; ++e) more[e] = 0.0f;
        unsigned char* dst = operand + h * L::planes * L::panel + r0 * 128 +
                             (((c >> 3) ^ (r0 & 7)) << 4) + (c & 7) * 2;
        if (vec) {
            const uint32_t s = smem_u32(src + r0 * cols + col);
            const uint32_t z = smem_u32(pre + r0 * cols + col);
            const uint32_t pitch = (uint32_t)(kStep * cols) * (uint32_t)sizeof(T);
#pragma unroll
            for (int i0 = 0; i0 < kRows / kStep; i0 += kBatch) {
                typename Pack<T, V>::Raw a[kBatch], b[kBatch];   // (all loads, then all stores)
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {   // (what lies behind the last row is shared too)
                    a[i] = lds16<T>(s + (i0 + i) * pitch);
                    if (kAct != kActNone) b[i] = lds16<T>(z + (i0 + i) * pitch);
                }
                float v[kBatch][V], w[kBatch][V];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    Pack<T, V>::open(a[i], v[i]);
                    if (kAct != kActNone) Pack<T, V>::open(b[i], w[i]);
                    to_dz<kAct>(v[i], w[i]);
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const bool in = r0 + (i0 + i) * kStep < rows && col < cols;
#pragma unroll
                    for (int e = 0; e < V; ++e) v[i][e] = in ? v[i][e] : 0.0f;
                    if (kDz)
#pragma unroll
                        for (int e = 0; e < V; ++e) more[e] += v[i][e];
                    put_columns<L::planes>(dst + (i0 + i) * kStep * 128, L::panel, v[i]);
                }
            }
        } else if (shared) {
            const uint32_t s = smem_u32(src + r0 * cols + col), z = smem_u32(pre + r0 * cols + col);
            const uint32_t pitch = (uint32_t)(kStep * cols) * (uint32_t)sizeof(T);
#pragma unroll
            for (int i = 0; i < kRows / kStep; ++i) {   // (what lies behind the last is shared too)
                Window<T, V> a, b;
                a.load_shared(s + i * pitch);
                if (kAct != kActNone) b.load_shared(z + i * pitch);
                float v[V], w[V];
                a.open(v);
                if (kAct != kActNone) b.open(w);
                to_dz<kAct>(v, w);
                const bool row = r0 + i * kStep < rows;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    v[e] = row && col + e < cols ? v[e] : 0.0f;
                    if (kDz) more[e] += v[e];
                }
                put_columns<L::planes>(dst + i * kStep * 128, L::panel, v);
            }
        } else {
#pragma unroll 1
            for (int r = r0; r < kRows; r += kStep) {
                float v[V], w[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float one[1] = {0.0f}, z[1] = {0.0f};
                    if (r < rows && col + e < cols) {
                        Pack<T, 1>::load(src + (int64_t)r * cols + col + e, one);
                        if (kAct != kActNone) Pack<T, 1>::load(pre + (int64_t)r * cols + col + e, z);
                    }
                    v[e] = one[0];
                    w[e] = z[0];
                }
                to_dz<kAct>(v, w);
                if (kDz)
#pragma unroll
                    for (int e = 0; e < V; ++e) more[e] += v[e];
                put_columns<L::planes>(dst + (r - r0) * 128, L::panel, v);
            }
        }
        if (kDz)
#pragma unroll
            for (int e = 0; e < V; ++e) sum[h][e] += more[e];
    }
}

// 32 sums of a row, or the `left` that there are, into a part of dW: added to what it has where
// `more`.  (All loads, then all stores; by fours where rows begin on them: a lane has a row, and
// one by one the sectors are asked for eight times.)
__device__ __forceinline__ void add_part(float* part, uint32_t (&w)[32], int left, bool more) {
    if ((reinterpret_cast<uintptr_t>(part) & 15u) == 0 && left % 4 == 0) {
        float4* at = reinterpret_cast<float4*>(part);
        float4 u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            u[e] = more && 4 * e < left ? at[e] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (4 * e < left)
                at[e] = make_float4(u[e].x + __uint_as_float(w[4 * e]),
                                    u[e].y + __uint_as_float(w[4 * e + 1]),
                                    u[e].z + __uint_as_float(w[4 * e + 2]),
                                    u[e].w + __uint_as_float(w[4 * e + 3]));
    } else {
        float u[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) u[e] = more && e < left ? part[e] : 0.0f;
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (e < left) part[e] = u[e] + __uint_as_float(w[e]);
    }
}

// kForm: 2, rows of dy, z, x and dx are whole vectors; 1, those of dx are; 0, none need be.  (One
// kernel of forms 1 and 2 takes 67 us, not 62, of 777600 x 64 -> 64 in 16 bits; form 0 in place of 1
// 124, not 113, of 590465 x 96 -> 7 with SiLU.)
template <typename T, int kAct, int kPanels, int kForm>
__global__ void __launch_bounds__(kBackThreads, 1)
k_linear_narrow(const __grid_constant__ Narrow q, LearnState* st) {
    using L = BackSmem<T, kPanels, kAct != kActNone>;
    constexpr int kPlanes = L::planes, V = VecOf<T>::n;
    constexpr bool kSplit = kPlanes == 3;
    constexpr int kRowsX = L::rows_x, kRowsZ = kAct == kActNone ? L::rows_x : L::rows_x / 2;
    constexpr uint32_t kDw = kSplit ? 192 : 256;   // columns: dx below, dW from here
    extern __shared__ unsigned char raw_smem[];
    unsigned char* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + L::bars);
    uint64_t* raw_empty = raw_full + L::pieces;
    uint64_t* dz_full = raw_empty + L::pieces;
    uint64_t* x_full = dz_full + 2;
    uint64_t* dz_empty = x_full + 2;
    uint64_t* x_empty = dz_empty + 2;
    uint64_t* dx_full = x_empty + 2;
    uint64_t* dx_empty = dx_full + 2;
    uint64_t* dw_full = dx_empty + 2;
    uint64_t* dw_empty = dw_full + 2;
    uint64_t* drain = dw_empty + 2;
    static_assert((2 * L::pieces + 17) * 8 + 8 <= 256, "barriers");
    uint32_t* s_taddr = reinterpret_cast<uint32_t*>(drain + 1);
    volatile uint32_t* s_fail = s_taddr + 1;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (known to be the same in a warp)
    if (tid == 0) {
        for (int s = 0; s < L::pieces; ++s) {
            mbar_init(raw_full + s);
            mbar_init_n(raw_empty + s, 8);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init_n(dz_full + s, 8);
            mbar_init_n(x_full + s, 8);
            mbar_init(dz_empty + s);
            mbar_init(x_empty + s);
            mbar_init(dx_full + s);
            mbar_init_n(dx_empty + s, 8);
            mbar_init(dw_full + s);
            mbar_init_n(dw_empty + s, 8);
        }
        mbar_init(drain);
        *s_fail = 0u;
    }
    if (warp == 0) tmem_alloc(s_taddr, 512);
    pdl_begin();
    if (q.want_x) {   // W, rows of outputs: an MN-major operand; zeros in the rows up to the next 16
        const int rows = (q.n + 15) / 16 * 16, chunks = (q.k + 7) / 8;
        for (int t = tid; t < rows * chunks; t += kBackThreads) {
            const int r = t / chunks, c = t % chunks, n = q.k - c * 8;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            if (r < q.n)
                load8(static_cast<const T*>(q.weight) + r * q.k + c * 8, n, q.vec_w && n >= 8, v);
            put_chunk<kPlanes>(smem + L::weight + (c >> 3) * kPlanes * L::weight_panel + r * 128 +
                                   (((c & 7) ^ (r & 7)) << 4),
                               L::weight_panel, v);
        }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_taddr;
    pdl_next();   // (not before this block has its tensor memory: the next one's would wait with it)
    const int first = blockIdx.x, step = gridDim.x;
    if (warp == 17) {
        if (q.raw && elect_one()) {   // ---- raw pieces, in the order in which they are used
            int f = 0;
            bool ok = true;
            // `rows` rows of one tensor or two from row r on
            const auto piece = [&](const void* p, const void* p2, int64_t r, int rows, int cols) {
                const int s = f % L::pieces;
                ok = mbar_wait(raw_empty + s, ((f / L::pieces) & 1) ^ 1) && !*s_fail;
                if (!ok) return;
                ++f;
                const int64_t left = q.rows - r;
                if (left < rows) rows = left > 0 ? (int)left : 0;
                const uint32_t bytes = (uint32_t)rows * cols * (uint32_t)sizeof(T);
                const uint32_t bulk = bytes & ~15u;   // (the last rows need not end on 16 bytes)
                T* dst = reinterpret_cast<T*>(smem + L::raw + s * L::piece);
                T* dst2 = dst + L::piece / 2 / (int)sizeof(T);
                const T* src = static_cast<const T*>(p) + r * cols;
                const T* src2 = static_cast<const T*>(p2) + r * cols;
                for (uint32_t e = bulk / sizeof(T); e < bytes / sizeof(T); ++e) {
                    dst[e] = src[e];
                    if (p2) dst2[e] = src2[e];
                }
                expect_bytes(raw_full + s, p2 ? 2 * bulk : bulk);
                if (bulk) {
                    bulk_copy(dst, src, bulk, raw_full + s);
                    if (p2) bulk_copy(dst2, src2, bulk, raw_full + s);
                }
            };
            // a tile's tensors, on their way to the L2: the pieces' own way in is short then
            const auto ahead = [&](int64_t t) {
                if (t >= q.tiles) return;
                const int64_t left = q.rows - t * kBlock;
                const uint32_t rows = (uint32_t)(left < kBlock ? left : kBlock);
                const auto one = [&](const void* p, int cols) {
                    prefetch_l2(static_cast<const T*>(p) + t * kBlock * cols,
                                rows * cols * (uint32_t)sizeof(T) & ~15u);
                };
                one(q.grad_y, q.n);
                if (kAct != kActNone) one(q.pre, q.n);
                if (q.want_w) one(q.x, q.k);
            };
            constexpr bool kAhead = L::pieces * L::piece < 96 * 1024;   // (with these, no need)
            if (kAhead) ahead(first + step);
            for (int64_t t = first; t < q.tiles && ok; t += step) {
                const int64_t r = t * kBlock;
                if (kAhead) ahead(t + 2 * step);
                for (int i = 0; i < kBlock && ok; i += kRowsZ)
                    piece(q.grad_y, kAct != kActNone ? q.pre : nullptr, r + i, kRowsZ, q.n);
                if (q.want_w)
                    for (int i = 0; i < kBlock && ok; i += kRowsX)
                        piece(q.x, nullptr, r + i, kRowsX, q.k);
            }
            if (!ok) {   // give the copies in flight one more bounded wait
                *s_fail = 1u;
                for (int k = f > L::pieces ? f - L::pieces : 0; k < f; ++k)
                    mbar_wait(raw_full + k % L::pieces, (k / L::pieces) & 1);
            }
        }
    } else if (warp == 0) {
        if (elect_one()) {   // ---- MMAs
            constexpr uint32_t kBase = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) |
                                       ((uint32_t)(kBlock >> 4) << 24);   // B MN-major
            constexpr uint32_t kAMn = 1u << 15;
            const uint32_t base = smem_u32(smem);
            const uint32_t k16 = (uint32_t)(q.k + 15) / 16 * 16;
            const int steps_n = (q.n + 15) / 16;
            int u = 0;
            bool ok = true;
            for (int64_t t = first; t < q.tiles; t += step, ++u) {
                const int sz = u % L::dzs, sx = u % L::xs;
                ok = mbar_wait(dz_full + sz, (u / L::dzs) & 1) && !*s_fail;
                if (!ok) break;
                const uint32_t dz = base + sz * L::operand, x = base + L::x + sx * L::operand;
                if (q.want_x) {   // (while x's operand is made)
                    // (one accumulator in 32 bits, two in 16)
                    const int buf = kSplit ? 0 : u & 1, turn = kSplit ? u : u >> 1;
                    ok = mbar_wait(dx_empty + buf, (turn & 1) ^ 1) && !*s_fail;
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * 128;
                    const uint64_t b = desc_sw128(base + L::weight, L::weight_panel);
                    for (int e = 0; e < steps_n; ++e) {
                        const uint32_t at = dz + (e >> 2) * kPlanes * L::panel + (e & 3) * 32;
                        const uint64_t be = b + (2048u * e >> 4);
                        if constexpr (kSplit) {
                            mma_f16(d, desc_sw128(at, 16), be, kBase | (192u >> 3 << 17), e > 0);
                            mma_f16(d + 64, desc_sw128(at + L::panel, 16), be,
                                    kBase | (128u >> 3 << 17), 1);
                            mma_f16(d + 128, desc_sw128(at + 2 * L::panel, 16), be,
                                    kBase | (64u >> 3 << 17), 1);
                        } else {
                            mma_f16(d, desc_sw128(at, 16), be, kBase | (k16 >> 3 << 17), e > 0);
                        }
                    }
                    mma_commit(dx_full + buf);
                }
                if (q.want_w) {
                    // (in 32 bits one accumulator, drained every tile; in 16 two, every piece)
                    const int piece = kSplit ? u : u / kPieceTiles, buf = kSplit ? 0 : piece & 1;
                    const bool begins = kSplit || u % kPieceTiles == 0;
                    const bool ends = kSplit || u % kPieceTiles == kPieceTiles - 1;
                    ok = mbar_wait(x_full + sx, (u / L::xs) & 1) && !*s_fail;
                    if (begins && ok)
                        ok = mbar_wait(dw_empty + buf, ((kSplit ? piece : piece >> 1) & 1) ^ 1) &&
                             !*s_fail;
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + kDw + buf * 128;
                    const uint64_t a = desc_sw128(dz, L::panel), b = desc_sw128(x, L::panel);
                    const uint64_t lo = desc_sw128(dz + 2 * L::panel, L::panel);
                    for (int e = 0; e < kBlock / 16; ++e) {
                        const uint32_t off = 2048u * e >> 4;
                        if constexpr (kSplit) {
                            mma_f16(d, a + off, b + off, kBase | kAMn | (192u >> 3 << 17), e > 0);
                            mma_f16(d + 128, lo + off, b + off, kBase | kAMn | (64u >> 3 << 17), 1);
                        } else {
                            mma_f16(d, a + off, b + off, kBase | kAMn | (k16 >> 3 << 17),
                                    !begins || e > 0);
                        }
                    }
                    if (ends || t + step >= q.tiles) mma_commit(dw_full + buf);
                    mma_commit(x_empty + sx);
                }
                mma_commit(dz_empty + sz);
            }
            if (!ok) {
                *s_fail = 1u;
                mma_commit(drain);
                mbar_wait(drain, 0);
            }
        }
    } else if (warp < 9) {   // ---- operands
        const int mine = tid - 32;
        float sum[kPanels][V], none[kPanels][V];
#pragma unroll
        for (int h = 0; h < kPanels; ++h)
#pragma unroll
            for (int e = 0; e < V; ++e) sum[h][e] = none[h][e] = 0.0f;
        int u = 0, f = 0;
        bool ok = true;
        // the piece in turn (where the tensors do not begin on 16 bytes there are none)
        const auto wait_piece = [&]() {
            if (kForm == 2 || q.raw)
                ok = warp_all(mbar_wait(raw_full + f % L::pieces, (f / L::pieces) & 1) && !*s_fail);
            return ok;
        };
        const auto done_piece = [&]() {
            __syncwarp();
            if ((kForm == 2 || q.raw) && lane == 0) mbar_arrive(raw_empty + f % L::pieces);
            ++f;
        };
        for (int64_t t = first; t < q.tiles; t += step, ++u) {
            const int sz = u % L::dzs, sx = u % L::xs;
            const int64_t row0 = t * kBlock, left = q.rows - row0;
            const int rows = (int)(left < kBlock ? left : kBlock);
            const auto given = [&](uint64_t* full) {   // an operand is complete
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full);
            };
            ok = warp_all(mbar_wait(dz_empty + sz, ((u / L::dzs) & 1) ^ 1) && !*s_fail);
#pragma unroll 1
            for (int i = 0; i < kBlock && ok; i += kRowsZ) {
                if (!wait_piece()) break;
                const T* raw = reinterpret_cast<const T*>(smem + L::raw + f % L::pieces * L::piece);
                const T* z = raw + L::piece / 2 / (int)sizeof(T);
                unsigned char* to = smem + sz * L::operand + i * 128;
                if (kForm == 2 || q.vec_n) {
                    make_operand<T, kAct, kPanels, true, kRowsZ>(to, raw, z, rows - i, q.n, true,
                                                                 true, mine, sum);
                } else {
                    const int64_t at = (row0 + i) * q.n;
                    make_operand<T, kAct, kPanels, true, kRowsZ>(
                        to, q.raw ? raw : static_cast<const T*>(q.grad_y) + at,
                        q.raw ? z : static_cast<const T*>(q.pre) + at, rows - i, q.n, q.raw,
                        false, mine, sum);
                }
                done_piece();
            }
            if (!ok) break;
            given(dz_full + sz);
            if (q.want_w) {
                ok = warp_all(mbar_wait(x_empty + sx, ((u / L::xs) & 1) ^ 1) && !*s_fail);
#pragma unroll 1
                for (int i = 0; i < kBlock && ok; i += kRowsX) {
                    if (!wait_piece()) break;
                    const T* raw =
                        reinterpret_cast<const T*>(smem + L::raw + f % L::pieces * L::piece);
                    unsigned char* to = smem + L::x + sx * L::operand + i * 128;
                    if (kForm == 2 || q.vec_k)
                        make_operand<T, kActNone, kPanels, false, kRowsX>(to, raw, nullptr, rows - i,
                                                                          q.k, true, true, mine,
                                                                          none);
                    else
                        make_operand<T, kActNone, kPanels, false, kRowsX>(
                            to, q.raw ? raw : static_cast<const T*>(q.x) + (row0 + i) * q.k, nullptr,
                            rows - i, q.k, q.raw, false, mine, none);
                    done_piece();
                }
                if (!ok) break;
                given(x_full + sx);
            }
        }
        if (!ok) *s_fail = 1u;
        if (q.sums) {   // the rows of threads: in a warp, then between the warps
            constexpr int kLanes = kPanel / V;
#pragma unroll
            for (int h = 0; h < kPanels; ++h)
#pragma unroll
                for (int e = 0; e < V; ++e)
#pragma unroll
                    for (int d = kLanes; d < 32; d *= 2)
                        sum[h][e] += __shfl_xor_sync(0xffffffffu, sum[h][e], d);
            // (every raw piece has been read by all of these warps)
            float* all = reinterpret_cast<float*>(smem + L::raw);
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (lane < kLanes)
#pragma unroll
                for (int h = 0; h < kPanels; ++h)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        all[(warp - 1) * L::side + h * kPanel + lane * V + e] = sum[h][e];
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (mine < q.n) {
                float v[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) v[w] = all[w * L::side + mine];
                q.sums[(int64_t)blockIdx.x * q.n + mine] =
                    ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            }
        }
    } else {   // ---- epilogue
        const int e0 = warp - 9, quarter = warp & 3, group = e0 >> 2;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        float dw[kSplit ? 32 : 1];
#pragma unroll
        for (int e = 0; e < (kSplit ? 32 : 1); ++e) dw[e] = 0.0f;
        float4* x = reinterpret_cast<float4*>(smem + L::exchange) + e0 * (kSplit ? 64 : 256);
        // 32 columns of dx, a row in each lane
        auto store_dx = [&](const float (&v)[32], int64_t t, int c0) {
            const int64_t r0 = t * kBlock + quarter * 32;
            if constexpr (kSplit) {
                finish_small<T, kActNone, true, kForm >= 1>(q.out, x, v, r0, c0, 0, lane);
            } else {
                Share<T, kForm >= 1, false> share;
                const float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                share.begin(q.out, r0, c0, 0, lane);
                share.template end<kActNone>(q.out, x, v, bias, r0, c0, 0, lane);
            }
        };
        // a lane has a row of its part of dW
        const int row = kSplit ? (quarter & 1) * 32 + lane : quarter * 32 + lane;
        const auto part_of = [&]() {
            return q.parts + ((int64_t)blockIdx.x * (kSplit ? 2 : 1) +
                              (kSplit ? quarter >> 1 : 0)) * q.part +
                   (int64_t)row * q.k;
        };
        bool ok = true;
        int u = 0;
        for (int64_t t = first; t < q.tiles; t += step, ++u) {
            if (q.want_x) {
                const int buf = kSplit ? 0 : u & 1, turn = kSplit ? u : u >> 1;
                ok = warp_all(mbar_wait(dx_full + buf, turn & 1) && !*s_fail);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = group * 32; c < (kSplit ? 64 : q.k); c += 64) {
                    float v[32];
#pragma unroll
                    for (int p = 0; p < kPlanes; ++p) {
                        uint32_t w[32];
                        __syncwarp();
                        tmem_ld32(tmem + buf * 128 + lanes + p * 64 + c, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[e] = p ? v[e] + __uint_as_float(w[e]) : __uint_as_float(w[e]);
                    }
                    if (c + 64 >= (kSplit ? 64 : q.k)) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(dx_empty + buf);
                    }
                    store_dx(v, t, c);
                }
                if (!kSplit && group * 32 >= q.k && lane == 0) mbar_arrive(dx_empty + buf);
            }
            if (kSplit && q.want_w) {
                ok = warp_all(mbar_wait(dw_full, u & 1) && !*s_fail);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    if (p == 2 && quarter >= 2) continue;   // mid lo, and what lies behind lo
                    uint32_t w[32];
                    __syncwarp();
                    tmem_ld32(tmem + kDw + lanes + p * 64 + group * 32, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) dw[kSplit ? e : 0] += __uint_as_float(w[e]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dw_empty);
            }
            if (!kSplit && q.want_w &&
                (u % kPieceTiles == kPieceTiles - 1 || t + step >= q.tiles)) {
                const int piece = u / kPieceTiles, buf = piece & 1;
                ok = warp_all(mbar_wait(dw_full + buf, (piece >> 1) & 1) && !*s_fail);
                if (!ok) break;
                tc_fence_after();
                float* part = part_of();
#pragma unroll 1
                for (int c = group * 32; c < q.k; c += 64) {
                    uint32_t w[32];
                    __syncwarp();
                    tmem_ld32(tmem + kDw + buf * 128 + lanes + c, w);
                    tmem_wait_ld();
                    if (row >= q.n) continue;
                    add_part(part + c, w, q.k - c, piece > 0);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(dw_empty + buf);
            }
        }
        if constexpr (kSplit) {
            if (ok && q.want_w && row < q.n) {
                float* part = part_of();
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (group * 32 + e < q.k) part[group * 32 + e] = dw[e];
            }
        }
        if (!ok) *s_fail = 1u;
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *s_fail) atomicOr(&st->error, kErrTimeout);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ plans --
// The plan of a narrow layer; false where it is none.
template <typename T>
bool stream_plan(const LinearCall& c, Stream* q, int* smem) {
    constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
    if (!is_stream<T>(c.inputs, c.outputs)) return false;
    q->x = c.x;
    q->weight = c.weight;
    q->tiles = ceil_div(c.rows, kBlock);
    q->k = (int)c.inputs;
    q->panels = (int)ceil_div(c.inputs, kPanel);
    q->blocks = (int)ceil_div(c.outputs, kStreamN<T>);
    q->np = q->blocks > 1 ? kStreamN<T> : (int)ceil_div(c.outputs, 16) * 16;
    q->shift = (int)(reinterpret_cast<uintptr_t>(c.x) & 15u);
    q->vec = c.inputs % VecOf<T>::n == 0 && q->shift == 0;
    q->vec_w = c.inputs % VecOf<T>::n == 0 && aligned16(c.weight);
    // as many operands, then raw tiles in flight as fit
    const auto fits = [&](int raws, int units) {
        *smem = stream_smem(kPlanes, sizeof(T), q->k, q->panels, q->np, raws, units, q->shift)
                    .bytes;
        return *smem <= kStreamSmemMax;
    };
    for (int units = 2; units >= 1; --units)
        for (int raws = 4; raws >= units; --raws)
            if (fits(raws, units)) {
                q->raws = raws;
                q->units = units;
                return true;
            }
    return false;
}

template <typename T, int kPanels>
constexpr size_t back_smem(bool act) {
    return act ? BackSmem<T, kPanels, true>::bytes : BackSmem<T, kPanels, false>::bytes;
}

template <typename T, int kPanels>
cudaError_t prepare_back() {
    cudaError_t e = cudaSuccess;
    for (auto* f : {k_linear_narrow<T, kActNone, kPanels, 2>, k_linear_narrow<T, kActSilu, kPanels, 2>,
                    k_linear_narrow<T, kActRelu, kPanels, 2>, k_linear_narrow<T, kActNone, kPanels, 1>,
                    k_linear_narrow<T, kActSilu, kPanels, 1>, k_linear_narrow<T, kActRelu, kPanels, 1>,
                    k_linear_narrow<T, kActNone, kPanels, 0>, k_linear_narrow<T, kActSilu, kPanels, 0>,
                    k_linear_narrow<T, kActRelu, kPanels, 0>})
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)(back_smem<T, kPanels>(true) > back_smem<T, kPanels>(false)
                                               ? back_smem<T, kPanels>(true)
                                               : back_smem<T, kPanels>(false)));
    return e;
}

}  // namespace

template <typename T>
bool is_stream(int64_t inputs, int64_t outputs) {
    return inputs <= kStreamMaxK && outputs <= kStreamBlocks * kStreamN<T>;
}
template bool is_stream<float>(int64_t, int64_t);
template bool is_stream<__nv_bfloat16>(int64_t, int64_t);

template <typename T>
bool launch_stream(const LinearCall& c, const Result& q, LearnState* st, int n_sms, cudaStream_t s,
                   cudaError_t* e) {
    Stream narrow{};
    int smem = 0;
    if (!stream_plan<T>(c, &narrow, &smem)) return false;
    narrow.out = q;
    narrow.skip = q.residual && aligned16(q.residual) && narrow.blocks == 1;
    const int64_t per = n_sms / narrow.blocks;
    const int64_t grid = narrow.blocks * (narrow.tiles < per ? narrow.tiles : per);
    auto* kernel = !q.vec       ? k_linear_stream<T, false, true>
                   : q.residual ? k_linear_stream<T, true, true>
                                : k_linear_stream<T, true, false>;
    *e = launch_pdl(kernel, dim3((unsigned)grid), dim3(kStreamThreads),
                      (size_t)smem, s, narrow, st);
    return true;
}
template bool launch_stream<float>(const LinearCall&, const Result&, LearnState*, int, cudaStream_t,
                                   cudaError_t*);
template bool launch_stream<__nv_bfloat16>(const LinearCall&, const Result&, LearnState*, int,
                                           cudaStream_t, cudaError_t*);

template <typename T>
bool is_narrow(int64_t inputs, int64_t outputs) {
    return inputs <= kBackSide<T> && outputs <= kBackSide<T>;
}
template bool is_narrow<float>(int64_t, int64_t);
template bool is_narrow<__nv_bfloat16>(int64_t, int64_t);

// A CTA's, or in 32 bits its two.
template <typename T>
int narrow_parts(int64_t rows, int n_sms) {
    const int64_t tiles = ceil_div(rows, kBlock);
    return (int)(tiles < n_sms ? tiles : n_sms) * (sizeof(T) == 4 ? 2 : 1);
}
template int narrow_parts<float>(int64_t, int);
template int narrow_parts<__nv_bfloat16>(int64_t, int);

template <typename T>
cudaError_t launch_narrow(const LinearCall& c, float* parts, float* sums, LearnState* st, int n_sms,
                          cudaStream_t s) {
    const int64_t m = c.rows, k = c.inputs, n = c.outputs;
    Narrow q{};
    q.grad_y = c.grad_y;
    q.pre = c.pre;
    q.x = c.x;
    q.weight = c.weight;
    q.rows = m;
    q.tiles = ceil_div(m, kBlock);
    q.k = (int)k;
    q.n = (int)n;
    const bool act = c.act != kActNone;
    q.raw = aligned16(c.grad_y) && (!act || aligned16(c.pre)) && aligned16(c.x);
    q.vec_n = q.raw && n % VecOf<T>::n == 0;
    q.vec_k = q.raw && k % VecOf<T>::n == 0;
    q.vec_w = aligned16(c.weight) && k % 8 == 0;
    q.want_x = c.grad_x != nullptr;
    q.want_w = c.grad_weight != nullptr;
    q.parts = parts;
    q.part = part_size(n, k);
    q.sums = c.grad_bias ? sums : nullptr;
    q.out.m = m;
    q.out.n = k;
    q.out.out = c.grad_x;
    q.out.vec = vec4<T>(q.out);
    const unsigned ctas = (unsigned)(q.tiles < n_sms ? q.tiles : n_sms);
    const auto run = [&](auto panels) {
        constexpr int kPanels = decltype(panels)::value;
        const auto pick = [&](auto form) {
            constexpr int kForm = decltype(form)::value;
            return c.act == kActSilu   ? k_linear_narrow<T, kActSilu, kPanels, kForm>
                   : c.act == kActRelu ? k_linear_narrow<T, kActRelu, kPanels, kForm>
                                       : k_linear_narrow<T, kActNone, kPanels, kForm>;
        };
        return launch_pdl(!q.out.vec             ? pick(std::integral_constant<int, 0>())
                          : q.vec_n && q.vec_k ? pick(std::integral_constant<int, 2>())
                                               : pick(std::integral_constant<int, 1>()),
                          dim3(ctas), dim3(kBackThreads), back_smem<T, kPanels>(act), s, q, st);
    };
    return k <= kPanel && n <= kPanel ? run(std::integral_constant<int, 1>())
                                      : run(std::integral_constant<int, kBackSide<T> / kPanel>());
}
template cudaError_t launch_narrow<float>(const LinearCall&, float*, float*, LearnState*, int,
                                          cudaStream_t);
template cudaError_t launch_narrow<__nv_bfloat16>(const LinearCall&, float*, float*, LearnState*,
                                                  int, cudaStream_t);

cudaError_t prepare_narrow() {
    cudaError_t e = prepare_back<float, 1>();
    if (e == cudaSuccess) e = prepare_back<__nv_bfloat16, 1>();
    if (e == cudaSuccess) e = prepare_back<__nv_bfloat16, 2>();
    for (auto* f : {k_linear_stream<float, true, true>, k_linear_stream<float, true, false>,
                    k_linear_stream<float, false, true>, k_linear_stream<__nv_bfloat16, true, true>,
                    k_linear_stream<__nv_bfloat16, true, false>,
                    k_linear_stream<__nv_bfloat16, false, true>})
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kStreamSmemMax);
    return e;
}

}  // namespace linear
}  // namespace pulsar
