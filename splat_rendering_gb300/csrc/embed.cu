// Codebook embedding with scaling, and its gradient by sorted tokens.
//
//   out_i = s table[t_i]                    (a zero row where t_i < 0)
//   dtable_v = s sum_{i: t_i = v} dout_i    (in the order of i)
//
// Forward: one pass, bound by the bytes of `out`.  Lanes take 16-byte vectors
// of a row; four rows per thread are in flight (eight: 21.5 us against 16.0),
// and the output goes past the caches (16.0 -> 11.7 us at 1M x 16 floats from
// 8192 rows, 5.8 TB/s).
//
// Backward: the tokens are sorted (a stable radix sort of (token, i) pairs),
// so that a table row's terms lie in a run of sorted positions and are summed
// in the order of i by threads that own the run's columns: no floating-point
// atomics, the same result every time.  Runs longer than a thread's share are
// cut, and the parts joined in order, first inside a block and then between
// blocks.  The second join is one block's: a token that takes every position
// costs little more than others in rows of up to some 64 floats (1M x 16: 58
// us against 62 with cold caches; 262144 x 64: 48 against 38), but its chain
// of tiles is what wide rows wait for (16381 x 1024 in 16 bits: 152 us against
// 46, and 83 where it takes half of the positions).
// Sums are held in 32 bits and scaled and rounded once.
#include "learn_internal.cuh"

namespace pulsar {
namespace {

constexpr int kThreads = 256;

// --------------------------------------------------------------- forward --
constexpr int kFwdRows = 4;   // rows in flight per thread

// A thread's lane covers columns lane, lane + L, ... (vectors of V elements)
// of the rows slot, slot + S, ... of its block, S = kThreads / L.
template <typename T, typename I, int V>
__global__ void __launch_bounds__(kThreads)
k_embed_rows(const T* __restrict__ table, const I* __restrict__ tokens, int64_t n, int64_t rows,
             int nv, int lshift, float scale, T* __restrict__ out, LearnState* st) {
    pdl_begin();
    const int lane = threadIdx.x & ((1 << lshift) - 1);
    const int slots = kThreads >> lshift;
    const int64_t i0 = (int64_t)blockIdx.x * (slots * kFwdRows) + (threadIdx.x >> lshift);
    int64_t t[kFwdRows];
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kFwdRows; ++u) {
        const int64_t i = i0 + (int64_t)u * slots;
        t[u] = i < n ? (int64_t)tokens[i] : -1;
        if (t[u] >= rows) {
            t[u] = -1;
            bad = true;
        }
    }
    if (bad) atomicOr(&st->error, kErrIndex);
    for (int v = lane; v < nv; v += 1 << lshift) {
        float x[kFwdRows][V];
#pragma unroll
        for (int u = 0; u < kFwdRows; ++u) {
            if (t[u] >= 0) {
                Pack<T, V>::load(table + (t[u] * nv + v) * V, x[u]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) x[u][j] = 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < kFwdRows; ++u) {
            const int64_t i = i0 + (int64_t)u * slots;
            if (i >= n) break;
            // a masked row stays zero whatever the scale
            if (t[u] >= 0) {
#pragma unroll
                for (int j = 0; j < V; ++j) x[u][j] *= scale;
            }
            Pack<T, V>::store_through(out + (i * nv + v) * V, x[u]);
        }
    }
}

// ------------------------------------------------------------------ sort --
// (key, position) pairs in the order of the keys, equal keys in the order of
// the positions.  Keys are the tokens, `rows` standing for a token that
// contributes nothing.
template <typename I>
__device__ __forceinline__ uint32_t token_key(I t, uint32_t rows, bool* bad) {
    const int64_t v = (int64_t)t;
    if (v >= (int64_t)rows) *bad = true;
    return v >= 0 && v < (int64_t)rows ? (uint32_t)v : rows;
}

// The table rows' marks (set by the reduction where a row is written) start
// at zero: the grid's threads clear them.
__device__ __forceinline__ void clear_marks(unsigned char* __restrict__ marks, uint32_t rows) {
    uint32_t* w = reinterpret_cast<uint32_t*>(marks);   // (padded to whole words)
    for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < (rows + 3) / 4;
         i += gridDim.x * blockDim.x)
        w[i] = 0u;
}

// Few tokens: one launch, a token's place is the number of keys before it,
// counted against all of them in shared memory by sixteen threads (one thread
// a token, bound by its own chain of additions, took 43 us at 4000 tokens; now
// 7, and the radix sort's four launches 18 at 6000).
constexpr int kRankMost = 4096;
constexpr int kRankThreads = 512, kRankLanes = 16;
constexpr int kRankTokens = kRankThreads / kRankLanes;   // of a block

template <typename I>
__global__ void __launch_bounds__(kRankThreads)
k_sort_rank(const I* __restrict__ tokens, uint32_t n, uint32_t rows,
            uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out,
            unsigned char* __restrict__ marks, LearnState* st) {
    pdl_begin();
    __shared__ __align__(16) uint32_t key[kRankMost];
    bool bad = false;
    const uint32_t padded = (n + 3) / 4 * 4;
#pragma unroll 8
    for (uint32_t i = threadIdx.x; i < padded; i += kRankThreads)
        key[i] = i < n ? token_key(tokens[i], rows, &bad) : 0xffffffffu;
    if (bad) atomicOr(&st->error, kErrIndex);
    clear_marks(marks, rows);
    __syncthreads();
    const uint32_t i = blockIdx.x * kRankTokens + threadIdx.x / kRankLanes;
    const uint32_t lane = threadIdx.x % kRankLanes;
    const uint32_t k = i < n ? key[i] : 0u, own = i / 4;
    uint32_t at[4] = {0u, 0u, 0u, 0u};
    // keys at or below its own in the vectors before its own, keys below it from there on ...
#pragma unroll 4
    for (uint32_t v = lane; v < padded / 4; v += kRankLanes) {
        const uint4 u = reinterpret_cast<const uint4*>(key)[v];
        const uint32_t t = k + (v < own ? 1u : 0u);
        at[0] += u.x < t;
        at[1] += u.y < t;
        at[2] += u.z < t;
        at[3] += u.w < t;
    }
    // ... and those equal to it that stand before it in its own vector
    if (lane == 0)
        for (uint32_t e = own * 4; e < i; ++e) at[0] += key[e] == k;
    uint32_t sum = at[0] + at[1] + at[2] + at[3];
#pragma unroll
    for (int o = kRankLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0 && i < n) {
        keys_out[sum] = k;
        pos_out[sum] = i;
    }
}

// More: a stable LSD radix sort.  A pass is two launches: every block counts
// the digits of its contiguous chunk; then every block sums the count matrix
// to its own offsets, orders its chunk by the digit in shared memory and
// writes it out from there, so that stores of a digit lie side by side.
// 1M tokens of 14 bits: count 2 us, scatter 11 us a pass -- offsets 2.5,
// items 2.2, ranking 3.5 (ballots: the integer pipe), ordering 2, writing 1
// -- of which every part is latency or issue, not bytes (16 MB, 2.4 us).
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 8;                               // most per thread at a time
constexpr int kSortTile = kSortThreads * kSortItems;        // 8192
constexpr int kMaxDigit = 8;                                // bits
constexpr int kMaxBins = 1 << kMaxDigit;
constexpr size_t kSortSmem = kSortTile * 8;
constexpr uint32_t kSortBlocks = 152;                       // at most, one per SM

// counts[digit][block] of one pass; `keys` NULL: from the tokens.
template <typename I, int kDigit>
__global__ void __launch_bounds__(kSortThreads)
k_sort_count(const I* __restrict__ tokens, const uint32_t* __restrict__ keys, uint32_t n,
             uint32_t rows, uint32_t chunk, int shift, int bits, uint32_t* __restrict__ counts,
             unsigned char* __restrict__ marks, LearnState* st) {
    pdl_begin();
    constexpr int kBins = 1 << kDigit;
    __shared__ uint32_t h[kSortWarps][kBins];
    const int bins = 1 << bits, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < kSortWarps * kBins; e += kSortThreads) (&h[0][0])[e] = 0u;
    __syncthreads();
    const uint32_t lo = blockIdx.x * chunk, hi = min(n, lo + chunk);
    bool bad = false;
#pragma unroll 4
    for (uint32_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
        const uint32_t k = keys ? keys[i] : token_key(tokens[i], rows, &bad);
        atomicAdd(&h[warp][(k >> shift) & (bins - 1)], 1u);
    }
    if (bad) atomicOr(&st->error, kErrIndex);
    if (!keys) clear_marks(marks, rows);
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += kSortThreads) {
        uint32_t s = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) s += h[w][d];
        counts[(size_t)d * gridDim.x + blockIdx.x] = s;
    }
}

template <typename I, int kDigit>
__global__ void __launch_bounds__(kSortThreads)
k_sort_scatter(const I* __restrict__ tokens, const uint32_t* __restrict__ keys,
               const uint32_t* __restrict__ pos, uint32_t n, uint32_t rows, uint32_t chunk,
               int shift, int bits, const uint32_t* __restrict__ counts,
               uint32_t* __restrict__ keys_out, uint32_t* __restrict__ pos_out) {
    pdl_begin();
    constexpr int kBins = 1 << kDigit, kPerWarp = kBins / kSortWarps;   // digits a warp sums
    static_assert(kBins % 32 == 0 && kPerWarp >= 1, "digits");
    extern __shared__ uint2 s_pair[];                 // [kSortTile] the tile in order
    __shared__ uint32_t base[kBins];               // next output position of each digit
    __shared__ uint32_t total[kBins];              // of the sort; then of the tile
    __shared__ uint32_t start[kBins];              // where a digit begins in the tile
    __shared__ uint32_t wh[kSortWarps][kBins];     // per warp: count, then offset in the tile
    const int bins = 1 << bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t nb = gridDim.x, b = blockIdx.x;
    {   // a warp's digits together, so that their counts load together
        uint32_t all[kPerWarp], before[kPerWarp];
#pragma unroll
        for (int e = 0; e < kPerWarp; ++e) all[e] = before[e] = 0u;
        for (uint32_t q = lane; q < nb; q += 32) {
#pragma unroll
            for (int e = 0; e < kPerWarp; ++e) {
                const int d = warp + e * kSortWarps;
                const uint32_t c = d < bins ? counts[(size_t)d * nb + q] : 0u;
                all[e] += c;
                before[e] += q < b ? c : 0u;
            }
        }
#pragma unroll
        for (int e = 0; e < kPerWarp; ++e) {
            const int d = warp + e * kSortWarps;
            const uint32_t s = __reduce_add_sync(0xffffffffu, all[e]);
            const uint32_t f = __reduce_add_sync(0xffffffffu, before[e]);
            if (lane == 0) {
                total[d] = s;
                base[d] = f;
            }
        }
    }
    __syncthreads();
    // exclusive scan of the totals, by one warp: digit d's sum to f(d, sum)
    const auto scan_totals = [&](auto&& f) {
        uint32_t c[kBins / 32], sum = 0;
#pragma unroll
        for (int e = 0; e < kBins / 32; ++e) sum += c[e] = total[lane * (kBins / 32) + e];
        uint32_t s = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += up;
        }
        s -= sum;
#pragma unroll
        for (int e = 0; e < kBins / 32; ++e) {
            f(lane * (kBins / 32) + e, s);
            s += c[e];
        }
    };
    if (warp == 0) scan_totals([&](int d, uint32_t s) { base[d] += s; });
    const uint32_t lo = b * chunk, hi = min(n, lo + chunk);
    bool bad = false;
    for (uint32_t t0 = lo; t0 < hi; t0 += kSortTile) {
        // the warps share the tile's items evenly, each a contiguous run of 32 x rounds
        const int rounds = (int)((min(hi - t0, (uint32_t)kSortTile) + kSortThreads - 1) / kSortThreads);
        for (int e = threadIdx.x; e < kSortWarps * kBins; e += kSortThreads)
            (&wh[0][0])[e] = 0u;
        uint32_t key[kSortItems], val[kSortItems], rank[kSortItems];
        const uint32_t i0 = t0 + warp * (32 * rounds) + lane;
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            const uint32_t i = i0 + 32 * j;
            key[j] = 0;
            val[j] = i;
            if (j < rounds && i < hi) {
                key[j] = keys ? keys[i] : token_key(tokens[i], rows, &bad);
                if (pos) val[j] = pos[i];
            }
        }
        __syncthreads();
        // rank inside the warp's items, in their order
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            if (j < rounds) {
                const bool on = i0 + 32 * j < hi;
                const uint32_t d = (key[j] >> shift) & (bins - 1);
                uint32_t same = __ballot_sync(0xffffffffu, on);   // (faster than a match)
#pragma unroll
                for (int q = 0; q < kDigit; ++q) {
                    const uint32_t m = __ballot_sync(0xffffffffu, (d >> q) & 1u);
                    same &= (d >> q) & 1u ? m : ~m;
                }
                const uint32_t before = __popc(same & ((1u << lane) - 1u));
                rank[j] = on ? wh[warp][d] + before : 0u;
                __syncwarp();
                if (on && before == 0) wh[warp][d] += __popc(same);
                __syncwarp();
            }
        }
        __syncthreads();
        for (int d = threadIdx.x; d < kBins; d += kSortThreads) {
            uint32_t run = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = wh[w][d];
                wh[w][d] = run;
                run += c;
            }
            total[d] = run;
        }
        __syncthreads();
        if (warp == 0) scan_totals([&](int d, uint32_t s) { start[d] = s; });
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            if (j < rounds && i0 + 32 * j < hi) {
                const uint32_t d = (key[j] >> shift) & (bins - 1);
                s_pair[start[d] + wh[warp][d] + rank[j]] = make_uint2(key[j], val[j]);
            }
        }
        __syncthreads();
        const uint32_t count = min(hi - t0, (uint32_t)kSortTile);
#pragma unroll 4
        for (uint32_t i = threadIdx.x; i < count; i += kSortThreads) {
            const uint2 u = s_pair[i];
            const uint32_t d = (u.x >> shift) & (bins - 1), at = base[d] + i - start[d];
            keys_out[at] = u.x;
            pos_out[at] = u.y;
        }
        __syncthreads();
        for (int d = threadIdx.x; d < kBins; d += kSortThreads) base[d] += total[d];
        __syncthreads();
    }
}

// ------------------------------------------------------------- reduction --
constexpr int kAhead = 8;        // gathered rows in flight per thread
constexpr int kMostQ = 32;       // positions per slot

// A block's tile is S slots x q sorted positions, S = kThreads / L; the L
// lanes of a slot own columns (vectors of V) and walk the slot's positions.
// Equal tiles, whatever rows they hold, are one wave of blocks; the gather of
// rows in sorted order is what bounds it: 64 MB of 64-byte rows in 16 us (4
// TB/s), 33 MB of 2 KB rows and 22 MB of results in 12 us.
// A run that lies inside a slot goes straight to the table.  A slot keeps two
// parts of runs that do not: `head`, of a run that began before the slot (and
// may pass through it), and `tail`, of a run that begins in it and goes on.
// The slot where a run begins joins its parts in order; what leaves the tile
// goes to tile_head / tile_tail for k_embed_join.  Where a row is written its
// mark is set.
enum : int { kHasHead = 1, kThrough = 2, kHasTail = 4 };

constexpr int reduce_blocks_per_sm(int v) { return v == 8 ? 3 : 4; }

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, reduce_blocks_per_sm(V))
k_embed_reduce(const T* __restrict__ grad, const uint32_t* __restrict__ keys,
               const uint32_t* __restrict__ pos, uint32_t n, uint32_t rows, int nv, int lshift,
               int q, float scale, T* __restrict__ out, float* __restrict__ tile_head,
               float* __restrict__ tile_tail, int* __restrict__ tile_flag,
               unsigned char* __restrict__ marks) {
    pdl_begin();
    extern __shared__ __align__(16) unsigned char smem[];
    const int L = 1 << lshift, S = kThreads >> lshift;
    const int lane = threadIdx.x & (L - 1), slot = threadIdx.x >> lshift;
    const int v = blockIdx.y * L + lane;
    float* s_head = reinterpret_cast<float*>(smem);   // [kThreads][V]
    float* s_tail = s_head + kThreads * V;
    int* s_flag = reinterpret_cast<int*>(s_tail + kThreads * V);   // [S]
    uint32_t* s_key = reinterpret_cast<uint32_t*>(s_flag + S);     // [S q + 2]: with both neighbours
    uint32_t* s_pos = s_key + S * q + 2;                           // [S q]
    const uint32_t t0 = blockIdx.x * (uint32_t)(S * q), len = min((uint32_t)(S * q), n - t0);
    for (uint32_t i = threadIdx.x; i < len + 2; i += kThreads) {
        // (a key that is no token's beyond both ends)
        s_key[i] = t0 + i == 0 || t0 + i - 1 >= n ? 0xffffffffu : keys[t0 + i - 1];
        if (i < len) s_pos[i] = pos[t0 + i];
    }
    __syncthreads();
    const uint32_t* key = s_key + 1;   // key[-1], key[len]: the neighbours'
    const int p0 = min((int)len, slot * q), p1 = min((int)len, p0 + q);
    const bool col = v < nv;
    int flag = 0;
    auto emit = [&](uint32_t row, const float (&a)[V]) {
        if (row >= rows) return;
        if (v == 0) marks[row] = 1;
        if (!col) return;
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = a[j] * scale;
        Pack<T, V>::store(out + ((size_t)row * nv + v) * V, y);
    };
    uint32_t cur = rows;
    if (p0 < p1) {
        cur = key[p0];
        bool head = key[p0 - 1] == cur;   // the current run began before the slot
        float acc[V] = {};
        for (int p = p0; p < p1; p += kAhead) {
            typename Pack<T, V>::Raw x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (p + u < p1 && key[p + u] < rows && col)
                    x[u] = Pack<T, V>::raw_last(grad + ((size_t)s_pos[p + u] * nv + v) * V);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (p + u >= p1) break;
                const uint32_t k = key[p + u];
                if (k != cur) {
                    if (head) {
                        flag |= kHasHead;
#pragma unroll
                        for (int j = 0; j < V; ++j) s_head[threadIdx.x * V + j] = acc[j];
                        head = false;
                    } else {
                        emit(cur, acc);
                    }
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
                    cur = k;
                }
                if (k < rows && col) {
                    float f[V];
                    Pack<T, V>::open(x[u], f);
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[j] += f[j];
                }
            }
        }
        const bool goes_on = key[p1] == cur;
        if (head) {
            flag |= kHasHead | (goes_on ? kThrough : 0);
#pragma unroll
            for (int j = 0; j < V; ++j) s_head[threadIdx.x * V + j] = acc[j];
        } else if (goes_on) {
            flag |= kHasTail;
#pragma unroll
            for (int j = 0; j < V; ++j) s_tail[threadIdx.x * V + j] = acc[j];
        } else {
            emit(cur, acc);
        }
    }
    if (lane == 0) s_flag[slot] = flag;
    __syncthreads();
    // ---- join the parts of the runs that begin in this slot, and (slot 0)
    // of the run that began before the tile
    const size_t at = ((size_t)blockIdx.x * nv + v) * V;
    auto follow = [&](float (&a)[V], int s) {   // parts of the slots from s on; true: to the tile's end
        for (; s < S; ++s) {
            const int f = s_flag[s];
            if (!(f & kHasHead)) return false;
#pragma unroll
            for (int j = 0; j < V; ++j) a[j] += s_head[((s << lshift) + lane) * V + j];
            if (!(f & kThrough)) return false;
        }
        return true;
    };
    int tile_bits = 0;
    if (slot == 0 && (flag & kHasHead)) {
        float a[V] = {};
        const bool through = follow(a, 0);
        tile_bits |= kHasHead | (through ? kThrough : 0);
        if (col) {
#pragma unroll
            for (int j = 0; j < V; ++j) tile_head[at + j] = a[j];
        }
    }
    bool leaves = false;
    if (flag & kHasTail) {
        float a[V];
#pragma unroll
        for (int j = 0; j < V; ++j) a[j] = s_tail[threadIdx.x * V + j];
        // at the tile's end the run goes on if the next tile begins with its key
        leaves = follow(a, slot + 1) && key[len] == cur;
        if (leaves && v == 0 && cur < rows) marks[cur] = 1;   // k_embed_join writes it
        if (!leaves) {
            emit(cur, a);
        } else if (col) {
#pragma unroll
            for (int j = 0; j < V; ++j) tile_tail[at + j] = a[j];
        }
    }
    const bool any_leaves = __syncthreads_or(leaves);
    if (threadIdx.x == 0 && blockIdx.y == 0)
        tile_flag[blockIdx.x] = tile_bits | (any_leaves ? kHasTail : 0);
}

// The runs that leave the tile they begin in: one block per tile (and column
// block), its slots striding over the tiles the run covers, joined in the
// order of the slots.  Behind them, blocks that clear the rows without a mark,
// kZeroRows rows each (80 MB of them in 10 to 15 us, DRAM writes; marks, not a
// search of the sorted keys per row, which took 12 us before the first store).
constexpr int kZeroRows = 64;

template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
k_embed_join(const uint32_t* __restrict__ keys, uint32_t n, uint32_t rows, int nv, int lshift, int q,
             uint32_t tiles, float scale, T* __restrict__ out, const float* __restrict__ tile_head,
             const float* __restrict__ tile_tail, const int* __restrict__ tile_flag,
             const unsigned char* __restrict__ marks) {
    pdl_begin();
    if (blockIdx.x >= tiles - 1) {
        const uint32_t r0 = (blockIdx.x - (tiles - 1)) * kZeroRows;
        const int count = (int)min((uint32_t)kZeroRows, rows - r0);
        const int c0 = (blockIdx.y << lshift), width = min(nv - c0, 1 << lshift);
        const float zero[V] = {};
        for (int e = threadIdx.x; e < count * width; e += kThreads) {
            const int r = e / width;
            if (!marks[r0 + r])
                Pack<T, V>::store(out + ((size_t)(r0 + r) * nv + c0 + (e - r * width)) * V, zero);
        }
        return;
    }
    if (!(tile_flag[blockIdx.x] & kHasTail)) return;
    const int L = 1 << lshift, S = kThreads >> lshift;
    const int lane = threadIdx.x & (L - 1), slot = threadIdx.x >> lshift;
    const int v = blockIdx.y * L + lane;
    const uint32_t key = keys[(blockIdx.x + 1) * (uint32_t)(S * q) - 1];
    if (key >= rows) return;
    // the run's last tile: the first that it does not pass through
    uint32_t last = blockIdx.x + 1;
    for (;; last += kThreads) {
        const uint32_t t = last + threadIdx.x;
        const bool passes = t < tiles && (tile_flag[t] & kThrough);
        const uint32_t stop = __ballot_sync(0xffffffffu, !passes);
        __shared__ uint32_t first[kThreads / 32];
        if ((threadIdx.x & 31) == 0) first[threadIdx.x >> 5] = stop ? __ffs(stop) - 1 : 32u;
        __syncthreads();
        uint32_t found = kThreads;
#pragma unroll
        for (int w = kThreads / 32 - 1; w >= 0; --w)
            if (first[w] < 32u) found = 32u * w + first[w];
        __syncthreads();
        if (found < kThreads) {
            last += found;
            break;
        }
    }
    __shared__ float part[kThreads * V];
    float a[V] = {};
    if (v < nv) {
#pragma unroll 4
        for (uint32_t t = blockIdx.x + 1 + slot; t <= last; t += S) {
            const float* h = tile_head + ((size_t)t * nv + v) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) a[j] += h[j];
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) part[threadIdx.x * V + j] = a[j];
    __syncthreads();
    if (slot == 0 && v < nv) {
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = tile_tail[((size_t)blockIdx.x * nv + v) * V + j];
        for (int s = 0; s < S; ++s) {
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] += part[((s << lshift) + lane) * V + j];
        }
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] *= scale;
        Pack<T, V>::store(out + ((size_t)key * nv + v) * V, y);
    }
}

// ----------------------------------------------------------------- plans --
int log2_up(int64_t v) {
    int s = 0;
    while (((int64_t)1 << s) < v) ++s;
    return s;
}

struct SortPlan {
    int passes, bits;
    uint32_t blocks, chunk;
};
SortPlan sort_plan(int64_t n, int64_t rows) {
    SortPlan p;
    const int kb = log2_up(rows + 1) > 0 ? log2_up(rows + 1) : 1;   // keys 0 .. rows
    p.passes = (kb + kMaxDigit - 1) / kMaxDigit;
    p.bits = (kb + p.passes - 1) / p.passes;
    const int64_t per = ceil_div(n, kSortBlocks);
    p.chunk = (uint32_t)(ceil_div(per, kSortThreads) * kSortThreads);
    p.blocks = (uint32_t)ceil_div(n, p.chunk);
    return p;
}

// Tile shape of the reduction for rows of nv vectors: as many positions per
// slot as give one wave of resident blocks, kAhead to kMostQ.
struct ReducePlan {
    int lshift, q;
    uint32_t tiles;
    unsigned cols;
    size_t smem;
};
ReducePlan reduce_plan(int64_t n, int64_t nv, int v) {
    ReducePlan r;
    r.lshift = log2_up(nv);
    r.lshift = r.lshift < 2 ? 2 : r.lshift > 8 ? 8 : r.lshift;
    const int64_t S = kThreads >> r.lshift;
    const int64_t q = ceil_div(n, S * 152 * reduce_blocks_per_sm(v));
    r.q = (int)(q < kAhead ? kAhead : q > kMostQ ? kMostQ : q);
    r.tiles = (uint32_t)ceil_div(n, S * r.q);
    r.cols = (unsigned)ceil_div(nv, 1 << r.lshift);
    r.smem = 4 * (2 * (size_t)kThreads * v + S + 2 * S * r.q + 2);
    return r;
}

struct BackwardSpace {
    uint32_t *keys[2], *pos[2], *counts;
    float *head, *tail;
    int* flag;
    unsigned char* marks;
};
// V only splits a row: nv * V is dim, so the pieces have one size for both.
BackwardSpace carve(Carve& w, int64_t n, int64_t rows, int64_t dim, uint32_t tiles) {
    BackwardSpace s;
    for (int k = 0; k < 2; ++k) {
        s.keys[k] = w.take<uint32_t>(n);
        s.pos[k] = w.take<uint32_t>(n);
    }
    s.counts = w.take<uint32_t>((size_t)kMaxBins * kSortBlocks);
    s.head = w.take<float>((size_t)tiles * dim);
    s.tail = w.take<float>((size_t)tiles * dim);
    s.flag = w.take<int>(tiles);
    s.marks = w.take<unsigned char>(rows);
    return s;
}

template <typename T, typename I, int V>
cudaError_t forward(const EmbedCall& c, LearnState* st, cudaStream_t s) {
    const int64_t nv = c.dim / V;
    int ls = log2_up(nv);
    ls = ls > 5 ? 5 : ls;
    const int64_t per = (int64_t)(kThreads >> ls) * kFwdRows;
    return launch_pdl(k_embed_rows<T, I, V>, dim3((unsigned)ceil_div(c.n, per)), dim3(kThreads), 0,
                      s, (const T*)c.src, (const I*)c.tokens, c.n, c.rows, (int)nv, ls, c.scale,
                      (T*)c.dst, st);
}

template <typename T, int V>
cudaError_t reduce(const EmbedCall& c, const BackwardSpace& w, int from, const ReducePlan& r,
                   cudaStream_t s) {
    const int nv = (int)(c.dim / V);
    const uint32_t n = (uint32_t)c.n, rows = (uint32_t)c.rows;
    cudaError_t e = launch_pdl(k_embed_reduce<T, V>, dim3(r.tiles, r.cols), dim3(kThreads), r.smem,
                               s, (const T*)c.src, (const uint32_t*)w.keys[from],
                               (const uint32_t*)w.pos[from], n, rows, nv, r.lshift, r.q, c.scale,
                               (T*)c.dst, w.head, w.tail, w.flag, w.marks);
    if (e != cudaSuccess) return e;
    const unsigned zero_blocks = (unsigned)ceil_div(rows, kZeroRows);
    return launch_pdl(k_embed_join<T, V>, dim3(r.tiles - 1 + zero_blocks, r.cols), dim3(kThreads),
                      0, s, (const uint32_t*)w.keys[from], n, rows, nv, r.lshift, r.q, r.tiles,
                      c.scale, (T*)c.dst, (const float*)w.head, (const float*)w.tail,
                      (const int*)w.flag, (const unsigned char*)w.marks);
}

template <typename T, typename I>
cudaError_t backward(const EmbedCall& c, LearnState* st, void* ws, cudaStream_t s) {
    const bool wide = c.dim % VecOf<T>::n == 0 && aligned16(c.src) && aligned16(c.dst);
    const int v = wide ? VecOf<T>::n : 1;
    const ReducePlan r = reduce_plan(c.n, c.dim / v, v);
    Carve cv{static_cast<unsigned char*>(ws)};
    const BackwardSpace w = carve(cv, c.n, c.rows, c.dim, r.tiles);
    const uint32_t n = (uint32_t)c.n, rows = (uint32_t)c.rows;
    int from = 0;
    cudaError_t e = cudaSuccess;
    if (n <= kRankMost) {
        e = launch_pdl(k_sort_rank<I>, dim3((unsigned)ceil_div(n, kRankTokens)),
                       dim3(kRankThreads), 0, s, (const I*)c.tokens, n, rows, w.keys[0], w.pos[0], w.marks, st);
    } else {
        const SortPlan p = sort_plan(c.n, c.rows);
        for (int k = 0; k < p.passes && e == cudaSuccess; ++k) {
            const uint32_t* ki = k ? w.keys[(k - 1) & 1] : nullptr;
            const uint32_t* pi = k ? w.pos[(k - 1) & 1] : nullptr;
            // (the forms differ in the bins they have room for: 14 bits in two passes of 128
            // bins take 3.3 us less than with room for 256)
            const auto pass = [&](auto count, auto scatter) {
                cudaError_t f = launch_pdl(count, dim3(p.blocks), dim3(kSortThreads), 0, s,
                                           (const I*)c.tokens, ki, n, rows, p.chunk, k * p.bits,
                                           p.bits, w.counts, w.marks, st);
                if (f == cudaSuccess)
                    f = launch_pdl(scatter, dim3(p.blocks), dim3(kSortThreads), kSortSmem, s,
                                   (const I*)c.tokens, ki, pi, n, rows, p.chunk, k * p.bits, p.bits,
                                   (const uint32_t*)w.counts, w.keys[k & 1], w.pos[k & 1]);
                return f;
            };
            e = p.bits <= 6   ? pass(k_sort_count<I, 6>, k_sort_scatter<I, 6>)
                : p.bits == 7 ? pass(k_sort_count<I, 7>, k_sort_scatter<I, 7>)
                              : pass(k_sort_count<I, 8>, k_sort_scatter<I, 8>);
        }
        from = (p.passes - 1) & 1;
    }
    if (e != cudaSuccess) return e;
    return wide ? reduce<T, VecOf<T>::n>(c, w, from, r, s) : reduce<T, 1>(c, w, from, r, s);
}

}  // namespace

size_t embed_workspace(int64_t n, int64_t rows, int64_t dim) {
    if (n == 0) return 0;
    // the largest of the plans of the vector and the element forms
    uint32_t tiles = 0;
    for (int v : {1, 4, 8})
        if (dim % v == 0) {
            const uint32_t t = reduce_plan(n, dim / v, v).tiles;
            tiles = t > tiles ? t : tiles;
        }
    Carve cv{nullptr};
    carve(cv, n, rows, dim, tiles);
    return cv.used;
}

cudaError_t prepare_embed() {
    cudaError_t e = cudaSuccess;
    for (const void* k : {(const void*)k_sort_scatter<int32_t, 6>, (const void*)k_sort_scatter<int32_t, 7>,
                          (const void*)k_sort_scatter<int32_t, 8>, (const void*)k_sort_scatter<int64_t, 6>,
                          (const void*)k_sort_scatter<int64_t, 7>, (const void*)k_sort_scatter<int64_t, 8>})
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSortSmem);
    return e;
}

cudaError_t launch_embed_forward(const EmbedCall& c, LearnState* st, cudaStream_t s) {
    if (c.n == 0) return cudaSuccess;
    using B = __nv_bfloat16;
    const int v = c.dtype == kBf16 ? 8 : 4;
    const bool wide = c.dim % v == 0 && aligned16(c.src) && aligned16(c.dst);
    if (c.dtype == kF32)
        return c.index == kI32 ? (wide ? forward<float, int32_t, 4>(c, st, s)
                                       : forward<float, int32_t, 1>(c, st, s))
                               : (wide ? forward<float, int64_t, 4>(c, st, s)
                                       : forward<float, int64_t, 1>(c, st, s));
    return c.index == kI32 ? (wide ? forward<B, int32_t, 8>(c, st, s)
                                   : forward<B, int32_t, 1>(c, st, s))
                           : (wide ? forward<B, int64_t, 8>(c, st, s)
                                   : forward<B, int64_t, 1>(c, st, s));
}

cudaError_t launch_embed_backward(const EmbedCall& c, LearnState* st, void* ws, int n_sms,
                                  cudaStream_t s) {
    (void)n_sms;
    if (c.n == 0)
        return cudaMemsetAsync(c.dst, 0, (size_t)c.rows * c.dim * (c.dtype == kBf16 ? 2 : 4), s);
    if (c.dtype == kF32)
        return c.index == kI32 ? backward<float, int32_t>(c, st, ws, s)
                               : backward<float, int64_t>(c, st, ws, s);
    return c.index == kI32 ? backward<__nv_bfloat16, int32_t>(c, st, ws, s)
                           : backward<__nv_bfloat16, int64_t>(c, st, ws, s);
}

}  // namespace pulsar
