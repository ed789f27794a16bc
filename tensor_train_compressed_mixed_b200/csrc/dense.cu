#ifndef WT
#define WT 24
#endif
#ifndef SW
#define SW 8
#endif
#ifndef CW4
#define CW4 1
#endif
#ifndef CW8
#define CW8 1
#endif
#ifndef SA
#define SA 8
#endif
#ifndef CA
#define CA 2
#endif
// Dense tables: scaled lookup of rows, and the table's gradient by sorted tokens.
//
// Both move rows and do one or two operations a value, so memory bounds them.
//
// Lookup.  One thread moves 16 bytes (of the wider type) of up to four rows, whose loads are all
// issued before the first store.
//
// Gradient.  The tokens are sorted by row (stable, so equal rows stay in input order) and the sorted
// positions are cut into tiles.  A warp adds up its columns of a tile's upstream rows in fp32
// registers, one run of equal rows after the other; a run that lies inside its tile is written to
// the gradient at once, and the parts of one that crosses tiles go to the workspace and are
// added in tile order by the next kernel, which also clears the rows that no token names.  So every
// row of the gradient is written once, a row that many tokens name is spread over many warps, and
// no sum depends on the order in which blocks run.
#include <cooperative_groups.h>
#include <new>
#include <type_traits>

#include "types.cuh"

using namespace tt;

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ int64_t token_at(const void* tokens, int token_bytes, int64_t i)
{
    return token_bytes == 8 ? ((const int64_t*)tokens)[i] : (int64_t)((const int32_t*)tokens)[i];
}

struct LookupArgs {
    const void* tokens;
    int64_t n, rows, out_stride;
    int token_bytes, dim;
    float scale;
    int lanes;           // lanes that share a row, a power of two
    int slabs;           // units of the same tokens, 32 * kCols vectors of a row each
    int32_t* status;
};

// A warp takes a unit: some tokens and a slab of their rows.  A step moves 32 / lanes rows; the loads
// of all kSteps steps are issued before the first store.  No load hangs on a condition, so that
// none waits for another: places behind the last token read the last one's row, tokens outside the
// table row 0.
template <typename T, typename O, int V, int kCols, int kSteps>
__global__ void __launch_bounds__(kThreads) k_lookup(LookupArgs a, const T* __restrict__ table, O* __restrict__ out)
{
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), group = unit / a.slabs;
    const int rows = 32 / a.lanes;
    const int64_t i0 = group * (rows * kSteps < 32 ? rows * kSteps : 32);
    if (i0 >= a.n) return;
    const int cnt = (int)min64(min(32, rows * kSteps), a.n - i0);
    int64_t token = token_at(a.tokens, a.token_bytes, i0 + min(lane, cnt - 1));
    const bool stop = has_error(a.status);
    const bool bad = token < 0 || token >= a.rows;
    if (bad) token = 0;
    const int sub = lane & (a.lanes - 1), own = lane / a.lanes;
    const int c0 = ((int)(unit - group * a.slabs) * kCols * 32 + sub) * V;
    Pack<T, V> x[kSteps][kCols];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int64_t row = __shfl_sync(kFull, token, min(s * rows + own, cnt - 1));
#pragma unroll
        for (int k = 0; k < kCols; ++k) {
            const int c = c0 + k * 32 * V;
            x[s][k] = *reinterpret_cast<const Pack<T, V>*>(table + row * a.dim + (c < a.dim ? c : 0));
        }
    }
    if (stop) return;
    if (bad && lane < cnt) raise_error(a.status, TT_ERR_INDEX_RANGE, (int)min64(i0 + lane, INT32_MAX));
    const unsigned good = __ballot_sync(kFull, !bad);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int i = s * rows + own;
        if (i >= cnt || !(good >> i & 1u)) continue;
#pragma unroll
        for (int k = 0; k < kCols; ++k) {
            const int c = c0 + k * 32 * V;
            float y[V];
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = to_f32(x[s][k].v[j]) * a.scale;
            if (c < a.dim) store_pack(out + (i0 + i) * a.out_stride + c, y);
        }
    }
}

// ---------------------------------------------------------------------------
// Sorted tokens: keys ascending, each with its input position, equal keys in input order.  A key is
// the token, or `rows` (behind every row) for one that gets no gradient.  `touched`, where wanted, has
// a bit for every row that gets one; it is clear when a kernel that sets bits begins.
// ---------------------------------------------------------------------------
struct TokenArgs {
    const void* tokens;
    int64_t n, rows, pad;
    int token_bytes;
    uint32_t* touched;       // or null
    int32_t* status;
};

__device__ __forceinline__ uint32_t token_key(const TokenArgs& a, int64_t i, int64_t t)
{
    if (t < 0 || t >= a.rows) {
        raise_error(a.status, TT_ERR_INDEX_RANGE, (int)min64(i, INT32_MAX));
        return (uint32_t)a.rows;
    }
    if (t == a.pad) return (uint32_t)a.rows;
    if (a.touched) atomicOr(a.touched + (t >> 5), 1u << (t & 31));
    return (uint32_t)t;
}

__global__ void __launch_bounds__(kThreads) k_token_keys(TokenArgs a, uint32_t* __restrict__ keys, int32_t* __restrict__ vals)
{
    if (has_error(a.status)) return;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.n) return;
    keys[i] = token_key(a, i, token_at(a.tokens, a.token_bytes, i));
    vals[i] = (int32_t)i;
}

// Up to kClusterTokens tokens in one launch: a cluster of blocks holds all keys in registers, kItems a
// thread, and sorts them by digits from the lowest up.  A digit's pass ranks the keys within
// their warp by matching lanes, adds the counts of the warps before (shared memory) and of the blocks
// before (the cluster's shared memory), and moves each key to its new place in whichever block
// that is.  One launch instead of ten: 4 to 10 us instead of 30.
// It goes on after an error: a cluster's blocks must all reach its barriers, and it writes
// nothing but workspace.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kCluster = 8;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int64_t kClusterTokens = (int64_t)kCluster * kSortThreads * 8;

template <int kItems> struct SortShared {
    uint2 come[kSortThreads * kItems];      // (key, position) from all blocks: this block's share of a pass's result
    uint2 mine[kSortThreads * kItems];      // this block's keys in the order of their digits
    uint16_t before[kSortWarps][kDigits];   // keys of a digit in the warps before, of this block
    uint32_t count[kDigits];                // keys of a digit in this block
    uint32_t here[kDigits];                 // place in `mine` of its first key of a digit
    uint32_t there[kDigits];                // place among all keys of that one
    uint32_t scan[2][kSortWarps];
};

template <int kItems>
__global__ void __launch_bounds__(kSortThreads, 1) k_token_sort(TokenArgs a, int bits, uint32_t* __restrict__ keys_out,
                                                                int32_t* __restrict__ vals_out, int64_t touched_words)
{
    extern __shared__ __align__(16) char s_raw[];
    SortShared<kItems>& s = *reinterpret_cast<SortShared<kItems>*>(s_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    constexpr int kChunk = kSortThreads * kItems;
    const unsigned lt = (1u << lane) - 1u;

    if (a.touched) {
        for (int64_t i = (int64_t)me * kSortThreads + tid; i < touched_words; i += (int64_t)blocks * kSortThreads) a.touched[i] = 0;
        cluster.sync();
    }
    const int first = wid * 32 * kItems + lane;             // the thread's keys: first, first + 32, ..
    const int cnt = (int)max((int64_t)0, min64(kChunk, a.n - (int64_t)me * kChunk));
    uint2 key[kItems];
    {
        int64_t t[kItems];
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int e = first + j * 32;
            t[j] = token_at(a.tokens, a.token_bytes, e < cnt ? (int64_t)me * kChunk + e : 0);
        }
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int e = first + j * 32;
            const int64_t i = (int64_t)me * kChunk + e;
            key[j] = make_uint2(e < cnt ? token_key(a, i, t[j]) : 0u, (uint32_t)i);
        }
    }
    const int passes = (bits + kDigitBits - 1) / kDigitBits, width = (bits + passes - 1) / passes, digits = 1 << width;
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * width;
        for (int i = tid; i < kSortWarps * kDigits / 2; i += kSortThreads) reinterpret_cast<uint32_t*>(s.before)[i] = 0;
        __syncthreads();
        // lanes with the same digit: a vote for each of its bits (those above the width are zero)
        uint32_t rank[kItems];
        unsigned same[kItems];
#pragma unroll
        for (int j = 0; j < kItems; ++j) same[j] = __ballot_sync(kFull, first + j * 32 < cnt);
#pragma unroll
        for (int b = 0; b < kDigitBits; ++b)
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
                const bool one = b < width && (key[j].x >> (shift + b) & 1u);
                const unsigned ones = __ballot_sync(kFull, one);
                same[j] &= one ? ones : ~ones;
            }
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int d = (int)((key[j].x >> shift) & (digits - 1));
            const uint32_t seen = s.before[wid][d];
            rank[j] = seen + __popc(same[j] & lt);
            __syncwarp();
            if (first + j * 32 < cnt && (same[j] & lt) == 0) s.before[wid][d] = (uint16_t)(seen + __popc(same[j]));
            __syncwarp();
        }
        __syncthreads();
        // counts of the warps before, and of the block: two threads for a digit, half of the warps each
        {
            constexpr int kHalf = kSortWarps / 2;
            const int d = tid >> 1, half = tid & 1;
            uint32_t c[kHalf], run = 0;
            if (d < digits)
#pragma unroll
                for (int w = 0; w < kHalf; ++w) c[w] = s.before[half * kHalf + w][d];
            else
#pragma unroll
                for (int w = 0; w < kHalf; ++w) c[w] = 0;
#pragma unroll
            for (int w = 0; w < kHalf; ++w) run += c[w];
            const uint32_t other = __shfl_xor_sync(kFull, run, 1);
            if (d < digits) {
                uint32_t sum = half ? other : 0u;
#pragma unroll
                for (int w = 0; w < kHalf; ++w) {
                    s.before[half * kHalf + w][d] = (uint16_t)sum;
                    sum += c[w];
                }
                if (half) s.count[d] = sum;
            }
        }
        cluster.sync();
        // places of a digit's first key in this block and among all: scans over the digits
        {
            uint32_t own = 0, earlier = 0, all = 0;
            if (tid < digits) {
                uint32_t x[kCluster];
#pragma unroll
                for (int c = 0; c < kCluster; ++c) x[c] = c < blocks ? *cluster.map_shared_rank(&s.count[tid], c) : 0u;
#pragma unroll
                for (int c = 0; c < kCluster; ++c) {
                    if (c == me) own = x[c];
                    earlier += c < me ? x[c] : 0u;
                    all += x[c];
                }
            }
            uint32_t x = own, y = all;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(kFull, x, o), v = __shfl_up_sync(kFull, y, o);
                if (lane >= o) {
                    x += u;
                    y += v;
                }
            }
            if (lane == 31) {
                s.scan[0][wid] = x;
                s.scan[1][wid] = y;
            }
            __syncthreads();
            const uint32_t sx = __reduce_add_sync(kFull, lane < wid ? s.scan[0][lane] : 0u);
            const uint32_t sy = __reduce_add_sync(kFull, lane < wid ? s.scan[1][lane] : 0u);
            if (tid < digits) {
                s.here[tid] = sx + x - own;
                s.there[tid] = sy + y - all + earlier;
            }
        }
        __syncthreads();
        // into the order of their digits here first, so that neighbours then go to neighbouring places
#pragma unroll
        for (int j = 0; j < kItems; ++j)
            if (first + j * 32 < cnt) {
                const int d = (int)((key[j].x >> shift) & (digits - 1));
                s.mine[s.here[d] + s.before[wid][d] + rank[j]] = key[j];
            }
        __syncthreads();
        const bool last = pass + 1 == passes;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int e = j * kSortThreads + tid;
            if (e < cnt) {
                const uint2 k = s.mine[e];
                const int d = (int)((k.x >> shift) & (digits - 1));
                const uint32_t to = s.there[d] + (e - s.here[d]);
                if (last) {
                    keys_out[to] = k.x;
                    vals_out[to] = (int32_t)k.y;
                } else {
                    cluster.map_shared_rank(s.come, to / kChunk)[to % kChunk] = k;
                }
            }
        }
        cluster.sync();   // also keeps every block's counts in place until they are read
        if (!last) {
#pragma unroll
            for (int j = 0; j < kItems; ++j)
                if (first + j * 32 < cnt) key[j] = s.come[first + j * 32];
        }
    }
}

// ---------------------------------------------------------------------------
// Sums.  A unit is one tile of sorted positions and 32 * V columns, and belongs to one warp.
// ---------------------------------------------------------------------------
struct SumArgs {
    const uint32_t* keys;     // sorted
    const int32_t* vals;      // input position of each
    int64_t n;
    int64_t rows;
    int dim;
    float scale;
    int accumulate;
    int tile;                 // positions per tile, a multiple of 32
    int64_t tiles;
    int slabs;                // units of a tile
    float* head;              // [tiles][dim] part of a run that began in an earlier tile
    float* tail;              // [tiles][dim] part of a run that begins here and goes on
    const uint32_t* touched;  // a bit for every row that a token names (without accumulate)
    const int32_t* status;
};

template <typename W, int V>
__device__ __forceinline__ void finish_row(W* at, const float (&x)[V], const Pack<W, V>& old, float scale)
{
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = fmaf(x[j], scale, to_f32(old.v[j]));
    store_pack(at, y);
}

#ifndef UU
#define UU 4
#endif
#ifndef UA
#define UA 2
#endif
template <typename G, typename W, int V, bool kAdd>
__global__ void __launch_bounds__(kThreads) k_token_sum(SumArgs a, const G* __restrict__ up, int64_t stride, W* __restrict__ grad)
{
    constexpr int kRows = kAdd ? UA : UU;                             // rows on their way at a time
    if (has_error(a.status)) return;
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t tile = unit / a.slabs;
    if (tile >= a.tiles) return;
    const int c = ((int)(unit - tile * a.slabs) * 32 + lane) * V;
    const bool on = c < a.dim;
    const int at_c = on ? c : 0;      // lanes behind the last column load the first ones
    const uint32_t none = (uint32_t)a.rows;
    const int64_t p0 = tile * a.tile, p1 = min64(p0 + a.tile, a.n);
    bool began = p0 > 0 && a.keys[p0 - 1] == a.keys[p0];  // the current run began in an earlier tile
    F2 acc[(V + 1) / 2];
#pragma unroll
    for (int j = 0; j < (V + 1) / 2; ++j) acc[j] = both(0.f);
    for (int64_t p = p0; p < p1; p += 32) {
        // a lane holds one position, and whether its run ends there or at the tile's end
        const bool in = p + lane < p1;
        const uint32_t key = in ? a.keys[p + lane] : none;
        const int32_t val = in ? a.vals[p + lane] : 0;
        const uint32_t next = p + lane + 1 < a.n ? a.keys[p + lane + 1] : none;
        const bool last = next != key;
        const int cnt = __popc(__ballot_sync(kFull, key < none));   // the others, behind, get no gradient
        const unsigned ends = __ballot_sync(kFull, last || p + lane + 1 == p1);
        const unsigned whole = __ballot_sync(kFull, last);
#pragma unroll 1
        for (int q = 0; q < cnt; q += kRows) {
            // No load hangs on a condition, so that none waits for another.  Places without a sum read a
            // row they do not use (position 0's, row 0); with kAdd each place loads its row of the
            // gradient as it is, which equal neighbours find in the cache.
            Pack<G, V> x[kRows];
            Pack<W, V> old[kAdd ? kRows : 1];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int64_t row = __shfl_sync(kFull, val, q + u);
                x[u] = *reinterpret_cast<const Pack<G, V>*>(up + row * stride + at_c);
                if constexpr (kAdd) {
                    const uint32_t k = __shfl_sync(kFull, key, q + u);
                    old[u] = *reinterpret_cast<const Pack<W, V>*>(grad + (int64_t)(k < none ? k : 0u) * a.dim + at_c);
                }
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                if (q + u >= cnt) break;
                if constexpr (V > 1) {
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) acc[j] = add2(acc[j], {to_f32(x[u].v[2 * j]), to_f32(x[u].v[2 * j + 1])});
                } else {
                    acc[0].x += to_f32(x[u].v[0]);
                }
                if (!(ends >> (q + u) & 1u)) continue;
                float sum[V];
#pragma unroll
                for (int j = 0; j < V; ++j) sum[j] = j & 1 ? acc[j / 2].y : acc[j / 2].x;
                const bool here = whole >> (q + u) & 1u;
                const uint32_t k = __shfl_sync(kFull, key, q + u);
                if (on) {
                    if (began) {
                        store_pack(a.head + tile * a.dim + c, sum);
                    } else if (!here) {
                        store_pack(a.tail + tile * a.dim + c, sum);
                    } else {
                        if constexpr (!kAdd) memset(&old[0], 0, sizeof(old[0]));
                        finish_row(grad + (int64_t)k * a.dim + c, sum, old[kAdd ? u : 0], a.scale);
                    }
                }
                began = false;
#pragma unroll
                for (int j = 0; j < (V + 1) / 2; ++j) acc[j] = both(0.f);
            }
        }
        if (cnt < 32) break;
    }
}

// The first `joins` blocks: where a run begins in a tile and goes on, they add up its parts, a warp
// for each of its slabs, in the order of the tiles.  The other blocks clear the rows that no token
// names.
constexpr int kClear = 16;        // vectors of 16 bytes a thread clears

// What one block clears: vectors of 16 bytes of the buffer, whatever rows they lie in.  The values in
// front of the buffer's first 16-byte place and behind its last are left to block 0.
template <typename W> struct Clear {
    static constexpr int N = 16 / sizeof(W);
    int64_t values, vectors, at, row0;
    int skip;
    unsigned col0;
    __device__ __forceinline__ Clear(const SumArgs& a, int64_t block, const W* grad)
    {
        values = a.rows * a.dim;
        skip = (int)((16 - ((uintptr_t)grad & 15)) & 15) / (int)sizeof(W);
        vectors = values > skip ? (values - skip) / N : 0;
        at = block * (kThreads * kClear);
        row0 = (at * N + skip) / a.dim;
        col0 = (unsigned)(at * N + skip - row0 * a.dim);
    }
    // hit: whether a token names a row of this block's vectors; far: any row
    template <typename Hit, typename Far>
    __device__ __forceinline__ void run(const SumArgs& a, W* grad, Hit hit, Far far) const
    {
        if (at == 0) {
            const int64_t e = threadIdx.x < skip ? threadIdx.x : skip + vectors * N + threadIdx.x - skip;
            if (e < values && !far(e / a.dim)) grad[e] = W(0.f);
        }
        const unsigned dim = a.dim;
        Pack<W, N> zero;
        memset(&zero, 0, sizeof(zero));
#pragma unroll 1
        for (int i0 = 0; i0 < kClear; i0 += 4) {
            unsigned col[4];
            int64_t row[4];
            bool named[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {     // all four are looked up first
                const unsigned off = col0 + ((i0 + i) * kThreads + threadIdx.x) * N, more = off / dim;
                col[i] = off - more * dim;
                row[i] = row0 + more;
                named[i] = hit(min64(row[i], a.rows - 1));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t v = at + (i0 + i) * kThreads + threadIdx.x;
                if (v >= vectors) return;
                W* const p = grad + skip + v * N;
                if (col[i] + N <= dim) {
                    if (!named[i]) *reinterpret_cast<Pack<W, N>*>(p) = zero;
                } else {
                    for (int j = 0; j < N; ++j)
                        if (!hit(row[i] + (col[i] + j) / dim)) p[j] = W(0.f);
                }
            }
        }
    }
};

template <typename W, int V>
__global__ void __launch_bounds__(kThreads) k_token_join(SumArgs a, int64_t joins, W* __restrict__ grad)
{
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int groups = (a.slabs + kWarps - 1) / kWarps;           // blocks of a tile
    const int64_t tile = blockIdx.x / groups, p0 = tile * a.tile, p1 = p0 + a.tile;
    const bool join = blockIdx.x < joins && p1 < a.n;
    const uint32_t k = join ? a.keys[p1 - 1] : 0u, then = join ? a.keys[p1] : 0u, front = join && p0 > 0 ? a.keys[p0 - 1] : ~0u;
    if (has_error(a.status)) return;
    if (blockIdx.x >= joins) {
        auto hit = [&](int64_t row) { return a.touched[row >> 5] >> (row & 31) & 1u; };
        Clear<W>(a, blockIdx.x - joins, grad).run(a, grad, hit, hit);
        return;
    }
    // nothing goes on, or it began earlier
    if (!join || k >= (uint32_t)a.rows || then != k || front == k) return;
    const int c = ((int)((blockIdx.x - tile * groups) * kWarps + wid) * 32 + lane) * V;
    if (c - lane * V >= a.dim) return;
    const bool on = c < a.dim;
    const int at_c = on ? c : 0;
    // the run's end: each step the lanes split what is left, (lo, hi), into 33
    int64_t lo = p1, hi = a.n;                                    // keys[lo] = k; keys[hi] is above k or past the end
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 32) / 33, at = lo + step * (lane + 1);
        const unsigned below = __ballot_sync(kFull, at < hi && a.keys[at] == k);
        const int m = __popc(below);
        hi = min64(hi, lo + step * (m + 1));
        lo = lo + step * m;
    }
    const int64_t last = lo / a.tile;                             // heads of tiles tile + 1 .. last
    W* const at = grad + (int64_t)k * a.dim + at_c;
    Pack<W, V> old;
    if (a.accumulate) old = *reinterpret_cast<const Pack<W, V>*>(at);
    else memset(&old, 0, sizeof(old));
    float acc[V];
    load_pack(a.tail + tile * a.dim + at_c, acc);
    constexpr int kParts = 8;                                     // parts on their way at a time
    for (int64_t t = tile + 1; t <= last; t += kParts) {
        Pack<float, V> x[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            x[i] = *reinterpret_cast<const Pack<float, V>*>(a.head + min64(t + i, last) * a.dim + at_c);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            if (t + i > last) break;
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] += x[i].v[j];
        }
    }
    if (on) finish_row(at, acc, old, a.scale);
}

// ---------------------------------------------------------------------------
// Few tokens: one launch.  A block of the first `slabs` sorts the tokens by itself (each key's place is
// the number of keys in front of it, counted) and adds up one slab, each warp a part of the sorted
// positions, whose ends are joined in shared memory.  The others clear rows; each looks
// up the few tokens in the rows that it covers.
// ---------------------------------------------------------------------------
constexpr int kFew = 512;
constexpr int kFewRows = kThreads * kClear * 8;   // rows that a block's vectors lie in at most

template <typename G, typename W, int V, bool kAdd>
__global__ void __launch_bounds__(kThreads) k_token_few(TokenArgs t, SumArgs a, const G* __restrict__ up, int64_t stride, W* __restrict__ grad)
{
    constexpr int kRows = 4;
    __shared__ alignas(16) uint32_t s_key[kFew + 4];
    __shared__ uint32_t s_bits[kFewRows / 32 + 1];
    __shared__ uint32_t s_sorted[kFew + 1];
    __shared__ int32_t s_place[kFew];
    __shared__ float s_part[kWarps][32 * V];
    const int n = (int)t.n, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const uint32_t none = (uint32_t)a.rows;
    constexpr int kMine = kFew / kThreads;
    int64_t token[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) token[j] = token_at(t.tokens, t.token_bytes, min(tid + j * kThreads, n - 1));
    bool bad = has_error(t.status);
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int i = tid + j * kThreads;
        if (i < n && (token[j] < 0 || token[j] >= a.rows)) {
            raise_error(t.status, TT_ERR_INDEX_RANGE, i);
            bad = true;
        }
        s_key[i] = i < n && token[j] != t.pad ? (uint32_t)token[j] : none;
    }
    if (tid < 4) s_key[kFew + tid] = none;
    if (__syncthreads_or(bad)) return;
    if ((int)blockIdx.x >= a.slabs) {
        // the rows of this block's vectors that a token names, as bits
        const Clear<W> clear(a, blockIdx.x - a.slabs, grad);
        for (int i = tid; i < kFewRows / 32 + 1; i += kThreads) s_bits[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            const int64_t r = (int64_t)s_key[i] - clear.row0;
            if (s_key[i] < none && r >= 0 && r < kFewRows + 32) atomicOr(&s_bits[r >> 5], 1u << (r & 31));
        }
        __syncthreads();
        auto hit = [&](int64_t row) { return s_bits[(row - clear.row0) >> 5] >> ((row - clear.row0) & 31) & 1u; };
        auto far = [&](int64_t row) {
            bool found = false;
            for (int i = 0; i < n; ++i) found |= s_key[i] == (uint32_t)row;
            return found;
        };
        clear.run(a, grad, hit, far);
        return;
    }
    // places: keys below mine, and equal ones in front
    {
        uint32_t mine[kMine];
        int place[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            mine[j] = s_key[tid + j * kThreads];
            place[j] = 0;
        }
        for (int i = 0; i < n; i += 4) {
            const uint4 q = *reinterpret_cast<const uint4*>(s_key + i);
            const uint32_t k[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < kMine; ++j)
                    place[j] += i + e < n && (k[e] < mine[j] || (k[e] == mine[j] && i + e < tid + j * kThreads));
        }
#pragma unroll
        for (int j = 0; j < kMine; ++j)
            if (tid + j * kThreads < n) {
                s_sorted[place[j]] = mine[j];
                s_place[place[j]] = tid + j * kThreads;
            }
        if (tid == 0) s_sorted[n] = none;
    }
    __syncthreads();
    const int c = ((int)blockIdx.x * 32 + lane) * V;
    const bool on = c < a.dim;
    const int at_c = on ? c : 0;
    const int each = (n + kWarps - 1) / kWarps, p0 = min(n, wid * each), p1 = min(n, p0 + each);
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    auto row_of = [&](uint32_t k) { return grad + (int64_t)k * a.dim + at_c; };
    // a run that goes over this part's end is left in acc, and what ends one that began before in s_part
    bool began = p0 > 0 && p0 < n && s_sorted[p0 - 1] == s_sorted[p0];
    uint32_t k = none;
    for (int p = p0; p < p1; p += kRows) {
        Pack<G, V> x[kRows];
        Pack<W, V> old[kAdd ? kRows : 1];
        memset(&old[0], 0, sizeof(old[0]));
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int q = min(p + u, p1 - 1);
            x[u] = *reinterpret_cast<const Pack<G, V>*>(up + (int64_t)s_place[q] * stride + at_c);
            if constexpr (kAdd) old[u] = *reinterpret_cast<const Pack<W, V>*>(row_of(s_sorted[q] < none ? s_sorted[q] : 0u));
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (p + u >= p1) break;
            k = s_sorted[p + u];
            if (k >= none) break;
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] += to_f32(x[u].v[j]);
            if (s_sorted[p + u + 1] == k) continue;
            if (began) {
#pragma unroll
                for (int j = 0; j < V; ++j) s_part[wid][j * 32 + lane] = acc[j];
                began = false;
            } else if (on) {
                finish_row(row_of(k), acc, old[kAdd ? u : 0], a.scale);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = 0.f;
        }
    }
    // what is left in acc goes on behind this part, or is all of a part that a run covers
    const bool goes_on = p1 > p0 && p1 < n && k < none && s_sorted[p1] == k;
    if (goes_on && began)
#pragma unroll
        for (int j = 0; j < V; ++j) s_part[wid][j * 32 + lane] = acc[j];
    __syncthreads();
    if (!goes_on || began) return;
    for (int w = wid + 1; w < kWarps && w * each < n && s_sorted[w * each] == k; ++w)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += s_part[w][j * 32 + lane];
    Pack<W, V> old;
    memset(&old, 0, sizeof(old));
    if constexpr (kAdd) old = *reinterpret_cast<const Pack<W, V>*>(row_of(k));
    if (on) finish_row(row_of(k), acc, old, a.scale);
}

// Positions a tile has: longer tiles cut fewer runs, shorter ones give every warp of the card a unit.
int tile_of(int64_t n, int slabs, int sms)
{
    const int64_t units = ceil_div(n, 32) * slabs, want = (int64_t)sms * WT;
    return 32 * (int)(units <= want ? 1 : units / want >= 8 ? 8 : units / want);
}

struct DenseLayout {
    size_t keys[2], vals[2], hist, digit_total, touched, head, tail, total;
};

DenseLayout dense_layout(int64_t n, int dim, int64_t rows)
{
    DenseLayout y;
    size_t p = 0;
    auto take = [&](size_t bytes) {
        const size_t at = p;
        p = (p + bytes + 255) / 256 * 256;
        return at;
    };
    const size_t nz = (size_t)(n > 0 ? n : 1);
    const size_t tiles = (size_t)ceil_div((int64_t)nz, 32);
    for (int i = 0; i < 2; ++i) {
        y.keys[i] = take(nz * 4);
        y.vals[i] = take(nz * 4);
    }
    y.hist = take(256 * (size_t)ceil_div((int64_t)nz, kSortTile) * 4);
    y.digit_total = take(256 * 4);
    y.touched = take((size_t)ceil_div(rows, 32) * 4);
    y.head = take(tiles * (size_t)dim * 4);
    y.tail = take(tiles * (size_t)dim * 4);
    y.total = p;
    return y;
}

// whether rows of `stride` values at p can be moved eight values at a time
bool wide_rows(const void* p, int64_t stride, int type)
{
    return ((uintptr_t)p & 15) == 0 && (stride * type_bytes(type)) % 16 == 0;
}

}  // namespace

struct tt_emb_dense_handle {
    int64_t rows = 0, pad = -1;
    int dim = 0, table_type = TT_F32, grad_type = TT_F32;
    float scale = 1.f;
    const void* table = nullptr;
    void* grad = nullptr;
    char* ws = nullptr;
    int64_t ws_n = -1;
    int32_t* d_status = nullptr;
    int device = 0, num_sms = 148;
    cudaStream_t last_stream = nullptr;
    bool used_stream = false;
    int last_error = TT_OK;
};

namespace {

int note(tt_emb_dense_t h, int rc)
{
    if (h && rc != TT_OK) h->last_error = rc;
    return rc;
}

int ready(tt_emb_dense_t h)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return TT_ERR_CUDA;
    return dev == h->device ? TT_OK : TT_ERR_STATE;
}

bool tokens_ok(const void* tokens, int32_t token_bytes, int64_t n)
{
    if (n < 0 || n >= INT32_MAX || (token_bytes != 4 && token_bytes != 8)) return false;
    return n == 0 || (tokens && ((uintptr_t)tokens & (token_bytes - 1)) == 0);
}

bool rows_ok(const void* p, int32_t type, int64_t stride, int64_t least, int64_t n)
{
    if (!type_known(type) || stride < least) return false;
    return n == 0 || (p && ((uintptr_t)p & (type_bytes(type) - 1)) == 0);
}

int forward(tt_emb_dense_t h, const void* tokens, int32_t token_bytes, int64_t n, void* out, int32_t out_type,
            int64_t out_stride, cudaStream_t s)
{
    if (!h || !tokens_ok(tokens, token_bytes, n) || !rows_ok(out, out_type, out_stride, h->dim, n)) return TT_ERR_ARG;
    if (!h->table) return TT_ERR_STATE;
    if (const int rc = ready(h)) return rc;
    h->last_stream = s;
    h->used_stream = true;
    if (n == 0) return TT_OK;
    const bool wide = h->dim % 8 == 0 && wide_rows(h->table, h->dim, h->table_type) && wide_rows(out, out_stride, out_type);
    // 16 bytes a lane of the narrower type; where rows begin anywhere, single values, two to a lane
    const int V = !wide ? 1 : h->table_type == TT_F32 && out_type == TT_F32 ? 4 : 8;
    const int64_t vectors = ceil_div(h->dim, V);
    LookupArgs a;
    a.tokens = tokens;
    a.n = n;
    a.rows = h->rows;
    a.out_stride = out_stride;
    a.token_bytes = token_bytes;
    a.dim = h->dim;
    a.scale = h->scale;
    a.status = h->d_status;
    for (a.lanes = 1; a.lanes < vectors && a.lanes < 32;) a.lanes *= 2;
    const int cols = wide ? V == 4 ? CW4 : CW8 : CA, rows = 32 / a.lanes;
    a.slabs = (int)ceil_div(vectors, 32 * cols);
    // as many steps to a unit as leave every warp of the card a unit or more
    const bool many = ceil_div(n, rows * 4) * a.slabs >= (int64_t)h->num_sms * 16;
    const int steps = many ? wide ? SW : SA : 1;
    const unsigned grid = (unsigned)ceil_div(ceil_div(n, rows * steps < 32 ? rows * steps : 32) * a.slabs, kWarps);
    by_type(h->table_type, [&](auto t) {
        by_type(out_type, [&](auto o) {
            using T = decltype(t);
            using O = decltype(o);
            auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, s>>>(a, (const T*)h->table, (O*)out); };
            constexpr bool f32 = sizeof(T) == 4 && sizeof(O) == 4;
            constexpr int kWide = f32 ? 4 : 8, kCols = f32 ? CW4 : CW8;
            if (wide) go(many ? k_lookup<T, O, kWide, kCols, SW> : k_lookup<T, O, kWide, kCols, 1>);
            else go(many ? k_lookup<T, O, 1, CA, SA> : k_lookup<T, O, 1, CA, 1>);
        });
    });
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

// Sorted keys and positions in buffer *which of the workspace.
cudaError_t sort_tokens(tt_emb_dense_t h, const TokenArgs& a, const DenseLayout& y, int bits, int* which, cudaStream_t s)
{
    uint32_t* const keys = (uint32_t*)(h->ws + y.keys[0]);
    int32_t* const vals = (int32_t*)(h->ws + y.vals[0]);
    const int64_t words = ceil_div(h->rows, 32);
    if (a.n <= kClusterTokens) {
        auto go = [&](auto kernel, size_t smem) {
            cudaLaunchConfig_t c = {};
            cudaLaunchAttribute at[1];
            // one block where a thread's one key is enough; the cluster's barriers are dearer than the block's
            const unsigned blocks = a.n <= kSortThreads ? 1 : kCluster;
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = blocks;
            at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
            c.gridDim = dim3(blocks);
            c.blockDim = dim3(kSortThreads);
            c.dynamicSmemBytes = smem;
            c.stream = s;
            c.attrs = at;
            c.numAttrs = 1;
            return cudaLaunchKernelEx(&c, kernel, a, bits, keys, vals, words);
        };
        *which = 0;
        const int64_t each = ceil_div(a.n, kCluster * kSortThreads);
        if (each <= 1) return go(k_token_sort<1>, sizeof(SortShared<1>));
        if (each <= 2) return go(k_token_sort<2>, sizeof(SortShared<2>));
        if (each <= 4) return go(k_token_sort<4>, sizeof(SortShared<4>));
        return go(k_token_sort<8>, sizeof(SortShared<8>));
    }
    if (a.touched) {
        const cudaError_t e = cudaMemsetAsync(a.touched, 0, (size_t)words * 4, s);
        if (e != cudaSuccess) return e;
    }
    k_token_keys<<<(unsigned)ceil_div(a.n, kThreads), kThreads, 0, s>>>(a, keys, vals);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    SortBuffers sb;
    for (int i = 0; i < 2; ++i) {
        sb.keys[i] = h->ws + y.keys[i];
        sb.vals[i] = (int32_t*)(h->ws + y.vals[i]);
    }
    sb.hist = (uint32_t*)(h->ws + y.hist);
    sb.digit_total = (uint32_t*)(h->ws + y.digit_total);
    int nl = 0;
    return radix_sort_pairs(false, a.n, bits, sb, which, h->d_status, s, &nl);
}

int backward(tt_emb_dense_t h, const void* tokens, int32_t token_bytes, int64_t n, const void* up, int32_t up_type,
             int64_t up_stride, int32_t accumulate, cudaStream_t s)
{
    if (!h || !tokens_ok(tokens, token_bytes, n) || !rows_ok(up, up_type, up_stride, 0, n)) return TT_ERR_ARG;
    if (accumulate != 0 && accumulate != 1) return TT_ERR_ARG;
    if (!h->grad) return TT_ERR_STATE;
    if (!h->ws || n > h->ws_n) return TT_ERR_WORKSPACE;
    if (const int rc = ready(h)) return rc;
    h->last_stream = s;
    h->used_stream = true;
    if (n == 0) {
        if (!accumulate &&
            cudaMemsetAsync(h->grad, 0, (size_t)h->rows * h->dim * type_bytes(h->grad_type), s) != cudaSuccess)
            return TT_ERR_CUDA;
        return TT_OK;
    }
    const DenseLayout y = dense_layout(h->ws_n, h->dim, h->rows);
    TokenArgs ta;
    ta.tokens = tokens;
    ta.n = n;
    ta.rows = h->rows;
    ta.pad = h->pad;
    ta.token_bytes = token_bytes;
    ta.touched = accumulate ? nullptr : (uint32_t*)(h->ws + y.touched);
    ta.status = h->d_status;
    const bool wide = h->dim % 8 == 0 && wide_rows(h->grad, h->dim, h->grad_type) && wide_rows(up, up_stride, up_type);
    // 16 bytes a lane of the narrower type
    const int V = !wide ? 1 : h->grad_type == TT_F32 && up_type == TT_F32 ? 4 : 8;
    SumArgs a;
    a.n = n;
    a.rows = h->rows;
    a.dim = h->dim;
    a.scale = h->scale;
    a.accumulate = accumulate;
    a.slabs = (int)ceil_div(h->dim, 32 * V);
    a.tile = tile_of(n, a.slabs, h->num_sms);
    a.tiles = ceil_div(n, a.tile);
    a.head = (float*)(h->ws + y.head);
    a.tail = (float*)(h->ws + y.tail);
    a.touched = ta.touched;
    a.status = h->d_status;
    const int64_t joins = a.tiles > 1 ? a.tiles * ceil_div(a.slabs, kWarps) : 0;
    const int64_t clears = accumulate ? 0 : ceil_div(ceil_div(h->rows * h->dim, 16 / type_bytes(h->grad_type)), kThreads * kClear);
    const unsigned grid = (unsigned)ceil_div(a.tiles * a.slabs, kWarps);
    if (joins + clears > INT32_MAX) return TT_ERR_ARG;   // sizes that no device holds
    if (n <= kFew) {
        by_type(h->grad_type, [&](auto w) {
            by_type(up_type, [&](auto g) {
                using W = decltype(w);
                using G = decltype(g);
                auto go = [&](auto kernel) {
                    kernel<<<(unsigned)(a.slabs + clears), kThreads, 0, s>>>(ta, a, (const G*)up, up_stride, (W*)h->grad);
                };
                constexpr int kWide = sizeof(W) == 4 && sizeof(G) == 4 ? 4 : 8;
                if (wide) go(accumulate ? k_token_few<G, W, kWide, true> : k_token_few<G, W, kWide, false>);
                else go(accumulate ? k_token_few<G, W, 1, true> : k_token_few<G, W, 1, false>);
            });
        });
        return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
    }
    int bits = 1, which = 0;
    while (h->rows >> bits) ++bits;
    if (sort_tokens(h, ta, y, bits, &which, s) != cudaSuccess) return TT_ERR_CUDA;
    a.keys = (const uint32_t*)(h->ws + y.keys[which]);
    a.vals = (const int32_t*)(h->ws + y.vals[which]);
    by_type(h->grad_type, [&](auto w) {
        using W = decltype(w);
        by_type(up_type, [&](auto g) {
            using G = decltype(g);
            auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, s>>>(a, (const G*)up, up_stride, (W*)h->grad); };
            constexpr int kWide = sizeof(W) == 4 && sizeof(G) == 4 ? 4 : 8;
            if (wide) go(accumulate ? k_token_sum<G, W, kWide, true> : k_token_sum<G, W, kWide, false>);
            else go(accumulate ? k_token_sum<G, W, 1, true> : k_token_sum<G, W, 1, false>);
        });
        if (joins + clears == 0) return;
        auto go = [&](auto kernel) { kernel<<<(unsigned)(joins + clears), kThreads, 0, s>>>(a, joins, (W*)h->grad); };
        if (V == 1) go(k_token_join<W, 1>);
        else if (V == 8) go(k_token_join<W, 8>);
        else if constexpr (sizeof(W) == 4) go(k_token_join<W, 4>);
    });
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // namespace

extern "C" {

int tt_emb_dense_create(int64_t num_rows, int32_t dim, int32_t table_type, float scale, int64_t padding_row,
                        tt_emb_dense_t* out)
{
    if (!out) return TT_ERR_ARG;
    *out = nullptr;
    if (!type_known(table_type)) return TT_ERR_ARG;
    if (num_rows < 1 || num_rows >= INT32_MAX || dim < 1 || dim > 1 << 20) return TT_ERR_SHAPE;
    if (padding_row < -1 || padding_row >= num_rows) return TT_ERR_SHAPE;
    tt_emb_dense_handle* h = new (std::nothrow) tt_emb_dense_handle();
    if (!h) return TT_ERR_ARG;
    h->rows = num_rows;
    h->dim = dim;
    h->table_type = table_type;
    h->scale = scale;
    h->pad = padding_row;
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
        cudaMalloc((void**)&h->d_status, 256) != cudaSuccess) {
        delete h;
        return TT_ERR_CUDA;
    }
    auto room = [](auto kernel, size_t smem) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    };
    if (cudaMemset(h->d_status, 0, 256) != cudaSuccess ||
        room(k_token_sort<1>, sizeof(SortShared<1>)) != cudaSuccess || room(k_token_sort<2>, sizeof(SortShared<2>)) != cudaSuccess ||
        room(k_token_sort<4>, sizeof(SortShared<4>)) != cudaSuccess || room(k_token_sort<8>, sizeof(SortShared<8>)) != cudaSuccess) {
        cudaFree(h->d_status);
        delete h;
        return TT_ERR_CUDA;
    }
    *out = h;
    return TT_OK;
}

int tt_emb_dense_set_table(tt_emb_dense_t h, const void* table, void* grad, int32_t grad_type)
{
    if (!h || !table || !type_known(grad_type)) return note(h, TT_ERR_ARG);
    if (((uintptr_t)table & (type_bytes(h->table_type) - 1)) || ((uintptr_t)grad & (type_bytes(grad_type) - 1)))
        return note(h, TT_ERR_ARG);
    h->table = table;
    h->grad = grad;
    h->grad_type = grad_type;
    return TT_OK;
}

int tt_emb_dense_workspace_size(tt_emb_dense_t h, int64_t max_tokens, size_t* bytes)
{
    if (!h || !bytes || max_tokens < 0 || max_tokens >= INT32_MAX) return note(h, TT_ERR_ARG);
    *bytes = dense_layout(max_tokens, h->dim, h->rows).total;
    return TT_OK;
}

int tt_emb_dense_set_workspace(tt_emb_dense_t h, void* workspace, size_t bytes, int64_t max_tokens)
{
    if (!h || !workspace || ((uintptr_t)workspace & 255) || max_tokens < 0 || max_tokens >= INT32_MAX)
        return note(h, TT_ERR_ARG);
    if (bytes < dense_layout(max_tokens, h->dim, h->rows).total) return note(h, TT_ERR_WORKSPACE);
    h->ws = (char*)workspace;
    h->ws_n = max_tokens;
    return TT_OK;
}

int tt_emb_dense_forward(tt_emb_dense_t h, const void* tokens, int32_t token_bytes, int64_t num_tokens, void* out,
                         int32_t out_type, int64_t out_stride, tt_stream_t stream)
{
    return note(h, forward(h, tokens, token_bytes, num_tokens, out, out_type, out_stride, (cudaStream_t)stream));
}

int tt_emb_dense_backward(tt_emb_dense_t h, const void* tokens, int32_t token_bytes, int64_t num_tokens,
                          const void* grad_out, int32_t grad_out_type, int64_t grad_out_stride, int32_t accumulate,
                          tt_stream_t stream)
{
    return note(h, backward(h, tokens, token_bytes, num_tokens, grad_out, grad_out_type, grad_out_stride, accumulate,
                            (cudaStream_t)stream));
}

int tt_emb_dense_sync(tt_emb_dense_t h)
{
    if (!h) return TT_ERR_ARG;
    cudaStream_t s = h->used_stream ? h->last_stream : (cudaStream_t)0;
    int32_t st = 0;
    if (cudaMemcpyAsync(&st, h->d_status, sizeof(st), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return note(h, TT_ERR_CUDA);
    if (st != 0 && (cudaMemsetAsync(h->d_status, 0, 256, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess))
        return note(h, TT_ERR_CUDA);
    return note(h, st);
}

int tt_emb_dense_last_error(tt_emb_dense_t h)
{
    if (!h) return TT_ERR_ARG;
    const int rc = h->last_error;
    h->last_error = TT_OK;
    return rc;
}

const int32_t* tt_emb_dense_status_word(tt_emb_dense_t h) { return h ? h->d_status : nullptr; }

void tt_emb_dense_destroy(tt_emb_dense_t h)
{
    if (!h) return;
    if (h->d_status) cudaFree(h->d_status);
    delete h;
}

}  // extern "C"
