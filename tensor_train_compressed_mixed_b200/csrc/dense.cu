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
    int per_unit;        // tokens of a unit, 1 .. 32
    int lanes;           // lanes that share a row, a power of two
    int slabs;           // units of the same tokens, 32 vectors (times kCols) of a row each
    int32_t* status;
};

// A warp takes a unit: up to 32 tokens, one a lane, and a slab of their rows.  A step moves 32 / lanes
// rows; the loads of kSteps steps are on their way while the kSteps before them are stored.  No
// load hangs on a condition, so that none waits for another: places behind the last token read
// the last one's row, tokens outside the table row 0.
template <typename T, typename O, int V, int kCols, int kSteps>
__global__ void __launch_bounds__(kThreads) k_lookup(LookupArgs a, const T* __restrict__ table, O* __restrict__ out)
{
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), group = unit / a.slabs;
    const int64_t i0 = group * a.per_unit;
    if (i0 >= a.n) return;
    const int cnt = (int)min64(a.per_unit, a.n - i0);
    int64_t token = token_at(a.tokens, a.token_bytes, i0 + min(lane, cnt - 1));
    if (has_error(a.status)) return;
    const bool bad = token < 0 || token >= a.rows;
    if (bad && lane < cnt) raise_error(a.status, TT_ERR_INDEX_RANGE, (int)min64(i0 + lane, INT32_MAX));
    const unsigned good = __ballot_sync(kFull, !bad);
    if (bad) token = 0;
    const int sub = lane & (a.lanes - 1), own = lane / a.lanes, rows = 32 / a.lanes, steps = (cnt + rows - 1) / rows;
    const int c0 = ((int)(unit - group * a.slabs) * kCols * 32 + sub) * V;
    Pack<T, V> x[2][kSteps][kCols];
    auto load = [&](Pack<T, V> (&to)[kSteps][kCols], int s0) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t row = __shfl_sync(kFull, token, min((s0 + s) * rows + own, cnt - 1));
#pragma unroll
            for (int k = 0; k < kCols; ++k) {
                const int c = c0 + k * 32 * V;
                to[s][k] = *reinterpret_cast<const Pack<T, V>*>(table + row * a.dim + (c < a.dim ? c : 0));
            }
        }
    };
    auto store = [&](const Pack<T, V> (&from)[kSteps][kCols], int s0) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int i = (s0 + s) * rows + own;
            if (i >= cnt || !(good >> i & 1u)) continue;
#pragma unroll
            for (int k = 0; k < kCols; ++k) {
                const int c = c0 + k * 32 * V;
                float y[V];
#pragma unroll
                for (int j = 0; j < V; ++j) y[j] = to_f32(from[s][k].v[j]) * a.scale;
                if (c < a.dim) store_pack(out + (i0 + i) * a.out_stride + c, y);
            }
        }
    };
    load(x[0], 0);
    for (int s0 = 0; s0 < steps; s0 += 2 * kSteps) {
        load(x[1], s0 + kSteps);
        store(x[0], s0);
        if (s0 + kSteps >= steps) break;
        load(x[0], s0 + 2 * kSteps);
        store(x[1], s0 + kSteps);
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
    uint32_t key[kSortThreads * kItems];
    int32_t val[kSortThreads * kItems];
    uint16_t before[kSortWarps][kDigits];   // keys of a digit in the warps before, of this block
    uint32_t count[kDigits];                // keys of a digit in this block
    uint32_t first[kDigits];                // place of this block's first key of a digit
    uint32_t scan[kSortWarps];
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
    uint32_t key[kItems];
    int32_t val[kItems];
    bool in[kItems];
    {
        int64_t t[kItems];
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            val[j] = me * kChunk + wid * 32 * kItems + j * 32 + lane;
            in[j] = val[j] < a.n;
            t[j] = token_at(a.tokens, a.token_bytes, in[j] ? val[j] : 0);
        }
#pragma unroll
        for (int j = 0; j < kItems; ++j) key[j] = in[j] ? token_key(a, val[j], t[j]) : 0u;
    }
    const int passes = (bits + kDigitBits - 1) / kDigitBits, width = (bits + passes - 1) / passes, digits = 1 << width;
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * width;
        for (int i = tid; i < kSortWarps * kDigits / 2; i += kSortThreads) reinterpret_cast<uint32_t*>(s.before)[i] = 0;
        __syncthreads();
        uint32_t rank[kItems];
        int digit[kItems];
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            digit[j] = (int)((key[j] >> shift) & (digits - 1));
            // lanes with the same digit, a vote for each of its bits (a match instruction takes three times as long)
            unsigned same = __ballot_sync(kFull, in[j]);
            for (int b = 0; b < width; ++b) {
                const bool one = digit[j] >> b & 1;
                const unsigned ones = __ballot_sync(kFull, one);
                same &= one ? ones : ~ones;
            }
            const uint32_t seen = in[j] ? s.before[wid][digit[j]] : 0u;
            rank[j] = seen + __popc(same & lt);
            __syncwarp();
            if (in[j] && (same & lt) == 0) s.before[wid][digit[j]] = (uint16_t)(seen + __popc(same));
            __syncwarp();
        }
        __syncthreads();
        // counts of the warps before, and of the block: two threads for a digit, half of the warps each
        {
            const int d = tid >> 1, half = tid & 1;
            uint32_t run = 0;
            if (d < digits)
                for (int w = half * (kSortWarps / 2); w < (half + 1) * (kSortWarps / 2); ++w) {
                    const uint32_t c = s.before[w][d];
                    s.before[w][d] = (uint16_t)run;
                    run += c;
                }
            const uint32_t other = __shfl_xor_sync(kFull, run, 1);
            if (d < digits && half)
                for (int w = kSortWarps / 2; w < kSortWarps; ++w) s.before[w][d] += (uint16_t)other;
            if (d < digits && !half) s.count[d] = run + other;
        }
        cluster.sync();
        // a digit's keys in the blocks before and in all; their places by a scan over the digits
        {
            uint32_t earlier = 0, all = 0;
            if (tid < digits) {
                uint32_t x[kCluster];
#pragma unroll
                for (int c = 0; c < kCluster; ++c) x[c] = c < blocks ? *cluster.map_shared_rank(&s.count[tid], c) : 0u;
#pragma unroll
                for (int c = 0; c < kCluster; ++c) {
                    earlier += c < me ? x[c] : 0u;
                    all += x[c];
                }
            }
            uint32_t x = all;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(kFull, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) s.scan[wid] = x;
            __syncthreads();
            uint32_t sum = 0;
            for (int w = 0; w < wid; ++w) sum += s.scan[w];
            if (tid < digits) s.first[tid] = sum + x - all + earlier;
        }
        __syncthreads();
        const bool last = pass + 1 == passes;
#pragma unroll
        for (int j = 0; j < kItems; ++j)
            if (in[j]) {
                const uint32_t to = s.first[digit[j]] + s.before[wid][digit[j]] + rank[j];
                if (last) {
                    keys_out[to] = key[j];
                    vals_out[to] = val[j];
                } else {
                    SortShared<kItems>* there = cluster.map_shared_rank(&s, to / kChunk);
                    there->key[to % kChunk] = key[j];
                    there->val[to % kChunk] = val[j];
                }
            }
        cluster.sync();   // also keeps every block's counts in place until they are read
        if (!last) {
#pragma unroll
            for (int j = 0; j < kItems; ++j)
                if (in[j]) {
                    key[j] = s.key[wid * 32 * kItems + j * 32 + lane];
                    val[j] = s.val[wid * 32 * kItems + j * 32 + lane];
                }
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

template <typename G, typename W, int V, bool kAdd>
__global__ void __launch_bounds__(kThreads) k_token_sum(SumArgs a, const G* __restrict__ up, int64_t stride, W* __restrict__ grad)
{
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
    uint32_t key = a.keys[p0];
    bool began = p0 > 0 && a.keys[p0 - 1] == key;         // the current run began in an earlier tile
    constexpr int U = 8;                                  // rows on their way at a time
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int64_t p = p0; p < p1; p += 32) {
        // a lane holds one position; past the tile's end the key that follows, past the last one none
        const uint32_t my_key = p + lane < a.n ? a.keys[p + lane] : none;
        const int32_t my_val = p + lane < p1 ? a.vals[p + lane] : 0;
        const uint32_t after = p + 32 < a.n ? a.keys[p + 32] : none;
        const int cnt = (int)min64(32, p1 - p);
        const uint32_t up1 = __shfl_down_sync(kFull, my_key, 1);
        const uint32_t my_next = lane == 31 ? after : up1;
        if (__shfl_sync(kFull, my_key, 0) >= none) break;  // what follows gets no gradient
#pragma unroll 1
        for (int q = 0; q < cnt; q += U) {
            // No load hangs on a condition, so that all are on their way together.  Places without a sum
            // read a row they do not use (position 0's, row 0); with kAdd each place loads its row of the
            // gradient as it is, which equal neighbours find in the cache.
            Pack<G, V> x[U];
            Pack<W, V> old[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = __shfl_sync(kFull, my_val, q + u);
                x[u] = *reinterpret_cast<const Pack<G, V>*>(up + row * stride + at_c);
                if (kAdd) {
                    const uint32_t k = __shfl_sync(kFull, my_key, q + u);
                    old[u] = *reinterpret_cast<const Pack<W, V>*>(grad + (int64_t)(k < none ? k : 0u) * a.dim + at_c);
                } else {
                    memset(&old[u], 0, sizeof(old[u]));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t k = __shfl_sync(kFull, my_key, q + u), next = __shfl_sync(kFull, my_next, q + u);
                if (q + u >= cnt || k >= none) break;
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] += to_f32(x[u].v[j]);
                const bool at_end = p + q + u + 1 == p1;
                if (!at_end && next == k) continue;
                if (on) {
                    if (began) store_pack(a.head + tile * a.dim + c, acc);
                    else if (next == k) store_pack(a.tail + tile * a.dim + c, acc);
                    else finish_row(grad + (int64_t)k * a.dim + c, acc, old[u], a.scale);
                }
                began = false;
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] = 0.f;
            }
        }
    }
}

// The first `joins` blocks, one for each unit: where a run begins in the unit's tile and goes on, they
// add up its parts, each warp a row of tiles, then the warps' sums in order.  The other blocks
// clear the rows that no token names.
constexpr int kClear = 16;        // vectors of 16 bytes a thread clears

template <typename W>
__device__ __forceinline__ void clear_rows(const SumArgs& a, int64_t block, W* grad)
{
    constexpr int N = 16 / sizeof(W);
    const int64_t values = a.rows * a.dim;
    // vectors of the buffer, whatever rows they lie in; those in front of its first 16-byte place
    // and behind its last are left to the first block
    const int skip = (int)((16 - ((uintptr_t)grad & 15)) & 15) / (int)sizeof(W);
    const int64_t vectors = values > skip ? (values - skip) / N : 0;
    const int64_t at = block * (kThreads * kClear), first = at * N + skip, row0 = first / a.dim;
    const unsigned col0 = (unsigned)(first - row0 * a.dim), dim = a.dim;
    auto touched = [&](int64_t row) { return a.touched[row >> 5] >> (row & 31) & 1u; };
    Pack<W, N> zero;
    memset(&zero, 0, sizeof(zero));
#pragma unroll 4
    for (int i = 0; i < kClear; ++i) {
        const int64_t v = at + i * kThreads + threadIdx.x;
        if (v >= vectors) break;
        const unsigned off = col0 + (i * kThreads + threadIdx.x) * N, more = off / dim, col = off - more * dim;
        const int64_t row = row0 + more;
        W* const p = grad + skip + v * N;
        if (col + N <= dim) {
            if (!touched(row)) *reinterpret_cast<Pack<W, N>*>(p) = zero;
        } else {
            for (int j = 0; j < N; ++j)
                if (!touched(row + (col + j) / dim)) p[j] = W(0.f);
        }
    }
    if (block == 0) {
        const int64_t behind = skip + vectors * N;
        const int64_t e = threadIdx.x < skip ? threadIdx.x : behind + threadIdx.x - skip;
        if (e < values && (threadIdx.x < skip || e >= behind) && !touched(e / a.dim)) grad[e] = W(0.f);
    }
}

template <typename W, int V>
__global__ void __launch_bounds__(kThreads) k_token_join(SumArgs a, int64_t joins, W* __restrict__ grad)
{
    __shared__ float s_part[kWarps][32 * V];
    if (has_error(a.status)) return;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    if (blockIdx.x >= joins) {
        clear_rows(a, blockIdx.x - joins, grad);
        return;
    }
    const int64_t tile = blockIdx.x / a.slabs;
    const int64_t p0 = tile * a.tile, p1 = p0 + a.tile;
    if (p1 >= a.n) return;
    const uint32_t k = a.keys[p1 - 1];
    if (k >= (uint32_t)a.rows || a.keys[p1] != k) return;         // nothing goes on
    if (p0 > 0 && a.keys[p0 - 1] == k) return;                    // it began earlier
    // the run's end: each step the lanes split what is left, (lo, hi], into 33
    int64_t lo = p1, hi = a.n;                                    // keys[lo] = k; keys[hi] is above k or past the end
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 32) / 33, at = lo + step * (lane + 1);
        const unsigned below = __ballot_sync(kFull, at < hi && a.keys[at] == k);
        const int m = __popc(below);
        hi = min64(hi, lo + step * (m + 1));
        lo = lo + step * m;
    }
    const int64_t last = lo / a.tile, parts = last - tile;        // heads of tiles tile + 1 .. last
    const int c = ((int)(blockIdx.x - tile * a.slabs) * 32 + lane) * V;
    const bool on = c < a.dim;
    const int64_t each = (parts + kWarps - 1) / kWarps, from = tile + 1 + wid * each, to = min64(from + each, last + 1);
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    if (on)
#pragma unroll 4
        for (int64_t t = from; t < to; ++t) {
            float x[V];
            load_pack(a.head + t * a.dim + c, x);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] += x[j];
        }
#pragma unroll
    for (int j = 0; j < V; ++j) s_part[wid][j * 32 + lane] = acc[j];
    __syncthreads();
    if (wid > 0 || !on) return;
    float sum[V];
    load_pack(a.tail + tile * a.dim + c, sum);
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += s_part[w][j * 32 + lane];
    W* const at = grad + (int64_t)k * a.dim + c;
    Pack<W, V> old;
    memset(&old, 0, sizeof(old));
    if (a.accumulate) old = *reinterpret_cast<const Pack<W, V>*>(at);
    finish_row(at, sum, old, a.scale);
}

// Positions a tile has: longer tiles cut fewer runs, shorter ones give every warp of the card a unit.
int tile_of(int64_t n, int slabs, int sms)
{
    const int64_t units = ceil_div(n, 32) * slabs, want = (int64_t)sms * 24;
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
    // 16 bytes a lane of the wider type; where rows begin anywhere, single values, four to a lane
    const int V = !wide ? 1 : h->table_type == TT_F32 || out_type == TT_F32 ? 4 : 8;
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
    a.slabs = (int)ceil_div(vectors, wide ? 32 : 32 * 4);
    // as many tokens to a unit as leave every warp of the card a few
    a.per_unit = 32;
    while (a.per_unit > 1 && ceil_div(n, a.per_unit) * a.slabs < (int64_t)h->num_sms * 64) a.per_unit /= 2;
    const unsigned grid = (unsigned)ceil_div(ceil_div(n, a.per_unit) * a.slabs, kWarps);
    by_type(h->table_type, [&](auto t) {
        by_type(out_type, [&](auto o) {
            using T = decltype(t);
            using O = decltype(o);
            auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, s>>>(a, (const T*)h->table, (O*)out); };
            constexpr int kWide = sizeof(T) == 4 || sizeof(O) == 4 ? 4 : 8;
            if (wide) go(k_lookup<T, O, kWide, 1, 4>);
            else go(k_lookup<T, O, 1, 4, 2>);
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
    // 16 bytes a lane of the wider type
    const int V = !wide ? 1 : h->grad_type == TT_F32 || up_type == TT_F32 ? 4 : 8;
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
    const int64_t joins = a.tiles > 1 ? a.tiles * a.slabs : 0;
    const int64_t clears = accumulate ? 0 : ceil_div(ceil_div(h->rows * h->dim, 16 / type_bytes(h->grad_type)), kThreads * kClear);
    const unsigned grid = (unsigned)ceil_div(a.tiles * a.slabs, kWarps);
    if (joins + clears > INT32_MAX) return TT_ERR_ARG;   // sizes that no device holds
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
            constexpr int kWide = sizeof(W) == 4 || sizeof(G) == 4 ? 4 : 8;
            if (wide) go(accumulate ? k_token_sum<G, W, kWide, true> : k_token_sum<G, W, kWide, false>);
            else go(accumulate ? k_token_sum<G, W, 1, true> : k_token_sum<G, W, 1, false>);
        });
        if (joins + clears == 0) return;
        auto go = [&](auto kernel) { kernel<<<(unsigned)(joins + clears), kThreads, 0, s>>>(a, joins, (W*)h->grad); };
        if (V == 1) go(k_token_join<W, 1>);
        else if (V == 4) go(k_token_join<W, 4>);
        else if constexpr (sizeof(W) == 2) go(k_token_join<W, 8>);
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
