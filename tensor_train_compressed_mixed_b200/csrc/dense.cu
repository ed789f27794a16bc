// Dense tables: scaled lookup of rows, and the table's gradient by sorted tokens.
//
// Both move rows and do one or two operations a value, so memory bounds them.
//
// Lookup.  A lane moves 16 bytes (of the narrower type) of four rows at a time, whose loads are all
// issued before the first store.
//
// Gradient.  The tokens are sorted by row (stable, so equal rows stay in input order) and the sorted
// positions are cut into tiles.  A warp adds up its columns of a tile's upstream rows in fp32
// registers, one run of equal rows after the other; a run that lies inside its tile is written to
// the gradient at once, and the parts of one that crosses tiles go to the workspace and are
// added in tile order by the next kernel.  Both kernels also clear rows that no token names.  So every
// row of the gradient is written once, a row that many tokens name is spread over many warps, and
// no sum depends on the order in which blocks run.
#include <cooperative_groups.h>
#include <new>
#include <type_traits>

#include "dense.cuh"

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
    int lane_bits;       // 2^lane_bits lanes share a row
    unsigned slabs;      // units of the same tokens; a slab is 32 * kCols vectors of a row
    int32_t* status;
};

// A warp takes a unit: up to 32 tokens, one a lane, and a slab of their rows.  A step moves 32 / lanes
// rows; the loads of kSteps steps are issued before the first store.  No load hangs on a
// condition, so that none waits for another: places behind the last token read the last one's row,
// tokens outside the table row 0.
template <typename T, typename O, int V, int kCols, int kSteps>
__global__ void __launch_bounds__(kThreads) k_lookup(LookupArgs a, const T* __restrict__ table, O* __restrict__ out)
{
    const int lane = threadIdx.x & 31;
    const unsigned unit = blockIdx.x * kWarps + (threadIdx.x >> 5), group = unit / a.slabs, slab = unit - group * a.slabs;
    const int64_t i0 = (int64_t)group * a.per_unit;
    if (i0 >= a.n) return;
    const int cnt = (int)min64(a.per_unit, a.n - i0);
    int64_t token = token_at(a.tokens, a.token_bytes, i0 + min(lane, cnt - 1));
    const bool stop = has_error(a.status);
    const bool bad = token < 0 || token >= a.rows;
    if (bad) token = 0;
    const int lanes = 1 << a.lane_bits, rows = 32 >> a.lane_bits, sub = lane & (lanes - 1), own = lane >> a.lane_bits;
    const int steps = (cnt + rows - 1) >> (5 - a.lane_bits);
    const int c0 = ((int)slab * kCols * 32 + sub) * V;
    const unsigned good = __ballot_sync(kFull, !bad);
    for (int s0 = 0; s0 < steps; s0 += kSteps) {
        Pack<T, V> x[kSteps][kCols];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t row = __shfl_sync(kFull, token, min(((s0 + s) << (5 - a.lane_bits)) + own, cnt - 1));
#pragma unroll
            for (int k = 0; k < kCols; ++k) {
                const int c = c0 + k * 32 * V;
                x[s][k] = *reinterpret_cast<const Pack<T, V>*>(table + row * a.dim + (c < a.dim ? c : 0));
            }
        }
        if (stop) return;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int i = ((s0 + s) << (5 - a.lane_bits)) + own;
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
    if (bad && lane < cnt) raise_error(a.status, TT_ERR_INDEX_RANGE, (int)min64(i0 + lane, INT32_MAX));
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
    return (uint32_t)(t == a.pad ? a.rows : t);
}

// The bit of a key's row.  A lane whose left neighbour has the same key leaves it to that one: the bits of
// a batch of one token would otherwise be set one after the other.  All lanes of a warp call it.
__device__ __forceinline__ void touch(const TokenArgs& a, uint32_t key, bool in)
{
    const uint32_t left = __shfl_up_sync(kFull, in ? key : 0xffffffffu, 1);
    if (a.touched && in && key < (uint32_t)a.rows && ((threadIdx.x & 31) == 0 || left != key)) atomicOr(a.touched + (key >> 5), 1u << (key & 31));
}

__global__ void __launch_bounds__(kThreads) k_token_keys(TokenArgs a, uint32_t* __restrict__ keys, int32_t* __restrict__ vals)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const bool in = i < a.n;
    const uint32_t key = in ? token_key(a, i, token_at(a.tokens, a.token_bytes, i)) : 0u;
    touch(a, key, in);
    if (!in) return;
    keys[i] = key;
    vals[i] = (int32_t)i;
}

// Up to kClusterTokens tokens in one launch: a cluster of blocks holds all keys in registers, kItems a
// thread, and sorts them by digits from the lowest up.  A digit's pass ranks the keys within
// their warp by matching lanes, adds the counts of the warps before (shared memory) and of the blocks
// before (the cluster's shared memory), and moves each key to its new place in whichever block
// that is.  One launch instead of ten: a gradient of 2000 tokens over 5000 x 512 fp32 takes 21 us with it and
// 40 with the radix sort's launches, one of 65536 tokens 60 and 81, one of 131072 tokens 104 and 118.
// It goes on after an error: a cluster's blocks must all reach its barriers, and it writes
// nothing but workspace.
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kCluster = 16;     // needs leave for more than eight blocks (see sort_fits)
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int64_t kClusterTokens = (int64_t)kCluster * kSortThreads * 16;
static_assert(kDigits == kSortThreads, "a thread for each digit");

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
    let_next_kernel_start();
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
            touch(a, key[j].x, e < cnt);
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
        // counts of the warps before, and of the block: a thread for each digit
        {
            uint32_t c[kSortWarps], sum = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) c[w] = s.before[w][tid];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                s.before[w][tid] = (uint16_t)sum;
                sum += c[w];
            }
            s.count[tid] = sum;
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
// Sums.  A unit is one tile of sorted positions and a slab of columns, a lane's (see Cols) for each lane of
// the warp that it belongs to.
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
    int64_t sums;             // blocks of the first kernel that add up; its others clear rows,
    int64_t first_clear;      // and the second kernel's go on from here
    int clear_each;           // clearing blocks' worth that a block of the kernel for few tokens takes
    float* head;              // [tiles][dim] part of a run that began in an earlier tile
    float* tail;              // [tiles][dim] part of a run that begins here and goes on
    const uint32_t* touched;  // a bit for every row that a token names (without accumulate)
    const int32_t* status;
};

// A lane's columns of a row: V neighbours, or, where rows begin at places for pairs (V = 2) or for single
// values only, four of those, each 32 of them behind the last.  Columns behind the row's last are
// read as its first and not written.
template <int V> constexpr int kColumns = V <= 2 ? 4 * V : V;
template <int V> constexpr int kRuns = kColumns<V> / V;
template <typename T, int V> struct Cols {
    Pack<T, V> p[kRuns<V>];
    __device__ __forceinline__ void load(const T* row, int c, int dim)
    {
#pragma unroll
        for (int k = 0; k < kRuns<V>; ++k) {
            const int at = c + k * 32 * V;
            p[k] = *reinterpret_cast<const Pack<T, V>*>(row + (at < dim ? at : 0));
        }
    }
    __device__ __forceinline__ void clear() { memset(p, 0, sizeof(p)); }
    __device__ __forceinline__ float get(int e) const { return to_f32(p[e / V].v[e % V]); }
};
template <int V, typename T>
__device__ __forceinline__ void store_cols(T* row, int c, int dim, const float (&x)[kColumns<V>])
{
#pragma unroll
    for (int k = 0; k < kRuns<V>; ++k) {
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = x[k * V + j];
        if (c + k * 32 * V < dim) store_pack(row + c + k * 32 * V, y);
    }
}
template <int V, typename W>
__device__ __forceinline__ void finish_row(W* row, int c, int dim, const float (&x)[kColumns<V>], const Cols<W, V>& old, float scale)
{
    float y[kColumns<V>];
#pragma unroll
    for (int e = 0; e < kColumns<V>; ++e) y[e] = fmaf(x[e], scale, old.get(e));
    store_cols<V>(row, c, dim, y);
}

// What one block clears: vectors of 16 bytes of the buffer, whatever rows they lie in.  The values in
// front of the buffer's first 16-byte place and behind its last are left to block 0.
constexpr int kClearVectors = 4096;   // of a block
template <typename W, int kBlock> struct Clear {
    static constexpr int N = 16 / sizeof(W), kEach = kClearVectors / kBlock;
    static_assert(kEach % 4 == 0, "four at a time");
    int64_t values, vectors, at, row0;
    int skip;
    unsigned col0;
    __device__ __forceinline__ Clear(const SumArgs& a, int64_t block, const W* grad)
    {
        values = a.rows * a.dim;
        skip = (int)((16 - ((uintptr_t)grad & 15)) & 15) / (int)sizeof(W);
        vectors = values > skip ? (values - skip) / N : 0;
        at = block * kClearVectors;
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
        if (at >= vectors) return;
        const unsigned dim = a.dim;
        Pack<W, N> zero;
        memset(&zero, 0, sizeof(zero));
        // from one of the thread's vectors to the next
        const unsigned ahead = kBlock * N / dim, aside = kBlock * N - ahead * dim;
        const unsigned off = col0 + threadIdx.x * N, more = off / dim;
        unsigned col = off - more * dim;
        int64_t row = row0 + more;
        int64_t v = at + threadIdx.x;
        W* p = grad + skip + v * N;
        if (skip == 0 && dim % N == 0) {          // no vector lies in two rows
#pragma unroll 1
            for (int i0 = 0; i0 < kEach; i0 += 4) {
                bool named[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {     // all four are looked up first
                    named[i] = hit(min64(row, a.rows - 1));
                    row += ahead;
                    col += aside;
                    if (col >= dim) {
                        col -= dim;
                        ++row;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (v < vectors && !named[i]) *reinterpret_cast<Pack<W, N>*>(p) = zero;
                    v += kBlock;
                    p += kBlock * N;
                }
            }
            return;
        }
#pragma unroll 1
        for (int i0 = 0; i0 < kEach; i0 += 4) {
            unsigned cols[4];
            int64_t rows[4];
            bool named[4], next[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                cols[i] = col;
                rows[i] = row;
                named[i] = hit(min64(row, a.rows - 1));
                next[i] = col + N > dim && hit(min64(row + 1, a.rows - 1));
                row += ahead;
                col += aside;
                if (col >= dim) {
                    col -= dim;
                    ++row;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (v < vectors) {
                    if (dim >= N && !named[i] && !next[i]) {      // in one row, or in two that no token names
                        *reinterpret_cast<Pack<W, N>*>(p) = zero;
                    } else if (dim >= N) {
                        for (unsigned j = 0; j < N; ++j)
                            if (!(cols[i] + j < dim ? named[i] : next[i])) p[j] = W(0.f);
                    } else {
                        for (unsigned j = 0; j < N; ++j)
                            if (!hit(rows[i] + (cols[i] + j) / dim)) p[j] = W(0.f);
                    }
                }
                v += kBlock;
                p += kBlock * N;
            }
        }
    }
};

template <typename W>
__device__ __forceinline__ void clear_block(const SumArgs& a, int64_t block, W* grad)
{
    auto hit = [&](int64_t row) { return a.touched[row >> 5] >> (row & 31) & 1u; };
    Clear<W, kThreads>(a, block, grad).run(a, grad, hit, hit);
}

// kRows rows are on their way at a time.  With many units few of them, because what hides the memory's
// latency then is warps: a gradient of 32768 tokens over 128000 x 4096 bf16 takes 212 us with four blocks an
// SM and four rows of 8 columns a lane, 224 with eight rows.  With few units, for which eight rows'
// registers leave room, more: 16205 rows of 4 fp32 values added to a gradient of 250000 take 26 us two
// at a time, 21 eight at a time.
constexpr int rows_many(bool add) { return add ? 2 : 4; }
constexpr int kRowsFew = 8;
template <typename G, typename W, int V, bool kAdd, int kRows>
__global__ void __launch_bounds__(kThreads, kRows == kRowsFew ? 1 : 4) k_token_sum(SumArgs a, const G* __restrict__ up, int64_t stride, W* __restrict__ grad)
{
    let_next_kernel_start();
    wait_for_kernel_before();
    if (has_error(a.status)) return;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x >= a.sums) {
        clear_block<W>(a, blockIdx.x - a.sums, grad);
        return;
    }
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t tile = unit / a.slabs;
    if (tile >= a.tiles) return;
    const int c = (int)(unit - tile * a.slabs) * 32 * kColumns<V> + lane * V;
    const uint32_t none = (uint32_t)a.rows;
    const int64_t p0 = tile * a.tile, p1 = min64(p0 + a.tile, a.n);
    bool began = p0 > 0 && a.keys[p0 - 1] == a.keys[p0];  // the current run began in an earlier tile
    constexpr int E = kColumns<V>;
    F2 acc[E / 2];
#pragma unroll
    for (int j = 0; j < E / 2; ++j) acc[j] = both(0.f);
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
            Cols<G, V> x[kRows];
            Cols<W, V> old[kAdd ? kRows : 1];
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const int64_t row = __shfl_sync(kFull, val, q + u);
                x[u].load(up + row * stride, c, a.dim);
                if constexpr (kAdd) {
                    const uint32_t k = __shfl_sync(kFull, key, q + u);
                    old[u].load(grad + (int64_t)(k < none ? k : 0u) * a.dim, c, a.dim);
                }
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                if (q + u >= cnt) break;
#pragma unroll
                for (int j = 0; j < E / 2; ++j) acc[j] = add2(acc[j], {x[u].get(2 * j), x[u].get(2 * j + 1)});
                if (!(ends >> (q + u) & 1u)) continue;
                float sum[E];
#pragma unroll
                for (int e = 0; e < E; ++e) sum[e] = e & 1 ? acc[e / 2].y : acc[e / 2].x;
                const bool here = whole >> (q + u) & 1u;
                const uint32_t k = __shfl_sync(kFull, key, q + u);
                if (began) {
                    store_cols<V>(a.head + tile * a.dim, c, a.dim, sum);
                } else if (!here) {
                    store_cols<V>(a.tail + tile * a.dim, c, a.dim, sum);
                } else {
                    if constexpr (!kAdd) old[0].clear();
                    finish_row<V>(grad + (int64_t)k * a.dim, c, a.dim, sum, old[kAdd ? u : 0], a.scale);
                }
                began = false;
#pragma unroll
                for (int j = 0; j < E / 2; ++j) acc[j] = both(0.f);
            }
        }
        if (cnt < 32) break;
    }
}

// Its first `joins` blocks: where a run begins in a tile and goes on, they add up its parts, kSplit
// warps for a slab, each a row of tiles, and then the warps' sums, all in order.  The other blocks
// clear rows that no token names.
constexpr int kSplit = 4, kJoinSlabs = kWarps / kSplit;
template <typename W, int V>
__global__ void __launch_bounds__(kThreads) k_token_join(SumArgs a, int64_t joins, W* __restrict__ grad)
{
    wait_for_kernel_before();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    constexpr int E = kColumns<V>;
    __shared__ float s_part[kWarps][32 * E];
    const int groups = (a.slabs + kJoinSlabs - 1) / kJoinSlabs;   // blocks of a tile
    const int64_t tile = blockIdx.x / groups, p0 = tile * a.tile, p1 = p0 + a.tile;
    const bool join = blockIdx.x < joins && p1 < a.n;
    const uint32_t k = join ? a.keys[p1 - 1] : 0u, then = join ? a.keys[p1] : 0u, front = join && p0 > 0 ? a.keys[p0 - 1] : ~0u;
    if (has_error(a.status)) return;
    if (blockIdx.x >= joins) {
        clear_block<W>(a, a.first_clear + (blockIdx.x - joins), grad);
        return;
    }
    // nothing goes on, or it began earlier
    if (!join || k >= (uint32_t)a.rows || then != k || front == k) return;
    const int split = wid % kSplit, slab = (int)(blockIdx.x - tile * groups) * kJoinSlabs + wid / kSplit;
    const int c = slab * 32 * E + lane * V;
    // the last tile that the run reaches: 32 tiles' first keys at a time
    int64_t last = tile;                                          // heads of tiles tile + 1 .. last
    for (;;) {
        const int64_t p = (last + 1 + lane) * a.tile;
        const unsigned same = __ballot_sync(kFull, p < a.n && a.keys[min64(p, a.n - 1)] == k);
        const int m = same == kFull ? 32 : __ffs(~same) - 1;
        last += m;
        if (m < 32) break;
    }
    W* const row = grad + (int64_t)k * a.dim;
    Cols<W, V> old;
    old.clear();
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    if (split == 0) {
        Cols<float, V> x;
        x.load(a.tail + tile * a.dim, c, a.dim);
        if (a.accumulate) old.load(row, c, a.dim);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = x.get(e);
    }
    const int64_t each = (last - tile + kSplit - 1) / kSplit, from = tile + 1 + split * each, to = min64(from + each, last + 1);
    constexpr int kParts = 8;                                     // parts on their way at a time
    for (int64_t t = from; t < to; t += kParts) {
        Cols<float, V> x[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i) x[i].load(a.head + min64(t + i, to - 1) * a.dim, c, a.dim);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            if (t + i >= to) break;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += x[i].get(e);
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_part[wid][e * 32 + lane] = acc[e];
    __syncthreads();
    if (split > 0) return;
    for (int w = wid + 1; w < wid + kSplit; ++w)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += s_part[w][e * 32 + lane];
    finish_row<V>(row, c, a.dim, acc, old, a.scale);
}

// ---------------------------------------------------------------------------
// Few tokens: one launch.  A block of the first `slabs` sorts the tokens by itself (each key's place is
// the number of keys in front of it, counted) and adds up one slab, each warp a part of the sorted
// positions, whose ends are joined in shared memory.  The others clear rows; each looks
// up the few tokens in the rows that it covers.
// ---------------------------------------------------------------------------
//
// The counting grows with the square of the tokens: over 5000 x 512 fp32, 256 tokens take 9 us (16 by
// sort, sums and joins), 512 took 19 (16).
constexpr int kFew = 256;
constexpr int kFewThreads = 1024, kFewWarps = kFewThreads / 32;
constexpr int kFewRows = kClearVectors * 8;   // rows that a block's vectors lie in at most

template <typename G, typename W, int V, bool kAdd>
__global__ void __launch_bounds__(kFewThreads) k_token_few(TokenArgs t, SumArgs a, const G* __restrict__ up, int64_t stride, W* __restrict__ grad)
{
    constexpr int kRows = 4;
    __shared__ alignas(16) uint32_t s_key[kFew];
    __shared__ uint32_t s_sorted[kFew + 1];
    __shared__ int32_t s_place[kFew], s_front[kFew];
    __shared__ uint32_t s_bits[kFewRows / 32 + 1];
    constexpr int E = kColumns<V>;
    __shared__ float s_part[kFewWarps][32 * E];
    const int n = (int)t.n, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const uint32_t none = (uint32_t)a.rows;
    // kParts threads for a key, which count a part of the others each
    constexpr int kParts = kFewThreads / kFew;
    const int mine = tid & (kFew - 1), part = tid / kFew;
    const int64_t token = token_at(t.tokens, t.token_bytes, min(mine, n - 1));
    const bool bad = token < 0 || token >= a.rows;
    if (part == 0) {
        s_key[mine] = mine < n && !bad && token != t.pad ? (uint32_t)token : none;
        s_front[mine] = 0;
        if (bad && mine < n) raise_error(t.status, TT_ERR_INDEX_RANGE, mine);
    }
    if (__syncthreads_or(bad || has_error(t.status))) return;
    if ((int)blockIdx.x >= a.slabs) {
        // the rows of this block's vectors that a token names, as bits
        const int64_t chunk = ((int64_t)blockIdx.x - a.slabs) * a.clear_each, row0 = Clear<W, kFewThreads>(a, chunk, grad).row0;
        for (int i = tid; i < kFewRows / 32 + 1; i += kFewThreads) s_bits[i] = 0;
        __syncthreads();
        if (tid < n) {
            const int64_t r = (int64_t)s_key[tid] - row0;
            if (s_key[tid] < none && r >= 0 && r < kFewRows + 32) atomicOr(&s_bits[r >> 5], 1u << (r & 31));
        }
        __syncthreads();
        auto hit = [&](int64_t row) { return s_bits[(row - row0) >> 5] >> ((row - row0) & 31) & 1u; };
        auto far = [&](int64_t row) {
            bool found = false;
            for (int i = 0; i < n; ++i) found |= s_key[i] == (uint32_t)row;
            return found;
        };
        for (int i = 0; i < a.clear_each; ++i) Clear<W, kFewThreads>(a, chunk + i, grad).run(a, grad, hit, far);
        return;
    }
    // places: keys below mine, and equal ones in front
    {
        const uint32_t key = s_key[mine];
        const int quads = (n + 3) / 4, each = (quads + kParts - 1) / kParts, from = part * each, to = min(quads, from + each);
        int front = 0;
        for (int i = from; i < to; ++i) {     // what is behind the last token is `none`, never below, and never in front of one
            const uint4 q = reinterpret_cast<const uint4*>(s_key)[i];
            front += (q.x < key || (q.x == key && 4 * i < mine)) + (q.y < key || (q.y == key && 4 * i + 1 < mine)) +
                     (q.z < key || (q.z == key && 4 * i + 2 < mine)) + (q.w < key || (q.w == key && 4 * i + 3 < mine));
        }
        if (mine < n) atomicAdd(&s_front[mine], front);
    }
    __syncthreads();
    if (tid < n) {
        s_sorted[s_front[tid]] = s_key[tid];
        s_place[s_front[tid]] = tid;
    }
    if (tid == 0) s_sorted[n] = none;
    __syncthreads();
    const int c = (int)blockIdx.x * 32 * E + lane * V;
    const int each = (n + kFewWarps - 1) / kFewWarps, p0 = min(n, wid * each), p1 = min(n, p0 + each);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    auto row_of = [&](uint32_t k) { return grad + (int64_t)k * a.dim; };
    // a run that goes over this part's end is left in acc, and what ends one that began before in s_part
    bool began = p0 > 0 && p0 < n && s_sorted[p0 - 1] == s_sorted[p0];
    uint32_t k = none;
    for (int p = p0; p < p1; p += kRows) {
        Cols<G, V> x[kRows];
        Cols<W, V> old[kAdd ? kRows : 1];
        old[0].clear();
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            const int q = min(p + u, p1 - 1);
            x[u].load(up + (int64_t)s_place[q] * stride, c, a.dim);
            if constexpr (kAdd) old[u].load(row_of(s_sorted[q] < none ? s_sorted[q] : 0u), c, a.dim);
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (p + u >= p1) break;
            k = s_sorted[p + u];
            if (k >= none) break;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += x[u].get(e);
            if (s_sorted[p + u + 1] == k) continue;
            if (began) {
#pragma unroll
                for (int e = 0; e < E; ++e) s_part[wid][e * 32 + lane] = acc[e];
                began = false;
            } else {
                finish_row<V>(row_of(k), c, a.dim, acc, old[kAdd ? u : 0], a.scale);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = 0.f;
        }
    }
    // what is left in acc goes on behind this part, or is all of a part that a run covers
    const bool goes_on = p1 > p0 && p1 < n && k < none && s_sorted[p1] == k;
    if (goes_on && began)
#pragma unroll
        for (int e = 0; e < E; ++e) s_part[wid][e * 32 + lane] = acc[e];
    __syncthreads();
    if (!goes_on || began) return;
    for (int w = wid + 1; w < kFewWarps && w * each < n && s_sorted[w * each] == k; ++w)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += s_part[w][e * 32 + lane];
    Cols<W, V> old;
    old.clear();
    if constexpr (kAdd) old.load(row_of(k), c, a.dim);
    finish_row<V>(row_of(k), c, a.dim, acc, old, a.scale);
}

// Positions a tile has: longer tiles cut fewer runs, shorter ones give every warp of the card a unit.  24
// units an SM: 32768 tokens over 128000 x 4096 bf16 take 212 us so, 221 with 12 and 218 with 48.
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

// whether rows of `stride` values at p begin at multiples of `bytes`
bool rows_at(const void* p, int64_t stride, int type, int bytes)
{
    return ((uintptr_t)p & (bytes - 1)) == 0 && (stride * type_bytes(type)) % bytes == 0;
}

// Neighbouring values that one access may move in rows of both kinds: 16 bytes of the narrower type, or a
// pair, or one.  Against 16 bytes of the wider type and 8 of the other: 65536 bf16 rows of 2048 added to an fp32
// gradient of 256000 take 147 us, 188 so; fp32 rows of 2048 looked up into bf16 13.0 us, 13.7 so, for 8192 tokens, and as
// long for 131072 (164 us).  It loses where a wide type is written by few warps: 8192 bf16 rows looked up into fp32
// take 19.1 us, 15.6 so, and 200 of 512 summed into fp32 12.1 us, 8.5 so.
int width_of(int dim, const void* p, int64_t p_stride, int p_type, const void* q, int64_t q_stride, int q_type)
{
    const int most = p_type == TT_F32 && q_type == TT_F32 ? 4 : 8;
    if (dim % most == 0 && rows_at(p, p_stride, p_type, 16) && rows_at(q, q_stride, q_type, 16)) return most;
    return dim % 2 == 0 && rows_at(p, p_stride, p_type, 2 * type_bytes(p_type)) && rows_at(q, q_stride, q_type, 2 * type_bytes(q_type)) ? 2 : 1;
}

}  // namespace

namespace {

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
    const int V = width_of(h->dim, h->table, h->dim, h->table_type, out, out_stride, out_type);
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
    for (a.lane_bits = 0; (1 << a.lane_bits) < vectors && a.lane_bits < 5;) ++a.lane_bits;
    const int rows = 32 >> a.lane_bits;
    constexpr int kAnyCols = 2, kAnySteps = 8;            // of pairs and single values
    a.slabs = (unsigned)ceil_div(vectors, 32 * (V > 2 ? 1 : kAnyCols));
    // As many tokens to a unit as leave 64 units an SM: 8192 rows of 4096 bf16 take 20.5 us so, 21.3 with 24
    // units and 22.5 with 128.
    a.per_unit = rows;
    while (a.per_unit < 32 && ceil_div(n, a.per_unit * 2) * a.slabs >= (int64_t)h->num_sms * 64) a.per_unit *= 2;
    const int64_t units = ceil_div(n, a.per_unit) * a.slabs;
    if (units > UINT32_MAX - kWarps) return TT_ERR_ARG;   // sizes that no device holds
    const unsigned grid = (unsigned)ceil_div(units, kWarps);
    by_type(h->table_type, [&](auto t) {
        by_type(out_type, [&](auto o) {
            using T = decltype(t);
            using O = decltype(o);
            auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, s>>>(a, (const T*)h->table, (O*)out); };
            constexpr int kWide = sizeof(T) == 4 && sizeof(O) == 4 ? 4 : 8;
            const bool many = a.per_unit > rows;
            if (V > 2) go(many ? k_lookup<T, O, kWide, 1, 4> : k_lookup<T, O, kWide, 1, 1>);
            else if (V == 2) go(many ? k_lookup<T, O, 2, kAnyCols, kAnySteps> : k_lookup<T, O, 2, kAnyCols, 1>);
            else go(many ? k_lookup<T, O, 1, kAnyCols, kAnySteps> : k_lookup<T, O, 1, kAnyCols, 1>);
        });
    });
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

// The launch of k_token_sort: one cluster of blocks with `smem` bytes each.
struct SortLaunch {
    cudaLaunchConfig_t config = {};
    cudaLaunchAttribute at[1];
    SortLaunch(size_t smem, cudaStream_t s)
    {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = kCluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        config.gridDim = dim3(kCluster);
        config.blockDim = dim3(kSortThreads);
        config.dynamicSmemBytes = smem;
        config.stream = s;
        config.attrs = at;
        config.numAttrs = 1;
    }
    SortLaunch(const SortLaunch&) = delete;
};

// Gives k_token_sort leave for its shared memory and for more than eight blocks a cluster on the current device, and
// tells whether such a cluster fits there.  It fits a whole B200; a part of one without sixteen SMs side by side sorts
// by the radix sort's launches, whatever the number of tokens.
bool sort_fits()
{
    auto fits = [](auto kernel, size_t smem) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return false;
        const SortLaunch l(smem, nullptr);
        int clusters = 0;
        return cudaOccupancyMaxActiveClusters(&clusters, kernel, &l.config) == cudaSuccess && clusters > 0;
    };
    const bool all = fits(k_token_sort<1>, sizeof(SortShared<1>)) && fits(k_token_sort<2>, sizeof(SortShared<2>)) &&
                     fits(k_token_sort<4>, sizeof(SortShared<4>)) && fits(k_token_sort<8>, sizeof(SortShared<8>)) &&
                     fits(k_token_sort<16>, sizeof(SortShared<16>));
    if (!all) cudaGetLastError();     // a refusal here is an answer, not an error of the next launch
    return all;
}

// Sorted keys and positions in buffer *which of the workspace.
cudaError_t sort_tokens(tt_emb_dense_t h, const TokenArgs& a, const DenseLayout& y, int bits, int* which, cudaStream_t s)
{
    uint32_t* const keys = (uint32_t*)(h->ws + y.keys[0]);
    int32_t* const vals = (int32_t*)(h->ws + y.vals[0]);
    const int64_t words = ceil_div(h->rows, 32);
    if (a.n <= kClusterTokens && h->clusters) {
        auto go = [&](auto kernel, size_t smem) {
            const SortLaunch l(smem, s);
            return cudaLaunchKernelEx(&l.config, kernel, a, bits, keys, vals, words);
        };
        *which = 0;
        const int64_t each = ceil_div(a.n, kCluster * kSortThreads);
        if (each <= 1) return go(k_token_sort<1>, sizeof(SortShared<1>));
        if (each <= 2) return go(k_token_sort<2>, sizeof(SortShared<2>));
        if (each <= 4) return go(k_token_sort<4>, sizeof(SortShared<4>));
        if (each <= 8) return go(k_token_sort<8>, sizeof(SortShared<8>));
        return go(k_token_sort<16>, sizeof(SortShared<16>));
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
    const int V = width_of(h->dim, h->grad, h->dim, h->grad_type, up, up_stride, up_type);
    SumArgs a;
    a.n = n;
    a.rows = h->rows;
    a.dim = h->dim;
    a.scale = h->scale;
    a.accumulate = accumulate;
    a.slabs = (int)ceil_div(h->dim, 32 * (V > 2 ? V : V == 2 ? kColumns<2> : kColumns<1>));
    a.tile = tile_of(n, a.slabs, h->num_sms);
    a.tiles = ceil_div(n, a.tile);
    a.head = (float*)(h->ws + y.head);
    a.tail = (float*)(h->ws + y.tail);
    a.touched = ta.touched;
    a.status = h->d_status;
    const int64_t joins = a.tiles * ceil_div(a.slabs, kJoinSlabs);
    const int64_t clears = accumulate ? 0 : ceil_div(ceil_div(h->rows * h->dim, 16 / type_bytes(h->grad_type)), kClearVectors);
    // Half of the clearing goes with the sums and half with the joins: few tokens leave the memory idle
    // in both, and many fill it in either (128000 x 4096 bf16: 212 us so, 221 with all of it with the joins).
    a.sums = ceil_div(a.tiles * a.slabs, kWarps);
    a.first_clear = clears / 2;
    const unsigned grid = (unsigned)(a.sums + a.first_clear), grid2 = (unsigned)(joins + clears - a.first_clear);
    if (a.sums + joins + clears > INT32_MAX) return TT_ERR_ARG;   // sizes that no device holds
    if (n <= kFew) {
        // two blocks an SM clear all, if the rows of what one of them clears fit its bits
        a.clear_each = (int)min64(ceil_div(clears, 2 * h->num_sms) + (clears == 0), h->dim);
        by_type(h->grad_type, [&](auto w) {
            by_type(up_type, [&](auto g) {
                using W = decltype(w);
                using G = decltype(g);
                auto go = [&](auto kernel) {
                    kernel<<<(unsigned)(a.slabs + ceil_div(clears, a.clear_each)), kFewThreads, 0, s>>>(ta, a, (const G*)up, up_stride, (W*)h->grad);
                };
                constexpr int kWide = sizeof(W) == 4 && sizeof(G) == 4 ? 4 : 8;
                if (V > 2) go(accumulate ? k_token_few<G, W, kWide, true> : k_token_few<G, W, kWide, false>);
                else if (V == 2) go(accumulate ? k_token_few<G, W, 2, true> : k_token_few<G, W, 2, false>);
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
    cudaError_t e = cudaSuccess;
    by_type(h->grad_type, [&](auto w) {
        using W = decltype(w);
        by_type(up_type, [&](auto g) {
            using G = decltype(g);
            auto go = [&](auto kernel) { e = launch_early(kernel, grid, kThreads, s, a, (const G*)up, up_stride, (W*)h->grad); };
            constexpr int kWide = sizeof(W) == 4 && sizeof(G) == 4 ? 4 : 8;
            const bool few = a.tiles * a.slabs <= (int64_t)h->num_sms * 16;
            auto pick = [&](auto v) {
                constexpr int kV = decltype(v)::value;
                if (accumulate) go(few ? k_token_sum<G, W, kV, true, kRowsFew> : k_token_sum<G, W, kV, true, rows_many(true)>);
                else go(few ? k_token_sum<G, W, kV, false, kRowsFew> : k_token_sum<G, W, kV, false, rows_many(false)>);
            };
            if (V > 2) pick(std::integral_constant<int, kWide>());
            else if (V == 2) pick(std::integral_constant<int, 2>());
            else pick(std::integral_constant<int, 1>());
        });
        if (e != cudaSuccess) return;
        auto go = [&](auto kernel) { e = launch_early(kernel, grid2, kThreads, s, a, joins, (W*)h->grad); };
        if (V == 1) go(k_token_join<W, 1>);
        else if (V == 2) go(k_token_join<W, 2>);
        else if (V == 8) go(k_token_join<W, 8>);
        else if constexpr (sizeof(W) == 4) go(k_token_join<W, 4>);
    });
    return e == cudaSuccess ? TT_OK : TT_ERR_CUDA;
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
    h->clusters = sort_fits();
    // the memset is waited for, as the first call may run on a stream that is not ordered behind this one
    if (cudaMemset(h->d_status, 0, 256) != cudaSuccess || cudaStreamSynchronize(0) != cudaSuccess) {
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
    // the last stream may be a device's default one, which is another stream where another device is current
    if (const int rc = ready(h)) return note(h, rc);
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
