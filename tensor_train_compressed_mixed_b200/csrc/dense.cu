// Dense tables: scaled lookup of rows, and the table's gradient by sorted tokens.
//
// Both move rows and do one or two operations a value, so memory bounds them.
//
// Lookup.  One thread moves eight neighbouring values (16 bytes of 16-bit ones) of up to four
// rows, whose loads are all issued before the first store.
//
// Gradient.  The tokens are sorted by row (stable, so equal rows stay in input order) and the sorted
// positions are cut into tiles of kTile.  A block adds up the upstream rows of its tiles in fp32
// registers, one run of equal rows after the other; a run that lies inside its tile is written to
// the gradient at once, and the parts of one that crosses tiles go to the workspace and are
// added in tile order by a second kernel.  So a row that many tokens name is spread over many
// blocks, and no sum depends on the order in which blocks run.
#include <new>

#include "types.cuh"

using namespace tt;

namespace {

constexpr int kTile = 32;        // sorted positions per tile
constexpr int kThreads = 256;

__device__ __forceinline__ int64_t token_at(const void* tokens, int token_bytes, int64_t i)
{
    return token_bytes == 8 ? ((const int64_t*)tokens)[i] : (int64_t)((const int32_t*)tokens)[i];
}

template <typename T, typename O, int V, int R>
__global__ void __launch_bounds__(kThreads) k_lookup(const T* __restrict__ table, int64_t rows, int dim, float scale,
                                                     const void* __restrict__ tokens, int token_bytes, int64_t n,
                                                     O* __restrict__ out, int64_t out_stride, int32_t* status)
{
    const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
    const int64_t i0 = ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * R;
    if (c >= dim || has_error(status)) return;
    int64_t row[R];
    float x[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        row[r] = i0 + r < n ? token_at(tokens, token_bytes, i0 + r) : -1;
        if (i0 + r < n && (row[r] < 0 || row[r] >= rows)) {
            raise_error(status, TT_ERR_INDEX_RANGE, (int)min64(i0 + r, INT32_MAX));
            row[r] = -1;
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (row[r] >= 0) load_pack(table + row[r] * dim + c, x[r]);
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (row[r] >= 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) x[r][j] *= scale;
            store_pack(out + (i0 + r) * out_stride + c, x[r]);
        }
}

// sort keys: the token, or `rows` (behind every row) for one that gets no gradient
__global__ void __launch_bounds__(kThreads) k_token_keys(const void* __restrict__ tokens, int token_bytes, int64_t n,
                                                         int64_t rows, int64_t pad, uint32_t* __restrict__ keys,
                                                         int32_t* __restrict__ vals, int32_t* status)
{
    if (has_error(status)) return;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    int64_t t = token_at(tokens, token_bytes, i);
    if (t < 0 || t >= rows) {
        raise_error(status, TT_ERR_INDEX_RANGE, (int)min64(i, INT32_MAX));
        t = rows;
    }
    keys[i] = (uint32_t)(t == pad ? rows : t);
    vals[i] = (int32_t)i;
}

struct SumArgs {
    const uint32_t* keys;     // sorted
    const int32_t* vals;      // input position of each
    int64_t n;
    int64_t rows;
    int dim;
    float scale;
    int accumulate;
    int64_t tiles;
    float* head;              // [tiles][dim] part of a run that began in an earlier tile
    float* tail;              // [tiles][dim] part of a run that begins here and goes on
    const int32_t* status;
};

template <typename W, int V>
__device__ __forceinline__ void finish_row(W* at, float (&x)[V], const SumArgs& a)
{
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] *= a.scale;
    if (a.accumulate) {
        float old[V];
        load_pack(at, old);
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] += old[j];
    }
    store_pack(at, x);
}

template <typename G, typename W, int V>
__global__ void __launch_bounds__(kThreads) k_token_sum(SumArgs a, const G* __restrict__ up, int64_t stride, W* __restrict__ grad)
{
    if (has_error(a.status)) return;
    const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
    const int64_t tile = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (tile >= a.tiles || c >= a.dim) return;
    const int64_t p0 = tile * kTile;
    const int cnt = (int)min64(kTile, a.n - p0);
    const uint32_t* key = a.keys + p0;
    const int32_t* val = a.vals + p0;
    bool began = p0 > 0 && key[-1] == key[0];             // the current run began in an earlier tile
    const bool goes_on = p0 + cnt < a.n && key[cnt] == key[cnt - 1];
    constexpr int U = 4;
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int q0 = 0; q0 < cnt; q0 += U) {
        float x[U][V];
        uint32_t k[U + 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            k[u] = q0 + u < cnt ? key[q0 + u] : (uint32_t)a.rows;
            if (k[u] < (uint32_t)a.rows) load_pack(up + (int64_t)val[q0 + u] * stride + c, x[u]);
        }
        k[U] = q0 + U < cnt ? key[q0 + U] : (uint32_t)a.rows;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k[u] >= (uint32_t)a.rows) break;
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] += x[u][j];
            const bool at_end = q0 + u + 1 == cnt;
            if (!at_end && k[u + 1] == k[u]) continue;
            if (began)
                store_pack(a.head + tile * a.dim + c, acc);
            else if (at_end && goes_on)
                store_pack(a.tail + tile * a.dim + c, acc);
            else
                finish_row(grad + (int64_t)k[u] * a.dim + c, acc, a);
            began = false;
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = 0.f;
        }
    }
}

// Runs that cross tiles: the tile where one begins adds up its parts.
template <typename W, int V>
__global__ void __launch_bounds__(kThreads) k_token_join(SumArgs a, W* __restrict__ grad)
{
    if (has_error(a.status)) return;
    const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
    const int64_t tile = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (tile + 1 >= a.tiles || c >= a.dim) return;
    const int64_t p0 = tile * kTile, p1 = p0 + kTile;
    const uint32_t k = a.keys[p1 - 1];
    if (k >= (uint32_t)a.rows || a.keys[p1] != k) return;         // nothing goes on
    if (p0 > 0 && a.keys[p0 - 1] == k) return;                    // it began earlier
    int64_t lo = p1, hi = a.n;                                    // end of the run: first key above k
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.keys[mid] <= k) lo = mid + 1; else hi = mid;
    }
    const int64_t last = (lo - 1) / kTile;
    float acc[V], x[V];
    load_pack(a.tail + tile * a.dim + c, acc);
#pragma unroll 4
    for (int64_t t = tile + 1; t <= last; ++t) {
        load_pack(a.head + t * a.dim + c, x);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += x[j];
    }
    finish_row(grad + (int64_t)k * a.dim + c, acc, a);
}

struct DenseLayout {
    size_t keys[2], vals[2], hist, digit_total, head, tail, total;
};

DenseLayout dense_layout(int64_t n, int dim)
{
    DenseLayout y;
    size_t p = 0;
    auto take = [&](size_t bytes) {
        const size_t at = p;
        p = (p + bytes + 255) / 256 * 256;
        return at;
    };
    const size_t nz = (size_t)(n > 0 ? n : 1);
    const size_t tiles = (size_t)ceil_div((int64_t)nz, kTile);
    for (int i = 0; i < 2; ++i) {
        y.keys[i] = take(nz * 4);
        y.vals[i] = take(nz * 4);
    }
    y.hist = take(256 * (size_t)ceil_div((int64_t)nz, kSortTile) * 4);
    y.digit_total = take(256 * 4);
    y.head = take(tiles * (size_t)dim * 4);
    y.tail = take(tiles * (size_t)dim * 4);
    y.total = p;
    return y;
}

// threads of a block over the vectors of a row (a power of two) and over rows
dim3 block_for(int64_t vectors)
{
    unsigned x = 1;
    while (x < vectors && x < kThreads) x *= 2;
    return dim3(x, kThreads / x);
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
    const int V = wide ? 8 : 1;
    const int64_t vectors = ceil_div(h->dim, V);
    const dim3 block = block_for(vectors);
    const int64_t by = ceil_div(vectors, block.x);
    // four rows a thread where that still fills the card
    const int64_t rows4 = ceil_div(n, (int64_t)block.y * 4);
    const bool four = rows4 * by >= 4 * h->num_sms;
    const dim3 grid((unsigned)(four ? rows4 : ceil_div(n, block.y)), (unsigned)by);
    by_type(h->table_type, [&](auto t) {
        by_type(out_type, [&](auto o) {
            using T = decltype(t);
            using O = decltype(o);
            auto go = [&](auto kernel) {
                kernel<<<grid, block, 0, s>>>((const T*)h->table, h->rows, h->dim, h->scale, tokens, token_bytes, n,
                                              (O*)out, out_stride, h->d_status);
            };
            if (wide) go(four ? k_lookup<T, O, 8, 4> : k_lookup<T, O, 8, 1>);
            else go(four ? k_lookup<T, O, 1, 4> : k_lookup<T, O, 1, 1>);
        });
    });
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
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
    if (!accumulate &&
        cudaMemsetAsync(h->grad, 0, (size_t)h->rows * h->dim * type_bytes(h->grad_type), s) != cudaSuccess)
        return TT_ERR_CUDA;
    if (n == 0) return TT_OK;
    const DenseLayout y = dense_layout(h->ws_n, h->dim);
    SortBuffers sb;
    for (int i = 0; i < 2; ++i) {
        sb.keys[i] = h->ws + y.keys[i];
        sb.vals[i] = (int32_t*)(h->ws + y.vals[i]);
    }
    sb.hist = (uint32_t*)(h->ws + y.hist);
    sb.digit_total = (uint32_t*)(h->ws + y.digit_total);
    k_token_keys<<<(unsigned)ceil_div(n, kThreads), kThreads, 0, s>>>(tokens, token_bytes, n, h->rows, h->pad,
                                                                      (uint32_t*)sb.keys[0], sb.vals[0], h->d_status);
    if (cudaGetLastError() != cudaSuccess) return TT_ERR_CUDA;
    int bits = 1, which = 0, nl = 0;
    while (h->rows >> bits) ++bits;
    if (radix_sort_pairs(false, n, bits, sb, &which, h->d_status, s, &nl) != cudaSuccess) return TT_ERR_CUDA;

    SumArgs a;
    a.keys = (const uint32_t*)sb.keys[which];
    a.vals = sb.vals[which];
    a.n = n;
    a.rows = h->rows;
    a.dim = h->dim;
    a.scale = h->scale;
    a.accumulate = accumulate;
    a.tiles = ceil_div(n, kTile);
    a.head = (float*)(h->ws + y.head);
    a.tail = (float*)(h->ws + y.tail);
    a.status = h->d_status;
    const bool wide = h->dim % 8 == 0 && wide_rows(h->grad, h->dim, h->grad_type) && wide_rows(up, up_stride, up_type);
    const int64_t vectors = ceil_div(h->dim, wide ? 8 : 1);
    const dim3 block = block_for(vectors);
    const dim3 grid((unsigned)ceil_div(a.tiles, block.y), (unsigned)ceil_div(vectors, block.x));
    by_type(h->grad_type, [&](auto w) {
        using W = decltype(w);
        by_type(up_type, [&](auto g) {
            using G = decltype(g);
            auto go = [&](auto kernel) { kernel<<<grid, block, 0, s>>>(a, (const G*)up, up_stride, (W*)h->grad); };
            if (wide) go(k_token_sum<G, W, 8>); else go(k_token_sum<G, W, 1>);
        });
        if (a.tiles > 1) {
            auto go = [&](auto kernel) { kernel<<<grid, block, 0, s>>>(a, (W*)h->grad); };
            if (wide) go(k_token_join<W, 8>); else go(k_token_join<W, 1>);
        }
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
    if (cudaMemset(h->d_status, 0, 256) != cudaSuccess) {
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
    *bytes = dense_layout(max_tokens, h->dim).total;
    return TT_OK;
}

int tt_emb_dense_set_workspace(tt_emb_dense_t h, void* workspace, size_t bytes, int64_t max_tokens)
{
    if (!h || !workspace || ((uintptr_t)workspace & 255) || max_tokens < 0 || max_tokens >= INT32_MAX)
        return note(h, TT_ERR_ARG);
    if (bytes < dense_layout(max_tokens, h->dim).total) return note(h, TT_ERR_WORKSPACE);
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
