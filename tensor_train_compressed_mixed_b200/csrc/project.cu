// A dense table W [rows][dim] read as a matrix, and the gradients of that.
//
//   z = x W^T + bias,   out = act(z) + residual
//   dz = grad_out . act'(z),   grad_x = dz W,   grad_W = dz^T x,   grad_bias = sum over rows of dz
//
// Three products of the same kind: C[r][c] = sum over k of A(r, k) B(c, k).
#include <math.h>

#include "dense.cuh"
#include "project.cuh"

using namespace tt;

namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// products on the FP32 pipes: any type, stride and size
// ---------------------------------------------------------------------------
constexpr int kSide = 64, kDeep = 16;

struct SmallArgs {
    Matrix a, b;          // A(r, k) and B(c, k)
    Upstream u;           // where u.up is set, A is its dz (u_t = 0) or the transpose (u_t = 1)
    Epilogue e;
    int64_t rows, cols, deep;
    int32_t u_t;
    const int32_t* status;
};

// A block computes 64 x 64 values, a thread 4 x 4 of them, 16 steps of k at a time through shared memory.
__global__ void __launch_bounds__(kThreads) k_product(const __grid_constant__ SmallArgs g)
{
    if (has_error(g.status)) return;
    __shared__ float As[kDeep][kSide + 4], Bs[kDeep][kSide + 4];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t tiles_c = ceil_div(g.cols, kSide);
    const int64_t r0 = blockIdx.x / tiles_c * kSide, c0 = blockIdx.x % tiles_c * kSide;
    float acc[4][4] = {};
    // neighbouring threads read neighbouring places: along k, or along r and c where those are the near ones
    const bool a_k = g.u.up ? !g.u_t : g.a.sk == 1, b_k = g.b.sk == 1;
    for (int64_t k0 = 0; k0 < g.deep; k0 += kDeep) {
#pragma unroll
        for (int q = 0; q < kSide * kDeep / kThreads; ++q) {
            const int at = threadIdx.x + q * kThreads;
            const int ak = a_k ? at % kDeep : at / kSide, ar = a_k ? at / kDeep : at % kSide;
            const int bk = b_k ? at % kDeep : at / kSide, bc = b_k ? at / kDeep : at % kSide;
            float a = 0.f, b = 0.f;
            if (r0 + ar < g.rows && k0 + ak < g.deep) {
                if (!g.u.up) a = load_any(g.a.p, g.a.type, (r0 + ar) * g.a.si + (k0 + ak) * g.a.sk);
                else a = g.u_t ? upstream(g.u, k0 + ak, r0 + ar) : upstream(g.u, r0 + ar, k0 + ak);
            }
            if (c0 + bc < g.cols && k0 + bk < g.deep) b = load_any(g.b.p, g.b.type, (c0 + bc) * g.b.si + (k0 + bk) * g.b.sk);
            As[ak][ar] = a;
            Bs[bk][bc] = b;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = As[k][ty * 4 + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = Bs[k][tx + 16 * j];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r0 + ty * 4 + i < g.rows && c0 + tx + 16 * j < g.cols) finish(g.e, r0 + ty * 4 + i, c0 + tx + 16 * j, acc[i][j]);
}

// ---------------------------------------------------------------------------
// the bias's gradient
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) k_bias_grad(Upstream u, int64_t rows, int64_t cols, void* out, int32_t out_type, int32_t accumulate,
                                                        const int32_t* status)
{
    if (has_error(status)) return;
    __shared__ float part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < cols)
        for (int64_t r = warp; r < rows; r += 8) sum += upstream(u, r, c);
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < cols) {
        for (int i = 1; i < 8; ++i) sum += part[i][lane];
        if (accumulate) sum += load_any(out, out_type, c);
        store_any(out, out_type, c, sum);
    }
}

// ---------------------------------------------------------------------------
// checks
// ---------------------------------------------------------------------------
struct Rows {       // n rows of `bytes`, `stride` bytes apart
    uintptr_t at;
    int64_t bytes, stride, n;
    bool none() const { return n == 0 || bytes == 0; }
    uintptr_t end() const { return at + (uintptr_t)((n - 1) * stride + bytes); }
};
Rows rows_of(const void* p, int type, int64_t width, int64_t stride, int64_t n)
{
    return {(uintptr_t)p, p ? width * type_bytes(type) : 0, stride * type_bytes(type), n};
}
// Whether two of them share memory: also not where one lies between the other's rows, as parts of one wider buffer do.
bool overlap(const Rows& a, const Rows& b)
{
    if (a.none() || b.none() || a.end() <= b.at || b.end() <= a.at) return false;
    if (a.stride != b.stride || a.stride <= 0) return true;
    const int64_t apart = (int64_t)(b.at - a.at) % a.stride, from = apart < 0 ? apart + a.stride : apart;
    return !(from >= a.bytes && from + b.bytes <= a.stride);
}
bool matrix_ok(const void* p, int type, int64_t stride, int64_t least)
{
    return p && type_known(type) && ((uintptr_t)p & (type_bytes(type) - 1)) == 0 && stride >= least;
}

int check_forward(tt_emb_dense_t h, const tt_emb_project* a)
{
    if (!h || !a || a->n < 0 || a->n >= INT32_MAX || !activation_known(a->activation)) return TT_ERR_ARG;
    if (a->activation == TT_ACT_SOFTCAP && !(a->cap > 0.f && a->cap < INFINITY)) return TT_ERR_ARG;
    if (!h->table) return TT_ERR_STATE;
    if (a->n == 0) return TT_OK;
    if (!matrix_ok(a->x, h->table_type, a->x_stride, 0) || !matrix_ok(a->out, a->out_type, a->out_stride, h->rows)) return TT_ERR_ARG;
    if (a->residual && !matrix_ok(a->residual, a->residual_type, a->residual_stride, 0)) return TT_ERR_ARG;
    if (a->pre && !matrix_ok(a->pre, a->pre_type, a->pre_stride, h->rows)) return TT_ERR_ARG;
    if (a->bias && !matrix_ok(a->bias, a->bias_type, 0, 0)) return TT_ERR_ARG;
    const Rows out = rows_of(a->out, a->out_type, h->rows, a->out_stride, a->n);
    const Rows pre = rows_of(a->pre, a->pre ? a->pre_type : TT_F32, h->rows, a->pre_stride, a->n);
    const Rows res = rows_of(a->residual, a->residual ? a->residual_type : TT_F32, h->rows, a->residual_stride, a->n);
    const Rows in[3] = {rows_of(a->x, h->table_type, h->dim, a->x_stride, a->n), rows_of(h->table, h->table_type, h->dim, h->dim, h->rows),
                        rows_of(a->bias, a->bias ? a->bias_type : TT_F32, h->rows, h->rows, 1)};
    if (overlap(out, pre)) return TT_ERR_ARG;
    for (const Rows& x : in)
        if (overlap(out, x) || overlap(pre, x)) return TT_ERR_ARG;
    const bool in_place = a->residual == a->out && a->residual_type == a->out_type && a->residual_stride == a->out_stride;
    if (overlap(pre, res) || (!in_place && overlap(out, res))) return TT_ERR_ARG;
    return TT_OK;
}

int check_backward(tt_emb_dense_t h, const tt_emb_project_grad* a)
{
    if (!h || !a || a->n < 0 || a->n >= INT32_MAX || !activation_known(a->activation)) return TT_ERR_ARG;
    if (a->activation == TT_ACT_SOFTCAP && !(a->cap > 0.f && a->cap < INFINITY)) return TT_ERR_ARG;
    if ((a->accumulate != 0 && a->accumulate != 1) || (a->table_grad != 0 && a->table_grad != 1)) return TT_ERR_ARG;
    if (a->grad_bias && !matrix_ok(a->grad_bias, a->grad_bias_type, 0, 0)) return TT_ERR_ARG;
    if (!h->table || (a->table_grad && !h->grad)) return TT_ERR_STATE;
    const bool act = a->activation != TT_ACT_NONE;
    if (a->n > 0) {
        if (!matrix_ok(a->grad_out, a->grad_out_type, a->grad_out_stride, 0)) return TT_ERR_ARG;
        if (a->table_grad && !matrix_ok(a->x, h->table_type, a->x_stride, 0)) return TT_ERR_ARG;
        if (act && !matrix_ok(a->pre, a->pre_type, a->pre_stride, 0)) return TT_ERR_ARG;
        if (a->grad_x && !matrix_ok(a->grad_x, a->grad_x_type, a->grad_x_stride, h->dim)) return TT_ERR_ARG;
    }
    const Rows none = rows_of(nullptr, TT_F32, 0, 0, 0);
    const Rows in[4] = {a->table_grad ? rows_of(a->x, h->table_type, h->dim, a->x_stride, a->n) : none,
                        rows_of(h->table, h->table_type, h->dim, h->dim, h->rows),
                        a->n > 0 ? rows_of(a->grad_out, a->grad_out_type, h->rows, a->grad_out_stride, a->n) : none,
                        a->n > 0 && act ? rows_of(a->pre, a->pre_type, h->rows, a->pre_stride, a->n) : none};
    const Rows out[3] = {a->grad_x ? rows_of(a->grad_x, a->grad_x_type, h->dim, a->grad_x_stride, a->n) : none,
                         a->table_grad ? rows_of(h->grad, h->grad_type, h->dim, h->dim, h->rows) : none,
                         a->grad_bias ? rows_of(a->grad_bias, a->grad_bias_type, h->rows, h->rows, 1) : none};
    for (int i = 0; i < 3; ++i) {
        for (const Rows& x : in)
            if (overlap(out[i], x)) return TT_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return TT_ERR_ARG;
    }
    return TT_OK;
}

// ---------------------------------------------------------------------------
// calls
// ---------------------------------------------------------------------------
int launch_product(const SmallArgs& g, cudaStream_t s)
{
    const int64_t blocks = ceil_div(g.rows, kSide) * ceil_div(g.cols, kSide);
    if (blocks > INT32_MAX) return TT_ERR_ARG;     // sizes that no device holds
    k_product<<<(unsigned)blocks, kThreads, 0, s>>>(g);
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

int project(tt_emb_dense_t h, const tt_emb_project* a, cudaStream_t s)
{
    if (const int rc = check_forward(h, a)) return rc;
    if (const int rc = ready(h)) return rc;
    h->last_stream = s;
    h->used_stream = true;
    if (a->n == 0) return TT_OK;
    SmallArgs g = {};
    g.a = {a->x, a->x_stride, 1, h->table_type};
    g.b = {h->table, h->dim, 1, h->table_type};
    g.e = {a->out, a->residual, a->pre, a->bias, a->out_stride, a->residual_stride, a->pre_stride, -1,
           a->out_type, a->residual_type, a->pre_type, a->bias_type, a->activation, a->cap};
    g.rows = a->n;
    g.cols = h->rows;
    g.deep = h->dim;
    g.status = h->d_status;
    return launch_product(g, s);
}

int project_backward(tt_emb_dense_t h, const tt_emb_project_grad* a, cudaStream_t s)
{
    if (const int rc = check_backward(h, a)) return rc;
    if (const int rc = ready(h)) return rc;
    h->last_stream = s;
    h->used_stream = true;
    if (a->n == 0) {
        if (a->accumulate) return TT_OK;
        if (a->table_grad && cudaMemsetAsync(h->grad, 0, (size_t)h->rows * h->dim * type_bytes(h->grad_type), s) != cudaSuccess) return TT_ERR_CUDA;
        if (a->grad_bias && cudaMemsetAsync(a->grad_bias, 0, (size_t)h->rows * type_bytes(a->grad_bias_type), s) != cudaSuccess) return TT_ERR_CUDA;
        return TT_OK;
    }
    const Upstream u = {a->grad_out, a->pre, a->grad_out_stride, a->pre_stride, a->grad_out_type, a->pre_type, a->activation, a->cap};
    SmallArgs g = {};
    g.u = u;
    g.status = h->d_status;
    if (a->grad_x) {
        g.b = {h->table, 1, h->dim, h->table_type};
        g.e = {};
        g.e.out = a->grad_x;
        g.e.out_stride = a->grad_x_stride;
        g.e.out_type = a->grad_x_type;
        g.e.skip_row = -1;
        g.rows = a->n;
        g.cols = h->dim;
        g.deep = h->rows;
        g.u_t = 0;
        if (const int rc = launch_product(g, s)) return rc;
    }
    if (a->table_grad) {
        g.b = {a->x, 1, a->x_stride, h->table_type};
        g.e = {};
        g.e.out = h->grad;
        g.e.out_stride = h->dim;
        g.e.out_type = h->grad_type;
        if (a->accumulate) {
            g.e.residual = h->grad;
            g.e.residual_stride = h->dim;
            g.e.residual_type = h->grad_type;
        }
        g.e.skip_row = h->pad;
        g.rows = h->rows;
        g.cols = h->dim;
        g.deep = a->n;
        g.u_t = 1;
        if (const int rc = launch_product(g, s)) return rc;
    }
    if (a->grad_bias) {
        k_bias_grad<<<(unsigned)ceil_div(h->rows, 32), kThreads, 0, s>>>(u, a->n, h->rows, a->grad_bias, a->grad_bias_type, a->accumulate, h->d_status);
        if (cudaGetLastError() != cudaSuccess) return TT_ERR_CUDA;
    }
    return TT_OK;
}

}  // namespace

extern "C" {

int tt_emb_dense_project_workspace_size(tt_emb_dense_t h, const tt_emb_project* call, size_t* bytes)
{
    if (!bytes) return note(h, TT_ERR_ARG);
    if (const int rc = check_forward(h, call)) return note(h, rc);
    *bytes = 0;
    return TT_OK;
}

int tt_emb_dense_project_backward_workspace_size(tt_emb_dense_t h, const tt_emb_project_grad* call, size_t* bytes)
{
    if (!bytes) return note(h, TT_ERR_ARG);
    if (const int rc = check_backward(h, call)) return note(h, rc);
    *bytes = 0;
    return TT_OK;
}

int tt_emb_dense_set_project_workspace(tt_emb_dense_t h, void* workspace, size_t bytes)
{
    if (!h || !workspace || ((uintptr_t)workspace & 255)) return note(h, TT_ERR_ARG);
    h->project_ws = (char*)workspace;
    h->project_bytes = bytes;
    return TT_OK;
}

int tt_emb_dense_project(tt_emb_dense_t h, const tt_emb_project* call, tt_stream_t stream)
{
    return note(h, project(h, call, (cudaStream_t)stream));
}

int tt_emb_dense_project_backward(tt_emb_dense_t h, const tt_emb_project_grad* call, tt_stream_t stream)
{
    return note(h, project_backward(h, call, (cudaStream_t)stream));
}

}  // extern "C"
