// A dense table W [rows][dim] read as a matrix, and the gradients of that.
//
//   z = x W^T + bias,   out = act(z) + residual
//   dz = grad_out . act'(z),   grad_x = dz W,   grad_W = dz^T x,   grad_bias = sum over rows of dz
//
// Three products of the same kind.  The tensor cores take them (matmul.cu) on 16-bit operands whose rows begin at 16-byte
// places.  What is not like that is laid out first, in the workspace: rows at other places are copied; fp32
// values (and dz, where its rounding to 16 bits would show in a result) are written as three bf16 terms
// x = t0 + t1 + t2, each the nearest bf16 to what the ones before leave, which hold all bits of a value above 2^-110, fp16 values beside
// them as two.  dz is formed in the same pass, and the bias's gradient with it.  Small products, whose time is that of their
// launches, run on the FP32 pipes from where their operands lie, in one launch each.
#include <math.h>

#include <initializer_list>

#include "dense.cuh"
#include "matmul.cuh"

using namespace tt;

namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// products on the FP32 pipes: any type, stride and size
// ---------------------------------------------------------------------------
constexpr int kDeep = 32;

struct SmallArgs {
    Matrix a, b;          // A(r, k) and B(c, k)
    Upstream u;           // with u.act, A's values are times the slope at those of u.pre, which lie likewise
    Epilogue e;
    int64_t pre_si, pre_sk;
    int64_t rows, cols, deep;
    const int32_t* status;
};

// A thread's N values of a tile, `step` apart from the first one's place on, all on their way before the first is used; the first n
// of them are in the matrix, the others 0.
template <typename T, int N>
__device__ __forceinline__ void bring(const T* p, int64_t step, int n, float (&x)[N])
{
    T q[N];
#pragma unroll
    for (int i = 0; i < N; ++i, p += step) q[i] = i < n ? *p : T(0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(q[i]);
}
template <int N>
__device__ __forceinline__ void bring(const void* p, int type, int64_t at, int64_t step, int n, float (&x)[N])
{
    if (type == TT_BF16) bring((const __nv_bfloat16*)p + at, step, n, x);
    else if (type == TT_F16) bring((const __half*)p + at, step, n, x);
    else bring((const float*)p + at, step, n, x);
}
// places o, o + step, .. below `end`
__device__ __forceinline__ int count_below(int64_t o, int step, int64_t end) { return o >= end ? 0 : (int)min64(64, (end - o + step - 1) / step); }

// A block computes R x C values, a thread 4 x 4 of them, 32 steps of k at a time through shared memory; the next 32 are
// on their way meanwhile.
template <int R, int C>
__global__ void __launch_bounds__(kThreads) k_product(const __grid_constant__ SmallArgs g)
{
    if (has_error(g.status)) return;
    static_assert(R * C == 16 * kThreads, "");
    constexpr int kAcross = C / 4;      // threads side by side
    constexpr int kA = R * kDeep / kThreads, kB = C * kDeep / kThreads;     // values of the operands that a thread brings
    __shared__ __align__(16) float As[kDeep][R + 4], Bs[kDeep][C + 1];      // (writes along k fall into different banks)
    const int tx = threadIdx.x % kAcross, ty = threadIdx.x / kAcross;
    const int64_t tiles_c = ceil_div(g.cols, C);
    const int64_t r0 = blockIdx.x / tiles_c * R, c0 = blockIdx.x % tiles_c * C;
    const bool busy = r0 + ty * 4 < g.rows;
    float acc[4][4] = {};
    // neighbouring threads read neighbouring places: along k, or along r and c where those are the near ones
    const bool a_k = g.a.sk == 1, b_k = g.b.sk == 1;
    float a[kA], z[kA], b[kB];
    // the thread's values: of one k and every eighth r or c, or of one r or c and every kThreads / R-th k
    const int ka = a_k ? threadIdx.x % kDeep : threadIdx.x / R, kb = b_k ? threadIdx.x % kDeep : threadIdx.x / C;
    const int64_t ra = r0 + (a_k ? threadIdx.x / kDeep : threadIdx.x % R), cb = c0 + (b_k ? threadIdx.x / kDeep : threadIdx.x % C);
    constexpr int kEighth = kThreads / kDeep;
    const int n_r = a_k ? count_below(ra, kEighth, g.rows) : ra < g.rows ? kA : 0, n_c = b_k ? count_below(cb, kEighth, g.cols) : cb < g.cols ? kB : 0;
    auto fetch = [&](int64_t k0) {
        const int64_t i = k0 + kb, j = k0 + ka;
        bring(g.b.p, g.b.type, cb * g.b.si + i * g.b.sk, b_k ? kEighth * g.b.si : kThreads / C * g.b.sk,
              b_k ? (i < g.deep ? n_c : 0) : min(n_c, count_below(i, kThreads / C, g.deep)), b);
        const int n = a_k ? (j < g.deep ? n_r : 0) : min(n_r, count_below(j, kThreads / R, g.deep));
        bring(g.a.p, g.a.type, ra * g.a.si + j * g.a.sk, a_k ? kEighth * g.a.si : kThreads / R * g.a.sk, n, a);
        if (g.u.act != TT_ACT_NONE) bring(g.u.pre, g.u.pre_type, ra * g.pre_si + j * g.pre_sk, a_k ? kEighth * g.pre_si : kThreads / R * g.pre_sk, n, z);
    };
    fetch(0);
    for (int64_t k0 = 0; k0 < g.deep; k0 += kDeep) {
        if (g.u.act != TT_ACT_NONE) {
#pragma unroll
            for (int q = 0; q < kA; q += 2) {
                const F2 d = slope(g.u.act, F2{z[q], z[q + 1]}, g.u.cap);
                a[q] *= d.x;
                a[q + 1] *= d.y;
            }
        }
#pragma unroll
        for (int q = 0; q < kA; ++q) {
            const int i = threadIdx.x + q * kThreads;
            As[a_k ? i % kDeep : i / R][a_k ? i / kDeep : i % R] = a[q];
        }
#pragma unroll
        for (int q = 0; q < kB; ++q) {
            const int i = threadIdx.x + q * kThreads;
            Bs[b_k ? i % kDeep : i / C][b_k ? i / kDeep : i % C] = b[q];
        }
        __syncthreads();
        if (k0 + kDeep < g.deep) fetch(k0 + kDeep);
        if (busy) {
#pragma unroll 8
            for (int k = 0; k < kDeep; ++k) {
                float x[4], y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = As[k][ty * 4 + i];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = Bs[k][tx + kAcross * j];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
            }
        }
        __syncthreads();
    }
    if (!busy) return;
    const Epilogue& e = g.e;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
        const int64_t c = c0 + tx + kAcross * j;
        if (c >= g.cols) break;
        const int64_t r = r0 + ty * 4;
        const int rows = (int)min64(4, g.rows - r);
        const float bias = e.bias ? load_any(e.bias, e.bias_type, c) : 0.f;
        float y[4], res[4] = {};
        if (e.residual) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < rows) res[i] = load_any(e.residual, e.residual_type, (r + i) * e.residual_stride + c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float s = j == 0 ? acc[i][0] : j == 1 ? acc[i][1] : j == 2 ? acc[i][2] : acc[i][3];
            y[i] = (r + i == e.skip_row ? 0.f : s) + bias;
            if (e.pre && i < rows) store_any(e.pre, e.pre_type, (r + i) * e.pre_stride + c, y[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const F2 v = activate(e.act, F2{y[i], y[i + 1]}, e.cap);
            y[i] = v.x + res[i];
            y[i + 1] = v.y + res[i + 1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < rows) store_any(e.out, e.out_type, (r + i) * e.out_stride + c, y[i]);
    }
}

// ---------------------------------------------------------------------------
// operands laid out, dz, the bias's gradient
// ---------------------------------------------------------------------------
constexpr int kPackCols = 256;       // columns of a block: eight a lane

struct PackArgs {
    Upstream u;           // the values: u.up, times the slope at u.pre
    int64_t rows, cols, ld;
    int64_t each;         // rows of a block
    void* narrow;         // [rows][ld] of narrow_type; may be null
    uint16_t* wide;       // [parts][rows][ld] bf16 terms; may be null
    float* sums;          // [blocks of rows][cols] sums over a block's rows; may be null
    void* total;          // with one block of rows: the bias's gradient itself; may be null
    int32_t total_type, accumulate;
    const int32_t* status;
    int32_t narrow_type, parts;
    int32_t vectors;      // every row begins at a place that vector loads can take, and is a multiple of eight values
    int32_t across;       // blocks side by side
};
constexpr int kJobs = 3;
struct PackList {
    PackArgs job[kJobs];
    unsigned first[kJobs + 1];     // blocks
    int32_t early;                 // so few blocks that the next kernel's may wait beside them
};

// Eight neighbouring values as they lie in memory, 16-byte aligned.
struct Raw8 { uint4 a, b; };
__device__ __forceinline__ Raw8 load8(const void* p, int type, int64_t at)
{
    Raw8 q;
    if (type == TT_F32) {
        q.a = ((const uint4*)((const float*)p + at))[0];
        q.b = ((const uint4*)((const float*)p + at))[1];
    } else {
        q.a = *(const uint4*)((const uint16_t*)p + at);
    }
    return q;
}
template <typename T>
__device__ __forceinline__ void widen8(const Raw8& q, float (&x)[8])
{
    T v[32 / sizeof(T)];
    memcpy(v, &q, 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(v[i]);
}
__device__ __forceinline__ void widen8(const Raw8& q, int type, float (&x)[8])
{
    if (type == TT_BF16) widen8<__nv_bfloat16>(q, x);
    else if (type == TT_F16) widen8<__half>(q, x);
    else widen8<float>(q, x);
}
// A row of up to 256 values from any place: neighbouring lanes read neighbouring values, which go to shared memory, from
// where each lane takes its eight.
template <typename T>
__device__ __forceinline__ void load_row(const T* p, int n, int lane, float* buf)
{
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = lane + 32 * i < n ? p[lane + 32 * i] : T(0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) buf[lane + 32 * i] = to_f32(v[i]);
}
__device__ __forceinline__ void load_row(const void* p, int type, int64_t at, int n, int lane, float* buf)
{
    if (type == TT_BF16) load_row((const __nv_bfloat16*)p + at, n, lane, buf);
    else if (type == TT_F16) load_row((const __half*)p + at, n, lane, buf);
    else load_row((const float*)p + at, n, lane, buf);
}
__device__ __forceinline__ void take8(const float* buf, int lane, float (&x)[8])
{
    const float4 a = ((const float4*)buf)[2 * lane], b = ((const float4*)buf)[2 * lane + 1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// One bf16 term of eight values, which become what it leaves.  `odd`: some value is not finite, or its nearest bf16 value is not:
// an infinity then leaves 0, and the largest bf16 value stands for what rounds to one.
__device__ __forceinline__ uint4 next_term(float (&x)[8], bool odd)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        memcpy(&w[i], &h, 4);
        if (odd) {
            const bool big0 = fabsf(x[2 * i]) < INFINITY && (w[i] & 0x7fffu) == 0x7f80u, big1 = fabsf(x[2 * i + 1]) < INFINITY && (w[i] >> 16 & 0x7fffu) == 0x7f80u;
            w[i] -= (big0 ? 1u : 0u) + (big1 ? 0x10000u : 0u);
        }
        x[2 * i] -= __uint_as_float(w[i] << 16);
        x[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
        if (odd) {      // infinity less itself
            x[2 * i] = x[2 * i] == x[2 * i] ? x[2 * i] : 0.f;
            x[2 * i + 1] = x[2 * i + 1] == x[2 * i + 1] ? x[2 * i + 1] : 0.f;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One row's eight values of a lane (those beyond the last column 0): times the slope, summed, and written in the forms wanted.
__device__ __forceinline__ void pack_row(const PackArgs& g, int64_t r, int64_t c, float (&x)[8], const float (&z)[8], float (&sum)[8])
{
    auto times = [&](auto act) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const F2 d = mul2(slope(decltype(act)::value, F2{z[i], z[i + 1]}, g.u.cap), F2{x[i], x[i + 1]});
            x[i] = d.x;
            x[i + 1] = d.y;
        }
    };
    if (g.u.act == TT_ACT_RELU) times(std::integral_constant<int, TT_ACT_RELU>());
    else if (g.u.act == TT_ACT_GELU) times(std::integral_constant<int, TT_ACT_GELU>());
    else if (g.u.act == TT_ACT_SILU) times(std::integral_constant<int, TT_ACT_SILU>());
    else if (g.u.act == TT_ACT_SOFTCAP) times(std::integral_constant<int, TT_ACT_SOFTCAP>());
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const F2 t = add2({sum[i], sum[i + 1]}, {x[i], x[i + 1]});
        sum[i] = t.x;
        sum[i + 1] = t.y;
    }
    if (c >= g.cols) return;
    if (g.narrow) {
        if (g.narrow_type == TT_F16) store_pack((__half*)g.narrow + r * g.ld + c, x);
        else store_pack((__nv_bfloat16*)g.narrow + r * g.ld + c, x);
    }
    if (g.wide) {
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(fabsf(x[i])));
        const bool odd = !(most < 0x1.fep127f);
        uint16_t* to = g.wide + r * g.ld + c;
        for (int p = 0; p < g.parts; ++p, to += g.rows * g.ld) *(uint4*)to = next_term(x, odd);
    }
}

__global__ void __launch_bounds__(kThreads, 4) k_pack(const __grid_constant__ PackList list)
{
    constexpr int kWarps = kThreads / 32;
    __shared__ float part[2 * kWarps][kPackCols];
    if (list.early) let_next_kernel_start();
    const int job = blockIdx.x >= list.first[2] ? 2 : blockIdx.x >= list.first[1] ? 1 : 0;
    const PackArgs& g = list.job[job];
    if (has_error(g.status)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned block = blockIdx.x - list.first[job], bx = block % g.across, by = block / g.across;
    const int64_t c0 = (int64_t)bx * kPackCols, c = c0 + lane * 8;
    const int64_t to = min64(g.rows, ((int64_t)by + 1) * g.each);
    int64_t r = (int64_t)by * g.each + warp;
    const bool act = g.u.act != TT_ACT_NONE;
    float sum[8] = {}, x[8], z[8];
    if (g.vectors) {        // (the columns are whole vectors then)
        Raw8 v = {}, w = {};
        auto fetch = [&] {
            if (c >= g.cols || r >= to) return;
            v = load8(g.u.up, g.u.up_type, r * g.u.up_stride + c);
            if (act) w = load8(g.u.pre, g.u.pre_type, r * g.u.pre_stride + c);
        };
        fetch();
        while (r < to) {
            widen8(v, g.u.up_type, x);
            if (act) widen8(w, g.u.pre_type, z);
            const int64_t here = r;
            r += kWarps;
            fetch();
            pack_row(g, here, c, x, z, sum);
        }
    } else {
        float *a = part[2 * warp], *b = part[2 * warp + 1];
        const int n = (int)min64(kPackCols, g.cols - c0);
        for (; r < to; r += kWarps) {
            load_row(g.u.up, g.u.up_type, r * g.u.up_stride + c0, n, lane, a);
            if (act) load_row(g.u.pre, g.u.pre_type, r * g.u.pre_stride + c0, n, lane, b);
            __syncwarp();
            take8(a, lane, x);
            if (act) take8(b, lane, z);
            __syncwarp();
            pack_row(g, r, c, x, z, sum);
        }
    }
    if (!g.sums && !g.total) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) part[warp][i * 32 + lane] = sum[i];
    __syncthreads();
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) all += part[i][threadIdx.x];
    const int64_t at = c0 + (threadIdx.x & 31) * 8 + (threadIdx.x >> 5);
    if (at >= g.cols) return;
    if (g.total) store_any(g.total, g.total_type, at, g.accumulate ? all + load_any(g.total, g.total_type, at) : all);
    else g.sums[by * g.cols + at] = all;
}

// The sums of the blocks of rows: 32 columns of a block of threads, each warp an eighth of the sums.
__global__ void __launch_bounds__(kThreads) k_bias_grad(const float* sums, int64_t blocks, int64_t cols, void* out, int32_t type, int32_t accumulate,
                                                        const int32_t* status)
{
    wait_for_kernel_before();
    if (has_error(status)) return;
    __shared__ float part[kThreads / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int64_t i = warp; i < blocks; i += kThreads / 32) sum += sums[i * cols + c];
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp > 0 || c >= cols) return;
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) sum += part[i][lane];
    if (accumulate) sum += load_any(out, type, c);
    store_any(out, type, c, sum);
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
template <int R, int C>
int launch_product(const SmallArgs& g, cudaStream_t s)
{
    const int64_t blocks = ceil_div(g.rows, R) * ceil_div(g.cols, C);
    if (blocks > INT32_MAX) return TT_ERR_ARG;     // sizes that no device holds
    k_product<R, C><<<(unsigned)blocks, kThreads, 0, s>>>(g);
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

// The workspace's parts, one after another.
struct Space {
    char* base;
    size_t used = 0;
    explicit Space(char* at) : base(at) {}
    void* take(int64_t bytes)
    {
        const size_t at = used;
        used += (size_t)(bytes + 255) / 256 * 256;
        return base ? base + at : nullptr;
    }
};

// Rows whose sums one block of rows makes, which saves the launch that joins several: 2 us of the host's, while the device takes as long
// (32 rows by 4000 x 256 bf16, all gradients: 17.2 us, 16.9 with it).
constexpr int64_t kAlone = 32;
// One matrix of a call in the forms that its products want.
struct Forms {
    PackArgs pack = {};
    bool packs = false;       // the pass over the values is needed
    Operand narrow, wide;
};

// How far apart rows of `cols` values are laid out: at 16-byte places, which tensor maps want; at 128-byte places, where a copied row
// of 64 values is no more cache lines than it has to be, unless rows are that short (515 fp32 columns, three terms: 8.4 us for 24
// stages at 1040 bytes a row).
int64_t laid_out(int64_t cols) { return cols >= 64 ? ceil_div(cols, 64) * 64 : ceil_div(cols, 8) * 8; }

// forms of u's values [rows][cols], which are values of the narrow form's 16 bits as they lie if `plain`
Forms forms_of(Space& w, const Upstream& u, bool plain, int64_t rows, int64_t cols, int narrow_type, bool want_narrow, int wide_parts, bool want_sums,
               int sms, int32_t* status)
{
    Forms f;
    const int64_t ld = laid_out(cols);
    const bool direct = plain && mappable(u.up, u.up_stride, rows, cols);
    f.pack.u = u;
    f.pack.rows = rows;
    f.pack.cols = cols;
    f.pack.ld = ld;
    f.pack.status = status;
    f.pack.narrow_type = narrow_type;
    // one bf16 term is the value itself
    if (wide_parts == 1) want_narrow = true;
    if (want_narrow) {
        f.narrow.type = narrow_type;
        f.narrow.outer = rows;
        f.narrow.inner = cols;
        f.narrow.stride = direct ? u.up_stride : ld;
        f.narrow.p = direct ? u.up : f.pack.narrow = w.take(rows * ld * 2);
        f.packs = !direct;
    }
    if (wide_parts == 1) f.wide = f.narrow;
    if (wide_parts > 1) {
        f.pack.wide = (uint16_t*)w.take(wide_parts * rows * ld * 2);
        f.pack.parts = wide_parts;
        f.wide = {f.pack.wide, rows, cols, ld, rows * ld, TT_BF16, wide_parts};
        f.packs = true;
    }
    f.packs = f.packs || want_sums;
    // Blocks of rows: eight blocks an SM in all, of eight rows, one a warp, at least.
    const int64_t across = ceil_div(cols, kPackCols);
    int64_t down = ceil_div((int64_t)sms * 8, across);
    if (down > ceil_div(rows, 8)) down = ceil_div(rows, 8);
    if (want_sums && rows <= kAlone) down = 1;
    if (down > 65535) down = 65535;
    f.pack.each = ceil_div(rows, down);
    if (want_sums && f.pack.each < rows) f.pack.sums = (float*)w.take(ceil_div(rows, f.pack.each) * cols * 4);
    auto vectors = [&](const void* p, int type, int64_t stride) {
        return ((uintptr_t)p & 15) == 0 && (stride * type_bytes(type) & 15) == 0;
    };
    f.pack.vectors = (cols & 7) == 0 && vectors(u.up, u.up_type, u.up_stride) && (u.act == TT_ACT_NONE || vectors(u.pre, u.pre_type, u.pre_stride));
    return f;
}
Forms forms_of(Space& w, const void* p, int64_t stride, int64_t rows, int64_t cols, int type, bool want_narrow, bool want_wide, int sms, int32_t* status)
{
    const Upstream u = {p, nullptr, stride, 0, type, TT_F32, TT_ACT_NONE, 0.f};
    return forms_of(w, u, type != TT_F32, rows, cols, type, want_narrow, !want_wide ? 0 : type == TT_F32 ? 3 : type == TT_F16 ? 2 : 1, false, sms, status);
}
// all passes of a call in one launch; *any: whether there was one
int launch_pack(std::initializer_list<const Forms*> forms, int sms, bool* any, cudaStream_t s)
{
    PackList list = {};
    int64_t blocks = 0;
    int jobs = 0;
    for (const Forms* f : forms) {
        if (!f->packs) continue;
        const int64_t across = ceil_div(f->pack.cols, kPackCols);
        list.job[jobs] = f->pack;
        list.job[jobs].across = (int)across;
        list.first[jobs++] = (unsigned)blocks;
        blocks += across * ceil_div(f->pack.rows, f->pack.each);
        if (blocks > INT32_MAX) return TT_ERR_ARG;     // sizes that no device holds
    }
    *any = jobs > 0;
    if (jobs == 0) return TT_OK;
    for (int i = jobs; i <= kJobs; ++i) list.first[i] = (unsigned)blocks;
    list.early = blocks <= 2 * sms;
    k_pack<<<(unsigned)blocks, kThreads, 0, s>>>(list);
    return cudaGetLastError() == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

// Products by the FP32 pipes, where the tensor cores would want an operand laid out first: one launch instead of two, which the host feels (256
// x 256 x 64 fp32: 9.0 us a call by the pipes, 12.3 by the tensor cores) and the device mostly not (in a replayed graph 7.4 and 6.7), and
// no row of a few values copied (33000 x 4 x 9: 11.8 and 31.2; 520 x 4100 x 17: 16.0 and 19.2).  What costs less is told by a model of
// both times, in us, whose numbers come from 4 to 33000 rows and columns by 1 to 257 k of all three products: the pipes take so long a step of
// 32 k for each tile of 64 x 64 on an SM, and no less than one tile's steps do; the others lay out `short_rows` rows that k runs along, and
// write whole tiles of 128 columns.  (Its choices cost 1.5 % more than the better ones in the mean.)  Long sums, for which the host counts
// less, want 3 us more.  Operands that can be read as they lie take the tensor cores at any size (16 x 96 x 48 bf16: 3.9 us, 6.8 by the pipes).
bool is_small(tt_emb_dense_t h, int64_t rows, int64_t cols, int64_t deep, int64_t short_rows, int result_type)
{
    const double steps = (double)ceil_div(deep, 32), tiles = (double)ceil_div(rows, 64) * (double)ceil_div(cols, 64) / h->num_sms;
    const double pipes = fmax(9.0, 6.5 + steps * fmax(1.6, 1.21 * tiles) + 1.04 * tiles);
    const double written = (double)rows * (double)(ceil_div(cols, 128) * 128 * type_bytes(result_type));
    const double laid = fmax(12.3, (h->table_type == TT_F32 ? 12.0 : 11.5) + 0.4e-3 * (double)short_rows + written / 2.3e6);
    return pipes + (deep > 64 ? 3.0 : 0.0) < laid;
}

// Few rows by a table that would have to be laid out for the tensor cores: reading it once as it lies may cost less than writing and
// reading that.  What is less is told by a model of both times, in us, whose numbers come from 1 to 32 rows by 2000 to 84712 x 65 to
// 4095: the pipes take so long a step of 32 k for each block of 128 columns on an SM, and no less than one block's steps do; laying out
// moves the table, its copy or three terms twice.  (26 rows by 84712 x 280 fp32: 66 us by the pipes, 105 laid out; 32 rows by 12000 x 4095:
// 210 and 179, bf16 290 and 81; 8 rows by 5844 x 280 fp32: 16.8 and 19.0.)  Calls one after another take the host 9 us and 12.5.
constexpr int kFewRows = 32;
bool is_few(tt_emb_dense_t h, int64_t n)
{
    const bool fp32 = h->table_type == TT_F32, as_it_lies = !fp32 && mappable(h->table, h->dim, h->rows, h->dim);
    if (as_it_lies || n > kFewRows || h->dim > 4096) return false;
    const double steps = (double)ceil_div(h->dim, 32), blocks = (double)ceil_div(ceil_div(h->rows, 128), h->num_sms);
    const double step = fmax(n <= 16 ? 1.13 : 1.55, blocks * (0.65 + 0.022 * (double)n));
    const double pipes = fp32 ? 6.5 + steps * step : 5.0 + 1.3 * steps * step;
    const double moved = (double)h->rows * ((fp32 ? 4.0 : 2.0) * h->dim + (fp32 ? 12.0 : 4.0) * laid_out(h->dim));
    const double laid = fp32 ? 13.0 + moved / 5.3e6 : 9.5 + moved / 4.4e6 + 8.6e-5 * (double)h->rows;
    return fmax(pipes, 9.0) < fmax(laid, 12.5);
}

// What the handle's device holds of the product kernels.  Asked for once, when a product is first planned: most tables are never
// read as a matrix.  Sizes may be asked for while another device is current.
const MatmulFits& fits_of(tt_emb_dense_t h)
{
    if (!h->has_fits) {
        int current = h->device;
        const bool elsewhere = cudaGetDevice(&current) == cudaSuccess && current != h->device;
        if (!elsewhere || cudaSetDevice(h->device) == cudaSuccess) {
            h->fits = matmul_fits(h->num_sms);
            h->has_fits = true;
        }
        if (elsewhere) cudaSetDevice(current);
    }
    return h->fits;
}

int take_injection(tt_emb_dense_t h)
{
    const int what = h->inject;
    h->inject = TT_INJECT_NONE;
    return what;
}

Matrix matrix(const void* p, int64_t si, int64_t sk, int type) { return {p, si, sk, type}; }

int enter(tt_emb_dense_t h, cudaStream_t s)
{
    if (const int rc = ready(h)) return rc;
    h->last_stream = s;
    h->used_stream = true;
    return TT_OK;
}

// The call, or with `size` only the workspace that it needs.
int project(tt_emb_dense_t h, const tt_emb_project* a, size_t* size, cudaStream_t s)
{
    if (size) *size = 0;
    if (const int rc = check_forward(h, a)) return rc;
    if (!size)
        if (const int rc = enter(h, s)) return rc;
    if (a->n == 0) return TT_OK;
    const Epilogue e = {a->out, a->residual, a->pre, a->bias, a->out_stride, a->residual_stride, a->pre_stride, -1,
                        a->out_type, a->residual_type, a->pre_type, a->bias_type, a->activation, a->cap};
    const bool few = is_few(h, a->n);
    const bool as_they_lie = h->table_type != TT_F32 && mappable(h->table, h->dim, h->rows, h->dim) && mappable(a->x, a->x_stride, a->n, h->dim);
    if (few || (!as_they_lie && is_small(h, a->n, h->rows, h->dim, a->n + h->rows, a->out_type))) {
        if (size) return TT_OK;
        SmallArgs g = {};
        g.a = matrix(a->x, a->x_stride, 1, h->table_type);
        g.b = matrix(h->table, h->dim, 1, h->table_type);
        g.e = e;
        g.rows = a->n;
        g.cols = h->rows;
        g.deep = h->dim;
        g.status = h->d_status;
        return few ? launch_product<kFewRows, 128>(g, s) : launch_product<64, 64>(g, s);
    }
    Space w(size ? nullptr : h->project_ws);
    const bool wide = h->table_type == TT_F32;
    const Forms x = forms_of(w, a->x, a->x_stride, a->n, h->dim, h->table_type, !wide, wide, h->num_sms, h->d_status);
    const Forms t = forms_of(w, h->table, h->dim, h->rows, h->dim, h->table_type, !wide, wide, h->num_sms, h->d_status);
    Product p;
    p.a = wide ? t.wide : t.narrow;
    p.b = wide ? x.wide : x.narrow;
    p.rows = a->n;
    p.cols = h->rows;
    p.deep = h->dim;
    p.e = e;
    p.has_pre = a->pre != nullptr;
    const MatmulPlan plan = matmul_plan(p, fits_of(h));
    void* const scratch = w.take(plan.scratch);
    if (size) {
        *size = w.used;
        return TT_OK;
    }
    if (w.used > h->project_bytes) return TT_ERR_WORKSPACE;
    bool packed = false;
    if (const int rc = launch_pack({&t, &x}, h->num_sms, &packed, s)) return rc;
    p.fail = take_injection(h);
    return matmul(p, plan, scratch, h->d_status, h->fits, packed, s);
}

int project_backward(tt_emb_dense_t h, const tt_emb_project_grad* a, size_t* size, cudaStream_t s)
{
    if (size) *size = 0;
    if (const int rc = check_backward(h, a)) return rc;
    if (!size)
        if (const int rc = enter(h, s)) return rc;
    if (a->n == 0) {
        if (a->accumulate || size) return TT_OK;
        if (a->table_grad && cudaMemsetAsync(h->grad, 0, (size_t)h->rows * h->dim * type_bytes(h->grad_type), s) != cudaSuccess) return TT_ERR_CUDA;
        if (a->grad_bias && cudaMemsetAsync(a->grad_bias, 0, (size_t)h->rows * type_bytes(a->grad_bias_type), s) != cudaSuccess) return TT_ERR_CUDA;
        return TT_OK;
    }
    const Upstream u = {a->grad_out, a->pre, a->grad_out_stride, a->pre_stride, a->grad_out_type, a->pre_type, a->activation, a->cap};
    Epilogue ex = {}, et = {};
    ex.out = a->grad_x;
    ex.out_stride = a->grad_x_stride;
    ex.out_type = a->grad_x_type;
    ex.skip_row = -1;
    et.out = h->grad;
    et.out_stride = h->dim;
    et.out_type = h->grad_type;
    et.skip_row = h->pad;
    if (a->accumulate) {
        et.residual = h->grad;
        et.residual_stride = h->dim;
        et.residual_type = h->grad_type;
    }
    // Which operands each product takes.  Where grad_out is of the table's 16 bits and is dz itself, as they lie.  Elsewhere a bf16
    // result beside a bf16 table takes dz rounded to bf16: its own rounding is as large (200 by 5000 x 512 with silu: 0.0024 of the norm
    // against 0.0017).  fp32 and fp16 results, which have more bits, take it in full by terms, and so does all that an fp16 table
    // gets: fp32 and bf16 values have more range than fp16, and products with slopes leave fp16's at both ends.
    const int type = h->table_type, up = a->grad_out_type;
    const bool computed = a->activation != TT_ACT_NONE, plain = type != TT_F32 && up == type && !computed;
    auto wide_for = [&](int result) { return type == TT_F32 || (!plain && (result != TT_BF16 || type == TT_F16)); };
    // bf16 terms that hold dz: bf16 values are one, as they lie or copied.  16-bit results beside a 16-bit table take the first two of
    // three, whose rest is at most 2^-17 of it, where the result's own rounding is 2^-11 or more (8192 by 4096 x 128 fp16 with gelu, the
    // table's gradient of fp32: 185 us, 198 with three).
    const int terms = computed || up == TT_F32 ? 3 : up == TT_F16 ? 2 : 1;
    auto terms_for = [&](int result) { return type == TT_F32 || result == TT_F32 || terms < 2 ? terms : 2; };
    const int dz_type = terms == 1 ? TT_BF16 : type;
    const bool dz_lies = plain && mappable(a->grad_out, a->grad_out_stride, a->n, h->rows);
    const bool small_x = a->grad_x && is_small(h, a->n, h->dim, h->rows, a->n, a->grad_x_type) && !(dz_lies && mappable(h->table, h->dim, h->rows, h->dim));
    const bool small_t = a->table_grad && is_small(h, h->rows, h->dim, a->n, 0, h->grad_type) && !(dz_lies && mappable(a->x, a->x_stride, a->n, h->dim));
    const bool big_x = a->grad_x && !small_x, big_t = a->table_grad && !small_t;
    const bool wide_x = big_x && wide_for(a->grad_x_type), wide_t = big_t && wide_for(h->grad_type);
    const int terms_x = wide_x ? terms_for(a->grad_x_type) : 0, terms_t = wide_t ? terms_for(h->grad_type) : 0;
    const int most_terms = terms_x > terms_t ? terms_x : terms_t;
    Space w(size ? nullptr : h->project_ws);
    Forms d = forms_of(w, u, !computed && up != TT_F32 && up == dz_type, a->n, h->rows, dz_type, (big_x && !wide_x) || (big_t && !wide_t),
                       most_terms, a->grad_bias != nullptr, h->num_sms, h->d_status);
    const Forms t = forms_of(w, h->table, h->dim, h->rows, h->dim, type, big_x && !wide_x, wide_x, h->num_sms, h->d_status);
    const Forms x = forms_of(w, a->x, a->x_stride, a->n, h->dim, type, big_t && !wide_t, wide_t, h->num_sms, h->d_status);
    Product px, pt;
    px.cols = pt.cols = h->dim;
    px.a_mn = pt.a_mn = pt.b_mn = true;
    px.rows = pt.deep = a->n;
    px.deep = pt.rows = h->rows;
    px.a = wide_x ? t.wide : t.narrow;
    px.b = wide_x ? d.wide : d.narrow;
    pt.a = wide_t ? x.wide : x.narrow;
    pt.b = wide_t ? d.wide : d.narrow;
    if (wide_x) px.b.parts = terms_x;
    if (wide_t) pt.b.parts = terms_t;
    px.e = ex;
    pt.e = et;
    const MatmulPlan plan_x = big_x ? matmul_plan(px, fits_of(h)) : MatmulPlan(), plan_t = big_t ? matmul_plan(pt, fits_of(h)) : MatmulPlan();
    void* const scratch = w.take(plan_x.scratch > plan_t.scratch ? plan_x.scratch : plan_t.scratch);     // one after the other
    if (size) {
        *size = w.used;
        return TT_OK;
    }
    if (w.used > h->project_bytes) return TT_ERR_WORKSPACE;
    if (a->grad_bias && !d.pack.sums) {
        d.pack.total = a->grad_bias;
        d.pack.total_type = a->grad_bias_type;
        d.pack.accumulate = a->accumulate;
    }
    bool early = false;
    if (const int rc = launch_pack({&d, &t, &x}, h->num_sms, &early, s)) return rc;
    SmallArgs g = {};
    g.u = u;
    g.status = h->d_status;
    if (small_x) {
        g.a = matrix(u.up, u.up_stride, 1, u.up_type);
        g.pre_si = u.pre_stride;
        g.pre_sk = 1;
        g.b = matrix(h->table, 1, h->dim, type);
        g.e = ex;
        g.rows = a->n;
        g.cols = h->dim;
        g.deep = h->rows;
        if (const int rc = launch_product<64, 64>(g, s)) return rc;
    }
    if (small_t) {
        g.a = matrix(u.up, 1, u.up_stride, u.up_type);
        g.pre_si = 1;
        g.pre_sk = u.pre_stride;
        g.b = matrix(a->x, 1, a->x_stride, type);
        g.e = et;
        g.rows = h->rows;
        g.cols = h->dim;
        g.deep = a->n;
        if (const int rc = launch_product<64, 64>(g, s)) return rc;
    }
    if (big_x || big_t) (big_x ? px : pt).fail = take_injection(h);
    if (big_x) {
        if (const int rc = matmul(px, plan_x, scratch, h->d_status, h->fits, early, s)) return rc;
        early = true;
    }
    if (big_t)
        if (const int rc = matmul(pt, plan_t, scratch, h->d_status, h->fits, early, s)) return rc;
    if (d.pack.sums &&
        launch_early(k_bias_grad, (unsigned)ceil_div(h->rows, 32), kThreads, s, (const float*)d.pack.sums, ceil_div(a->n, d.pack.each), h->rows,
                     a->grad_bias, a->grad_bias_type, a->accumulate, (const int32_t*)h->d_status) != cudaSuccess)
        return TT_ERR_CUDA;
    return TT_OK;
}

}  // namespace

extern "C" {

int tt_emb_dense_project_workspace_size(tt_emb_dense_t h, const tt_emb_project* call, size_t* bytes)
{
    if (!bytes) return note(h, TT_ERR_ARG);
    return note(h, project(h, call, bytes, nullptr));
}

int tt_emb_dense_project_backward_workspace_size(tt_emb_dense_t h, const tt_emb_project_grad* call, size_t* bytes)
{
    if (!bytes) return note(h, TT_ERR_ARG);
    return note(h, project_backward(h, call, bytes, nullptr));
}

int tt_emb_dense_set_project_workspace(tt_emb_dense_t h, void* workspace, size_t bytes)
{
    if (!h || !workspace || ((uintptr_t)workspace & 255)) return note(h, TT_ERR_ARG);
    h->project_ws = (char*)workspace;
    h->project_bytes = bytes;
    return TT_OK;
}

int tt_emb_dense_debug_inject(tt_emb_dense_t h, int32_t what)
{
    if (!h || (what != TT_INJECT_NONE && what != TT_INJECT_COPIES && what != TT_INJECT_PRODUCTS && what != TT_INJECT_SUMS)) return note(h, TT_ERR_ARG);
    h->inject = what;
    return TT_OK;
}

int tt_emb_dense_project(tt_emb_dense_t h, const tt_emb_project* call, tt_stream_t stream)
{
    return note(h, project(h, call, nullptr, (cudaStream_t)stream));
}

int tt_emb_dense_project_backward(tt_emb_dense_t h, const tt_emb_project_grad* call, tt_stream_t stream)
{
    return note(h, project_backward(h, call, nullptr, (cudaStream_t)stream));
}

}  // extern "C"
