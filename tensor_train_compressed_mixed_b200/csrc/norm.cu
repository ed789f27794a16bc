// The norm over the gradients of many tensors, and gradients scaled by it.
//
//   norm = sqrt(sum over all values of g^2),   factor = bound / norm where norm > bound, else 1
//
// The sums read every gradient once and memory bounds them (66.6 M fp32 values: 46 us, 5.8 TB/s; 403 M bf16 values: 107 to 140), the
// scaling reads and writes them (80 us; the cache spares it some of the 532 MB).  A thread squares and adds the 32 or 64 values of its
// eight vectors in fp32 and goes on in fp64: squares of values beyond 2^63, or all below 2^-45, leave fp32, and such
// a group is squared again in fp64, so that the norm is right over the whole range of the types.  Each block has a
// place for its sum, and the last block adds them in their order: the same gradients give the same bits.
#include <algorithm>
#include <math.h>
#include <new>
#include <type_traits>
#include <utility>

#include "norm.cuh"

using namespace tt;

namespace {

constexpr int kThreads = 256;
constexpr int kVectors = 8;                          // of 16 bytes, on their way per thread
constexpr int kTile = kThreads * kVectors;           // vectors of a tile
constexpr int kFit = 4;                              // blocks of threads on an SM

template <typename T> struct Vec {
    static constexpr int n = 16 / sizeof(T);
    T v[n];
};

// The squares of a thread's vectors v0, v0 + kThreads, .. of a tensor in fp64, read once more: of values whose squares fp32
// cannot hold, or would lose.
template <typename T>
__device__ __noinline__ double squares64(const Vec<T>* body, int64_t v0, int64_t vectors)
{
    double s = 0.0;
    for (int k = 0; k < kVectors; ++k) {
        const int64_t v = v0 + k * kThreads;
        if (v >= vectors) break;
        for (int i = 0; i < Vec<T>::n; ++i) {
            const double x = (double)to_f32(body[v].v[i]);
            s = fma(x, x, s);
        }
    }
    return s;
}

__device__ __forceinline__ const NormRec& tensor_of(const NormList& L, int64_t tile)
{
    int lo = 0, hi = L.count;   // r[lo].tile0 <= tile < r[hi].tile0
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (L.r[mid].tile0 <= tile) lo = mid; else hi = mid;
    }
    return L.r[lo];
}

// Values of a tensor: `lead` single ones, whole vectors from there on, single ones behind the last.  kStay: nothing in this launch
// writes them, so that they may come by the read-only path.
template <typename T, bool kStay>
__device__ __forceinline__ double tile_squares(const NormRec& r, int64_t tile)
{
    const T* g = (const T*)r.grad;
    const Vec<T>* body = (const Vec<T>*)(g + r.lead);
    const int64_t vectors = (r.size - r.lead) / Vec<T>::n;
    const int64_t v0 = (tile - r.tile0) * kTile + threadIdx.x;
    uint4 w[kVectors];
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
        const uint4* p = (const uint4*)(body + v0 + k * kThreads);
        w[k] = v0 + k * kThreads >= vectors ? make_uint4(0, 0, 0, 0) : kStay ? __ldg(p) : *p;
    }
    F2 a[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
    bool some = false;          // gradients of rows that no token touched are all zero
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
        Vec<T> q;
        memcpy(&q, &w[k], 16);
        some |= ((w[k].x | w[k].y | w[k].z | w[k].w) & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) != 0;
#pragma unroll
        for (int i = 0; i < Vec<T>::n; i += 2) {
            const F2 v = {to_f32(q.v[i]), to_f32(q.v[i + 1])};
            a[i / 2 + 2 * k & 3] = fma2(v, v, a[i / 2 + 2 * k & 3]);
        }
    }
    const F2 p = add2(add2(a[0], a[1]), add2(a[2], a[3]));
    const float s = p.x + p.y;
    // all squares of fp16 values fit: 2^-48 to 2^32
    const bool fits = std::is_same_v<T, __half> || (s >= 0x1p-90f && s < 0x1p126f);
    double sum = fits ? (double)s : some ? squares64(body, v0, vectors) : 0.0;
    if (tile == r.tile0) {      // the single values, at most 14 of them
        const int64_t behind = r.lead + vectors * Vec<T>::n;
        const int64_t at = threadIdx.x < r.lead ? threadIdx.x : behind + threadIdx.x - r.lead;
        if (at < r.size) {
            const double x = (double)to_f32(g[at]);
            sum = fma(x, x, sum);
        }
    }
    return sum;
}

// sum over the block, in thread 0
__device__ __forceinline__ double block_sum(double x)
{
    __shared__ double part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
        x = 0.0;
        for (int i = 0; i < kThreads / 32; ++i) x += part[i];
    }
    __syncthreads();
    return x;
}

__device__ __forceinline__ NormResult result_of(double sum, float bound)
{
    const double root = sqrt(sum);
    NormResult q = {};
    q.finite = root < INFINITY;      // also false for NaN
    q.factor = root > (double)bound ? (float)((double)bound / root) : 1.f;
    return q;
}

__global__ void __launch_bounds__(kThreads, kFit) k_norm(const __grid_constant__ NormList L, char* mem, int slots, float bound, float* norm)
{
    let_next_kernel_start();
    double sum = 0.0;
    for (int64_t b = blockIdx.x; b < L.tiles; b += gridDim.x) {
        const NormRec& r = tensor_of(L, b);
        if (r.guard && has_error(r.guard)) continue;
        if (r.type == TT_BF16) sum += tile_squares<__nv_bfloat16, true>(r, b);
        else if (r.type == TT_F16) sum += tile_squares<__half, true>(r, b);
        else sum += tile_squares<float, true>(r, b);
    }
    NormResult* res = (NormResult*)mem;
    double* part = (double*)(mem + 256);
    __shared__ bool last;
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        part[L.first_slot + blockIdx.x] = sum;
        __threadfence();
        last = slots > 0 && atomicAdd(&res->ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;      // the call's last launch alone has slots; those before it have ended
    __threadfence();
    double all = 0.0;
    for (int i = threadIdx.x; i < slots; i += kThreads) all += *(volatile double*)(part + i);
    all = block_sum(all);
    if (threadIdx.x == 0) {
        *res = result_of(all, bound);
        if (norm) *norm = (float)sqrt(all);
    }
}

template <typename T>
__device__ __forceinline__ void tile_scale(const NormRec& r, int64_t tile, float by)
{
    T* g = (T*)r.grad;
    Vec<T>* body = (Vec<T>*)(g + r.lead);
    const int64_t vectors = (r.size - r.lead) / Vec<T>::n;
    const int64_t v0 = (tile - r.tile0) * kTile + threadIdx.x;
    uint4 w[kVectors];
#pragma unroll
    for (int k = 0; k < kVectors; ++k) w[k] = v0 + k * kThreads < vectors ? *(const uint4*)(body + v0 + k * kThreads) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < kVectors; ++k) {
        Vec<T> q;
        memcpy(&q, &w[k], 16);
#pragma unroll
        for (int i = 0; i < Vec<T>::n; ++i) q.v[i] = from_f32<T>(to_f32(q.v[i]) * by);
        memcpy(&w[k], &q, 16);
        if (v0 + k * kThreads < vectors) *(uint4*)(body + v0 + k * kThreads) = w[k];
    }
    if (tile == r.tile0) {
        const int64_t behind = r.lead + vectors * Vec<T>::n;
        const int64_t at = threadIdx.x < r.lead ? threadIdx.x : behind + threadIdx.x - r.lead;
        if (at < r.size) g[at] = from_f32<T>(to_f32(g[at]) * by);
    }
}

__global__ void __launch_bounds__(kThreads, kFit) k_scale(const __grid_constant__ NormList L, const NormResult* res)
{
    wait_for_kernel_before();
    const float by = res->factor;
    if (by == 1.f || !res->finite) return;
    // from the end, where the sums have just been and the cache still holds the gradients
    for (int64_t b = L.tiles - 1 - blockIdx.x; b >= 0; b -= gridDim.x) {
        const NormRec& r = tensor_of(L, b);
        if (r.guard && has_error(r.guard)) continue;
        if (r.type == TT_BF16) tile_scale<__nv_bfloat16>(r, b, by);
        else if (r.type == TT_F16) tile_scale<__half>(r, b, by);
        else tile_scale<float>(r, b, by);
    }
}

// ---------------------------------------------------------------------------
// short lists: sums and scaling in one launch of one cluster, whose blocks exchange their sums
// ---------------------------------------------------------------------------
constexpr int kCluster = 8;
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads) k_clip_few(const __grid_constant__ NormList L, NormResult* res, float bound, float* norm)
{
    __shared__ double mine;
    __shared__ float factor;
    double sum = 0.0;
    for (int64_t b = blockIdx.x; b < L.tiles; b += kCluster) {
        const NormRec& r = tensor_of(L, b);
        if (r.guard && has_error(r.guard)) continue;
        if (r.type == TT_BF16) sum += tile_squares<__nv_bfloat16, false>(r, b);
        else if (r.type == TT_F16) sum += tile_squares<__half, false>(r, b);
        else sum += tile_squares<float, false>(r, b);
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) mine = sum;
    cluster_sync();
    if (threadIdx.x == 0) {
        double all = 0.0;       // in the order of the blocks, in every block alike
        for (int i = 0; i < kCluster; ++i) {
            uint32_t there;
            double part;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"((uint32_t)__cvta_generic_to_shared(&mine)), "r"(i));
            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(part) : "r"(there) : "memory");
            all += part;
        }
        const NormResult q = result_of(all, bound);
        factor = q.finite ? q.factor : 1.f;
        if (blockIdx.x == 0) {
            *res = q;
            if (norm) *norm = (float)sqrt(all);
        }
    }
    cluster_sync();         // nor does a block end while another may read its sum
    const float by = factor;
    if (by == 1.f) return;
    for (int64_t b = blockIdx.x; b < L.tiles; b += kCluster) {
        const NormRec& r = tensor_of(L, b);
        if (r.guard && has_error(r.guard)) continue;
        if (r.type == TT_BF16) tile_scale<__nv_bfloat16>(r, b, by);
        else if (r.type == TT_F16) tile_scale<__half>(r, b, by);
        else tile_scale<float>(r, b, by);
    }
}

struct FewLaunch {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[1];
    explicit FewLaunch(cudaStream_t s)
    {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = kCluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        c.gridDim = dim3(kCluster);
        c.blockDim = dim3(kThreads);
        c.stream = s;
        c.attrs = at;
        c.numAttrs = 1;
    }
    FewLaunch(const FewLaunch&) = delete;
};

}  // namespace

namespace tt {

// Whether a list can be taken at all.
static bool tensors_ok(int32_t count, const tt_emb_norm_tensor* tensors)
{
    if (!tensors || count < 1) return false;
    for (int32_t i = 0; i < count; ++i) {
        const tt_emb_norm_tensor& x = tensors[i];
        if (x.size < 0 || x.size > (int64_t)1 << 40 || !type_known(x.grad_type) || x.reserved != 0) return false;
        if ((uintptr_t)x.guard & 3) return false;
        if (x.size > 0 && (!x.grad || ((uintptr_t)x.grad & (type_bytes(x.grad_type) - 1)))) return false;
    }
    return true;
}

void norm_plan(NormPlan& p, int sms, bool clips, int32_t count, const tt_emb_norm_tensor* tensors)
{
    NormList empty;
    memset(&empty, 0, sizeof(empty));
    p.lists.push_back(empty);
    for (int32_t i = 0; i < count; ++i) {
        const tt_emb_norm_tensor& x = tensors[i];
        if (x.size == 0) continue;
        if (p.lists.back().count == kNormTensors) p.lists.push_back(empty);
        NormList& L = p.lists.back();
        const int bytes = type_bytes(x.grad_type);
        const int64_t lead = min64(x.size, (int64_t)((16 - ((uintptr_t)x.grad & 15)) & 15) / bytes);
        L.r[L.count++] = {x.grad, x.guard, x.size, L.tiles, x.grad_type, (int32_t)lead};
        L.tiles += std::max<int64_t>(1, ((x.size - lead) / (16 / bytes) + kTile - 1) / kTile);
    }
    for (NormList& L : p.lists) {
        L.first_slot = p.slots;
        p.grids.push_back((int)std::max<int64_t>(1, min64(L.tiles, (int64_t)sms * kFit)));
        p.slots += p.grids.back();
    }
    // One launch where each block of the cluster takes one tile of 32 KB, or two: 6.5 us for three tensors of 1334 to 42620 values, 9.5
    // by two launches, but 12.5 us for forty tensors of up to 4099, 9.1 by two.
    if (clips && p.lists.size() == 1 && p.lists[0].tiles <= 2 * kCluster) {
        const FewLaunch l(nullptr);
        int clusters = 0;
        p.few = cudaOccupancyMaxActiveClusters(&clusters, k_clip_few, &l.c) == cudaSuccess && clusters > 0;
        cudaGetLastError();     // a refusal here is an answer, not an error of the next launch
    }
}

cudaError_t cleared(void** mem, size_t bytes)
{
    cudaError_t e = cudaMalloc(mem, bytes);
    if (e != cudaSuccess) {
        *mem = nullptr;
        return e;
    }
    e = cudaMemset(*mem, 0, bytes);
    if (e == cudaSuccess) e = cudaStreamSynchronize(0);
    if (e != cudaSuccess) {
        cudaFree(*mem);
        *mem = nullptr;
    }
    return e;
}

cudaError_t norm_launch(const NormPlan& p, float bound, float* norm, cudaStream_t s)
{
    for (size_t i = 0; i < p.lists.size(); ++i)
        k_norm<<<p.grids[i], kThreads, 0, s>>>(p.lists[i], p.mem, i + 1 == p.lists.size() ? p.slots : 0, bound, norm);
    return cudaGetLastError();
}

cudaError_t norm_clip(const NormPlan& p, float bound, float* norm, cudaStream_t s)
{
    if (p.few) {
        const FewLaunch l(s);
        return cudaLaunchKernelEx(&l.c, k_clip_few, p.lists[0], p.result(), bound, norm);
    }
    const cudaError_t first = norm_launch(p, bound, norm, s);
    if (first != cudaSuccess) return first;
    for (size_t i = p.lists.size(); i-- > 0;) {
        const cudaError_t e = launch_early(k_scale, p.grids[i], kThreads, s, p.lists[i], (const NormResult*)p.result());
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace tt

struct tt_emb_norm_handle {
    NormPlan plan;
    int device = 0;
    bool apart = true;
    std::vector<std::pair<uintptr_t, uintptr_t>> spans;   // of the gradients, sorted
};

namespace {

int measure(tt_emb_norm_t h, bool scale, float max_norm, float* norm, cudaStream_t s)
{
    if (!h || ((uintptr_t)norm & 3) || !(max_norm > 0.f)) return TT_ERR_ARG;
    if (scale && !h->apart) return TT_ERR_ARG;
    for (const auto& x : h->spans)
        if (norm && (uintptr_t)norm < x.second && (uintptr_t)(norm + 1) > x.first) return TT_ERR_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return TT_ERR_CUDA;
    if (dev != h->device) return TT_ERR_STATE;
    return (scale ? norm_clip(h->plan, max_norm, norm, s) : norm_launch(h->plan, max_norm, norm, s)) == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // namespace

extern "C" {

int tt_emb_norm_create(int32_t count, const tt_emb_norm_tensor* tensors, tt_emb_norm_t* out)
{
    if (!out) return TT_ERR_ARG;
    *out = nullptr;
    if (!tensors_ok(count, tensors)) return TT_ERR_ARG;
    tt_emb_norm_handle* h = new (std::nothrow) tt_emb_norm_handle();
    if (!h) return TT_ERR_ARG;
    int rc = TT_OK;
    try {
        for (int32_t i = 0; i < count; ++i)
            if (tensors[i].size > 0)
                h->spans.emplace_back((uintptr_t)tensors[i].grad, (uintptr_t)tensors[i].grad + tensors[i].size * type_bytes(tensors[i].grad_type));
        std::sort(h->spans.begin(), h->spans.end());
        for (size_t i = 1; i < h->spans.size(); ++i) h->apart = h->apart && h->spans[i - 1].second <= h->spans[i].first;
        int sms = 0;
        if (cudaGetDevice(&h->device) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess) {
            rc = TT_ERR_CUDA;
        } else {
            norm_plan(h->plan, sms, true, count, tensors);
            if (cleared((void**)&h->plan.mem, h->plan.bytes()) != cudaSuccess) rc = TT_ERR_CUDA;
        }
    } catch (...) {
        rc = TT_ERR_ARG;
    }
    if (rc != TT_OK) {
        delete h;
        return rc;
    }
    *out = h;
    return TT_OK;
}

int tt_emb_norm_measure(tt_emb_norm_t h, float* norm, tt_stream_t stream)
{
    if (!norm) return TT_ERR_ARG;
    return measure(h, false, INFINITY, norm, (cudaStream_t)stream);
}

int tt_emb_norm_clip(tt_emb_norm_t h, float max_norm, float* norm, tt_stream_t stream)
{
    return measure(h, true, max_norm, norm, (cudaStream_t)stream);
}

void tt_emb_norm_destroy(tt_emb_norm_t h)
{
    if (!h) return;
    cudaFree(h->plan.mem);
    delete h;
}

}  // extern "C"
