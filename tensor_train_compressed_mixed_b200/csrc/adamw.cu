// AdamW over many tensors in one launch, moments in 32 bits or in 8 bits with one scale for each
// block of 256 values.
//
// Every value is read and written once: 28 bytes a value in fp32, 10 with 16-bit weights and
// gradients and 8-bit moments, for about 15 operations, so memory bounds it.  A warp takes one
// block of 256 values, eight in a row per lane: 16-byte loads of every operand, all issued
// before the first use, and a block's largest magnitude is one warp reduction, so an 8-bit
// block is read, updated, scaled and written without leaving registers.
#include <math.h>
#include <new>
#include <vector>

#include "types.cuh"

using namespace tt;

namespace {

constexpr int kBlk = TT_ADAMW_BLOCK;
constexpr int kPerLane = kBlk / 32;
constexpr int kWarps = 8;
constexpr int kLaunchTensors = 128;   // tensors of one launch; their records travel as its parameters
constexpr uint64_t kGamma = 0x9E3779B97F4A7C15ull;

struct Rec {
    void* param;
    const void* grad;
    void* m;
    void* v;
    float* ms;
    float* vs;
    const int32_t* guard;
    int64_t size;
    int64_t blk0;      // first block of the tensor, counted over the launch
    uint64_t quad0;    // first group of four values, counted over all tensors of the optimiser
    double decay;
};

struct List {
    int32_t count;
    int32_t last;      // the step's last launch: it advances the step count
    int64_t blocks;
    double log_b1, log_b2;
    float b1, b2, c1, c2, eps;   // c = 1 - b, rounded from 64 bits
    uint64_t seed;
    int64_t* steps;
    uint32_t* ticket;
    Rec r[kLaunchTensors];
};

// SplitMix64's finaliser (Steele, Lea and Flood, 2014)
__device__ __forceinline__ uint64_t mix64(uint64_t z)
{
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

// largest finite magnitude of a block of 256 (zero below 2^-100, where 448 / a could overflow)
__device__ __forceinline__ float block_max(const float (&x)[kPerLane])
{
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const float y = fabsf(x[i]);
        a = y < INFINITY ? fmaxf(a, y) : a;
    }
    // magnitudes order like their bits, so one integer reduction does
    a = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(a)));
    return a < 0x1p-100f ? 0.f : a;
}

__device__ __forceinline__ float decode8(uint32_t code)   // e4m3 to fp32, exact
{
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3);
    return __half2float(__half(h));
}

template <typename P, typename G, bool k8>
__global__ void __launch_bounds__(kWarps * 32) k_adamw(const __grid_constant__ List L, float lr,
                                                       const float* __restrict__ lr_device)
{
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int64_t t = *L.steps + 1;
    if (lr_device) lr = *lr_device;
    // 1 - beta^t without cancellation: the product is formed in 64 bits, the rest in 32
    const float fix1 = -expm1f((float)((double)t * L.log_b1));
    const float root2 = sqrtf(-expm1f((float)((double)t * L.log_b2)));
    const float lr1 = lr / fix1;
    const uint64_t start = k8 ? mix64((uint64_t)t * kGamma + L.seed) : 0;

    for (int64_t b = (int64_t)blockIdx.x * kWarps + wid; b < L.blocks; b += (int64_t)gridDim.x * kWarps) {
        int lo = 0, hi = L.count;   // r[lo].blk0 <= b < r[hi].blk0
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (L.r[mid].blk0 <= b) lo = mid; else hi = mid;
        }
        const Rec& r = L.r[lo];
        if (r.guard && has_error(r.guard)) continue;
        const int64_t blk = b - r.blk0;
        const int64_t e0 = blk * kBlk + lane * kPerLane;
        const int n = (int)max((int64_t)0, min64(kPerLane, r.size - e0));   // this lane's values
        P* p_at = (P*)r.param + e0;
        const G* g_at = (const G*)r.grad + e0;
        const uintptr_t where = (uintptr_t)p_at | (uintptr_t)g_at | (k8 ? 0 : (uintptr_t)r.m | (uintptr_t)r.v);
        const bool wide = n == kPerLane && (where & 15) == 0 &&
                          (!k8 || (((uintptr_t)r.m | (uintptr_t)r.v) & 7) == 0);

        float p[kPerLane], g[kPerLane], m[kPerLane], v[kPerLane];
        uint32_t mc[kPerLane], vc[kPerLane];
        float ms = 0.f, vs = 0.f;
        if (k8) {
            ms = r.ms[blk];
            vs = r.vs[blk];
        }
        if (wide) {
            load_pack(p_at, p);
            load_pack(g_at, g);
            if (k8) {
                const uint2 a = *(const uint2*)((const uint8_t*)r.m + e0), c = *(const uint2*)((const uint8_t*)r.v + e0);
#pragma unroll
                for (int i = 0; i < kPerLane; ++i) {
                    mc[i] = ((i < 4 ? a.x : a.y) >> (8 * (i & 3))) & 255u;
                    vc[i] = ((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 255u;
                }
            } else {
                load_pack((const float*)r.m + e0, m);
                load_pack((const float*)r.v + e0, v);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                const bool in = i < n;
                p[i] = in ? to_f32(p_at[i]) : 0.f;
                g[i] = in ? to_f32(g_at[i]) : 0.f;
                if (k8) {
                    mc[i] = in ? ((const uint8_t*)r.m)[e0 + i] : 0u;
                    vc[i] = in ? ((const uint8_t*)r.v)[e0 + i] : 0u;
                } else {
                    m[i] = in ? ((const float*)r.m)[e0 + i] : 0.f;
                    v[i] = in ? ((const float*)r.v)[e0 + i] : 0.f;
                }
            }
        }
        const float keep = (float)(1.0 - (double)lr * r.decay);
        float u[kPerLane];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            if (k8) {
                m[i] = __fmul_rn(decode8(mc[i]), ms);
                u[i] = __fmul_rn(decode8(vc[i]), vs);
                v[i] = __fmul_rn(u[i], u[i]);
            }
            // each operation rounded on its own (no fused multiply-add), and the root to nearest, so
            // that an 8-bit code is a function of the formula and not of the instructions chosen
            m[i] = __fadd_rn(__fmul_rn(m[i], L.b1), __fmul_rn(g[i], L.c1));
            v[i] = __fadd_rn(__fmul_rn(v[i], L.b2), __fmul_rn(__fmul_rn(g[i], g[i]), L.c2));
            u[i] = __fsqrt_rn(v[i]);
            p[i] = p[i] * keep - lr1 * m[i] / (u[i] / root2 + L.eps);
        }
        if (k8) {
            const float am = block_max(m), au = block_max(u);
            const float im = am > 0.f ? 448.f / am : 0.f, iu = au > 0.f ? 448.f / au : 0.f;
            uint64_t word[2];
            const uint64_t q = r.quad0 + (uint64_t)(e0 >> 2);
            word[0] = mix64(start + (q + 1) * kGamma);
            word[1] = mix64(start + (q + 2) * kGamma);
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                // an infinite moment is NaN in 8 bits, which has no infinity; conversion saturates
                const float x = fabsf(m[i]) < INFINITY ? __fmul_rn(m[i], im) : NAN;
                mc[i] = __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
                // times 2^-120 the format's exponents are those of fp32 (its subnormals fp32's), so
                // that the code is the top bits; 16 random ones below them round up or down
                const float y = __fmul_rn(fminf(__fmul_rn(u[i], iu), 448.f), 0x1p-120f);
                const uint32_t part = (uint32_t)(word[i >> 2] >> (16 * (i & 3))) & 0xffffu;
                const uint32_t c = (__float_as_uint(y) + (part << 4)) >> 20;
                vc[i] = u[i] < INFINITY ? (u[i] > 0.f ? max(c, 1u) : 0u) : 0x7fu;
            }
            if (lane == 0) {
                r.ms[blk] = am * (1.f / 448.f);
                r.vs[blk] = au * (1.f / 448.f);
            }
        }
        if (wide) {
            store_pack(p_at, p);
            if (k8) {
                uint2 a = {0, 0}, c = {0, 0};
#pragma unroll
                for (int i = 0; i < kPerLane; ++i) {
                    (i < 4 ? a.x : a.y) |= mc[i] << (8 * (i & 3));
                    (i < 4 ? c.x : c.y) |= vc[i] << (8 * (i & 3));
                }
                *(uint2*)((uint8_t*)r.m + e0) = a;
                *(uint2*)((uint8_t*)r.v + e0) = c;
            } else {
                store_pack((float*)r.m + e0, m);
                store_pack((float*)r.v + e0, v);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPerLane; ++i)
                if (i < n) {
                    p_at[i] = from_f32<P>(p[i]);
                    if (k8) {
                        ((uint8_t*)r.m)[e0 + i] = (uint8_t)mc[i];
                        ((uint8_t*)r.v)[e0 + i] = (uint8_t)vc[i];
                    } else {
                        ((float*)r.m)[e0 + i] = m[i];
                        ((float*)r.v)[e0 + i] = v[i];
                    }
                }
        }
    }

    // The block that is last to get here (all have read the count by then) advances it.
    if (L.last) {
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            if (atomicAdd(L.ticket, 1u) == gridDim.x - 1) {
                *L.ticket = 0;
                *L.steps = t;
            }
        }
    }
}

template <typename P, typename G, bool k8>
cudaError_t launch(const List& L, int sms, float lr, const float* lr_device, cudaStream_t s)
{
    static int per_sm = 0;   // resident blocks of this kernel on an SM; a race writes the same value
    if (per_sm == 0) {
        int n = 0;
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_adamw<P, G, k8>, kWarps * 32, 0);
        if (e != cudaSuccess) return e;
        per_sm = n > 0 ? n : 1;
    }
    int64_t grid = min64(ceil_div(L.blocks, kWarps), (int64_t)sms * per_sm);
    if (grid < 1) grid = 1;
    k_adamw<P, G, k8><<<(unsigned)grid, kWarps * 32, 0, s>>>(L, lr, lr_device);
    return cudaGetLastError();
}

}  // namespace

struct tt_emb_adamw_handle {
    struct Part { int32_t ptype, gtype; List list; };
    std::vector<Part> parts;
    bool k8 = false;
    int device = 0, sms = 148;
    uint32_t* ticket = nullptr;
};

extern "C" {

int tt_emb_adamw_create(int32_t count, const tt_emb_adamw_tensor* tensors, const tt_emb_adamw_options* opt,
                        int64_t* steps, tt_emb_adamw_t* out)
{
    if (!out) return TT_ERR_ARG;
    *out = nullptr;
    if (!tensors || !opt || !steps || ((uintptr_t)steps & 7) || count < 1) return TT_ERR_ARG;
    if (!(opt->beta1 >= 0.0 && opt->beta1 < 1.0 && opt->beta2 >= 0.0 && opt->beta2 < 1.0)) return TT_ERR_ARG;
    if (!((float)opt->eps > 0.f && (float)opt->eps < INFINITY) || opt->reserved != 0) return TT_ERR_ARG;
    if (opt->state_bits != 32 && opt->state_bits != 8) return TT_ERR_ARG;
    const bool k8 = opt->state_bits == 8;
    const int sb = k8 ? 1 : 4;
    for (int32_t i = 0; i < count; ++i) {
        const tt_emb_adamw_tensor& x = tensors[i];
        if (x.size < 0 || x.size > (int64_t)1 << 40 || !type_known(x.param_type) || !type_known(x.grad_type)) return TT_ERR_ARG;
        if (!(x.weight_decay >= 0.0 && x.weight_decay < INFINITY) || ((uintptr_t)x.guard & 3)) return TT_ERR_ARG;
        if (x.size == 0) continue;
        if (!x.param || !x.grad || !x.exp_avg || !x.exp_avg_sq) return TT_ERR_ARG;
        if (((uintptr_t)x.param & (type_bytes(x.param_type) - 1)) || ((uintptr_t)x.grad & (type_bytes(x.grad_type) - 1)))
            return TT_ERR_ARG;
        if ((((uintptr_t)x.exp_avg | (uintptr_t)x.exp_avg_sq) & (sb - 1))) return TT_ERR_ARG;
        if (k8 && (!x.m_scale || !x.v_scale || (((uintptr_t)x.m_scale | (uintptr_t)x.v_scale) & 3))) return TT_ERR_ARG;
    }
    tt_emb_adamw_handle* h = new (std::nothrow) tt_emb_adamw_handle();
    if (!h) return TT_ERR_ARG;
    h->k8 = k8;
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
        cudaMalloc((void**)&h->ticket, 256) != cudaSuccess) {
        delete h;
        return TT_ERR_CUDA;
    }
    if (cudaMemset(h->ticket, 0, 256) != cudaSuccess) {
        cudaFree(h->ticket);
        delete h;
        return TT_ERR_CUDA;
    }
    try {
        List base;
        memset(&base, 0, sizeof(base));
        base.log_b1 = log(opt->beta1);   // beta = 0: -inf, and 1 - beta^t = 1
        base.log_b2 = log(opt->beta2);
        base.b1 = (float)opt->beta1;
        base.b2 = (float)opt->beta2;
        base.c1 = (float)(1.0 - opt->beta1);
        base.c2 = (float)(1.0 - opt->beta2);
        base.eps = (float)opt->eps;
        base.seed = opt->seed;
        base.steps = steps;
        base.ticket = h->ticket;
        uint64_t quad = 0;
        for (int32_t i = 0; i < count; ++i) {
            const tt_emb_adamw_tensor& x = tensors[i];
            const int64_t blocks = ceil_div(x.size, kBlk);
            if (blocks > 0) {
                tt_emb_adamw_handle::Part* part = nullptr;
                for (auto& c : h->parts)
                    if (c.ptype == x.param_type && c.gtype == x.grad_type && c.list.count < kLaunchTensors) part = &c;
                if (!part) {
                    h->parts.push_back({x.param_type, x.grad_type, base});
                    part = &h->parts.back();
                }
                List& L = part->list;
                L.r[L.count++] = {x.param, x.grad, x.exp_avg, x.exp_avg_sq, x.m_scale, x.v_scale, x.guard,
                                  x.size, L.blocks, quad, x.weight_decay};
                L.blocks += blocks;
            }
            quad += (uint64_t)blocks * (kBlk / 4);
        }
        if (h->parts.empty()) h->parts.push_back({TT_F32, TT_F32, base});   // still advances the step
        h->parts.back().list.last = 1;
    } catch (...) {
        cudaFree(h->ticket);
        delete h;
        return TT_ERR_ARG;
    }
    *out = h;
    return TT_OK;
}

int tt_emb_adamw_step(tt_emb_adamw_t h, float lr, const float* lr_device, tt_stream_t stream)
{
    if (!h || ((uintptr_t)lr_device & 3)) return TT_ERR_ARG;
    if (!lr_device && !(lr >= 0.f && lr < INFINITY)) return TT_ERR_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return TT_ERR_CUDA;
    if (dev != h->device) return TT_ERR_STATE;
    cudaStream_t s = (cudaStream_t)stream;
    for (const auto& part : h->parts) {
        const cudaError_t e = by_type(part.ptype, [&](auto p) {
            return by_type(part.gtype, [&](auto g) {
                using P = decltype(p);
                using G = decltype(g);
                return h->k8 ? launch<P, G, true>(part.list, h->sms, lr, lr_device, s)
                             : launch<P, G, false>(part.list, h->sms, lr, lr_device, s);
            });
        });
        if (e != cudaSuccess) return TT_ERR_CUDA;
    }
    return TT_OK;
}

void tt_emb_adamw_destroy(tt_emb_adamw_t h)
{
    if (!h) return;
    if (h->ticket) cudaFree(h->ticket);
    delete h;
}

}  // extern "C"
