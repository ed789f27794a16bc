// AdamW over many tensors in one launch, moments in 32 bits or in 8 bits with one scale for each
// block of 256 values.
//
// Every value is read and written once: 28 bytes a value in fp32, 10 with 16-bit weights and
// gradients and 8-bit moments.  A warp takes one block of 256 values, eight per lane: all loads
// are issued before the first use, and a block's largest magnitude is one warp reduction, so an
// 8-bit block is read, updated, scaled and written without leaving registers.  In 32 bits memory
// bounds it; at 10 bytes a value the card's memory delivers a value every 55 issue slots, so
// there the arithmetic is packed in pairs and kept short, and a warp's next blocks travel to
// shared memory while it computes.
#include <algorithm>
#include <float.h>
#include <math.h>
#include <new>
#include <type_traits>
#include <utility>
#include <vector>

#include "roots.cuh"

using namespace tt;

namespace {

constexpr int kBlk = TT_ADAMW_BLOCK;
constexpr int kPerLane = kBlk / 32;
constexpr int kWarps = 8;
constexpr int kPerWarp = 16;          // blocks of a warp in a tile at most (half a warp of scales)
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
    int64_t tile0;     // first tile of the tensor, counted over the launch
    uint64_t quad0;    // first group of four values, counted over all tensors of the optimiser
    float decay;
    int32_t wide;      // every buffer begins at a place that vector loads can take
};

struct List {
    int32_t count;
    int32_t last;      // the step's last launch: it advances the step count
    int32_t per_warp;  // a tile is up to kWarps * per_warp blocks of one tensor
    int32_t pad;
    int64_t tiles;
    double log_b1, log_b2;
    uint64_t b1, b2, c1, c2, one, minus_b2, minus_c2;     // each twice in a pair; c = 1 - b, rounded from 64 bits
    float eps;
    int32_t pad2;
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

constexpr int kPairs = kPerLane / 2;

// largest magnitude of a block's values, NaN if one of them is; the same in every lane
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// the least of three words below 2^31, which order like the floats of their bits
__device__ __forceinline__ uint32_t min3(uint32_t a, uint32_t b, uint32_t c)
{
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return __float_as_uint(r);
}
__device__ __forceinline__ float block_max(const F2 (&x)[kPairs])
{
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) a = max3(a, x[i].x, x[i].y);
    // magnitudes order like their bits, NaN above infinity
    return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(a)));
}

// the same of the finite values only (blocks that hold others, or huge ones, take this second look)
__device__ __noinline__ float finite_max(F2 a, F2 b, F2 c, F2 d)
{
    F2 x[kPairs] = {a, b, c, d};
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        if (!(fabsf(x[i].x) < INFINITY)) x[i].x = 0.f;
        if (!(fabsf(x[i].y) < INFINITY)) x[i].y = 0.f;
    }
    return block_max(x);
}

// 1 / x to nearest where x is too large for `inverse`, whose approximation is 0 there
__device__ __noinline__ float any_inverse(float x) { return __frcp_rn(x); }

// four codes, NaN's in the place of those whose values are not finite
__device__ __noinline__ uint32_t without_infinities(uint32_t codes, F2 a, F2 b)
{
    const float x[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (!(fabsf(x[i]) < INFINITY)) codes = (codes & ~(255u << (8 * i))) | 0x7fu << (8 * i);
    return codes;
}

__device__ __forceinline__ F2 decode8(uint32_t codes)   // two e4m3 codes (low 16 bits) to fp32, exact
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return {f.x, f.y};
}

// A lane's eight values are kGroups runs of kRun neighbours, kRun * 32 apart: loads of 16 bytes a
// lane and 512 a warp in fp32, and of 16-bit values where no operand is wider than that.
template <typename P, typename G, bool k8> struct Shape {
    static constexpr int run = k8 && sizeof(P) == 2 && sizeof(G) == 2 ? 8 : 4;
    static constexpr int groups = kPerLane / run;
};

template <int run, typename T>
__device__ __forceinline__ void widen(const Pack<T, run>& q, F2* x)
{
#pragma unroll
    for (int i = 0; i < run / 2; ++i) x[i] = {to_f32(q.v[2 * i]), to_f32(q.v[2 * i + 1])};
}
template <int run, typename T>
__device__ __forceinline__ Pack<T, run> narrow(const F2* x)
{
    Pack<T, run> q;
#pragma unroll
    for (int i = 0; i < run / 2; ++i) {
        q.v[2 * i] = from_f32<T>(x[i].x);
        q.v[2 * i + 1] = from_f32<T>(x[i].y);
    }
    return q;
}
struct Factors {
    F2 den_u, den_1, keep;      // the update is m / (den_u u + den_1), u being the root, in 8 bits minus it
    uint64_t start;
};

// A tile, and a warp's share of it: `count` blocks in a row.
struct Tile {
    int64_t first;
    int count;
    int whole;         // those of them that are full and at places that vector loads can take
    __device__ __forceinline__ Tile(const Rec& r, const List& L, int64_t tile)
    {
        const int64_t from = (tile - r.tile0) * (L.per_warp * kWarps), blocks = ceil_div(r.size, kBlk);
        const int here = (int)min64(L.per_warp * kWarps, blocks - from), each = (here + kWarps - 1) / kWarps;
        const int skip = (int)(threadIdx.x >> 5) * each;
        first = from + skip;
        count = max(0, min(each, here - skip));
        whole = r.wide ? (int)max((int64_t)0, min64(count, r.size / kBlk - first)) : 0;
    }
};
__device__ __forceinline__ const Rec& tensor_of(const List& L, int64_t tile)
{
    int lo = 0, hi = L.count;   // r[lo].tile0 <= tile < r[hi].tile0
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (L.r[mid].tile0 <= tile) lo = mid; else hi = mid;
    }
    return L.r[lo];
}

// One lane's part of a block as it lies in memory.
template <typename P, typename G, bool k8> struct Raw {
    static constexpr int run = Shape<P, G, k8>::run, groups = Shape<P, G, k8>::groups;
    using M = std::conditional_t<k8, uint8_t, float>;
    using Moment = std::conditional_t<k8, std::conditional_t<run == 8, uint2, uint32_t>, Pack<float, run>>;
    Pack<P, run> p[groups];
    Pack<G, run> g[groups];
    Moment m[groups], v[groups];
    float ms, vs;
    __device__ __forceinline__ uint32_t codes(const Moment (&c)[groups], int w) const   // four codes of the lane's eight
    {
        if constexpr (run == 8) return w ? c[0].y : c[0].x;
        else return c[w];
    }
    __device__ __forceinline__ void set_codes(Moment (&c)[groups], int w, uint32_t x)
    {
        if constexpr (run == 8) (w ? c[0].y : c[0].x) = x;
        else c[w] = x;
    }
};

// The lane's values in memory, moving from one of the warp's blocks to the next.
template <typename P, typename G, bool k8> struct Place {
    using R = Raw<P, G, k8>;
    static constexpr int run = R::run;
    P* p;
    const G* g;
    typename R::M *m, *v;
    __device__ __forceinline__ Place(const Rec& r, int64_t blk, int lane)
    {
        const int64_t e = blk * kBlk + lane * run;
        p = (P*)r.param + e;
        g = (const G*)r.grad + e;
        m = (typename R::M*)r.m + e;
        v = (typename R::M*)r.v + e;
    }
    __device__ __forceinline__ void next(int blocks)
    {
        p += blocks * kBlk;
        g += blocks * kBlk;
        m += blocks * kBlk;
        v += blocks * kBlk;
    }
};

// n values at p (none of the others is touched) into or out of a vector of N
template <int N, typename Q, typename T>
__device__ __forceinline__ Q some_in(const T* p, int n)
{
    Q q;
    memset(&q, 0, sizeof(q));
    T x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < n ? p[i] : T(0);
    memcpy(&q, x, sizeof(q));
    return q;
}
template <int N, typename Q, typename T>
__device__ __forceinline__ void some_out(T* p, const Q& q, int n)
{
    T x[N];
    memcpy(x, &q, sizeof(q));
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < n) p[i] = x[i];
}

template <typename P, typename G, bool k8>
__device__ __forceinline__ void store_block(const Place<P, G, k8>& at, int from, const Raw<P, G, k8>& x, bool whole, int64_t left)
{
    using R = Raw<P, G, k8>;
#pragma unroll
    for (int k = 0; k < R::groups; ++k) {
        const int o = from + k * 32 * R::run;
        if (whole) {
            *(Pack<P, R::run>*)(at.p + o) = x.p[k];
            *(typename R::Moment*)(at.m + o) = x.m[k];
            *(typename R::Moment*)(at.v + o) = x.v[k];
        } else {
            const int n = (int)max((int64_t)0, min64(R::run, left - k * 32 * R::run));
            some_out<R::run>(at.p + o, x.p[k], n);
            some_out<R::run>(at.m + o, x.m[k], n);
            some_out<R::run>(at.v + o, x.v[k], n);
        }
    }
}

// `random`: the lane's place in the stream of random words
template <typename P, typename G, bool k8>
__device__ __forceinline__ void update(Raw<P, G, k8>& b, uint64_t random, const Factors& f, const List& L)
{
    constexpr int run = Shape<P, G, k8>::run, groups = Shape<P, G, k8>::groups;
    F2 p[kPairs], g[kPairs], m[kPairs], v[kPairs], u[kPairs];
#pragma unroll
    for (int k = 0; k < groups; ++k) {
        widen<run>(b.p[k], p + k * run / 2);
        widen<run>(b.g[k], g + k * run / 2);
        if constexpr (!k8) {
            widen<run>(b.m[k], m + k * run / 2);
            widen<run>(b.v[k], v + k * run / 2);
        }
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        if constexpr (k8) {
            m[i] = mul2(decode8(b.codes(b.m, i / 2) >> (16 * (i & 1)) & 0xffffu), both(b.ms));
            u[i] = mul2(decode8(b.codes(b.v, i / 2) >> (16 * (i & 1)) & 0xffffu), both(b.vs));
            v[i] = mul2(u[i], u[i]);
        }
        m[i] = fma2(mul2(m[i], pair(L.b1)), pair(L.one), mul2(g[i], pair(L.c1)));
        v[i] = fma2(mul2(v[i], pair(k8 ? L.minus_b2 : L.b2)), pair(L.one), mul2(mul2(g[i], g[i]), pair(k8 ? L.minus_c2 : L.c2)));
        if constexpr (k8) u[i] = minus_root2(v[i]);        // here v is minus v, and u minus the root
        else u[i] = {root(v[i].x), root(v[i].y)};
    }
    float am = 0.f, au = 0.f, by_m = 0.f;
    bool odd = false;                                // a value of the block is not finite, or beyond what inverse takes
    if constexpr (k8) {
        am = block_max(m);
        au = block_max(u);
        odd = !(am < 0x1p126f && au < INFINITY);     // (finite roots stay below 2^64)
        by_m = inverse(am);
        if (odd) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                if (v[i].x == -INFINITY) u[i].x = -INFINITY;
                if (v[i].y == -INFINITY) u[i].y = -INFINITY;
            }
            am = finite_max(m[0], m[1], m[2], m[3]);
            au = finite_max(u[0], u[1], u[2], u[3]);
            by_m = any_inverse(am);
        }
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const F2 den = fma2(u[i], f.den_u, f.den_1);
        p[i] = fma2(m[i], {rcp(den.x), rcp(den.y)}, mul2(p[i], f.keep));
    }
    if constexpr (k8) {
        if (am < 0x1p-100f) am = 0.f;
        if (au < 0x1p-100f) au = 0.f;
        b.ms = am * (1.f / 448.f);
        b.vs = au * (1.f / 448.f);
        const F2 im = both(am > 0.f ? __fmul_rn(448.f, by_m) : 0.f), iu = both(au > 0.f ? __fmul_rn(448.f, inverse(au)) : 0.f);
#pragma unroll
        for (int w = 0; w < kPairs / 2; ++w) {       // four neighbours: one word of random bits
            const uint64_t word = mix64(random + (run == 8 ? w : w * 32) * kGamma);
            uint32_t code[4], mc[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = 2 * w + h;
                const F2 x = mul2(m[i], im);
                mc[h] = __nv_cvt_float2_to_fp8x2(make_float2(x.x, x.y), __NV_SATFINITE, __NV_E4M3);
                // times 2^-120 the format's exponents are those of fp32 (its subnormals fp32's), so that
                // the code is the top bits; 16 random ones below them round up or down.  All are
                // shifted by 4, which makes the code the top byte.  A product a few ulps above 448 still
                // gives 448's code, as the random bits end 4 places above the lowest.
                const F2 y = mul2(mul2(u[i], iu), both(-0x1p-120f));
                const uint32_t part = (uint32_t)(word >> (32 * h));
                code[2 * h] = (__float_as_uint(y.x) << 4) + __byte_perm(part, 0u, 0x4104);
                code[2 * h + 1] = (__float_as_uint(y.y) << 4) + __byte_perm(part, 0u, 0x4324);
            }
            // A root above zero (its bits are above 2^24) keeps the least code at least.  Few blocks have a
            // code of zero, which is below every float whose exponent the code's lowest bit reaches.  Words of
            // roots that are not finite may be 2^31 or more, which do not order like floats: odd blocks
            // look at each value.
            if (odd || min3(min3(code[0], code[1], code[2]), code[3], code[3]) < 1u << 24) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    code[e] = max(code[e], min(__float_as_uint(fabsf(e & 1 ? u[2 * w + e / 2].y : u[2 * w + e / 2].x)), 1u << 24));
            }
            b.set_codes(b.m, w, mc[0] | mc[1] << 16);
            b.set_codes(b.v, w, __byte_perm(__byte_perm(code[0], code[1], 0x0073), __byte_perm(code[2], code[3], 0x0073), 0x5410));
        }
        if (odd) {   // the format has no infinity, and conversion saturates
#pragma unroll
            for (int w = 0; w < kPairs / 2; ++w) {
                b.set_codes(b.m, w, without_infinities(b.codes(b.m, w), m[2 * w], m[2 * w + 1]));
                b.set_codes(b.v, w, without_infinities(b.codes(b.v, w), u[2 * w], u[2 * w + 1]));
            }
        }
    }
#pragma unroll
    for (int k = 0; k < groups; ++k) {
        b.p[k] = narrow<run, P>(p + k * run / 2);
        if constexpr (!k8) {
            b.m[k] = narrow<run, float>(m + k * run / 2);
            b.v[k] = narrow<run, float>(v + k * run / 2);
        }
    }
}

__device__ __forceinline__ Factors factors(const List& L, int64_t t, float lr, bool minus_u)
{
    Factors f;
    // 1 - beta^t without cancellation: the product is formed in 64 bits, the rest in 32
    const float fix1 = -expm1f((float)((double)t * L.log_b1)), root2 = sqrtf(-expm1f((float)((double)t * L.log_b2)));
    // -lr / (fix1 (sqrt(v) / root2 + eps)) is the reciprocal of a product and a sum, which stay normal
    // numbers; a step below 1e-30, which moves no weight, makes them -sqrt(v) - infinity
    const bool moves = lr > 1e-30f;
    const float by = -fix1 / lr;
    const float den_u = moves ? by / root2 : -1.f;
    f.den_u = both(minus_u ? -den_u : den_u);
    f.den_1 = both(moves ? fminf(by * L.eps, -2.f * FLT_MIN) : -INFINITY);
    f.start = mix64((uint64_t)t * kGamma + L.seed);
    return f;
}

// The block that is last to get here (all have read the count by then) advances it.
__device__ __forceinline__ void count_step(const List& L, int64_t t)
{
    if (!L.last) return;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(L.ticket, 1u) == gridDim.x - 1) {
            *L.ticket = 0;
            *L.steps = t;
        }
    }
}

template <typename P, typename G>
__global__ void __launch_bounds__(kWarps * 32, 2) k_adamw32(const __grid_constant__ List L, float lr,
                                                          const float* __restrict__ lr_device)
{
    using R = Raw<P, G, false>;
    const int lane = threadIdx.x & 31;
    const int64_t t = *L.steps + 1;
    if (lr_device) lr = fmaxf(*lr_device, 0.f);
    Factors f = factors(L, t, lr, false);
    for (int64_t b = blockIdx.x; b < L.tiles; b += gridDim.x) {
        const Rec& r = tensor_of(L, b);
        if (r.guard && has_error(r.guard)) continue;
        f.keep = both(fmaf(-lr, r.decay, 1.f));
        const int64_t blk = (b - r.tile0) * kWarps + (threadIdx.x >> 5);
        const int64_t left = r.size - (blk * kBlk + lane * R::run);
        if (blk * kBlk >= r.size) continue;
        const bool whole = r.wide && (blk + 1) * kBlk <= r.size;
        const Place<P, G, false> at(r, blk, lane);
        R x;
#pragma unroll
        for (int k = 0; k < R::groups; ++k) {
            const int o = k * 32 * R::run;
            if (whole) {
                x.p[k] = *(const Pack<P, R::run>*)(at.p + o);
                x.g[k] = *(const Pack<G, R::run>*)(at.g + o);
                x.m[k] = *(const typename R::Moment*)(at.m + o);
                x.v[k] = *(const typename R::Moment*)(at.v + o);
            } else {
                const int n = (int)max((int64_t)0, min64(R::run, left - o));
                x.p[k] = some_in<R::run, Pack<P, R::run>>(at.p + o, n);
                x.g[k] = some_in<R::run, Pack<G, R::run>>(at.g + o, n);
                x.m[k] = some_in<R::run, typename R::Moment>(at.m + o, n);
                x.v[k] = some_in<R::run, typename R::Moment>(at.v + o, n);
            }
        }
        update<P, G, false>(x, 0, f, L);
        store_block<P, G, false>(at, 0, x, whole, left);
    }
    count_step(L, t);
}

template <int N>
__device__ __forceinline__ void copy_async(void* to, const void* from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "n"(N) : "memory");
}

// blocks of threads on an SM: 800 to 814 us for 403 M values, 814 to 818 with three, 879 with four (64 registers); 12.3, 13.2
// and 14.4 us for 4 M in twelve tensors
constexpr int kFit8 = 2;
constexpr int kStages = 2;   // blocks of a warp: one being computed, the next on its way

// Each thread copies its own values to its own place in shared memory and reads them back, so the
// copies need no barrier, only their own completion.
template <typename P, typename G> struct Stage {
    using R = Raw<P, G, true>;
    Pack<P, R::run> p[R::groups][kWarps * 32];
    Pack<G, R::run> g[R::groups][kWarps * 32];
    typename R::Moment m[R::groups][kWarps * 32], v[R::groups][kWarps * 32];
};

template <typename P, typename G>
__global__ void __launch_bounds__(kWarps * 32, kFit8) k_adamw8(const __grid_constant__ List L, float lr,
                                                          const float* __restrict__ lr_device)
{
    using R = Raw<P, G, true>;
    __shared__ Stage<P, G> st[kStages];
    const int lane = threadIdx.x & 31, me = threadIdx.x;
    const int64_t t = *L.steps + 1;
    if (lr_device) lr = fmaxf(*lr_device, 0.f);
    Factors f = factors(L, t, lr, true);
    for (int64_t b = blockIdx.x; b < L.tiles; b += gridDim.x) {
        const Rec& r = tensor_of(L, b);
        if (r.guard && has_error(r.guard)) continue;
        f.keep = both(fmaf(-lr, r.decay, 1.f));
        const Tile w(r, L, b);
        Place<P, G, true> at(r, w.first, lane);
        // lane j < 16 holds the scale of m of the warp's block j, lane 16 + j that of v
        float* const at_scale = (lane < 16 ? r.ms : r.vs) + w.first + (lane & 15);
        const bool has_scale = (lane & 15) < w.count;
        float scale = has_scale ? *at_scale : 0.f;
        uint64_t random = f.start + (r.quad0 + (uint64_t)((w.first * kBlk + lane * R::run) / 4) + 1) * kGamma;
        auto left = [&](int j) { return r.size - ((w.first + j) * kBlk + lane * R::run); };
        // block j, which is `ahead` blocks behind where `at` stands, to a stage
        auto fetch = [&](int j, int ahead, Stage<P, G>& s) {
            const int far = ahead * kBlk;
            if (j < w.whole) {
#pragma unroll
                for (int k = 0; k < R::groups; ++k) {
                    const int o = far + k * 32 * R::run;
                    copy_async<sizeof(s.p[0][0])>(&s.p[k][me], at.p + o);
                    copy_async<sizeof(s.g[0][0])>(&s.g[k][me], at.g + o);
                    copy_async<sizeof(s.m[0][0])>(&s.m[k][me], at.m + o);
                    copy_async<sizeof(s.v[0][0])>(&s.v[k][me], at.v + o);
                }
            } else if (j < w.count) {
#pragma unroll
                for (int k = 0; k < R::groups; ++k) {
                    const int o = far + k * 32 * R::run;
                    const int n = (int)max((int64_t)0, min64(R::run, left(j) - k * 32 * R::run));
                    s.p[k][me] = some_in<R::run, Pack<P, R::run>>(at.p + o, n);
                    s.g[k][me] = some_in<R::run, Pack<G, R::run>>(at.g + o, n);
                    s.m[k][me] = some_in<R::run, typename R::Moment>(at.m + o, n);
                    s.v[k][me] = some_in<R::run, typename R::Moment>(at.v + o, n);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) fetch(k, k, st[k]);
        for (int j0 = 0; j0 < w.count; j0 += kStages) {
#pragma unroll
            for (int u = 0; u < kStages; ++u) {   // unrolled over the stages, so that their places are constants
                const int j = j0 + u;
                if (j >= w.count) break;
                fetch(j + kStages - 1, u + kStages - 1, st[(u + kStages - 1) % kStages]);
                asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 1) : "memory");
                const Stage<P, G>& s = st[u];
                R x;
#pragma unroll
                for (int k = 0; k < R::groups; ++k) {
                    x.p[k] = s.p[k][me];
                    x.g[k] = s.g[k][me];
                    x.m[k] = s.m[k][me];
                    x.v[k] = s.v[k][me];
                }
                x.ms = __shfl_sync(kFull, scale, j);
                x.vs = __shfl_sync(kFull, scale, 16 + j);
                update<P, G, true>(x, random + (uint64_t)(u * kBlk / 4) * kGamma, f, L);
                store_block<P, G, true>(at, u * kBlk, x, j < w.whole, left(j));
                if ((lane & 15) == j) scale = lane < 16 ? x.ms : x.vs;
            }
            at.next(kStages);
            random += (uint64_t)(kStages * kBlk / 4) * kGamma;
        }
        if (has_scale) *at_scale = scale;
    }
    count_step(L, t);
}

template <typename P, typename G>
cudaError_t launch_step(bool k8, const List& L, int sms, float lr, const float* lr_device, cudaStream_t s)
{
    // Blocks that stay and take tile after tile.  Two on an SM keep enough 32-bit loads on their way, and
    // more of them spread the card's reads: 309 us for the rank-64 cores with three, 285 with two.
    int64_t grid = min64(L.tiles, (int64_t)sms * (k8 ? kFit8 : 2));
    if (grid < 1) grid = 1;
    if (k8) k_adamw8<P, G><<<(unsigned)grid, kWarps * 32, 0, s>>>(L, lr, lr_device);
    else k_adamw32<P, G><<<(unsigned)grid, kWarps * 32, 0, s>>>(L, lr, lr_device);
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

// Whether no two of the buffers that a step writes overlap, and no gradient one of them (false too where there is no
// memory to tell).
static bool apart(int32_t count, const tt_emb_adamw_tensor* tensors, bool k8, const int64_t* steps)
{
    using Span = std::pair<uintptr_t, uintptr_t>;
    try {
        std::vector<Span> spans;
        auto span = [](const void* p, int64_t bytes) { return Span((uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes); };
        spans.push_back(span(steps, sizeof(*steps)));
        for (int32_t i = 0; i < count; ++i) {
            const tt_emb_adamw_tensor& x = tensors[i];
            if (x.size == 0) continue;
            spans.push_back(span(x.param, x.size * type_bytes(x.param_type)));
            spans.push_back(span(x.exp_avg, x.size * (k8 ? 1 : 4)));
            spans.push_back(span(x.exp_avg_sq, x.size * (k8 ? 1 : 4)));
            if (k8) {
                spans.push_back(span(x.m_scale, ceil_div(x.size, kBlk) * 4));
                spans.push_back(span(x.v_scale, ceil_div(x.size, kBlk) * 4));
            }
        }
        std::sort(spans.begin(), spans.end());
        for (size_t i = 1; i < spans.size(); ++i)
            if (spans[i].first < spans[i - 1].second) return false;
        for (int32_t i = 0; i < count; ++i) {
            const tt_emb_adamw_tensor& x = tensors[i];
            if (x.size == 0) continue;
            const Span g = span(x.grad, x.size * type_bytes(x.grad_type));
            // the last span that begins before the gradient ends: the others of those end before that one begins
            const auto after = std::lower_bound(spans.begin(), spans.end(), Span(g.second, 0));
            if (after != spans.begin() && (after - 1)->second > g.first) return false;
        }
        return true;
    } catch (...) {
        return false;
    }
}

extern "C" {

int tt_emb_adamw_create(int32_t count, const tt_emb_adamw_tensor* tensors, const tt_emb_adamw_options* opt,
                        int64_t* steps, tt_emb_adamw_t* out)
{
    if (!out) return TT_ERR_ARG;
    *out = nullptr;
    if (!tensors || !opt || !steps || ((uintptr_t)steps & 7) || count < 1) return TT_ERR_ARG;
    if (!(opt->beta1 >= 0.0 && opt->beta1 < 1.0 && opt->beta2 >= 0.0 && opt->beta2 < 1.0)) return TT_ERR_ARG;
    if (!((float)opt->eps >= FLT_MIN && (float)opt->eps < INFINITY) || opt->reserved != 0) return TT_ERR_ARG;
    if (opt->state_bits != 32 && opt->state_bits != 8) return TT_ERR_ARG;
    const bool k8 = opt->state_bits == 8;
    const int sb = k8 ? 1 : 4;
    for (int32_t i = 0; i < count; ++i) {
        const tt_emb_adamw_tensor& x = tensors[i];
        if (x.size < 0 || x.size > (int64_t)1 << 40 || !type_known(x.param_type) || !type_known(x.grad_type)) return TT_ERR_ARG;
        if (!(x.weight_decay >= 0.0 && (float)x.weight_decay < INFINITY) || ((uintptr_t)x.guard & 3)) return TT_ERR_ARG;
        if (x.size == 0) continue;
        if (!x.param || !x.grad || !x.exp_avg || !x.exp_avg_sq) return TT_ERR_ARG;
        if (((uintptr_t)x.param & (type_bytes(x.param_type) - 1)) || ((uintptr_t)x.grad & (type_bytes(x.grad_type) - 1)))
            return TT_ERR_ARG;
        if ((((uintptr_t)x.exp_avg | (uintptr_t)x.exp_avg_sq) & (sb - 1))) return TT_ERR_ARG;
        if (k8 && (!x.m_scale || !x.v_scale || (((uintptr_t)x.m_scale | (uintptr_t)x.v_scale) & 3))) return TT_ERR_ARG;
    }
    if (!apart(count, tensors, k8, steps)) return TT_ERR_ARG;
    tt_emb_adamw_handle* h = new (std::nothrow) tt_emb_adamw_handle();
    if (!h) return TT_ERR_ARG;
    h->k8 = k8;
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
        cudaMalloc((void**)&h->ticket, 256) != cudaSuccess) {
        delete h;
        return TT_ERR_CUDA;
    }
    // waited for, as the first step may run on a stream that is not ordered behind this one
    if (cudaMemset(h->ticket, 0, 256) != cudaSuccess || cudaStreamSynchronize(0) != cudaSuccess) {
        cudaFree(h->ticket);
        delete h;
        return TT_ERR_CUDA;
    }
    try {
        List base;
        memset(&base, 0, sizeof(base));
        base.log_b1 = log(opt->beta1);   // beta = 0: -inf, and 1 - beta^t = 1
        base.log_b2 = log(opt->beta2);
        auto twice = [](double x) {
            const float f = (float)x;
            uint32_t bits;
            memcpy(&bits, &f, 4);
            return (uint64_t)bits << 32 | bits;
        };
        base.b1 = twice(opt->beta1);
        base.b2 = twice(opt->beta2);
        base.c1 = twice(1.0 - opt->beta1);
        base.c2 = twice(1.0 - opt->beta2);
        base.one = twice(1.0);
        base.minus_b2 = twice(-opt->beta2);
        base.minus_c2 = twice(-(1.0 - opt->beta2));
        base.eps = (float)opt->eps;
        base.seed = opt->seed;
        base.steps = steps;
        base.ticket = h->ticket;
        // In 8 bits, where instructions bound, a warp takes up to 16 blocks of a tensor at a time, which
        // spreads what it does once a tile (800 to 814 us for 403 M values against 879 with 4); fewer where
        // that already gives each tile a block of threads of its own.  In 32 bits, where memory
        // bounds, it takes one, so that the whole card reads neighbouring places (284 us for the 55 M
        // values of the rank-64 cores against 299 with 4 and 303 with 16).
        auto tiles = [&](int per_warp) {
            int64_t t = 0;
            for (int32_t i = 0; i < count; ++i) t += ceil_div(ceil_div(tensors[i].size, kBlk), (int64_t)per_warp * kWarps);
            return t;
        };
        base.per_warp = 1;
        while (k8 && base.per_warp < kPerWarp && tiles(base.per_warp) > (int64_t)h->sms * kFit8) ++base.per_warp;
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
                const uintptr_t at = (uintptr_t)x.param | (uintptr_t)x.grad | (k8 ? 0 : (uintptr_t)x.exp_avg | (uintptr_t)x.exp_avg_sq);
                const uintptr_t at8 = k8 ? (uintptr_t)x.exp_avg | (uintptr_t)x.exp_avg_sq : 0;
                L.r[L.count++] = {x.param, x.grad, x.exp_avg, x.exp_avg_sq, x.m_scale, x.v_scale, x.guard, x.size,
                                  L.tiles, quad, (float)x.weight_decay, (at & 15) == 0 && (at8 & 7) == 0};
                L.tiles += ceil_div(blocks, L.per_warp * kWarps);
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
                return launch_step<P, G>(h->k8, part.list, h->sms, lr, lr_device, s);
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
