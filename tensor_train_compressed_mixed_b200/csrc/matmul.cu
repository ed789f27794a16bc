// C[r][c] = sum over k of A(c, k) B(r, k) on the fifth-generation tensor cores, finished in the same kernel.
//
// The columns of the result are the M side of the tensor cores' tile (128 of them, a lane of tensor memory each) and its
// rows the N side (16 to 256, a column of tensor memory each).  A thread that reads a lane then holds one column of
// C, and the 32 threads of a warp write 32 neighbouring values of a row at a time whatever its stride or alignment; and few
// rows (single tokens) make a narrow tile that reads the large operand once and wastes nothing.
//
// One warp copies tiles of 64 k into a ring of stages (TMA, 128-byte swizzle), one thread issues the products, eight warps read the
// sums.  The sums of `chunk` steps of k are formed in tensor memory, which cuts the last bits off at each step, and those of
// all chunks in fp32 registers; two areas of tensor memory take turns, so that products go on meanwhile.
// Where there are fewer tiles than SMs a cluster of blocks shares one tile's k, and its partial sums are added through
// distributed shared memory in the order of the blocks.
#include <cuda.h>

#include <algorithm>

#include "matmul.cuh"
#include "tcgen05.cuh"

using namespace tt;

namespace {

constexpr int kThreads = 320;        // the copying warp, the issuing warp, eight that finish
constexpr int kDeep = 64;            // k of a stage: 128 bytes, one swizzle row
constexpr int kCols = 128;
constexpr int kGroup = 16;           // row tiles that are taken in turn before the next column tile: they stay in L2
constexpr int kMaxSplit = 8;

struct Args {
    CUtensorMap a, b;
    Epilogue e;
    int32_t* status;
    int64_t rows, cols;
    int32_t its;          // stages of one tile's sum: blocks of k times pairs of terms
    int32_t pairs;
    uint32_t pair_list;   // four bits each: A's term, B's term << 2
    int32_t chunk;        // stages whose sums stay in tensor memory
    uint32_t idesc;
    int32_t tiles_c, tiles_r;
    int32_t split;        // blocks of a cluster that share a tile
};

__host__ __device__ constexpr int stage_bytes(int bn) { return (kCols + bn) * kDeep * 2; }
__host__ __device__ constexpr int stages_of(int bn) { return bn == 256 ? 4 : bn == 128 ? 6 : bn == 64 ? 8 : bn == 32 ? 9 : 10; }

// waits that end early where another role of the block has given up, and tell it where this one does
constexpr int kGone = 1, kTimedOut = 2;
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* gone)
{
    const uint32_t a = smem_u32(bar);
    for (int it = 0; it < kMbarSpin; ++it) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.b32 %0, 1, 0, p;\n\t}"
                     : "=r"(done) : "r"(a), "r"(parity) : "memory");
        if (done) return true;
        if (it >= 64) {
            if (*gone) return false;
            __nanosleep(64);
        }
    }
    *gone = kTimedOut;
    return false;
}
__device__ __forceinline__ void arrive(uint64_t* bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory"); }
__device__ __forceinline__ void expect(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_tile(uint32_t to, const CUtensorMap* map, int x, int y, int part, uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(to), "l"(map), "r"(x), "r"(y), "r"(part), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float peer_value(uint32_t at, int rank)
{
    uint32_t there;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
    return v;
}

// Descriptor of an operand tile with the 128-byte swizzle.  k along the rows of 128 bytes: groups of eight rows 1024 bytes
// apart.  The other way round (mn): blocks of 64 values of m or n by 64 of k, 8192 bytes apart, in each
// groups of eight k 1024 bytes apart.
__device__ __forceinline__ uint64_t swizzled(uint32_t at, bool mn)
{
    return (uint64_t)((at >> 4) & 0x3FFFu) | (uint64_t)(mn ? 8192 >> 4 : 1) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// N columns of the warp's 32 lanes of tensor memory
template <int N>
__device__ __forceinline__ void load_columns(uint32_t at, uint32_t* r)
{
    static_assert(N == 8 || N == 16 || N == 32, "");
    if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(at) : "memory");
    else if constexpr (N == 16)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
                       "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]) : "r"(at) : "memory");
    else {
        load_columns<16>(at, r);
        load_columns<16>(at + 16, r + 16);
    }
}

// The epilogue of 8 or 16 rows of a thread's column.  Types and activation are the same for the whole launch, so each is
// looked at once for all of them.
template <typename T, int N>
__device__ __forceinline__ void load_rows(const void* p, int64_t at, int64_t stride, int n, float (&x)[N])
{
    const T* q = (const T*)p + at;
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = j < n ? to_f32(q[j * stride]) : 0.f;
}
template <typename T, int N>
__device__ __forceinline__ void store_rows(void* p, int64_t at, int64_t stride, int n, const float (&x)[N])
{
    T* q = (T*)p + at;
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < n) q[j * stride] = from_f32<T>(x[j]);
}
template <int N>
__device__ __forceinline__ void store_rows(void* p, int type, int64_t at, int64_t stride, int n, const float (&x)[N])
{
    if (type == TT_BF16) store_rows<__nv_bfloat16>(p, at, stride, n, x);
    else if (type == TT_F16) store_rows<__half>(p, at, stride, n, x);
    else store_rows<float>(p, at, stride, n, x);
}
template <int N>
__device__ __forceinline__ void finish_rows(const Epilogue& e, int64_t r, int64_t c, int n, float bias, float (&z)[N])
{
    if (e.skip_row >= r && e.skip_row < r + n) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (r + j == e.skip_row) z[j] = 0.f;
    }
    float res[N];
    if (e.residual) {
        const int64_t at = r * e.residual_stride + c;
        if (e.residual_type == TT_BF16) load_rows<__nv_bfloat16>(e.residual, at, e.residual_stride, n, res);
        else if (e.residual_type == TT_F16) load_rows<__half>(e.residual, at, e.residual_stride, n, res);
        else load_rows<float>(e.residual, at, e.residual_stride, n, res);
    }
    if (e.bias) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] += bias;
    }
    if (e.pre) store_rows(e.pre, e.pre_type, r * e.pre_stride + c, e.pre_stride, n, z);
    if (e.act == TT_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = activate(TT_ACT_RELU, z[j], 0.f);
    } else if (e.act == TT_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = activate(TT_ACT_GELU, z[j], 0.f);
    } else if (e.act == TT_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = activate(TT_ACT_SILU, z[j], 0.f);
    } else if (e.act == TT_ACT_SOFTCAP) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = activate(TT_ACT_SOFTCAP, z[j], e.cap);
    }
    if (e.residual) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] += res[j];
    }
    store_rows(e.out, e.out_type, r * e.out_stride + c, e.out_stride, n, z);
}

template <int BN, bool kAmn, bool kBmn>
__global__ void __launch_bounds__(kThreads, 1) k_matmul(const __grid_constant__ Args g)
{
    constexpr int kStages = stages_of(BN), kStage = stage_bytes(BN), kHalf = BN / 2;
    constexpr uint32_t kTmem = 2 * BN < 32 ? 32 : 2 * BN;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[kStages], empty[kStages], sums_full[2], sums_empty[2], drained;
    __shared__ uint32_t tmem_at;
    __shared__ volatile int gone;
    const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sums_full[i], 1);
            mbar_init(&sums_empty[i], 8);
        }
        mbar_init(&drained, 1);
        gone = has_error(g.status) ? kGone : 0;
    }
    if (warp == 1) tmem_alloc(&tmem_at, kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    const int split = g.split, rank = (int)blockIdx.x % split;
    const int first = (int)((int64_t)g.its * rank / split), last = (int)((int64_t)g.its * (rank + 1) / split);
    const int step = (int)gridDim.x / split, tiles = gone ? 0 : g.tiles_c * g.tiles_r;
    const int group_tiles = kGroup * g.tiles_c;
    // a tile's place: groups of kGroup row tiles, in each a column tile for all of the group's rows after another
    auto place = [&](int tile, int& c0, int& r0) {
        const int group = tile / group_tiles, in = tile - group * group_tiles;
        const int here = min(kGroup, g.tiles_r - group * kGroup);
        c0 = in / here * kCols;
        r0 = (group * kGroup + in % here) * BN;
    };

    if (warp == 0 && lane == 0) {
        int n = 0;      // stages filled
        bool ok = true;
        for (int tile = blockIdx.x / split; ok && tile < tiles; tile += step) {
            int c0, r0;
            place(tile, c0, r0);
            for (int it = first; it < last; ++it, ++n) {
                const int s = n % kStages;
                if (n >= kStages && !wait_for(&empty[s], (n / kStages - 1) & 1, &gone)) { ok = false; break; }
                const int kb = it / g.pairs;
                const uint32_t pair = g.pair_list >> (4 * (it - kb * g.pairs));
                const int k = kb * kDeep, pa = pair & 3, pb = (pair >> 2) & 3;
                const uint32_t a = ring + s * kStage, b = a + kCols * kDeep * 2;
                expect(&full[s], kStage);
                if constexpr (kAmn) {
#pragma unroll
                    for (int i = 0; i < kCols / 64; ++i) copy_tile(a + i * 8192, &g.a, c0 + 64 * i, k, pa, &full[s]);
                } else {
                    copy_tile(a, &g.a, k, c0, pa, &full[s]);
                }
                if constexpr (kBmn) {
#pragma unroll
                    for (int i = 0; i < BN / 64; ++i) copy_tile(b + i * 8192, &g.b, r0 + 64 * i, k, pb, &full[s]);
                } else {
                    copy_tile(b, &g.b, k, r0, pb, &full[s]);
                }
            }
        }
        if (gone == kTimedOut)      // copies on their way land before the block's memory is given up
            for (int i = max(0, n - kStages); i < n; ++i) mbar_wait(&full[i % kStages], (i / kStages) & 1);
    } else if (warp == 1 && lane == 0) {
        int n = 0, seq = 0;
        bool ok = true;
        for (int tile = blockIdx.x / split; ok && tile < tiles; tile += step)
            for (int c = first; ok && c < last; c += g.chunk, ++seq) {
                const int buf = seq & 1, end = min(c + g.chunk, last);
                if (seq >= 2 && !wait_for(&sums_empty[buf], (seq / 2 - 1) & 1, &gone)) { ok = false; break; }
                tc_fence_after();
                for (int it = c; it < end; ++it, ++n) {
                    const int s = n % kStages;
                    if (!wait_for(&full[s], (n / kStages) & 1, &gone)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a = ring + s * kStage, b = a + kCols * kDeep * 2;
                    uint64_t da = swizzled(a, kAmn), db = swizzled(b, kBmn);
#pragma unroll
                    for (int k = 0; k < kDeep / 16; ++k) {
                        tc_mma_bf16(tmem + buf * BN, da, db, g.idesc, it > c || k > 0);
                        da += (kAmn ? 2048 : 32) >> 4;
                        db += (kBmn ? 2048 : 32) >> 4;
                    }
                    tc_commit(&empty[s]);
                }
                if (ok) tc_commit(&sums_full[buf]);
            }
        if (gone == kTimedOut) {    // products on their way end before tensor memory is given up
            tc_commit(&drained);
            mbar_wait(&drained, 0);
        }
    } else if (warp >= 2) {
        const int quarter = warp & 3, half = (warp - 2) >> 2;     // a warp reaches the lanes of its quarter of tensor memory
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + half * kHalf;
        int seq = 0;
        bool ok = true;
        for (int tile = blockIdx.x / split; ok && tile < tiles; tile += step) {
            int c0, r0;
            place(tile, c0, r0);
            const int64_t col = c0 + quarter * 32 + lane;
            const bool mine = col < g.cols;
            const float bias = mine && g.e.bias ? load_any(g.e.bias, g.e.bias_type, col) : 0.f;
            float acc[kHalf];
            for (int c = first; c < last; c += g.chunk, ++seq) {
                const int buf = seq & 1;
                if (!wait_for(&sums_full[buf], (seq / 2) & 1, &gone)) { ok = false; break; }
                tc_fence_after();
                constexpr int kLoad = kHalf < 32 ? kHalf : kHalf > 64 ? 16 : 32;
#pragma unroll
                for (int j = 0; j < kHalf; j += kLoad) {
                    uint32_t x[kLoad];
                    load_columns<kLoad>(at + buf * BN + j, x);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    if (c == first) {
#pragma unroll
                        for (int i = 0; i < kLoad; ++i) acc[j + i] = __uint_as_float(x[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < kLoad; ++i) acc[j + i] += __uint_as_float(x[i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(&sums_empty[buf]);
            }
            if (!ok) break;
            if (split > 1) {        // the ring is free: every product that read it has ended
                float* part = (float*)(raw + (ring - smem_u32(raw)));
#pragma unroll
                for (int j = 0; j < kHalf; ++j) part[(half * kHalf + j) * kCols + quarter * 32 + lane] = acc[j];
                continue;
            }
            constexpr int kRows = kHalf < 16 || kHalf > 64 ? 8 : 16;
#pragma unroll 1
            for (int j = 0; j < kHalf; j += kRows) {
                const int64_t r = r0 + half * kHalf + j;
                if (r >= g.rows) break;
                float z[kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i) z[i] = acc[i];
                if (mine) finish_rows(g.e, r, col, (int)min64(kRows, g.rows - r), bias, z);
#pragma unroll
                for (int i = 0; i + kRows < kHalf; ++i) acc[i] = acc[i + kRows];      // registers have no index
            }
        }
    }
    __syncwarp();
    if (split > 1) {
        cluster_sync();
        if (warp >= 2 && !gone) {
            int c0, r0;
            place(blockIdx.x / split, c0, r0);
            const int each = BN / split;
            for (int i = threadIdx.x - 64; i < each * kCols; i += kThreads - 64) {
                const int j = rank * each + i / kCols, c = i % kCols;
                if (r0 + j >= g.rows || c0 + c >= g.cols) continue;
                float sum = 0.f;
                for (int s = 0; s < split; ++s) sum += peer_value(ring + (j * kCols + c) * 4, s);
                finish(g.e, r0 + j, c0 + c, sum);
            }
        }
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmem);
    if (threadIdx.x == 0 && gone == kTimedOut) raise_error(g.status, TT_ERR_TIMEOUT, (int)blockIdx.x);
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder()
{
    static const Encode f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (Encode)p;
    }();
    return f;
}

// boxes of 64 values of the inner side by `high` of the outer one
bool encode(CUtensorMap* map, const Operand& o, int high)
{
    const int64_t stride = o.outer == 1 ? (o.inner + 7) / 8 * 8 : o.stride;
    const cuuint64_t dims[3] = {(cuuint64_t)o.inner, (cuuint64_t)o.outer, (cuuint64_t)o.parts};
    const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, (cuuint64_t)(o.parts > 1 ? o.part_stride : stride * o.outer) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)high, 1}, one[3] = {1, 1, 1};
    const Encode f = encoder();
    return f && f(map, o.type == TT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p), dims, strides,
                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool kAmn, bool kBmn>
cudaError_t launch(Args& g, int sms, cudaStream_t s)
{
    constexpr int kBytes = stages_of(BN) * stage_bytes(BN) + 1024;
    auto* kernel = k_matmul<BN, kAmn, kBmn>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = g.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    const int64_t tiles = (int64_t)g.tiles_c * g.tiles_r;
    c.gridDim = dim3((unsigned)(g.split > 1 ? tiles * g.split : min64(tiles, sms)));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = kBytes;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, g);
}

}  // namespace

namespace tt {

int matmul(const Product& p, int32_t* status, int sms, cudaStream_t s)
{
    Args g = {};
    g.e = p.e;
    g.status = status;
    g.rows = p.rows;
    g.cols = p.cols;
    // terms i and j of the operands give a product of 2^-8(i + j) of the first ones: those beyond 2^-16 are below fp32's last bit
    for (int i = 0; i < p.a.parts; ++i)
        for (int j = 0; j < p.b.parts && i + j < 3; ++j) g.pair_list |= (uint32_t)(i | j << 2) << (4 * g.pairs++);
    const int64_t its = ceil_div(p.deep, kDeep) * g.pairs, tiles_c = ceil_div(p.cols, kCols);
    // The tile's height and the blocks that share a tile: what a model of the time likes best.  A stage takes what its
    // products take (half a cycle for each of its rows and 16 k, at 128 columns), or what its bytes take, about 40 a cycle.
    int bn = 0, split = 1;
    double best = 0.0;
    for (int n = p.b_mn ? 64 : 16; n <= 256; n *= 2) {
        const int64_t tiles = tiles_c * ceil_div(p.rows, n);
        const double stage = std::max(2.0 * n, stage_bytes(n) / 40.0);
        for (int k = 1; k <= kMaxSplit; k *= 2) {
            if (k > 1 && (tiles * k > sms || its < 4 * k)) break;
            const double t = (double)ceil_div(tiles * k, sms) * ((double)its / k * stage + 8.0 * n) + 1500.0 + (k > 1 ? 1500.0 : 0.0);
            if (bn == 0 || t < best) best = t, bn = n, split = k;
        }
    }
    const int64_t tiles_r = ceil_div(p.rows, bn);
    if (its > INT32_MAX || tiles_c * tiles_r > INT32_MAX / kMaxSplit) return TT_ERR_ARG;   // sizes that no device holds
    g.its = (int)its;
    // 64 products of 16 k: their sum in tensor memory is cut off at each, by up to 2^-23 of it
    g.chunk = 16;
    g.tiles_c = (int)tiles_c;
    g.tiles_r = (int)tiles_r;
    g.split = split;
    g.idesc = (1u << 4) | (p.a.type == TT_BF16 ? 1u << 7 | 1u << 10 : 0u) | (p.a_mn ? 1u << 15 : 0u) | (p.b_mn ? 1u << 16 : 0u) |
              (uint32_t)(bn >> 3) << 17 | (uint32_t)(kCols >> 4) << 24;
    if (!encode(&g.a, p.a, p.a_mn ? kDeep : kCols) || !encode(&g.b, p.b, p.b_mn ? kDeep : bn)) return TT_ERR_CUDA;
    auto by_height = [&](auto amn, auto bmn) {
        constexpr bool A = decltype(amn)::value, B = decltype(bmn)::value;
        if (bn == 256) return launch<256, A, B>(g, sms, s);
        if (bn == 128) return launch<128, A, B>(g, sms, s);
        if constexpr (!B) {
            if (bn == 16) return launch<16, A, B>(g, sms, s);
            if (bn == 32) return launch<32, A, B>(g, sms, s);
        }
        return launch<64, A, B>(g, sms, s);
    };
    const cudaError_t e = p.b_mn ? by_height(std::true_type(), std::true_type())
                                 : p.a_mn ? by_height(std::true_type(), std::false_type()) : by_height(std::false_type(), std::false_type());
    return e == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // namespace tt
