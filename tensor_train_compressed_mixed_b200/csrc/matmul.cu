// C[r][c] = sum over k of A(c, k) B(r, k) on the fifth-generation tensor cores, finished in the same kernel.
//
// The columns of the result are the M side of the tensor cores' tile (128 of them, a lane of tensor memory each) and its
// rows the N side (16 to 256, a column of tensor memory each), so that few rows (single tokens) make a narrow tile that reads the
// large operand once and wastes nothing.
//
// One warp copies tiles of 64 k into a ring of stages (TMA, 128-byte swizzle), one thread issues the products, sixteen warps take the
// sums from tensor memory through shared memory, 64 rows at a time, where rows lie as they do in the result: a warp
// then works on whole pieces of 128 values of a row, and reads the residual of the next rows ahead.  Two areas of tensor memory
// take turns, so that products go on meanwhile.
// Tensor cores cut the last bits of a sum off at each step.  Short sums of 16-bit results round far above that; for others (kLong) the
// sums of some blocks of k at a time are formed in tensor memory and added in fp32 registers.  Operands of several terms
// (x = t0 + t1 + t2, each 2^-8 of the one before) bring each term once for all products that it is part of: those of terms i and j
// with i + j < 3, as the others are below fp32's last bit.  All but the first terms' product are summed in an area of their
// own, so that few steps are made on a large sum.
//
// What bounds it.  Many k: the tensor cores and the power limit (4096 x 32000 x 4096 bf16: 1.58 PFLOP/s cold, 1.38 in a row,
// as the library's product).  Copies and products are issued by an elected thread: behind a comparison of the thread's number the
// same instructions took 763 us where they now take 680.  Few k: the finishing, whose instructions fill half of the issue slots
// (8192 x 4096 x 128 fp16 with gelu, residual and pre: 73 us, 60 without gelu, 31 for the bytes).  Few rows: memory (8 rows of
// 32000 x 4096 bf16: 50 us, 5.3 TB/s).
//
// Two blocks on neighbouring SMs make a pair where there are many tiles: one tile of 256 columns, of which each block brings its half of
// both operands and finishes its half, so that a block reads half of B.
// Where there are fewer tiles than SMs a cluster of blocks shares one tile's k, and its partial sums are added through
// distributed shared memory in the order of the blocks.  Where there are so few tiles and so many k that clusters leave most SMs
// idle, k is cut into slices whose sums go to the workspace; a second kernel adds them in their order and finishes them.
#include <cuda.h>

#include <math.h>

#include <algorithm>
#include <atomic>

#include "matmul.cuh"
#include "tcgen05.cuh"

using namespace tt;

namespace {

// Blocks of 64 k whose sum is formed in tensor memory, before it is added in fp32 registers.  Each block is four steps, and a step
// cuts off up to 2^-22 of the sum, always towards zero (measured on terms of one sign: 2^-23.3 of a growing sum, 2^-22.2 of one that is large
// from the start).  Results of fp32: with 16 blocks the gradients of 301 x 5003 x 257 were off by 1.2e-6 of their norm, with 4 by
// 2.5e-7 (fp32 products: 4.9e-7).  16-bit results: an eighth of half a step at most, 2^-14 for fp16 and 2^-11 for bf16.  Whole sums of
// 32768 terms of one sign were off by up to 3.9e-4 beyond their rounding, more than half a step of fp16, and of 65536 by 7.7e-4.
constexpr int kChunk = 4, kChunkF16 = 64, kChunkBf16 = 512;
constexpr int kDeep = 64;            // k of a stage: 128 bytes, one swizzle row
constexpr int kCols = 128;
constexpr double kMostSums = 1 << 26;      // of all slices together
// Row tiles that are taken in turn before the next column tile, so that they stay in L2 (4096 x 32000 x 4096 bf16: 671 us, 736 with
// 4 of them and 880 with one).
constexpr int kGroup = 16;

struct Args {
    CUtensorMap a, b;
    Epilogue e;
    int32_t* status;
    int64_t rows, cols;
    int32_t blocks;       // of 64 k
    int32_t chunk;        // of them, with kLong: those whose sum is formed in tensor memory
    int32_t a_terms, b_terms;     // of the operands' values, 1 to 3; with kLong only
    uint32_t idesc;
    int32_t tiles_c, tiles_r;
    int32_t split;        // blocks of a cluster that share a tile
    int32_t slices;       // of k, each a tile of its own whose sums go to rows of their own
    int32_t fail;         // TT_INJECT_COPIES, _PRODUCTS or _SUMS (tests): the role that gives up after its first chunk
    int32_t vectors;      // four neighbouring values of a row of the result, residual and pre make one access
};

// A tile's height bn, and whether a pair of blocks shares a tile: warps that finish, bytes of a stage (the block's own columns of
// A, its rows of B), stages of the ring, rows on their way through shared memory, blocks on an SM.
__host__ __device__ constexpr int finish_of(int bn) { return bn <= 32 ? 4 : 16; }
__host__ __device__ constexpr int threads_of(int bn) { return 64 + 32 * finish_of(bn); }
__host__ __device__ constexpr int stage_bytes(int bn, bool pair) { return (kCols + (pair ? bn / 2 : bn)) * kDeep * 2; }
__host__ __device__ constexpr int stages_of(int bn, bool pair) { return bn == 256 ? (pair ? 6 : 4) : bn == 128 ? (pair ? 8 : 6) : bn == 64 ? 8 : 5; }
__host__ __device__ constexpr int passing_of(int bn) { return bn <= 32 ? 16 : 64; }
__host__ __device__ constexpr int fit_of(int bn) { return bn <= 32 ? 2 : 1; }

// waits that end early where another role of the block has given up, and tell it where this one does
constexpr int kGone = 1, kTimedOut = 2;
constexpr int kTries = 1 << 18;      // of a wait: about a second
template <bool kCluster = false>      // whether other blocks of the cluster arrive there
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* gone)
{
    const uint32_t a = smem_u32(bar);
    for (int it = 0; it < kTries; ++it) {
        uint32_t done;
        if constexpr (kCluster)
            asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.b32 %0, 1, 0, p;\n\t}"
                         : "=r"(done) : "r"(a), "r"(parity) : "memory");
        else
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
// bar: shared-memory address; of a pair's, that of the first block's barrier
template <bool kPair>
__device__ __forceinline__ void copy_tile(uint32_t to, const CUtensorMap* map, int x, int y, int part, uint32_t bar)
{
    if constexpr (kPair)
        asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                     ::"r"(to), "l"(map), "r"(x), "r"(y), "r"(part), "r"(bar) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                     ::"r"(to), "l"(map), "r"(x), "r"(y), "r"(part), "r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t in_block(uint32_t at, int rank)      // the same place in another block of the cluster
{
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
    return there;
}
__device__ __forceinline__ void arrive_at_first(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_block(smem_u32(bar), 0)) : "memory");
}
// the pair's products: operands' halves and the accumulators' in both blocks at the same places
template <bool kPair>
__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (kPair)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
    else
        tc_mma_bf16(d, a, b, idesc, accumulate);
}
// arrives at the barrier, of a pair's at those of both blocks, when all products issued so far have ended
template <bool kPair>
__device__ __forceinline__ void commit(uint64_t* bar)
{
    if constexpr (kPair)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
    else
        tc_commit(bar);
}
// One thread of a warp, told so that the compiler knows that what it guards runs in one: it keeps descriptors in the
// warp's own registers then.
__device__ __forceinline__ bool elected()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a row's sums from another block's shared memory, as row_sums takes them
__device__ __forceinline__ void peer_four(uint32_t row, int rank, bool vectors, int lane, F2 (&z)[2])
{
    const uint32_t there = in_block(row, rank);
    float x[4];
    if (vectors) {
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(there + lane * 16) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x[i]) : "r"(there + (lane + 32 * i) * 4) : "memory");
    }
    z[0] = {x[0], x[1]};
    z[1] = {x[2], x[3]};
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
    static_assert(N == 4 || N == 8 || N == 16, "");
    if constexpr (N == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
    else if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(at) : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
                       "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]) : "r"(at) : "memory");
}

// Four values of a row as a thread holds them: neighbours where they make one access (kVec; two words hold four 16-bit
// values), else those 32 apart, so that a warp's accesses are of neighbouring places either way.
struct Four { uint32_t w[4]; };

// A thread's place in the result's rows: its first column, how many of its four values are in the matrix, the bias of each.
struct Lane {
    int64_t c;
    int n;
    bool vectors;
    F2 bias[2];
    __device__ __forceinline__ Lane(const Epilogue& e, int64_t c0, int64_t cols, bool v, int lane)
    {
        vectors = v;
        c = c0 + (v ? 4 * lane : lane);
        n = 0;
        float b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at = c + (v ? i : 32 * i);
            n += at < cols;
            b[i] = at < cols && e.bias ? load_any(e.bias, e.bias_type, at) : 0.f;
        }
        bias[0] = {b[0], b[1]};
        bias[1] = {b[2], b[3]};
    }
};
// a row's sums from shared memory
__device__ __forceinline__ void row_sums(const float* row, bool vectors, int lane, F2 (&z)[2])
{
    if (vectors) {
        const float4 q = *(const float4*)(row + 4 * lane);
        z[0] = {q.x, q.y};
        z[1] = {q.z, q.w};
    } else {
        z[0] = {row[lane], row[lane + 32]};
        z[1] = {row[lane + 64], row[lane + 96]};
    }
}
template <typename T>
__device__ __forceinline__ uint32_t packed(F2 x)      // two 16-bit values
{
    uint32_t r;
    if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(x.x, x.y);
        memcpy(&r, &h, 4);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
        memcpy(&r, &h, 4);
    }
    return r;
}
template <typename T>
__device__ __forceinline__ F2 unpacked(uint32_t w)
{
    if constexpr (std::is_same_v<T, __half>) {
        __half2 h;
        memcpy(&h, &w, 4);
        const float2 f = __half22float2(h);
        return {f.x, f.y};
    }
    return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
}
template <typename T, bool kVec, int R>
__device__ __forceinline__ void store_rows(T* p, int64_t stride, int n, int rows, const F2 (&z)[R][2])
{
#pragma unroll
    for (int j = 0; j < R; ++j, p += stride) {
        if (j >= rows) break;
        if constexpr (!kVec) {
            const float x[4] = {z[j][0].x, z[j][0].y, z[j][1].x, z[j][1].y};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) p[32 * i] = from_f32<T>(x[i]);
        } else if constexpr (sizeof(T) == 4) {
            *(float4*)p = make_float4(z[j][0].x, z[j][0].y, z[j][1].x, z[j][1].y);
        } else {
            *(uint2*)p = make_uint2(packed<T>(z[j][0]), packed<T>(z[j][1]));
        }
    }
}
template <bool kVec, int R>
__device__ __forceinline__ void store_rows(void* p, int type, int64_t at, int64_t stride, int n, int rows, const F2 (&z)[R][2])
{
    if (type == TT_BF16) store_rows<__nv_bfloat16, kVec>((__nv_bfloat16*)p + at, stride, n, rows, z);
    else if (type == TT_F16) store_rows<__half, kVec>((__half*)p + at, stride, n, rows, z);
    else store_rows<float, kVec>((float*)p + at, stride, n, rows, z);
}
// the residual of up to R rows, and what it adds
template <typename T, bool kVec, int R>
__device__ __forceinline__ void fetch_rows(const T* p, int64_t stride, int n, int rows, Four (&res)[R])
{
#pragma unroll
    for (int j = 0; j < R; ++j, p += stride) {
        if (j >= rows) break;
        if constexpr (!kVec) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) res[j].w[i] = p[32 * i];
        } else if constexpr (sizeof(T) == 4) {
            const uint4 q = *(const uint4*)p;
            res[j] = {{q.x, q.y, q.z, q.w}};
        } else {
            const uint2 q = *(const uint2*)p;
            res[j].w[0] = q.x;
            res[j].w[1] = q.y;
        }
    }
}
template <int R>
__device__ __forceinline__ void fetch_rows(const Epilogue& e, const Lane& l, int64_t r, int rows, Four (&res)[R])
{
    if (!e.residual || l.n == 0) return;
    const int64_t at = r * e.residual_stride + l.c;
    if (e.residual_type == TT_F32) {
        const uint32_t* p = (const uint32_t*)e.residual + at;
        l.vectors ? fetch_rows<uint32_t, true>(p, e.residual_stride, l.n, rows, res) : fetch_rows<uint32_t, false>(p, e.residual_stride, l.n, rows, res);
    } else {
        const uint16_t* p = (const uint16_t*)e.residual + at;
        l.vectors ? fetch_rows<uint16_t, true>(p, e.residual_stride, l.n, rows, res) : fetch_rows<uint16_t, false>(p, e.residual_stride, l.n, rows, res);
    }
}
template <typename T, bool kVec, int R>
__device__ __forceinline__ void add_rows(const Four (&res)[R], F2 (&z)[R][2])
{
#pragma unroll
    for (int j = 0; j < R; ++j) {
        const uint32_t(&w)[4] = res[j].w;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            F2 x = {};
            if constexpr (sizeof(T) == 4) x = {__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])};
            else if constexpr (kVec) x = unpacked<T>(w[i]);
            else x = unpacked<T>(__byte_perm(w[2 * i], w[2 * i + 1], 0x5410));
            z[j][i] = add2(z[j][i], x);
        }
    }
}
// Up to R rows finished from their sums.  Types and activation are the same for the whole launch: each is looked at once
// for all of them.
template <int R, bool kCoarse, bool kVec>
__device__ __forceinline__ void finish_rows(const Epilogue& e, const Lane& l, int r, int rows, F2 (&z)[R][2], const Four (&res)[R])
{
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) z[j][i] = add2(z[j][i], l.bias[i]);
    if (e.pre) store_rows<kVec>(e.pre, e.pre_type, r * e.pre_stride + l.c, e.pre_stride, l.n, rows, z);
    auto all = [&](auto act) {
        constexpr int kAct = decltype(act)::value;
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (kCoarse) z[j][i] = {activate_coarse(kAct, z[j][i].x, e.cap), activate_coarse(kAct, z[j][i].y, e.cap)};
                else z[j][i] = activate(kAct, z[j][i], e.cap);
            }
    };
    if (e.act == TT_ACT_RELU) all(std::integral_constant<int, TT_ACT_RELU>());
    else if (e.act == TT_ACT_GELU) all(std::integral_constant<int, TT_ACT_GELU>());
    else if (e.act == TT_ACT_SILU) all(std::integral_constant<int, TT_ACT_SILU>());
    else if (e.act == TT_ACT_SOFTCAP) all(std::integral_constant<int, TT_ACT_SOFTCAP>());
    if (e.residual) {
        if (e.residual_type == TT_BF16) add_rows<__nv_bfloat16, kVec>(res, z);
        else if (e.residual_type == TT_F16) add_rows<__half, kVec>(res, z);
        else add_rows<float, kVec>(res, z);
    }
    store_rows<kVec>(e.out, e.out_type, r * e.out_stride + l.c, e.out_stride, l.n, rows, z);
}
template <int R, bool kCoarse>
__device__ __forceinline__ void finish_rows(const Epilogue& e, const Lane& l, int r, int rows, F2 (&z)[R][2], const Four (&res)[R])
{
    const int skip = (int)e.skip_row - r;        // (rows are below 2^31)
    if (skip >= 0 && skip < rows) {
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (j == skip) z[j][0] = z[j][1] = both(0.f);
    }
    if (l.n == 0) return;
    if (l.vectors) finish_rows<R, kCoarse, true>(e, l, r, rows, z, res);
    else finish_rows<R, kCoarse, false>(e, l, r, rows, z, res);
}

// Barriers of the four warps that finish the same part of a tile; the first tells whether all of them say yes.
__device__ __forceinline__ bool all_agree(int part, bool yes)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %2, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"((uint32_t)yes), "r"(1 + part) : "memory");
    return r != 0;
}
__device__ __forceinline__ void part_sync(int part) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + part) : "memory"); }

// Tiles of less than kHigh rows take kTermChunks for single terms too: memory bounds them.  Higher ones are bound by the thread that issues the products, which the loops over terms delay
// (2048 rows by 32000 x 1024 fp16, x's gradient: 119 us so, 167 by the loops over terms).  The highest spill some sums, which costs
// 5 us a tile (4096 rows by 32000 x 4096 fp16: 815 us, 795 as whole sums).
constexpr int kHigh = 128;
template <int BN, bool kAmn, bool kBmn, int kSums, bool kPair>
__global__ void __launch_bounds__(threads_of(BN), fit_of(BN)) k_matmul(const __grid_constant__ Args g)
{
    constexpr int kFinish = finish_of(BN), kStages = stages_of(BN, kPair), kStage = stage_bytes(BN, kPair), kPart = BN / (kFinish / 4);
    constexpr int kPass = passing_of(BN), kRows = kPass / kFinish;       // rows at a time of a block and of a finishing warp
    constexpr bool kLong = kSums != kWhole, kTerms = kSums == kTermChunks;
    constexpr int kSide = kPair ? 2 : 1, kOwn = BN / kSide;              // blocks of a pair, rows of B that each brings
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[kStages], empty[kStages], sums_full[2], sums_empty[2], drained;
    __shared__ uint32_t tmem_at;
    __shared__ volatile int gone;
    const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u;
    const int terms = kTerms ? max(g.a_terms, g.b_terms) : 1;
    const uint32_t area = terms > 1 ? 4 * BN : 2 * BN, columns = area < 32 ? 32 : area;      // of tensor memory: two of sums, and two of the small terms'
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sums_full[i], 1);
            mbar_init(&sums_empty[i], kFinish * kSide);
        }
        mbar_init(&drained, 1);
        asm volatile("prefetch.tensormap [%0];" ::"l"(&g.a) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&g.b) : "memory");
    }
    let_next_kernel_start();
    if (warp == 1) {
        if constexpr (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_at)), "r"(columns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            tmem_alloc(&tmem_at, columns);
        }
    }
    wait_for_kernel_before();
    if (threadIdx.x == 0) gone = has_error(g.status) ? kGone : 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    // blocks that share a tile: a pair halves its columns, others its k
    const int split = kPair ? 1 : g.split, share = kPair ? 2 : split, rank = (int)blockIdx.x % share;
    int skip = gone;
    if constexpr (kPair) {      // either both work or none
        cluster_sync();
        uint32_t other;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(other) : "r"(in_block(smem_u32((const void*)&gone), rank ^ 1)) : "memory");
        skip |= (int)other;
    }
    const int start = blockIdx.x / share, step = (int)gridDim.x / share, slices = kPair ? 1 : g.slices;
    const int tiles = skip ? 0 : g.tiles_c * g.tiles_r * slices;
    const int group_tiles = kGroup * g.tiles_c;
    // A tile's place: groups of kGroup row tiles, in each a column tile for all of the group's rows after another; and its k.
    struct Tile { int c0, r0, first, last, shift; };
    auto place = [&](int tile) {
        Tile t;
        const int slice = slices > 1 ? tile % slices : 0, at = slices > 1 ? tile / slices : tile;
        const int group = at / group_tiles, in = at - group * group_tiles;
        const int here = min(kGroup, g.tiles_r - group * kGroup);
        t.c0 = in / here * (kCols * kSide) + (kPair ? rank * kCols : 0);
        t.r0 = (group * kGroup + in % here) * BN;
        const int of = slices > 1 ? slices : split, which = slices > 1 ? slice : kPair ? 0 : rank;
        t.first = (int)((int64_t)g.blocks * which / of);
        t.last = (int)((int64_t)g.blocks * (which + 1) / of);
        t.shift = slice * (int)g.rows;
        return t;
    };

    const int chunk = kLong ? g.chunk : g.blocks;      // blocks of k whose sums stay in tensor memory
    if (warp == 0 && elected()) {
        int n = 0;      // stages filled
        bool ok = true;
        for (int tile = start; ok && tile < tiles; tile += step) {
            const Tile at = place(tile);
            const int c0 = at.c0, rb = at.r0 + (kPair ? rank * kOwn : 0);
            for (int k0 = at.first; ok && k0 < at.last; k0 += chunk) {
                const int end = min(k0 + chunk, at.last);
                for (int kb = k0; ok && kb < end; ++kb)
                    for (int t = 0; t < terms; ++t, ++n) {
                        const int s = n % kStages, k = kb * kDeep;
                        if (n >= kStages && !wait_for(&empty[s], (n / kStages - 1) & 1, &gone)) { ok = false; break; }
                        const uint32_t a = ring + s * kStage, b = a + kCols * kDeep * 2, bar = kPair ? in_block(smem_u32(&full[s]), 0) : smem_u32(&full[s]);
                        const bool with_a = !kTerms || t < g.a_terms, with_b = !kTerms || t < g.b_terms;
                        if (!kPair || rank == 0) expect(&full[s], ((with_a ? kCols : 0) + (with_b ? kOwn : 0)) * kDeep * 2 * kSide);
                        if (with_a) {
                            if constexpr (kAmn) {
#pragma unroll
                                for (int i = 0; i < kCols / 64; ++i) copy_tile<kPair>(a + i * 8192, &g.a, c0 + 64 * i, k, t, bar);
                            } else {
                                copy_tile<kPair>(a, &g.a, k, c0, t, bar);
                            }
                        }
                        if (with_b) {
                            if constexpr (kBmn) {
#pragma unroll
                                for (int i = 0; i < kOwn / 64; ++i) copy_tile<kPair>(b + i * 8192, &g.b, rb + 64 * i, k, t, bar);
                            } else {
                                copy_tile<kPair>(b, &g.b, k, rb, t, bar);
                            }
                        }
                    }
                if (g.fail == TT_INJECT_COPIES) gone = kTimedOut, ok = false;
            }
        }
        // All copies have landed before the block's memory is given up, also where another role gives up after the last of them was
        // asked for.  (A pair's arrive at the first block's barriers.)
        if (!kPair || rank == 0)
            for (int i = max(0, n - kStages); i < n; ++i)
                if (!mbar_wait(&full[i % kStages], (i / kStages) & 1, kTries)) break;
    } else if (warp == 1 && (!kPair || rank == 0) && elected()) {
        int n = 0, seq = 0;
        bool ok = true;
        for (int tile = start; ok && tile < tiles; tile += step) {
            const Tile at = place(tile);
            for (int k0 = at.first; ok && k0 < at.last; k0 += chunk, ++seq) {
                const int buf = seq & 1, end = min(k0 + chunk, at.last);
                if (seq >= 2 && !wait_for<kPair>(&sums_empty[buf], (seq / 2 - 1) & 1, &gone)) { ok = false; break; }
                tc_fence_after();
                const uint32_t sums = tmem + buf * BN;
                auto product = [&](uint32_t to, int a_slot, int b_slot, bool add) {
                    uint64_t da = swizzled(ring + a_slot * kStage, kAmn), db = swizzled(ring + b_slot * kStage + kCols * kDeep * 2, kBmn);
#pragma unroll
                    for (int k = 0; k < kDeep / 16; ++k) {
                        multiply<kPair>(to, da, db, g.idesc, add || k > 0);
                        da += (kAmn ? 2048 : 32) >> 4;
                        db += (kBmn ? 2048 : 32) >> 4;
                    }
                };
                if (!kTerms || terms == 1) {
                    for (int kb = k0; kb < end; ++kb, ++n) {
                        const int s = n % kStages;
                        if (!wait_for(&full[s], (n / kStages) & 1, &gone)) { ok = false; break; }
                        tc_fence_after();
                        product(sums, s, s, kb > k0);
                        commit<kPair>(&empty[s]);
                    }
                } else {
                    for (int kb = k0; ok && kb < end; ++kb, n += terms) {
                        int slot[3];
#pragma unroll
                        for (int t = 0; t < 3; ++t) slot[t] = (n + t) % kStages;
                        bool small = kb > k0;       // the small terms' sum has begun
#pragma unroll
                        for (int t = 0; t < 3; ++t) {
                            if (t >= terms) break;
                            if (!wait_for(&full[slot[t]], ((n + t) / kStages) & 1, &gone)) { ok = false; break; }
                            tc_fence_after();
                            if (t == 0) product(sums, slot[0], slot[0], kb > k0);
                            // the products whose later term is this one
#pragma unroll
                            for (int i = 0; i <= t; ++i)
#pragma unroll
                                for (int j = 0; j <= t; ++j)
                                    if ((i == t || j == t) && i + j > 0 && i + j < 3 && i < g.a_terms && j < g.b_terms) {
                                        product(sums + 2 * BN, slot[i], slot[j], small);
                                        small = true;
                                    }
                        }
#pragma unroll
                        for (int t = 0; t < 3; ++t)
                            if (ok && t < terms) commit<kPair>(&empty[slot[t]]);
                    }
                }
                if (g.fail == TT_INJECT_PRODUCTS) gone = kTimedOut, ok = false;
                if (ok) commit<kPair>(&sums_full[buf]);
            }
        }
        if (gone == kTimedOut) {    // products on their way end before tensor memory is given up
            commit<kPair>(&drained);
            mbar_wait(&drained, 0, kTries);
        }
    } else if (warp >= 2) {
        const int quarter = warp & 3, part = kFinish == 4 ? 0 : (warp - 2) >> 2;     // a warp reaches the lanes of its quarter of tensor memory
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + part * kPart;
        float* const passing = (float*)(raw + (ring - smem_u32(raw)) + kStages * kStage);
        constexpr int kLoad = kPass / (kFinish / 4);              // rows that a warp takes from tensor memory at a time
        const int mine = (warp - 2) * kRows;                      // the first of the passing rows that this warp finishes
        const int height = (int)g.rows;
        int seq = 0;
        for (int tile = start; tile < tiles; tile += step) {
            const Tile at = place(tile);
            const int first = at.first, last = at.last;
            const Lane l(g.e, at.c0, g.cols, g.vectors, lane);
            // each part of the tile gives kLoad of the passing rows in turn
            const int row = at.r0 + mine / kLoad * kPart + mine % kLoad;
            Four res[kRows];
            if (split == 1) fetch_rows(g.e, l, row, min(kRows, height - row), res);
            float acc[kLong ? kPart : 1];
            bool ok = true;
            int buf = 0;
            if constexpr (kLong) {
                for (int k0 = first; ok && k0 < last; k0 += chunk, ++seq) {
                    buf = seq & 1;
                    ok = wait_for(&sums_full[buf], (seq / 2) & 1, &gone);
                    if (g.fail == TT_INJECT_SUMS) gone = kTimedOut, ok = false;
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < kPart; j += kLoad) {
                        uint32_t x[kLoad];
                        load_columns<kLoad>(lanes + buf * BN + j, x);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                        for (int i = 0; i < kLoad; ++i) acc[j + i] = (k0 == first ? 0.f : acc[j + i]) + __uint_as_float(x[i]);
                        if (kTerms && terms > 1) {
                            load_columns<kLoad>(lanes + 2 * BN + buf * BN + j, x);
                            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                            for (int i = 0; i < kLoad; ++i) acc[j + i] += __uint_as_float(x[i]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) kPair ? arrive_at_first(&sums_empty[buf]) : arrive(&sums_empty[buf]);
                }
            } else {
                buf = seq & 1;
                ok = wait_for(&sums_full[buf], (seq / 2) & 1, &gone);
                if (g.fail == TT_INJECT_SUMS) gone = kTimedOut, ok = false;
                tc_fence_after();
                ++seq;
            }
            // all four warps give up, or none: the barriers below want all
            if (!all_agree(part, ok)) break;
            // of a shared tile all sums go to the ring, which is free: every product that read it has ended
            float* const to = split > 1 ? (float*)(raw + (ring - smem_u32(raw))) + part * kPart * kCols : passing + part * kLoad * kCols;
#pragma unroll 1
            for (int j = 0; j < kPart; j += kLoad) {
                uint32_t x[kLoad];
                if constexpr (kLong) {
#pragma unroll
                    for (int i = 0; i < kLoad; ++i) x[i] = __float_as_uint(acc[i]);
#pragma unroll
                    for (int i = 0; i + kLoad < kPart; ++i) acc[i] = acc[i + kLoad];      // registers have no index
                } else {
                    load_columns<kLoad>(lanes + buf * BN + j, x);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    if (j + kLoad == kPart) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) kPair ? arrive_at_first(&sums_empty[buf]) : arrive(&sums_empty[buf]);
                    }
                }
                if (split > 1) {
#pragma unroll
                    for (int i = 0; i < kLoad; ++i) to[(j + i) * kCols + quarter * 32 + lane] = __uint_as_float(x[i]);
                    continue;
                }
                if (j > 0) part_sync(part);        // the rows before have been read
#pragma unroll
                for (int i = 0; i < kLoad; ++i) to[i * kCols + quarter * 32 + lane] = __uint_as_float(x[i]);
                part_sync(part);
                const int r = row + j, rows = min(kRows, height - r);
                F2 z[kRows][2];
#pragma unroll
                for (int i = 0; i < kRows; ++i) row_sums(passing + (mine + i) * kCols, l.vectors, lane, z[i]);
                finish_rows<kRows, !kLong>(g.e, l, r + at.shift, rows, z, res);
                if (j + kLoad < kPart) fetch_rows(g.e, l, r + kLoad, min(kRows, height - r - kLoad), res);
            }
        }
    }
    __syncwarp();
    if (split > 1) {
        cluster_sync();
        if (warp >= 2 && !skip && !gone) {
            const Tile at = place(start);
            const Lane l(g.e, at.c0, g.cols, g.vectors, lane);
            // eight pieces of rows on their way to a warp, of all blocks of the cluster
            auto join = [&](auto of) {
                constexpr int kBlocks = decltype(of)::value, kBatch = 8 / kBlocks, kEach = BN / kBlocks;
#pragma unroll 1
                for (int j = (warp - 2) * kBatch; j < kEach; j += kFinish * kBatch) {
                    const int r = at.r0 + rank * kEach + j, rows = max(0, min(min(kBatch, kEach - j), (int)g.rows - r));
                    Four res[kBatch];
                    fetch_rows(g.e, l, r, rows, res);
                    F2 x[kBatch][kBlocks][2], z[kBatch][2];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
#pragma unroll
                        for (int s = 0; s < kBlocks; ++s) peer_four(ring + ((rank * kEach + j + (i < rows ? i : 0)) * kCols) * 4, s, l.vectors, lane, x[i][s]);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            z[i][h] = x[i][0][h];
#pragma unroll
                            for (int s = 1; s < kBlocks; ++s) z[i][h] = add2(z[i][h], x[i][s][h]);
                        }
                    finish_rows<kBatch, !kLong>(g.e, l, r, rows, z, res);
                }
            };
            if (split == 2) join(std::integral_constant<int, 2>());
            else if (split == 4) join(std::integral_constant<int, 4>());
            else join(std::integral_constant<int, 8>());
        }
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) cluster_sync();       // neither block's memory is given up while the other's products may read it
    tc_fence_after();
    if (warp == 1) {
        if constexpr (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
        else tmem_dealloc(tmem, columns);
    }
    if (threadIdx.x == 0 && gone == kTimedOut) raise_error(g.status, TT_ERR_TIMEOUT, (int)blockIdx.x);
}

// The slices' sums added in their order and finished: 32 columns of a row of a block of threads, each warp an eighth of the slices.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) k_join(const float* sums, int slices, int64_t rows, int64_t cols, const __grid_constant__ Epilogue e,
                                                       const int32_t* status)
{
    wait_for_kernel_before();
    if (has_error(status)) return;
    __shared__ float part[kJoinThreads / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t across = ceil_div(cols, 32), r = blockIdx.x / across, c = blockIdx.x % across * 32 + lane;
    float sum = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int i = warp; i < slices; i += kJoinThreads / 32) sum += sums[(i * rows + r) * cols + c];
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp > 0 || c >= cols) return;
#pragma unroll
    for (int i = 1; i < kJoinThreads / 32; ++i) sum += part[i][lane];
    float z = r == e.skip_row ? 0.f : sum;
    if (e.bias) z += load_any(e.bias, e.bias_type, c);
    if (e.pre) store_any(e.pre, e.pre_type, r * e.pre_stride + c, z);
    float y = activate(e.act, F2{z, z}, e.cap).x;
    if (e.residual) y += load_any(e.residual, e.residual_type, r * e.residual_stride + c);
    store_any(e.out, e.out_type, r * e.out_stride + c, y);
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

template <int BN, bool kPair>
constexpr int block_bytes() { return stages_of(BN, kPair) * stage_bytes(BN, kPair) + passing_of(BN) * kCols * 4 + 1024; }

// A launch of `blocks` blocks in clusters of `cluster`.
struct Launch {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[2];
    Launch(int64_t blocks, int threads, int bytes, int cluster, bool early, cudaStream_t s)
    {
        int n = 0;
        if (cluster > 1) {
            at[n].id = cudaLaunchAttributeClusterDimension;
            at[n].val.clusterDim.x = cluster;
            at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
            ++n;
        }
        if (early) {
            at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[n].val.programmaticStreamSerializationAllowed = 1;
            ++n;
        }
        c.gridDim = dim3((unsigned)blocks);
        c.blockDim = dim3(threads);
        c.dynamicSmemBytes = bytes;
        c.stream = s;
        c.attrs = at;
        c.numAttrs = n;
    }
    Launch(const Launch&) = delete;
};

// leave for its shared memory, once for each device
template <typename Kernel>
cudaError_t allow(Kernel kernel, int bytes, std::atomic<uint64_t>& told)
{
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e == cudaSuccess && (device >= 64 || !(told.load(std::memory_order_relaxed) >> device & 1))) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess && device < 64) told.fetch_or((uint64_t)1 << device, std::memory_order_relaxed);
    }
    return e;
}

template <int BN, bool kAmn, bool kBmn, int kSums, bool kPair>
cudaError_t launch(Args& g, const MatmulFits& fits, bool early, cudaStream_t s)
{
    static std::atomic<uint64_t> told{0};
    auto* kernel = k_matmul<BN, kAmn, kBmn, kSums, kPair>;
    const cudaError_t e = allow(kernel, block_bytes<BN, kPair>(), told);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)g.tiles_c * g.tiles_r * g.slices;
    const int64_t blocks = kPair ? 2 * min64(tiles, fits.one[1]) : g.split > 1 ? tiles * g.split : min64(tiles, (int64_t)fits.sms * fit_of(BN));
    const Launch l(blocks, threads_of(BN), block_bytes<BN, kPair>(), kPair ? 2 : g.split, early, s);
    return cudaLaunchKernelEx(&l.c, kernel, g);
}

// clusters of 2, 4 and 8 blocks of a kernel that the current device holds at a time
template <int BN, bool kPair>
void count_clusters(int (&n)[4])
{
    auto* kernel = k_matmul<BN, false, false, kWhole, kPair>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, block_bytes<BN, kPair>()) != cudaSuccess) return;
    for (int i = 1; i < 4; ++i) {
        const Launch l(1 << i, threads_of(BN), block_bytes<BN, kPair>(), 1 << i, false, nullptr);
        if (cudaOccupancyMaxActiveClusters(&n[i], kernel, &l.c) != cudaSuccess) n[i] = 0;
    }
}

}  // namespace

namespace tt {

MatmulFits matmul_fits(int sms)
{
    MatmulFits f;
    f.sms = sms;
    f.one[0] = sms;
    f.two[0] = 2 * sms;
    count_clusters<256, true>(f.one);
    count_clusters<16, false>(f.two);
    cudaGetLastError();     // a refusal here is an answer, not an error of the next launch
    return f;
}

// products of the operands' terms: of terms i and j with i + j < 3
static int products_of(const Product& p)
{
    int n = 0;
    for (int i = 0; i < p.a.parts; ++i)
        for (int j = 0; j < p.b.parts && i + j < 3; ++j) ++n;
    return n;
}

MatmulPlan matmul_plan(const Product& p, const MatmulFits& fits)
{
    MatmulPlan q;
    const int64_t blocks = ceil_div(p.deep, kDeep);
    const int products = products_of(p);
    // Results of fp32 and operands of several terms are formed by chunks of kChunk blocks, 16-bit results by as many as their roundings
    // hide.
    auto any = [&](int type) { return p.e.out_type == type || (p.has_pre && p.e.pre_type == type); };
    const bool fine = any(TT_F32) || products > 1;
    q.chunk = fine ? kChunk : any(TT_F16) ? kChunkF16 : kChunkBf16;
    // The tile's height and the blocks that share a tile: what a model of the time likes best, in cycles.  64 k take what their
    // products take (half a cycle for each row and 16 k, at 128 columns), or what their bytes take, about 55 a cycle and SM; a tile
    // a few cycles for each of its rows, a launch 1500, a cluster 1500 more, a joining kernel 6000.  Of 300 drawn products (10^7 to 2 10^11
    // multiplications, all three kinds, bf16 and fp32) what it likes takes 1.5 % more than the best of all choices in the mean, and 41 % at
    // most (2008 x 80 by sums of 10704, fp32: 27 us in slices, 19 shared).
    double best = 0.0;
    for (int n = p.b_mn ? 64 : 16; n <= (fine ? 128 : 256); n *= 2) {
        const double tiles = (double)ceil_div(p.cols, kCols) * ceil_div(p.rows, n), work = 2.0 * n * products;
        const double each = std::max(work, (kCols * p.a.parts + n * p.b.parts) * (kDeep * 2 / 55.0));
        const int fit = fit_of(n);
        const int(&room)[4] = fit > 1 ? fits.two : fits.one;
        for (int i = 0; i < 4; ++i) {
            const int k = 1 << i;
            if (i > 0 && (tiles > room[i] || blocks < 2 * k)) break;
            // two blocks on an SM share its bandwidth
            const double turns = fit > 1 ? std::max(1.0, tiles * k / fits.sms) : ceil(tiles * k / fits.sms);
            const double t = turns * ((double)blocks / k * each + 8.0 * n) + 1500.0 + (k > 1 ? 1500.0 : 0.0);
            if (q.height == 0 || t < best) best = t, q.height = n, q.split = k, q.slices = 1, q.pair = false;
        }
        const int k = (int)std::min((double)fits.sms * fit / tiles, blocks / 4.0);
        if (k > 8 && (double)p.rows * p.cols * k <= kMostSums) {
            const double t = std::max(1.0, tiles * k / fits.sms) * ((double)blocks / k * each + 8.0 * n) + 1500.0 + 6000.0;
            if (t < best) best = t, q.height = n, q.split = 1, q.slices = k, q.pair = false;
        }
        // (Not for fp32 results of single terms, whose short chunks both blocks wait for: the gradient of a table of 43000 x 1616 bf16 from 2240
        // rows took 464 us by pairs, 384 by single blocks, and of 120 drawn products nine such ones 10 to 25 % more.)
        if (n >= 128 && fits.one[1] > 0 && !(fine && products == 1)) {
            const double count = (double)ceil_div(p.cols, 2 * kCols) * ceil_div(p.rows, n);
            const double two = std::max(work, (kCols * p.a.parts + n / 2 * p.b.parts) * (kDeep * 2 / 55.0));
            const double t = ceil(count / fits.one[1]) * ((double)blocks * two + 8.0 * n) + 2000.0;
            if (t < best) best = t, q.height = n, q.split = q.slices = 1, q.pair = true;
        }
    }
    if (fine || ceil_div(blocks, q.split * q.slices) > q.chunk) q.sums = q.height >= kHigh && p.a.parts == 1 && p.b.parts == 1 ? kChunks : kTermChunks;
    q.scratch = q.slices > 1 ? (size_t)(q.slices * p.rows * p.cols) * sizeof(float) : 0;
    return q;
}

int matmul(const Product& p, const MatmulPlan& q, void* scratch, int32_t* status, const MatmulFits& fits, bool early, cudaStream_t s)
{
    Args g = {};
    g.e = p.e;
    if (q.slices > 1) {
        g.e = {};
        g.e.out = scratch;
        g.e.out_type = TT_F32;
        g.e.out_stride = p.cols;
        g.e.skip_row = -1;
    }
    g.status = status;
    g.rows = p.rows;
    g.cols = p.cols;
    g.a_terms = p.a.parts;
    g.b_terms = p.b.parts;
    const int64_t blocks = ceil_div(p.deep, kDeep);
    const int bn = q.height;
    const bool pair = q.pair;
    const int64_t tiles_c = ceil_div(p.cols, pair ? 2 * kCols : kCols), tiles_r = ceil_div(p.rows, bn);
    if (blocks > INT32_MAX / 8 || tiles_c * tiles_r > INT32_MAX / 8) return TT_ERR_ARG;   // sizes that no device holds
    g.blocks = (int)blocks;
    g.tiles_c = (int)tiles_c;
    g.tiles_r = (int)tiles_r;
    g.chunk = q.chunk;
    g.fail = p.fail;
    g.split = q.split;
    g.slices = q.slices;
    auto four = [&](const void* x, int type, int64_t stride) {
        return !x || (((uintptr_t)x & (4 * type_bytes(type) - 1)) == 0 && (stride & 3) == 0);
    };
    g.vectors = (p.cols & 3) == 0 && four(g.e.out, g.e.out_type, g.e.out_stride) && four(g.e.pre, g.e.pre_type, g.e.pre_stride) &&
                four(g.e.residual, g.e.residual_type, g.e.residual_stride);
    g.idesc = (1u << 4) | (p.a.type == TT_BF16 ? 1u << 7 | 1u << 10 : 0u) | (p.a_mn ? 1u << 15 : 0u) | (p.b_mn ? 1u << 16 : 0u) |
              (uint32_t)(bn >> 3) << 17 | (uint32_t)((pair ? 2 * kCols : kCols) >> 4) << 24;
    if (!encode(&g.a, p.a, p.a_mn ? kDeep : kCols) || !encode(&g.b, p.b, p.b_mn ? kDeep : pair ? bn / 2 : bn)) return TT_ERR_CUDA;
    auto by_height = [&](auto amn, auto bmn, auto sums) {
        constexpr bool A = decltype(amn)::value, B = decltype(bmn)::value;
        constexpr int S = decltype(sums)::value;
        if constexpr (S != kTermChunks) {       // (whose sums of their own leave tensor memory for half that height)
            if (bn == 256) return pair ? launch<256, A, B, S, true>(g, fits, early, s) : launch<256, A, B, S, false>(g, fits, early, s);
        }
        if (bn == 128) return pair ? launch<128, A, B, S, true>(g, fits, early, s) : launch<128, A, B, S, false>(g, fits, early, s);
        if constexpr (S == kChunks) {
            return cudaErrorInvalidValue;       // (no plan has it)
        } else {
            if constexpr (!B) {
                if (bn == 16) return launch<16, A, B, S, false>(g, fits, early, s);
                if (bn == 32) return launch<32, A, B, S, false>(g, fits, early, s);
            }
            return launch<64, A, B, S, false>(g, fits, early, s);
        }
    };
    auto by_sides = [&](auto sums) {
        using Yes = std::true_type;
        using No = std::false_type;
        return p.b_mn ? by_height(Yes(), Yes(), sums) : p.a_mn ? by_height(Yes(), No(), sums) : by_height(No(), No(), sums);
    };
    cudaError_t e = q.sums == kWhole    ? by_sides(std::integral_constant<int, kWhole>())
                    : q.sums == kChunks ? by_sides(std::integral_constant<int, kChunks>())
                                        : by_sides(std::integral_constant<int, kTermChunks>());
    if (e == cudaSuccess && q.slices > 1) {
        const int64_t blocks_of_rows = p.rows * ceil_div(p.cols, 32);      // (below kMostSums)
        e = launch_early(k_join, (unsigned)blocks_of_rows, kJoinThreads, s, (const float*)scratch, (int)q.slices, p.rows, p.cols, p.e, (const int32_t*)status);
    }
    return e == cudaSuccess ? TT_OK : TT_ERR_CUDA;
}

}  // namespace tt
