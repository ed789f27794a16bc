// Products on the tensor cores (matmul.cu) as project.cu calls them.
#pragma once

#include "project.cuh"

namespace tt {

// A 16-bit matrix [outer][inner] that tensor maps can take: rows `stride` values apart, and `parts` such matrices
// part_stride values apart (the bf16 terms of values that have more bits than one holds).
struct Operand {
    const void* p = nullptr;
    int64_t outer = 0, inner = 0, stride = 0, part_stride = 0;
    int32_t type = TT_BF16, parts = 1;
};
// whether a matrix can be read as it lies: 16-byte aligned rows
inline bool mappable(const void* p, int64_t stride, int64_t outer, int64_t inner)
{
    return ((uintptr_t)p & 15) == 0 && (outer == 1 || ((stride & 7) == 0 && stride >= inner && stride < (int64_t)1 << 38));
}

// Blocks of the product kernels that a device holds at a time: those of one an SM and those of two, alone and in clusters of
// 2, 4 and 8 (0: none of that size).
struct MatmulFits {
    int sms = 148;
    int one[4] = {}, two[4] = {};
};
MatmulFits matmul_fits(int sms);     // of the current device

// C[r][c] = sum over k of A(c, k) B(r, k), finished by e: r < rows, c < cols, k < deep.  A is [cols][deep], or with a_mn
// [deep][cols]; B is [rows][deep], or with b_mn [deep][rows].  Both of one type.
struct Product {
    Operand a, b;
    bool a_mn = false, b_mn = false, has_pre = false;
    int64_t rows = 0, cols = 0, deep = 0;
    Epilogue e = {};
    int fail = TT_INJECT_NONE;       // the role that gives up, in tests
};
// How a tile's sums are formed: whole ones in tensor memory, chunks of single terms, or chunks of operands of several terms.
enum { kWhole, kChunks, kTermChunks };
// How a product of these sizes, types and terms (no pointer of it is looked at) is computed.
struct MatmulPlan {
    int height = 0, split = 1, slices = 1;
    int sums = kWhole;
    int chunk = 0;            // blocks of 64 k of a chunk
    bool pair = false;
    size_t scratch = 0;       // device memory for slices' sums
};
MatmulPlan matmul_plan(const Product& p, const MatmulFits& fits);
// early: a kernel of the same call is before it on the stream.  Returns a tt_status.
int matmul(const Product& p, const MatmulPlan& q, void* scratch, int32_t* status, const MatmulFits& fits, bool early, cudaStream_t s);

}  // namespace tt
