// Which kernel the products of given sizes take: each line of the input is a product, each line of the output its plan.
//   input:  sides (0: forward, 1: x's gradient, 2: the table's), terms of A and of B, rows, cols, deep, type of the result, 1 if z is kept in it too
//   output: height, whether a pair of blocks shares a tile, blocks that share its k, slices of k, sums (0: whole, 1: chunks of single
//           terms, 2: chunks of operands of several), and blocks of 64 k of a chunk
// Arguments: what the device holds at a time, or none to ask the current device and print that.
#include <stdio.h>
#include <stdlib.h>

#include "matmul.cuh"

int main(int argc, char** argv)
{
    tt::MatmulFits fits;
    if (argc != 10) {
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, 0) != cudaSuccess) return 1;
        fits = tt::matmul_fits(sms);
        printf("%d", fits.sms);
        for (int i = 0; i < 4; ++i) printf(" %d", fits.one[i]);
        for (int i = 0; i < 4; ++i) printf(" %d", fits.two[i]);
        printf("\n");
        return 0;
    }
    fits.sms = atoi(argv[1]);
    for (int i = 0; i < 4; ++i) fits.one[i] = atoi(argv[2 + i]), fits.two[i] = atoi(argv[6 + i]);
    int sides, a, b, type, keep;
    long long rows, cols, deep;
    while (scanf("%d %d %d %lld %lld %lld %d %d", &sides, &a, &b, &rows, &cols, &deep, &type, &keep) == 8) {
        tt::Product p;
        p.a_mn = sides >= 1;
        p.b_mn = sides == 2;
        p.a.parts = a;
        p.b.parts = b;
        p.rows = rows;
        p.cols = cols;
        p.deep = deep;
        p.has_pre = keep != 0;
        p.e.out_type = p.e.pre_type = type;
        const tt::MatmulPlan q = tt::matmul_plan(p, fits);
        printf("%d %d %d %d %d %d\n", q.height, (int)q.pair, q.split, q.slices, q.sums, q.chunk);
    }
    return 0;
}
