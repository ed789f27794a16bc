"""Which kernel a product of given sizes takes on a whole B200, and that the sizes below reach every one of them.

test_gpu_project_plans.py computes them.  The plan comes from a small program that asks the library (plans.cu).
"""
import os
import subprocess

import pytest
import torch

from tensor_train_compressed_mixed_b200.build import CSRC, INCLUDE, NVCC, PKG

HERE = os.path.dirname(os.path.abspath(__file__))
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
CODE = {F32: 0, BF16: 1, F16: 2}
TERMS = {F32: 3, F16: 2, BF16: 1}
# blocks of a kernel that the device holds at a time: SMs, then clusters of 1, 2, 4 and 8 of one block an SM and of two
B200 = [148, 148, 74, 33, 15, 296, 74, 33, 15]
WHOLE, CHUNKS, TERM_CHUNKS = 0, 1, 2

# product (0: forward, 1: x's gradient, 2: the table's), table, grad_out, result, activation, n, rows, dim,
# and its plan: height, pair, sums, blocks that share a tile, slices of k
CASES = [
    (0, BF16, None, F16, "relu", 5543, 130, 69, (128, 0, 0, 1, 1)), (0, F16, None, F16, None, 70, 3, 31704, (128, 0, 0, 1, 124)),
    (0, F16, None, F16, None, 402, 276, 967, (128, 0, 0, 8, 1)), (0, F16, None, F32, None, 3538, 266, 88, (128, 0, 1, 1, 1)),
    (0, F16, None, F32, None, 67, 4, 31829, (128, 0, 1, 1, 124)), (0, F16, None, F32, None, 584, 168, 984, (128, 0, 1, 8, 1)),
    (0, F32, None, F32, None, 4765, 284, 84, (128, 0, 2, 1, 1)), (0, F32, None, BF16, "relu", 65, 4, 29825, (128, 0, 2, 1, 116)),
    (0, F32, None, F32, None, 457, 141, 972, (128, 0, 2, 8, 1)), (0, F16, None, F16, None, 1176, 916, 196, (128, 1, 0, 1, 1)),
    (0, BF16, None, F16, "relu", 1228, 984, 4284, (128, 1, 1, 1, 1)), (0, F32, None, BF16, "relu", 4827, 148, 77, (128, 1, 2, 1, 1)),
    (0, BF16, None, BF16, None, 16, 5, 72, (16, 0, 0, 1, 1)), (0, F16, None, F16, None, 3, 5, 10824, (16, 0, 0, 1, 42)),
    (0, F16, None, F16, None, 4, 3, 520, (16, 0, 0, 4, 1)), (0, F16, None, F32, None, 16, 8, 72, (16, 0, 2, 1, 1)),
    (0, F32, None, F32, None, 33, 4, 71, (16, 0, 2, 1, 1)), (0, F16, None, F32, None, 4, 5, 9152, (16, 0, 2, 1, 35)),
    (0, BF16, None, F16, "relu", 15, 3133, 45400, (16, 0, 2, 1, 11)), (0, F32, None, F32, None, 35, 5, 4439, (16, 0, 2, 1, 17)),
    (0, F16, None, F32, None, 4, 6, 464, (16, 0, 2, 4, 1)), (0, BF16, None, F16, "relu", 8, 4304, 8640, (16, 0, 2, 2, 1)),
    (0, F32, None, F32, None, 34, 3, 194, (16, 0, 2, 2, 1)), (0, F16, None, F16, None, 6262, 514, 82, (256, 0, 0, 1, 1)),
    (0, BF16, None, BF16, None, 140, 4, 38206, (256, 0, 0, 1, 148)), (0, BF16, None, F16, "relu", 424, 544, 1744, (256, 0, 0, 8, 1)),
    (0, BF16, None, F16, "relu", 3136, 1304, 4728, (256, 0, 1, 1, 1)), (0, F16, None, F16, None, 266, 817, 42055, (256, 0, 1, 1, 10)),
    (0, BF16, None, F16, "relu", 808, 664, 16888, (256, 0, 1, 4, 1)), (0, F16, None, F16, None, 4845, 406, 84, (256, 1, 0, 1, 1)),
    (0, F16, None, F16, None, 1515, 1570, 4138, (256, 1, 1, 1, 1)), (0, BF16, None, BF16, None, 3019, 3, 68, (32, 0, 0, 1, 1)),
    (0, F16, None, F16, None, 18, 3, 25040, (32, 0, 0, 1, 98)), (0, BF16, None, BF16, None, 248, 8, 976, (32, 0, 0, 8, 1)),
    (0, F16, None, F32, None, 3040, 8, 72, (32, 0, 2, 1, 1)), (0, F32, None, F32, None, 2776, 8, 104, (32, 0, 2, 1, 1)),
    (0, F32, None, F32, None, 33, 3, 15488, (32, 0, 2, 1, 60)), (0, BF16, None, F16, "relu", 24, 3136, 47768, (32, 0, 2, 1, 11)),
    (0, F16, None, F32, None, 36, 5, 16311, (32, 0, 2, 1, 63)), (0, F32, None, BF16, "relu", 264, 136, 472, (32, 0, 2, 4, 1)),
    (0, BF16, None, F16, "relu", 32, 4824, 8672, (32, 0, 2, 2, 1)), (0, F16, None, F32, None, 246, 6, 982, (32, 0, 2, 8, 1)),
    (0, BF16, None, BF16, None, 7379, 4, 72, (64, 0, 0, 1, 1)), (0, BF16, None, BF16, None, 34, 7, 25778, (64, 0, 0, 1, 100)),
    (0, F16, None, F16, None, 537, 144, 516, (64, 0, 0, 4, 1)), (0, F16, None, F32, None, 7232, 8, 72, (64, 0, 2, 1, 1)),
    (0, BF16, None, F16, "relu", 514, 2020, 4710, (64, 0, 2, 1, 1)), (0, F32, None, BF16, "relu", 2231, 260, 81, (64, 0, 2, 1, 1)),
    (0, F32, None, BF16, "relu", 35, 4, 23705, (64, 0, 2, 1, 92)), (0, BF16, None, F16, "relu", 40, 1728, 41232, (64, 0, 2, 1, 10)),
    (0, F16, None, F32, None, 35, 3, 25616, (64, 0, 2, 1, 100)), (0, F32, None, BF16, "relu", 244, 136, 975, (64, 0, 2, 8, 1)),
    (0, BF16, None, F16, "relu", 701, 656, 9079, (64, 0, 2, 2, 1)), (0, F16, None, F32, None, 244, 141, 1032, (64, 0, 2, 8, 1)),
    (1, F16, F16, F16, None, 5828, 74, 154, (128, 0, 0, 1, 1)), (1, BF16, BF16, BF16, "relu", 68, 32637, 6, (128, 0, 0, 1, 127)),
    (1, F16, F16, F16, None, 536, 992, 200, (128, 0, 0, 8, 1)), (1, F16, F16, F32, None, 1160, 72, 1040, (128, 0, 1, 1, 1)),
    (1, F16, F16, F32, None, 68, 32489, 6, (128, 0, 1, 1, 127)), (1, F16, F16, F32, None, 517, 1014, 144, (128, 0, 1, 8, 1)),
    (1, F32, BF16, F32, None, 3227, 67, 259, (128, 0, 2, 1, 1)), (1, BF16, BF16, F32, "relu", 4746, 81, 313, (128, 0, 2, 1, 1)),
    (1, F16, BF16, BF16, None, 5152, 72, 152, (128, 0, 2, 1, 1)), (1, F32, BF16, F32, None, 65, 25629, 10, (128, 0, 2, 1, 100)),
    (1, BF16, BF16, F32, "relu", 72, 34105, 5, (128, 0, 2, 1, 133)), (1, F16, BF16, BF16, None, 72, 26496, 8, (128, 0, 2, 1, 103)),
    (1, F16, BF16, BF16, None, 711, 475, 279, (128, 0, 2, 4, 1)), (1, BF16, BF16, F32, "relu", 440, 1008, 264, (128, 0, 2, 8, 1)),
    (1, F32, F32, F32, None, 488, 1046, 135, (128, 0, 2, 8, 1)), (1, BF16, BF16, BF16, "relu", 1868, 231, 523, (128, 1, 0, 1, 1)),
    (1, F16, F16, F16, None, 1337, 4130, 909, (128, 1, 1, 1, 1)), (1, BF16, BF16, F32, "relu", 5712, 80, 136, (128, 1, 2, 1, 1)),
    (1, F16, F16, F16, "relu", 1013, 136, 1277, (128, 1, 2, 1, 1)), (1, F32, F32, F32, None, 460, 73, 2343, (128, 1, 2, 1, 1)),
    (1, F16, F16, F16, None, 17, 68, 4, (16, 0, 0, 1, 1)), (1, F16, F16, F16, None, 3, 9727, 3, (16, 0, 0, 1, 38)),
    (1, F16, F16, F16, None, 3, 515, 4, (16, 0, 0, 4, 1)), (1, F16, F16, F32, None, 16, 67, 3, (16, 0, 2, 1, 1)),
    (1, BF16, BF16, F32, "relu", 17, 78, 4, (16, 0, 2, 1, 1)), (1, F32, BF16, F32, None, 16, 69, 4, (16, 0, 2, 1, 1)),
    (1, F32, BF16, F32, None, 3, 5683, 3, (16, 0, 2, 1, 22)), (1, BF16, BF16, F32, "relu", 3, 7744, 3, (16, 0, 2, 1, 30)),
    (1, F16, F16, F16, "relu", 3, 6240, 3, (16, 0, 2, 1, 24)), (1, F32, F32, F32, None, 3, 227, 4, (16, 0, 2, 2, 1)),
    (1, BF16, BF16, F32, "relu", 4, 598, 3, (16, 0, 2, 4, 1)), (1, F16, F16, F16, "relu", 4, 263, 3, (16, 0, 2, 2, 1)),
    (1, F16, F16, F16, None, 6249, 75, 543, (256, 0, 0, 1, 1)), (1, BF16, BF16, BF16, None, 134, 37515, 5, (256, 0, 0, 1, 146)),
    (1, F16, F16, F16, None, 438, 1829, 527, (256, 0, 0, 8, 1)), (1, F16, F16, F16, None, 1576, 4521, 2604, (256, 0, 1, 1, 1)),
    (1, F16, F16, F16, None, 592, 41352, 528, (256, 0, 1, 1, 9)), (1, F16, F16, F16, None, 1646, 16681, 279, (256, 0, 1, 4, 1)),
    (1, BF16, BF16, BF16, "relu", 6491, 71, 262, (256, 1, 0, 1, 1)), (1, F16, F16, F16, None, 1436, 4393, 1557, (256, 1, 1, 1, 1)),
    (1, F16, F16, F16, None, 2962, 73, 3, (32, 0, 0, 1, 1)), (1, BF16, BF16, BF16, "relu", 17, 22564, 9, (32, 0, 0, 1, 88)),
    (1, BF16, BF16, BF16, None, 551, 457, 5, (32, 0, 0, 4, 1)), (1, F16, F16, F16, "relu", 2861, 68, 12, (32, 0, 2, 1, 1)),
    (1, BF16, BF16, F32, "relu", 1637, 65, 132, (32, 0, 2, 1, 1)), (1, F32, BF16, F32, None, 2656, 104, 8, (32, 0, 2, 1, 1)),
    (1, F32, BF16, F32, None, 18, 21871, 4, (32, 0, 2, 1, 85)), (1, BF16, BF16, F32, "relu", 17, 29561, 5, (32, 0, 2, 1, 115)),
    (1, F16, F16, F32, None, 18, 25395, 3, (32, 0, 2, 1, 99)), (1, F16, F16, F32, None, 243, 962, 7, (32, 0, 2, 8, 1)),
    (1, BF16, BF16, F32, "relu", 568, 454, 4, (32, 0, 2, 4, 1)), (1, F32, F32, F32, None, 242, 968, 7, (32, 0, 2, 8, 1)),
    (1, BF16, BF16, BF16, None, 6720, 72, 8, (64, 0, 0, 1, 1)), (1, BF16, BF16, BF16, "relu", 34, 26539, 4, (64, 0, 0, 1, 103)),
    (1, BF16, BF16, BF16, "relu", 237, 1091, 139, (64, 0, 0, 8, 1)), (1, F16, F16, F32, None, 7048, 80, 8, (64, 0, 2, 1, 1)),
    (1, BF16, BF16, F32, "relu", 1907, 85, 391, (64, 0, 2, 1, 1)), (1, F32, BF16, F32, None, 5496, 144, 8, (64, 0, 2, 1, 1)),
    (1, F32, BF16, F32, None, 38, 21812, 3, (64, 0, 2, 1, 85)), (1, BF16, BF16, F32, "relu", 34, 28645, 11, (64, 0, 2, 1, 112)),
    (1, F16, BF16, BF16, None, 34, 22707, 8, (64, 0, 2, 1, 88)), (1, F32, F32, F32, None, 592, 464, 144, (64, 0, 2, 4, 1)),
    (1, BF16, BF16, F32, "relu", 326, 974, 134, (64, 0, 2, 8, 1)), (1, F16, BF16, BF16, None, 232, 1059, 154, (64, 0, 2, 8, 1)),
    (2, BF16, BF16, BF16, "relu", 76, 4861, 132, (128, 0, 0, 1, 1)), (2, F16, F16, F16, None, 31536, 72, 8, (128, 0, 0, 1, 123)),
    (2, BF16, BF16, BF16, "relu", 480, 528, 416, (128, 0, 0, 4, 1)), (2, F16, F16, F32, None, 70, 5142, 153, (128, 0, 1, 1, 1)),
    (2, F16, F16, F32, None, 33296, 72, 8, (128, 0, 1, 1, 130)), (2, F16, F16, F32, None, 1040, 208, 432, (128, 0, 1, 8, 1)),
    (2, F16, F16, F16, "relu", 71, 4779, 148, (128, 0, 2, 1, 1)), (2, BF16, BF16, F32, "relu", 68, 4766, 264, (128, 0, 2, 1, 1)),
    (2, F32, BF16, F32, None, 72, 4840, 192, (128, 0, 2, 1, 1)), (2, F32, BF16, F32, None, 25336, 72, 8, (128, 0, 2, 1, 99)),
    (2, BF16, BF16, F32, "relu", 35577, 75, 3, (128, 0, 2, 1, 139)), (2, F16, BF16, BF16, None, 27135, 74, 6, (128, 0, 2, 1, 106)),
    (2, F16, BF16, BF16, None, 453, 1031, 144, (128, 0, 2, 4, 1)), (2, BF16, BF16, F32, "relu", 1016, 376, 264, (128, 0, 2, 8, 1)),
    (2, F32, BF16, F32, None, 456, 528, 416, (128, 0, 2, 4, 1)), (2, BF16, BF16, BF16, None, 227, 2392, 387, (128, 1, 0, 1, 1)),
    (2, F16, F16, F16, None, 4136, 1584, 656, (128, 1, 1, 1, 1)), (2, F32, F32, F32, None, 95, 4828, 129, (128, 1, 2, 1, 1)),
    (2, BF16, BF16, F32, "relu", 76, 5430, 137, (128, 1, 2, 1, 1)), (2, F16, F16, F16, "relu", 131, 2026, 520, (128, 1, 2, 1, 1)),
    (2, F16, F16, F16, None, 66, 588, 6238, (256, 0, 0, 1, 1)), (2, F16, F16, F16, None, 38687, 133, 4, (256, 0, 0, 1, 148)),
    (2, BF16, BF16, BF16, None, 912, 656, 776, (256, 0, 0, 4, 1)), (2, F16, F16, F16, None, 4537, 2593, 1620, (256, 0, 1, 1, 1)),
    (2, F16, F16, F16, None, 43796, 296, 770, (256, 0, 1, 1, 10)), (2, F16, F16, F16, None, 16600, 1072, 552, (256, 0, 1, 4, 1)),
    (2, BF16, BF16, BF16, "relu", 80, 6488, 280, (256, 1, 0, 1, 1)), (2, F16, F16, F16, None, 4272, 2328, 946, (256, 1, 1, 1, 1)),
    (2, BF16, BF16, BF16, None, 66, 64, 5, (64, 0, 0, 1, 1)), (2, F16, F16, F16, None, 7883, 3, 3, (64, 0, 0, 1, 31)),
    (2, BF16, BF16, BF16, None, 443, 3, 3, (64, 0, 0, 2, 1)), (2, F16, F16, F32, None, 65, 67, 3, (64, 0, 2, 1, 1)),
    (2, BF16, BF16, F32, "relu", 65, 84, 5, (64, 0, 2, 1, 1)), (2, F32, BF16, F32, None, 71, 65, 5, (64, 0, 2, 1, 1)),
    (2, F32, F32, F32, None, 3927, 3, 3, (64, 0, 2, 1, 15)), (2, BF16, BF16, F32, "relu", 6845, 3, 3, (64, 0, 2, 1, 26)),
    (2, F16, F16, F16, "relu", 4837, 5, 3, (64, 0, 2, 1, 19)), (2, F32, F32, F32, None, 200, 3, 3, (64, 0, 2, 2, 1)),
    (2, BF16, BF16, F32, "relu", 266, 4, 3, (64, 0, 2, 2, 1)), (2, F16, F16, F16, "relu", 230, 4, 3, (64, 0, 2, 2, 1)),
]


def terms(product, kind, up, result, act):
    """bf16 terms, or values as they are, of the table's (or x's) and the other operand."""
    if product == 0:
        return (3, 3) if kind == F32 else (1, 1)
    if kind != F32 and up == kind and act is None:
        return 1, 1
    if kind == result == BF16:
        return 1, 1
    dz = 3 if act or up == F32 else TERMS[up]
    return TERMS[kind], dz if kind == F32 or result == F32 else min(dz, 2)


def kernels():
    """Every kernel that the library has: product, height, pair, sums."""
    every = set()
    for product in range(3):
        for sums in (WHOLE, CHUNKS, TERM_CHUNKS):
            for height in (16, 32, 64, 128, 256):
                if (height == 256 and sums == TERM_CHUNKS) or (height < 128 and sums == CHUNKS) or (height < 64 and product == 2):
                    continue
                every |= {(product, height, pair, sums) for pair in ((0, 1) if height >= 128 else (0,))}
    return every


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """A function from lines of products to lines of plans."""
    out = str(tmp_path_factory.mktemp("plans") / "plans")
    subprocess.run([NVCC, "-std=c++17", "--expt-relaxed-constexpr", "-gencode", "arch=compute_100a,code=sm_100a", "-I", INCLUDE, "-I", CSRC,
                    os.path.join(HERE, "plans.cu"), "-o", out, "-L", PKG, "-lttemb", "-Xlinker", "-rpath=" + PKG], check=True)

    def asked(products):
        text = "\n".join(" ".join(map(str, p)) for p in products)
        got = subprocess.run([out, *map(str, B200)], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in got.splitlines()]
    return asked


def _product(product, kind, up, result, act, n, rows, dim):
    a, b = terms(product, kind, up, result, act)
    sizes = {0: (n, rows, dim), 1: (n, dim, rows), 2: (rows, dim, n)}[product]
    return (product, a, b, *sizes, CODE[result], 0)


def test_the_cases_reach_every_kernel(ask):
    got = ask([_product(*c[:8]) for c in CASES])
    assert len(got) == len(CASES)
    for c, (height, pair, split, slices, sums, _) in zip(CASES, got):
        assert (height, pair, sums, split, slices) == c[8], c
    assert {(c[0], c[8][0], c[8][1], c[8][2]) for c in CASES} == kernels()
    for product in range(3):        # shared tiles and slices of each kind of sums
        for sums in (WHOLE, CHUNKS, TERM_CHUNKS):
            mine = [c[8] for c in CASES if c[0] == product and c[8][2] == sums]
            assert any(p[3] > 1 for p in mine) and any(p[4] > 1 for p in mine) and any(p[1] for p in mine)


def test_long_sums_are_cut_into_chunks(ask):
    """4096 k at most in tensor memory for fp16 results, 32768 for bf16, 256 where a result has 32 bits or an operand several terms."""
    for kind, most in ((F16, 64), (BF16, 512)):
        for blocks, sums in ((most, WHOLE), (most + 1, CHUNKS), (40 * most, CHUNKS)):
            (height, pair, split, slices, got, chunk), = ask([(0, 1, 1, 20000, 20000, blocks * 64, CODE[kind], 0)])
            assert (split, slices, got, chunk) == (1, 1, sums, most), (kind, blocks)
    for p in ((0, 1, 1, 20000, 20000, 64, 0, 0), (1, 1, 3, 20000, 20000, 64, 1, 0), (0, 1, 1, 4, 200, 64, 0, 0)):
        assert ask([p])[0][4:] == (CHUNKS if p[:3] == (0, 1, 1) and p[3] > 4 else TERM_CHUNKS, 4)
    # z kept in another type than the result: the finer of the two
    assert ask([(0, 1, 1, 20000, 20000, 8192, CODE[F32], 1)])[0][4:] == (CHUNKS, 4)
