"""The roots and reciprocals that 8-bit codes depend on are those rounded to nearest, for every mantissa and exponent
of their stated ranges, against the device's correctly rounded square root and reciprocal."""
import ctypes
import os
import subprocess

import pytest

from tensor_train_compressed_mixed_b200 import build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "exact_roots.cu")


@pytest.fixture(scope="module")
def lib():
    out = os.path.join(build.ROOT, "_build", "libexact_roots.so")
    if build._stale(out, [SRC] + build._deps()):
        os.makedirs(os.path.dirname(out), exist_ok=True)
        tmp = f"{out}.tmp{os.getpid()}"
        subprocess.run([build.NVCC] + build.ARCH + build.FLAGS + ["-shared", "-o", tmp, SRC, "-lcudart"], check=True, capture_output=True)
        os.replace(tmp, out)
    handle = ctypes.CDLL(out)
    for name in ("different_roots", "different_reciprocals"):
        fn = getattr(handle, name)
        fn.argtypes, fn.restype = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_float)], ctypes.c_longlong
    return handle


@pytest.mark.parametrize("name,first,last", [("different_roots", -102, 127), ("different_reciprocals", -100, 125)])
def test_every_value_of_the_stated_range(lib, name, first, last):
    example = ctypes.c_float()
    n = getattr(lib, name)(first, last, ctypes.byref(example))
    assert n == 0, f"{n} values differ, one of them {example.value.hex()}"
