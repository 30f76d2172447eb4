"""The choice among the forms of the products' kernel, compiled with the host
compiler alone: every form that some size takes is among those that the GPU tests
run, and those take the forms they are listed for."""
import ctypes
import math
import os
import random
import subprocess

import pytest

from product_forms import FORMS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 148
SHIM = """
#include "grouped_form.h"
extern "C" void form(int rows, int experts, int N, long long k_bytes, int sms, int* out) {
  const moeq::ProductForm f = moeq::choose_form(rows, experts, N, k_bytes, sms);
  out[0] = f.cg; out[1] = f.width; out[2] = f.S;
}
extern "C" int parts(int rest, int clusters) { return moeq::last_turn_parts(rest, clusters); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("forms")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "bit_quantized_moe_top_b200", "csrc"), str(d / "shim.cpp"), "-o", str(d / "shim.so")],
                   check=True)
    so = ctypes.CDLL(str(d / "shim.so"))
    so.form.argtypes = [ctypes.c_int] * 3 + [ctypes.c_longlong, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    return so


def form(lib, rows, experts, N, k_bytes):
    out = (ctypes.c_int * 3)()
    lib.form(rows, experts, N, k_bytes, SMS, out)
    return tuple(out)


def last_turn(lib, counts, N, width):
    """Pieces of the last turn's tiles, as the pairs of a launch divide them; 1 where nothing is left over."""
    NF = (N - 1) // 256 + 1
    groups = min(sum(counts), len(counts))
    launched = min((groups + (sum(counts) - groups) // width) * NF, SMS // 2)
    rest = sum(-(-c // width) for c in counts) * NF % launched
    return lib.parts(rest, launched) if rest else 1


@pytest.mark.parametrize("op,counts,N,K,want,parts", FORMS)
def test_listed_products_take_their_forms(lib, op, counts, N, K, want, parts):
    assert all(c >= 0 for c in counts)
    assert form(lib, sum(counts), len(counts), N, K * (1 if op == "int8" else 2)) == want
    if want[0] == 2 and parts is not None:
        assert last_turn(lib, counts, N, want[1]) == parts


def test_every_form_is_listed(lib):
    """Over sizes from one row and channel to 20000 x 32768 x 16384 in up to 256 experts."""
    rng = random.Random(0)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    seen = set()
    for _ in range(60000):
        seen.add(form(lib, log(1, 20000), rng.choice([1, 2, 4, 8, 16, 64, 256]), log(1, 32768), log(1, 32768)))
    for op in ("bf16", "int8"):
        assert seen <= {f[4] for f in FORMS if f[0] == op}
    listed = {f[4] for f in FORMS}
    assert listed <= seen  # and no form is there that no size takes
    for op in ("bf16", "int8"):
        assert {f[5] for f in FORMS if f[0] == op and f[4][0] == 2} >= {1, 2, 4}


def test_last_turn_fills_no_more_than_the_pairs(lib):
    for clusters in range(1, SMS // 2 + 1):
        for rest in range(clusters):
            assert lib.parts(rest, clusters) * rest <= clusters and lib.parts(rest, clusters) in (1, 2, 4)
