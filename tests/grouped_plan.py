"""The library's own rules for the products grouped by expert (csrc/grouped_plan.h, arithmetic of the host), compiled for
the tests: which instance takes a call, and how many workgroups it launches."""
import ctypes
import functools
import os
import subprocess
import tempfile

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_routed_moe_router_amd", "csrc",
                      "grouped_plan.h")
SOURCE = """
#include "%s"
using namespace ds4;
extern "C" {
int few(int r, int64_t E, int64_t P) { return grouped_is_few(r, E, P); }
int form(int r, int64_t E, int64_t P, int64_t N) { const auto f = grouped_form(r, E, P, N); return f.waves * 1000 + f.height; }
int turned(int64_t E, int64_t P, int64_t N) { const auto f = grouped_turned_form(E, P, N); return f.waves * 1000 + f.height; }
int64_t groups(int w, int h, int r, int64_t E, int64_t P, int64_t N) { return grouped_workgroups(GroupedForm{w, h}, r, E, P, N); }
int64_t tiles(int w, int h, int r, int64_t E, int64_t P) { return grouped_max_tiles(r, E, P, GroupedForm{w, h}.lowest()); }
int64_t columns(int w, int h, int64_t N) { return grouped_col_tiles(GroupedForm{w, h}, N); }
int large(int64_t E, int64_t N, int64_t K) { return grouped_dw_large(E, N, K); }
int64_t dw_groups(int l, int64_t E, int64_t N, int64_t K) { return grouped_dw_workgroups(l, E, N, K); }
}
"""


@functools.lru_cache(None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE % HEADER)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", src, "-o", so], check=True)
        L = ctypes.CDLL(so)
    I, I64 = ctypes.c_int, ctypes.c_int64
    for name, args, res in (("few", [I, I64, I64], I), ("form", [I] + [I64] * 3, I), ("turned", [I64] * 3, I),
                            ("groups", [I, I, I, I64, I64, I64], I64), ("tiles", [I, I, I, I64, I64], I64),
                            ("columns", [I, I, I64], I64), ("large", [I64] * 3, I), ("dw_groups", [I] + [I64] * 3, I64)):
        getattr(L, name).argtypes, getattr(L, name).restype = args, res
    return L


def forward(ragged, E, P, N):
    """(waves, height) of the kernel that takes P rows, or "few"."""
    return "few" if _lib().few(ragged, E, P) else divmod(_lib().form(ragged, E, P, N), 1000)


def turned(E, P, N):
    """(waves, height) of the kernel of the rows' gradient, N values long."""
    return divmod(_lib().turned(E, P, N), 1000)


def workgroups(form, ragged, E, P, N):
    return _lib().groups(*form, ragged, E, P, N)


def row_tiles(form, ragged, E, P):
    return _lib().tiles(*form, ragged, E, P)


def col_tiles(form, N):
    return _lib().columns(*form, N)


def dw_large(E, N, K):
    """Whether the weights' gradient goes in tiles of 256 x 256."""
    return bool(_lib().large(E, N, K))


def dw_workgroups(large, E, N, K):
    return _lib().dw_groups(large, E, N, K)
