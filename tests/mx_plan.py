"""The launches that a projection with 4-bit weights makes, asked of the rule
itself: csrc/mx_plan.h is host code, compiled here by the C++ compiler."""
import collections
import ctypes
import functools
import os
import shutil
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_state_layer_amd", "csrc")
SOURCE = """
#include "mx_plan.h"
extern "C" int fits(int64_t n_tok, int64_t n_out) { return gdn::mx_proj_fits(n_tok, n_out); }
extern "C" int plan(int64_t n_tok, int32_t n_in, int64_t n_out, int64_t* out) {
    const gdn::MxPlan p = gdn::mx_plan(n_tok, n_in, n_out);
    for (int i = 0; i < p.n; ++i, out += 6) {
        const gdn::MxLaunch& l = p.launch[i];
        out[0] = l.tile; out[1] = l.tokens; out[2] = l.channels; out[3] = l.c0; out[4] = l.c1; out[5] = l.workgroups;
    }
    return p.n;
}
"""
Launch = collections.namedtuple("Launch", "tile tokens channels c0 c1 workgroups")


@functools.lru_cache(None)
def _lib():
    cxx = shutil.which("g++") or shutil.which("c++") or "/opt/rocm/llvm/bin/clang++"
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib],
                       check=True)
        so = ctypes.CDLL(lib)
    so.plan.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
    so.fits.argtypes = [ctypes.c_int64, ctypes.c_int64]
    return so


def plan(n_tok, n_in, n_out):
    out = (ctypes.c_int64 * 12)()
    n = _lib().plan(n_tok, n_in, n_out, out)
    return [Launch(*out[6 * i: 6 * i + 6]) for i in range(n)]


def fits(n_tok, n_out):
    return bool(_lib().fits(n_tok, n_out))


def paths(n_tok, n_in, n_out):
    """The launches' kernels: "skinny", "tile128", "tile192", "strip" (the skinny
    kernel behind tiles)."""
    return [f"tile{p.channels}" if p.tile else "strip" if p.c0 else "skinny" for p in plan(n_tok, n_in, n_out)]


# Sizes that reach the tile kernels, with the launches they take: both tiles,
# with and without a strip behind them; inputs that end inside 64 and inside
# 128, fewer than four groups of inputs; even and odd widths.
TILE_CASES = [
    (300, 96, 700, ["tile128"]), (129, 64, 4097, ["tile128"]), (700, 544, 1500, ["tile128"]),
    (700, 2080, 3000, ["tile128"]), (300, 1056, 12301, ["tile192"]), (2600, 1184, 2050, ["tile192"]),
    (700, 512, 8200, ["tile192", "strip"]), (500, 1184, 12353, ["tile192", "strip"]),
]
# In-projections: tokens, hidden, h_k, h_v, d; the gates are the last channels.
TILE_IN_PROJ = [
    (1100, 512, 4, 8, 128, ["tile128"]), (300, 544, 16, 32, 128, ["tile192"]),
    (500, 544, 16, 32, 128, ["tile192", "strip"]),
]


def in_proj_channels(h_k, h_v, d):
    return 2 * h_k * d + 2 * h_v * d + 2 * h_v
