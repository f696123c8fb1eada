"""Buffers of the residual norm that overlap are refused before a device is touched (an
output in the place of an input is not: the tests on the GPU).  CPU only."""
import os
import subprocess

import pytest

from deepseek_v4_sparse_indexer_gb300 import _binding as B
from test_more_abi import NORM, call

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, D = 4, 4096
AT = {k: (i + 1) << 24 for i, k in enumerate(("x", "res", "res_out", "weight", "out", "codes", "scales", "n_live"))}
GOOD = dict(NORM, T=T, D=D, res_type=B.DS4A_BF16, **AT)
END = {"x": T * D * 2, "res": T * D * 2, "res_out": T * D * 2, "weight": D * 4, "out": T * D * 2, "codes": T * D,
       "scales": T * D // 128 * 4, "n_live": 4}


@pytest.fixture(scope="module")
def lib():
    return B.load()


@pytest.mark.parametrize("one,other", [(a, b) for a in ("res_out", "out", "codes", "scales") for b in AT if a != b])
def test_partial_overlaps(lib, one, other):
    # `one` begins 16 bytes before the end of `other`, and the other way round
    for a, b in ((one, other), (other, one)):
        last = (END[b] - 1) // 16 * 16
        assert call(lib.ds4a_add_rms_norm, GOOD, **{a: AT[b] + last}) == B.DS4A_EINVAL


@pytest.mark.parametrize("change", [
    dict(out=AT["x"], out_type=B.DS4A_F16), dict(out=AT["x"], out_type=B.DS4A_F32), dict(out=AT["res_out"]),
    dict(out=AT["x"], x_stride=D + 8), dict(res_out=AT["x"], out=AT["x"]), dict(res_out=AT["res"], out=AT["res"]),
    dict(res_out=AT["x"], res_type=B.DS4A_F32), dict(res_out=AT["x"], x_stride=2 * D), dict(codes=AT["x"]),
    dict(codes=AT["out"]), dict(scales=AT["codes"]), dict(scales=AT["weight"]), dict(out=AT["x"] + 2 * D),
    dict(x_stride=2 * D, res_out=AT["x"] + 2 * D - 16, res_out_stride=2 * D),
    dict(x_stride=2 * D, res_out=AT["x"] + 2 * D + 16, res_out_stride=2 * D)])
def test_overlaps(lib, change):
    assert call(lib.ds4a_add_rms_norm, GOOD, **change) == B.DS4A_EINVAL


PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "span.h"
using ds4a::Span;
static unsigned long long state = 1;
static int pick(int n) { state = state * 6364136223846793005ULL + 1442695040888963407ULL; return int((state >> 33) % unsigned(n)); }
int main() {
    char *base = reinterpret_cast<char *>(1 << 20);
    long hits = 0;
    for (int n = 0; n < 400000; ++n) {
        Span s[2];
        std::vector<int> bytes(4096, 0);
        for (int k = 0; k < 2; ++k) {
            s[k].width = 1 + pick(k && pick(2) ? 200 : 12);
            s[k].rows = 1 + pick(6);
            s[k].stride = s[k].rows > 1 ? s[k].width + pick(pick(2) ? 40 : 3) : 0;
            s[k].type = 0;
        }
        if (pick(2) && s[0].rows > 1 && s[1].rows > 1)
            s[0].stride = s[1].stride = s[0].stride > s[1].stride ? s[0].stride : s[1].stride;
        bool want = false;
        for (int k = 0; k < 2; ++k) {
            const int at = pick(pick(2) ? 600 : 60);
            s[k].at = base + at;
            for (int i = 0; i < s[k].rows; ++i)
                for (int j = 0; j < s[k].width; ++j) {
                    int &v = bytes[at + i * s[k].stride + j];
                    want = want || (k && v);
                    if (!k) v = 1;
                }
        }
        hits += want;
        if (ds4a::overlap(s[0], s[1]) != want || ds4a::overlap(s[1], s[0]) != want) {
            std::printf("%d: %lld %lld %lld, %lld %lld %lld, apart %ld: %d\n", n, s[0].rows, s[0].stride, s[0].width, s[1].rows,
                        s[1].stride, s[1].width, long((const char *)s[1].at - (const char *)s[0].at), want);
            return 1;
        }
    }
    Span none = {nullptr, 1, 0, 4, 0}, some = {base, 1, 0, 4, 0};
    if (ds4a::overlap(none, some) || ds4a::overlap(some, none)) return 2;
    return hits > 100000 && hits < 300000 ? 0 : 3;
}
"""


def test_overlap_against_bytes(tmp_path):
    """Rows of two buffers, byte by byte."""
    src, exe = tmp_path / "span.cpp", tmp_path / "span"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "deepseek_v4_sparse_indexer_gb300", "csrc"), "-o",
                    str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
