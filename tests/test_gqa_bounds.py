"""Index arithmetic of the grouped-head kernels at the ends of their integer ranges, run on the host: the same
inline functions that the kernels call, compiled by nvcc into a small program that makes no CUDA call."""
import os
import subprocess

import pytest

from compressed_sparse_attention_13_b200 import build

SOURCE = r"""
#include <cstdio>
#include <cstdint>
#include "gqa_tiles.cuh"
#include "paged_split.cuh"

namespace csa { __device__ unsigned int g_status; }

int main() {
    const int ts[] = {INT32_MIN, INT32_MIN + 1, -2147483, -5, -3, -2, -1, 0, 1, 63, 64, 2047, INT32_MAX - 1, INT32_MAX};
    const int ws[] = {0, 1, 2, 64, 2048, INT32_MAX - 1, INT32_MAX};
    for (int t : ts)
        for (int w : ws) printf("first %d %d %d\n", t, w, csa::first_seen(t, w));
    const int64_t far[] = {INT64_MIN, INT64_MIN + 1, INT64_MIN + 30, -(int64_t(1) << 40), -5, -1, 0, 1, 19, 20, 94, 95, 96, 97,
                           int64_t(1) << 40, INT64_MAX - 30, INT64_MAX - 1, INT64_MAX};
    for (int64_t t : far)
        for (int w : {0, 1, 20, INT32_MAX})
            for (int64_t cap : {int64_t(0), int64_t(96), int64_t(INT32_MAX)}) {
                const csa::Span v = csa::span_at<64>(t, w, cap);
                printf("span %lld %d %lld %lld %d %d\n", (long long)t, w, (long long)cap, (long long)v.lo, v.n, v.steps);
            }
    return 0;
}
"""


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    d = tmp_path_factory.mktemp("bounds")
    src, exe = str(d / "bounds.cu"), str(d / "bounds")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([build.NVCC, *build.ARCH, "-std=c++17", "-O1", "-rdc=true", "--expt-relaxed-constexpr", f"-I{build.CSRC}",
                    f"-I{os.path.join(build.ROOT, 'include')}", src, "-o", exe], check=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    return [ln.split() for ln in out.splitlines()]


def test_first_key_of_a_window_of_any_length(lines):
    got = [tuple(map(int, x[1:])) for x in lines if x[0] == "first"]
    assert len(got) == 14 * 7
    for t, w, first in got:
        assert first == (max(t - w + 1, 0) if w else 0), (t, w)


def test_visible_tokens_of_any_position(lines):
    """A position below 0 sees nothing; of one past the cache's places those that exist are seen."""
    got = [tuple(map(int, x[1:])) for x in lines if x[0] == "span"]
    assert len(got) == 18 * 4 * 3
    for t, w, cap, lo, n, steps in got:
        first, end = (max(t - w + 1, 0) if w else 0), min(t + 1, cap)
        assert n == max(end - first, 0) and steps == max(-(-n // 64), 1), (t, w, cap)
        assert n == 0 or (lo == first and 0 <= lo and lo + n <= cap)
