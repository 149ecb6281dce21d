"""The arithmetic that bounds a request's rows in the kernels (csrc/bq_rows.h),
built for the CPU with checks for overflow: offsets of any value, against whole
numbers of any size."""
import itertools
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DRIVER = r"""
#include <stdio.h>
#include "bq_rows.h"
int main(void)
{
    long long lo, hi, tokens;
    while (scanf("%lld %lld %lld", &lo, &hi, &tokens) == 3) {
        const bq::Rows r = bq::rows_between((int)lo, (int)hi, tokens);
        printf("%d %d\n", r.first, r.n);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def rows_between(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    (d / "s.cpp").write_text(DRIVER)
    csrc = os.path.join(ROOT, "ternary_quantized_gemv_amd", "csrc")
    build = ["g++", "-std=c++17", "-O1", "-I", csrc, str(d / "s.cpp"), "-o", str(d / "s")]
    check = ["-fsanitize=undefined", "-fno-sanitize-recover=all"]
    if subprocess.run(build + check, capture_output=True).returncode:  # no runtime for it here
        subprocess.run(build, check=True)

    def call(cases):
        text = "".join("%d %d %d\n" % c for c in cases)
        r = subprocess.run([str(d / "s")], input=text, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        return [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]
    return call


def test_rows_of_any_offsets(rows_between):
    least, most = -(1 << 31), (1 << 31) - 1
    offsets = sorted({least, least + 1, -5, -1, 0, 1, 2, 5, 7, 8, 9, 100, 1 << 20, 1 << 30, most - 1, most})
    cases = list(itertools.product(offsets, offsets, (1, 2, 7, 8, 100, 1 << 30, most)))
    for (lo, hi, tokens), (first, n) in zip(cases, rows_between(cases)):
        end = min(hi, tokens)
        want = (lo, end - lo) if 0 <= lo < end else (0, 0)
        assert (first, n) == want, (lo, hi, tokens)
        assert 0 <= first and n >= 0 and first + n <= tokens
