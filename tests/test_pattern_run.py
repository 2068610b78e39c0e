"""The part of a pattern's run that is copied in whole 16-byte lines stays inside the caller's array (CPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <stdio.h>
#include "pattern_run.h"
// every alignment of arrays of up to 3 rows of 1 to 21 entries, every run of every row
int main() {
    long long runs = 0;
    for (int rows = 1; rows <= 3; ++rows)
        for (int ld = 1; ld <= 21; ++ld)
            for (int word = 0; word < 4; ++word)
                for (int h = 0; h < rows; ++h) {
                    const uintptr_t base = 4096 + 4 * word, row = base + 4ull * h * ld;
                    const long long before = (long long)h * ld, behind = (long long)(rows - h) * ld;
                    for (int lo = 0; lo < ld; ++lo)
                        for (int hi = lo; hi < ld; ++hi, ++runs) {
                            const saf::PatternRun x = saf::pattern_run(row, before, behind, lo, hi);
                            const long long first = (long long)row + 4ll * x.first, end = (long long)row + 4ll * x.end;
                            if (first % 16 || end % 16) return puts("not a line"), 1;
                            if (x.first < x.end && (first < (long long)base || end > (long long)base + 4ll * rows * ld))
                                return puts("outside the array"), 1;
                            // what is left is at most three entries at either end
                            const int left = x.first < x.end ? (x.first > lo ? x.first - lo : 0) : hi - lo + 1;
                            const int right = x.first < x.end && hi >= x.end ? hi - x.end + 1 : 0;
                            if (left > (x.first < x.end ? 3 : 6) || right > 3) return puts("too much is left"), 1;
                            // and only where a line is not a part of the array
                            const long long line = (long long)row + 4ll * lo, last = (long long)row + 4ll * hi;
                            const bool cut = line / 16 * 16 < (long long)base || last / 16 * 16 + 16 > (long long)base + 4ll * rows * ld;
                            if ((left || right) && !cut) return puts("left without a reason"), 1;
                        }
                }
    printf("%lld runs\n", runs);
    return 0;
}
"""


def test_lines_of_a_run_stay_inside_the_array(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "run.cc", tmp_path / "run"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", os.path.join(ROOT, "softmax_attention_hybrid_gb300", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
    assert int(out.stdout.split()[0]) > 10000
