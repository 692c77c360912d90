"""Host-side tests of how the experts' linear layers cut their sums: the counts of the kernel's own header,
compiled for the host with overflow checks, against whole numbers of any size."""
import os
import subprocess

import pytest

from tp_reduce_residual_gb300 import build as nbuild

LARGEST = 2 ** 31 - 1024  # rows of a call, at most
PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "bn_experts.h"
int main(int n, char **v)
{
    for (int i = 2; i < n; ++i)
        std::printf("%d %d\\n", bn::sum_stages(std::atoi(v[i])), bn::sum_runs(std::atoi(v[i]), std::atoi(v[1])));
}
"""


@pytest.fixture(scope="module")
def counts(tmp_path_factory):
    folder = tmp_path_factory.mktemp("sums")
    source, program = folder / "sums.cc", folder / "sums"
    source.write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nbuild.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", cuda, "-I", nbuild.CSRC,
                    "-I", nbuild.INCLUDE, str(source), "-o", str(program)], check=True)

    def of(log, lengths):
        out = subprocess.run([str(program), str(log), *map(str, lengths)], capture_output=True, text=True)
        assert out.returncode == 0, out.stderr
        return [tuple(map(int, line.split())) for line in out.stdout.splitlines()]

    return of


@pytest.mark.parametrize("log", [2, 6])  # a weight gradient in FP32, and in 16 bits
def test_counts_over_the_whole_range(counts, log):
    """Both sides of a run's and a stage's end, up to the longest sum: the warp that issues products takes a run
    for every 2^log stages, and the warps that take sums out have to count as many."""
    run = 2 ** log
    step = 64 * run
    lengths = {1, 2, 63, 64, 65, LARGEST, LARGEST - 1}
    for at in (step, 2 * step, 5 * step, 2 ** 20, 2 ** 30, 2 ** 31 - step - 1024, LARGEST // step * step):
        lengths |= {at + d for d in (-64, -1, 0, 1, 63, 64, 65) if 0 < at + d <= LARGEST}
    lengths |= {2 ** 31 - 4096, 2 ** 31 - 4095, 2 ** 31 - 4094}  # where adding 4095 leaves 31 bits
    lengths = sorted(lengths)
    got = counts(log, lengths)
    assert got == [(-(-d // 64), -(-(-(-d // 64)) // run)) for d in lengths]


def test_no_values_are_one_run(counts):
    assert counts(6, [0, -5]) == [(0, 1), (0, 1)]
