"""How the optimiser step spreads its tensors over launches, on the host: every element once, in order,
within the limits of a launch (its blocks of 256 threads are counted as work items in 32 bits)."""
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "semi_structured_sparsity_amd" / "csrc"

PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "nm_adamw_pieces.h"
int main(int argc, char** argv) {   // chunk, pieces a launch, blocks a launch (0: the kernel's), sizes
    std::vector<long long> n;
    for (int i = 4; i < argc; ++i) n.push_back(atoll(argv[i]));
    const long long most = atoll(argv[3]);
    nm::adamw_pieces((int)n.size(), atoll(argv[1]), atoi(argv[2]), most ? most : nm::kAdamWMostBlocks,
                     [&](int i) { return (int64_t)n[i]; },
                     [&](int i, int64_t at, int64_t m, int64_t block) {
                         printf("%d %lld %lld %lld\\n", i, (long long)at, (long long)m, (long long)block);
                     },
                     [] { puts("launch"); return true; });
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("pieces")
    (d / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", str(CSRC), str(d / "p.cpp"), "-o", str(d / "p")], check=True)
    return d / "p"


def _launches(program, chunk, pieces, most, sizes):
    out = subprocess.run([str(program), str(chunk), str(pieces), str(most), *map(str, sizes)], capture_output=True, text=True,
                         check=True, timeout=60).stdout.split("\n")[:-1]
    runs, now = [], []
    for line in out:
        if line == "launch":
            runs.append(now)
            now = []
        else:
            now.append(tuple(map(int, line.split())))
    assert not now, "pieces without a launch"
    return runs


def _check(runs, chunk, pieces, most, sizes):
    done = [0] * len(sizes)
    last = 0
    for run in runs:
        assert 1 <= len(run) <= pieces
        block = 0
        for i, at, m, b in run:
            assert i >= last and at == done[i] and m > 0 and at % chunk == 0 and b == block
            block += -(-m // chunk)
            done[i] += m
            last = i
        assert block <= most and block * 256 < 2 ** 32
    assert done == list(sizes)


LIMIT = (1 << 24) - 1     # blocks of 256 threads in a launch


@pytest.mark.parametrize("sizes", [[], [0], [1], [0, 5, 0], [2048] * 3, [700] * 131, [LIMIT * 2048], [LIMIT * 2048 + 1], [1 << 39],
                                   [34400000000, 77, 1], [900000000] * 44, [3, (1 << 36) + 5, 0, 4097], [1 << 30] * 100])
def test_kernel_limits(program, sizes):
    runs = _launches(program, 2048, 44, 0, sizes)
    _check(runs, 2048, 44, LIMIT, sizes)
    blocks = sum(-(-n // 2048) for n in sizes)
    assert len(runs) >= max(-(-blocks // LIMIT), -(-sum(n > 0 for n in sizes) // 44))


@pytest.mark.parametrize("most", [1, 2, 5])
def test_small_limits(program, most):
    for sizes in ([1, 255, 256, 257, 0, 2000], [10000], [256 * most] * 4, [256 * most + 1] * 4):
        _check(_launches(program, 256, 3, most, sizes), 256, 3, most, sizes)
