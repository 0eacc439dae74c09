"""How the kernels of the attention over a paged cache number what they leave in the workspace, on the host (CPU).

When a wait of the first kernel runs out, the tiles that it did not finish have no entry, and the second one finds whatever
the workspace held.  What it takes for shares has to stay inside the workspace, and their number bounded, whatever that is."""
import itertools
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "latent_compressed_attention_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "attend_shares.h"
// Lines of first, last, shares: whether they are gone through, and if so the smallest and largest part that is read.
int main() {
    int first, last, shares;
    while (std::scanf("%d %d %d", &first, &last, &shares) == 3) {
        if (!mla::shares_written(first, last, shares)) {
            std::puts("no");
            continue;
        }
        long long lo = mla::part_number(first, true), hi = lo, n = 0;
        for (long long c = first; c <= last; ++c, ++n) {
            const long long part = mla::part_number(static_cast<int>(c), c == first);
            lo = part < lo ? part : lo, hi = part > hi ? part : hi;
        }
        std::printf("%lld %lld %lld\n", lo, hi, n);
    }
}
"""


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    folder = tmp_path_factory.mktemp("shares")
    (folder / "shares.cpp").write_text(PROGRAM)
    cxx = shutil.which("g++") or shutil.which("c++")
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(folder / "shares"), str(folder / "shares.cpp")],
                   check=True)

    def run(triples):
        text = "".join("%d %d %d\n" % t for t in triples)
        out = subprocess.run([str(folder / "shares")], input=text, capture_output=True, text=True, check=True).stdout
        return [None if line == "no" else tuple(map(int, line.split())) for line in out.splitlines()]

    return run


@pytest.mark.parametrize("shares", [1, 2, 76, 304])
def test_whatever_the_workspace_held(parts, shares):
    rng = random.Random(shares)
    odd = [-2**31, -2**31 + 1, -1, 0, 1, shares - 1, shares, shares + 1, 2**30, 2**31 - 1, 0x3F800000, 0x7F7F7F7F]
    pairs = list(itertools.product(odd, odd)) + [(rng.getrandbits(32) - 2**31, rng.getrandbits(32) - 2**31) for _ in range(500)]
    pairs += [(rng.randrange(shares), rng.getrandbits(32) - 2**31) for _ in range(500)]
    taken = 0
    for (first, last), got in zip(pairs, parts([(a, b, shares) for a, b in pairs])):
        if got is not None:
            assert 0 <= got[0] and got[1] < 2 * shares and got[2] <= shares, (first, last, got)
            taken += 1
    assert taken < len(pairs)


@pytest.mark.parametrize("shares", [1, 2, 5, 76])
def test_every_tile_that_there_is(parts, shares):
    """All first and last shares of real tiles are taken, with a part each and none of them twice."""
    pairs = [(a, b) for a in range(shares) for b in range(a, shares)]
    for (first, last), got in zip(pairs, parts([(a, b, shares) for a, b in pairs])):
        assert got is not None and got[2] == last - first + 1
        numbers = [2 * c + (c == first) for c in range(first, last + 1)]
        assert (got[0], got[1]) == (min(numbers), max(numbers))
    # what a share leaves of the tile before and of the one that starts in it are two parts
    assert parts([(0, 0, 1)])[0][:2] == (1, 1)
