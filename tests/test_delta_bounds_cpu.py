"""What the delta rule's backward may read of a piece's chunks, checked on the
host: the rule is the kernel's own header, compiled by g++."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mamba_ssd_chunked_03_b200", "csrc")
PROGRAM = r"""
#include <cstdio>
#include "ssd_delta_blocks.h"
int main() {
  for (int chunks = 1; chunks <= 2; ++chunks)
    for (int mt = 0; mt < 4; ++mt)
      for (int sb = 0; sb < 4; ++sb) std::printf("%d %d %d %d\n", chunks, mt, sb, (int)ssd::delta::block_exists(mt, sb, chunks));
}
"""


@pytest.fixture(scope="module")
def blocks(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("blocks")
    (d / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "p.cpp"), "-o", str(d / "p")], check=True)
    rows = subprocess.run([str(d / "p")], check=True, capture_output=True, text=True).stdout.split("\n")[:-1]
    return {tuple(map(int, r.split()[:3])): r.split()[3] == "1" for r in rows}


def reads(blocks, chunks):
    """Chunks of the piece (0, 1) whose decays the blocks that exist may read: their rows' chunk."""
    return {mt // 2 for (c, mt, _), e in blocks.items() if c == chunks and e}


def pieces(L):
    """(first chunk, tokens) of the pieces of one row, and how many places for chunks there are."""
    return [(2 * i, min(64, L - 64 * i)) for i in range(-(-L // 64))], -(-L // 32)


@pytest.mark.parametrize("L", list(range(1, 200)))
def test_no_decays_of_a_chunk_that_does_not_exist(blocks, L):
    list_, places = pieces(L)
    for first, n in list_:
        chunks = 2 if n > 32 else 1
        assert all(first + c < places and 32 * c < n for c in reads(blocks, chunks)), (L, first, n)


@pytest.mark.parametrize("n", list(range(1, 65)))
def test_no_block_with_tokens_is_left_out(blocks, n):
    """Tokens s <= t < n, so their block counts; above the diagonal none does."""
    chunks = 2 if n > 32 else 1
    for t in range(n):
        for s in range(t + 1):
            assert blocks[chunks, t // 16, s // 16]
    assert not any(e for (c, mt, sb), e in blocks.items() if sb > mt)


def test_the_check_sees_the_fault():
    """Every block on or below the diagonal, whether its chunk exists or not, fails the first test."""
    old = {(c, mt, sb): sb <= mt for c in (1, 2) for mt in range(4) for sb in range(4)}
    assert reads(old, 1) == {0, 1}  # a second chunk's decays, of a piece of one


def test_the_kernel_asks_the_rule():
    src = open(os.path.join(CSRC, "ssd_delta_grads.cuh")).read()
    at = src.index("plain[mt >> 1]")
    assert "block_exists(mt, sb, nch)" in src[at - 200:at]
