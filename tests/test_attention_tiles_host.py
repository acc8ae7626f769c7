"""Tile numbers of the attention kernels against the rows that they have to cover (no GPU: the kernels' own rule, compiled
for the host): every row of every sequence in exactly one tile, no number outside the sequences."""
import os
import random
import subprocess

import pytest

from sparse_attention_kpool_gb300 import build as kbuild
from tests import attention_reference as A

HERE = os.path.dirname(os.path.abspath(__file__))
PACKS = [[1], [0], [2], [0, 2], [3, 0, 0], [1, 0, 1], [1, 1, 1], [0, 2, 1, 0], [0, 0, 5, 0], [70, 0, 1, 40, 9, 129], [300],
         [128, 127, 129, 1]]
TOKENS = [1, 2, 3, 16, 25, 32, 64, 128, 256]      # of a row tile; 1: groups of 65 to 128 heads


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("tiles") / "tiles")
    subprocess.run([kbuild.nvcc(), *kbuild.ARCH, *kbuild.NVCC_FLAGS, "-I", kbuild.CSRC, "-o", exe,
                    os.path.join(HERE, "attention_tiles.cu")], check=True, capture_output=True)

    def ask(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        lines = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(lines) == len(cases)
        out = []
        for line in lines:
            tiles, *rest = map(int, line.split())
            assert len(rest) == 2 * tiles
            out.append(list(zip(rest[::2], rest[1::2])))
        return out
    return ask


def covers(tiles, q_lens, tt):
    """The first tokens that each sequence's tiles begin at, every one once."""
    assert all(0 <= b < len(q_lens) for b, _ in tiles), "a tile of a sequence that does not exist"
    got = sorted((b, t) for b, t in tiles if 0 <= t < q_lens[b])
    return got == [(b, t) for b, n in enumerate(q_lens) for t in range(0, n, tt)]


def test_every_row_has_one_tile(places):
    rng = random.Random(1)
    packs = PACKS + [[rng.choice([0, 1, 2, rng.randrange(300)]) for _ in range(rng.randrange(1, 12))] for _ in range(60)]
    asked = [(q, tt, paged) for q in packs for tt in TOKENS for paged in (0, 1)]
    # behind cu_q: what looks like the cumulative lengths of more sequences
    cases = [(paged, 0, tt, len(q), len(q) + 9, *A.cu(q + [0, 1, 0, 2, 0, 0, 1, 0])) for q, tt, paged in asked]
    for (q, tt, paged), tiles in zip(asked, places(cases)):
        assert covers(tiles, q, tt), (q, tt, paged)


@pytest.mark.parametrize("rows", [0, 1], ids=["tiles", "rows"])
def test_a_row_of_every_sequence(rows, places):
    """Without cu_q: tiles of any number of tokens, and the form that numbers its tiles by the sequences."""
    asked = [(S, tt) for S in (1, 2, 7, 300) for tt in ((1,) if rows else TOKENS)]
    for (S, tt), tiles in zip(asked, places([(1, rows, tt, S, 0) for S, tt in asked])):
        assert covers(tiles, [1] * S, tt), (S, tt)
        assert not rows or len(tiles) == S
