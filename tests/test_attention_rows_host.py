"""Partial results hold every row of the layout that the kernels write (no GPU): row tiles of 128 / G
tokens, the second one from row 128 on, whatever the group size G is."""
import pytest

from sparse_attention_kpool_gb300 import build as kbuild
from sparse_attention_kpool_gb300 import kpool as K

RUNS = 152          # two partial results each: [rows][head_dim] sums and (m, l) per row, fp32


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return K.load()


@pytest.mark.parametrize("d", [64, 128])
def test_workspace_holds_the_rows_of_both_row_tiles(lib, d):
    before = 0
    for group in range(1, 129):
        tt = 128 // group
        for rows in range(1, 2 * tt + 2):
            last = rows * group if rows <= tt else 128 + min(rows - tt, tt) * group
            sh = K.kpool_attention_shape(group, 1, d, K.KPOOL_BF16, 0.1, 0)
            got = lib.kpool_attention_workspace_bytes(rows, 1, sh)
            # what else lies there for so few rows: header, join items, row list, mask bits
            other = 256 + 256 + RUNS * 64 + (rows * 4 + 255) // 256 * 256 + rows * ((rows + 127) // 128) * 16
            assert got >= 2 * RUNS * last * (d + 2) * 4 + other, (group, rows)
            assert rows == 1 or got >= before, (group, rows)
            before = got
