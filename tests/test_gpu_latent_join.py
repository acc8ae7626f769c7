"""Latent rows cut over CTAs and joined in each of the ways that the join has, on either side of their borders, with rows in
their own places and in the runs': against a plain 64-bit implementation, twice, bit for bit."""
import pytest
import torch

from tests.test_gpu_latent import BF, BIG, run, verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,heads", [(1, 1), (9, 16), (10, 16), (6, 32), (7, 32), (3, 64), (4, 64), (2, 128), (1, 193), (12, 64),
                                        (11, 64), (48, 16), (47, 16), (24, 32), (23, 32), (6, 128), (5, 128), (152, 4),
                                        (153, 4), (160, 5), (76, 128), (77, 128), (200, 3), (192, 4)], ids=str)
def test_whole_caches(rows, heads):
    lengths = [(1500 + 37 * r) % 4000 for r in range(rows)] if rows < 20 else [(300 + 61 * r) % 700 for r in range(rows)]
    lengths[rows // 2] = 0 if rows > 2 else lengths[rows // 2]
    made, out, lse = run(lengths, 64, heads, BIG, BF, "auto", seed=rows)
    verify(made, out, lse, lengths, 64, pick=sorted({0, rows // 2, rows - 1, rows // 3, rows // 5}))
    assert torch.isfinite(out).all()
    _, again, alse = run(lengths, 64, heads, BIG, BF, "auto", tensors=made[:2], pool=(None, made[2]))
    assert torch.equal(out, again) and torch.equal(lse, alse)


@pytest.mark.parametrize("rows,heads,width", [(3, 64, 2052), (4, 64, 2052), (11, 64, 2052), (12, 64, 2052), (2, 128, 4000), (5, 128, 900),
                                              (6, 128, 900), (9, 16, 2052), (153, 4, 300), (47, 16, 500)], ids=str)
def test_lists(rows, heads, width):
    g = torch.Generator().manual_seed(rows)
    ids = torch.stack([torch.randperm(4000, generator=g)[:width] for _ in range(rows)]).to(torch.int32)
    ids[rows // 2, 1:] = -1
    seq = [0] * rows
    made, out, lse = run([4000], 64, heads, BIG, BF, "auto", ids=ids, seq=seq, seed=rows)
    verify(made, out, lse, [4000], 64, ids, seq, pick=sorted({0, rows // 2, rows - 1, rows // 3}))
    _, again, alse = run([4000], 64, heads, BIG, BF, "auto", ids=ids, seq=seq, tensors=made[:2], pool=(None, made[2]))
    assert torch.equal(out, again) and torch.equal(lse, alse)
