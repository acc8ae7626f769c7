"""Rotary positions at the ends of int32 on the GPU, against cosines and sines of 60-digit angles."""
import decimal
import math

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests.test_rotary_table_host import FAR, KINDS, turns

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rd,kw", KINDS, ids=str)
def test_far_positions(rd, kw):
    pos = torch.tensor(FAR, dtype=torch.int32)
    x = torch.zeros((len(FAR), 1, rd), device="cuda")
    x[..., :rd // 2] = 1.0
    out, _ = K.kpool_rotary(x, pos.cuda(), K.new_rotary_table(rd, **kw))
    out = out.cpu().double()[:, 0]
    with decimal.localcontext(decimal.Context(prec=60)):
        angle = torch.tensor([[float(2 * ((t * f) % 1)) for f in turns(rd, **kw)] for t in FAR], dtype=torch.float64) * math.pi
    # the angle within 2^-24 of a half turn, cosine and sine within two steps below one
    tol = math.pi * 2.0 ** -24 + 2.0 ** -23
    assert (out[:, :rd // 2] - torch.cos(angle)).abs().max() <= tol
    assert (out[:, rd // 2:] - torch.sin(angle)).abs().max() <= tol
