"""The example layer: selection and attention together, against the plain 64-bit attention."""
import importlib.util
import os

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import attention_reference as A

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("sparse_layer", os.path.join(ROOT, "examples", "sparse_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_runs(example, capsys):
    sparse, dense = example.main(tokens=700, steps=2)
    # 700 tokens are fewer than index_topk: every row keeps every earlier token, in another order
    # (both within a bf16 weight and output rounding of the true value, |v| sums below 4)
    assert ((sparse.float() - dense.float()).abs() <= 2.0 ** -7 * dense.float().abs() + 2.0 ** -6).all()
    assert "verified a tree" in capsys.readouterr().out


def test_layer_steps_match_the_reference(example):
    gen = torch.Generator(device="cuda").manual_seed(3)
    layer = example.SparseLayer(capacity=400, q_heads=8, kv_heads=2, pool=4, index_topk=64)
    x = example.random_tokens(300, layer, gen)
    layer.append(x["k"], x["v"], x["index_k"])
    out = layer.prompt(x["q"], x["index_q"], x["index_w"])
    cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    ids = K.kpool_select(x["index_q"], x["index_k"], x["index_w"], cu, 4, 64, layer.index_scale)[1]
    pick = [0, 1, 63, 64, 150, 299]
    ref = A.reference(x["q"][pick], x["k"], x["v"], A.see_selected(ids[pick], [0] * 6, [300]), layer.scale)
    A.check(out[pick], None, ref, "prompt")
    y = example.random_tokens(1, layer, gen)
    layer.append(y["k"], y["v"], y["index_k"])
    out = layer.decode(y["q"], y["index_q"], y["index_w"])
    pooled = K.kpool_pool_keys(layer.index_k, layer.cu, 4)
    row = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = K.kpool_select_rows(y["index_q"], y["index_w"], row, row + 300, pooled, layer.cu, 400, 4, 64,
                              layer.index_scale)[1]
    see = A.see_selected(ids, [0], [301])
    assert see[0].max() == 300 and see[0].numel() == 64 + 1  # the row's own token is its incomplete trailing pool
    A.check(out, None, A.reference(y["q"], layer.k, layer.v, see, layer.scale), "decode")
    z = example.random_tokens(4, layer, gen)
    layer.append(z["k"], z["v"], z["index_k"])
    out = layer.verify(z["q"], [-1, 0, 0, 2])
    see = A.see_tree([4], [400], [301], [[0b0001, 0b0011, 0b0101, 0b1101]])
    A.check(out, None, A.reference(z["q"], layer.k, layer.v, see, layer.scale), "verify")
