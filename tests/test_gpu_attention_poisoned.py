"""The attention checks again with outputs full of NaN and a workspace of ones before every call, so that a place
which no kernel writes, or reads before it is written, cannot hold an earlier call's right values."""
import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import test_gpu_attention as G
from tests.test_gpu_attention import BF, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def poison(monkeypatch):
    new = K.new_attention_workspace

    def poisoned(call):
        def run(q, *a, **kw):
            if kw.get("out") is None:
                kw["out"] = torch.full_like(q, float("nan"), memory_format=torch.contiguous_format)
            if kw.get("out_lse") is None and kw.pop("return_lse", False):
                kw["out_lse"] = torch.full(q.shape[:2], float("nan"), device="cuda")
            if kw.get("workspace") is not None:
                kw["workspace"].fill_(0xFF)
            return call(q, *a, **kw)
        return run
    monkeypatch.setattr(K, "new_attention_workspace", lambda *a, **kw: new(*a, **kw).fill_(0xFF))
    for name in ("kpool_attention_prompt", "kpool_attention_tree", "kpool_attention_selected"):
        monkeypatch.setattr(K, name, poisoned(getattr(K, name)))


@pytest.mark.parametrize("heads", [(8, 2, 128, BF), (6, 2, 128, BF), (16, 1, 64, BF), (4, 4, 32, F32)], ids=str)
@pytest.mark.parametrize("pack", range(len(G.PACKS)))
def test_packs(pack, heads):
    G.test_prompt(pack, heads, "auto")


@pytest.mark.parametrize("heads", [(4, 1, 128, BF), (80, 2, 128, BF), (2, 1, 64, F32)], ids=str)
def test_longer_prompts(heads):
    G.test_prompt_longer(heads)


@pytest.mark.parametrize("heads", [(8, 2, 128, BF), (6, 2, 128, BF), (8, 8, 64, F32)], ids=str)
@pytest.mark.parametrize("chain", [True, False])
def test_trees(chain, heads):
    G.test_tree(chain, heads, "auto")


@pytest.mark.parametrize("heads,nodes,prefixes", [((64, 1, 128), [1, 1], [20000, 3000]),
                                                  ((16, 1, 64), [40, 3], [8000, 200]),
                                                  ((32, 8, 128), [16, 30, 8], [3000, 1000, 9000])], ids=str)
def test_cut_rows(heads, nodes, prefixes):
    G.test_rows_cut_into_many_runs(heads, nodes, prefixes)


@pytest.mark.parametrize("ql,kl,heads", [([70, 500, 3], [900, 500, 1500], (128, 1, 64)), ([4000], [4000], (32, 8, 128)),
                                         ([20, 7, 1], [300, 20000, 4000], (24, 4, 64)), ([30], [5000], (24, 4, 64)),
                                         ([1] * 40, [3000] * 40, (8, 2, 128))], ids=str)
def test_runs(ql, kl, heads):
    G.test_runs_of_many_segments(ql, kl, heads)


@pytest.mark.parametrize("heads", [(8, 2, 128), (40, 1, 128)], ids=str)
@pytest.mark.parametrize("rows", [1, 40, 700])
def test_selected_rows(rows, heads):
    G.test_selected_few_and_many_rows(rows, heads, "auto")


@pytest.mark.parametrize("kind", ["causal", "twice", "bad_ids"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (12, 2, 128)], ids=str)
def test_selected_prompts(heads, kind):
    G.test_selected_whole_prompt(kind, heads)


def test_errors_and_empty_calls():
    G.test_device_errors_are_reported()
    G.test_no_keys_at_all()
    G.test_tree_rows_that_see_nothing("auto")
