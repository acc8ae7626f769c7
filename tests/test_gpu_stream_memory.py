"""Calls on another stream that allocate their own workspace and outputs: no memory that the current stream
still uses is written, and none of theirs is handed out before their kernels are done."""
import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import attention_reference as A
from tests.test_gpu_attention import BF, i32, make

pytestmark = pytest.mark.gpu
HEADS, ROWS, TOKENS, SCALE = (8, 2, 128), 40, 3000, 0.1
BUSY = 100_000_000      # clock cycles, tens of milliseconds


@pytest.fixture
def case():
    q, k, v = make(3, ROWS, TOKENS, HEADS, BF)
    return q, k, v, i32([0, ROWS]), i32([0, TOKENS]), A.reference(q, k, v, A.see_prompt([ROWS], [TOKENS]), SCALE)


@pytest.fixture
def workspaces(monkeypatch):
    made, new = [], K.new_attention_workspace

    def keep(*a, **kw):
        t = new(*a, **kw)
        made.append((t.data_ptr(), t.numel()))
        return t
    monkeypatch.setattr(K, "new_attention_workspace", keep)
    return made


def raw(stream, as_handle):
    return stream.cuda_stream if as_handle else stream


@pytest.mark.parametrize("as_handle", [False, True], ids=["stream", "handle"])
def test_its_memory_is_not_handed_out_while_it_runs(as_handle, case, workspaces):
    q, k, v, cq, ck, ref = case
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    out, lse = K.kpool_attention_prompt(q, k, v, cq, ck, SCALE, return_lse=True, stream=raw(side, as_handle))
    (at, size), = workspaces
    others = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert all(t.data_ptr() + size <= at or at + size <= t.data_ptr() for t in others)
    side.synchronize()
    A.check(out, lse, ref)


def test_memory_that_the_current_stream_still_reads_is_not_taken(case, workspaces):
    q, k, v, cq, ck, ref = case
    side = torch.cuda.Stream()
    size = K.load().kpool_attention_workspace_bytes(ROWS, 1, K._attention_shape(*HEADS, BF, SCALE))
    mine = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
    kept = torch.empty_like(mine)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    kept.copy_(mine)
    del mine                          # free for the current stream's later work, which follows the copy
    out, lse = K.kpool_attention_prompt(q, k, v, cq, ck, SCALE, return_lse=True, stream=side)
    torch.cuda.synchronize()
    assert workspaces[0][1] == size and (kept == 7).all()
    A.check(out, lse, ref)


def test_outputs_outlive_the_call_for_the_current_stream(case):
    """A result read on the current stream and dropped is not written by the side stream's next call."""
    q, k, v, cq, ck, ref = case
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = K.kpool_attention_prompt(q, k, v, cq, ck, SCALE, return_lse=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    other = q * 0.5
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    kept, kept_lse = out.clone(), lse.clone()
    del out, lse
    K.kpool_attention_prompt(other, k, v, cq, ck, SCALE, return_lse=True, stream=side)
    torch.cuda.synchronize()
    A.check(kept, kept_lse, ref)
