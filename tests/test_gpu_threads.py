"""Calls of different sizes from two host threads: each launch gets the shared memory that it needs, whatever
another thread's calls of the same kernel need."""
import threading

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import attention_reference as A
from tests.test_gpu_attention import BF, F32, i32, make

pytestmark = pytest.mark.gpu


def both(first, second, calls):
    """Runs the two functions `calls` times each, side by side; their exceptions."""
    errors, gate = [], threading.Barrier(2)

    def loop(call):
        try:
            gate.wait(timeout=30)
            for _ in range(calls):
                call()
        except Exception as e:  # noqa: BLE001 (whatever it is, the test shows it)
            errors.append(e)
    threads = [threading.Thread(target=loop, args=(c,)) for c in (first, second)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


@pytest.mark.parametrize("dtype,dims", [(F32, (64, 128)), (BF, (32, 120)), (F32, (160, 256))], ids=str)
def test_cuda_core_attention_of_two_head_sizes(dtype, dims):
    jobs = []
    for d in dims:
        heads = (4, 2, d)
        q, k, v = make(d, 5, 70, heads, dtype)
        ws = K.new_attention_workspace(5, 1, *heads, dtype)
        out, lse = torch.empty_like(q), torch.empty((5, 4), device="cuda")
        cq, ck, stream = i32([0, 5]), i32([0, 70]), torch.cuda.Stream()
        ref = A.reference(q, k, v, A.see_prompt([5], [70]), 0.1)

        def call(q=q, k=k, v=v, cq=cq, ck=ck, out=out, lse=lse, ws=ws, stream=stream):
            K.kpool_attention_prompt(q, k, v, cq, ck, 0.1, out=out, out_lse=lse, workspace=ws, stream=stream)
        jobs.append((call, out, lse, ref))
    torch.cuda.synchronize()
    assert both(jobs[0][0], jobs[1][0], 30000) == []
    for _, out, lse, ref in jobs:
        A.check(out, lse, ref)


def test_cuda_core_selection_of_two_budgets():
    """64 KB of shared memory a block on one side, 96 KB on the other."""
    jobs = []
    for budget in (1000, 2000):
        T, H, d = 3, 2, 64
        g = torch.Generator().manual_seed(budget)
        q, k = torch.randn((T, H, d), generator=g).cuda(), torch.randn((T, d), generator=g).cuda()
        w, cu = torch.rand((T, H), generator=g).cuda(), i32([0, T])
        want = K.kpool_select_ex(q, k, w, cu, 1, budget, 0.1, score_kernel=K.KPOOL_SCORE_SIMT)
        ids, toks = (torch.empty_like(t) for t in want[:2])
        ws = K.new_workspace(T, 1, H, d, K.KPOOL_F32, 1, budget)
        stream = torch.cuda.Stream()

        def call(q=q, k=k, w=w, cu=cu, budget=budget, ids=ids, toks=toks, ws=ws, stream=stream):
            K.kpool_select_ex(q, k, w, cu, 1, budget, 0.1, out_pool_ids=ids, out_token_ids=toks, workspace=ws,
                              stream=stream, score_kernel=K.KPOOL_SCORE_SIMT)
        jobs.append((call, ids, toks, want))
    torch.cuda.synchronize()
    assert both(jobs[0][0], jobs[1][0], 3000) == []
    for _, ids, toks, want in jobs:
        assert torch.equal(ids, want[0]) and torch.equal(toks, want[1])
