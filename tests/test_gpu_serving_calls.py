"""Rotary, paged and latent calls side by side: two host threads, graphs that share a workspace, calls that allocate for
themselves on another stream, and one workspace for calls of different operators and sizes in a row."""
import math
import random

import pytest
import torch

from sparse_attention_kpool_gb300 import kpool as K
from tests import attention_reference as A
from tests import serving_reference as S
from tests.test_gpu_threads import both

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
BUSY = 100_000_000      # clock cycles, tens of milliseconds


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Paged:
    """A decode step and what it has to give."""

    def __init__(self, lengths, page, heads, seed, dtype=BF):
        hq, hkv, d = heads
        total, table = S.pool(lengths, page, random.Random(seed))
        g = torch.Generator().manual_seed(seed)
        self.q = (torch.randn((len(lengths), hq, d), generator=g) * 2).to(dtype).cuda()
        self.k = torch.randn((total, page, hkv, d), generator=g).to(dtype).cuda()
        self.v = torch.randn((total, page, hkv, d), generator=g).to(dtype).cuda()
        self.table, self.lengths = table.cuda(), i32(lengths)
        see = S.see_paged(table, lengths, page, [1] * len(lengths))
        self.ref = S.attend(self.q, self.k.flatten(0, 1), self.v.flatten(0, 1), see, 0.1)
        self.out, self.lse = torch.empty_like(self.q), torch.empty((len(lengths), hq), device="cuda")
        self.size = (len(lengths), len(lengths), *heads, dtype)

    def workspace(self):
        return K.new_attention_workspace(*self.size)

    def __call__(self, **kw):
        return K.kpool_attention_paged(self.q, self.k, self.v, self.table, self.lengths, 0.1,
                                       **{"out": self.out, "out_lse": self.lse, **kw})


class Latent:
    def __init__(self, lengths, page, heads, seed, dims=(512, 64), dtype=BF):
        total, table = S.pool(lengths, page, random.Random(seed))
        g = torch.Generator().manual_seed(seed)
        self.q = (torch.randn((len(lengths), heads, sum(dims)), generator=g) * 1.2).to(dtype).cuda()
        self.cache = torch.randn((total, page, sum(dims)), generator=g).to(dtype).cuda()
        self.table, self.lengths, self.dim = table.cuda(), i32(lengths), dims[0]
        flat = self.cache.reshape(-1, 1, sum(dims))
        self.ref = S.attend(self.q, flat, flat[..., :dims[0]], S.slots(table, lengths, page), 0.07)
        self.out = torch.empty((len(lengths), heads, dims[0]), dtype=dtype, device="cuda")
        self.lse = torch.empty((len(lengths), heads), device="cuda")
        self.size = (len(lengths), len(lengths), heads, *dims, dtype)

    def workspace(self):
        return K.new_latent_workspace(*self.size)

    def __call__(self, **kw):
        return K.kpool_attention_latent(self.q, self.cache, self.table, self.lengths, self.dim, 0.07,
                                        **{"out": self.out, "out_lse": self.lse, **kw})


def jobs():
    return [Paged([3000, 5, 800], 16, (8, 2, 128), 1), Paged([70, 0], 24, (4, 2, 64), 2), Latent([4000, 90], 64, 32, 3),
            Latent([200], 16, 80, 4), Paged([90], 8, (4, 4, 32), 5, F32), Latent([60, 7], 16, 3, 6, (64, 16), F32)]


def clear(job):
    job.out.fill_(math.nan)
    job.lse.fill_(math.nan)


@pytest.mark.parametrize("pair", [(0, 1), (2, 3), (4, 5), (0, 2)], ids=str)
def test_two_threads(pair):
    made = jobs()
    two = [made[i] for i in pair]
    calls = []
    for job in two:
        ws, stream = job.workspace(), torch.cuda.Stream()
        calls.append(lambda job=job, ws=ws, stream=stream: job(workspace=ws, stream=stream))
    torch.cuda.synchronize()
    assert both(*calls, 3000) == []
    for job in two:
        A.check(job.out, job.lse, job.ref)


def test_tensor_core_calls_of_a_thread_that_has_made_no_others():
    """A thread's first call on the GPU is one that makes tensor maps."""
    import threading
    q, kv = torch.randn((40, 8, 128), device="cuda").to(BF), torch.randn((90, 2, 128), device="cuda").to(BF)
    cq, ck = i32([0, 40]), i32([0, 90])
    ws, out = K.new_attention_workspace(40, 1, 8, 2, 128, BF), torch.empty_like(q)
    want, _ = K.kpool_attention_prompt(q, kv, kv, cq, ck, 0.1)
    stream, errors = torch.cuda.current_stream().cuda_stream, []
    torch.cuda.synchronize()

    def call():
        try:
            K.kpool_attention_prompt(q, kv, kv, cq, ck, 0.1, out=out, workspace=ws, stream=stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    t = threading.Thread(target=call)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert errors == [] and torch.equal(out, want)


def test_rotary_from_two_threads():
    sides = []
    for dim, dtype in ((128, BF), (40, F32)):
        x, pos = torch.randn((30, 4, dim), device="cuda").to(dtype), torch.arange(30, dtype=torch.int32, device="cuda")
        table, stream = K.new_rotary_table(dim), torch.cuda.Stream()
        want, _ = K.kpool_rotary(x, pos, table)
        out = torch.empty_like(x)
        sides.append((lambda x=x, pos=pos, table=table, out=out, stream=stream:
                      K.kpool_rotary(x, pos, table, out_q=out, stream=stream), out, want))
    torch.cuda.synchronize()
    assert both(sides[0][0], sides[1][0], 3000) == []
    assert all(torch.equal(out, want) for _, out, want in sides)


def test_one_workspace_for_calls_in_a_row():
    """Every operator in turn, large and small, on one workspace that holds what the call before left."""
    made = jobs()
    ws = max((job.workspace() for job in made), key=lambda t: t.numel())
    for _ in range(2):
        for job in made + made[::-1]:
            clear(job)
            job(workspace=ws)
            assert K.kpool_last_device_error(ws) == K.KPOOL_OK
            A.check(job.out, job.lse, job.ref)


def test_two_graphs_share_a_workspace():
    made = jobs()[:4]
    ws = max((job.workspace() for job in made), key=lambda t: t.numel())
    for job in made:
        job(workspace=ws)
    graphs = []
    for job in made:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            job(workspace=ws)
        graphs.append(g)
    for order in ([0, 1, 2, 3], [3, 2, 1, 0], [2, 0, 3, 1]):
        for job in made:
            clear(job)
        ws.fill_(0xA5)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for job in made:
            A.check(job.out, job.lse, job.ref)


@pytest.mark.parametrize("which", [0, 2])
def test_memory_of_a_call_on_another_stream(which):
    """It allocates its workspace and outputs; nobody gets them while it waits behind other work."""
    job = jobs()[which]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    out, lse = job(out=None, out_lse=None, return_lse=True, stream=side)
    others = [torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(40)]
    side.synchronize()
    A.check(out, lse, job.ref)
    del others
