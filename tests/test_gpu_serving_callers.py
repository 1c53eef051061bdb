"""Serving attention called in other ways than from the main thread on memory of the default allocator:
other threads, other allocators, the C ABI's own binding, and arguments that only such callers can pass."""
from __future__ import annotations

import threading

import pytest
import torch

from tests.serving_ref import offsets

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from temporal_block_sparse_sm_b200 import build, liteattn
    build.build()
    liteattn.load()


def _randn(*shape, dtype=BF16, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def _ints(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _in_new_thread(fn):
    """fn in a thread that has never used CUDA; what it raised is raised here."""
    raised = []

    def run():
        try:
            fn()
        except BaseException as e:
            raised.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    if raised:
        raise raised[0]


@pytest.mark.parametrize("call", ["prompt", "append", "attend", "step"])
def test_first_call_of_a_thread(call):
    """A thread's first use of CUDA is a call on tensors that other threads made."""
    from temporal_block_sparse_sm_b200 import liteattn, serving
    q, k, v = (_randn(100, h, 128, seed=h) for h in (8, 2, 3))
    v = v[:, :2]
    plan, lens, cu, table = serving.GroupedPlan(8, 2, 128), _ints(100), offsets([100]), _ints([0, 1])
    cache = serving.PagedCache(plan, *(torch.zeros(2, 2, 64, 128, dtype=BF16, device="cuda") for _ in range(2)))
    cache.append(k, v, lens, cu, table)
    step = liteattn.Plan(1, 2, 1024, 128, 128, 128, [-10.0])
    x = _randn(3, 1, 2, 1024, 128)
    outs = []

    def run():
        o = outs[-1]
        if call == "prompt":
            plan.prompt(q, k, v, o, cu, stream=0)
        elif call == "append":
            cache.append(k, v, lens, cu, table, q=q, q_out=o, stream=0)
        elif call == "attend":
            cache.attend(q, o, lens, cu, table, max_new=100, stream=0)
        else:
            step.step(x[0], x[1], x[2], o, masks[len(outs) - 1], masks[len(outs) - 1], 0, stream=0)
    masks = [step.mask(), step.mask()]
    for way in (lambda f: f(), _in_new_thread):
        outs.append(torch.full_like(x[0] if call == "step" else q, 7.0))
        torch.cuda.synchronize()
        way(run)
        torch.cuda.synchronize()
    plan.check()
    assert torch.equal(outs[0], outs[1]) and not bool((outs[1] == 7).all())
