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


def _other_allocator(conf):
    """In a process of its own under PYTORCH_CUDA_ALLOC_CONF=conf: pools of many mapped pieces serve, and an
    extent that ends behind what is mapped is refused."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, PYTORCH_CUDA_ALLOC_CONF=conf, PYTHONPATH=root)
    code = "from tests.test_gpu_serving_callers import _allocator_child; _allocator_child()"
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


def _allocator_child():
    import ctypes
    import math

    from temporal_block_sparse_sm_b200 import liteattn, serving
    from tests.serving_ref import assert_close, seq_reference
    Hq, Hk, d, page, n, pages = 8, 2, 128, 64, 300, 4096           # pools of 134 MB
    q, k, v = (_randn(n, h, d, seed=i) for i, h in enumerate((Hq, Hk, Hk)))
    plan = serving.GroupedPlan(Hq, Hk, d)
    cache = serving.PagedCache(plan, *(torch.zeros(pages, Hk, page, d, dtype=BF16, device="cuda") for _ in range(2)))
    lens, cu = _ints(n), offsets([n])
    table = torch.tensor([[pages - 1, 0, 7, 2000, 999]], dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    cache.append(k, v, lens, cu, table)
    cache.attend(q, o, lens, cu, table, max_new=n)
    plan.check()
    assert_close(o, *seq_reference(q, k, v, True, 1 / math.sqrt(d)))
    # keys said to be 2^27 tokens long, 64 GiB: behind the memory of this process
    rows = lambda t, tokens: liteattn.Rows(t.data_ptr(), tokens, t.stride(0), t.stride(1))   # noqa: E731
    before = liteattn.lite_attn_launch_count()
    for tokens in (1 << 27, 1 << 28):
        ws = torch.empty(liteattn.lite_attn_gqa_workspace(plan.handle, 1, n, n, tokens), dtype=torch.uint8, device="cuda")
        args = liteattn.PromptArgs(q=rows(q, n), o=rows(o, n), k=rows(k, tokens), v=rows(v, tokens), cu_q=cu.data_ptr(), cu_k=cu.data_ptr(),
                                   workspace=ws.data_ptr(), workspace_bytes=ws.numel(), B=1, causal=1, scale=0.1)
        rc = liteattn.load().lite_attn_prompt(plan.handle, ctypes.addressof(args), None)
        assert rc == liteattn.LITE_ERR_INVALID_ARG, rc
    assert liteattn.lite_attn_launch_count() == before
    print("ok")


@pytest.mark.parametrize("conf", ["expandable_segments:False", "expandable_segments:True", "backend:cudaMallocAsync"])
def test_memory_of_other_allocators(conf):
    _other_allocator(conf)
