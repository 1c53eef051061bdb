"""Serving attention called in other ways than from the main thread on memory of the default allocator:
other threads, other allocators, the C ABI's own binding, and arguments that only such callers can pass."""
from __future__ import annotations

import threading

import pytest
import torch

from tests.serving_ref import assert_close, offsets, seq_reference

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


# ---------------------------------------------------------------- inputs and outputs in one another's memory
def _append_args(T=6, Hq=4, Hk=2, d=64, dtype=BF16):
    from temporal_block_sparse_sm_b200 import serving
    plan = serving.GroupedPlan(Hq, Hk, d, dtype=dtype)
    pools = [torch.zeros(2, Hk, 16, d, dtype=dtype, device="cuda") for _ in range(2)]
    cos, sin = serving.rotation_table(range(40), [0.3 * i + 0.1 for i in range(d // 2)], device="cuda")
    return plan, serving.PagedCache(plan, *pools), pools, dict(lens=_ints(T), cu_new=offsets([T]), table=_ints(1, 0).view(1, 2), cos=cos, sin=sin)


def test_queries_rotated_in_place_must_not_be_keys_or_values():
    """q_out == q, and k or v reads some of the elements that are written."""
    from temporal_block_sparse_sm_b200 import liteattn
    plan, cache, pools, kw = _append_args()
    x = _randn(9, 8, 64)
    q, other = x[1:7, 1:5], _randn(6, 2, 64)
    per_head = _randn(6, 4, 2, 64)                # [token][head][a, b]
    heads_first = _randn(4, 8, 64).transpose(0, 1)
    cases = [(q, x[1:7, 1:3]), (q, x[1:7, 4:6]), (q, x[1:7, 0:2]), (q, x[2:8, 3:5]), (q, x[0:6, 2:4]),
             (q, x[1:7, 0:8:4]), (per_head[:, :, 0], per_head[:, 1:3, 0]), (heads_first[:6], heads_first[2:, 1:3]),
             (q, x.flatten()[512 + 320 - 32:].as_strided((6, 2, 64), (512, 64, 1))),
             (q, x.flatten()[512 + 64:].as_strided((6, 2, 64), (384, 64, 1)))]
    before = liteattn.lite_attn_launch_count()
    for i, (a, b) in enumerate(cases):
        for k, v in ((b, other), (other, b)):
            with pytest.raises(liteattn.LiteAttnError) as e:
                cache.append(k, v, q=a, q_out=a, **kw)
            assert e.value.code == liteattn.LITE_ERR_INVALID_ARG, i
    assert liteattn.lite_attn_launch_count() == before


@pytest.mark.parametrize("T", [1, 6])
@pytest.mark.parametrize("form", ["fused", "per head", "heads first", "apart", "pieces of a wide row"])
def test_queries_rotated_in_place_between_keys_and_values(form, T):
    """The same elements' neighbours are fine: slices of one projection, whatever their order in it."""
    Hq, Hk, d = (4, 4, 64) if form == "per head" else (4, 2, 64)
    plan, cache, pools, kw = _append_args(T, Hq, Hk)
    if form == "fused":
        q, k, v = _randn(T, Hq + 2 * Hk, d).split([Hq, Hk, Hk], dim=1)
    elif form == "per head":
        q, k, v = _randn(T, Hq, 3, d).unbind(2)
    elif form == "heads first":
        q, k, v = _randn(Hq + 2 * Hk, T, d).transpose(0, 1).split([Hq, Hk, Hk], dim=1)
    elif form == "apart":
        q, k, v = (_randn(T, h, d, seed=h + i) for i, h in enumerate((Hq, Hk, Hk)))
    else:
        x = _randn(T, 40, d)
        k, q, v = x[:, 3:3 + Hk], x[:, 10:10 + 3 * Hq:3], x[:, 11:11 + 4 * Hk:6][:, :Hk]
    want_q, saved = torch.empty(T, Hq, d, dtype=BF16, device="cuda"), (q.clone(), k.clone(), v.clone())
    cache.append(k, v, q=saved[0], q_out=want_q, **kw)
    want_pools = [p.clone() for p in pools]
    for p in pools:
        p.zero_()
    cache.append(k, v, q=q, q_out=q, **kw)
    plan.check()
    assert torch.equal(q, want_q) and torch.equal(k, saved[1]) and torch.equal(v, saved[2])
    assert all(torch.equal(a, b) for a, b in zip(pools, want_pools))
    assert torch.equal(q, saved[0]) == (T == 1)        # position 0 turns by angles of 0: cos 1, sin 0


def _rows(t):
    from temporal_block_sparse_sm_b200 import liteattn
    return liteattn.Rows(t.data_ptr(), t.shape[0], t.stride(0), t.stride(1))


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("call", ["attend", "prompt"])
def test_a_workspace_over_other_arguments_is_refused(call, new):
    """Through the C ABI's binding, with a workspace in an allocation that holds an argument as well: behind
    it, which is fine, and reaching into it from either side."""
    import ctypes

    from temporal_block_sparse_sm_b200 import liteattn, serving
    Hq, Hk, d, m, page, pages = 4, 1, 64, 20000, 64, 320
    plan = serving.GroupedPlan(Hq, Hk, d)
    bytes_ = liteattn.lite_attn_gqa_workspace(plan.handle, 1, new, new, pages * page if call == "attend" else m)
    assert bytes_ > 0
    made = dict(q=_randn(new, Hq, d), o=torch.full((new, Hq, d), 7.0, dtype=BF16, device="cuda"), cu_q=offsets([new]))
    if call == "attend":
        made.update(k=_randn(pages, Hk, page, d), v=_randn(pages, Hk, page, d, seed=1), lens=_ints(m),
                    table=torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages))
    else:
        made.update(k=_randn(m, Hk, d), v=_randn(m, Hk, d, seed=1), cu_k=offsets([m]))

    def run(t, ws):
        if call == "attend":
            args = liteattn.AttendArgs(q=_rows(t["q"]), o=_rows(t["o"]), k_pages=t["k"].data_ptr(), v_pages=t["v"].data_ptr(), pages=pages,
                                       cu_new=t["cu_q"].data_ptr(), lens=t["lens"].data_ptr(), table=t["table"].data_ptr(), workspace=ws,
                                       workspace_bytes=bytes_, B=1, table_width=pages, page=page, layout=0, max_new=new, causal=1, scale=0.125)
            liteattn.lite_attn_cache_attend(plan.handle, ctypes.addressof(args))
        else:
            args = liteattn.PromptArgs(q=_rows(t["q"]), o=_rows(t["o"]), k=_rows(t["k"]), v=_rows(t["v"]), cu_q=t["cu_q"].data_ptr(),
                                       cu_k=t["cu_k"].data_ptr(), workspace=ws, workspace_bytes=bytes_, B=1, causal=1, scale=0.125)
            liteattn.lite_attn_prompt(plan.handle, ctypes.addressof(args))

    own = torch.empty(bytes_, dtype=torch.uint8, device="cuda")
    run(made, own.data_ptr())
    plan.check()
    want = made["o"].clone()
    for name, t in made.items():
        size = -(-t.numel() * t.element_size() // 256) * 256
        pad = -(-bytes_ // 256) * 256
        flat = torch.zeros(2 * pad + size, dtype=torch.uint8, device="cuda")
        inside = flat[pad:pad + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        inside.copy_(t)
        moved = dict(made, **{name: inside})
        used = t.numel() * t.element_size()
        run(moved, flat.data_ptr() + pad + size)
        run(moved, flat.data_ptr() + pad - (bytes_ + 15) // 16 * 16)
        plan.check()
        assert torch.equal(moved["o"], want), name
        before = liteattn.lite_attn_launch_count()
        for at in (pad - (bytes_ - 1) // 16 * 16, pad, pad + (used - 1) // 16 * 16):
            with pytest.raises(liteattn.LiteAttnError) as e:
                run(moved, flat.data_ptr() + at)
            assert e.value.code == liteattn.LITE_ERR_INVALID_ARG, (name, at)
        assert liteattn.lite_attn_launch_count() == before


@pytest.mark.parametrize("new", [1, 40])
def test_scales_at_the_end_of_the_range(new):
    """The kernels' factor is scale * log2 e: a scale whose factor is no 32-bit number is refused, and the
    largest others give what they say on logits that are 0 or small."""
    from temporal_block_sparse_sm_b200 import liteattn, serving
    plan, Hq, Hk, d = serving.GroupedPlan(4, 2, 64), 4, 2, 64
    q, k, v = torch.zeros(new, Hq, d, dtype=BF16, device="cuda"), _randn(200, Hk, d), _randn(200, Hk, d, seed=1)
    o, cu_q, cu_k = torch.empty_like(q), offsets([new]), offsets([200])
    before = liteattn.lite_attn_launch_count()
    for scale in (2.4e38, 3.4e38):
        with pytest.raises(liteattn.LiteAttnError) as e:
            plan.prompt(q, k, v, o, cu_q, cu_k, scale=scale)
        assert e.value.code == liteattn.LITE_ERR_INVALID_ARG
    assert liteattn.lite_attn_launch_count() == before
    for factor, scale in ((0.0, 2.3e38), (2.0 ** -120, 2.0 ** 117), (2.0 ** -120, 2.0 ** 120)):
        q.fill_(factor)
        plan.prompt(q, k, v, o, cu_q, cu_k, scale=scale, causal=False)
        plan.check()
        want, tol = seq_reference(q, k, v, False, scale)
        assert_close(o, want, tol, f"scale {scale}")


def test_outputs_over_lengths_offsets_tables_and_angles_are_refused():
    from temporal_block_sparse_sm_b200 import liteattn, serving
    Hq, Hk, d, T = 4, 2, 64, 6
    plan, cache, pools, kw = _append_args(T)
    q, k, v = (_randn(T, h, d, seed=h + i) for i, h in enumerate((Hq, Hk, Hk)))
    kw["positions"] = torch.zeros(T, dtype=torch.int32, device="cuda")
    before = liteattn.lite_attn_launch_count()

    def within(host, t):
        """t's values in the memory of host, somewhere in its middle."""
        flat = host.flatten().view(torch.uint8)
        at = flat.numel() // 2 // 16 * 16
        out = flat[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        out.copy_(t)
        return out

    for name in ("lens", "cu_new", "table", "positions"):
        out = torch.zeros(T, Hq, d, dtype=BF16, device="cuda")
        for host in (out, pools[0], pools[1]):
            with pytest.raises(liteattn.LiteAttnError) as e:
                cache.append(k, v, q=q, q_out=out, **dict(kw, **{name: within(host, kw[name])}))
            assert e.value.code == liteattn.LITE_ERR_INVALID_ARG, name
        if name != "positions":
            args = dict(lens=kw["lens"], cu_new=kw["cu_new"], table=kw["table"])
            with pytest.raises(liteattn.LiteAttnError):
                cache.attend(q, out, max_new=T, **dict(args, **{name: within(out, kw[name])}))
    wide = torch.zeros(64, Hq, d, dtype=BF16, device="cuda")
    for name in ("cos", "sin"):
        with pytest.raises(liteattn.LiteAttnError):
            cache.append(_randn(64, Hk, d), _randn(64, Hk, d), q=_randn(64, Hq, d), q_out=wide,
                         **dict(kw, lens=_ints(32), cu_new=offsets([32]), positions=torch.zeros(64, dtype=torch.int32, device="cuda"),
                                **{name: within(wide, kw[name])}))
    out = torch.zeros(T, Hq, d, dtype=BF16, device="cuda")
    for name in ("cu_q", "cu_k"):
        with pytest.raises(liteattn.LiteAttnError):
            plan.prompt(q, k, v, out, **dict(dict(cu_q=offsets([T]), cu_k=offsets([T])), **{name: within(out, offsets([T]))}))
    assert liteattn.lite_attn_launch_count() == before


@pytest.mark.parametrize("way", ["data", "attribute", "set_"])
def test_pages_that_get_other_memory(way):
    """The caller's page tensors move to other memory (with another number of pages) after the cache was made:
    calls go to where they are; tensors that are no pages of this plan any more are refused."""
    from temporal_block_sparse_sm_b200 import serving
    Hq, Hk, d, T = 4, 2, 64, 20
    q, k, v = (_randn(T, h, d, seed=h + i) for i, h in enumerate((Hq, Hk, Hk)))
    plan = serving.GroupedPlan(Hq, Hk, d)
    first, fresh, wrong = ([torch.zeros(*s, dtype=BF16, device="cuda") for _ in range(2)] for s in ((8, Hk, 16, d), (3, Hk, 32, d), (8, Hk, 16, 2 * d)))
    cache = serving.PagedCache(plan, *first)
    lens, cu, o = _ints(T), offsets([T]), [torch.empty_like(q) for _ in range(2)]
    cache.append(k, v, lens, cu, _ints(7, 2).view(1, 2))
    cache.attend(q, o[0], lens, cu, _ints(7, 2).view(1, 2), max_new=T)
    plan.check()
    kept, old = [x.clone() for x in first], [x.detach() for x in first]

    def move(tensors):
        for name, x in zip(("k_pages", "v_pages"), tensors):
            if way == "attribute":
                setattr(cache, name, x)
            elif way == "data":
                getattr(cache, name).data = x
            else:
                getattr(cache, name).set_(x)
    move(fresh)
    cache.append(k, v, lens, cu, _ints(2).view(1, 1))
    cache.attend(q, o[1], lens, cu, _ints(2).view(1, 1), max_new=T)
    plan.check()
    want, tol = seq_reference(q, k, v, True, d ** -0.5)
    for x in o:
        assert_close(x, want, tol)
    assert all(torch.equal(a, b) for a, b in zip(old, kept)), "the memory of before was written"
    move(wrong)
    with pytest.raises(ValueError):
        cache.append(k, v, lens, cu, _ints(2).view(1, 1))
    with pytest.raises(ValueError):
        cache.attend(q, o[0], lens, cu, _ints(2).view(1, 1), max_new=T)


def _first_calls_child():
    """The library's first serving calls in the process are captured, and run when the graph is replayed."""
    from temporal_block_sparse_sm_b200 import serving
    Hq, Hk, d, T, page = 8, 2, 128, 70, 16
    plan = serving.GroupedPlan(Hq, Hk, d)
    q, k, v = (_randn(T, h, d, seed=h + i) for i, h in enumerate((Hq, Hk, Hk)))
    cache = serving.PagedCache(plan, *(torch.zeros(200, Hk, page, d, dtype=BF16, device="cuda") for _ in range(2)))
    lens, cu, one = _ints(T), offsets([T]), offsets([1])
    table = torch.arange(199, -1, -1, dtype=torch.int32, device="cuda").view(1, 200)
    outs = [torch.full_like(q, 7.0) for _ in range(2)] + [torch.full_like(q[:1], 7.0)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan.prompt(q, k, v, outs[0], cu)
        cache.append(k, v, lens, cu, table)
        cache.attend(q, outs[1], lens, cu, table, max_new=T)
        cache.attend(q[-1:], outs[2], lens, one, table, max_new=1)
    graph.replay()
    plan.check()
    want, tol = seq_reference(q, k, v, True, d ** -0.5)
    for o, rows in zip(outs, (slice(0, T), slice(0, T), slice(T - 1, T))):
        assert_close(o, want[rows], tol[rows])
    print("ok")


def test_the_first_calls_of_a_process_are_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = "from tests.test_gpu_serving_callers import _first_calls_child; _first_calls_child()"
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, PYTHONPATH=root), cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


@pytest.mark.parametrize("stream_of", ["argument", "current"])
def test_calls_on_a_forked_stream_of_a_capture(stream_of):
    """A capture that forks to a second stream and joins it again, both with calls that need a workspace: the
    graph's replays are right while other work takes the allocator's free memory."""
    from temporal_block_sparse_sm_b200 import serving
    Hq, Hk, d, page, m = 4, 1, 64, 64, 20000
    plan = serving.GroupedPlan(Hq, Hk, d)
    cache = serving.PagedCache(plan, _randn(320, Hk, page, d), _randn(320, Hk, page, d, seed=1))
    table, lens = torch.arange(320, dtype=torch.int32, device="cuda").view(1, 320), _ints(m)
    qs = [_randn(n, Hq, d, seed=n) for n in (1, 60)]
    outs, cus = [torch.empty_like(q) for q in qs], [offsets([q.shape[0]]) for q in qs]
    call = lambda i, s=None: cache.attend(qs[i], outs[i], lens, cus[i], table, max_new=qs[i].shape[0], stream=s)   # noqa: E731
    call(0), call(1)
    plan.check()
    want = [o.clone() for o in outs]
    main, side, graph = torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        if stream_of == "argument":
            call(0, side)
        else:
            with torch.cuda.stream(side):
                call(0)
        call(1)
        main.wait_stream(side)
    for _ in range(5):
        for o in outs:
            o.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        junk = [torch.full((n,), float("nan"), device="cuda") for n in (1 << 10, 1 << 16, 1 << 20, 1 << 23)]
        with torch.cuda.stream(side):
            junk += [torch.full((n,), float("nan"), device="cuda") for n in (1 << 10, 1 << 16, 1 << 20, 1 << 23)]
        torch.cuda.synchronize()
        del junk
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    plan.check()


@pytest.mark.parametrize("heads_first", [False, True])
def test_packed_rows_far_into_large_tensors(heads_first):
    """q, k, v and o of over 2^31 elements each, the sequences in their last rows: offsets beyond 32 bits, in both
    kernels, in the rotation, and where a value that is not finite is looked up again."""
    import math

    from temporal_block_sparse_sm_b200 import serving
    Hq, Hk, d, n, m = 2, 1, 128, 60, 300
    T = (1 << 31) // d + 1000                   # tokens of one head
    def big(heads):
        shape = (heads, T // heads, d) if heads_first else (T // heads, heads, d)
        x = torch.empty(shape, dtype=BF16, device="cuda")
        return x.transpose(0, 1) if heads_first else x
    q, o, k, v = big(Hq), big(Hq), big(Hk), big(Hk)
    tq, tk = q.shape[0], k.shape[0]
    q[-n:], k[-m:], v[-m:] = _randn(n, Hq, d), _randn(m, Hk, d, seed=1), _randn(m, Hk, d, seed=2)
    o[-n - 1:] = 7
    v[-10, 0, 3] = math.inf                     # seen by the last rows only
    plan = serving.GroupedPlan(Hq, Hk, d)
    cu_q, cu_k = torch.tensor([tq - n, tq], dtype=torch.int32, device="cuda"), torch.tensor([tk - m, tk], dtype=torch.int32, device="cuda")
    plan.prompt(q, k, v, o, cu_q, cu_k)
    plan.check()
    want, tol = seq_reference(q[-n:], k[-m:], v[-m:], True, d ** -0.5)
    assert_close(o[-n:], want, tol)
    assert bool((o[-n - 1] == 7).all())
    # the same rows into a cache, turned by nothing, and attended over by few rows and by many
    pools = [torch.zeros(5, Hk, 64, d, dtype=BF16, device="cuda") for _ in range(2)]
    cache, table = serving.PagedCache(plan, *pools), _ints(4, 2, 0, 1, 3).view(1, 5)
    kq = big(Hq)                                # queries beside the new keys: as many rows
    cu = torch.tensor([tq - m, tq], dtype=torch.int32, device="cuda")
    kq[-m:] = _randn(m, Hq, d, seed=3)
    o[-m:] = 7
    cos, sin = serving.rotation_table([0] * m, [1.0] * (d // 2), device="cuda")
    cache.append(k[tk - tq:], v[tk - tq:], _ints(m), cu, table, q=kq, q_out=o, cos=cos, sin=sin)
    plan.check()
    assert torch.equal(o[-m:], kq[-m:])
    for rows in (2, n):
        o[-n:] = 7
        cache.attend(q, o, _ints(m), torch.tensor([tq - rows, tq], dtype=torch.int32, device="cuda"), table, max_new=rows)
        plan.check()
        assert_close(o[-rows:], want[-rows:], tol[-rows:])
        assert bool((o[-n:-rows] == 7).all() if rows < n else True)


@pytest.mark.parametrize("Hq,Hk,B", [(4, 4, 20000), (8, 1, 5000)])
def test_a_large_batch_of_short_sequences(Hq, Hk, B):
    """Thousands of sequences of one new token, keys by the dozen: every result against 64 bits at once."""
    from temporal_block_sparse_sm_b200 import serving
    d, page, m = 64, 16, 16
    plan = serving.GroupedPlan(Hq, Hk, d)
    kp, vp, q = _randn(B, Hk, page, d), _randn(B, Hk, page, d, seed=1), _randn(B, Hq, d, seed=2)
    lens = torch.arange(B, device="cuda").remainder(m + 1).int()
    o = torch.full_like(q, 7.0)
    serving.PagedCache(plan, kp, vp).attend(q, o, lens, torch.arange(B + 1, device="cuda").int(),
                                            torch.arange(B, device="cuda").int().view(B, 1), max_new=1)
    plan.check()
    s = torch.einsum("bhgd,bhkd->bhgk", q.view(B, Hk, Hq // Hk, d).double(), kp.double()) / 8
    hide = torch.arange(m, device="cuda")[None, :] >= lens[:, None]
    w = torch.softmax(s.masked_fill(hide[:, None, None], float("-inf")), -1).nan_to_num(0.0)
    want, A = (torch.einsum("bhgk,bhkd->bhgd", w, x).reshape(B, Hq, d) for x in (vp.double(), vp.double().abs()))
    # u for the output, 2 u A for the weights; logits of up to 64 products of a few units each: 1e-4 is plenty for those
    u = 2.0 ** -8
    assert_close(o, want, u * want.abs() + (2 * u / (1 - u) + 1e-4) * A + 1e-30)


@pytest.mark.parametrize("new", [1, 30])
def test_pages_that_sequences_share(new):
    """Sequences with a common beginning hold it once; a page may even come twice in one sequence; and keys may
    be values (one tensor for both)."""
    from temporal_block_sparse_sm_b200 import serving
    Hq, Hk, d, page, m = 4, 2, 64, 16, 90
    kp, vp = _randn(12, Hk, page, d), _randn(12, Hk, page, d, seed=1)
    table = _ints([3, 7, 1, 0, 5, 2], [3, 7, 1, 4, 6, 8], [3, 3, 3, 3, 9, 3])
    plan = serving.GroupedPlan(Hq, Hk, d)
    q = _randn(3 * new, Hq, d, seed=2)
    o = torch.empty_like(q)
    serving.PagedCache(plan, kp, vp).attend(q, o, _ints(m, m, m), offsets([new] * 3), table, max_new=new)
    plan.check()
    for b in range(3):
        k, v = (torch.cat([p[int(j)].transpose(0, 1) for j in table[b]])[:m] for p in (kp, vp))
        rows = slice(b * new, (b + 1) * new)
        want, tol = seq_reference(q[rows], k, v, True, d ** -0.5)
        assert_close(o[rows], want, tol, f"sequence {b}")
    plan.prompt(q, k, k, o, offsets([3 * new]), offsets([m]))
    plan.check()
    want, tol = seq_reference(q, k, k, True, d ** -0.5)
    assert_close(o, want, tol)
