"""Serving attention on the GPU: how a batch is divided among the blocks -- whole items by a counter, in graphs
too, cut items of many sequences, and that no tile of a long cache is left out or counted twice."""
from __future__ import annotations

import math

import pytest
import torch

from tests.serving_ref import assert_close, offsets, paged, seq_reference

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from temporal_block_sparse_sm_b200 import build, liteattn
    build.build()
    liteattn.load()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=BF16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _workspace(plan, *sizes):
    from temporal_block_sparse_sm_b200 import liteattn
    return liteattn.lite_attn_gqa_workspace(plan.handle, *sizes)


COUNTER = 4    # bytes of workspace of a call that hands out whole items by a counter


def _replays(run, o, eager):
    """Two calls in a captured graph, replayed: the eager results, again and again."""
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        run()
        o.add_(1)          # the second call starts behind other work on o
        run()
    for _ in range(4):
        o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager)


@pytest.mark.parametrize("Hq,Hk,d,dtype,nq,nk", [
    (64, 4, 128, BF16, [500, 1, 120, 300, 0, 79], [500, 1, 120, 300, 10, 79]),      # few keys: nothing is cut
    (64, 4, 64, FP16, [100, 350, 350, 1, 150], [50, 400, 300, 20, 200]),
    (10, 10, 128, BF16, [30000 // k for k in range(1, 8)], None),                   # many items per block
    (16, 8, 64, FP16, [9001, 5000, 3, 8000, 1, 12000], None),
])
def test_prompts_by_the_counter(Hq, Hk, d, dtype, nq, nk):
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(1)
    nk = nq if nk is None else nk
    q, k, v = (_randn(g, n, h, d, dtype=dtype) for n, h in ((sum(nq), Hq), (sum(nk), Hk), (sum(nk), Hk)))
    plan, cu_q, cu_k, o = serving.GroupedPlan(Hq, Hk, d, dtype=dtype), offsets(nq), offsets(nk), torch.full_like(q, 7.0)
    assert _workspace(plan, len(nq), sum(nq), sum(nq), sum(nk)) == COUNTER
    plan.prompt(q, k, v, o, cu_q, cu_k)
    plan.check()
    i = j = 0
    heads = slice(0, Hq) if sum(nq) < 5000 else None
    for b, (n, m) in enumerate(zip(nq, nk)):
        if heads is not None:
            want, tol = seq_reference(q[i:i + n], k[j:j + m], v[j:j + m], True, d ** -0.5)
            assert_close(o[i:i + n], want, tol, f"sequence {b}")
        else:               # of long sequences the last rows, which see all, and some before
            for last in {n, n // 2, min(n, 257), 1}:
                t = slice(max(0, last - 40), last)
                want, tol = seq_reference(q[i:i + n][t], k[j:j + last], v[j:j + last], True, d ** -0.5)
                assert_close(o[i:i + n][t], want, tol, f"sequence {b}, rows before {last}")
        i, j = i + n, j + m
    _replays(lambda: plan.prompt(q, k, v, o, cu_q, cu_k), o, o.clone())
    plan.check()


@pytest.mark.parametrize("Hq,Hk,d,dtype,new,total", [
    (32, 8, 128, BF16, [100] * 20, [600 - 13 * b for b in range(20)]),
    (8, 2, 128, FP16, [3] * 500, [20 + (b * 29) % 280 for b in range(500)]),        # the kernel of few rows
    (64, 4, 64, BF16, [1] * 400, [1 + (b * 31) % 310 for b in range(400)]),
])
def test_caches_by_the_counter(Hq, Hk, d, dtype, new, total):
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(2)
    ks, vs = ([_randn(g, m, Hk, d, dtype=dtype) for m in total] for _ in range(2))
    kp, vp, table = paged(ks, vs, 16, "bhnd", g)
    plan = serving.GroupedPlan(Hq, Hk, d, dtype=dtype)
    cache = serving.PagedCache(plan, kp, vp)
    q = _randn(g, sum(new), Hq, d, dtype=dtype)
    o, lens, cu = torch.full_like(q, 7.0), torch.tensor(total, dtype=torch.int32, device="cuda"), offsets(new)
    assert _workspace(plan, len(new), sum(new), max(new), table.shape[1] * 16) == COUNTER
    run = lambda: cache.attend(q, o, lens, cu, table, max_new=max(new))   # noqa: E731
    run()
    plan.check()
    at = 0
    for b, (n, m) in enumerate(zip(new, total)):
        want, tol = seq_reference(q[at:at + n], ks[b], vs[b], True, d ** -0.5)
        assert_close(o[at:at + n], want, tol, f"sequence {b}")
        at += n
    _replays(run, o, o.clone())
    plan.check()


def _by_tile(m, d, dtype, gen):
    """Values that say where a key is: 1 to 2 in the column of its 64-key tile (modulo d), 0 elsewhere.  A
    column's output is then what few tiles weigh, so that a tile or a 16-key part of one that is left
    out or counted twice is a change of 3% or more, at any length of the cache."""
    v = torch.zeros(m, 1, d, device="cuda")
    key = torch.arange(m, device="cuda")
    v[key, 0, (key // 64) % d] = 1 + torch.rand(m, generator=gen, device="cuda")
    return v.to(dtype)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (FP16, 128), (FP16, 64)])
@pytest.mark.parametrize("Hq,new,total", [
    (4, [1], [40001]), (4, [1], [70001]), (4, [4], [40004]), (1, [1], [30063]), (4, [64], [40064]), (16, [100], [20100]),
    (8, [1, 1, 1], [33000, 5, 12345]), (8, [40, 1, 30], [20000, 9000, 30]),
    (4, [1] * 40, [3000 + 17 * b for b in range(40)]),                    # more sequences than a warp has lanes,
    (8, [20] * 40, [5000 + 61 * b for b in range(40)]),                   # in both kernels, cut
])
def test_every_tile_counts_once(dtype, d, Hq, new, total):
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(len(new) + total[0])
    ks = [_randn(g, m, 1, d, dtype=dtype) for m in total]
    vs = [_by_tile(m, d, dtype, g) for m in total]
    kp, vp, table = paged(ks, vs, 64, "bhnd", g)
    plan = serving.GroupedPlan(Hq, 1, d, dtype=dtype)
    q = (0.3 * torch.randn(sum(new), Hq, d, generator=g, device="cuda")).to(dtype)     # weights of like size
    o, lens, cu = torch.full_like(q, 7.0), torch.tensor(total, dtype=torch.int32, device="cuda"), offsets(new)
    assert _workspace(plan, len(new), sum(new), max(new), table.shape[1] * 64) > COUNTER      # items may be cut
    serving.PagedCache(plan, kp, vp).attend(q, o, lens, cu, table, max_new=max(new))
    plan.check()
    at = 0
    for b, (n, m) in enumerate(zip(new, total)):
        want, tol = seq_reference(q[at:at + n], ks[b], vs[b], True, d ** -0.5)
        assert_close(o[at:at + n], want, tol, f"sequence {b}")
        at += n


@pytest.mark.parametrize("m,d,dtype", [(70001, 128, BF16), (40064, 64, FP16)])
def test_the_bound_sees_a_lost_tile(m, d, dtype):
    """The reference with a tile, or 16 keys, left out or counted twice is outside the bound (no kernel runs)."""
    g = _gen(9)
    k, v = _randn(g, m, 1, d, dtype=dtype), _by_tile(m, d, dtype, g)
    q = (0.3 * torch.randn(1, 4, d, generator=g, device="cuda")).to(dtype)
    want, tol = seq_reference(q, k, v, False, d ** -0.5)
    for at, n in ((0, 64), (m // 2 // 64 * 64, 64), (m // 3 // 16 * 16, 16), (m - 16, 16)):
        for keep in (torch.cat([torch.arange(at), torch.arange(at + n, m)]), torch.cat([torch.arange(m), torch.arange(at, min(m, at + n))])):
            keep = keep.cuda()
            other, _ = seq_reference(q, k[keep], v[keep], False, d ** -0.5)
            with pytest.raises(AssertionError):
                assert_close(other, want, tol)
