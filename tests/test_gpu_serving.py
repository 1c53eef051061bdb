"""Serving attention on the GPU: the append to a paged cache, attention over it and attention over
packed prompts, against the 64-bit reference of tests/serving_ref.py and its derived bound."""
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


def _randn(g, *shape, dtype, scale=1.25):
    return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)


# ---------------------------------------------------------------- attention over the cache
def _attend_case(Hq, Hk, d, dtype, page, layout, new, total, causal=True, seed=0, pad=0, lead=0, max_new=None,
                 edit=None, scale=None, fill=None, std=1.25):
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(seed)
    T = lead + sum(new) + pad
    q = _randn(g, T, Hq, d, dtype=dtype, scale=std)
    ks = [_randn(g, m, Hk, d, dtype=dtype, scale=std) for m in total]
    vs = [_randn(g, m, Hk, d, dtype=dtype, scale=std) for m in total]
    if edit is not None:
        edit(q, ks, vs)
    kp, vp, table = paged(ks, vs, page, layout, g, fill=fill)
    plan = serving.GroupedPlan(Hq, Hk, d, dtype=dtype)
    cache = serving.PagedCache(plan, kp, vp, layout=layout)
    o = torch.full((T, Hq, d), 7.0, dtype=dtype, device="cuda")
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    cu = offsets(new, start=lead)
    cache.attend(q, o, lens, cu, table, max_new=max(new) if max_new is None else max_new, causal=causal, scale=scale)
    plan.check()
    at = lead
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    for b, (n, m) in enumerate(zip(new, total)):
        want, tol = seq_reference(q[at:at + n], ks[b], vs[b], causal, sc)
        assert_close(o[at:at + n], want, tol, f"sequence {b} ({n} new, {m} keys)")
        at += n
    assert bool((o[:lead] == 7).all()) and bool((o[at:] == 7).all()), "rows outside the sequences were written"
    return o


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("layout,page", [("bhnd", 16), ("bnhd", 64), ("bhnd", 256), ("bnhd", 32)])
def test_attend_single_tokens(d, dtype, layout, page):
    _attend_case(8, 2, d, dtype, page, layout, [1] * 9, [1, 2, 15, 16, 17, 63, 64, 65, 1000], seed=d + page, pad=2)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (6, 1), (7, 1), (12, 4), (24, 4), (40, 8), (16, 1), (20, 1), (128, 1)])
@pytest.mark.parametrize("new,total", [([1, 1], [129, 700]), ([3, 1, 0, 2], [3, 65, 40, 300]), ([70, 200], [500, 200])])
def test_attend_group_sizes(Hq, Hk, new, total):
    _attend_case(Hq, Hk, 128, BF16, 16, "bhnd", new, total, seed=Hq)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,total", [([1, 5, 130, 257], [1, 5, 130, 257]),              # no context
                                       ([64, 128, 129], [1064, 4000, 129]),
                                       ([300, 5, 40], [100, 3, 0]),                         # rows that see nothing
                                       ([0, 0, 1, 0], [0, 50, 50, 7]),                      # nothing new
                                       ([513], [20000]), ([1], [70001])])
@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, FP16)])
def test_attend_chunks(causal, new, total, d, dtype):
    _attend_case(8, 2, d, dtype, 64, "bnhd", new, total, causal=causal, seed=len(new) + d, lead=3, pad=4)


@pytest.mark.parametrize("max_new", [0, 1, 1000])
def test_attend_any_max_new_is_correct(max_new):
    _attend_case(8, 2, 128, BF16, 32, "bhnd", [1, 40, 2], [900, 333, 2], max_new=max_new)


def test_attend_many_sequences():
    r = torch.Generator().manual_seed(3)
    total = torch.randint(0, 300, (1500,), generator=r).tolist()
    new = [min(m, int(x)) for m, x in zip(total, torch.randint(0, 3, (1500,), generator=r).tolist())]
    _attend_case(4, 2, 64, BF16, 16, "bnhd", new, total, seed=8)


@pytest.mark.parametrize("n,m", [(1, 500), (5, 500), (100, 500), (130, 300)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_attend_hidden_nonfinite_values_do_not_leak(n, m, dtype, value):
    """A NaN or infinite value that some rows see and others do not reaches only the rows that see it."""
    def edit(q, ks, vs):
        for j in {m - 1, m - n // 2 - 1, max(0, m - n)}:
            vs[0][j, 0, 5] = value
        ks[0][m - 1, 1, 3] = value
    if n == 1:
        edit = None   # the only row sees every key; the pools' unused places hold NaN
    _attend_case(4, 2, 128, dtype, 16, "bhnd", [n], [m], edit=edit)


def test_attend_large_logits_and_empty_weights():
    """Logits that differ by hundreds: one key takes all the weight, the others underflow."""
    _attend_case(4, 1, 128, BF16, 64, "bhnd", [1, 33], [700, 500], std=6.0)


def test_attend_all_visible_logits_minus_infinity_is_nan():
    """A row whose every visible logit is -inf has no softmax: NaN, as exp(-inf - -inf) gives."""
    def edit(q, ks, vs):
        q[:, :, 0] = 1.0
        ks[0][:, :, 0] = -math.inf
    o = _attend_case(4, 2, 64, BF16, 16, "bhnd", [2], [40], edit=edit)
    assert bool(torch.isnan(o).all())


def test_attend_scale():
    _attend_case(4, 2, 64, FP16, 16, "bhnd", [1, 50], [300, 80], scale=0.3)


def test_attend_deterministic_and_on_a_stream():
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(5)
    total, Hq, Hk, d = [5000, 37, 2000], 8, 2, 128
    ks, vs = ([_randn(g, m, Hk, d, dtype=BF16) for m in total] for _ in range(2))
    kp, vp, table = paged(ks, vs, 32, "bhnd", g)
    plan = serving.GroupedPlan(Hq, Hk, d)
    cache = serving.PagedCache(plan, kp, vp)
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    for new in ([1, 1, 1], [200, 30, 1]):
        cu, q = offsets(new), _randn(g, sum(new), Hq, d, dtype=BF16)
        outs = []
        streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for s in streams:
            o = torch.empty_like(q)
            cache.attend(q, o, lens, cu, table, max_new=max(new), stream=s)   # two streams at the same time
            outs.append(o)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ---------------------------------------------------------------- attention over packed prompts
def _prompt_case(Hq, Hk, d, dtype, nq, nk=None, causal=True, seed=0, pad=0, lead=0, fused=False, scale=None, edit=None):
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(seed)
    T = lead + sum(nq) + pad
    if fused:
        x = _randn(g, T, Hq + 2 * Hk, d, dtype=dtype)
        q, k, v = x.split([Hq, Hk, Hk], dim=1)
        out = torch.full((T, Hq + 3, d), 7.0, dtype=dtype, device="cuda")
        o = out[:, 1:1 + Hq]
    else:
        Tk = T if nk is None else lead + sum(nk) + pad
        q, k, v = (_randn(g, n, h, d, dtype=dtype) for n, h in ((T, Hq), (Tk, Hk), (Tk, Hk)))
        o = torch.full((T, Hq, d), 7.0, dtype=dtype, device="cuda")
    cu_q = offsets(nq, start=lead)
    cu_k = None if nk is None else offsets(nk, start=lead)
    k[:lead], v[:lead] = math.nan, math.nan                     # nobody's rows
    k[int((cu_q if nk is None else cu_k)[-1]):], v[int((cu_q if nk is None else cu_k)[-1]):] = math.nan, math.nan
    if edit is not None:
        edit(q, k, v)
    plan = serving.GroupedPlan(Hq, Hk, d, dtype=dtype)
    plan.prompt(q, k, v, o, cu_q, cu_k=cu_k, causal=causal, scale=scale)
    plan.check()
    i = j = lead
    for b, (n, m) in enumerate(zip(nq, nq if nk is None else nk)):
        want, tol = seq_reference(q[i:i + n], k[j:j + m], v[j:j + m], causal, 1.0 / math.sqrt(d) if scale is None else scale)
        assert_close(o[i:i + n], want, tol, f"sequence {b} ({n} queries, {m} keys)")
        i, j = i + n, j + m
    assert bool((o[:lead] == 7).all()) and bool((o[i:] == 7).all()), "rows outside the sequences were written"
    if fused:
        assert bool((out[:, 0] == 7).all()) and bool((out[:, 1 + Hq:] == 7).all()), "neighbouring heads were written"


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("nq", [[1], [2, 1, 0, 17], [127, 128, 129], [255, 256, 257, 64], [1000, 3, 700], [2500]])
def test_prompt(causal, d, dtype, nq):
    _prompt_case(4, 2, d, dtype, nq, causal=causal, seed=sum(nq), lead=2, pad=5)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (5, 1), (7, 1), (12, 12), (28, 4), (64, 1), (100, 1), (128, 1)])
def test_prompt_group_sizes(Hq, Hk):
    _prompt_case(Hq, Hk, 128, BF16, [130, 1, 300], seed=Hq)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", [([5, 300, 40], [300, 5, 40]), ([200, 1], [0, 1000]), ([64, 64, 64], [63, 64, 65]),
                                   ([1, 1, 1], [400, 0, 1])])
@pytest.mark.parametrize("d,dtype", [(128, FP16), (64, BF16)])
def test_prompt_keys_and_queries_of_different_lengths(causal, nq, nk, d, dtype):
    _prompt_case(6, 2, d, dtype, nq, nk, causal=causal, seed=len(nq), pad=1)


def test_prompt_without_any_key():
    _prompt_case(4, 2, 64, BF16, [5, 3], [0, 0])


@pytest.mark.parametrize("d,dtype", [(128, BF16), (64, FP16)])
def test_prompt_fused_projection_views(d, dtype):
    _prompt_case(8, 2, d, dtype, [100, 300], fused=True, seed=4)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("value", [math.inf, math.nan])
@pytest.mark.parametrize("n", [9, 129, 400])
def test_prompt_later_nonfinite_values_do_not_leak(dtype, value, n):
    """Causal: a NaN or infinite value at a token reaches that token's row and later ones only."""
    def edit(q, k, v):
        for j in (n - 1, n // 2, n // 3):
            v[j, 0, 7] = value
            v[j, 1, 70] = -value
    _prompt_case(4, 2, 128, dtype, [n, 5], edit=edit, seed=n)


def test_prompt_masked_infinite_keys():
    """Infinite and NaN keys at later tokens give masked logits: earlier rows do not change."""
    def edit(q, k, v):
        k[70, 0, 3], k[71, 1, 9], k[99, 0, 0] = math.inf, math.nan, -math.inf
    _prompt_case(2, 2, 64, BF16, [100], edit=edit)


# ---------------------------------------------------------------- append
def _append_case(Hq, Hk, d, dtype, page, layout, new, total, rot, interleaved, fused=False, own_pos=False, with_q=True,
                 in_place=False, pad=0, lead=0, seed=0):
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(seed)
    T = lead + sum(new) + pad
    ks, vs = ([_randn(g, m, Hk, d, dtype=dtype) for m in total] for _ in range(2))
    kp, vp, table = paged(ks, vs, page, layout, g, fill=3.0)
    x = _randn(g, T, Hq + 2 * Hk, d, dtype=dtype)
    q, k, v = x.split([Hq, Hk, Hk], dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q0 = q.clone()
    qo = None if not with_q else q if in_place else torch.full((T, Hq, d), 7.0, dtype=dtype, device="cuda")
    n_rows = 2 * max(total) + 5
    cos = sin = pos = None
    if rot:
        cos, sin = serving.rotation_table(range(n_rows), [10000.0 ** (-2 * i / rot) for i in range(rot // 2)], device="cuda")
        pos = torch.randint(0, n_rows, (T,), generator=g, device="cuda", dtype=torch.int32) if own_pos else None
    plan = serving.GroupedPlan(Hq, Hk, d, dtype=dtype)
    cache = serving.PagedCache(plan, kp, vp, layout=layout)
    want_k, want_v = kp.double().clone(), vp.clone()
    want_q = (q0 if in_place else torch.full((T, Hq, d), 7.0, device="cuda")).double().clone()
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    cu = offsets(new, start=lead)
    cache.append(k, v, lens, cu, table, q=q if with_q else None, q_out=qo, cos=cos, sin=sin, positions=pos,
                 interleaved=interleaved)
    plan.check()
    size_k, size_q = want_k.abs(), want_q.abs()   # what a rotated element's rounding errors scale with

    def turn(y, row):
        y = y.double()
        z, mag = y.clone(), y.abs()
        if rot:
            a, b = (y[:, 0:rot:2], y[:, 1:rot:2]) if interleaved else (y[:, :rot // 2], y[:, rot // 2:rot])
            c, s = cos[row].double(), sin[row].double()
            ra, rb, big = a * c - b * s, a * s + b * c, a.abs() + b.abs()
            if interleaved:
                z[:, 0:rot:2], z[:, 1:rot:2], mag[:, 0:rot:2], mag[:, 1:rot:2] = ra, rb, big, big
            else:
                z[:, :rot // 2], z[:, rot // 2:rot], mag[:, :rot // 2], mag[:, rot // 2:rot] = ra, rb, big, big
        return z, mag

    i = lead
    for b, (n, m) in enumerate(zip(new, total)):
        for t in range(n):
            slot = m - n + t
            row = int(pos[i]) if own_pos else slot
            pg, r = int(table[b, slot // page]), slot % page
            at = (pg, slice(None), r) if layout == "bhnd" else (pg, r)
            want_k[at], size_k[at] = turn(k[i] if not fused else k[i].clone(), row)
            want_v[at] = v[i]
            want_q[i], size_q[i] = turn(q0[i], row)
            i += 1
    # one rounding of a 32-bit a c - b s: half a step of the result, and three 32-bit roundings of |a| + |b|
    u = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert_close(kp, want_k, u * want_k.abs() + 3 * 2.0 ** -24 * size_k * (1 + u) + tiny, "k")
    assert torch.equal(vp.view(torch.int16), want_v.view(torch.int16)), "values are copied bit for bit"
    if with_q:
        assert_close(qo, want_q, u * want_q.abs() + 3 * 2.0 ** -24 * size_q * (1 + u) + tiny, "q")


@pytest.mark.parametrize("layout,page", [("bhnd", 16), ("bnhd", 64), ("bhnd", 256)])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 96), (64, 64), (64, 48), (64, 16), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(layout, page, d, rot, interleaved):
    _append_case(6, 2, d, BF16, page, layout, [1, 20, 0, 7], [1, 20, 5, 300], rot, interleaved, pad=3, lead=2, seed=rot + d)


@pytest.mark.parametrize("kw", [dict(fused=True), dict(own_pos=True), dict(with_q=False), dict(in_place=True),
                                dict(in_place=True, fused=True, own_pos=True)])
@pytest.mark.parametrize("Hq,Hk", [(5, 1), (12, 12), (32, 8), (130, 2)])
def test_append_forms(kw, Hq, Hk):
    _append_case(Hq, Hk, 128, FP16, 32, "bnhd", [1, 1, 9], [100, 1, 50], 128, True, seed=Hq, **kw)


def test_append_many_tokens():
    _append_case(4, 2, 64, BF16, 128, "bhnd", [700, 1, 900], [1000, 1, 900], 64, False, seed=2)


# ---------------------------------------------------------------- together, as they are used
@pytest.mark.parametrize("dtype,Hq,Hk,d,page,layout", [(BF16, 8, 2, 128, 16, "bhnd"), (FP16, 6, 6, 64, 64, "bnhd")])
def test_prompt_then_decode(dtype, Hq, Hk, d, page, layout):
    """Two prompts are read at once and appended, then both sequences decode token by token and one
    takes a chunk; every step's output equals attention over the sequence's rotated history."""
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(11)
    plan = serving.GroupedPlan(Hq, Hk, d, dtype=dtype)
    width = 8
    pools = [torch.full((2 * width + 1, Hk, page, d) if layout == "bhnd" else (2 * width + 1, page, Hk, d), math.nan, dtype=dtype,
                        device="cuda") for _ in range(2)]
    cache = serving.PagedCache(plan, *pools, layout=layout)
    table = torch.randperm(2 * width + 1, generator=g, device="cuda")[:2 * width].view(2, width).int()
    cos, sin = serving.rotation_table(range(width * page), [1000.0 ** (-2 * i / d) for i in range(d // 2)], device="cuda")
    hist_k, hist_v = [[], []], [[], []]
    lens = [0, 0]
    for step, new in enumerate([[37, 50], [1, 1], [1, 1], [20, 1], [0, 1], [1, 0]]):
        T = sum(new)
        q, k, v = (_randn(g, T, h, d, dtype=dtype) for h in (Hq, Hk, Hk))
        qr, o = torch.empty_like(q), torch.zeros(T, Hq, d, dtype=dtype, device="cuda")
        cu = offsets(new)
        lens = [a + b for a, b in zip(lens, new)]
        dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cache.append(k, v, dl, cu, table, q=q, q_out=qr, cos=cos, sin=sin)
        cache.attend(qr, o, dl, cu, table, max_new=max(new))
        plan.check()
        at = 0
        for b, n in enumerate(new):
            for t in range(n):   # the rotated key as the cache holds it
                slot = lens[b] - n + t
                pg, r = int(table[b, slot // page]), slot % page
                hist_k[b].append(pools[0][pg, :, r] if layout == "bhnd" else pools[0][pg, r])
                hist_v[b].append(v[at + t])
            if n:
                want, tol = seq_reference(qr[at:at + n], torch.stack(hist_k[b]), torch.stack(hist_v[b]), True, 1 / math.sqrt(d))
                assert_close(o[at:at + n], want, tol, f"step {step} sequence {b}")
            at += n
        if step == 0:   # the prompt pass gives the same rows
            kr = torch.cat([torch.stack(h) for h in hist_k])
            o2 = torch.zeros_like(o)
            plan.prompt(qr, kr, v, o2, cu)
            plan.check()
            at = 0
            for b, n in enumerate(new):
                want, tol = seq_reference(qr[at:at + n], kr[at:at + n], v[at:at + n], True, 1 / math.sqrt(d))
                assert_close(o2[at:at + n], want, tol, f"prompt {b}")
                at += n


def test_captured_graph_replays_on_other_lengths():
    """Append and attend captured once; replayed after lengths, tables and inputs changed in place."""
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(21)
    Hq, Hk, d, page, width, B, T = 8, 2, 128, 16, 40, 3, 8
    plan = serving.GroupedPlan(Hq, Hk, d)
    kp, vp = (torch.full((B * width, Hk, page, d), math.nan, dtype=BF16, device="cuda") for _ in range(2))
    cache = serving.PagedCache(plan, kp, vp)
    table = torch.arange(B * width, device="cuda").view(B, width).int()
    q, k, v = (_randn(g, T, h, d, dtype=BF16) for h in (Hq, Hk, Hk))
    qr, o = torch.empty_like(q), torch.empty_like(q)
    lens, cu = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cos, sin = serving.rotation_table(range(width * page), [100.0 ** (-2 * i / d) for i in range(d // 2)], device="cuda")

    def step():
        cache.append(k, v, lens, cu, table, q=q, q_out=qr, cos=cos, sin=sin)
        cache.attend(qr, o, lens, cu, table, max_new=T)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    hist = [[], [], []]
    total = [0, 0, 0]
    for new in ([5, 1, 2], [1, 1, 1], [0, 8, 0], [2, 2, 2], [1, 0, 1]):
        total = [a + b for a, b in zip(total, new)]
        lens.copy_(torch.tensor(total, dtype=torch.int32))
        cu.copy_(offsets(new, device="cpu"))
        q.copy_(_randn(g, T, Hq, d, dtype=BF16))
        k.copy_(_randn(g, T, Hk, d, dtype=BF16))
        v.copy_(_randn(g, T, Hk, d, dtype=BF16))
        o.fill_(7)
        graph.replay()
        plan.check()
        at = 0
        for b, n in enumerate(new):
            for t in range(n):
                slot = total[b] - n + t
                hist[b].append((kp[int(table[b, slot // page]), :, slot % page].clone(), v[at + t].clone()))
            if n:
                ks, vs = (torch.stack([x[i] for x in hist[b]]) for i in range(2))
                want, tol = seq_reference(qr[at:at + n], ks, vs, True, 1 / math.sqrt(d))
                assert_close(o[at:at + n], want, tol, f"{new} sequence {b}")
            at += n
        assert bool((o[at:] == 7).all())


# ---------------------------------------------------------------- device data that cannot be used
def _status_case(mutate, call="attend"):
    """Runs a call whose device data was changed by `mutate`; returns (error code, o, q_out, pools before, pools after)."""
    from temporal_block_sparse_sm_b200 import liteattn, serving
    g = _gen(31)
    Hq, Hk, d, page = 4, 2, 64, 16
    new, total = [2, 3], [40, 70]
    ks, vs = ([_randn(g, m, Hk, d, dtype=BF16) for m in total] for _ in range(2))
    kp, vp, table = paged(ks, vs, page, "bhnd", g, fill=1.0)
    plan = serving.GroupedPlan(Hq, Hk, d)
    cache = serving.PagedCache(plan, kp, vp)
    lens, cu = torch.tensor(total, dtype=torch.int32, device="cuda"), offsets(new)
    q, k, v = (_randn(g, 5, h, d, dtype=BF16) for h in (Hq, Hk, Hk))
    o = torch.full((5, Hq, d), 7.0, dtype=BF16, device="cuda")
    cos, sin = serving.rotation_table(range(100), [1.0] * 32, device="cuda")
    pos = torch.zeros(5, dtype=torch.int32, device="cuda")
    mutate(lens, cu, table, pos)
    before = kp.clone(), vp.clone()
    if call == "attend":
        cache.attend(q, o, lens, cu, table, max_new=3)
    elif call == "prompt":
        plan.prompt(q, k, v, o, cu, cu_k=lens)   # lens stands in for cu_k
    else:
        cache.append(k, v, lens, cu, table, q=q, q_out=o, cos=cos, sin=sin, positions=pos)
    code = 0
    try:
        plan.check()
    except liteattn.LiteAttnError as e:
        code = e.code
    return code, o, before, (kp, vp)


@pytest.mark.parametrize("call", ["attend", "append"])
@pytest.mark.parametrize("what", ["page", "negative page", "long", "negative", "rows", "backwards"])
def test_bad_device_data_is_reported_and_not_used(call, what):
    from temporal_block_sparse_sm_b200 import liteattn

    def mutate(lens, cu, table, pos):
        if what == "page":
            table[0, 2] = 1 << 20
        elif what == "negative page":
            table[0, 2] = -5
        elif what == "long":
            lens[0] = 1 << 20
        elif what == "negative":
            lens[0] = -1
        elif what == "rows":
            cu[2] = 1000
        else:
            cu[0], cu[1] = 2, 1
    code, o, before, after = _status_case(mutate, call)
    assert code == liteattn.LITE_ERR_DEVICE_CHECK
    if call == "append" and what in ("page", "negative page", "long", "negative"):
        assert bool((o[:2] == 7).all()), "the refused tokens were written"
        assert not bool((o[2:] == 7).all())
    if call == "append" and what == "rows":
        assert bool((o[2:] == 7).all())


def test_append_refuses_negative_slots_and_angle_rows():
    from temporal_block_sparse_sm_b200 import liteattn
    for mutate in (lambda lens, cu, table, pos: lens.__setitem__(0, 1), lambda lens, cu, table, pos: pos.__setitem__(0, 100),
                   lambda lens, cu, table, pos: pos.__setitem__(0, -1)):
        code, o, before, after = _status_case(mutate, "append")
        assert code == liteattn.LITE_ERR_DEVICE_CHECK
        assert bool((o[0] == 7).all()) and not bool((o[1:] == 7).all(dim=-1).any())


def test_good_device_data_reports_nothing():
    for call in ("attend", "append"):
        assert _status_case(lambda *a: None, call)[0] == 0


def test_arguments_refused_on_the_host():
    from temporal_block_sparse_sm_b200 import liteattn, serving
    plan = serving.GroupedPlan(4, 2, 64)
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    kp, vp = z(3, 2, 16, 64), z(3, 2, 16, 64)
    cache = serving.PagedCache(plan, kp, vp)
    q, k, v, o = z(5, 4, 64), z(5, 2, 64), z(5, 2, 64), z(5, 4, 64)
    lens, cu, table = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1,), (2,), (1, 3)))
    n0 = liteattn.lite_attn_launch_count()
    for bad in (dict(q=q.half()), dict(q=q[:, :3]), dict(o=o[:4]), dict(lens=lens.long()), dict(lens=lens[:0]), dict(cu_new=cu.cpu()),
                dict(table=table[:, ::2]), dict(o=q), dict(q=z(5, 4, 68)[:, :, :64]), dict(q=z(5, 64, 4).transpose(1, 2)),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(max_new=-1)):
        args = dict(q=q, o=o, lens=lens, cu_new=cu, table=table, max_new=1)
        args.update(bad)
        with pytest.raises((ValueError, liteattn.LiteAttnError)):
            cache.attend(**args)
    for bad in (dict(k=k[:4]), dict(q=q), dict(q=q, q_out=k), dict(q=q, q_out=q[:, :, :32]), dict(positions=lens),
                dict(cos=z(4, 8, dt=torch.float32)), dict(cos=z(4, 8), sin=z(4, 8)),
                dict(cos=z(4, 12, dt=torch.float32), sin=z(4, 12, dt=torch.float32)),
                dict(cos=z(4, 40, dt=torch.float32), sin=z(4, 40, dt=torch.float32)),
                dict(k=kp.view(-1, 2, 64)[:5])):
        args = dict(k=k, v=v, lens=lens, cu_new=cu, table=table)
        args.update(bad)
        with pytest.raises((ValueError, liteattn.LiteAttnError)):
            cache.append(**args)
    for bad in (dict(k=k[:4]), dict(o=q), dict(cu_k=cu[:1]), dict(q=q.float())):
        args = dict(q=q, k=k, v=v, o=o, cu_q=cu)
        args.update(bad)
        with pytest.raises((ValueError, liteattn.LiteAttnError)):
            plan.prompt(**args)
    for shape, layout in (((3, 2, 24, 64), "bhnd"), ((3, 2, 8, 64), "bhnd"), ((3, 16, 3, 64), "bnhd"), ((3, 2, 16, 64), "other")):
        with pytest.raises(ValueError):
            serving.PagedCache(plan, z(*shape), z(*shape), layout=layout)
    with pytest.raises(liteattn.LiteAttnError):
        serving.PagedCache(plan, kp, kp).attend(q, o, lens, cu, table, max_new=1)   # one pool for both
    assert liteattn.lite_attn_launch_count() == n0, "a refused call launched a kernel"


def test_empty_calls_do_nothing():
    from temporal_block_sparse_sm_b200 import serving
    plan = serving.GroupedPlan(4, 2, 64)
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    cache = serving.PagedCache(plan, z(3, 2, 16, 64), z(3, 2, 16, 64))
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")   # noqa: E731
    cache.attend(z(0, 4, 64), z(0, 4, 64), i(2), i(3), i(2, 3), max_new=0)
    cache.append(z(0, 2, 64), z(0, 2, 64), i(2), i(3), i(2, 3))
    plan.prompt(z(0, 4, 64), z(0, 2, 64), z(0, 2, 64), z(0, 4, 64), i(1))
    o = torch.full((4, 4, 64), 7.0, dtype=BF16, device="cuda")
    cache.attend(z(4, 4, 64), o, i(2), i(3), i(2, 3), max_new=0)   # four rows, no sequence has any
    plan.check()
    assert bool((o == 7).all())


def test_plan_of_another_device_than_the_current_one():
    from temporal_block_sparse_sm_b200 import serving
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    with torch.cuda.device(1):
        plan = serving.GroupedPlan(4, 2, 64)
        g = torch.Generator(device="cuda:1").manual_seed(0)
        q, k, v = (torch.randn(50, h, 64, generator=g, device="cuda:1").to(BF16) for h in (4, 2, 2))
        cu = torch.tensor([0, 50], dtype=torch.int32, device="cuda:1")
        o1 = torch.empty_like(q)
        plan.prompt(q, k, v, o1, cu)
        torch.cuda.synchronize()
    o2 = torch.empty_like(q)
    plan.prompt(q, k, v, o2, cu)
    plan.check()
    assert torch.equal(o1, o2) and torch.cuda.current_device() == 0


# ---------------------------------------------------------------- failures, graphs, far offsets
@pytest.mark.parametrize("new", [1, 40])
def test_a_wait_that_runs_out_ends_the_kernel_and_is_reported(monkeypatch, new):
    """A warp made to wait on a barrier that nothing arrives on: its bounded wait runs out, the block
    gives up, the call ends, the plan's status says so, and another plan works on."""
    from temporal_block_sparse_sm_b200 import liteattn, serving
    g = _gen(41)
    ks, vs = ([_randn(g, 500, 2, 128, dtype=BF16)] for _ in range(2))
    kp, vp, table = paged(ks, vs, 16, "bhnd", g)
    q = _randn(g, new, 8, 128, dtype=BF16)
    lens, cu = torch.tensor([500], dtype=torch.int32, device="cuda"), offsets([new])
    plan = serving.GroupedPlan(8, 2, 128)
    o = torch.empty_like(q)
    monkeypatch.setenv("LITE_ATTN_FAULT", "device_wait")
    serving.PagedCache(plan, kp, vp).attend(q, o, lens, cu, table, max_new=new)
    monkeypatch.delenv("LITE_ATTN_FAULT")
    with pytest.raises(liteattn.LiteAttnError) as e:
        plan.check()
    assert e.value.code == liteattn.LITE_ERR_DEVICE_TIMEOUT
    other = serving.GroupedPlan(8, 2, 128)
    serving.PagedCache(other, kp, vp).attend(q, o, lens, cu, table, max_new=new)
    other.check()
    want, tol = seq_reference(q, ks[0], vs[0], True, 1 / math.sqrt(128))
    assert_close(o, want, tol)


def test_host_faults_are_reported_without_a_launch(monkeypatch):
    from temporal_block_sparse_sm_b200 import liteattn, serving
    plan = serving.GroupedPlan(4, 2, 64)
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device="cuda")   # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")   # noqa: E731
    cache = serving.PagedCache(plan, z(3, 2, 16, 64), z(3, 2, 16, 64))
    monkeypatch.setenv("LITE_ATTN_FAULT", "launch")
    n0 = liteattn.lite_attn_launch_count()
    for call in (lambda: cache.attend(z(2, 4, 64), z(2, 4, 64), i(1), i(2), i(1, 3), max_new=1),
                 lambda: cache.append(z(2, 2, 64), z(2, 2, 64), i(1), i(2), i(1, 3)),
                 lambda: plan.prompt(z(2, 4, 64), z(2, 2, 64), z(2, 2, 64), z(2, 4, 64), i(2))):
        with pytest.raises(liteattn.LiteAttnError) as e:
            call()
        assert e.value.code == liteattn.LITE_ERR_CUDA
    assert liteattn.lite_attn_launch_count() == n0
    monkeypatch.setenv("LITE_ATTN_FAULT", "status")
    with pytest.raises(liteattn.LiteAttnError) as e:
        plan.check()
    assert e.value.code == liteattn.LITE_ERR_DEVICE_TIMEOUT


def test_two_graphs_of_one_plan_replayed_at_the_same_time():
    """Two captures of one plan, each with a workspace of its own, replayed together on two streams."""
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(51)
    Hq, Hk, d = 8, 2, 128
    plan = serving.GroupedPlan(Hq, Hk, d)
    work = []
    for new, total in (([1, 1], [30000, 7]), ([100, 3], [9000, 5000])):
        ks, vs = ([_randn(g, m, Hk, d, dtype=BF16) for m in total] for _ in range(2))
        kp, vp, table = paged(ks, vs, 64, "bhnd", g)
        q = _randn(g, sum(new), Hq, d, dtype=BF16)
        lens, cu, o = torch.tensor(total, dtype=torch.int32, device="cuda"), offsets(new), torch.empty_like(q)
        cache = serving.PagedCache(plan, kp, vp)
        cache.attend(q, o, lens, cu, table, max_new=max(new))
        torch.cuda.synchronize()
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s):
            cache.attend(q, o, lens, cu, table, max_new=max(new))
        work.append((graph, s, o, o.clone(), (ks, vs, kp, vp, table, q, lens, cu, cache)))
    for _ in range(20):
        for _, _, o, _, _ in work:
            o.zero_()
        torch.cuda.synchronize()
        for graph, s, *_ in work:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, o, want, _ in work:
            assert torch.equal(o, want)
    plan.check()


@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
@pytest.mark.parametrize("new", [1, 30])
def test_pages_far_into_a_large_pool(layout, new):
    """A pool of over 2^32 bytes and 2^31 elements, its last pages in use."""
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(61)
    Hq, Hk, d, page = 8, 2, 128, 256
    pages = (1 << 31) // (page * Hk * d) + 40
    shape = (pages, Hk, page, d) if layout == "bhnd" else (pages, page, Hk, d)
    kp, vp = (torch.empty(shape, dtype=BF16, device="cuda") for _ in range(2))
    m = 3000
    table = torch.arange(pages - 1, pages - 1 - 12, -1, device="cuda").int().view(1, 12)
    ks, vs = (_randn(g, m, Hk, d, dtype=BF16) for _ in range(2))
    plan = serving.GroupedPlan(Hq, Hk, d)
    cache = serving.PagedCache(plan, kp, vp, layout=layout)
    lens = torch.tensor([m], dtype=torch.int32, device="cuda")
    cache.append(ks, vs, lens, offsets([m]), table)
    q = _randn(g, new, Hq, d, dtype=BF16)
    o = torch.empty_like(q)
    cache.attend(q, o, lens, offsets([new]), table, max_new=new)
    plan.check()
    want, tol = seq_reference(q, ks, vs, True, 1 / math.sqrt(d))
    assert_close(o, want, tol)


def test_many_splits_of_one_item_and_long_keys():
    """One key head, few rows, a long cache: one item cut over all blocks, in both kernels."""
    for new in (1, 4, 5, 64):
        _attend_case(4, 1, 128, BF16, 64, "bhnd", [new], [40000 + new], seed=new)
    _attend_case(128, 1, 64, FP16, 16, "bnhd", [1], [30011], seed=9)


def test_ragged_batches_of_every_kind():
    """Random batches over both kernels and both divisions, lengths from nothing to thousands."""
    import random
    r = random.Random(7)
    for k in range(12):
        Hk = r.choice([1, 2, 3])
        Hq = Hk * r.choice([1, 2, 5, 8])
        B = r.choice([1, 2, 7, 33, 40])
        top = r.choice([1, 3, 60, 300])
        ctx = r.choice([0, 50, 3000, 9000 if B < 8 else 300])
        new = [r.randint(0, top) for _ in range(B)]
        total = [n + r.randint(0, ctx) if r.random() < 0.9 else r.randint(0, n) for n in new]
        _attend_case(Hq, Hk, r.choice([64, 128]), r.choice([BF16, FP16]), r.choice([16, 64, 512]), r.choice(["bhnd", "bnhd"]), new, total,
                     causal=r.random() < 0.8, seed=100 + k, pad=r.randint(0, 3), lead=r.randint(0, 3))


def test_misaligned_views_are_refused():
    from temporal_block_sparse_sm_b200 import liteattn, serving
    plan = serving.GroupedPlan(4, 2, 64)
    base = torch.zeros(5 * 4 * 64 + 8, dtype=BF16, device="cuda")
    q = base[4:4 + 5 * 256].view(5, 4, 64)        # 8 bytes past a 16-byte boundary
    k, v, o = (torch.zeros(5, h, 64, dtype=BF16, device="cuda") for h in (2, 2, 4))
    with pytest.raises(liteattn.LiteAttnError):
        plan.prompt(q, k, v, o, offsets([5]))
    with pytest.raises(liteattn.LiteAttnError):
        plan.prompt(k[:, :1].expand(5, 4, 64), k, v, o, offsets([5]))   # one head four times: overlapping rows


def test_outputs_whose_rows_overlap_are_refused():
    from temporal_block_sparse_sm_b200 import liteattn, serving
    plan = serving.GroupedPlan(4, 2, 64)
    q = torch.zeros(5, 4, 64, dtype=BF16, device="cuda")
    k, v = (torch.zeros(5, 2, 64, dtype=BF16, device="cuda") for _ in range(2))
    flat = torch.zeros(4096, dtype=BF16, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")   # noqa: E731
    cache = serving.PagedCache(plan, *(torch.zeros(3, 2, 16, 64, dtype=BF16, device="cuda") for _ in range(2)))
    for bad in (flat.as_strided((5, 4, 64), (64, 64, 1)), flat.as_strided((5, 4, 64), (128, 64, 1)), flat.as_strided((5, 4, 64), (64, 256, 1))):
        for call in (lambda: plan.prompt(q, k, v, bad, offsets([5])),
                     lambda: cache.attend(q, bad, i(1), i(2), i(1, 3), max_new=1),
                     lambda: cache.append(k, v, i(1), i(2), i(1, 3), q=q, q_out=bad)):
            with pytest.raises(liteattn.LiteAttnError) as e:
                call()
            assert e.value.code == liteattn.LITE_ERR_INVALID_ARG
    heads_first = torch.zeros(4, 5, 64, dtype=BF16, device="cuda").transpose(0, 1)
    plan.prompt(q, k, v, heads_first, offsets([5]))
    plan.check()


@pytest.mark.parametrize("new", [1, 50])
def test_the_smallest_and_a_large_scale(new):
    """A scale so small that every visible key weighs the same, and one that leaves the largest logit."""
    for scale in (1e-42, 1e-30, 30.0):
        _attend_case(8, 2, 64, FP16, 16, "bhnd", [new, new], [400, new], scale=scale, seed=new)


def test_too_many_keys_are_refused():
    from temporal_block_sparse_sm_b200 import liteattn, serving
    plan = serving.GroupedPlan(4, 2, 64)
    cache = serving.PagedCache(plan, *(torch.zeros(1, 2, 65536, 64, dtype=BF16, device="cuda") for _ in range(2)))
    q = torch.zeros(1, 4, 64, dtype=BF16, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")   # noqa: E731
    with pytest.raises(liteattn.LiteAttnError) as e:
        cache.attend(q, torch.zeros_like(q), i(1), i(2), i(1, (1 << 14) + 1), max_new=1)
    assert e.value.code == liteattn.LITE_ERR_UNSUPPORTED


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hk,d,dtype,new,total", [
    (32, 8, 128, BF16, [100] * 20, [600] * 20),         # two slots to an item, whole items, more than one per block
    (20, 4, 64, FP16, [130, 1, 64, 65] * 12, [200, 1, 64, 900] * 12),
    (16, 4, 128, BF16, [64], [1000]),                   # one slot to an item
    (10, 2, 64, BF16, [25, 26, 51, 1], [700, 26, 600, 30]),
    (5, 1, 128, FP16, [1000], [1000]),
])
def test_items_of_one_slot_and_of_two(Hq, Hk, d, dtype, new, total, causal):
    _attend_case(Hq, Hk, d, dtype, 32, "bhnd", new, total, causal=causal, seed=len(new), pad=3)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("new", [1, 40])
def test_calls_wait_for_whatever_is_in_front_of_them(new, captured):
    """Inputs written right before each call by kernels, copies and another stream, outputs read right
    after it, without a wait on the host: the same as with one between all of them."""
    from temporal_block_sparse_sm_b200 import serving
    g = _gen(71)
    Hq, Hk, d, page, steps = 8, 2, 128, 16, 6
    plan = serving.GroupedPlan(Hq, Hk, d)
    src = [[_randn(g, 2 * new, h, d, dtype=BF16) for h in (Hq, Hk, Hk)] for _ in range(steps)]
    table = torch.randperm(2 * 140, device="cuda", generator=g).int().view(2, 140)
    big = _randn(g, 4096, 4096, dtype=BF16)
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def run(sync):
        kp, vp = (torch.zeros(2 * 140, Hk, page, d, dtype=BF16, device="cuda") for _ in range(2))
        lens = torch.full((2,), 2000, dtype=torch.int32, device="cuda")
        cu, outs = offsets([new, new]), [torch.zeros(2 * new, Hq, d, dtype=BF16, device="cuda") for _ in range(steps)]
        q, k, v = (torch.zeros_like(x) for x in src[0])
        o, y = torch.zeros_like(q), torch.empty_like(big)
        cache = serving.PagedCache(plan, kp, vp)

        def step():
            for i in range(steps):
                torch.mul(big, 2, out=y)              # keeps the GPU busy, so that what comes next queues up
                ev = torch.cuda.Event()
                ev.record()
                side.wait_event(ev)
                with torch.cuda.stream(side):
                    torch.add(y, 1, out=y)
                    torch.add(src[i][2], 0, out=v)
                    done = torch.cuda.Event()
                    done.record()
                lens.add_(new)
                q.copy_(src[i][0])
                k.copy_(src[i][1])
                torch.cuda.current_stream().wait_event(done)
                if sync:
                    torch.cuda.synchronize()
                cache.append(k, v, lens, cu, table)
                if sync:
                    torch.cuda.synchronize()
                cache.attend(q, o, lens, cu, table, max_new=new)
                if sync:
                    torch.cuda.synchronize()
                outs[i].copy_(o)
                o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(main):
            if captured and not sync:
                step()                                # warm-up
                torch.cuda.synchronize()
                for t in (kp, vp):
                    t.zero_()
                lens.fill_(2000)
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=main):
                    step()
                graph.replay()
            else:
                step()
        torch.cuda.synchronize()
        plan.check()
        return outs, kp, vp

    want, got = run(True), run(False)
    for a, b in zip(want[0], got[0]):
        assert torch.equal(a, b)
    assert torch.equal(want[1], got[1]) and torch.equal(want[2], got[2])


@pytest.mark.parametrize("Hq,Hk,d,dtype,B,top", [(16, 8, 64, BF16, 60, 300), (12, 12, 128, FP16, 33, 1), (8, 8, 64, BF16, 400, 2)])
def test_items_handed_out_by_a_counter(Hq, Hk, d, dtype, B, top):
    """More items than blocks in a ragged batch, eager and in a graph that is replayed: the same, and right."""
    import random
    from temporal_block_sparse_sm_b200 import serving
    r, g = random.Random(B), _gen(B)
    new = [r.randint(1, top) for _ in range(B)]
    nk = [n + r.randint(0, 300) for n in new]
    q = _randn(g, sum(new), Hq, d, dtype=dtype)
    k, v = (_randn(g, sum(nk), Hk, d, dtype=dtype) for _ in range(2))
    plan, cu_q, cu_k, o = serving.GroupedPlan(Hq, Hk, d, dtype=dtype), offsets(new), offsets(nk), torch.zeros_like(q)
    plan.prompt(q, k, v, o, cu_q, cu_k)
    plan.check()
    eager = o.clone()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        plan.prompt(q, k, v, o, cu_q, cu_k)
        plan.prompt(q, k, v, o, cu_q, cu_k)
    for _ in range(3):
        o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager)
    for b in range(0, B, max(1, B // 20)):
        i, j = sum(new[:b]), sum(nk[:b])
        want, tol = seq_reference(q[i:i + new[b]], k[j:j + nk[b]], v[j:j + nk[b]], True, 1 / math.sqrt(d))
        assert_close(eager[i:i + new[b]], want, tol, f"sequence {b}")
