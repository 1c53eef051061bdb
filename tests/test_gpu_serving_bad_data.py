"""Serving attention on the GPU with lengths, offsets, pages and angle rows that cannot be used: each call says
so, leaves out exactly what the header says, and does the rest of its work."""
from __future__ import annotations

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


def _code(plan):
    from temporal_block_sparse_sm_b200 import liteattn
    try:
        plan.check()
    except liteattn.LiteAttnError as e:
        return e.code
    return 0


FEW, MANY = [1, 2, 1], [40, 3, 90]       # new tokens: for the kernel of few rows, and for that of many
TOTAL = [300, 70, 150]

# what is wrong -> (lens, cu, table) changed, the sequences left out
ATTEND = {
    "long": (lambda lens, cu, table: lens.__setitem__(1, 1 << 20), {1}),
    "a page too long": (lambda lens, cu, table: lens.__setitem__(0, table.shape[1] * 16 + 1), {0}),
    "negative length": (lambda lens, cu, table: lens.__setitem__(2, -1), {2}),
    "rows behind the tensor": (lambda lens, cu, table: cu.__setitem__(3, 1000), {2}),
    "negative row": (lambda lens, cu, table: cu.__setitem__(0, -1), {0}),
    "offsets backwards": (lambda lens, cu, table: cu.__setitem__(1, int(cu[2]) + 1), {1}),    # one row named by two others
    "all": (lambda lens, cu, table: lens.fill_(-7), {0, 1, 2}),
}


@pytest.mark.parametrize("what", sorted(ATTEND))
@pytest.mark.parametrize("new", [FEW, MANY])
@pytest.mark.parametrize("dtype,d,layout", [(BF16, 128, "bhnd"), (FP16, 64, "bnhd")])
def test_attend_leaves_out_sequences_outside_the_tensors(what, new, dtype, d, layout):
    from temporal_block_sparse_sm_b200 import liteattn, serving
    g, mutate, (Hq, Hk) = _gen(1), ATTEND[what][0], (4, 2)
    ks, vs = ([_randn(g, m, Hk, d, dtype=dtype) for m in TOTAL] for _ in range(2))
    kp, vp, table = paged(ks, vs, 16, layout, g)
    plan = serving.GroupedPlan(Hq, Hk, d, dtype=dtype)
    lens, cu = torch.tensor(TOTAL, dtype=torch.int32, device="cuda"), offsets(new)
    q = _randn(g, sum(new) + 2, Hq, d, dtype=dtype)
    o = torch.full_like(q, 7.0)
    mutate(lens, cu, table)
    pools = kp.clone(), vp.clone()
    serving.PagedCache(plan, kp, vp, layout=layout).attend(q, o, lens, cu, table, max_new=max(new))
    assert _code(plan) == liteattn.LITE_ERR_DEVICE_CHECK
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(pools, (kp, vp)))
    named = [(int(cu[b]), int(cu[b + 1]), ks[b], vs[b]) for b in range(3) if b not in ATTEND[what][1]]
    _check_named_rows(q, o, named, d)


def _check_named_rows(q, o, named, d):
    """Rows of one sequence [i, j) with its keys and values hold its attention; rows of none are untouched; of a
    row that two sequences name it is only said that one of them writes it."""
    count = torch.zeros(q.shape[0], dtype=torch.int32, device="cuda")
    for i, j, _, _ in named:
        count[i:j] += 1
    for i, j, k, v in named:
        want, tol = seq_reference(q[i:j], k, v, True, d ** -0.5)
        alone = count[i:j] == 1
        assert_close(o[i:j][alone], want[alone], tol[alone], f"rows {i} to {j}")
    assert bool((o[count == 0] == 7).all()), "rows of a sequence that was left out were written"


@pytest.mark.parametrize("page", [1 << 20, -5, -(1 << 31), (1 << 31) - 1])
@pytest.mark.parametrize("new", [FEW, MANY])
@pytest.mark.parametrize("size,layout", [(16, "bhnd"), (64, "bnhd"), (128, "bhnd")])
def test_attend_takes_keys_of_a_page_that_does_not_exist_as_zeros(page, new, size, layout):
    from temporal_block_sparse_sm_b200 import liteattn, serving
    g, Hq, Hk, d = _gen(2), 4, 2, 128
    ks, vs = ([_randn(g, m, Hk, d) for m in TOTAL] for _ in range(2))
    kp, vp, table = paged(ks, vs, size, layout, g)
    plan = serving.GroupedPlan(Hq, Hk, d)
    lens, cu = torch.tensor(TOTAL, dtype=torch.int32, device="cuda"), offsets(new)
    q = _randn(g, sum(new), Hq, d)
    o = torch.full_like(q, 7.0)
    for b, j in ((0, 1), (2, (TOTAL[2] - 1) // size)):        # in the middle, and the last one
        table[b, j] = page
        ks[b][j * size:(j + 1) * size], vs[b][j * size:(j + 1) * size] = 0, 0
    serving.PagedCache(plan, kp, vp, layout=layout).attend(q, o, lens, cu, table, max_new=max(new))
    assert _code(plan) == liteattn.LITE_ERR_DEVICE_CHECK
    for b, n in enumerate(new):
        at = int(cu[b])
        want, tol = seq_reference(q[at:at + n], ks[b], vs[b], True, d ** -0.5)
        assert_close(o[at:at + n], want, tol, f"sequence {b}")


PROMPT = {
    "queries backwards": ("q", lambda cu, T: cu.__setitem__(1, int(cu[2]) + 1), {1}),
    "queries behind the tensor": ("q", lambda cu, T: cu.__setitem__(3, T + 1), {2}),
    "negative query row": ("q", lambda cu, T: cu.__setitem__(0, -3), {0}),
    "keys backwards": ("k", lambda cu, T: cu.__setitem__(1, int(cu[2]) + 1), {1}),
    "keys behind the tensor": ("k", lambda cu, T: cu.__setitem__(3, T + 1), {2}),
    "keys far behind": ("k", lambda cu, T: cu.__setitem__(3, (1 << 31) - 1), {2}),
    "negative key row": ("k", lambda cu, T: cu.__setitem__(0, -(1 << 31)), {0}),
}


@pytest.mark.parametrize("what", sorted(PROMPT))
@pytest.mark.parametrize("nq", [[3, 4, 5], [90, 40, 130]])
@pytest.mark.parametrize("dtype,d,Hq", [(BF16, 128, 1), (FP16, 64, 6)])
def test_prompt_leaves_out_sequences_outside_the_tensors(what, nq, dtype, d, Hq):
    from temporal_block_sparse_sm_b200 import liteattn, serving
    g, (side, mutate, out) = _gen(3), PROMPT[what]
    Hk = 1 if Hq == 1 else 2
    q, k, v = (_randn(g, n, h, d, dtype=dtype) for n, h in ((sum(nq) + 2, Hq), (sum(TOTAL) + 2, Hk), (sum(TOTAL) + 2, Hk)))
    cu_q, cu_k, plan, o = offsets(nq), offsets(TOTAL), serving.GroupedPlan(Hq, Hk, d, dtype=dtype), torch.full_like(q, 7.0)
    mutate(cu_q if side == "q" else cu_k, q.shape[0] if side == "q" else k.shape[0])
    plan.prompt(q, k, v, o, cu_q, cu_k)
    assert _code(plan) == liteattn.LITE_ERR_DEVICE_CHECK
    named = [(int(cu_q[b]), int(cu_q[b + 1]), k[int(cu_k[b]):int(cu_k[b + 1])], v[int(cu_k[b]):int(cu_k[b + 1])]) for b in range(3) if b not in out]
    _check_named_rows(q, o, named, d)


# what is wrong -> (lens, cu, table, pos) changed, the token rows left out (of 3 sequences of 2, 20 and 5 new tokens)
APPEND = {
    "nothing": (lambda lens, cu, table, pos: None, []),
    "page": (lambda lens, cu, table, pos: table.__setitem__((1, 3), 1 << 20), list(range(2, 16))),      # slots 50 to 63 of 50 to 69
    "negative page": (lambda lens, cu, table, pos: table.__setitem__((1, 4), -1), list(range(16, 22))),
    "long": (lambda lens, cu, table, pos: lens.__setitem__(1, 1 << 30), list(range(2, 22))),
    "negative length": (lambda lens, cu, table, pos: lens.__setitem__(0, -2), [0, 1]),
    "more new tokens than there are": (lambda lens, cu, table, pos: lens.__setitem__(2, 3), [22, 23]),
    "rows behind the tensor": (lambda lens, cu, table, pos: cu.__setitem__(3, 10 ** 6), list(range(22, 29))),
    "offsets backwards": (lambda lens, cu, table, pos: cu.__setitem__(1, -1), None),
    "angle row": (lambda lens, cu, table, pos: pos.__setitem__(5, 100), [5]),
    "negative angle row": (lambda lens, cu, table, pos: pos.__setitem__(24, -1), [24]),
}


@pytest.mark.parametrize("what", sorted(APPEND))
@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
def test_append_leaves_out_tokens_and_writes_nothing_else(what, layout):
    """Angles of 0, so that every accepted row is a copy: the pools and q_out are known bit for bit."""
    from temporal_block_sparse_sm_b200 import liteattn, serving
    g, Hq, Hk, d, page, new = _gen(4), 4, 2, 64, 16, [2, 20, 5]
    mutate, out = APPEND[what]
    plan = serving.GroupedPlan(Hq, Hk, d)
    shape = (20, Hk, page, d) if layout == "bhnd" else (20, page, Hk, d)
    kp, vp = (_randn(g, *shape) for _ in range(2))
    want_k, want_v = kp.clone(), vp.clone()
    cache = serving.PagedCache(plan, kp, vp, layout=layout)
    table = torch.randperm(20, generator=g, device="cuda")[:15].int().view(3, 5)
    lens, cu = torch.tensor([40, 70, 16], dtype=torch.int32, device="cuda"), offsets(new)
    T = sum(new) + 2                                            # two rows behind the last sequence
    q, k, v = (_randn(g, T, h, d) for h in (Hq, Hk, Hk))
    q_out = torch.full_like(q, 7.0)
    want_q = q_out.clone()
    cos, sin = serving.rotation_table([0] * 100, [1.0] * (d // 2), device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    good_lens, good_cu = lens.tolist(), cu.tolist()
    mutate(lens, cu, table, pos)
    cache.append(k, v, lens, cu, table, q=q, q_out=q_out, cos=cos, sin=sin, positions=pos)
    assert _code(plan) == (liteattn.LITE_ERR_DEVICE_CHECK if what != "nothing" else 0)
    if out is None:                                             # which tokens are still named is not said
        out = list(range(sum(new)))
        assert bool((q_out[sum(new):] == 7).all())
        for p, want in ((kp, want_k), (vp, want_v)):            # no slot but those of the new tokens
            slots = torch.zeros(shape[:1] + ((page,)), dtype=torch.bool, device="cuda")
            for b, n in enumerate(new):
                for s in range(good_lens[b] - n, good_lens[b] + 22):
                    if 0 <= s < 80:
                        slots[int(table[b, s // page]), s % page] = True
            same = (p == want).all(-1).all(1 if layout == "bhnd" else 2)
            assert bool((same | slots).all())
        return
    for b, n in enumerate(new):
        for i in range(n):
            t = good_cu[b] + i
            if t in out:
                continue
            slot = int(lens[b]) - n + i
            pg, r = int(table[b, slot // page]), slot % page
            at = (pg, slice(None), r) if layout == "bhnd" else (pg, r)
            want_k[at], want_v[at], want_q[t] = k[t], v[t], q[t]
    assert torch.equal(q_out, want_q) and torch.equal(kp, want_k) and torch.equal(vp, want_v)
