"""Serving attention on the GPU where rows see only part of a key tile: what hidden places hold, and
what becomes of the shared memory that held it, against the 64-bit reference of tests/serving_ref.py."""
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


def _attend(q, ks, vs, new, page=16, layout="bhnd", causal=True, scale=None, seed=0, fill=None):
    """attend over pools that hold the sequences ks, vs: (o, the reference per sequence, its bound)."""
    from temporal_block_sparse_sm_b200 import serving
    Hq, d = q.shape[1:]
    kp, vp, table = paged(ks, vs, page, layout, _gen(seed), fill=fill)
    plan = serving.GroupedPlan(Hq, ks[0].shape[1], d, dtype=q.dtype)
    o = torch.full_like(q, 7.0)
    lens = torch.tensor([x.shape[0] for x in ks], dtype=torch.int32, device="cuda")
    serving.PagedCache(plan, kp, vp, layout=layout).attend(q, o, lens, offsets(new), table, max_new=max(new), causal=causal, scale=scale)
    plan.check()
    at, refs = 0, []
    for n, k, v in zip(new, ks, vs):
        refs.append((slice(at, at + n), *seq_reference(q[at:at + n], k, v, causal, 1 / math.sqrt(d) if scale is None else scale)))
        at += n
    return o, refs


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (FP16, 64)])
@pytest.mark.parametrize("new", [1, 3])
def test_stages_with_hidden_values_are_used_again(dtype, d, new):
    """Many short sequences whose last tile is partial, so that a block's ring stages hold zeroed values
    and then the next item's keys and values many times over."""
    g = _gen(3)
    lens = [17 + (37 * b) % 230 for b in range(700)]
    ks, vs = ([torch.randn(m, 2, d, generator=g, device="cuda").to(dtype) for m in lens] for _ in range(2))
    q = torch.randn(new * len(lens), 4, d, generator=g, device="cuda").to(dtype)
    o, refs = _attend(q, ks, vs, [new] * len(lens))
    for b, (rows, want, tol) in enumerate(refs):
        assert_close(o[rows], want, tol, f"sequence {b}")


def _one_key_and_many_far_ones(dtype, d, new, m, gap, far):
    """q and keys such that key 0 has the logit `gap` (in powers of two of the weight) above all others,
    which are equal; the values of key 0 are 0, the others' +-far by column."""
    q = torch.zeros(new, 2, d, device="cuda")
    k, v = torch.zeros(m, 1, d, device="cuda"), torch.zeros(m, 1, d, device="cuda")
    q[..., 0] = 1.0
    k[0, 0, 0] = gap
    v[1:] = far * torch.where(torch.arange(d, device="cuda") % 2 == 0, 1.0, -1.0)
    return q.to(dtype), k.to(dtype), v.to(dtype), math.log(2.0)


@pytest.mark.parametrize("dtype,far", [(FP16, 6e4), (BF16, 1e4)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gap,m", [(100, 1000), (40, 9000), (12, 1000)])
def test_weights_far_below_the_largest_count_as_what_they_are(dtype, far, d, gap, m):
    """Keys 2^-gap below the largest weight, whose key has no value: nothing is added to them, and what
    little they weigh (in fp16 down to 2^-32 of the largest) is not lost."""
    q, k, v, scale = _one_key_and_many_far_ones(dtype, d, 1, m, gap, far)
    o, refs = _attend(q, [k], [v], [1], scale=scale)
    for rows, want, tol in refs:
        assert_close(o[rows], want, tol)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("new", [1, 4, 40])
@pytest.mark.parametrize("gap", [0, 3, 30])
def test_values_that_are_not_finite_and_seen_by_all(dtype, value, new, gap):
    """An infinite value seen by every row, in the middle of a long cache and at its end, under a weight that
    is exactly a power of two and however small: the column is that infinity, or NaN, and no other is."""
    q, k, v, scale = _one_key_and_many_far_ones(dtype, 128, new, 700, gap, 2.0)
    for j, c in ((5, 7), (333, 8), (695, 100)):
        v[j, 0, c] = value
    v[40, 0, 8] = -value
    o, refs = _attend(q, [k], [v], [new], scale=scale, causal=False)
    for rows, want, tol in refs:
        assert_close(o[rows], want, tol)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("new", [1, 4, 40])
@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 15, 181 * 2.0 ** 4, 181 * 2.0 ** 7, 149 * 2.0 ** 8, 171 * 2.0 ** 8, 201 * 2.0 ** 8, 233 * 2.0 ** 8, 253 * 2.0 ** 8, 214 * 2.0 ** 8])
@pytest.mark.parametrize("where", [0, 500, 699])
def test_logits_so_large_that_a_key_or_two_take_all(dtype, new, size, where):
    """Logits of up to 4e8, exact in 32 bits (one product each): the keys with the largest, and no others,
    share the weight, whatever 2^x makes of arguments this far from zero."""
    d, m = 64, 700
    g = _gen(5)
    q, k = torch.zeros(new, 2, d, device="cuda"), torch.zeros(m, 1, d, device="cuda")
    q[:, 0, 0], q[:, 1, 1] = size, -size                       # head 0 sees column 0 of k, head 1 the negative of column 1
    k[:, 0, 0] = -size * (1 + torch.arange(m, device="cuda") % 3) / 4
    k[:, 0, 1] = size * 0.5
    k[where, 0, 0], k[where, 0, 1] = size, -size
    k[100, 0, 1] = -size
    v = torch.randn(m, 1, d, generator=g, device="cuda").to(dtype)
    q, k = q.to(dtype), k.to(dtype)
    o, _ = _attend(q, [k], [v], [new], scale=0.125, causal=False)
    want = torch.stack([v[where, 0].double(), (v[where, 0].double() + v[100, 0].double()) / 2])
    # weights and output are rounded to the type, 2^-22 of each for 2^x and the sums
    u = torch.finfo(dtype).eps / 2
    tol = (2 * u / (1 - u) + 2.0 ** -18) * torch.stack([v[where, 0].double().abs(), (v[where, 0].double().abs() + v[100, 0].double().abs()) / 2]) + u * want.abs()
    assert_close(o, want.expand(new, 2, d), (tol + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps).expand(new, 2, d))


@pytest.mark.parametrize("dtype,d", [(FP16, 128), (BF16, 64)])
@pytest.mark.parametrize("new", [3, 50])
def test_a_query_that_is_not_finite_spoils_its_own_row_only(dtype, d, new):
    g = _gen(6)
    k, v = (torch.randn(400, 2, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn(new, 4, d, generator=g, device="cuda").to(dtype)
    q[1, 2, 5], q[2, 0, 0], q[0, 3, 1] = math.nan, math.inf, -math.inf
    o, refs = _attend(q, [k], [v], [new])
    clean = q.clone()
    clean[1, 2, 5], clean[2, 0, 0], clean[0, 3, 1] = 0, 0, 0
    want, tol = seq_reference(clean, k, v, True, d ** -0.5)
    spoilt = torch.zeros(new, 4, dtype=torch.bool, device="cuda")
    spoilt[1, 2], spoilt[2, 0], spoilt[0, 3] = True, True, True
    assert bool(torch.isnan(o[spoilt]).all())
    assert_close(o[~spoilt], want[~spoilt], tol[~spoilt])
