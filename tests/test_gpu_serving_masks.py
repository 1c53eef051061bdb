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
