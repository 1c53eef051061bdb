"""Serving attention without a GPU: argument checks that come before any device call, the packed
argument blocks, the rotation table and the reference the GPU tests use."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from temporal_block_sparse_sm_b200 import build as lib_build
from temporal_block_sparse_sm_b200 import liteattn, serving
from tests.serving_ref import offsets, paged, seq_reference


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return liteattn.load()


@pytest.mark.parametrize("args,code", [
    ((0, 1, 64, 0), liteattn.LITE_ERR_INVALID_ARG), ((4, 0, 64, 0), liteattn.LITE_ERR_INVALID_ARG),
    ((4, 3, 64, 0), liteattn.LITE_ERR_INVALID_ARG), ((4, 2, 0, 0), liteattn.LITE_ERR_INVALID_ARG),
    ((4, 2, 64, 2), liteattn.LITE_ERR_INVALID_ARG), ((4, 2, 64, -1), liteattn.LITE_ERR_INVALID_ARG),
    ((4, 2, 96, 0), liteattn.LITE_ERR_UNSUPPORTED), ((4, 2, 256, 1), liteattn.LITE_ERR_UNSUPPORTED),
    ((129, 1, 64, 0), liteattn.LITE_ERR_UNSUPPORTED), ((1 << 17, 1 << 17, 64, 0), liteattn.LITE_ERR_UNSUPPORTED),
    ((128, 1, 64, 1), liteattn.LITE_ERR_ALLOC), ((28, 4, 128, 0), liteattn.LITE_ERR_ALLOC),   # valid: the injected fault
])
def test_plan_argument_checks(lib, monkeypatch, args, code):
    monkeypatch.setenv("LITE_ATTN_FAULT", "alloc")
    h = ctypes.c_void_p()
    assert lib.lite_attn_gqa_create(ctypes.byref(h), *args) == code
    assert not h.value
    assert lib.lite_attn_gqa_create(None, *args) == liteattn.LITE_ERR_INVALID_ARG


def test_null_handles_and_arguments(lib):
    n = ctypes.c_size_t()
    assert lib.lite_attn_gqa_destroy(None) == liteattn.LITE_OK
    assert lib.lite_attn_gqa_status(None, None) == liteattn.LITE_ERR_INVALID_ARG
    assert lib.lite_attn_gqa_workspace(None, 1, 1, 1, 1, ctypes.byref(n)) == liteattn.LITE_ERR_INVALID_ARG
    for fn, args in ((lib.lite_attn_cache_append, liteattn.AppendArgs()), (lib.lite_attn_cache_attend, liteattn.AttendArgs()),
                     (lib.lite_attn_prompt, liteattn.PromptArgs())):
        assert fn(None, ctypes.byref(args), None) == liteattn.LITE_ERR_INVALID_ARG
        assert fn(None, None, None) == liteattn.LITE_ERR_INVALID_ARG


def test_packed_arguments_match_the_structures():
    """The formats the object layer packs are the C structures, field by field."""
    for fmt, cls in ((serving._APPEND, liteattn.AppendArgs), (serving._ATTEND, liteattn.AttendArgs),
                     (serving._PROMPT, liteattn.PromptArgs)):
        assert fmt.size == ctypes.sizeof(cls)
        values = []

        def flat(c, base=0):
            for name, t in c._fields_:
                at = base + getattr(c, name).offset
                if issubclass(t, ctypes.Structure):
                    flat(t, at)
                else:
                    values.append((at, t))
        flat(cls)
        numbers = [0.5 if t is ctypes.c_float else 3 + i for i, (at, t) in enumerate(values)]
        blob = fmt.pack(*numbers)
        for (at, t), x in zip(values, numbers):
            assert t.from_buffer_copy(blob, at).value == x


def test_objects_need_a_known_type(lib, monkeypatch):
    with pytest.raises(ValueError):
        serving.GroupedPlan(4, 2, 64, dtype=torch.float32)
    monkeypatch.setenv("LITE_ATTN_FAULT", "alloc")
    with pytest.raises(liteattn.LiteAttnError) as e:
        serving.GroupedPlan(4, 2, 64)
    assert e.value.code == liteattn.LITE_ERR_ALLOC


def test_rotation_table():
    """Angles in 64 bits: at position 10^7 a 32-bit angle would be off by half a radian and more."""
    rates = [10000.0 ** (-2 * i / 64) for i in range(32)]
    cos, sin = serving.rotation_table([0, 1, 10_000_019], rates)
    assert cos.dtype == torch.float32 and cos.shape == (3, 32)
    for i, p in enumerate((0, 1, 10_000_019)):
        for j, w in enumerate(rates):
            assert abs(float(cos[i, j]) - math.cos(p * w)) < 2e-7 and abs(float(sin[i, j]) - math.sin(p * w)) < 2e-7
    # several axes: a position per pair
    pos = torch.tensor([[1.0, 5.0], [2.0, 7.0]])
    cos, sin = serving.rotation_table(pos, [0.5, 0.25])
    assert torch.allclose(cos.double(), torch.cos(pos.double() * torch.tensor([0.5, 0.25], dtype=torch.float64)), atol=1e-7)
    for bad in (torch.zeros(2, 3), torch.zeros(2, 2, 2)):
        with pytest.raises(ValueError):
            serving.rotation_table(bad, [0.5, 0.25])


# ---------------------------------------------------------------- the reference itself
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,m", [(1, 1), (4, 9), (9, 4), (3, 0)])
def test_reference_equals_sums_written_out(causal, n, m):
    g = torch.Generator().manual_seed(n * 10 + m)
    q, k, v = (torch.randn(t, h, 8, generator=g).bfloat16() for t, h in ((n, 4), (m, 2), (m, 2)))
    o, tol = seq_reference(q, k, v, causal, 0.3)
    for i in range(n):
        sees = max(0, m - n + i + 1) if causal else m
        for h in range(4):
            w = [math.exp(0.3 * float(q[i, h].double() @ k[j, h // 2].double())) for j in range(sees)]
            want = sum((x * v[j, h // 2].double() for j, x in enumerate(w)), torch.zeros(8, dtype=torch.float64))
            want = want / sum(w) if sees else want
            assert torch.allclose(o[i, h], want, atol=1e-12)
            assert bool((tol[i, h] >= 2.0 ** -8 * want.abs()).all())


def test_reference_leaves_hidden_places_out():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(5, 2, 8, generator=g).bfloat16() for _ in range(3))
    clean, _ = seq_reference(q, k, v, True, 0.3)
    v[4, 0, 2], k[4, 1, 1] = math.inf, math.nan
    o, _ = seq_reference(q, k, v, True, 0.3)
    assert torch.equal(o[:4], clean[:4]) and bool(torch.isinf(o[4, 0, 2])) and bool(torch.isnan(o[4, 1]).all())


@pytest.mark.parametrize("layout", ["bhnd", "bnhd"])
def test_paged_helper_round_trip(layout):
    g = torch.Generator().manual_seed(2)
    ks, vs = ([torch.randn(m, 2, 8, generator=g) for m in (5, 0, 33)] for _ in range(2))
    kp, vp, table = paged(ks, vs, 16, layout, g)
    for b, x in enumerate(ks):
        for j in range(x.shape[0]):
            pg = int(table[b, j // 16])
            assert torch.equal(kp[pg, :, j % 16] if layout == "bhnd" else kp[pg, j % 16], x[j])
    assert bool(torch.isnan(kp).any()) and offsets([2, 0, 3], device="cpu").tolist() == [0, 2, 2, 5]


def test_objects_call_the_binding_with_their_tensors(monkeypatch):
    """GroupedPlan and PagedCache hand addresses, lengths and strides to the binding's functions."""
    calls = []
    for name in ("lite_attn_prompt", "lite_attn_cache_append", "lite_attn_cache_attend"):
        monkeypatch.setattr(liteattn, name, lambda plan, args, stream=None, name=name: calls.append((name, plan, args, stream)))
    monkeypatch.setattr(liteattn, "lite_attn_gqa_workspace", lambda *a: 0)
    plan = object.__new__(serving.GroupedPlan)
    plan.Hq, plan.Hk, plan.d, plan.dtype, plan.device, plan.handle, plan._ws = 4, 2, 64, torch.bfloat16, 0, 77, {}
    plan._i32, plan._f32, plan._current = torch.int32, torch.float32, lambda device: 0
    x = torch.zeros(9, 8, 64, dtype=torch.bfloat16)
    q, k, v = x.split([4, 2, 2], dim=1)
    o = torch.zeros(9, 4, 64, dtype=torch.bfloat16)
    cu, lens, table = offsets([3, 6], "cpu"), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 5, dtype=torch.int32)
    plan.prompt(q, k, v, o, cu, scale=0.5, stream=5)
    cache = object.__new__(serving.PagedCache)
    cache.plan, cache.k_pages, cache.v_pages = plan, torch.zeros(7, 2, 16, 64), torch.zeros(7, 2, 16, 64)
    cache.pages, cache.page, cache._layout = 7, 16, liteattn.LITE_LAYOUT_BNHD
    cache._pool = cache.k_pages.data_ptr(), cache.v_pages.data_ptr(), 7
    cos, sin = serving.rotation_table(range(80), [1.0] * 16)
    cache.append(k, v, lens, cu, table, q=q, q_out=q, cos=cos, sin=sin, interleaved=True, stream=6)
    cache.attend(q, o, lens, cu, table, max_new=100, causal=False, stream=7)
    plan.handle = None                                          # nothing to free
    assert [(c[0], c[1], c[3]) for c in calls] == [("lite_attn_prompt", 77, 5), ("lite_attn_cache_append", 77, 6),
                                                   ("lite_attn_cache_attend", 77, 7)]
    args = [cls.from_buffer_copy(c[2]) for cls, c in zip((liteattn.PromptArgs, liteattn.AppendArgs, liteattn.AttendArgs), calls)]
    rows = lambda r: (r.ptr, r.tokens, r.stride_token, r.stride_head)   # noqa: E731
    view = lambda t: (t.data_ptr(), 9, t.stride(0), 64)                 # noqa: E731
    assert all(rows(getattr(args[0], n)) == view(t) for n, t in (("q", q), ("k", k), ("v", v), ("o", o)))
    assert (args[0].cu_q, args[0].cu_k, args[0].B, args[0].causal, args[0].scale) == (cu.data_ptr(), cu.data_ptr(), 2, 1, 0.5)
    assert all(rows(getattr(args[1], n)) == view(t) for n, t in (("q", q), ("q_out", q), ("k", k), ("v", v)))
    a = args[1]
    assert (a.k_pages, a.v_pages, a.pages, a.page, a.layout, a.table_width) == (*cache._pool, 16, liteattn.LITE_LAYOUT_BNHD, 5)
    assert (a.cos, a.sin, a.angle_rows, a.rot, a.interleaved, a.positions) == (cos.data_ptr(), sin.data_ptr(), 80, 32, 1, None)
    a = args[2]
    assert rows(a.q) == view(q) and rows(a.o) == view(o) and (a.max_new, a.causal, a.B) == (9, 0, 2)
    assert (a.cu_new, a.lens, a.table, a.scale) == (cu.data_ptr(), lens.data_ptr(), table.data_ptr(), 0.125)
