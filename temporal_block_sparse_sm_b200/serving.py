"""Serving attention: grouped query heads, packed sequences and a paged cache.

:class:`GroupedPlan` fixes the heads and the type; :meth:`GroupedPlan.prompt`
attends over whole packed sequences.  :class:`PagedCache` names a cache of
pages that the caller owns; :meth:`PagedCache.append` writes new tokens' keys
and values into it, rotated on the way, and :meth:`PagedCache.attend` lets the
new tokens attend over it (one token, a chunk, or a whole video frame).

Argument marshalling only, as in :mod:`.liteattn`: the work is done by the CUDA
library's ``lite_attn_prompt``, ``lite_attn_cache_append`` and
``lite_attn_cache_attend``, whose header comments give the conventions.  Lengths,
offsets and page tables stay on the device, so a captured graph can be replayed
on other lengths within the same tensors.
"""
from __future__ import annotations

import math
import struct
from typing import Optional, Sequence

from . import liteattn as _c

_APPEND = struct.Struct("=16q3q2q q 4q 6i")
_ATTEND = struct.Struct("=8q 3q 3q 2q 6i f i")
_PROMPT = struct.Struct("=16q 2q 2q 2i f i")
_NO_ROWS = (0, 0, 0, 0)


def rotation_table(positions, rates: Sequence[float], device=None):
    """cos and sin (float32 [n, len(rates)]) of the angles positions * rates, the angles in 64 bits.

    positions: [n] numbers, or [n, len(rates)] for a position of its own per pair (several
    axes: each pair takes the coordinate of the axis it belongs to)."""
    import torch
    p = torch.as_tensor(positions, dtype=torch.float64, device=device)
    w = torch.as_tensor(rates, dtype=torch.float64, device=p.device)
    if p.dim() == 1:
        p = p[:, None]
    if p.dim() != 2 or w.dim() != 1 or p.shape[1] not in (1, w.shape[0]):
        raise ValueError("positions must be [n] or [n, len(rates)]")
    angle = p * w
    return angle.cos().float().contiguous(), angle.sin().float().contiguous()


class GroupedPlan:
    """Hq query heads in groups over Hk key heads, head dim d (64 or 128), bf16 or fp16.

    The plan belongs to the device that is current when it is made.  It holds no
    scratch, so its calls may run on several streams at once.  Keep it as long as
    graphs that captured its calls are replayed."""

    def __init__(self, Hq: int, Hk: int, d: int, dtype=None):
        import torch
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("dtype must be torch.bfloat16 or torch.float16")
        self.Hq, self.Hk, self.d, self.dtype = int(Hq), int(Hk), int(d), dtype
        self.device = _c._current_device()
        self._torch, self._u8, self._i32, self._f32 = torch, torch.uint8, torch.int32, torch.float32
        self._dev = torch.device("cuda", self.device) if self.device is not None else None
        # the current stream's handle, without the stream object where torch offers that
        self._current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        self._ws = {}   # workspace bytes by (B, tokens, max_new, max_keys)
        self.handle = _c.lite_attn_gqa_create(self.Hq, self.Hk, self.d,
                                              _c.LITE_DTYPE_BF16 if dtype == torch.bfloat16 else _c.LITE_DTYPE_FP16)

    # ------------------------------------------------------------ arguments
    # (the library checks addresses and strides; these look at what it cannot see)
    def _stream(self, stream) -> int:
        if stream is None:
            return self._current(self.device)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _rows(self, t, heads: int, name: str):
        """(address, tokens, token stride, head stride) of a [tokens, heads, d] tensor."""
        if t.dtype is not self.dtype or t.dim() != 3:
            raise ValueError(f"{name} must be a CUDA tensor [tokens, {heads}, {self.d}] of {self.dtype}")
        n, h, d = t.shape
        st, sh, sd = t.stride()
        if h != heads or d != self.d or (sd != 1 and n):
            raise ValueError(f"{name} must be [tokens, {heads}, {self.d}] with contiguous rows of d")
        if h == 1:
            sh = d
        if n == 1 and st < h * d:
            st = h * d
        return t.data_ptr(), n, st, sh

    def _ints(self, t, n: int, name: str) -> int:
        if t.dtype is not self._i32 or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA int32 tensor of {n} elements")
        return t.data_ptr()

    def _workspace(self, B: int, tokens: int, max_new: int, max_keys: int, stream: int):
        key = (B, tokens, max_new, max_keys)
        n = self._ws.get(key)
        if n is None:
            if len(self._ws) >= 4096:
                self._ws.clear()
            n = self._ws[key] = _c.lite_attn_gqa_workspace(self.handle, B, tokens, max_new, max_keys)
        if not n:
            return None
        # from the caching allocator, on the call's own stream: reused in that stream's order, and a
        # captured graph's workspace is the graph's own
        torch = self._torch
        if stream == self._current(self.device):
            return torch.empty(n, dtype=self._u8, device=self._dev)
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=self._dev)):
            return torch.empty(n, dtype=self._u8, device=self._dev)

    def _scale(self, scale: Optional[float]) -> float:
        return 1.0 / math.sqrt(self.d) if scale is None else float(scale)

    # ------------------------------------------------------------ calls
    def prompt(self, q, k, v, o, cu_q, cu_k=None, causal: bool = True, scale: Optional[float] = None, stream=None):
        """Attention over packed sequences into o.

        q, o: [tokens, Hq, d]; k, v: [tokens, Hk, d]; cu_q, cu_k (default cu_q): int32
        [B + 1] row offsets.  With causal, the queries are the last of the sequence's
        positions."""
        rq, ro = self._rows(q, self.Hq, "q"), self._rows(o, self.Hq, "o")
        rk, rv = self._rows(k, self.Hk, "k"), self._rows(v, self.Hk, "v")
        cu_k = cu_q if cu_k is None else cu_k
        B = cu_q.numel() - 1
        s = self._stream(stream)
        w = self._workspace(B, rq[1], rq[1], rk[1], s)
        args = _PROMPT.pack(*rq, *ro, *rk, *rv, self._ints(cu_q, B + 1, "cu_q"), self._ints(cu_k, B + 1, "cu_k"),
                            w.data_ptr() if w is not None else 0, w.shape[0] if w is not None else 0, B,
                            1 if causal else 0, self._scale(scale), 0)
        _c.lite_attn_prompt(self.handle, args, s)

    def check(self, stream=None):
        """Waits for the stream and raises if a kernel of this plan reported an error."""
        _c.lite_attn_gqa_status(self.handle, self._stream(stream))

    def close(self):
        if getattr(self, "handle", None):
            _c.lite_attn_gqa_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedCache:
    """A paged cache of keys and values over tensors that the caller owns.

    k_pages, v_pages: contiguous [pages, Hk, page, d] ("bhnd") or [pages, page, Hk, d]
    ("bnhd"), page a power of two from 16 on.  Which pages belong to which sequence is
    said by each call's table: int32 [B, width], entry [b, j] the page that holds
    positions [j * page, (j + 1) * page) of sequence b (entries behind its length are not
    read)."""

    def __init__(self, plan: GroupedPlan, k_pages, v_pages, layout: str = "bhnd"):
        if layout not in _c._LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(_c._LAYOUTS)}")
        self.plan, self.k_pages, self.v_pages, self.layout = plan, k_pages, v_pages, layout
        self._layout = _c._LAYOUTS[layout]
        self._pool = self._check_pages()

    def _check_pages(self):
        """(addresses, number) of the pages, after a look at the tensors."""
        plan, k_pages, v_pages = self.plan, self.k_pages, self.v_pages
        for t, nm in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if t.dim() != 4 or not t.is_cuda or t.dtype != plan.dtype or not t.is_contiguous() or t.shape != k_pages.shape:
                raise ValueError(f"{nm} must be a contiguous CUDA tensor of {plan.dtype} with four dimensions")
        heads, page = (1, 2) if self.layout == "bhnd" else (2, 1)
        if k_pages.shape[heads] != plan.Hk or k_pages.shape[3] != plan.d:
            raise ValueError(f"the pages must hold {plan.Hk} heads of {plan.d}")
        self.pages, self.page = k_pages.shape[0], k_pages.shape[page]
        if self.page < 16 or self.page & (self.page - 1):
            raise ValueError("a page must hold a power of two of tokens, 16 or more")
        return k_pages.data_ptr(), v_pages.data_ptr(), self.pages

    def append(self, k, v, lens, cu_new, table, q=None, q_out=None, cos=None, sin=None, positions=None,
               interleaved: bool = False, stream=None):
        """New tokens' k and v ([tokens, Hk, d]) into the cache; q ([tokens, Hq, d]) into q_out.

        lens: int32 [B], tokens of each sequence including the new ones; cu_new: int32
        [B + 1], the rows of each sequence's new tokens; table: as above.  With cos and
        sin (float32 [rows, rot / 2], see rotation_table) the first rot elements of the heads
        of q and k are rotated by the token's row (positions: int32 [tokens]; default the
        token's position in the cache), in pairs (i, i + rot / 2) or, interleaved, (2i, 2i + 1)."""
        p = self.plan
        rk, rv = p._rows(k, p.Hk, "k"), p._rows(v, p.Hk, "v")
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out come together")
        rq, ro = (p._rows(q, p.Hq, "q"), p._rows(q_out, p.Hq, "q_out")) if q is not None else (_NO_ROWS, _NO_ROWS)
        if (cos is None) != (sin is None) or (cos is None and positions is not None):
            raise ValueError("cos and sin come together, positions with them")
        a, rot = (0, 0, 0), 0
        if cos is not None:
            f32 = p._f32
            if cos.dtype is not f32 or sin.dtype is not f32 or cos.dim() != 2 or sin.shape != cos.shape or not (
                    cos.is_contiguous() and sin.is_contiguous()):
                raise ValueError("cos and sin must be contiguous CUDA float32 tensors [rows, rot / 2]")
            rows, half = cos.shape
            rot = 2 * half
            if rot % 16 or not 16 <= rot <= p.d:
                raise ValueError("rot must be a multiple of 16, at most d")
            a = (cos.data_ptr(), sin.data_ptr(), rows)
        pool = self._pool      # the pages where they are now: the caller may have given the tensors other memory
        if self.k_pages.data_ptr() != pool[0] or self.v_pages.data_ptr() != pool[1]:
            pool = self._pool = self._check_pages()
        B, width = cu_new.numel() - 1, table.shape[-1]
        args = _APPEND.pack(*rq, *ro, *rk, *rv, *pool, *a,
                            p._ints(positions, rk[1], "positions") if positions is not None else 0,
                            p._ints(cu_new, B + 1, "cu_new"), p._ints(lens, B, "lens"),
                            p._ints(table, B * width, "table"), B, width, self.page, self._layout, rot, 1 if interleaved else 0)
        _c.lite_attn_cache_append(p.handle, args, p._stream(stream))

    def attend(self, q, o, lens, cu_new, table, max_new: int, causal: bool = True, scale: Optional[float] = None,
               stream=None):
        """Attention of the new tokens q ([tokens, Hq, d]) over the cache into o.

        lens, cu_new, table: as for append (lens includes the new tokens, which have been
        appended).  max_new: an upper bound of the new tokens of a sequence, known on the
        host; it selects the kernel.  causal=False: every new token sees all keys of its
        sequence."""
        p = self.plan
        rq, ro = p._rows(q, p.Hq, "q"), p._rows(o, p.Hq, "o")
        pool = self._pool      # as in append
        if self.k_pages.data_ptr() != pool[0] or self.v_pages.data_ptr() != pool[1]:
            pool = self._pool = self._check_pages()
        B, width = cu_new.numel() - 1, table.shape[-1]
        if max_new > rq[1]:
            max_new = rq[1]
        s = p._stream(stream)
        w = p._workspace(B, rq[1], max_new, width * self.page, s)
        args = _ATTEND.pack(*rq, *ro, *pool, p._ints(cu_new, B + 1, "cu_new"), p._ints(lens, B, "lens"),
                            p._ints(table, B * width, "table"), w.data_ptr() if w is not None else 0,
                            w.shape[0] if w is not None else 0, B, width, self.page, self._layout, max_new,
                            1 if causal else 0, p._scale(scale), 0)
        _c.lite_attn_cache_attend(p.handle, args, s)
