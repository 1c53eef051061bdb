"""64-bit reference of the serving attention calls, and the error bound they are held to.

One sequence at a time, from the definition: row i of the n queries sees the first
m - n + i + 1 of the m keys (causal) or all of them, o_i = sum_j w_ij v_j with
w_i = softmax(scale q_i . k_j) over what it sees, zero when it sees nothing.  Keys that a
row does not see are left out of its sums altogether.

The bound, per element.  Let u = eps / 2 of the 16-bit type (a rounding is off by at most
half a step), A = sum_j w_j |v_j| and o the exact output.
* The weights enter the product rounded to 16 bits, w_j (1 + e_j) with |e_j| <= u, and are
  normalised by the sum of the weights before or after that rounding: the result moves by at most
  u A, or |sum w_j e_j (v_j - o)| / (1 - u) <= u (A + |o|) / (1 - u) <= 2 u A / (1 - u).
* A logit is a sum of d products in 32 bits: off by at most d 2^-23 scale sum |q||k| =: s
  (twice the half-step, for accumulations that do not round to nearest), so a weight is off by
  a factor within exp(+-2 s) after normalisation: 2 (exp(2 s) - 1) A.
* The exponential is off by at most x = 2^-18 (the hardware's 2^x is off by 2^-22: in the weight, and
  in each rescaling of the sums that hold it, of which 15 are allowed for); and its argument, held
  in 32 bits, by 2^-23 of its own size (the size of the logits, at most 2 * scale sum |q||k|), so
  2 (x + 2^-22 L) A.
* Sums of m terms in 32 bits, in an order that is not fixed here: 2^-24 m^(1/2) would be typical,
  2^-24 m is sure: 2 m 2^-24 A.
* The output is rounded once: u |o| (and half the smallest step of the type).
"""
from __future__ import annotations

import math

import torch


def seq_reference(q, k, v, causal, scale):
    """(o, bound) of one sequence in 64 bits: q [n, Hq, d], k, v [m, Hk, d] of a 16-bit type."""
    n, Hq, d = q.shape
    m, Hk = k.shape[0], k.shape[1]
    G = Hq // Hk
    dt = q.dtype
    u = torch.finfo(dt).eps / 2
    x = 2.0 ** -18
    o = torch.zeros(n, Hq, d, dtype=torch.float64, device=q.device)
    tol = torch.full_like(o, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps)
    sees = torch.arange(n, device=q.device) + (m - n + 1) if causal else torch.full((n,), m, device=q.device)
    hide = torch.arange(m, device=q.device)[None, :] >= sees[:, None]
    rows = sees > 0
    if n == 0 or m == 0:
        return o, tol
    for h in range(Hq):
        kk, vv = k[:, h // G].double(), v[:, h // G].double()
        s = scale * (q[:, h].double() @ kk.T)
        s = torch.where(hide, torch.full_like(s, -math.inf), s)
        w = torch.softmax(s, dim=1)
        w = torch.where(hide, torch.zeros_like(w), w)
        size = torch.where(hide, torch.zeros_like(s), scale * (q[:, h].double().abs() @ kk.abs().T)).amax(1, keepdim=True)
        if bool(torch.isfinite(vv).all()):
            oh, A = w @ vv, w @ vv.abs()
        else:   # hidden places must not reach a row's sum as 0 * inf
            oh, A = torch.zeros(n, d, dtype=torch.float64, device=q.device), torch.zeros(n, d, dtype=torch.float64, device=q.device)
            for i in range(n):
                c = max(0, min(m, int(sees[i])))
                oh[i], A[i] = w[i, :c] @ vv[:c], w[i, :c] @ vv[:c].abs()
        sl = d * 2.0 ** -23 * size
        err = (2 * u / (1 - u) + 2 * torch.expm1(2 * sl) + 2 * (x + 2.0 ** -22 * size) + 2 * m * 2.0 ** -24) * A + u * oh.abs()
        o[:, h] = torch.where(rows[:, None], oh, torch.zeros_like(oh))
        tol[:, h] += torch.where(rows[:, None], err, torch.zeros_like(err))
    return o, tol


def assert_close(got, want, tol, what=""):
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    bad = (got - want).abs() > tol
    bad &= fine
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} elements off, worst "
                                 f"{float(((got - want).abs() / tol)[fine].max()):.3f} of the bound")


def offsets(lens, device="cuda", start=0):
    out = [start]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=device)


def paged(k_seqs, v_seqs, page, layout, gen, spare=3, fill=None, width=None):
    """Pools and a shuffled table holding the sequences' keys and values; every other place of
    the pools holds `fill` (NaN by default), unused table entries -1 or a far page number."""
    Hk, d = k_seqs[0].shape[1:]
    dt, dev = k_seqs[0].dtype, k_seqs[0].device
    need = [-(-x.shape[0] // page) for x in k_seqs]
    num = sum(need) + spare
    fill = float("nan") if fill is None else fill
    order = torch.randperm(num, generator=gen, device=dev)
    pools = [torch.full((num, Hk, page, d), fill, dtype=dt, device=dev) for _ in range(2)]
    width = max(1, max(need)) if width is None else width
    table = torch.full((len(k_seqs), width), -1, dtype=torch.int32, device=dev)
    table[:, 1::2] = 1 << 30
    at = 0
    for b, x in enumerate(k_seqs):
        ids = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = ids.int()
        for pool, src in zip(pools, (x, v_seqs[b])):
            for j in range(need[b]):
                part = src[j * page:(j + 1) * page]
                pool[ids[j], :, :part.shape[0]] = part.transpose(0, 1)
    if layout == "bnhd":
        pools = [x.transpose(1, 2).contiguous() for x in pools]
    return pools[0], pools[1], table
