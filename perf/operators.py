"""Cases of the serving attention operators: rotating and appending keys and values to a
paged cache, attention of new tokens over that cache, and attention over whole prompts.

Every case is one call on ragged batches of sequences.  `prepare` makes its inputs on the
GPU, `run` makes one pass (the plain form in elementary torch operations, or the library's
call where `own` is true), `exact` gives the same outputs from the definition in 64 bits and
`work` the bytes and operations that the call cannot do without."""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token for each of 64 running sequences: latency of a decoding step
        dict(name="append-64x1", op="append", B=64, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=2000, pad=0, Hq=32, Hk=8, d=128,
             rot=128, interleaved=False, page=16, layout="bnhd", dtype="bf16", fused=True, own_pos=False, shape=1),
        # a few prompts entering the cache at once, adjacent-pair rotation, padded batch
        dict(name="append-9-prompts", op="append", B=9, new_lo=1, new_hi=4000, ctx_lo=0, ctx_hi=0, pad=37, Hq=24, Hk=4, d=128,
             rot=128, interleaved=True, page=64, layout="bhnd", dtype="bf16", fused=False, own_pos=False, shape=2),
        # one video frame of 1560 tokens joining 20 cached ones, rotation index from its grid cell
        dict(name="append-frame", op="append", B=1, new_lo=1560, new_hi=1560, ctx_lo=31200, ctx_hi=31200, pad=0, Hq=12, Hk=12,
             d=128, rot=96, interleaved=True, page=128, layout="bhnd", dtype="fp16", fused=True, own_pos=True, shape=3),
        # a single token of a single short sequence: the smallest call
        dict(name="attend-1x1", op="attend", B=1, new_lo=1, new_hi=1, ctx_lo=999, ctx_hi=999, pad=0, Hq=32, Hk=8, d=128,
             page=16, layout="bnhd", dtype="bf16", causal=True, shape=4),
        # single tokens of 64 sequences of very different lengths: an ordinary decoding step
        dict(name="attend-64x1", op="attend", B=64, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=8191, pad=0, Hq=32, Hk=8, d=128,
             page=64, layout="bhnd", dtype="bf16", causal=True, shape=5),
        # a single token over the 108000 cached tokens of a long video, six query heads to a key head
        dict(name="attend-1x1-long", op="attend", B=1, new_lo=1, new_hi=1, ctx_lo=107999, ctx_hi=107999, pad=0, Hq=24, Hk=4,
             d=128, page=128, layout="bhnd", dtype="fp16", causal=True, shape=6),
        # a video frame of 1560 tokens attending to all of itself and to the 20 frames before it
        dict(name="attend-frame", op="attend", B=1, new_lo=1560, new_hi=1560, ctx_lo=31200, ctx_hi=31200, pad=0, Hq=12, Hk=12,
             d=128, page=128, layout="bnhd", dtype="bf16", causal=False, shape=7),
        # prompts entering in chunks beside sequences that decode: ragged on both sides
        dict(name="attend-chunks", op="attend", B=11, new_lo=1, new_hi=513, ctx_lo=0, ctx_hi=16001, pad=5, Hq=16, Hk=4, d=64,
             page=16, layout="bnhd", dtype="bf16", causal=True, shape=8),
        # one short prompt: latency to its first token
        dict(name="prompt-1x200", op="prompt", B=1, q_lo=200, q_hi=200, more_lo=0, more_hi=0, pad=0, Hq=32, Hk=8, d=128,
             dtype="bf16", causal=True, fused=True, shape=9),
        # sixteen packed prompts of different lengths
        dict(name="prompt-16-packed", op="prompt", B=16, q_lo=1, q_hi=2048, more_lo=0, more_hi=0, pad=3, Hq=32, Hk=8, d=128,
             dtype="bf16", causal=True, fused=False, shape=10),
        # one sequence of the 32760 tokens of a video, token by token in time
        dict(name="prompt-32760", op="prompt", B=1, q_lo=32760, q_hi=32760, more_lo=0, more_hi=0, pad=0, Hq=12, Hk=12, d=128,
             dtype="bf16", causal=True, fused=False, shape=11),
        # smaller heads, keys longer or shorter than the queries: some rows see nothing
        dict(name="prompt-5-uneven", op="prompt", B=5, q_lo=100, q_hi=4096, more_lo=-300, more_hi=3000, pad=0, Hq=28, Hk=4, d=64,
             dtype="fp16", causal=True, fused=False, shape=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "prompt"])
    Hk = rng.choice([1, 2, 3, 4, 8, 12])
    group = rng.choice([1, 1, 2, 3, 4, 5, 6, 7, 8, 12])
    c = dict(op=op, Hq=Hk * group, Hk=Hk, d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "fp16"]),
             pad=rng.choice([0, 0, 1, 19]), shape=rng.randrange(1 << 30))
    if op == "prompt":
        B = _log(rng, 1, 32)
        hi = _log(rng, 1, 20000)
        # no more products than the largest listed case
        while B * c["Hq"] * hi * (hi + 1) * c["d"] > 12 * 32760 * 32760 * 128:
            hi = max(1, hi // 2)
        c.update(B=B, q_lo=rng.choice([1, max(1, hi // 2), hi]), q_hi=hi, more_lo=0, more_hi=0,
                 causal=rng.random() < 0.8, fused=False)
        if rng.random() < 0.4:
            c.update(more_lo=-rng.randrange(1, 50), more_hi=rng.randrange(0, 2000))
        elif rng.random() < 0.5:
            c.update(fused=True)
        return c
    B = _log(rng, 1, 96)
    hi = rng.choice([1, 1, 2, 3, _log(rng, 4, 2000)])
    ctx = _log(rng, 1, 100000)
    while B * (ctx + hi) * Hk * c["d"] > 1 << 28 or B * hi * (ctx + hi) * c["Hq"] * c["d"] > 1 << 36:
        B, ctx, hi = max(1, B - B // 3), max(1, ctx // 2), max(1, hi - hi // 3)
    c.update(B=B, new_lo=rng.choice([1, hi]), new_hi=hi, ctx_lo=rng.choice([0, ctx]), ctx_hi=ctx,
             page=rng.choice([16, 32, 64, 128, 256]), layout=rng.choice(["bhnd", "bnhd"]))
    if op == "append":
        c.update(rot=rng.choice([c["d"], c["d"], c["d"] // 2, c["d"] - 16]), interleaved=rng.random() < 0.5,
                 fused=rng.random() < 0.5, own_pos=rng.random() < 0.3)
    else:
        c.update(causal=rng.random() < 0.8)
    return c


def _lengths(c):
    """The case's ragged lengths: new (or query) tokens and cached (or key) tokens per sequence."""
    r = random.Random(c["shape"])
    if c["op"] == "prompt":
        new = [r.randint(c["q_lo"], c["q_hi"]) for _ in range(c["B"])]
        return new, [max(0, n + r.randint(c["more_lo"], c["more_hi"])) for n in new]
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    return new, [n + r.randint(c["ctx_lo"], c["ctx_hi"]) for n in new]


def _visible(c, n, m):
    """Pairs of one query row and one key row that it sees, of a sequence of n queries and m keys."""
    if not c["causal"]:
        return n * m
    first = m - n + 1                       # keys that the first query sees
    return sum(max(0, first + i) for i in range(n))


def work(c):
    new, total = _lengths(c)
    T, d, Hq, Hk = sum(new), c["d"], c["Hq"], c["Hk"]
    if c["op"] == "append":
        rows = set() if c["own_pos"] else {m - n + i for n, m in zip(new, total) for i in range(n)}
        angles = (T if c["own_pos"] else len(rows)) * c["rot"] * 4
        return {"bytes": 2 * 2 * T * (Hq + 2 * Hk) * d + angles, "flops": 3 * T * (Hq + Hk) * c["rot"]}
    pairs = sum(_visible(c, n, m) for n, m in zip(new, total))
    return {"bytes": 2 * d * (2 * Hq * T + 2 * Hk * sum(total)), "flops": 4 * Hq * d * pairs}


# ------------------------------------------------------------------------------ inputs
def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _pages(c, total, g):
    """A shuffled page table with room for every sequence; unused entries name no page."""
    page = c["page"]
    need = [-(-m // page) for m in total]
    num = sum(need) + 3
    order = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["B"], max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return num, table


def _tokens(c, T, g, dt, heads):
    """[T, h, d] tensors for each h in heads: views of one fused projection, or separate."""
    d = c["d"]
    x = [torch.randn(T, h, d, generator=g, device="cuda").mul_(1.25).to(dt) for h in heads]
    if c.get("fused"):
        x = list(torch.cat(x, dim=1).split(list(heads), dim=1))
    return x


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    new, total = _lengths(c)
    T, d, Hq, Hk = sum(new) + c["pad"], c["d"], c["Hq"], c["Hk"]
    s = dict(c=c, new=new, total=total, cu=_offsets(new))
    if c["op"] == "prompt":
        if c["fused"]:
            s["q"], s["k"], s["v"] = _tokens(c, T, g, dt, (Hq, Hk, Hk))
        else:
            s["q"], = _tokens(c, T, g, dt, (Hq,))
            s["k"], s["v"] = _tokens(c, sum(total) + c["pad"], g, dt, (Hk, Hk))
        s["cu_k"] = _offsets(total)
        s["o"] = torch.zeros(T, Hq, d, dtype=dt, device="cuda")
    else:
        num, s["table"] = _pages(c, total, g)
        s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
        shape = (num, Hk, c["page"], d) if c["layout"] == "bhnd" else (num, c["page"], Hk, d)
        s["kp"], s["vp"] = (torch.randn(shape, generator=g, device="cuda", dtype=dt).mul_(1.25) for _ in range(2))
        if c["op"] == "attend":
            s["q"], = _tokens(c, T, g, dt, (Hq,))
            s["o"] = torch.zeros(T, Hq, d, dtype=dt, device="cuda")
        else:
            s["q"], s["k"], s["v"] = _tokens(c, T, g, dt, (Hq, Hk, Hk))
            s["qr"] = torch.zeros(T, Hq, d, dtype=dt, device="cuda")
            n_rows = max(total) if not c["own_pos"] else 1 + max(total) // 2
            half = c["rot"] // 2
            freq = torch.arange(half, dtype=torch.float64, device="cuda").div(-half).mul(math.log(10000.0)).exp()
            angle = torch.arange(n_rows, dtype=torch.float64, device="cuda")[:, None] * freq
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
            s["pos"] = torch.randint(0, n_rows, (T,), generator=g, device="cuda", dtype=torch.int32) if c["own_pos"] else None
    if own:
        from temporal_block_sparse_sm_b200 import serving

        s["plan"] = serving.GroupedPlan(Hq, Hk, d, dtype=dt)
        if c["op"] != "prompt":
            s["cache"] = serving.PagedCache(s["plan"], s["kp"], s["vp"], layout=c["layout"])
    return s


# ------------------------------------------------------------------------------ one pass
def run(s):
    c = s["c"]
    if own:
        if c["op"] == "append":
            s["cache"].append(s["k"], s["v"], s["lens"], s["cu"], s["table"], q=s["q"], q_out=s["qr"], cos=s["cos"],
                              sin=s["sin"], positions=s["pos"], interleaved=c["interleaved"])
            return {"q": s["qr"], "k": s["kp"], "v": s["vp"]}
        if c["op"] == "attend":
            s["cache"].attend(s["q"], s["o"], s["lens"], s["cu"], s["table"], max_new=max(s["new"]), causal=c["causal"])
        else:
            s["plan"].prompt(s["q"], s["k"], s["v"], s["o"], s["cu"], cu_k=s["cu_k"], causal=c["causal"])
        return {"o": s["o"]}
    return {"append": _plain_append, "attend": _plain_attend, "prompt": _plain_prompt}[c["op"]](s)


def _rotate(x, cos, sin, rot, interleaved):
    """x [T, H, d] in 32 bits, its first `rot` elements rotated pair by pair by cos, sin [T, rot / 2]."""
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    ra, rb = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([ra, rb], dim=-1).flatten(-2) if interleaved else torch.cat([ra, rb], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_append(s):
    c, dt = s["c"], s["q"].dtype
    n_new = (s["cu"][1:] - s["cu"][:-1]).long()
    T = sum(s["new"])
    seq = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), n_new, output_size=T)
    slot = torch.arange(T, device="cuda") - s["cu"][:-1].long()[seq] + (s["lens"].long() - n_new)[seq]
    at = (s["pos"][:T] if s["pos"] is not None else slot).long()
    cos, sin = s["cos"][at], s["sin"][at]
    s["qr"][:T] = _rotate(s["q"][:T].float(), cos, sin, c["rot"], c["interleaved"]).to(dt)
    kr = _rotate(s["k"][:T].float(), cos, sin, c["rot"], c["interleaved"]).to(dt)
    page, row = s["table"][seq, slot // c["page"]].long(), slot % c["page"]
    if c["layout"] == "bhnd":
        s["kp"][page, :, row] = kr
        s["vp"][page, :, row] = s["v"][:T]
    else:
        s["kp"][page, row] = kr
        s["vp"][page, row] = s["v"][:T]
    return {"q": s["qr"], "k": s["kp"], "v": s["vp"]}


def _plain_rows(q, k, v, causal, out):
    """softmax(q k^T / sqrt(d)) v of one sequence in 32 bits into out: q, out [n, Hq, d], k, v [m, Hk, d]; query i sees
    the keys up to m - n + i (causal) or all of them, and a row that sees none is zero."""
    n, Hq, d = q.shape
    m, Hk = k.shape[0], k.shape[1]
    if n == 0:
        return
    if m == 0:
        out.zero_()
        return
    G = Hq // Hk
    kt, vt = k.float().permute(1, 2, 0), v.float().transpose(0, 1)              # [Hk, d, m], [Hk, m, d]
    step = max(1, (1 << 28) // max(1, Hq * m))
    for i in range(0, n, step):
        j = min(n, i + step)
        see = m - n + j if causal else m                                        # no row of this piece sees further
        if see <= 0:
            out[i:j].zero_()
            continue
        x = q[i:j].float().reshape(j - i, Hk, G, d).permute(1, 2, 0, 3).reshape(Hk, G * (j - i), d)
        w = torch.matmul(x, kt[:, :, :see]).mul_(1.0 / math.sqrt(d)).view(Hk, G, j - i, see)
        if causal:
            last = torch.arange(m - n + i, m - n + j, device="cuda")            # the last key that each row sees
            w.masked_fill_(torch.arange(see, device="cuda")[None, :] > last[:, None], -math.inf)
        top = w.amax(dim=-1, keepdim=True)
        w = w.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
        total = w.sum(dim=-1, keepdim=True)
        y = torch.matmul(w.view(Hk, G * (j - i), see), vt[:, :see]).view(Hk, G, j - i, d) / total.masked_fill(total == 0, 1.0)
        out[i:j] = y.permute(2, 0, 1, 3).reshape(j - i, Hq, d).to(out.dtype)


def _plain_attend(s):
    c = s["c"]
    at = 0
    for b, (n, m) in enumerate(zip(s["new"], s["total"])):
        pages = s["table"][b, :-(-m // c["page"])].long()
        k, v = (p[pages] for p in (s["kp"], s["vp"]))
        if c["layout"] == "bhnd":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        k, v = (x.reshape(-1, c["Hk"], c["d"])[:m] for x in (k, v))
        _plain_rows(s["q"][at:at + n], k, v, c["causal"], s["o"][at:at + n])
        at += n
    return {"o": s["o"]}


def _plain_prompt(s):
    i = j = 0
    for n, m in zip(s["new"], s["total"]):
        _plain_rows(s["q"][i:i + n], s["k"][j:j + m], s["v"][j:j + m], s["c"]["causal"], s["o"][i:i + n])
        i, j = i + n, j + m
    return {"o": s["o"]}


# ------------------------------------------------------------------------------ 64 bits
def exact(c, seed):
    """The outputs of run() from the definition, in 64 bits: for attention one head at a time, weights exp(x - log sum exp x);
    for the rotation a product with complex numbers of length one."""
    global own
    keep, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = keep
    return _exact_append(s) if c["op"] == "append" else _exact_attention(s)


def _exact_attention(s):
    c = s["c"]
    G, d = c["Hq"] // c["Hk"], c["d"]
    out = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    i = j = 0
    for b, (n, m) in enumerate(zip(s["new"], s["total"])):
        for h in range(c["Hk"]):
            if c["op"] == "prompt":
                k, v = s["k"][j:j + m, h], s["v"][j:j + m, h]
            else:
                ids = s["table"][b].long()[torch.arange(m, device="cuda") // c["page"]]
                rows = torch.arange(m, device="cuda") % c["page"]
                k, v = ((p[ids, h, rows] if c["layout"] == "bhnd" else p[ids, rows, h]) for p in (s["kp"], s["vp"]))
            k, v = k.double(), v.double()
            for a in range(h * G, (h + 1) * G):
                for lo in range(0, n, 2048):
                    hi = min(n, lo + 2048)
                    sees = torch.arange(lo, hi, device="cuda") + (m - n + 1) if c["causal"] else torch.full((hi - lo,), m, device="cuda")
                    some = sees > 0
                    if m == 0 or not bool(some.any()):
                        continue
                    x = torch.einsum("id,jd->ij", s["q"][i + lo:i + hi, a].double(), k) / math.sqrt(d)
                    x = torch.where(torch.arange(m, device="cuda")[None, :] < sees[:, None], x, torch.full_like(x, -math.inf))
                    x = torch.exp(x - torch.logsumexp(x, dim=1, keepdim=True))
                    out[i + lo:i + hi, a] = torch.where(some[:, None], torch.einsum("ij,jd->id", x, v), torch.zeros((), dtype=torch.float64, device="cuda"))
        i, j = i + n, j + m
    return {"o": out}


def _exact_append(s):
    c = s["c"]
    rot, half = c["rot"], c["rot"] // 2
    kp, vp = s["kp"].double(), s["vp"].double()
    qr = torch.zeros(s["qr"].shape, dtype=torch.float64, device="cuda")

    def turn(x, at):
        y = x.double().clone()
        z = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None, :]
        lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, half), slice(half, rot))
        p = torch.complex(y[..., lo], y[..., hi]) * z
        y[..., lo], y[..., hi] = p.real, p.imag
        return y

    i = 0
    for b, (n, m) in enumerate(zip(s["new"], s["total"])):
        slots = torch.arange(m - n, m, device="cuda")
        at = s["pos"][i:i + n].long() if c["own_pos"] else slots
        qr[i:i + n] = turn(s["q"][i:i + n], at)
        kr, vr = turn(s["k"][i:i + n], at), s["v"][i:i + n].double()
        ids = s["table"][b].long()[slots // c["page"]]
        for h in range(c["Hk"]):
            if c["layout"] == "bhnd":
                kp[ids, h, slots % c["page"]], vp[ids, h, slots % c["page"]] = kr[:, h], vr[:, h]
            else:
                kp[ids, slots % c["page"], h], vp[ids, slots % c["page"], h] = kr[:, h], vr[:, h]
        i += n
    return {"q": qr, "k": kp, "v": vp}
