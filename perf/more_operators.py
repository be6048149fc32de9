"""Measured cases of a dense layer's cache side: rotation, append, chunks and windows.

Four operators that stand between a layer's projections and its output in a serving
loop: the norm of every head of queries and keys with the position rotation in the same
pass, the same with the keys and values going on into a paged cache (bf16, int8 or
e4m3), the attention of a chunk of any number of new tokens over that cache, and
attention with a sliding window and a few first tokens that stay visible, for single
tokens and short drafts (and, as a choice, for chunks).  ``run`` computes them in plain
torch operations, or, where ``own`` is true, through the library's entry points.
"""
import math
import random

import torch

own = False

BF16, INT8, E4M3 = "bf16", "int8", "e4m3"
QMAX = {INT8: 127.0, E4M3: 448.0}
DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one request's newest token, on its way to a layer that keeps its own cache
        dict(name="rotate_one", op="rotate", n=1, lq=1, len=100001, ragged=0, hq=8, hkv=1, d=128,
             rot=128, halves=True, norm=True),
        # a batch of prompts before their causal attention
        dict(name="rotate_prompt", op="rotate", n=8, lq=4096, len=4096, ragged=3, hq=32, hkv=8,
             d=128, rot=128, halves=True, norm=True),
        # the newest token of every sequence of a decode batch, 8-bit floats in the cache
        dict(name="append_decode", op="append", n=64, lq=1, len=5000, ragged=2, hq=32, hkv=8, d=128,
             rows=64, kind=E4M3, rot=128, halves=True, norm=True),
        # a batch of prompts on its way into the cache
        dict(name="append_prompt", op="append", n=8, lq=8192, len=8192, ragged=9, hq=32, hkv=8,
             d=128, rows=64, kind=BF16, rot=128, halves=True, norm=True),
        # chunks appended in 8-bit integers and read back, half of each head rotated, odd pages
        dict(name="append_back", op="append", n=5, lq=777, len=9000, ragged=6, hq=12, hkv=4, d=64,
             rows=48, kind=INT8, rot=32, halves=False, norm=False),
        # a short question after a cached preamble: latency
        dict(name="chunk_short", op="chunk", n=1, lq=77, mix=1, len=1100, ragged=0, hq=8, hkv=1,
             d=128, rows=64, kind=BF16, window=0, sinks=0),
        # two chunks of prompts in a batch whose other sequences decode one token each
        dict(name="chunk_mixed", op="chunk", n=32, lq=512, mix=2, len=8192, ragged=5, hq=32, hkv=8,
             d=128, rows=64, kind=BF16, window=0, sinks=0),
        # the last quarter of a long document, 8-bit integers in the cache
        dict(name="chunk_long", op="chunk", n=1, lq=8192, mix=1, len=32768, ragged=0, hq=16, hkv=1,
             d=128, rows=64, kind=INT8, window=0, sinks=0),
        # long chunks in a layer that attends locally, small pages, 8-bit floats
        dict(name="chunk_window", op="chunk", n=2, lq=4096, mix=2, len=16000, ragged=4, hq=32, hkv=8,
             d=64, rows=16, kind=E4M3, window=1024, sinks=4),
        # one request's newest token in a local layer, far into its text
        dict(name="window_one", op="window", n=1, q=1, len=100000, ragged=0, hq=8, hkv=1, d=128,
             rows=64, kind=BF16, window=4096, sinks=4),
        # a full decode batch in a local layer
        dict(name="window_batch", op="window", n=128, q=1, len=102400, ragged=7, hq=16, hkv=1, d=128,
             rows=64, kind=INT8, window=4096, sinks=4),
        # a whole step of a local layer while four draft tokens are verified: append, then attend
        dict(name="window_step", op="window", n=24, q=4, len=6000, ragged=8, hq=16, hkv=4, d=64,
             rows=32, kind=E4M3, window=1000, sinks=16, rot=64, halves=True, norm=True),
    ]


def _loguniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = [work(c) for c in listed()]
    while True:
        op = rng.choice(["rotate", "append", "append", "chunk", "chunk", "chunk", "window", "window"])
        hkv, d = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
        c = dict(op=op, hkv=hkv, d=d, ragged=rng.randrange(1000))
        c["hq"] = hkv * rng.choice([1, 2, 3, 4, 7, 8, 16])
        rotation = dict(rot=rng.choice([d, d, d // 2, d // 4]), halves=rng.random() < 0.7,
                        norm=rng.random() < 0.6)
        c["len"] = _loguniform(rng, 1, 110000)
        if op != "rotate":
            c.update(rows=rng.choice([16, 32, 48, 64, 100, 128]), kind=rng.choice([BF16, INT8, E4M3]))
        if op in ("rotate", "append"):
            c.update(n=_loguniform(rng, 1, 128), **rotation)
            c["lq"] = rng.randint(1, min(c["len"], 8)) if rng.random() < 0.4 else _loguniform(rng, 1, c["len"])
            if c["n"] * c["len"] * hkv * d > 1 << 29 or c["n"] * c["lq"] * c["hq"] * d > 1 << 28:
                continue
        else:
            local = op == "window" or rng.random() < 0.4
            c.update(n=_loguniform(rng, 1, 200 if op == "window" else 48),
                     window=_loguniform(rng, 1, 8192) if local else 0,
                     sinks=rng.choice([0, 1, 4, 16, 100]) if local else 0)
            if op == "window":
                c["q"] = rng.choice([1, 1, 1, 2, 4, 5, 8])
                if rng.random() < 0.3:
                    c.update(rotation)
                if c["q"] * c["hq"] // hkv > 128:
                    continue
            else:
                c.update(lq=_loguniform(rng, 1, min(c["len"], 8192)), mix=rng.randint(1, c["n"]))
            square = c["n"] * c["hq"] * c.get("lq", 8) * max(w for _, _, _, w in _spans(c))
            if square > 16 * 8192 * 32768 or c["n"] * c["len"] * hkv * d > 128 * 102400 * 128:
                continue
        w = work(c)
        if w["flops"] <= max(m["flops"] for m in most) and w["bytes"] <= max(m["bytes"] for m in most):
            return c


def _lens(case):
    """Per sequence: (new tokens, length with them), from the case alone."""
    n, top, rng = case["n"], case["len"], random.Random(case["ragged"])
    new, got = case["q"] if case["op"] == "window" else case["lq"], []
    for i in range(n):
        t = top if i == 0 or not case["ragged"] else rng.randint((top + 1) // 2, top)
        a = new
        if case["op"] != "window":
            if case["ragged"] and 1 < new < t and i:
                a = rng.randint(1, new)
            elif new == top:
                a = t  # a whole prompt
            if i >= case.get("mix", n):
                a = 0 if i % 7 == 3 else 1
        got.append((min(a, t) if case["op"] != "window" else a, max(t, a) if "rot" in case else t))
    return got


def _spans(case):
    """Per sequence: new tokens, length, first position after the sinks that any of them
    sees, and how many positions any of them sees."""
    got = []
    for a, t in _lens(case):
        w, s = case["window"], case["sinks"]
        lo = max(0, t - a - w + 1) if w else 0
        got.append((a, t, lo, min(s, lo) + t - lo if a else 0))
    return got


def _visible(case):
    """Pairs of a new token and a position that it sees."""
    w, s = case["window"], case["sinks"]

    def upto(x):  # the sum of those of positions 0 .. x - 1
        if not w or x <= w:
            return x * (x + 1) // 2
        y = x - w
        return w * (w + 1) // 2 + y * w + (y * (y + 1) // 2 if y <= s else s * (s + 1) // 2 + (y - s) * s)

    return sum(upto(t) - upto(max(0, t - a)) for a, t in _lens(case))


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    new = sum(a for a, _ in _lens(case))
    w = 2 if case.get("kind", BF16) == BF16 else 1
    row = 2 * hkv * (d * w + (0 if w == 2 else 4))  # a position's keys and values in the cache
    if case["op"] == "rotate":
        return {"bytes": new * (hq + hkv) * d * 4, "flops": new * (hq + hkv) * d * 8}
    if case["op"] == "append":
        back = 4 * hkv * d if case["kind"] == INT8 else 0
        return {"bytes": new * (4 * hq * d + 4 * hkv * d + row + back),
                "flops": new * (hq + 2 * hkv) * d * 8}
    cached = sum(x for _, _, _, x in _spans(case))
    got = {"bytes": cached * row + new * hq * (4 * d + 4), "flops": 4 * d * hq * _visible(case)}
    if "rot" in case:  # the queries come and go once more, the new rows come
        got["bytes"] += new * (4 * hq * d + 4 * hkv * d + row)
    return got


# ----------------------------------------------------------------- the inputs
def _normal(g, shape, outliers=False):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if outliers:  # a few channels of a key head are several times larger than the rest
        x *= 1.0 + 5.0 * (torch.rand(shape[-2:], generator=g, device=DEV) < 0.03)
    return x.to(torch.bfloat16)


def _cu(sizes):
    return torch.tensor([0] + sizes, device=DEV).cumsum(0).to(torch.int32)


def _pool(case, g, lens):
    """A cache with every page of every sequence in use, in a random order."""
    rows, kind, hkv, d = case["rows"], case["kind"], case["hkv"], case["d"]
    pages = [-(-t // rows) for _, t in lens]
    width, n_pages = max(1, max(pages)), max(1, sum(pages) + 3)
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    first, slot = _cu(pages)[:-1].long(), torch.arange(width, device=DEV)
    used = slot[None] < torch.tensor(pages, device=DEV)[:, None]
    st = dict(table=torch.where(used, order[(first[:, None] + slot).clamp(max=n_pages - 1)],
                                torch.full_like(order[:1], -1)).contiguous(),
              lens=torch.tensor([t for _, t in lens], dtype=torch.int32, device=DEV))
    shape = (n_pages, hkv, rows, d)
    if kind == BF16:
        kc, vc = (torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
                  for _ in range(2))
        ks = vs = None
    else:
        kc, vc = (torch.empty(shape, dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
                  for _ in range(2))
        ks, vs = (torch.rand(shape[:3], generator=g, device=DEV) * 0.02 + 0.01 for _ in range(2))
        if kind == E4M3:  # finite codes only
            kc, vc = (x.bitwise_and(-2).view(torch.float8_e4m3fn) for x in (kc, vc))
            ks, vs = ks * 0.1, vs * 0.1
    st.update(kc=kc, vc=vc, ks=ks, vs=vs)
    return st


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)
    lens, hq, hkv, d, op = _lens(case), case["hq"], case["hkv"], case["d"], case["op"]
    new = sum(a for a, _ in lens)
    st = dict(case=case, new_max=max(a for a, _ in lens))
    if "rot" in case:  # raw projections, the rotation and the norms' weights
        base = 10000.0 if case["halves"] else 500000.0
        pair = torch.arange(case["rot"] // 2, dtype=torch.float64)
        st["freqs"] = (base ** (-pair * 2 / case["rot"])).to(DEV)
        st["wq"], st["wk"] = ((1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
                               if case["norm"] else None) for _ in range(2))
        st.update(q=_normal(g, (new, hq, d)), k=_normal(g, (new, hkv, d), True),
                  q_out=torch.empty((new, hq, d), dtype=torch.bfloat16, device=DEV))
        if own:
            import hierarchical_sparse_kv_int8_gb300 as dhs
            st.update(dhs=dhs, rotation=dhs.Rotation(
                st["freqs"], dhs.ROTATE_HALVES if case["halves"] else dhs.ROTATE_NEIGHBOURS))
    if op == "rotate":
        st["k_out"] = torch.empty((new, hkv, d), dtype=torch.bfloat16, device=DEV)
        st["positions"] = torch.cat([torch.arange(t - a, t, device=DEV) for a, t in lens]).to(torch.int32)
        return st
    st.update(_pool(case, g, lens), cu=_cu([a for a, _ in lens]))
    if own:
        import hierarchical_sparse_kv_int8_gb300 as dhs
        st["cache"] = dhs.PageCache(st["kc"], st["vc"], st["ks"], st["vs"])
    if "rot" in case:
        st["v"] = _normal(g, (new, hkv, d))
    if op == "append":
        if case["kind"] == INT8:
            st.update(k_back=torch.empty_like(st["k"]), v_back=torch.empty_like(st["v"]))
        return st
    shape = (case["n"], case["q"], hq, d) if op == "window" else (new, hq, d)
    st["width"] = max(1, max(x for _, _, _, x in _spans(case)))
    st.update(out=torch.empty(shape, dtype=torch.bfloat16, device=DEV),
              lse=torch.empty(shape[:-1], dtype=torch.float32, device=DEV))
    if "rot" not in case:
        st["q"] = _normal(g, shape)
    if own:
        st["workspace"] = (st["cache"].attend_workspace(case["n"], case["q"], hq) if op == "window"
                           else st["cache"].chunk_workspace(new, case["n"], hq))
    return st


# ------------------------------------------------------- the library's entry points
def _run_own(st):
    case, op = st["case"], st["case"]["op"]
    if op == "rotate":
        st["dhs"].rotate(st["q"], st["k"], st["positions"], st["rotation"], st["q_out"], st["k_out"],
                         q_norm=st["wq"], k_norm=st["wk"], eps=EPS)
        return {"q": st["q_out"], "k": st["k_out"]}
    cache, got = st["cache"], {}
    if "rot" in case:
        cache.append(st["q"], st["k"], st["v"], st["cu"], st["lens"], st["table"], st["q_out"],
                     st["rotation"], q_norm=st["wq"], k_norm=st["wk"], eps=EPS)
        if op == "append" and case["kind"] == INT8:
            cache.read(st["k_back"], st["v_back"], st["cu"], st["lens"], st["table"])
            return {"q": st["q_out"], "k": st["k_back"], "v": st["v_back"]}
        got = _appended(st)
    if op == "window":
        q = st["q_out"].view(st["out"].shape) if "rot" in case else st["q"]
        cache.attend(q, st["lens"], st["table"], st["out"], st["workspace"], lse=st["lse"],
                     window=case["window"], sinks=case["sinks"])
    elif op == "chunk":
        cache.attend_chunk(st["q"], st["cu"], st["lens"], st["table"], st["out"], st["workspace"],
                           lse=st["lse"], window=case["window"], sinks=case["sinks"])
    if op != "append":
        got.update(out=st["out"], lse=st["lse"])
    return got


def _appended(st):
    """The queries and, of a cache whose numbers are floats, the cache."""
    got = {"q": st["q_out"]}
    if st["case"]["kind"] != INT8:
        got.update(k=st["kc"], v=st["vc"])
    if st["ks"] is not None:
        got.update(k_scale=st["ks"], v_scale=st["vs"])
    return got


# --------------------------------------------------------------- the plain forms
def _rotated(x, weight, cos, sin, halves):
    """Heads x [tokens, heads, d] after their norm and rotation, in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    pairs = cos.shape[-1]
    turned, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
    cos, sin = cos[:, None], sin[:, None]
    if halves:
        a, b = turned[..., :pairs], turned[..., pairs:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = turned[..., 0::2], turned[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _plain_rotation(st, pos):
    angle = pos.double()[:, None] * st["freqs"]  # (far positions: the angle in 64 bits)
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    halves = st["case"]["halves"]
    st["q_out"].copy_(_rotated(st["q"], st["wq"], cos, sin, halves))
    return _rotated(st["k"], st["wk"], cos, sin, halves)


def _plain_rotate(st):
    st["k_out"].copy_(_plain_rotation(st, st["positions"]))
    return {"q": st["q_out"], "k": st["k_out"]}


def _quantise(x, kind):
    """Codes (as values) and scales of rows x [..., d]; the division and what it is next
    to in 64 bits."""
    big = x.abs().amax(-1)
    scale = big / torch.full_like(big, QMAX[kind])
    y = x.double() / torch.where(scale > 0, scale, 1.0).double()[..., None]
    if kind == INT8:
        return y.round().clamp(-127, 127), scale
    step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
    return ((y / step).round() * step).clamp(-448, 448), scale


def _token_places(st):
    """Position, page and row of every packed token."""
    cu, lens, rows = st["cu"].long(), st["lens"].long(), st["case"]["rows"]
    tok = torch.arange(st["q"].shape[0], device=DEV)
    i = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    pos = lens[i] - cu[i + 1] + tok
    return pos, st["table"][i, pos // rows].long(), pos % rows


def _store(st, x, codes, scales, page, row):
    """Rows x in 32 bits into the cache; what they stand for there, in 32 bits."""
    kind = st["case"]["kind"]
    if kind == BF16:
        codes[page, :, row] = x.to(torch.bfloat16)
        return None
    c, s = _quantise(x, kind)
    if kind == INT8:
        codes[page, :, row] = c.to(torch.int8)
    else:
        codes.view(torch.uint8)[page, :, row] = c.float().to(torch.float8_e4m3fn).view(torch.uint8)
    scales[page, :, row] = s
    return c.float() * s[..., None]


def _plain_append(st):
    pos, page, row = _token_places(st)
    k = _store(st, _plain_rotation(st, pos), st["kc"], st["ks"], page, row)
    v = _store(st, st["v"].float(), st["vc"], st["vs"], page, row)
    if st["case"]["op"] == "append" and st["case"]["kind"] == INT8:
        return {"q": st["q_out"], "k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}
    return _appended(st)


def _rows_of(codes, scales, page, row):
    """Rows [..., hkv, d] of the cache in 32 bits (8-bit floats are indexed as bytes)."""
    e4m3 = codes.dtype == torch.float8_e4m3fn
    x = codes.view(torch.uint8)[page, :, row].view(codes.dtype) if e4m3 else codes[page, :, row]
    return x.float() if scales is None else x.float() * scales[page, :, row][..., None]


def _plain_attend(st, q, new):
    """q [n, lq, hq, d], of which new [n] tokens of each sequence are there: over the
    positions that any of a sequence's tokens sees (see _spans)."""
    case, lens = st["case"], st["lens"].long()
    n, lq, hq, d = q.shape
    hkv, w, s, rows = case["hkv"], case["window"], case["sinks"], case["rows"]
    first = lens - new                                    # of the new tokens
    lo = (first - w + 1).clamp(min=0) if w else torch.zeros_like(lens)
    kept = lo.clamp(max=s)
    x = torch.arange(st["width"], device=DEV)[None]
    pos = torch.where(x < kept[:, None], x, x + (lo - kept)[:, None])     # n t
    there = pos < lens[:, None]
    page = st["table"].gather(1, (pos // rows).clamp(max=st["table"].shape[1] - 1)).clamp(min=0).long()
    keep = there[..., None, None]
    k = torch.where(keep, _rows_of(st["kc"], st["ks"], page, pos % rows), 0.0).permute(0, 2, 3, 1)
    v = torch.where(keep, _rows_of(st["vc"], st["vs"], page, pos % rows), 0.0).permute(0, 2, 1, 3)
    qp = q.float().view(n, lq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)  # n hkv grp lq d
    u = torch.arange(lq, device=DEV)
    at = (first[:, None] + u)[..., None]                                  # n lq 1
    seen = there[:, None] & (pos[:, None] <= at)
    if w:
        seen &= (pos[:, None] > at - w) | (pos[:, None] < s)
    z = torch.matmul(qp.reshape(n, hkv, -1, d), k).view(n, hkv, -1, lq, st["width"])
    z = torch.where(seen[:, None, None], z * (1.0 / math.sqrt(d)), -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v[:, :, None]) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + m).squeeze(-1)
    return out.permute(0, 3, 1, 2, 4).reshape(n, lq, hq, d).to(torch.bfloat16), \
        lse.permute(0, 3, 1, 2).reshape(n, lq, hq)


def _plain_window(st):
    got = _plain_append(st) if "rot" in st["case"] else {}
    q = st["q_out"].view(st["out"].shape) if "rot" in st["case"] else st["q"]
    out, lse = _plain_attend(st, q, torch.full_like(st["lens"], q.shape[1]).long())
    got.update(out=out, lse=lse)
    return got


def _plain_chunk(st):
    cu = st["cu"].long()
    new, u = cu[1:] - cu[:-1], torch.arange(st["new_max"], device=DEV)
    at = (cu[:-1, None] + u).clamp(max=st["q"].shape[0] - 1)
    out, lse = _plain_attend(st, st["q"][at], new)
    keep = u < new[:, None]
    return {"out": out[keep], "lse": lse[keep]}


def run(state):
    if own:
        return _run_own(state)
    return {"rotate": _plain_rotate, "append": _plain_append, "chunk": _plain_chunk,
            "window": _plain_window}[state["case"]["op"]](state)


# ------------------------------------------------------------------- in 64 bits
def _exact_heads(st, x, weight, pos):
    y, case = x.double(), st["case"]
    if weight is not None:
        y = weight.double() * y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + EPS)
    n = case["rot"] // 2
    first = torch.arange(n, device=DEV) * (1 if case["halves"] else 2)
    second = first + (n if case["halves"] else 1)
    turn = torch.exp(1j * torch.outer(pos.double(), st["freqs"]))[:, None]  # complex rotation
    z = torch.complex(y[..., first], y[..., second]) * turn
    got = y.clone()
    got[..., first], got[..., second] = z.real, z.imag
    return got


def _e4m3_grid():
    """All finite non-negative e4m3 values, ascending; entry c is code c's value."""
    return torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                         for c in range(127)], dtype=torch.float64, device=DEV)


def _exact_codes(x, kind):
    top = x.abs().max(-1).values
    scale = (top / QMAX[kind]).float()   # a scale is a 32-bit number
    y = x / torch.where(scale > 0, scale, 1.0).double()[..., None]
    if kind == INT8:
        low = y.floor()
        up = (y - low > 0.5) | ((y - low == 0.5) & (low.remainder(2) == 1))
        return (low + up).clamp(-127, 127), scale
    grid, mag = _e4m3_grid(), y.abs()
    hi = torch.searchsorted(grid, mag).clamp(1, 126)
    over, under = grid[hi] - mag, mag - grid[hi - 1]
    take_hi = (over < under) | ((over == under) & (hi % 2 == 0))
    return torch.where(take_hi, grid[hi], grid[hi - 1]) * torch.sign(y), scale


def _exact_append(st, lens, got):
    """Fills `got`; the cache itself takes the exact rows, rounded to what it holds."""
    case, rows = st["case"], st["case"]["rows"]
    pos = torch.cat([torch.arange(t - a, t, device=DEV) for a, t in lens])
    seq = torch.cat([torch.full((a,), i, device=DEV) for i, (a, t) in enumerate(lens)])
    page, row = st["table"][seq, pos // rows].long(), pos % rows
    got["q"] = _exact_heads(st, st["q"], st["wq"], pos)
    back = case["op"] == "append" and case["kind"] == INT8
    for name, x in (("k", _exact_heads(st, st["k"], st["wk"], pos)), ("v", st["v"].double())):
        codes, scales = st[name + "c"], st[name + "s"]
        if case["kind"] == BF16:
            got[name] = codes.double()
            got[name][page, :, row] = x
            continue
        c, s = _exact_codes(x, case["kind"])
        scales[page, :, row] = s
        if back:
            got[name] = c * s.double()[..., None]
            continue
        got[name + "_scale"] = scales.clone()
        if case["kind"] == INT8:
            codes[page, :, row] = c.to(torch.int8)
        else:
            raw = codes.view(torch.uint8)
            raw[page, :, row] = c.float().to(torch.float8_e4m3fn).view(torch.uint8)
            got[name] = raw.view(torch.float8_e4m3fn).double()


def _exact_one(st, i, t, q, pos):
    """q [a, hq, d] of sequence i at positions pos, over its t cached rows."""
    case, (a, hq, d) = st["case"], q.shape
    hkv, w, s = case["hkv"], case["window"], case["sinks"]
    out, lse = torch.zeros_like(q), torch.full((a, hq), -math.inf, dtype=torch.float64, device=DEV)
    if not a or not t:
        return out, lse
    key = torch.arange(t, device=DEV)
    if w:  # positions that no query sees are left out
        key = key[(key < s) | (key > int(pos.min()) - w)]
    page, row = st["table"][i].long()[key // case["rows"]], key % case["rows"]
    kv = []
    for codes, scales in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
        e4m3 = codes.dtype == torch.float8_e4m3fn
        x = (codes.view(torch.uint8)[page, :, row].view(codes.dtype) if e4m3 else codes[page, :, row]).double()
        kv.append(x if scales is None else x * scales[page, :, row].double()[..., None])
    hidden = key[None] > pos[:, None]
    if w:
        hidden |= (key[None] <= pos[:, None] - w) & (key[None] >= s)
    for h in range(hq):
        g = h // (hq // hkv)
        z = (q[:, h] @ kv[0][:, g].T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
        lse[:, h] = torch.logsumexp(z, -1)
        some = (lse[:, h] > -math.inf)[:, None]
        out[:, h] = torch.where(some, torch.nan_to_num(torch.softmax(z, -1)) @ kv[1][:, g], 0.0)
    return out, lse


def exact(case, seed):
    st, lens, got = prepare(case, seed), _lens(case), {}
    if case["op"] == "rotate":
        return {x: _exact_heads(st, st[x], st["w" + x], st["positions"]) for x in ("q", "k")}
    q = st["q"]
    if "rot" in case:
        _exact_append(st, lens, got)
        if case["op"] == "append":
            return got
        # (queries and, in a bf16 cache, keys are rounded before they are attended with)
        q = got["q"].to(torch.bfloat16)
        if case["kind"] == BF16:
            st["kc"], st["vc"] = got["k"].to(torch.bfloat16), got["v"].to(torch.bfloat16)
    q = q.reshape(-1, case["hq"], case["d"]).double()
    parts, at = [], 0
    for i, (a, t) in enumerate(lens):
        parts.append(_exact_one(st, i, t, q[at:at + a], torch.arange(t - a, t, device=DEV)))
        at += a
    shape = st["out"].shape
    got.update(out=torch.cat([o for o, _ in parts]).view(shape),
               lse=torch.cat([x for _, x in parts]).view(shape[:-1]))
    return got
