"""Measured cases of the paged-cache and prompt operators.

Four operators, used one after another by a serving loop: the causal attention
of packed prompts, the write of their keys and values into a paged cache (bf16,
or quantised to int8 or e4m3 with one scale per token and head), the read of
cached rows back (the earlier part of a prompt that comes in chunks), and the
attention of the newest one to eight tokens of every sequence over the pages.
``run`` computes them in plain torch operations, or, where ``own`` is true,
through the library's entry points.
"""
import math
import random

import torch

own = False

BF16, INT8, E4M3 = "bf16", "int8", "e4m3"
QMAX = {INT8: 127.0, E4M3: 448.0}
TINY = 2.0 ** -100  # rows whose largest magnitude is smaller are stored as zeros
DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the first turn of a chat: one short prompt, a single-head-group layer
        dict(name="prompt_short", op="prompt", n=1, lq=77, lk=77, ragged=0, hq=8, hkv=1, d=128),
        # a prefill batch of unequal prompts packed without padding
        dict(name="prompt_packed", op="prompt", n=16, lq=2048, lk=2048, ragged=11, hq=32, hkv=8,
             d=128),
        # one long document
        dict(name="prompt_long", op="prompt", n=1, lq=16384, lk=16384, ragged=0, hq=16, hkv=1,
             d=128),
        # a chunk of a long prompt against everything before it
        dict(name="prompt_chunk", op="prompt", n=2, lq=500, lk=32768, ragged=0, hq=8, hkv=2, d=64),
        # one request, one token: the latency of a decode step
        dict(name="decode_one", op="attend", n=1, q=1, len=4096, ragged=0, hq=8, hkv=1, d=128,
             rows=64, kind=BF16),
        # verification of four draft tokens for a batch of eight
        dict(name="verify_4", op="attend", n=8, q=4, len=32768, ragged=5, hq=8, hkv=1, d=128,
             rows=64, kind=BF16),
        # a full decode batch at 100K context, int8 cache
        dict(name="decode_100k", op="attend", n=128, q=1, len=102400, ragged=7, hq=16, hkv=1,
             d=128, rows=64, kind=INT8),
        # many sequences with several kv heads, e4m3 cache, small pages
        dict(name="decode_heads", op="attend", n=61, q=1, len=8000, ragged=3, hq=32, hkv=8, d=64,
             rows=16, kind=E4M3),
        # the newest token of each sequence of a decode batch, on its way into the cache
        dict(name="write_decode", op="write", n=64, lq=1, len=5000, ragged=2, hkv=8, d=128, rows=64,
             kind=INT8),
        # a prefill batch on its way into the cache
        dict(name="write_prompt", op="write", n=8, lq=8192, len=8192, ragged=9, hkv=8, d=128,
             rows=64, kind=E4M3),
        # a short cached prefix, read back for the next chunk
        dict(name="read_short", op="read", n=3, lq=333, len=333, ragged=4, hkv=2, d=64, rows=48,
             kind=E4M3),
        # a long cached prefix
        dict(name="read_long", op="read", n=2, lq=65536, len=65536, ragged=0, hkv=8, d=128, rows=64,
             kind=INT8),
    ]


def _loguniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["prompt", "prompt", "attend", "attend", "attend", "write", "read"])
        hkv = rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([64, 128])
        kind = rng.choice([BF16, INT8, E4M3])
        rows = rng.choice([16, 32, 48, 64, 100, 128])
        c = dict(op=op, hkv=hkv, d=d, ragged=rng.randrange(1000))
        if op == "prompt":
            lk = _loguniform(rng, 1, 32768)
            lq = lk if rng.random() < 0.6 else _loguniform(rng, 1, min(lk, 2048))
            c.update(n=_loguniform(rng, 1, 32), lq=lq, lk=lk, hq=hkv * rng.choice([1, 2, 3, 4, 7, 8, 16]))
            square = c["n"] * c["hq"] * lq * lk
            if square > 16 * 16384 ** 2 or c["n"] * lk * hkv * d > 1 << 30:
                continue
        elif op == "attend":
            c.update(n=_loguniform(rng, 1, 200), len=_loguniform(rng, 1, 110000), rows=rows, kind=kind,
                     q=rng.choice([1, 1, 1, 2, 4, 5, 8]),
                     hq=hkv * rng.choice([1, 2, 3, 4, 7, 8, 16]))
            if c["q"] * c["hq"] // hkv > 128 or c["n"] * c["len"] * hkv * d > 128 * 102400 * 128:
                continue
        else:
            length = _loguniform(rng, 1, 70000)
            lq = length if op == "read" or rng.random() < 0.6 else rng.randint(1, min(length, 8))
            c.update(n=_loguniform(rng, 1, 128), lq=lq, len=length, rows=rows, kind=kind)
            if c["n"] * length * hkv * d > 1 << 27:
                continue
        if work(c)["flops"] <= work(listed()[2])["flops"] and work(c)["bytes"] <= work(listed()[6])["bytes"]:
            return c


def _lens(case):
    """Per sequence: (new or query tokens, cached or key tokens), from the case alone."""
    n, seed = case["n"], case["ragged"]
    rng = random.Random(seed)
    top = case["lk"] if case["op"] == "prompt" else case["len"]
    new = case["q"] if case["op"] == "attend" else case["lq"]
    if not seed:
        return [(new, top)] * n
    got = []
    for i in range(n):
        t = top if i == 0 else rng.randint((top + 1) // 2 if case["op"] == "attend" else 1, top)
        if case["op"] == "attend":
            got.append((new, 0 if i == 2 else t))  # one idle slot
        elif new == top:
            got.append((t, t))
        else:
            got.append((min(new, t), t))
    return got


def _visible(lens):
    return sum(sum(max(0, t - a + u + 1) for u in range(a)) if a <= 8 else
               a * t - a * (a - 1) // 2 for a, t in lens)


def work(case):
    lens, hkv, d = _lens(case), case["hkv"], case["d"]
    a, t = sum(x for x, _ in lens), sum(y for _, y in lens)
    w = 2 if case.get("kind", BF16) == BF16 else 1
    s = 0 if w == 2 else 4
    if case["op"] == "prompt":
        return {"bytes": 2 * d * (2 * a * case["hq"] + 2 * t * hkv) + 4 * a * case["hq"],
                "flops": 4 * d * case["hq"] * _visible(lens)}
    if case["op"] == "attend":
        return {"bytes": t * hkv * 2 * (d * w + s) + 4 * a * case["hq"] * d + 4 * a * case["hq"],
                "flops": 4 * d * case["hq"] * _visible(lens)}
    return {"bytes": a * hkv * 2 * (d * (2 + w) + s), "flops": 0}


# ----------------------------------------------------------------- the inputs
def _normal(g, shape, outliers=False):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if outliers:  # a few channels of a key head are several times larger than the rest
        x *= 1.0 + 5.0 * (torch.rand(shape[-2:], generator=g, device=DEV) < 0.03)
    return x.to(torch.bfloat16)


def _cu(sizes):
    return torch.tensor([0] + sizes, device=DEV).cumsum(0).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 13)
    lens, hkv, d = _lens(case), case["hkv"], case["d"]
    a, t = [x for x, _ in lens], [y for _, y in lens]
    st = dict(case=case, lq_max=max(a), lk_max=max(t))
    if case["op"] == "prompt":
        hq = case["hq"]
        st.update(q=_normal(g, (sum(a), hq, d)), k=_normal(g, (sum(t), hkv, d), True),
                  v=_normal(g, (sum(t), hkv, d)), cu_q=_cu(a), cu_k=_cu(t),
                  out=torch.empty((sum(a), hq, d), dtype=torch.bfloat16, device=DEV),
                  lse=torch.empty((sum(a), hq), dtype=torch.float32, device=DEV))
        if own:
            import hierarchical_sparse_kv_int8_gb300 as dhs
            st.update(dhs=dhs, workspace=dhs.prompt_workspace(st["q"], st["k"], len(lens)))
        return st
    rows, kind = case["rows"], case["kind"]
    pages = [-(-y // rows) for y in t]
    width = max(1, max(pages))
    n_pages = max(1, sum(pages) + 3)
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    first = _cu(pages)[:-1].long()
    slot = torch.arange(width, device=DEV)
    used = slot[None] < torch.tensor(pages, device=DEV)[:, None]
    st["table"] = torch.where(used, order[(first[:, None] + slot).clamp(max=n_pages - 1)],
                              torch.full_like(order[:1], -1)).contiguous()
    st["lens"] = torch.tensor(t, dtype=torch.int32, device=DEV)
    shape = (n_pages, hkv, rows, d)
    if kind == BF16:
        kc, vc = (torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(2))
        ks = vs = None
    else:
        kc, vc = (torch.empty(shape, dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
                  for _ in range(2))
        ks, vs = (torch.rand(shape[:3], generator=g, device=DEV) * 0.02 + 0.01 for _ in range(2))
        if kind == E4M3:  # finite codes only
            kc, vc = ((x.bitwise_and(-2)).view(torch.float8_e4m3fn) for x in (kc, vc))
            ks, vs = ks * 0.1, vs * 0.1
    st.update(kc=kc, vc=vc, ks=ks, vs=vs)
    if case["op"] == "attend":
        n, qn, hq = case["n"], case["q"], case["hq"]
        st.update(q=_normal(g, (n, qn, hq, d)),
                  out=torch.empty((n, qn, hq, d), dtype=torch.bfloat16, device=DEV),
                  lse=torch.empty((n, qn, hq), dtype=torch.float32, device=DEV))
    else:
        st["cu"] = _cu(a)
        if case["op"] == "write":
            st.update(k=_normal(g, (sum(a), hkv, d), True), v=_normal(g, (sum(a), hkv, d)))
        else:
            st.update(k=torch.empty((sum(a), hkv, d), dtype=torch.bfloat16, device=DEV),
                      v=torch.empty((sum(a), hkv, d), dtype=torch.bfloat16, device=DEV))
    if own:
        import hierarchical_sparse_kv_int8_gb300 as dhs
        st["cache"] = dhs.PageCache(kc, vc, ks, vs)
        if case["op"] == "attend":
            st["workspace"] = st["cache"].attend_workspace(case["n"], case["q"], case["hq"])
    return st


# ------------------------------------------------------- the library's entry points
def _run_own(st):
    op = st["case"]["op"]
    if op == "prompt":
        st["dhs"].prompt_attend(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], st["out"],
                                lse=st["lse"], workspace=st["workspace"])
        return {"out": st["out"], "lse": st["lse"]}
    cache = st["cache"]
    if op == "attend":
        cache.attend(st["q"], st["lens"], st["table"], st["out"], st["workspace"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "write":
        cache.write(st["k"], st["v"], st["cu"], st["lens"], st["table"])
        return _cache_of(st)
    cache.read(st["k"], st["v"], st["cu"], st["lens"], st["table"])
    return {"k": st["k"], "v": st["v"]}


def _cache_of(st):
    got = {"k": st["kc"], "v": st["vc"]}
    if st["ks"] is not None:
        got.update(k_scale=st["ks"], v_scale=st["vs"])
    return got


# --------------------------------------------------------------- the plain forms
def _softmax_av(s, seen, v, scale):
    """softmax over the seen places of s [..., q, t] times v [..., t, d], and the log-sum-exp."""
    s = torch.where(seen, s * scale, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(z > 0, z, 1.0)
    return out, (torch.log(z) + m).squeeze(-1)


def _plain_prompt(st):
    q, k, v, cu_q, cu_k = (st[x] for x in ("q", "k", "v", "cu_q", "cu_k"))
    lq, lk = st["lq_max"], st["lk_max"]
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    n, grp = cu_q.numel() - 1, hq // hkv
    nq, nk = (cu_q[1:] - cu_q[:-1])[:, None], (cu_k[1:] - cu_k[:-1])[:, None]
    iq, ik = torch.arange(lq, device=DEV)[None], torch.arange(lk, device=DEV)[None]
    at_q = (cu_q[:-1, None] + iq).clamp(max=q.shape[0] - 1).long()
    at_k = (cu_k[:-1, None] + ik).clamp(max=k.shape[0] - 1).long()
    qp = q[at_q].float().view(n, lq, hkv, grp, d).permute(0, 2, 3, 1, 4)     # n hkv grp lq d
    kp = torch.where((ik < nk)[..., None, None], k[at_k].float(), 0.0).permute(0, 2, 3, 1)
    vp = torch.where((ik < nk)[..., None, None], v[at_k].float(), 0.0).permute(0, 2, 1, 3)
    seen = (ik[:, None] < nk[..., None]) & (ik[:, None] <= (nk - nq)[..., None] + iq[..., None])
    s = torch.matmul(qp.reshape(n, hkv, grp * lq, d), kp).view(n, hkv, grp, lq, lk)
    out, lse = _softmax_av(s, seen[:, None, None], vp[:, :, None], 1.0 / math.sqrt(d))
    keep = (iq < nq).reshape(-1)
    out = out.permute(0, 3, 1, 2, 4).reshape(n * lq, hq, d)[keep]
    lse = lse.permute(0, 3, 1, 2).reshape(n * lq, hq)[keep]
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _places(st, width):
    """Page and row of positions 0 .. width - 1 of every sequence."""
    rows = st["case"]["rows"]
    pos = torch.arange(width, device=DEV)
    page = st["table"][:, (pos // rows).clamp(max=st["table"].shape[1] - 1)].clamp(min=0).long()
    return page, (pos % rows).expand_as(page)


def _rows_of(codes, scales, page, row):
    """Rows [..., hkv, d] of the cache in 32 bits (8-bit floats are indexed as bytes)."""
    e4m3 = codes.dtype == torch.float8_e4m3fn
    x = codes.view(torch.uint8)[page, :, row].view(codes.dtype) if e4m3 else codes[page, :, row]
    return x.float() if scales is None else x.float() * scales[page, :, row][..., None]


def _plain_attend(st):
    q, lens = st["q"], st["lens"].long()
    n, qn, hq, d = q.shape
    hkv = st["case"]["hkv"]
    grp, width = hq // hkv, max(1, st["lk_max"])
    page, row = _places(st, width)
    pos = torch.arange(width, device=DEV)
    there = (pos[None] < lens[:, None])[..., None, None]
    k = torch.where(there, _rows_of(st["kc"], st["ks"], page, row), 0.0).permute(0, 2, 3, 1)
    v = torch.where(there, _rows_of(st["vc"], st["vs"], page, row), 0.0).permute(0, 2, 1, 3)
    qp = q.float().view(n, qn, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, qn * grp, d)
    s = torch.matmul(qp, k).view(n, hkv, qn, grp, width)
    last = lens[:, None] - qn + torch.arange(qn, device=DEV)[None]
    seen = pos[None, None] <= last[..., None]                                  # n qn t
    out, lse = _softmax_av(s, seen[:, None, :, None], v[:, :, None], 1.0 / math.sqrt(d))
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(n, qn, hq, d).to(torch.bfloat16),
            "lse": lse.permute(0, 2, 1, 3).reshape(n, qn, hq)}


def _token_places(st):
    """Page and row of every packed token."""
    cu, lens, rows = st["cu"].long(), st["lens"].long(), st["case"]["rows"]
    tok = torch.arange(st["k"].shape[0], device=DEV)
    i = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    pos = lens[i] - cu[i + 1] + tok
    return st["table"][i, pos // rows].long(), pos % rows


def _quantise(x, kind):
    """Codes (as float32 values) and scales of rows x [..., d], the division in 64 bits."""
    x = x.float()
    big = x.abs().amax(-1)
    scale = big / torch.full_like(big, QMAX[kind])  # (a division: by a number it would be a product)
    scale = torch.where(big < TINY, 0.0, scale)
    scale = torch.where(torch.isfinite(big), scale, math.nan)
    y = x.double() / torch.where(scale > 0, scale, 1.0).double()[..., None]
    y = torch.where((scale > 0)[..., None], y, 0.0)
    if kind == INT8:
        return y.round().clamp(-127, 127), scale
    step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
    return ((y / step).round() * step).clamp(-448, 448), scale


def _plain_write(st):
    page, row = _token_places(st)
    for new, codes, scales in (("k", "kc", "ks"), ("v", "vc", "vs")):
        if st[scales] is None:
            st[codes][page, :, row] = st[new]
        else:
            c, s = _quantise(st[new], st["case"]["kind"])
            if st["case"]["kind"] == E4M3:
                st[codes].view(torch.uint8)[page, :, row] = c.float().to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                st[codes][page, :, row] = c.to(torch.int8)
            st[scales][page, :, row] = s
    return _cache_of(st)


def _plain_read(st):
    page, row = _token_places(st)
    return {"k": _rows_of(st["kc"], st["ks"], page, row).to(torch.bfloat16),
            "v": _rows_of(st["vc"], st["vs"], page, row).to(torch.bfloat16)}


def run(state):
    if own:
        return _run_own(state)
    return {"prompt": _plain_prompt, "attend": _plain_attend, "write": _plain_write,
            "read": _plain_read}[state["case"]["op"]](state)


# ------------------------------------------------------------------- in 64 bits
def _e4m3_grid():
    """All finite non-negative e4m3 values, ascending; entry c is code c's value."""
    return torch.tensor([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                         for c in range(127)], dtype=torch.float64, device=DEV)


def _exact_codes(x, kind):
    x = x.double()
    top = x.abs().max(-1).values
    scale = torch.div(top, torch.full_like(top, QMAX[kind])).float()   # a scale is a 32-bit number
    safe = torch.where(top >= TINY, scale.double(), torch.ones_like(top))[..., None]
    y = torch.where((top >= TINY)[..., None], x, torch.zeros_like(x)) / safe
    scale = torch.where(top >= TINY, scale, torch.zeros_like(scale))
    if kind == INT8:
        low = y.floor()
        up = (y - low > 0.5) | ((y - low == 0.5) & (low.remainder(2) == 1))
        return (low + up).clamp(-127, 127), scale
    grid, mag = _e4m3_grid(), y.abs()
    hi = torch.searchsorted(grid, mag).clamp(1, 126)
    lo = hi - 1
    over, under = grid[hi] - mag, mag - grid[lo]
    take_hi = (over < under) | ((over == under) & (hi % 2 == 0))
    return torch.where(take_hi, grid[hi], grid[lo]) * torch.sign(y), scale


def _exact_rows(st, i, upto, codes, scales):
    """Rows 0 .. upto - 1 of sequence i in 64 bits, [hkv, upto, d]."""
    rows = st["case"]["rows"]
    pages = st["table"][i, :-(-upto // rows)].long()
    x = codes.view(torch.uint8)[pages].view(codes.dtype) if codes.dtype == torch.float8_e4m3fn else codes[pages]
    x = x.double()
    if scales is not None:
        x = x * scales[pages].double()[..., None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[-1])[:, :upto]


def _exact_one(q, k, v):
    """q [hq, a, d] over k, v [hkv, t, d], causal from the end: out [hq, a, d], lse [hq, a]."""
    hq, a, d = q.shape
    hkv, t, _ = k.shape
    out, lse = torch.zeros_like(q), torch.full((hq, a), -math.inf, dtype=q.dtype, device=DEV)
    if not t:
        return out, lse
    hidden = torch.ones((a, t), dtype=torch.bool, device=DEV).triu(t - a + 1)
    for h in range(hq):
        s = (q[h] @ k[h // (hq // hkv)].T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
        lse[h] = torch.logsumexp(s, -1)
        some = (lse[h] > -math.inf)[:, None]
        out[h] = torch.where(some, torch.nan_to_num(torch.softmax(s, -1)) @ v[h // (hq // hkv)], 0.0)
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    lens = _lens(case)
    if case["op"] in ("prompt", "attend"):
        outs, lses = [], []
        for i, (a, t) in enumerate(lens):
            if case["op"] == "prompt":
                q0, k0 = int(st["cu_q"][i]), int(st["cu_k"][i])
                q = st["q"][q0:q0 + a]
                k, v = (st[x][k0:k0 + t].double().transpose(0, 1) for x in ("k", "v"))
            else:
                q = st["q"][i]
                k, v = (_exact_rows(st, i, t, st[c], st[s]) for c, s in (("kc", "ks"), ("vc", "vs")))
            o, l = _exact_one(q.double().transpose(0, 1), k, v)
            outs.append(o.transpose(0, 1))
            lses.append(l.T)
        join = torch.cat if case["op"] == "prompt" else torch.stack
        return {"out": join(outs), "lse": join(lses)}
    if case["op"] == "read":
        got = {}
        for name, codes, scales in (("k", "kc", "ks"), ("v", "vc", "vs")):
            got[name] = torch.cat([_exact_rows(st, i, t, st[codes], st[scales])[:, t - a:].transpose(0, 1)
                                   for i, (a, t) in enumerate(lens)])
        return got
    rows, got = case["rows"], {}
    for name, codes, scales in (("k", "kc", "ks"), ("v", "vc", "vs")):
        full = (st[codes].view(torch.uint8).view(st[codes].dtype) if case["kind"] == E4M3 else st[codes]).double()
        sc = None if st[scales] is None else st[scales].clone()
        for i, (a, t) in enumerate(lens):
            pos = torch.arange(t - a, t, device=DEV)
            page, row = st["table"][i].long()[pos // rows], pos % rows
            new = st[name][int(st["cu"][i]):int(st["cu"][i]) + a]
            if sc is None:
                full[page, :, row] = new.double()
            else:
                full[page, :, row], sc[page, :, row] = _exact_codes(new, case["kind"])
        got[name] = full if case["kind"] != INT8 else full.round().to(torch.int8)
        if sc is not None:
            got[name + "_scale"] = sc
    return got
