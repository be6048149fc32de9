"""Every key of the two attentions met once: needles and counts.

Needles.  Keys are rows of signs, and a query is 8 times the key at one position t: its
score there is 8 sqrt(d), exactly (whole numbers), and what all other keys weigh beside
it is computed and at most 1e-4 of it.  So out is row t of the values and the log-sum-exp
8 sqrt(d).  A key that is left out leaves another row and a log-sum-exp smaller by some
9, one that is met twice a log-sum-exp larger by log 2.  The log-sum-exp's error is the other
keys' 1e-4 and fp32's (90 times 2^-22 = 2e-5): 1e-3 is far above the one and far below
the other.  out: half a step for the weight's rounding to bf16 and half a step for the
result's (2^-8 each), the other keys' 2e-4 of the largest value (once for their rows, once
for the sum), and from an 8-bit cache f16's least weight as in test_gpu_dense.

Counts.  With keys of zeros every weight is 1, sums of them are exact, and the
log-sum-exp is log(n) to 2e-6 (below 2^16 the base-2 logarithm has steps of 2^-20 at most,
and it and its product with log 2 are off by one and a half of them): one key more or
less makes 1 / n, half of which is 7.6e-6 there.
"""
import math

import numpy as np
import pytest

from test_gpu_dense import BF16, E4M3, INT8, KINDS, Paged, _np, dhs, torch  # noqa: F401
from test_gpu_dense_plans import _assert_few_long_items

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ needles
def _signs(torch, n, hkv, d, g):  # noqa: F811
    return torch.randint(0, 2, (n, hkv, d), generator=g, device="cuda").float() * 2 - 1


def _others(torch, k):  # noqa: F811
    """The most that all other keys weigh beside the needle's own, k [n, d]."""
    worst, (n, d) = 0.0, k.shape
    for i in range(0, n, 2048):
        s = (k[i:i + 2048] @ k.T).double() * (8 / math.sqrt(d))
        w = torch.exp(s - 8 * math.sqrt(d)).sum(1) - 1
        worst = max(worst, w.max().item())
    return worst


def _store(torch, pc, k, seed):  # noqa: F811
    """Signs as the keys of every sequence and random values; the values as they read back,
    fp32 [n, hkv, d] per sequence."""
    c, got = pc.cache, []
    g = torch.Generator(device="cuda").manual_seed(seed)
    for i, n in enumerate(pc.lens):
        pos = torch.arange(n, device="cuda")
        page, row = pc.table[i].long()[pos // pc.rows], pos % pc.rows
        if pc.kind == BF16:
            v = torch.randn((n, pc.hkv, pc.d), generator=g, device="cuda").bfloat16()
            c.k[page, :, row], c.v[page, :, row] = k[i].bfloat16(), v
            got.append(v.float())
            continue
        codes = torch.randint(-127, 128, (n, pc.hkv, pc.d), generator=g, device="cuda").to(torch.int8)
        one, scale = k[i].to(torch.int8), 1 / 64
        if pc.kind == E4M3:
            codes = (codes & -2).view(torch.float8_e4m3fn)       # finite codes
            one, scale = k[i].to(torch.float8_e4m3fn), 1 / 128
        for at, scales, x, s in ((c.k, c.k_scale, one, 1.0), (c.v, c.v_scale, codes, scale)):
            at.view(torch.uint8)[page, :, row] = x.view(torch.uint8)
            scales[page, :, row] = s
        got.append(codes.float() * scale)
    return got


def _check_needles(torch, out, lse, v, d, nk, kind):  # noqa: F811
    """out and lse of rows whose needles' values are v."""
    vmax = 3.5 if kind == E4M3 else 2.0 if kind == INT8 else 6.0
    tol = v.abs() * 2.0 ** -7 + 2e-4 * vmax + (0 if kind == BF16 else nk * 2.0 ** -31 * 2 * vmax)
    wrong = ((out.float() - v).abs() > tol).any(-1) | ((lse - 8 * math.sqrt(d)).abs() > 1e-3)
    assert not wrong.any(), "%d needles, first %s" % (wrong.sum(), wrong.nonzero()[0].tolist())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,q_len,hq,hkv,d,rows,few", [
    ([20011, 18999], 1, 8, 1, 128, 64, True),          # the plan for few long items
    ([9001, 777, 64, 1, 2500], 1, 16, 2, 128, 48, False),
    ([5003, 6100], 2, 16, 1, 64, 7, False),
    ([3001, 700], 8, 8, 1, 128, 64, False),
    ([4099], 1, 128, 1, 64, 100, False),
    ([2500, 1300], 8, 16, 1, 128, 64, False)])
def test_attend_meets_every_key_once(torch, dhs, kind, lens, q_len, hq, hkv, d, rows, few):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(7)
    pc = Paged(torch, dhs, lens, rows, hkv, d, kind)
    k = [_signs(torch, n, hkv, d, g) for n in lens]
    assert max(_others(torch, x[:, h]) for x in k for h in range(hkv)) <= 1e-4
    v = _store(torch, pc, k, 8)
    ws = pc.cache.attend_workspace(len(lens), q_len, hq)
    out = torch.empty((len(lens), q_len, hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((len(lens), q_len, hq), device="cuda")
    head = torch.arange(hq, device="cuda") // (hq // hkv)
    grp, each = hq // hkv, torch.arange(hq, device="cuda") % (hq // hkv)
    j = torch.arange(q_len, device="cuda")[:, None]
    for base in range(0, max(lens), grp * q_len):      # every position of every kv head
        want, q = [], []
        for i, n in enumerate(lens):
            t = (base + j * grp + each) % (n - q_len + 1 + j).clamp(min=1)
            q.append(8 * k[i][t, head])
            want.append(v[i][t, head])
        pc.cache.attend(torch.stack(q).bfloat16(), pc.seq_lens, pc.table, out, ws, lse=lse)
        see = torch.tensor(lens, device="cuda")[:, None] - q_len + 1 + j[None, :, 0] > 0
        _check_needles(torch, out[see], lse[see], torch.stack(want)[see], d, max(lens), kind)
    pc.cache.check()
    if few:
        _assert_few_long_items(ws, len(lens), hkv, len(lens) * hkv)


@pytest.mark.parametrize("lq,lk,hq,hkv,d,split", [
    ([40], [9000], 8, 2, 128, True), ([300], [12000], 4, 1, 64, True), ([2, 130], [7001, 3000], 16, 1, 128, True),
    ([700, 129], [700, 129], 8, 2, 128, False), ([500] * 20, [1100] * 20, 32, 8, 64, False)])
def test_prompt_meets_every_key_once(torch, dhs, lq, lk, hq, hkv, d, split):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(9)
    k = [_signs(torch, n, hkv, d, g) for n in lk]
    assert max(_others(torch, x[:, h]) for x in k for h in range(hkv)) <= 1e-4
    v = [torch.randn((n, hkv, d), generator=g, device="cuda").bfloat16() for n in lk]
    cq, ck = (torch.tensor([0] + x).cumsum(0).int().cuda() for x in (lq, lk))
    kc, vc = torch.cat(k).bfloat16(), torch.cat(v)
    q0 = torch.empty((sum(lq), hq, d), dtype=torch.bfloat16, device="cuda")
    ws = dhs.prompt_workspace(q0, kc, len(lq))
    assert (ws is not None) == split
    head = torch.arange(hq, device="cuda") // (hq // hkv)
    grp, each = hq // hkv, torch.arange(hq, device="cuda") % (hq // hkv)
    rows = min(lq) * grp
    for base in range(0, max(lk), rows):
        q, want = [], []
        for i, (a, b) in enumerate(zip(lq, lk)):
            u = torch.arange(a, device="cuda")[:, None]
            t = (base + u * grp + each) % (b - a + 1 + u)
            q.append(8 * k[i][t, head])
            want.append(v[i][t, head])
        q = torch.cat(q).bfloat16()
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        dhs.prompt_attend(q, kc, vc, cq, ck, out, lse=lse, workspace=ws)
        _check_needles(torch, out, lse, torch.cat(want).float(), d, max(lk), BF16)
    dhs.check_errors()


# ------------------------------------------------------------------ counts
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,d", [(1, 128), (16, 64), (32, 128), (128, 128)])
def test_attend_counts_every_length(torch, dhs, kind, hq, d):  # noqa: F811
    """All lengths to 600 beside one another, and long ones that many CTAs share."""
    for lens in (list(range(601)), [65535, 20011], [40000, 3, 9999, 0, 1]):
        pc = Paged(torch, dhs, lens, 16, 1, d, kind)
        _store(torch, pc, [torch.zeros((n, 1, d), device="cuda") for n in lens], 3)
        q = torch.randn((len(lens), 1, hq, d)).bfloat16().cuda()
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(len(lens), 1, hq), lse=lse)
        pc.cache.check()
        with np.errstate(divide="ignore"):
            want = np.log(np.array(lens, dtype=np.float64))
        some = np.array(lens) > 0
        got = _np(lse)[:, 0]
        assert np.all(np.isneginf(got[~some]))
        assert np.all(np.abs(got[some] - want[some, None]) * np.array(lens)[some, None] < 0.5)


@pytest.mark.parametrize("a,b,hq,hkv,d,split", [(2000, 2000, 16, 2, 128, False), (300, 65000, 4, 1, 64, True),
                                                (7, 30000, 8, 1, 128, True)])
def test_prompt_counts_every_length(torch, dhs, a, b, hq, hkv, d, split):  # noqa: F811
    q = torch.randn((a, hq, d)).bfloat16().cuda()
    k, v = torch.zeros((b, hkv, d), dtype=torch.bfloat16, device="cuda"), torch.randn((b, hkv, d)).bfloat16().cuda()
    cq, ck = (torch.tensor([0, n], dtype=torch.int32).cuda() for n in (a, b))
    out, lse = torch.empty_like(q), torch.empty((a, hq), device="cuda")
    ws = dhs.prompt_workspace(q, k, 1)
    assert (ws is not None) == split
    dhs.prompt_attend(q, k, v, cq, ck, out, lse=lse, workspace=ws)
    dhs.check_errors()
    n = b - a + 1 + np.arange(a)
    assert np.all(np.abs(_np(lse) - np.log(n.astype(np.float64))[:, None]) * n[:, None] < 0.5)
