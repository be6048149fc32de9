"""Paged-cache and prompt operators on the GPU against the fp64 oracle.

Tolerances.  bf16 output: half a step of the rounding at the end (2^-8 relative),
half a step of each weight's rounding to bf16 before the product with V (2^-8
of sum p|v|), and what the 32-bit scores and sums are off by: a score of
magnitude at most `reach` is a sum of d products (d + 16 half-steps of 2^-24, the
scaling and the base-2 exponential's argument among them), the exponential
itself 2^-21, the sums one half-step per term.  Log-sum-exp: the same without the
two roundings to bf16.  From an 8-bit cache the weights, times their value's scale,
are rounded to f16 instead (2^-11, well inside the bf16 term): as multiples of 2^-6
of the largest scale at most, so that f16's smallest step near zero leaves an error
of up to 2^-25 2^-6 = 2^-31 of the largest weight times the largest scale in each,
and in all of nk positions nk 2^-31 max|v| (the largest weight over the sum is at
most 1; max|v| is taken twice for the largest scale standing on a row without its
largest code).
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

BF16, INT8, E4M3 = 0, 1, 2
KINDS = [BF16, INT8, E4M3]
NAME = {INT8: "int8", E4M3: "e4m3"}


@pytest.fixture(scope="module")
def dhs():
    import hierarchical_sparse_kv_int8_gb300 as m
    m.build()
    return m


@pytest.fixture(scope="module")
def torch():
    import torch as t
    return t


def _close(out, lse, want, d, nk, vmax=0.0):
    o, l, wt, reach = want
    e = reach * (d + 16) * 2.0 ** -24 + 2.0 ** -21
    tol = 2.0 ** -8 * np.abs(o) + wt * (2.0 ** -8 + 2 * e[..., None] + nk * 2.0 ** -24) + 1e-37 \
        + nk * 2.0 ** -31 * 2 * vmax
    fine = np.isfinite(o)
    assert np.array_equal(np.isnan(out), np.isnan(o))
    bad = fine & ~(np.abs(np.where(fine, out - o, 0)) <= np.where(fine, tol, 0))
    assert not bad.any(), "worst %g of its tolerance at %s" % (
        np.nanmax(np.where(fine, np.abs(out - o) / tol, 0)), np.argwhere(bad)[0])
    if lse is None:
        return
    fin = np.isfinite(l)
    assert np.array_equal(np.isneginf(lse), np.isneginf(l))
    tl = 2 * e + nk * 2.0 ** -24 + np.abs(np.where(fin, l, 0)) * 2.0 ** -22
    assert np.all(np.abs(np.where(fin, lse - np.where(fin, l, 0), 0)) <= tl)


def _np(t):
    return t.double().cpu().numpy()


class Paged:
    """A cache whose unused rows are poisoned, with a shuffled page table."""

    def __init__(self, torch, dhs, lens, rows, hkv, d, kind, seed=0, spare=2, huge_pages=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.rows, self.hkv, self.d, self.kind = lens, rows, hkv, d, kind
        need = [-(-max(0, x) // rows) for x in lens]
        self.n_pages = max(1, sum(need)) + spare
        base = max(0, huge_pages - self.n_pages)
        perm = torch.randperm(self.n_pages, generator=g)
        width = max(1, max(need)) + 1
        table = torch.full((len(lens), width), -7, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = (perm[at:at + n] + base).int()
            at += n
        self.table = table.cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32).cuda()
        shape = (self.n_pages + base, hkv, rows, d)
        if kind == BF16:
            k, v = (torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            ks = vs = None
        else:
            k, v = (torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in range(2))
            if kind == E4M3:
                k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
            ks, vs = (torch.full(shape[:3], math.nan, dtype=torch.float32, device="cuda") for _ in range(2))
        self.cache = dhs.PageCache(k, v, ks, vs)
        self.torch = torch

    def fill(self, seed=1, outlier=1.0):
        """Random rows for every position, written by hand (not by the operator).
        Returns float64 K, V per sequence, [len, hkv, d]."""
        torch, got = self.torch, []
        g = torch.Generator().manual_seed(seed)
        c = self.cache
        for i, n in enumerate(self.lens):
            n = max(0, n)
            pos = torch.arange(n)
            page, row = self.table.cpu()[i].long()[pos // self.rows], pos % self.rows
            pair = []
            for codes, scales in ((c.k, c.k_scale), (c.v, c.v_scale)):
                if self.kind == BF16:
                    x = (torch.randn((n, self.hkv, self.d), generator=g) * outlier).bfloat16()
                    codes[page.cuda(), :, row.cuda()] = x.cuda()
                    pair.append(x.double().numpy())
                    continue
                s = torch.rand((n, self.hkv), generator=g) * 0.02 + 0.005
                if self.kind == INT8:
                    b = torch.randint(-127, 128, (n, self.hkv, self.d), generator=g, dtype=torch.int8)
                    val = b.double()
                else:
                    s = s * 0.2
                    b = torch.randint(0, 256, (n, self.hkv, self.d), generator=g, dtype=torch.uint8)
                    b[(b & 127) == 127] = 0x35
                    val = b.view(torch.float8_e4m3fn).double()
                codes.view(torch.uint8)[page.cuda(), :, row.cuda()] = b.view(torch.uint8).cuda()
                scales[page.cuda(), :, row.cuda()] = s.cuda()
                pair.append((val * s.double()[..., None]).numpy())
            got.append(pair)
        return got


def _attend(torch, dhs, pc, kv, q_len, hq, q_lens=None, scale=0.0, seed=5, workspace=None, qmul=1.0):
    from oracle import dense_oracle as oracle
    n, d = len(pc.lens), pc.d
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((n, q_len, hq, d), generator=g) * qmul).bfloat16().cuda()
    out = torch.full_like(q, 77.0)
    lse = torch.full((n, q_len, hq), 77.0, dtype=torch.float32, device="cuda")
    ws = pc.cache.attend_workspace(n, q_len, hq) if workspace is None else workspace
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32).cuda()
    pc.cache.attend(q, pc.seq_lens, pc.table, out, ws, lse=lse, q_lens=ql, scale=scale)
    pc.cache.check()
    for i in range(n):
        nq = q_len if q_lens is None else q_lens[i]
        want = oracle.attend(_np(q[i, :nq]), kv[i][0], kv[i][1], scale or 1 / math.sqrt(d))
        vmax = np.abs(kv[i][1]).max() if pc.kind != BF16 and pc.lens[i] else 0.0
        _close(_np(out[i, :nq]), _np(lse[i, :nq]), want, d, max(1, pc.lens[i]), vmax)
        assert torch.all(out[i, nq:] == 77) and torch.all(lse[i, nq:] == 77)


# ------------------------------------------------------------------ write and read
def _tokens(torch, n, hkv, d, seed, hard=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, hkv, d), generator=g) * torch.exp2(
        torch.randint(-12, 12, (n, hkv, 1), generator=g).float())
    x = x.bfloat16()
    if hard and n > 8:
        x[0] = 0                                   # a row of zeros
        x[1] = 2.0 ** -110                         # below the smallest scale
        x[2, :, 3] = math.inf
        x[3, :, d - 1] = math.nan
        x[4] = 3.3e38                              # the largest scales
        x[5, :, ::2] = x[5].abs().amax(-1, keepdim=True) / 2     # values half way between two codes
        x[6, :, ::3] = x[6].abs().amax(-1, keepdim=True) * 0.75
        x[7] = -x[7].abs().amax(-1, keepdim=True)
    return x


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,hkv,rows", [(128, 1, 64), (64, 3, 16), (128, 8, 7), (64, 2, 1)])
def test_write_then_read(torch, dhs, kind, d, hkv, rows):
    from oracle import dense_oracle as oracle
    lens, new = [0, 1, 40, 129, 5], [0, 1, 40, 3, 5]
    pc = Paged(torch, dhs, lens, rows, hkv, d, kind)
    c = pc.cache
    cu = torch.tensor([2] + new).cumsum(0).int().cuda()     # two tokens of padding before, three after
    n = 2 + sum(new) + 3
    k, v = _tokens(torch, n, hkv, d, 1), _tokens(torch, n, hkv, d, 2)
    before = [None if t is None else t.clone().view(torch.uint8) for t in (c.k, c.v, c.k_scale, c.v_scale)]
    c.write(k.cuda(), v.cuda(), cu, pc.seq_lens, pc.table)
    c.check()
    table, touched = pc.table.cpu(), torch.zeros((pc.n_pages, hkv, rows), dtype=torch.bool)
    back = {}
    for i, (a, b) in enumerate(zip(new, lens)):
        for u in range(a):
            p, tok = b - a + u, int(cu[i]) + u
            page, row = int(table[i, p // rows]), p % rows
            touched[page, :, row] = True
            for h in range(hkv):
                for x, codes, scales in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
                    got = codes[page, h, row].view(torch.uint8).cpu().numpy()
                    if kind == BF16:
                        assert np.array_equal(got, x[tok, h].view(torch.uint8).numpy())
                        continue
                    want, s = oracle.quantise(x[tok, h].double().numpy(), NAME[kind])
                    assert np.array_equal(got, want.astype(np.uint8)), (tok, h)
                    assert np.array_equal(np.float32(scales[page, h, row].item()), s, equal_nan=True)
                    back[tok, h, x is k] = oracle.value(want, s, NAME[kind])
    for was, t in zip(before, (c.k, c.v, c.k_scale, c.v_scale)):
        if was is not None:
            now = t.view(torch.uint8)
            keep = ~touched.cuda()
            assert torch.equal(now.view(*touched.shape, -1)[keep], was.view(*touched.shape, -1)[keep])
    ko, vo = (torch.full((n, hkv, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.read(ko, vo, cu, pc.seq_lens, pc.table)
    c.check()
    for x, o, is_k in ((k, ko, True), (v, vo, False)):
        assert torch.all(o[:2] == 5) and torch.all(o[n - 3:] == 5)
        if kind == BF16:
            assert torch.equal(o[2:n - 3].cpu().view(torch.int16), x[2:n - 3].view(torch.int16))
        else:
            for (tok, h, side), val in back.items():
                if side == is_k:
                    got = _np(o[tok, h])
                    with np.errstate(invalid="ignore"):
                        # one rounding to fp32 and one to bf16
                        assert np.array_equal(np.isnan(got), np.isnan(val))
                        assert np.all(np.isnan(val) | (np.abs(got - val) <= np.abs(val) * (2.0 ** -8 + 2.0 ** -24)
                                                       + 2.0 ** -133))


@pytest.mark.parametrize("kind", [INT8, E4M3])
def test_every_bf16_ratio_is_rounded_exactly(torch, dhs, kind):
    """Rows of one largest value and many others: all 128 mantissas against all
    128, where ties and near-ties sit."""
    from oracle import dense_oracle as oracle
    d, hkv = 128, 4
    pc = Paged(torch, dhs, [128], 64, hkv, d, kind)
    bits = torch.arange(128, dtype=torch.int16)
    k = torch.zeros((128, hkv, d), dtype=torch.int16)
    for h in range(hkv):
        k[:, h] = (0x3F80 - 128 * h) + bits[None]       # 1 .. 2, an octave lower per head
        k[:, h, 0] = 0x4000 + bits                      # the largest
    k = k.view(torch.bfloat16)
    v = -k
    cu = torch.tensor([0, 128], dtype=torch.int32).cuda()
    pc.cache.write(k.cuda(), v.cuda(), cu, pc.seq_lens, pc.table)
    for x, codes in ((k, pc.cache.k), (v, pc.cache.v)):
        for tok in range(128):
            page = int(pc.table[0, tok // 64])
            for h in range(hkv):
                want, _ = oracle.quantise(x[tok, h].double().numpy(), NAME[kind])
                got = codes[page, h, tok % 64].view(torch.uint8).cpu().numpy()
                assert np.array_equal(got, want.astype(np.uint8)), (tok, h)


@pytest.mark.parametrize("kind", KINDS)
def test_write_and_read_strided(torch, dhs, kind):
    """Keys and values as views of one fused projection, and of a padded buffer."""
    hkv, d, n = 2, 64, 150
    fused = torch.randn((n, (8 + 2 * hkv) * d)).bfloat16().cuda()
    k = fused[:, 8 * d:(8 + hkv) * d].view(n, hkv, d)
    v = fused[:, (8 + hkv) * d:].view(n, hkv, d)
    a, b = (Paged(torch, dhs, [100, 50], 48, hkv, d, kind, seed=3) for _ in range(2))
    cu = torch.tensor([0, 100, 150], dtype=torch.int32).cuda()
    a.cache.write(k, v, cu, a.seq_lens, a.table)
    b.cache.write(k.contiguous(), v.contiguous(), cu, b.seq_lens, b.table)
    assert torch.equal(a.cache.k.view(torch.uint8), b.cache.k.view(torch.uint8))
    assert torch.equal(a.cache.v.view(torch.uint8), b.cache.v.view(torch.uint8))
    wide = torch.zeros((n, hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    ko, vo = torch.empty_like(k), wide[:, :, 1]
    a.cache.read(ko, vo, cu, a.seq_lens, a.table)
    k2, v2 = torch.empty_like(k.contiguous()), torch.empty_like(k.contiguous())
    a.cache.read(k2, v2, cu, a.seq_lens, a.table)
    assert torch.equal(ko, k2) and torch.equal(vo, v2) and torch.all(wide[:, :, 0] == 0)


def test_write_many_sequences(torch, dhs):
    """Hundreds of sequences of zero, one and a few tokens: each finds its own."""
    n = 700
    new = [(i * 7) % 4 for i in range(n)]
    lens = [x + (i % 5) for i, x in enumerate(new)]
    pc = Paged(torch, dhs, lens, 16, 1, 64, BF16)
    cu = torch.tensor([0] + new).cumsum(0).int().cuda()
    k = torch.randn((sum(new), 1, 64)).bfloat16().cuda()
    pc.cache.write(k, k + 1, cu, pc.seq_lens, pc.table)
    ko, vo = torch.zeros_like(k), torch.zeros_like(k)
    pc.cache.read(ko, vo, cu, pc.seq_lens, pc.table)
    pc.cache.check()
    assert torch.equal(ko, k) and torch.equal(vo, k + 1)


@pytest.mark.parametrize("what", ["page_high", "page_negative", "short", "long", "offsets"])
def test_bad_pages_and_lengths_are_reported_and_skipped(torch, dhs, what):
    lens = [70, 30]
    pc = Paged(torch, dhs, lens, 16, 2, 64, BF16)
    kv = pc.fill()
    c = pc.cache
    cu = torch.tensor([0, 70, 100], dtype=torch.int32).cuda()
    if what == "page_high":
        pc.table[0, 2] = c.n_pages
    elif what == "page_negative":
        pc.table[0, 0] = -1
    elif what == "short":
        pc.seq_lens[0] = 60                       # 70 tokens of a sequence of 60
    elif what == "long":
        pc.seq_lens[0] = pc.table.shape[1] * 16 + 1
    else:
        cu = torch.tensor([0, 120, 100], dtype=torch.int32).cuda()
    ko, vo = (torch.full((100, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    before = c.k.clone()
    c.read(ko, vo, cu, pc.seq_lens, pc.table)
    with pytest.raises(dhs.DhsError) as e:
        c.check()
    assert e.value.code == 5 and "dhs_page_read" in str(e.value)
    c.check()                                     # the record is taken once
    if what != "offsets":
        assert np.array_equal(_np(ko[70:]), kv[1][0])   # the other sequence is served
    c.write(ko, vo, cu, pc.seq_lens, pc.table)
    with pytest.raises(dhs.DhsError) as e:
        c.check()
    assert "dhs_page_write" in str(e.value)
    if what == "offsets":
        return
    untouched = torch.ones(c.n_pages, dtype=torch.bool)
    for i, n in enumerate(lens):
        untouched[pc.table[i, :-(-n // 16)].cpu().clamp(0, c.n_pages - 1).long()] = False
    assert torch.equal(c.k.view(torch.int16)[untouched.cuda()], before.view(torch.int16)[untouched.cuda()])


# ------------------------------------------------------------------ attention over pages
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv,d,rows,q_len", [
    (8, 1, 128, 64, 1), (16, 1, 128, 64, 4), (16, 1, 128, 64, 8), (4, 4, 64, 16, 1), (6, 2, 64, 48, 3),
    (14, 2, 128, 7, 1), (32, 8, 64, 128, 2), (5, 1, 128, 1, 5), (64, 1, 64, 32, 1), (128, 1, 128, 64, 1)])
def test_attend(torch, dhs, kind, hq, hkv, d, rows, q_len):
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 200, 7, 129]
    pc = Paged(torch, dhs, lens, rows, hkv, d, kind)
    kv = pc.fill()
    _attend(torch, dhs, pc, kv, q_len, hq)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_long_and_ragged(torch, dhs, kind):
    """Lengths that many CTAs share and one that none does; a scale of its own."""
    pc = Paged(torch, dhs, [20011, 3, 0, 7777, 1024], 64, 1, 128, kind)
    _attend(torch, dhs, pc, pc.fill(), 2, 8, scale=0.3)


@pytest.mark.parametrize("q_lens", [[0, 1, 2, 3, 4], [4, 0, 0, 0, 0]])
def test_attend_fewer_queries_than_room(torch, dhs, q_lens):
    pc = Paged(torch, dhs, [50, 1, 300, 2, 3], 16, 2, 128, BF16)
    _attend(torch, dhs, pc, pc.fill(), 4, 8, q_lens=q_lens)


def test_attend_many_sequences(torch, dhs):
    lens = [(i * 37) % 90 for i in range(500)]
    pc = Paged(torch, dhs, lens, 16, 1, 64, INT8)
    _attend(torch, dhs, pc, pc.fill(), 1, 2)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_large_scores(torch, dhs, kind):
    """Scores of several hundred: the running maximum grows many times."""
    pc = Paged(torch, dhs, [700, 64], 64, 1, 128, kind)
    _attend(torch, dhs, pc, pc.fill(outlier=8.0), 1, 8, qmul=30.0)


def test_attend_ignores_what_a_query_does_not_see(torch, dhs):
    """The last rows of a sequence hold NaN and infinities: queries before them
    are as if they were not there, queries from them on are not finite."""
    from oracle import dense_oracle as oracle
    for where, d in [(3, 128), (2, 64), (1, 128)]:
        pc = Paged(torch, dhs, [66, 130], 64, 1, d, BF16)
        kv = pc.fill()
        for i, n in enumerate(pc.lens):
            p = n - where
            pg, r = int(pc.table[i, p // 64]), p % 64
            pc.cache.k[pg, 0, r, 5], pc.cache.v[pg, 0, r, 7] = math.nan, math.inf
            pc.cache.v[pg, 0, r, 8] = -math.inf
        q = torch.randn((2, 4, 8, d)).bfloat16().cuda()
        out = torch.zeros_like(q)
        pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(2, 4, 8))
        for i, n in enumerate(pc.lens):
            want = oracle.attend(_np(q[i]), kv[i][0], kv[i][1], 1 / math.sqrt(d))
            first = 4 - where                    # the first query that sees the row
            _close(_np(out[i, :first]), None, [w[:first] for w in want], d, n)
            assert torch.isnan(out[i, first:]).all()


def test_attend_values_of_infinity_reach_the_queries_that_see_them(torch, dhs):
    for p in (0, 40, 63, 64):                    # before the last three rows, and among them
        pc = Paged(torch, dhs, [65], 64, 1, 128, BF16)
        kv = pc.fill()
        pg, r = int(pc.table[0, p // 64]), p % 64
        pc.cache.v[pg, 0, r, 7], pc.cache.v[pg, 0, r, 9] = math.inf, -math.inf
        kv[0][1][p] = 0
        q = torch.randn((1, 3, 8, 128)).bfloat16().cuda()
        out = torch.zeros_like(q)
        pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(1, 3, 8))
        for j in range(3):
            sees = p <= 65 - 3 + j
            assert torch.all(out[0, j, :, 7] == math.inf) == sees
            assert torch.all(out[0, j, :, 9] == -math.inf) == sees
            rest = [x for x in range(128) if x not in (7, 9)]
            assert torch.isfinite(out[0, j][:, rest]).all()


def test_attend_infinite_keys(torch, dhs):
    """A key row of infinities in one direction takes all the weight or none, as in the
    formula (inf - inf is NaN there)."""
    pc = Paged(torch, dhs, [40], 16, 1, 64, BF16)
    kv = pc.fill()
    pc.cache.k[int(pc.table[0, 1]), 0, 3, 0] = -math.inf
    q = torch.randn((1, 1, 2, 64)).bfloat16()
    q[0, 0, 0, 0], q[0, 0, 1, 0] = 1.0, -1.0
    q = q.cuda()
    out = torch.zeros_like(q)
    pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(1, 1, 2))
    keep = [t for t in range(40) if t != 19]
    from oracle import dense_oracle as oracle
    want = oracle.attend(_np(q[0]), kv[0][0][keep], kv[0][1][keep], 1 / 8)
    _close(_np(out[0])[:, :1], None, [w[:, :1] for w in want], 64, 40)
    assert torch.isnan(out[0, 0, 1]).all()


def test_attend_scores_of_minus_infinity_only(torch, dhs):
    """Every visible score is -infinity: 0 / 0, not the zeros of an empty row."""
    pc = Paged(torch, dhs, [20], 16, 1, 64, BF16)
    pc.fill()
    pc.cache.k[:, :, :, 0] = -math.inf
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    out = torch.zeros_like(q)
    lse = torch.zeros((1, 1, 1), device="cuda")
    pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(1, 1, 1), lse=lse)
    assert torch.isnan(out).all() and lse.item() == -math.inf


def test_attend_reports_bad_pages_and_lengths(torch, dhs):
    from oracle import dense_oracle as oracle
    pc = Paged(torch, dhs, [200, 40], 16, 1, 128, BF16)
    kv = pc.fill()
    q = torch.randn((2, 1, 8, 128)).bfloat16().cuda()
    out = torch.zeros_like(q)
    ws = pc.cache.attend_workspace(2, 1, 8)
    good = pc.table.clone()
    for page in (pc.cache.n_pages, -1, 2 ** 31 - 1):
        pc.table[0, 5] = page
        pc.cache.attend(q, pc.seq_lens, pc.table, out, ws)
        with pytest.raises(dhs.DhsError) as e:
            pc.cache.check()
        assert e.value.code == 5 and "page" in str(e.value) and "dhs_page_attend" in str(e.value)
        keep = [t for t in range(200) if t // 16 != 5]       # the rows in question are left out
        for i, (kk, vv) in enumerate([(kv[0][0][keep], kv[0][1][keep]), kv[1]]):
            _close(_np(out[i]), None, oracle.attend(_np(q[i]), kk, vv, 1 / math.sqrt(128)), 128, 200)
    pc.table.copy_(good)
    for bad in (-5, good.shape[1] * 16 + 1):
        pc.seq_lens[1] = bad
        pc.table[1, 3:] = good[1, 0]
        pc.cache.attend(q, pc.seq_lens, pc.table, out, ws)
        with pytest.raises(dhs.DhsError):
            pc.cache.check()
        _close(_np(out[0]), None, oracle.attend(_np(q[0]), *kv[0], 1 / math.sqrt(128)), 128, 200)
        if bad < 0:
            assert torch.all(out[1] == 0)
        # (a length past the table is cut to it: the poisoned rows behind the
        # sequence are then visible, so nothing finite is expected of out[1])
    ql = torch.tensor([2, -1], dtype=torch.int32).cuda()
    pc.seq_lens[1] = 40
    pc.cache.attend(q, pc.seq_lens, pc.table, out, ws, q_lens=ql)
    with pytest.raises(dhs.DhsError):
        pc.cache.check()


def test_attend_far_pages(torch, dhs):
    """Pages past 2^31 bytes and elements of the pool."""
    pc = Paged(torch, dhs, [300, 65], 64, 1, 128, INT8, huge_pages=(1 << 31) // (64 * 128) + 40)
    assert pc.cache.k.numel() > 1 << 31
    _attend(torch, dhs, pc, pc.fill(), 1, 8)
    k = torch.randn((365, 1, 128)).bfloat16().cuda()
    cu = torch.tensor([0, 300, 365], dtype=torch.int32).cuda()
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    pc.cache.write(k, -k, cu, pc.seq_lens, pc.table)
    pc.cache.read(ko, vo, cu, pc.seq_lens, pc.table)
    pc.cache.check()
    assert torch.equal(ko, -vo) and (ko - k).abs().max() < 0.05


def test_attend_ignores_scales_of_rows_it_does_not_see(torch, dhs):
    """Unused rows of an 8-bit cache have NaN scales (the poison of every test here);
    a visible row with a NaN scale makes its sequence NaN and no other."""
    for side in ("k_scale", "v_scale"):
        pc = Paged(torch, dhs, [50, 40], 16, 1, 64, INT8)
        kv = pc.fill()
        getattr(pc.cache, side)[int(pc.table[0, 1]), 0, 3] = math.nan
        q = torch.randn((2, 1, 4, 64)).bfloat16().cuda()
        out = torch.zeros_like(q)
        pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(2, 1, 4))
        from oracle import dense_oracle as oracle
        assert torch.isnan(out[0]).all()
        _close(_np(out[1]), None, oracle.attend(_np(q[1]), *kv[1], 1 / 8), 64, 40, np.abs(kv[1][1]).max())


def test_attend_scales_far_apart(torch, dhs):
    """Value scales that grow by 2^40 along the sequence, zeros among them: each row's
    result is as exact as its own largest terms."""
    from oracle import dense_oracle as oracle
    pc = Paged(torch, dhs, [640], 64, 1, 128, INT8)
    kv = pc.fill()
    grow = torch.exp2((torch.arange(640) // 16).float() - 20)
    grow[100:130] = 0
    pos = torch.arange(640)
    page, row = pc.table.cpu()[0].long()[pos // 64].cuda(), (pos % 64).cuda()
    pc.cache.v_scale[page, 0, row] *= grow.cuda()
    v = kv[0][1] * grow.double().numpy()[:, None, None]
    q = torch.randn((1, 2, 8, 128)).bfloat16().cuda()
    out = torch.zeros_like(q)
    pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(1, 2, 8))
    want = oracle.attend(_np(q[0]), kv[0][0], v, 1 / math.sqrt(128))
    _close(_np(out[0]), None, want, 128, 640, np.abs(v).max())


@pytest.mark.parametrize("kind", [INT8, E4M3])
@pytest.mark.parametrize("hq,d", [(2, 128), (4, 64), (8, 128), (16, 64), (32, 128)])
def test_attend_large_scales_that_some_queries_do_not_see(torch, dhs, kind, hq, d):
    """The last rows' value scales are 2^60 times the others': the queries before them are
    as exact as without (their tolerance counts only values that they see)."""
    from oracle import dense_oracle as oracle
    for where in (1, 3):
        pc = Paged(torch, dhs, [2, 3, 64, 65, 66, 67, 129, 130, 700], 64, 1, d, kind)
        kv = pc.fill()
        for i, n in enumerate(pc.lens):
            for p in range(max(0, n - where), n):
                pc.cache.v_scale[int(pc.table[i, p // 64]), 0, p % 64] *= 2.0 ** 60
                kv[i][1][p] *= 2.0 ** 60
        q = torch.randn((9, 4, hq, d)).bfloat16().cuda()
        out = torch.zeros_like(q)
        pc.cache.attend(q, pc.seq_lens, pc.table, out, pc.cache.attend_workspace(9, 4, hq))
        pc.cache.check()
        for i, n in enumerate(pc.lens):
            want = oracle.attend(_np(q[i]), *kv[i], 1 / math.sqrt(d))
            vmax = [np.abs(kv[i][1][:max(0, n - 3 + u)]).max(initial=0.0) for u in range(4)]
            _close(_np(out[i]), None, want, d, n, np.array(vmax)[:, None, None])


def test_attend_same_result_again_and_beside_others(torch, dhs):
    """Bits repeat; a sequence's result does not depend on its neighbours' values,
    and a workspace goes from one call to the next, whatever ran before."""
    pc = Paged(torch, dhs, [5000, 900, 1, 12000], 64, 2, 128, E4M3)
    pc.fill()
    q = torch.randn((4, 2, 8, 128)).bfloat16().cuda()
    ws = pc.cache.attend_workspace(4, 2, 8)
    outs = []
    for _ in range(3):
        o = torch.zeros_like(q)
        pc.cache.attend(q, pc.seq_lens, pc.table, o, ws)
        outs.append(o)
    other = torch.zeros((4, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
    pc.cache.attend(torch.randn_like(other), pc.seq_lens, pc.table, other, ws)
    q2 = q.clone()
    q2[1:] = 9.0
    o = torch.zeros_like(q)
    pc.cache.attend(q2, pc.seq_lens, pc.table, o, ws)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert torch.equal(o[0], outs[0][0])


def test_attend_refuses_a_small_workspace(torch, dhs):
    pc = Paged(torch, dhs, [5000], 64, 1, 128, BF16)
    q = torch.zeros((1, 1, 8, 128), dtype=torch.bfloat16, device="cuda")
    ws = pc.cache.attend_workspace(1, 1, 8)
    if ws.numel() > 16:
        with pytest.raises(dhs.DhsError) as e:
            pc.cache.attend(q, pc.seq_lens, pc.table, torch.empty_like(q), ws[:ws.numel() - 16])
        assert e.value.code == 1


# ------------------------------------------------------------------ prompts
def _prompt(torch, dhs, sizes, hq, hkv, d, pad=(0, 0), scale=0.0, strided=False, seed=0, qmul=1.0):
    from oracle import dense_oracle as oracle
    g = torch.Generator().manual_seed(seed)
    nq, nk = sum(a for a, _ in sizes) + sum(pad), sum(b for _, b in sizes) + sum(pad)
    if strided:                                   # q, k and v as views of one fused projection
        n = max(nq, nk)
        fused = torch.randn((n, (hq + 2 * hkv) * d), generator=g).bfloat16().cuda()
        q = fused[:nq, :hq * d].view(nq, hq, d)
        k = fused[:nk, hq * d:(hq + hkv) * d].view(nk, hkv, d)
        v = fused[:nk, (hq + hkv) * d:].view(nk, hkv, d)
    else:
        q, k, v = ((torch.randn(s, generator=g) * m).bfloat16().cuda()
                   for s, m in (((nq, hq, d), qmul), ((nk, hkv, d), 1.0), ((nk, hkv, d), 1.0)))
    cq = torch.tensor([pad[0]] + [a for a, _ in sizes]).cumsum(0).int().cuda()
    ck = torch.tensor([pad[0]] + [b for _, b in sizes]).cumsum(0).int().cuda()
    out = torch.full((nq, hq, d), 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((nq, hq), 77.0, dtype=torch.float32, device="cuda")
    err = torch.zeros(2, dtype=torch.int32, device="cuda")
    dhs.prompt_attend(q, k, v, cq, ck, out, lse=lse, scale=scale, errors=err,
                      workspace=dhs.prompt_workspace(q, k, len(sizes)))
    dhs.check_errors(err)
    for i, (a, b) in enumerate(sizes):
        q0, k0 = int(cq[i]), int(ck[i])
        want = oracle.attend(_np(q[q0:q0 + a]), _np(k[k0:k0 + b]), _np(v[k0:k0 + b]), scale or 1 / math.sqrt(d))
        _close(_np(out[q0:q0 + a]), _np(lse[q0:q0 + a]), want, d, max(1, b))
    for lo, hi in ((0, pad[0]), (nq - pad[1], nq)):
        assert torch.all(out[lo:hi] == 77) and torch.all(lse[lo:hi] == 77)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (2, 2), (6, 2), (7, 1), (16, 1)])
def test_prompt_packed(torch, dhs, hq, hkv, d):
    sizes = [(1, 1), (77, 77), (0, 0), (128, 128), (129, 129), (5, 200), (33, 33)]
    _prompt(torch, dhs, sizes, hq, hkv, d, pad=(3, 5))


@pytest.mark.parametrize("sizes", [[(1, 1)], [(2, 1)], [(10, 3), (4, 4)], [(5, 0), (3, 3)], [(0, 7), (2, 9)],
                                   [(1, 700)], [(260, 260)], [(200, 700)]])
def test_prompt_lengths(torch, dhs, sizes):
    """More queries than keys (rows that see nothing), no keys, no queries, chunks."""
    _prompt(torch, dhs, sizes, 4, 2, 128)
    _prompt(torch, dhs, sizes, 4, 1, 64)


def test_prompt_one_kv_head_for_many(torch, dhs):
    _prompt(torch, dhs, [(9, 9), (3, 40)], 128, 1, 128)
    _prompt(torch, dhs, [(9, 9), (3, 40)], 96, 1, 64)
    _prompt(torch, dhs, [(3, 3)], 99, 33, 64)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_strided(torch, dhs, d):
    _prompt(torch, dhs, [(70, 70), (130, 130)], 8, 2, d, strided=True)


def test_prompt_scale_and_large_scores(torch, dhs):
    _prompt(torch, dhs, [(150, 150)], 4, 2, 128, scale=0.02)
    _prompt(torch, dhs, [(300, 300)], 4, 2, 128, qmul=40.0)


def test_prompt_many_sequences(torch, dhs):
    _prompt(torch, dhs, [((i * 5) % 9, (i * 5) % 9 + i % 3) for i in range(600)], 2, 1, 64)


def test_prompt_long_chunk(torch, dhs):
    """Few queries against many keys: the keys are split and joined."""
    _prompt(torch, dhs, [(3, 9000), (17, 5000)], 4, 2, 128)
    _prompt(torch, dhs, [(3, 9000), (1, 3)], 2, 2, 64)


def test_prompt_split_among_many(torch, dhs):
    """Key splits of more items than SMs, sequences without queries or keys among them."""
    sizes = [(37, 2900), (0, 700), (64, 3100), (5, 0), (1, 2600), (50, 3000), (33, 2500), (3, 1)]
    q = torch.empty((sum(a for a, _ in sizes), 16, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((sum(b for _, b in sizes), 8, 64), dtype=torch.bfloat16, device="cuda")
    assert dhs.prompt_workspace(q, k, len(sizes)) is not None
    _prompt(torch, dhs, sizes, 16, 8, 64)


def test_prompt_refuses_a_small_workspace(torch, dhs):
    q = torch.zeros((8, 2, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((9000, 2, 64), dtype=torch.bfloat16, device="cuda")
    cq, ck = (torch.tensor([0, n], dtype=torch.int32).cuda() for n in (8, 9000))
    ws = dhs.prompt_workspace(q, k, 1)
    for bad in (None, ws[:ws.numel() - 16]):
        with pytest.raises(dhs.DhsError) as e:
            dhs.prompt_attend(q, k, k, cq, ck, torch.empty_like(q), workspace=bad)
        assert e.value.code == 1


@pytest.mark.parametrize("d", [64, 128])
def test_outputs_at_sixteen_bytes(torch, dhs, d):
    """Tensors that start 16 bytes into a 256-byte line."""
    from oracle import dense_oracle as oracle
    shift = lambda *s: torch.empty(math.prod(s) + 8, dtype=torch.bfloat16, device="cuda")[8:].view(s)  # noqa: E731
    q, k, v, out = shift(70, 4, d), shift(70, 2, d), shift(70, 2, d), shift(70, 4, d)
    for t in (q, k, v):
        t.copy_(torch.randn(t.shape))
    cu = torch.tensor([0, 70], dtype=torch.int32).cuda()
    dhs.prompt_attend(q, k, v, cu, cu, out)
    want = oracle.attend(_np(q), _np(k), _np(v), 1 / math.sqrt(d))
    _close(_np(out), None, want, d, 70)
    pc = Paged(torch, dhs, [70], 16, 2, d, BF16)
    pc.cache.write(k, v, cu, pc.seq_lens, pc.table)
    q1, o1 = shift(1, 1, 4, d), shift(1, 1, 4, d)
    q1.copy_(torch.randn(q1.shape))
    pc.cache.attend(q1, pc.seq_lens, pc.table, o1, pc.cache.attend_workspace(1, 1, 4))
    _close(_np(o1[0]), None, oracle.attend(_np(q1[0]), _np(k), _np(v), 1 / math.sqrt(d)), d, 70)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_masked_places_do_not_matter(torch, dhs, d):
    """NaN and infinities in keys and values that a query does not see: later ones
    of its own sequence, and those of the neighbours."""
    from oracle import dense_oracle as oracle
    sizes, hq, hkv = [60, 200, 90], 4, 2
    n = sum(sizes)
    q, k, v = (torch.randn((n, h, d)).bfloat16().cuda() for h in (hq, hkv, hkv))
    cu = torch.tensor([0] + sizes).cumsum(0).int().cuda()
    clean = [_np(x) for x in (k, v)]
    k[:60], v[:60] = math.nan, math.inf                       # the whole first sequence
    v[60 + 130, 1, 3], v[60 + 130, 1, 4], k[60 + 131, 0, 2] = math.nan, -math.inf, math.inf
    v[260:] = math.nan                                        # the whole third
    out = torch.zeros_like(q)
    dhs.prompt_attend(q, k, v, cu, cu, out, workspace=dhs.prompt_workspace(q, k, 3))
    want = oracle.attend(_np(q[60:260]), clean[0][60:260], clean[1][60:260], 1 / math.sqrt(d))
    got = _np(out[60:260])
    _close(got[:130], None, [w[:130] for w in want], d, 200)
    assert np.isnan(got[130:, 2:, 3]).all() and np.isneginf(got[130:, 2:, 4]).all()
    clear = [x for x in range(d) if x not in (3, 4)]
    assert np.isfinite(got[130:, 2:][:, :, clear]).all()
    _close(got[130:131, :2], None, [w[130:131, :2] for w in want], d, 200)
    assert torch.isnan(out[:60]).all() and torch.isnan(out[260:]).all()


def test_prompt_infinite_values_of_many_sequences(torch, dhs):
    """Some 400 short sequences (several to a CTA, most with one row tile), half of them
    with an infinite value: it reaches the rows that see it and no other sequence's."""
    from oracle import dense_oracle as oracle
    g = torch.Generator().manual_seed(11)
    sizes = torch.randint(1, 40, (400,), generator=g).tolist()
    sizes[100], sizes[200] = 150, 300
    cu = np.concatenate([[0], np.cumsum(sizes)])
    q, k, v = (torch.randn((int(cu[-1]), h, 64), generator=g).bfloat16() for h in (2, 1, 1))
    for i in range(0, 400, 2):
        v[cu[i] + sizes[i] * 2 // 3, 0, i % 64] = math.inf
    off = torch.tensor(cu, dtype=torch.int32).cuda()
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    out = torch.full_like(qd, 77.0)
    dhs.prompt_attend(qd, kd, vd, off, off, out, workspace=dhs.prompt_workspace(qd, kd, 400))
    for i in range(400):
        r = slice(cu[i], cu[i + 1])
        want = oracle.attend(_np(q[r]), _np(k[r]), _np(v[r]), 1 / 8)
        assert np.array_equal(np.isposinf(_np(out[r])), np.isposinf(want[0])), i
        _close(_np(out[r]), None, want, 64, sizes[i])


def test_prompt_from_cold_memory(torch, dhs):
    """The first tiles come from memory slowly and in any order: every run equals the
    others bit by bit, and sampled rows the oracle."""
    from oracle import dense_oracle as oracle
    sizes = [1500, 1856, 300, 1100, 700]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for hq, hkv, d in ((32, 8, 128), (8, 8, 64)):
        n = sum(sizes)
        q, k, v = (torch.randn((n, h, d), device="cuda").bfloat16() for h in (hq, hkv, hkv))
        cu = torch.tensor([0] + sizes).cumsum(0).int().cuda()
        ws = dhs.prompt_workspace(q, k, len(sizes))
        runs = []
        for _ in range(6):
            out, lse = torch.zeros_like(q), torch.zeros((n, hq), device="cuda")
            flush.zero_()
            torch.cuda.synchronize()
            dhs.prompt_attend(q, k, v, cu, cu, out, lse=lse, workspace=ws)
            runs.append((out, lse))
        for out, lse in runs[1:]:
            assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
        for i, ln in enumerate(sizes):
            at = int(cu[i])
            for u in (0, ln // 3, ln - 1):
                want = oracle.attend(_np(q[at + u:at + u + 1]), _np(k[at:at + u + 1]), _np(v[at:at + u + 1]),
                                     1 / math.sqrt(d))
                _close(_np(runs[0][0][at + u:at + u + 1]), _np(runs[0][1][at + u:at + u + 1]), want, d, u + 1)


def test_prompt_minus_infinity_scores(torch, dhs):
    n, d = 140, 64
    q, k, v = (torch.randn((n, 1, d)).bfloat16().cuda() for _ in range(3))
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    k[:100, :, 0] = -math.inf
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    out, lse = torch.zeros_like(q), torch.zeros((n, 1), device="cuda")
    dhs.prompt_attend(q, k, v, cu, cu, out, lse=lse)
    assert torch.isnan(out[:100]).all() and torch.all(lse[:100] == -math.inf)
    from oracle import dense_oracle as oracle
    want = oracle.attend(_np(q[100:]), _np(k[100:]), _np(v[100:]), 1 / 8)
    _close(_np(out[100:]), _np(lse[100:]), want, d, n)


def test_prompt_reports_bad_offsets(torch, dhs):
    q, k = torch.randn((50, 4, 64)).bfloat16().cuda(), torch.randn((50, 2, 64)).bfloat16().cuda()
    err = torch.zeros(2, dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 20, 50], dtype=torch.int32)
    for which, bad in (("q", [0, 20, 51]), ("k", [0, 20, 51]), ("k", [0, 60, 50]), ("q", [0, 60, 50]),
                       ("k", [-4, 20, 50]), ("q", [-4, 20, 50]), ("k", [0, 2 ** 31 - 1, 50])):
        cu = {x: (torch.tensor(bad, dtype=torch.int32) if x == which else good).cuda() for x in "qk"}
        out = torch.zeros_like(q)
        dhs.prompt_attend(q, k, k, cu["q"], cu["k"], out, errors=err,
                          workspace=dhs.prompt_workspace(q, k, 2))
        with pytest.raises(dhs.DhsError) as e:
            dhs.check_errors(err)
        assert e.value.code == 5 and "dhs_prompt_attend" in str(e.value)
        assert torch.isfinite(out).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("kind", KINDS)
def test_prompt_in_chunks_then_decode(torch, dhs, kind):
    """A prompt in two chunks and three decode steps of two tokens: attend, write,
    read the prefix back, attend the next chunk over it, then decode."""
    from oracle import dense_oracle as oracle
    hq, hkv, d, rows = 8, 2, 128, 16
    first, second, steps = [37, 70], [20, 1], 3
    final = [a + b + 2 * steps for a, b in zip(first, second)]
    pc = Paged(torch, dhs, final, rows, hkv, d, kind)
    c, table = pc.cache, pc.table
    g = torch.Generator().manual_seed(9)
    rnd = lambda n, h: torch.randn((n, h, d), generator=g).bfloat16().cuda()  # noqa: E731
    cum = lambda x: torch.tensor([0] + x).cumsum(0).int().cuda()  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    lens = [0, 0]
    scale = 1 / math.sqrt(d)
    for chunk in (first, second):
        n = sum(chunk)
        q, k, v = rnd(n, hq), rnd(n, hkv), rnd(n, hkv)
        lens = [a + b for a, b in zip(lens, chunk)]
        c.write(k, v, cum(chunk), ints(lens), table)
        kk, vv = (torch.empty((sum(lens), hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        c.read(kk, vv, cum(lens), ints(lens), table)
        out = torch.empty_like(q)
        dhs.prompt_attend(q, kk, vv, cum(chunk), cum(lens), out, workspace=dhs.prompt_workspace(q, kk, 2))
        for i in range(2):
            qs, ks = slice(sum(chunk[:i]), sum(chunk[:i + 1])), slice(sum(lens[:i]), sum(lens[:i + 1]))
            want = oracle.attend(_np(q[qs]), _np(kk[ks]), _np(vv[ks]), scale)
            _close(_np(out[qs]), None, want, d, lens[i])
    ws = c.attend_workspace(2, 2, hq)
    for _ in range(steps):
        k, v = rnd(4, hkv), rnd(4, hkv)
        q = torch.randn((2, 2, hq, d), generator=g).bfloat16().cuda()
        lens = [a + 2 for a in lens]
        c.write(k, v, cum([2, 2]), ints(lens), table)
        out = torch.empty_like(q)
        c.attend(q, ints(lens), table, out, ws)
        kk, vv = (torch.empty((sum(lens), hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        c.read(kk, vv, cum(lens), ints(lens), table)
        for i in range(2):
            ks = slice(sum(lens[:i]), sum(lens[:i + 1]))
            want = oracle.attend(_np(q[i]), _np(kk[ks]), _np(vv[ks]), scale)
            if kind != BF16:                 # rows read back are rounded to bf16 once more
                # keys off by 2^-8 move a score by 2^-8 of its reach, values move by 2^-8
                more = want[2] * (2.0 ** -8 + 2 * np.expm1(2.0 ** -8 * want[3][..., None]))
                assert np.all(np.abs(_np(out[i]) - want[0]) <= 2.0 ** -8 * np.abs(want[0]) * 1.1
                              + want[2] * 2.0 ** -8 * 1.1 + more)
            else:
                _close(_np(out[i]), None, want, d, lens[i])
    c.check()


def test_captured_decode_follows_lengths_and_pages(torch, dhs):
    """A graph of write and attend, replayed after the lengths, rows and page table
    in its tensors have changed; two such graphs, each with its own workspace,
    replayed at the same time on two streams."""
    from oracle import dense_oracle as oracle
    hq, hkv, d, rows, n = 8, 2, 128, 16, 3
    pcs, graphs = [], []
    for s in range(2):
        pc = Paged(torch, dhs, [3000, 40, 17], rows, hkv, d, BF16, seed=s)
        pc.kv = pc.fill(seed=s)
        pc.stream = torch.cuda.Stream()
        pc.q = torch.randn((n, 1, hq, d)).bfloat16().cuda()
        pc.new = [torch.randn((n, hkv, d)).bfloat16().cuda() for _ in range(2)]
        pc.cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
        pc.out = torch.zeros_like(pc.q)
        pc.ws = pc.cache.attend_workspace(n, 1, hq)
        torch.cuda.synchronize()
        gr = dhs.Graph.capture(pc.stream)
        with gr:
            pc.cache.write(*pc.new, pc.cu, pc.seq_lens, pc.table, stream=pc.stream)
            pc.cache.attend(pc.q, pc.seq_lens, pc.table, pc.out, pc.ws, stream=pc.stream)
        pcs.append(pc)
        graphs.append(gr)
    for lens in ([3000, 40, 17], [2990, 1, 0], [65, 39, 16]):
        for pc in pcs:
            pc.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
            for x in pc.new:
                x.copy_(torch.randn((n, hkv, d)).bfloat16())
        if lens[2] == 0:                       # nothing to write for an idle slot
            for pc in pcs:
                pc.cu.copy_(torch.tensor([0, 1, 2, 2], dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(5):
            for gr in graphs:
                gr.replay()
        torch.cuda.synchronize()
        for pc in pcs:
            pc.cache.check()
            for i, ln in enumerate(lens):
                for side in range(2):
                    if ln:
                        pc.kv[i][side][ln - 1] = _np(pc.new[side][i])
                want = oracle.attend(_np(pc.q[i]), pc.kv[i][0][:ln], pc.kv[i][1][:ln], 1 / math.sqrt(d))
                _close(_np(pc.out[i]), None, want, d, max(1, ln))
            pc.cu.copy_(torch.arange(n + 1, dtype=torch.int32))
    for gr in graphs:
        gr.close()


def test_captured_prompt(torch, dhs):
    from oracle import dense_oracle as oracle
    hq, hkv, d = 4, 2, 64
    q, k, v = (torch.randn((300, h, d)).bfloat16().cuda() for h in (hq, hkv, hkv))
    cq, ck = (torch.tensor([0, 100, 300], dtype=torch.int32).cuda() for _ in range(2))
    out = torch.zeros_like(q)
    ws = dhs.prompt_workspace(q, k, 2)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    gr = dhs.Graph.capture(st)
    with gr:
        dhs.prompt_attend(q, k, v, cq, ck, out, workspace=ws, stream=st)
    for cuts in ([0, 100, 300], [0, 299, 300], [10, 10, 150]):
        cq.copy_(torch.tensor(cuts, dtype=torch.int32))
        ck.copy_(torch.tensor(cuts, dtype=torch.int32))
        out.fill_(77.0)
        torch.cuda.synchronize()
        gr.replay()
        torch.cuda.synchronize()
        for a, b in zip(cuts, cuts[1:]):
            want = oracle.attend(_np(q[a:b]), _np(k[a:b]), _np(v[a:b]), 1 / 8)
            _close(_np(out[a:b]), None, want, d, max(1, b - a))
        assert torch.all(out[:cuts[0]] == 77) and torch.all(out[cuts[2]:] == 77)
    gr.close()


def test_calls_on_another_stream(torch, dhs):
    """A call is ordered on the stream it is given, the current one by default."""
    pc = Paged(torch, dhs, [2000, 100], 64, 1, 128, BF16)
    kv = pc.fill()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    from oracle import dense_oracle as oracle
    q = torch.randn((2, 1, 8, 128)).bfloat16().cuda()
    ws = pc.cache.attend_workspace(2, 1, 8)
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(2_000_000)
        q2 = q * 2
        pc.cache.attend(q2, pc.seq_lens, pc.table, out, ws)
        torch.cuda._sleep(2_000_000)
        q2.zero_()
    torch.cuda.synchronize()
    for i in range(2):
        want = oracle.attend(2 * _np(q[i]), *kv[i], 1 / math.sqrt(128))
        _close(_np(out[i]), None, want, 128, 2000)


def test_two_calls_at_once(torch, dhs):
    """The same calls on two streams at a time, each with a workspace of its own."""
    pc = Paged(torch, dhs, [9000, 300, 4000], 64, 2, 128, INT8)
    pc.fill()
    q = torch.randn((3, 2, 8, 128)).bfloat16().cuda()
    x, kv = torch.randn((700, 8, 128)).bfloat16().cuda(), torch.randn((6000, 2, 128)).bfloat16().cuda()
    cq, ck = (torch.tensor(c, dtype=torch.int32).cuda() for c in ([0, 300, 700], [0, 5000, 6000]))

    def calls(stream):
        with torch.cuda.stream(stream):
            a, b = torch.empty_like(q), torch.empty_like(x)
            ws, pw = pc.cache.attend_workspace(3, 2, 8), dhs.prompt_workspace(x, kv, 2)
            for _ in range(4):
                pc.cache.attend(q, pc.seq_lens, pc.table, a, ws)
                dhs.prompt_attend(x, kv, kv, cq, ck, b, workspace=pw)
            return a, b, ws, pw

    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    alone = calls(one)
    torch.cuda.synchronize()
    for s in (one, two):
        s.wait_stream(torch.cuda.current_stream())
    got = [calls(s) for s in (one, two)]
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], alone[0]) and torch.equal(g[1], alone[1])


def test_prompt_bad_offsets_among_many(torch, dhs):
    """One offset out of range among 300 sequences: the two that it belongs to are left
    alone and reported, the others are as without it."""
    n, t = 300, 5
    q, k = torch.randn((n * t, 4, 64)).bfloat16().cuda(), torch.randn((n * t, 2, 64)).bfloat16().cuda()
    cu = torch.arange(0, n * t + 1, t, dtype=torch.int32)
    bad = cu.clone()
    bad[150] = 10 ** 9
    ws, err = dhs.prompt_workspace(q, k, n), torch.zeros(2, dtype=torch.int32, device="cuda")
    outs = []
    for c in (cu, bad):
        out = torch.full_like(q, 77.0)
        dhs.prompt_attend(q, k, k, cu.cuda(), c.cuda(), out, workspace=ws, errors=err)
        outs.append(out)
    with pytest.raises(dhs.DhsError):
        dhs.check_errors(err)
    r = slice(149 * t, 151 * t)
    assert torch.all(outs[1][r] == 77)
    outs[1][r] = outs[0][r]
    assert torch.equal(outs[0], outs[1])


def test_prompt_past_2_to_the_31_elements(torch, dhs):
    """q and out of more than 2^31 elements: the last sequences are right, and as in a call
    of their own."""
    from oracle import dense_oracle as oracle
    n, t, hq, hkv, d = 500, 33, 1024, 8, 128
    q = torch.empty((n * t, hq, d), dtype=torch.bfloat16, device="cuda")
    assert q.numel() > 1 << 31
    for i in range(0, n * t, 1650):
        q[i:i + 1650] = torch.randn((1650, hq, d), device="cuda")
    k, v = (torch.randn((n * t, hkv, d), device="cuda").bfloat16() for _ in range(2))
    cu = torch.arange(0, n * t + 1, t, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 77.0)
    dhs.prompt_attend(q, k, v, cu, cu, out, workspace=dhs.prompt_workspace(q, k, n))
    last = slice((n - 2) * t, n * t)
    own = torch.empty_like(out[last])
    dhs.prompt_attend(q[last], k[last], v[last], cu[:3], cu[:3], own,
                      workspace=dhs.prompt_workspace(q[last], k[last], 2))
    r = slice((n - 1) * t, n * t)
    want = oracle.attend(_np(q[r, 1020:]), _np(k[r, 7:]), _np(v[r, 7:]), 1 / math.sqrt(d))
    _close(_np(out[r, 1020:]), None, want, d, t)
    assert not (out[:2 * t] == 77).any()
    assert torch.equal(out[last], own)


# ------------------------------------------------------------------ where rows may lie
@pytest.mark.parametrize("n,h", [(4, 2), (3, 4), (1, 3), (5, 1)])
def test_read_into_every_layout_whose_rows_do_not_meet(torch, dhs, n, h):
    """A grid of strides: a layout in which no two rows meet receives every row, heads
    among the tokens and values among the keys included; the others are refused."""
    d = 64
    pc = Paged(torch, dhs, [n], 16, h, d, BF16)
    kv = pc.fill()[0]
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    served = refused = 0
    grid = [8, d - 8, d, d + 8, 2 * d, 3 * d, h * d, 8 * d]
    for st in grid:
        for sh in grid:
            for off in (8, d, -d, 2 * d, st, sh, st + sh, 64 * d):
                buf = torch.full((128 * d,), 5.0, dtype=torch.bfloat16, device="cuda")
                first = 2 * d
                rows = [first + x + i * st + j * sh for x in (0, off) for i in range(n) for j in range(h)]
                ko, vo = (buf.as_strided((n, h, d), (st, sh, 1), first + x) for x in (0, off))
                gaps = np.diff(np.sort(rows))
                if gaps.min() < d:
                    refused += 1
                    with pytest.raises(dhs.DhsError) as e:
                        pc.cache.read(ko, vo, cu, pc.seq_lens, pc.table)
                    assert e.value.code == 1
                    continue
                served += 1
                pc.cache.read(ko, vo, cu, pc.seq_lens, pc.table)
                assert np.array_equal(_np(ko), kv[0]) and np.array_equal(_np(vo), kv[1])
                assert (buf == 5.0).sum().item() >= buf.numel() - 2 * n * h * d
    pc.cache.check()
    assert served and refused


# ------------------------------------------------------------------ what the checks find
def test_prompt_errors_without_a_record_are_kept(torch, dhs):
    """In one record of the device, also for a first call that is captured; calls with a
    record of their own stay out of it."""
    dhs.check_errors()
    q = torch.randn((20, 4, 64)).bfloat16().cuda()
    good, bad = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([0, 12, 20], [0, 25, 20]))
    out = torch.full_like(q, 77.0)
    err = torch.zeros(2, dtype=torch.int32, device="cuda")
    dhs.prompt_attend(q, q, q, bad, bad, out, errors=err)
    dhs.check_errors()
    with pytest.raises(dhs.DhsError):
        dhs.check_errors(err)
    dhs.prompt_attend(q, q, q, bad, bad, out)
    dhs.prompt_attend(q, q, q, good, good, out, errors=err)
    dhs.check_errors(err)
    with pytest.raises(dhs.DhsError) as e:
        dhs.check_errors()
    assert e.value.code == 5 and "dhs_prompt_attend" in str(e.value) and "offset" in str(e.value)
    dhs.check_errors()                            # the record is taken once
    cu, side = bad.clone(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dhs.prompt_attend(q, q, q, cu, cu, out)
    graph.replay()
    with pytest.raises(dhs.DhsError):
        dhs.check_errors()
    cu.copy_(good)
    want = out.clone()
    out.fill_(77.0)
    graph.replay()
    dhs.check_errors(stream=torch.cuda.current_stream())
    dhs.prompt_attend(q, q, q, good, good, want)
    assert torch.equal(out, want) and not (out == 77.0).any()


def test_write_and_read_of_the_last_of_2_30_sequences(torch, dhs):
    """The search among more than 2^30 sequences (all empty but the last; the arrays take
    13 GB) stays within 32 bits."""
    n = (1 << 30) + 5
    pc = Paged(torch, dhs, [1], 16, 1, 64, BF16)
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    lens, table = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
    cu[n], lens[n - 1], table[n - 1, 0] = 1, 1, pc.table[0, 0]
    k = torch.randn((1, 1, 64)).bfloat16().cuda()
    ko, vo = torch.zeros_like(k), torch.zeros_like(k)
    pc.cache.write(k, -k, cu, lens, table)
    pc.cache.read(ko, vo, cu, lens, table)
    pc.cache.check()
    assert torch.equal(ko, k) and torch.equal(vo, -k)
    page = int(pc.table[0, 0])
    assert torch.equal(pc.cache.k[page, 0, 0], k[0, 0])
