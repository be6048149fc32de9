"""Paged attention's plan for few long items, against the fp64 oracle."""
import math

import numpy as np
import pytest

from test_gpu_dense import BF16, KINDS, Paged, _attend, _close, _np, dhs, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def _assert_few_long_items(ws, n, hkv, items):
    """The call took the plan for few long items, by what it left for the join (first and
    last CTA of each item in parts): no CTA has a part of two items.  (Dealt evenly, the
    CTA that ends an item begins the next.)"""
    import torch as t
    got = [p for p in ws[:n * hkv * 8].view(t.int32).view(n * hkv, 2).tolist() if p[0] >= 0]
    assert len(got) == items and items > 1
    assert got[0][0] == 0 and all(last > first for first, last in got)
    assert all(first == last + 1 for (_, last), (first, _) in zip(got, got[1:]))


# two and three sequences; eight and an idle slot; one of two kv heads; two among 42 slots,
# most of them idle, one with rows and without a query
SPARSE = [0] * 17 + [35013] + [0] * 19 + [29777, 3000, 0, 0, 0]
LONG = [([20011, 18999], 1, 8, 1, 128, 64, None),
        ([20011, 30007, 12345], 2, 2, 1, 128, 48, None),
        ([8001, 19000, 0, 12345, 20011, 9999, 16384, 15000, 14001], 4, 1, 1, 128, 64, None),
        ([33333], 1, 4, 2, 64, 16, None),
        (SPARSE, 3, 4, 1, 64, 100, [2] * 18 + [3] * 20 + [0, 1, 2, 3])]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", range(len(LONG)))
def test_attend_few_long_items(torch, dhs, kind, case):  # noqa: F811
    lens, q_len, hq, hkv, d, rows, q_lens = LONG[case]
    pc = Paged(torch, dhs, lens, rows, hkv, d, kind, seed=case)
    kv = pc.fill(seed=case + 10)
    ws = pc.cache.attend_workspace(len(lens), q_len, hq)
    _attend(torch, dhs, pc, kv, q_len, hq, q_lens=q_lens, workspace=ws)
    live = sum(n > 0 and (q_lens is None or q_lens[i] > 0) for i, n in enumerate(lens))
    _assert_few_long_items(ws, len(lens), hkv, live * hkv)


@pytest.mark.parametrize("kind", KINDS)
def test_attend_few_long_items_values_out_of_sight(torch, dhs, kind):  # noqa: F811
    """The last row of a sequence holds what its earlier queries must not meet: NaN and
    infinities, or a value scale of 2^60 times the others."""
    from oracle import dense_oracle as oracle
    lens, d = [20011, 18999], 128
    pc = Paged(torch, dhs, lens, 64, 1, d, kind)
    kv = pc.fill()
    for i, n in enumerate(lens):
        pg, r = int(pc.table[i, (n - 1) // 64]), (n - 1) % 64
        if kind == BF16:
            pc.cache.k[pg, 0, r, 5], pc.cache.v[pg, 0, r, 7] = math.nan, math.inf
        else:
            pc.cache.v_scale[pg, 0, r] *= 2.0 ** 60
            kv[i][1][n - 1] *= 2.0 ** 60
    q = torch.randn((2, 4, 1, d)).bfloat16().cuda()
    out = torch.zeros_like(q)
    ws = pc.cache.attend_workspace(2, 4, 1)
    pc.cache.attend(q, pc.seq_lens, pc.table, out, ws)
    pc.cache.check()
    _assert_few_long_items(ws, 2, 1, 2)
    for i, n in enumerate(lens):
        want = oracle.attend(_np(q[i]), *kv[i], 1 / math.sqrt(d))
        last = 3 if kind == BF16 else 4
        vmax = np.array([np.abs(kv[i][1][:n - 3 + u]).max() for u in range(last)])[:, None, None]
        _close(_np(out[i, :last]), None, [w[:last] for w in want], d, n, vmax if kind != BF16 else 0.0)
        if kind == BF16:
            assert torch.isnan(out[i, 3:]).all()
