"""The chunk kernel's waits, made to run out in a build of its own in which their limit
is a variable: the call still ends, reports it, and writes whole right rows or none."""
import ctypes
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu

TIMEOUT, SITE = 4, 6
LEFT = 77.0


@pytest.fixture(scope="module")
def torch():
    import torch as t
    return t


@pytest.fixture(scope="module")
def libs(tmp_path_factory):
    """The library, and the chunk kernel with the variable."""
    import hierarchical_sparse_kv_int8_gb300 as dhs
    from hierarchical_sparse_kv_int8_gb300 import _build as b
    other = os.path.join(b.OUT_DIR, "k_page_attn.o")
    dhs.build()
    if not os.path.exists(other):
        b.build(force=True)
    d = tmp_path_factory.mktemp("waits")
    obj, so = str(d / "k_chunk.o"), str(d / "libwaits.so")
    subprocess.run([b._nvcc(), *b.ARCH, *b.NVCC_FLAGS, "-DDHS_TEST_WAITS", "-c",
                    os.path.join(b.CSRC, "k_chunk.cu"), "-o", obj], check=True, capture_output=True)
    subprocess.run([b._nvcc(), *b.ARCH, "-shared", "-o", so, obj, other, "-lcudart"], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(so)
    from hierarchical_sparse_kv_int8_gb300 import _SIGS
    for name in ("dhs_page_chunk", "dhs_page_chunk_workspace"):
        f = getattr(lib, name)
        f.argtypes, f.restype = _SIGS[name]
    return dhs, dhs.load(), lib, ctypes.c_uint32.in_dll(lib, "dhs_chunk_wait_us")


def _call(torch, lib, cache, q, cu, lens, table, window):
    out = torch.full_like(q, LEFT)
    lse = torch.full(q.shape[:2], LEFT, device="cuda")
    err = torch.zeros(2, dtype=torch.int32, device="cuda")
    n, hq, _ = q.shape
    nbytes = lib.dhs_page_chunk_workspace(cache._ref, n, lens.shape[0], hq)
    # what a workspace holds before a call does not matter
    ws = torch.randint(0, 256, (nbytes,), dtype=torch.uint8, device="cuda")
    rc = lib.dhs_page_chunk(cache._ref, q.data_ptr(), None, n, cu.data_ptr(), lens.data_ptr(),
                            table.data_ptr(), table.shape[1], lens.shape[0], hq, window, 0, 0.0,
                            out.data_ptr(), lse.data_ptr(), ws.data_ptr(), nbytes, err.data_ptr(),
                            torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    return out, lse, err.tolist()


# Many items a CTA; one row tile only, walked as two halves; cut items that are joined; a window.
# A poll is suspended for some 5 us at most: where no item is `long` all waits may end before.
CASES = [([2000, 33, 900], [2600, 33, 900], 16, 4, 128, 0, True), ([1, 1, 3], [4000, 2000, 900], 8, 2, 64, 0, False),
         ([40, 300], [9000, 3000], 8, 2, 128, 0, False), ([700, 1], [4000, 4000], 4, 2, 64, 500, False)]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("new,lens,hq,hkv,d,window,long", CASES)
def test_waits_that_run_out_leave_rows_out(torch, libs, kind, new, lens, hq, hkv, d, window, long):
    dhs, plain, lib, wait_us = libs
    rows, n = 64, len(lens)
    need = [-(-x // rows) for x in lens]
    cache = dhs.PageCache.empty(sum(need), rows, hkv, d, kind)
    g = torch.Generator(device="cuda").manual_seed(3)
    if kind == 0:
        cache.k.normal_(generator=g)
        cache.v.normal_(generator=g)
    else:
        cache.k.random_(-127, 128, generator=g)
        cache.v.random_(-127, 128, generator=g)
        cache.k_scale.fill_(0.01)
        cache.v_scale.fill_(0.02)
    table = torch.zeros((n, max(need)), dtype=torch.int32)
    at = 0
    for i, x in enumerate(need):
        table[i, :x] = torch.arange(at, at + x)
        at += x
    table, seq = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    cu = torch.tensor([0] + new).cumsum(0).int().cuda()
    q = torch.randn((sum(new), hq, d), generator=g, device="cuda").bfloat16()
    args = (cache, q, cu, seq, table, window)
    want, want_lse, err = _call(torch, plain, *args)
    assert err == [0, 0] and not (want == LEFT).any()
    ran_out = 0
    # from less than the first copies take to more than the call does, in microseconds
    for limit in [0, 0] + list(range(1, 30, 2)) + [40, 60, 100, 150, 2000000]:
        wait_us.value = limit
        out, lse, err = _call(torch, lib, *args)
        assert err in ([0, 0], [TIMEOUT, SITE])
        left = (out == LEFT).all(-1)
        assert torch.equal(left, lse == LEFT)
        assert torch.equal(out[~left], want[~left]) and torch.equal(lse[~left], want_lse[~left])
        if err == [0, 0]:
            assert not left.any()
        else:
            ran_out += 1
    assert err == [0, 0] and (ran_out >= 1 or not long)
    # the GPU is as it was: the library's own kernel gives what it gave
    again, again_lse, err = _call(torch, plain, *args)
    assert err == [0, 0] and torch.equal(again, want) and torch.equal(again_lse, want_lse)
