"""The prompt kernel's waits, made to run out in a build of its own in which their limit
is a variable: the call still ends, reports it, and writes whole right rows or none."""
import ctypes
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu

TIMEOUT, SITE = 4, 4
LEFT = 77.0


@pytest.fixture(scope="module")
def torch():
    import torch as t
    return t


@pytest.fixture(scope="module")
def libs(tmp_path_factory):
    """The library, and the prompt kernel with the variable."""
    import hierarchical_sparse_kv_int8_gb300 as dhs
    from hierarchical_sparse_kv_int8_gb300 import _build as b
    other = os.path.join(b.OUT_DIR, "k_page_attn.o")
    dhs.build()
    if not os.path.exists(other):
        b.build(force=True)
    d = tmp_path_factory.mktemp("waits")
    obj, so = str(d / "k_prompt.o"), str(d / "libwaits.so")
    subprocess.run([b._nvcc(), *b.ARCH, *b.NVCC_FLAGS, "-DDHS_TEST_WAITS", "-c",
                    os.path.join(b.CSRC, "k_prompt.cu"), "-o", obj], check=True, capture_output=True)
    subprocess.run([b._nvcc(), *b.ARCH, "-shared", "-o", so, obj, other, "-lcudart"], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(so)
    from hierarchical_sparse_kv_int8_gb300 import _SIGS
    for name in ("dhs_prompt_attend", "dhs_prompt_attend_workspace"):
        f = getattr(lib, name)
        f.argtypes, f.restype = _SIGS[name]
    return dhs.load(), lib, ctypes.c_uint32.in_dll(lib, "dhs_prompt_wait_us")


def _call(torch, lib, x, hq, hkv, d):
    q, k, v, cq, ck, n = x
    out = torch.full_like(q, LEFT)
    lse = torch.full((q.shape[0], hq), LEFT, device="cuda")
    err = torch.zeros(2, dtype=torch.int32, device="cuda")
    nbytes = lib.dhs_prompt_attend_workspace(q.shape[0], k.shape[0], n, hq, hkv, d)
    # what a workspace holds before a call does not matter
    ws = torch.randint(0, 256, (max(16, nbytes),), dtype=torch.uint8, device="cuda")
    rc = lib.dhs_prompt_attend(q.data_ptr(), k.data_ptr(), v.data_ptr(), None, q.shape[0], k.shape[0],
                               cq.data_ptr(), ck.data_ptr(), n, hq, hkv, d, 0.0, out.data_ptr(),
                               lse.data_ptr(), ws.data_ptr(), nbytes, err.data_ptr(),
                               torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0
    return out, lse, err.tolist(), nbytes > 0


# Whole prompts, many items a CTA; one row tile only (few tokens, many heads); chunks whose
# keys are split and joined.  A poll is suspended for some 5 us at most: with `long`, items
# of tens of tiles, some waits outlast several and a limit of zero is sure to run out.
CASES = [([700, 33, 2100], [700, 33, 2100], 16, 4, 128, True), ([3, 900], [2000, 900], 64, 32, 64, True),
         ([40, 5], [9000, 3000], 8, 2, 128, False), ([300], [12000], 4, 1, 64, False),
         ([1], [16384], 160, 160, 64, True)]


@pytest.mark.parametrize("lq,lk,hq,hkv,d,long", CASES)
def test_waits_that_run_out_leave_rows_out(torch, libs, lq, lk, hq, hkv, d, long):
    plain, lib, wait_us = libs
    g = torch.Generator().manual_seed(3)
    cu = [torch.tensor([0] + x).cumsum(0).int().cuda() for x in (lq, lk)]
    q, k, v = (torch.randn((sum(t), h, d), generator=g).bfloat16().cuda()
               for t, h in ((lq, hq), (lk, hkv), (lk, hkv)))
    x = (q, k, v, *cu, len(lq))
    want, want_lse, err, split = _call(torch, plain, x, hq, hkv, d)
    assert err == [0, 0] and not (want == LEFT).any()
    assert split == (sum(lk) > 4 * sum(lq))  # the last three cases are the ones with a join
    ran_out = 0
    # from less than the first copies take to more than the call does, in microseconds
    for limit in [0, 0] + list(range(1, 30, 2)) + [40, 60, 100, 150, 2000000]:
        wait_us.value = limit
        out, lse, err, _ = _call(torch, lib, x, hq, hkv, d)
        assert err in ([0, 0], [TIMEOUT, SITE])
        left = (out == LEFT).all(-1)
        assert torch.equal(left, lse == LEFT)
        assert torch.equal(out[~left], want[~left]) and torch.equal(lse[~left], want_lse[~left])
        if err == [0, 0]:
            assert not left.any()
        else:
            ran_out += 1
            assert left.all() or not split       # a join writes every row or none
        if limit == 0 and long:
            assert err == [TIMEOUT, SITE]
    assert (ran_out >= 2 or not long) and err == [0, 0]
    # the GPU is as it was: the library's own kernel gives what it gave
    again, again_lse, err, _ = _call(torch, plain, x, hq, hkv, d)
    assert err == [0, 0] and torch.equal(again, want) and torch.equal(again_lse, want_lse)
