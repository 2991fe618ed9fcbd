"""The bounded-wait failure path of the paged attention kernels: with the wait
limit at 0 ns the first wait that is not satisfied gives up, the status says so,
and the same call then runs normally (see test_gpu_wait_abort.py)."""

import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
from tests import test_gpu_paged as TP

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def C(cuda_device):
    from compressed_sparse_long_compress_b200 import cslc
    return cslc


@pytest.fixture(autouse=True)
def _restore_limits(cuda_device):
    yield
    from compressed_sparse_long_compress_b200 import cslc
    cslc.testing_set_wait_limits(cslc.WAIT_LIMIT_NS_DEFAULT, cslc.WAIT_SLEEP_NS_DEFAULT)


def _aborts(C, run, name):
    C.testing_set_wait_limits(0, 0)
    run()
    with pytest.raises(C.CslcError) as ei:
        C.sync_status()
    assert ei.value.status == 7 and "timed out" in str(ei.value) and name in str(ei.value)
    C.testing_set_wait_limits(C.WAIT_LIMIT_NS_DEFAULT, C.WAIT_SLEEP_NS_DEFAULT)


@pytest.mark.parametrize("H", [8, 16])
def test_decode_wait_abort_then_recovers(C, H):
    cache = TP.make_cache(700, 1, 64, 5)
    table = TP.i32(np.random.RandomState(3).randint(0, 700, (6, 100)))
    lens = [6400, 3000, 1, 0, 5000, 777]
    q, n = TP.randn((6, H, 128), 8), TP.i32(lens)
    run = lambda: C.page_decode_attn(q, *cache, table, n, TP.SCALE, lse=True)  # noqa: E731
    _aborts(C, run, "cslc_page_decode_attn")
    out, lse = run()
    C.sync_status()
    kc, vc, ks, vs = (x.cpu().numpy() for x in cache)
    ref = PO.page_decode_attention(TP.f64(q), kc, vc, ks.astype(float), vs.astype(float), table.cpu().numpy(), lens, TP.SCALE)
    TP.check_attention(out, lse, ref, max(lens), "decode after an abort")


def test_prompt_wait_abort_then_recovers(C):
    q, k, v = TP.randn((3000, 8, 128), 1), TP.randn((3000, 2, 128), 2), TP.randn((3000, 2, 128), 3)
    cu = [0, 1700, 3000]
    run = lambda: C.prompt_attn(q, k, v, TP.i32(cu), TP.i32(cu), TP.SCALE, lse=True)  # noqa: E731
    _aborts(C, run, "cslc_prompt_attn")
    out, lse = run()
    C.sync_status()
    ref = PO.prompt_attention(TP.f64(q), TP.f64(k), TP.f64(v), cu, cu, TP.SCALE, rows={0, 5, 1699, 1700, 1701, 2999})
    TP.check_attention(out, lse, ref, 1700, "prompt after an abort")


@pytest.mark.parametrize("limit_ns", [0, 100, 400, 1500, 6000, 25000])
def test_prompt_waits_that_run_out_at_any_time(C, limit_ns):
    """Limits in the range of the kernel's own waits: some run out, in any role, each call ends, and the next ones
    with the usual limit have the bits of before."""
    q, k, v = TP.randn((4000, 8, 128), 1), TP.randn((4000, 2, 128), 2), TP.randn((4000, 2, 128), 3)
    v[::300, 1] = math.nan                                    # products on the CUDA cores, too
    cu = TP.i32([0, 1700, 1810, 1811, 3000, 4000])
    want = C.prompt_attn(q, k, v, cu, cu, TP.SCALE, 500, lse=True)
    C.sync_status()
    C.testing_set_wait_limits(limit_ns, 0)
    for _ in range(10):
        C.prompt_attn(q, k, v, cu, cu, TP.SCALE, 500, lse=True)
        try:
            C.sync_status()
        except C.CslcError as e:
            assert e.status == 7 and "cslc_prompt_attn" in str(e)
    C.testing_set_wait_limits(C.WAIT_LIMIT_NS_DEFAULT, C.WAIT_SLEEP_NS_DEFAULT)
    got = C.prompt_attn(q, k, v, cu, cu, TP.SCALE, 500, lse=True)
    C.sync_status()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("H,limit_ns", [(8, 0), (8, 300), (16, 1000), (8, 4000), (16, 20000)])
def test_decode_waits_that_run_out_at_any_time(C, H, limit_ns):
    """As above for the paged decode: units that cross CTAs, pages of 16, and short units of one CTA each."""
    cache = TP.make_cache(500, 2, 16, 5)
    table = TP.i32(np.random.RandomState(3).randint(0, 500, (70, 120)))
    q, n = TP.randn((70, 2 * H, 128), 8), TP.i32(np.random.RandomState(4).randint(0, 1921, 70))
    run = lambda: [C.page_decode_attn(q, *cache, table, n, TP.SCALE, w, lse=True) for w in (0, 200)]  # noqa: E731
    want = run()
    C.sync_status()
    C.testing_set_wait_limits(limit_ns, 0)
    for _ in range(10):
        run()
        try:
            C.sync_status()
        except C.CslcError as e:
            assert e.status == 7 and "cslc_page_decode_attn" in str(e)
    C.testing_set_wait_limits(C.WAIT_LIMIT_NS_DEFAULT, C.WAIT_SLEEP_NS_DEFAULT)
    got = run()
    C.sync_status()
    for x, y in zip(got, want):
        for a, b in zip(x, y):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
