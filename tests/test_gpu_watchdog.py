"""Failure detection without a GPU fault: the test hook makes the forward
producer skip one K tile, so the MMA thread's wait can never be satisfied.
The bounded wait must run out, the CTA must drain and exit, the host must
read FA_ERR_TIMEOUT, and the context must stay usable."""

import pytest
import torch

import oracle
from exact_io_aware_56_b200 import fa, to_f64

from .parity import assert_close_abs, assert_close_lse, gpu_inputs, run_fwd

pytestmark = pytest.mark.gpu


def test_forward_wait_times_out_cleanly_and_context_recovers():
    dev, ref = gpu_inputs(1, 2, 2, 300, 64, seed=21, with_dout=False)
    o = torch.empty_like(dev["q"])
    lse = torch.empty((1, 2, 300), dtype=torch.float32, device="cuda")
    assert fa.fa_check_device_error() == fa.FA_OK
    fa.fa_set_watchdog_ns(50_000_000)
    fa.fa_test_set_fault(1)
    try:
        fa.fa_fwd(dev["q"], dev["k"], dev["v"], o, lse, False, 0.125)
        assert fa.fa_check_device_error() == fa.FA_ERR_TIMEOUT
        # The word was cleared by the read.
        assert fa.fa_check_device_error() == fa.FA_OK
    finally:
        fa.fa_test_set_fault(0)
        fa.fa_set_watchdog_ns(2_000_000_000)
    out, l2 = run_fwd(dev, False, 0.125)
    O, L = oracle.attn_fwd_ref(ref["q"], ref["k"], ref["v"], False, 0.125)
    assert_close_abs("O", to_f64(out), O)
    assert_close_lse(to_f64(l2), L)


@pytest.mark.parametrize("code,new,d", [(2, 150, 64), (2, 150, 128), (3, 2, 64), (3, 2, 128)])
def test_paged_waits_time_out_cleanly_and_context_recovers(code, new, d):
    import numpy as np

    from .packed import Cache, assert_forward, normal, offsets

    cache = Cache(23, [300, 700], 16, 2, d)
    kp, vp, table, ln = cache.cuda()
    q = normal(24, 2 * new, 4, d)
    args = (q.cuda(), kp, vp, table, ln, torch.from_numpy(offsets([new, new])).cuda(), new, True, 0.125)
    assert fa.fa_check_device_error() == fa.FA_OK
    fa.fa_set_watchdog_ns(50_000_000)
    fa.fa_test_set_fault(code)
    try:
        fa.attention_paged(*args)
        assert fa.fa_check_device_error() == fa.FA_ERR_TIMEOUT
        assert fa.fa_check_device_error() == fa.FA_OK
    finally:
        fa.fa_test_set_fault(0)
        fa.fa_set_watchdog_ns(2_000_000_000)
    o, lse = fa.attention_paged(*args)
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == fa.FA_OK
    assert_forward(o, lse, *oracle.paged_ref(to_f64(q), to_f64(cache.k), to_f64(cache.v), cache.table,
                                             np.asarray(cache.lens), offsets([new, new]), True, 0.125))


def test_long_items_do_not_run_into_the_wait_limit():
    """The warps that wait for an item's end wait as long as its tiles take: 1024 tiles, over a millisecond."""
    from .packed import normal

    T = 128 * 1024 - 1
    q, k, v, dout = (normal(25 + i, T, 1, 64).cuda() for i in range(4))
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")

    def run():
        o, lse = fa.attention_packed_forward(q, k, v, cu, False)
        return o, lse, *fa.attention_packed_backward(q, k, v, o, dout, lse, cu, False)[1:]

    want = run()
    assert fa.fa_check_device_error() == fa.FA_OK
    fa.fa_set_watchdog_ns(1_000_000)
    try:
        got = run()
        assert fa.fa_check_device_error() == fa.FA_OK
    finally:
        fa.fa_set_watchdog_ns(2_000_000_000)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
