"""Failure detection on the GPU without a fault: device-side waits that nothing satisfies
give up after their limit, report HYB_DEVERR_TIMEOUT through the device status word, and
leave the context usable for the next call."""
import time

import numpy as np
import pytest
import torch

import oracle
import workloads as W
from gpu_helpers import assert_out_close, assert_states_close, empty_rows, to_dev, to_host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_us", [2000, 50000])
def test_bounded_waits_expire_report_and_return(hyb, devstatus, limit_us):
    t0 = time.perf_counter()
    hyb.check(hyb.hyb_selftest_bounded_waits(limit_us))
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    st, flags = hyb.hyb_device_status(clear=True)
    assert st == hyb.HYB_ERR_DEVICE_CHECK
    assert flags == hyb.HYB_DEVERR_TIMEOUT
    assert took >= limit_us * 1e-6                   # the waits ran to their limit ...
    assert took < limit_us * 1e-6 + 5.0              # ... and then returned

    # the context is still usable: a linear decode step runs and matches the oracle
    g = W.rng(5)
    B, H, D, NS = 3, 4, 64, 5
    q, k, v = (W.rows(g, (B, H, D), D, W.BF16) for _ in range(3))
    pool = W.synthetic_state(g, NS, H, D, np.full(NS, 100))
    slots = np.array([4, 0, 2], np.int32)
    o_ref, s_ref = oracle.linear_step(q, k, v, pool, slots)
    pool_d = to_dev(pool)
    out = empty_rows((B, H, D), W.BF16)
    hyb.check(hyb.hyb_linear_attn_step(out, to_dev(q), to_dev(k), to_dev(v), pool_d, NS, to_dev(slots),
                                       B, H, D, W.BF16))
    torch.cuda.synchronize()
    assert_out_close(out, o_ref, "linear step after the self-test")
    assert_states_close(to_host(pool_d)[slots], s_ref, "states after the self-test")
    assert devstatus() == (0, 0)


def test_gated_delta_prefill_after_expired_waits(hyb, devstatus):
    """The waits of the gated delta prefill (barriers by the SM's clock, the handoff of a cut chain)
    are among the self-test's: after they ran out, a call that cuts chains gives the same bits as
    before."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B, H, D, n = sms // 2 + 1, 2, 128, 130
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (torch.randn(B * n, H, D, generator=gen, device="cuda").bfloat16() for _ in range(3))
    g = -torch.rand(B * n, H, generator=gen, device="cuda")
    beta = torch.rand(B * n, H, generator=gen, device="cuda")
    start = torch.randn(B, H, D, D, generator=gen, device="cuda")
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    d = hyb.delta_dims(H, H, D, qk_norm_eps=1e-6)
    ws = torch.empty(hyb.hyb_gated_delta_chunked_prefill_workspace_size(B, B * n, d), dtype=torch.uint8, device="cuda")

    def call():
        out, pool = torch.empty_like(v), start.clone()
        hyb.check(hyb.hyb_gated_delta_chunked_prefill(out, q, k, v, g, beta, cu, pool, B, slots, None, B, B * n, n, d, ws, ws.numel()))
        torch.cuda.synchronize()
        return out, pool

    before = call()
    assert devstatus() == (0, 0)
    hyb.check(hyb.hyb_selftest_bounded_waits(1000))
    assert devstatus() == (hyb.HYB_ERR_DEVICE_CHECK, hyb.HYB_DEVERR_TIMEOUT)
    after = call()
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert devstatus() == (0, 0)
