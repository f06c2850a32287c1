"""The bounded waits of attention with keys of its own length and of the decode step with a bias:
a launch that waits for what nothing completes gives up, says so, and the next call is right. (The
wait is made to run out from the host; nothing faults or hangs.)"""
import pytest
import torch

import io_aware_exact_07_gb300 as fa
from _cross import bucket, plain, within

pytestmark = pytest.mark.gpu

RULE = (32, 128, True)


def _inputs(d, rel, G=1):
    g = torch.Generator().manual_seed(d + rel)
    x = [torch.randn(s, generator=g).to(torch.bfloat16)
         for s in ((1, 2 * G, 200, d), (1, 2, 300, d), (1, 2, 300, d), (1, 2 * G, 200, d))]
    table = torch.randn((RULE[0], 2 * G), generator=g) if rel else None
    return x, table


def _bias(table):
    if table is None:
        return None, None

    def of(h, away):
        rows = torch.tensor([[bucket(RULE, int(a)) for a in r] for r in away.tolist()])
        return table[rows, h].double()
    return fa.rel_bias(table.cuda(), fa.rel_buckets(*RULE)), of


def _stalled(mode, call):
    fa.fa_device_status(clear=True)
    fa.fa_set_wait_timeout_ns(200_000_000)
    try:
        fa.fa_test_inject_stall(mode)
        call()
        return fa.fa_device_status(clear=True)
    finally:
        fa.fa_test_inject_stall(0)
        fa.fa_set_wait_timeout_ns(4_000_000_000)


@pytest.mark.parametrize("rel", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mode", [1, 2, 3])
def test_a_stalled_launch_times_out_and_the_next_call_is_right(mode, d, rel):
    (q, k, v, do), table = _inputs(d, rel)
    gpu = [t.cuda() for t in (q, k, v, do)]
    bias, of = _bias(table)

    def run():
        o, lse = fa.fwd(*gpu[:3], q_offset=50, rel_bias=bias)
        return (o, lse) + tuple(fa.bwd(*gpu[:3], o, gpu[3], lse, q_offset=50, rel_bias=bias))
    assert _stalled(mode, run) == fa.FA_ERR_TIMEOUT
    got = run()
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_OK
    ref, tol = plain(q, k, v, do, q_offset=50, bias=of)
    for n, x in zip(("o", "lse", "dq", "dk", "dv"), got):
        if n != "lse":
            within(n, x, ref[n], tol[n])


@pytest.mark.parametrize("d", [64, 128])
def test_a_stalled_step_times_out_and_the_next_call_is_right(d):
    """Enough query rows per K/V head for the kernel of 128-row tiles, whose waits are bounded."""
    (q, k, v, _), table = _inputs(d, True, G=4)
    q = q[:, :, :6].contiguous()
    bias, of = _bias(table)
    run = lambda: fa.decode(q.cuda(), k.cuda(), v.cuda(), causal=True, rel_bias=bias, num_ctas=3)
    assert _stalled(1, run) == fa.FA_ERR_TIMEOUT
    o, lse = run()
    torch.cuda.synchronize()
    assert fa.fa_device_status(clear=True) == fa.FA_OK
    ref, tol = plain(q, k, v, causal=True, starts=[294], bias=of)
    within("o", o, ref["o"], tol["o"])


def test_a_hook_for_dq_is_not_taken_by_the_other_launches():
    (q, k, v, do), table = _inputs(64, True)
    gpu = [t.cuda() for t in (q, k, v, do)]
    bias, _ = _bias(table)
    fa.fa_device_status(clear=True)
    fa.fa_set_wait_timeout_ns(200_000_000)
    try:
        fa.fa_test_inject_stall(3)
        o, lse = fa.fwd(*gpu[:3], rel_bias=bias)
        assert fa.fa_device_status(clear=True) == fa.FA_OK
        fa.bwd(*gpu[:3], o, gpu[3], lse, rel_bias=bias)
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_TIMEOUT
    finally:
        fa.fa_test_inject_stall(0)
        fa.fa_set_wait_timeout_ns(4_000_000_000)
