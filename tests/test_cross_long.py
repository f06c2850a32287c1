"""The gradient of a bias table over thousands of positions, with keys far to both sides of every query:
what corrects D for the rounding of O, the sums over far keys and the long sums by distance have to hold
there."""
import math

import pytest
import torch

import io_aware_exact_07_gb300 as fa
from _cross import bucket

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk,q_offset,length,causal", [
    (5000, 5000, 0, None, False), (3100, 6000, 1400, 5900, False), (4999, 4999, 0, None, True)])
def test_gradient_of_the_table_over_thousands_of_positions(Nq, Nk, q_offset, length, causal, d):
    H, rule = 2, (32, 128, not causal)
    g = torch.Generator(device="cuda").manual_seed(d + Nq)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    # V with a mean: O is large beside what tells keys apart, and so is what its rounding does to D
    q, k, v, do = (x.to(torch.bfloat16) for x in (r(1, H, Nq, d), r(1, 1, Nk, d),
                                                  r(1, 1, Nk, d) + 2, r(1, H, Nq, d)))
    table, b = r(32, H), fa.rel_buckets(*rule)
    lens = None if length is None else torch.tensor([length], dtype=torch.int32, device="cuda")
    kw = dict(causal=causal, q_offset=q_offset, seqlens_k=lens, rel_bias=fa.rel_bias(table, b))
    o, lse = fa.fwd(q, k, v, **kw)
    got = fa.bwd(q, k, v, o, do, lse, **kw)[3].double()
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK

    n = Nk if length is None else length
    row = torch.tensor([bucket(rule, x) for x in range(-Nq - q_offset, Nk + 1)], device="cuda")
    pos = torch.arange(Nq, device="cuda")[:, None] + q_offset
    j = torch.arange(n, device="cuda")[None]
    at = row[j - pos + Nq + q_offset]
    for h in range(H):
        kd, vd, gd = k[0, 0, :n].double(), v[0, 0, :n].double(), do[0, h].double()
        s = q[0, h].double() @ kd.T / math.sqrt(d) + table[:, h].double()[at]
        if causal:
            s = s.masked_fill(j > pos, -math.inf)
        p = s.softmax(1)
        dp = gd @ vd.T
        D = (p * dp).sum(1, keepdim=True)
        ds = p * (dp - D)
        by = lambda x: torch.zeros(32, dtype=torch.float64, device="cuda").index_add_(
            0, at.flatten(), x.flatten())
        rows = lambda x: torch.zeros((Nq, 32), dtype=torch.float64, device="cuda").scatter_add_(1, at, x)
        want = by(ds)
        # The errors of the rows, and of a row's weights among themselves, are independent roundings
        # to either side: by Hoeffding's bound the sum of such errors e exceeds 8 sqrt(sum of e^2)
        # with a probability below 2 exp(-32). They are
        # - a weight's own, 2^-17 of it (table_grad in _cross.py), times what it multiplies;
        # - the row's, of lse and D: 2^-20 (lse of at most 2^4 in 24 bits, and its exponent);
        # - the sums of a row, which the kernel keeps as one number each: N / 8 additions to a
        #   thread's accumulators, each off by 2^-24 of at most the row's sum of |dS|, and twice
        #   that for the difference that a far side is. They count by the row's weights in the bucket.
        a = p * (dp.abs() + D.abs())
        own = by((2.0 ** -17 * a) ** 2)
        common = ((2.0 ** -20 * rows(a)) ** 2).sum(0)
        steps = 2 * math.sqrt(n / 8) * 2.0 ** -24 * ds.abs().sum(1, keepdim=True)
        summed = ((steps * rows(p)) ** 2).sum(0)
        bound = 8 * (own.sqrt() + common.sqrt() + summed.sqrt()) + 1e-6
        off = (got[:, h] - want).abs()
        assert (off - bound).max() <= 0, (off.max(), bound[off.argmax()])
        # a D from the rounded O alone would not do
        rounded = by(p * (dp - (gd * o[0, h].double()).sum(1, keepdim=True)))
        assert ((rounded - want).abs() > bound).any()
