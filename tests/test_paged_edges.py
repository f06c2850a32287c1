"""Paged caches at the edges of what the calls take, on the GPU against the fp64 oracle."""
import numpy as np
import pytest
import torch

import io_aware_exact_07_gb300 as fa
from _paged import Batch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -8  # half a step of bf16, relative to the value


def sync():
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK


def attn(b, x, **kw):
    return fa.paged_attn(x.q, x.k, x.v, x.table, x.kv, cu_seqlens_q=x.cu, **x.sc, **kw)


# ------------------------------------------------------------------ scales by key tile

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,kv", [
    ([40] * 60, [300, 380, 257] * 20),               # pieces of 3 tiles, cut by the runs' ends
    ([33] * 40, [600, 130, 890, 100] * 10),          # 5, 2, 7 and 1 tiles
    ([200] * 9, [1100, 640, 333] * 3),               # rounds of whole units
])
def test_scales_that_differ_from_tile_to_tile(nq, kv, d):
    # every 128 keys the scales of K and of V change by up to 2^6 and 2^12, so that a tile that
    # took another one's would be far off. Within a tile they are alike, so that the f16 tiles
    # are exact; P's rounding to f16 adds 2^-32 of the row's largest weight times value scale,
    # once a key.
    b = Batch(nq, kv, 32, 2, d, True, G=2, seed=51)
    g = torch.Generator().manual_seed(51)
    for i, L in enumerate(kv):
        for n, lo, hi in (("k", -6, 1), ("v", -10, 3)):
            e = torch.randint(lo, hi, (-(-L // 128), 1, 1), generator=g).repeat_interleave(128, 0)
            b.rows[n][i] = (b.rows[n][i].float() * torch.exp2(e[:L].float())).to(torch.bfloat16)
    x = b.fill().on(DEV)
    o_ref, lse_ref, o_abs = b.oracle(True)
    tol = 1.05 * U * (o_abs + np.abs(o_ref)) + max(kv) * 2.0 ** -32 * 448 * 2.0 ** -4
    assert int(b.scale["v"][b.scale["v"] != 133].max()) - 127 <= -4  # |V| < 28 = 448 * 2^-4
    for _ in range(5):
        o, lse = attn(b, x, causal=True, max_q=max(nq))
        sync()
        assert np.all(np.abs(o.double().cpu().numpy() - o_ref) <= tol)
        assert np.abs(lse.double().cpu().numpy() - lse_ref).max() <= 2e-4
