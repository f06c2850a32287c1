"""Attention with keys of their own length and a bias by relative position, from the definition in
64 bits on the CPU, with the bounds that the rounding of the kernels' operands allows."""
import math

import numpy as np
import torch

import oracle

F64 = torch.float64
HALF = 2.0 ** -8  # half a step of bf16, relative to the value


def bucket(rule, distance):
    """Row of the table for a distance (key minus query): rule = (num_buckets, max_distance, both)."""
    nb, far, both = rule
    half = nb // 2 if both else nb
    n = abs(distance) if both else max(0, -distance)
    e = half // 2
    b = n
    if n >= e:
        # floor(log(n / e) / log(far / e) * (half - e)) without rounding: n^E against far^t e^(E-t)
        E, t = half - e, 0
        while t + 1 < E and n ** E >= far ** (t + 1) * e ** (E - t - 1):
            t += 1
        b = e + t
    return b + half if both and distance > 0 else b


def keep_bits(B, H, Nq, Nk, p, seed, offset):
    """Dropout keep mask [B, H, Nq, Nk], from the Philox stream that include/fa.h defines."""
    p8 = oracle.p8(p)
    keep = np.zeros((B * H * Nq, (Nk + 15) // 16 * 16), dtype=np.uint8)
    key = (seed & 0xFFFFFFFF, seed >> 32)
    for row in range(B * H * Nq):
        for g in range(keep.shape[1] // 16):
            w = oracle.philox4x32_10((g, row, offset & 0xFFFFFFFF, offset >> 32), key)
            keep[row, 16 * g:16 * g + 16] = w.astype("<u4").view(np.uint8) >= p8
    return torch.from_numpy(keep[:, :Nk].reshape(B, H, Nq, Nk).astype(np.float64))


def plain(q, k, v, do=None, scale=None, causal=False, q_offset=0, window=(-1, -1), lens=None,
          bias=None, keep=None, p8=0, starts=None, exact_d=False):
    """q, do [B, H, Nq, d], k, v [B, H_kv, Nk, d] (any type), lens: list of key lengths or None,
    bias(h, distances) -> biases, starts: positions of the first queries instead of q_offset,
    exact_d: the bounds leave out what a D from the rounded O costs.
    Returns o, lse, (dq, dk, dv, S's gradient), and the bounds of the kernels' errors by name."""
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    G = H // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    z = lambda *s: torch.zeros(s, dtype=F64)
    out = {"o": z(B, H, Nq, d), "lse": torch.full((B, H, Nq), -math.inf, dtype=F64)}
    tol = {"o": z(B, H, Nq, d)}
    if do is not None:
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            out[n], tol[n] = z(*x.shape), z(*x.shape)
        out["ds"], tol["ds"] = z(B, H, Nq, Nk), z(B, H, Nq, Nk)
    j = torch.arange(Nk)[None]
    for b in range(B):
        L = Nk if lens is None else min(max(int(lens[b]), 0), Nk)
        pos = torch.arange(Nq)[:, None] + (q_offset if starts is None else starts[b])
        see = (j < L).expand(Nq, Nk)
        if causal:
            see = see & (j <= pos)
        if window[0] >= 0:
            see = see & (j >= pos - window[0])
        if window[1] >= 0:
            see = see & (j <= pos + window[1])
        for h in range(H):
            qh, kh, vh = q[b, h].to(F64), k[b, h // G].to(F64), v[b, h // G].to(F64)
            kh = torch.where((j < L).T, kh, torch.zeros((), dtype=F64))  # the padding counts for
            vh = torch.where((j < L).T, vh, torch.zeros((), dtype=F64))  # nothing, NaN included
            s = scale * (qh @ kh.T)
            if bias is not None:
                s = s + bias(h, j - pos)
            s = torch.where(see, s, torch.tensor(-math.inf, dtype=F64))
            lse = torch.logsumexp(s, 1)
            out["lse"][b, h] = lse
            P = torch.where(see, torch.exp(s - lse[:, None]), torch.zeros((), dtype=F64))
            P = torch.nan_to_num(P)
            Z = torch.ones_like(P) if keep is None else keep[b, h] / (1.0 - p8 / 256.0)
            o = (P * Z) @ vh
            out["o"][b, h] = o
            # weights rounded to bf16, and the output
            tol["o"][b, h] = HALF * ((P * Z) @ vh.abs() + o.abs())
            if do is None:
                continue
            g = do[b, h].to(F64)
            D = (g * o).sum(1, keepdim=True)
            dP = Z * (g @ vh.T)
            dS = P * (dP - D)
            # D comes from the rounded O; what it costs dS, and dS's own rounding
            e = HALF * dS.abs()
            if exact_d:  # fp32: the scores' error (see table_grad), and D's sum
                e = e + 2.0 ** -17 * P * (dP.abs() + (P * dP.abs()).sum(1, keepdim=True))
            else:
                e = e + HALF * (g * o).abs().sum(1, keepdim=True) * P
            out["ds"][b, h], tol["ds"][b, h] = dS, P * (dP.abs() + D.abs())
            out["dv"][b, h // G] += (P * Z).T @ g
            tol["dv"][b, h // G] += HALF * ((P * Z).T @ g.abs())
            out["dq"][b, h] = scale * (dS @ kh)
            tol["dq"][b, h] = scale * (e @ kh.abs())
            out["dk"][b, h // G] += scale * (dS.T @ qh)
            tol["dk"][b, h // G] += scale * (e.T @ qh.abs())
    for n in tol:
        if n in ("dq", "dk", "dv"):
            tol[n] += HALF * out[n].abs()
    return out, tol


def table_grad(out, tol, rule_row, rows, pos):
    """Gradient [rows, H] of a bias table from S's gradient: rule_row(distance) is the row of a
    distance, pos [B, Nq] the queries' positions. And a bound: the weights' relative error is that
    of the scores, which fp32 sums of products, the exponent's rounding and exp2's own error
    keep below 2^-17 at these sizes (|s| < 2^5, d <= 128: 8 partial sums of 2^-23 of at most 2^4
    each, 2^-24 of 2^5 for the exponent and lse, 2^-22 for exp2)."""
    ds, size = out["ds"], tol["ds"]
    B, H, Nq, Nk = ds.shape
    grad, bound = torch.zeros((rows, H), dtype=F64), torch.zeros((rows, H), dtype=F64)
    for b in range(B):
        row = torch.tensor([[rule_row(j - int(p)) for j in range(Nk)] for p in pos[b]])
        for h in range(H):
            grad[:, h].index_add_(0, row.flatten(), ds[b, h].flatten())
            bound[:, h].index_add_(0, row.flatten(), size[b, h].flatten())
    return grad, 2.0 ** -17 * bound + 1e-7


def within(name, got, want, bound, slack=2.0 ** -9):
    """|got - want| <= bound, with `slack` of it for what fp32 adds to the operands' rounding."""
    got = got.detach().to("cpu", F64)
    assert got.shape == want.shape, name
    assert torch.isfinite(got).all(), name
    over = (got - want).abs() - (bound * (1 + slack) + 2.0 ** -18)
    assert over.max() <= 0, f"{name}: off by {over.max()} more than allowed"
