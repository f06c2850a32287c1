"""Shared helpers of the paged-cache tests: a batch of sequences in a pool of pages, and
what the oracle says about it."""
import math

import numpy as np
import torch

import oracle

U = 2.0 ** -8  # half a step of bf16, relative to the value


class Batch:
    """Sequences of given lengths whose last nq[b] tokens are new, in a pool filled with
    `garbage` where no sequence has written. Tensors are on the CPU; on(dev) moves them."""

    def __init__(self, nq, kv, page, Hkv, d, e4m3=False, G=1, seed=0, spare=2, layout="head",
                 garbage=1.0, extra_rows=0, table_pad=0):
        g = torch.Generator().manual_seed(seed)
        self.nq, self.kv, self.page, self.Hkv, self.d, self.G = nq, kv, page, Hkv, d, G
        self.e4m3, self.B, self.H = e4m3, len(nq), Hkv * G
        self.cu = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
        self.T = int(self.cu[-1]) + extra_rows
        count = [-(-n // page) for n in kv]
        self.P = sum(count) + spare
        order = torch.randperm(self.P, generator=g).to(torch.int32)
        width = max(max(count), 1)
        table = torch.full((self.B, width + table_pad), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(count):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table[:, :width]
        bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
        self.q = bf(self.T, self.H, d)
        self.rows = {n: [bf(L, Hkv, d) for L in kv] for n in "kv"}  # whole sequences
        self.new = {n: torch.full((self.T, Hkv, d), 3.0, dtype=torch.bfloat16) for n in "kv"}
        for n in "kv":
            for b in range(self.B):
                m = min(nq[b], kv[b])  # tokens at negative positions have no row
                if m:
                    self.new[n][self.cu[b + 1] - m:self.cu[b + 1]] = self.rows[n][b][kv[b] - m:]
        shape = (self.P, Hkv, page, d)
        dtype = torch.uint8 if e4m3 else torch.bfloat16
        self.pages = {n: torch.full(shape, 0x7E if e4m3 else garbage, dtype=dtype) for n in "kv"}
        self.scale = {n: torch.full(shape[:3], 255 if math.isnan(garbage) else 133,
                                    dtype=torch.uint8) if e4m3 else None
                      for n in "kv"}
        self.layout = layout

    def stored(self, n, b):
        """Rows of sequence b as the cache holds them, [L, Hkv, d] fp64."""
        x = self.rows[n][b].double().numpy()
        return oracle.dequantize_rows(*oracle.quantize_rows(x)) if self.e4m3 else x

    def fill(self, upto=None):
        """Put positions 0 .. upto[b] - 1 of every sequence into the pages (host)."""
        for n in "kv":
            for b in range(self.B):
                L = self.kv[b] if upto is None else upto[b]
                if L == 0:
                    continue
                at, row = oracle.paged_positions(self.table.numpy(), self.page, b, np.arange(L))
                x = self.rows[n][b][:L]
                if self.e4m3:
                    x, s = oracle.quantize_rows(x.double().numpy())
                    self.scale[n][at, :, row] = torch.from_numpy(s)
                    x = torch.from_numpy(x)
                self.pages[n][at, :, row] = x
        return self

    def laid_out(self, x):
        """Pages [P, Hkv, page, d] in another order in memory, same indexing."""
        if self.layout == "row":  # [P, page, Hkv, d] in memory
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        return x.contiguous()

    def on(self, dev):
        c = type("OnDevice", (), {})()
        if self.layout == "pair":  # K and V of a page next to each other
            both = torch.stack([self.pages["k"], self.pages["v"]], 1).to(dev)
            c.k, c.v = both[:, 0], both[:, 1]
        else:
            c.k, c.v = (self.laid_out(self.pages[n].to(dev)) for n in "kv")
        c.sc = {f"{n}_scale": None if self.scale[n] is None else self.scale[n].to(dev)
                for n in "kv"}
        c.table = self.table.to(dev) if self.table.is_contiguous() else \
            torch.nn.functional.pad(self.table, (0, 3)).to(dev)[:, :self.table.shape[1]]
        c.kv = torch.tensor(self.kv, dtype=torch.int32, device=dev)
        c.cu = torch.from_numpy(self.cu).to(dev)
        c.q, c.k_new, c.v_new = self.q.to(dev), self.new["k"].to(dev), self.new["v"].to(dev)
        return c

    def oracle(self, causal, window_left=-1, scale=None):
        k, v = ([self.stored(n, b) for b in range(self.B)] for n in "kv")
        return oracle.fwd_paged(self.q.double().numpy(), k, v, self.cu, self.kv,
                                scale or 1.0 / math.sqrt(self.d), causal, window_left)


def check_attn(o, lse, ref, rows=None):
    """O within the roundings of P and of O to bf16, each at most 2^-8 of the value: an
    element is off by at most 2^-8 sum_j P_ij |v_j| + 2^-8 |O_ij|, and by what scores and
    exponentials in fp32 add. lse, fp32: a score is a sum of d products, off by at most about
    d 2^-24 scale sum |q k| < 1.3e-4 at d = 128 for normal inputs (scale sum |q k| < 16); the
    sum and the logarithm add less than 2^-20 each: 2e-4 in all, which as a relative error of
    P is 5 % of 2^-8, so O gets that much more. Rows without keys are exact."""
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    o_ref, lse_ref, o_abs = ref
    if rows is not None:
        o, lse, o_ref, lse_ref, o_abs = o[:rows], lse[:rows], o_ref[:rows], lse_ref[:rows], \
            o_abs[:rows]
    empty = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(lse), empty), "rows without keys differ"
    assert np.all(o[empty] == 0)
    tol = 1.05 * U * (o_abs + np.abs(o_ref)) + 1e-30
    assert np.all(np.isfinite(o))
    excess = np.abs(o - o_ref) / tol
    assert excess.max(initial=0) <= 1, f"O error is {excess.max()} of its bound"
    if (~empty).any():
        err = np.abs(lse[~empty] - lse_ref[~empty]).max()
        assert err <= 2e-4, f"lse error {err}"
