"""The operators over a paged key/value cache, as they are measured: writing new
tokens into the cache (bf16, or quantised to e4m3 as they are written), reading a
cache back into contiguous rows, and attention of new tokens (one per sequence, or
a chunk) over it.

``run`` computes them in plain torch operations, or with this package's calls where
``own`` is true. Every case holds a batch of sequences whose keys and values lie in
pages of ``page`` positions, scattered over a pool in random order; ``lens`` seeds the
lengths of the sequences, so that they belong to the case and not to the inputs.
"""
import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
SPARE_PAGES = 3      # pages of the pool that no sequence of the case holds
E_MIN, E_MAX = -117, 7  # exponents of the power-of-two scales of an e4m3 row


def _case(name, op, kind, B, Hkv, d, page, kv, q, lens, G=1, causal=True, window=-1):
    return {"name": name, "op": op, "type": kind, "B": B, "Hkv": Hkv, "G": G, "d": d,
            "page": page, "kv_min": kv[0], "kv_max": kv[1], "q_min": q[0], "q_max": q[1],
            "causal": causal, "window": window, "lens": lens}


def listed():
    return [
        # a decode step's write: one new token for each of 16 sequences; latency alone
        _case("write_step_bf16", "write", "bf16", 16, 8, 128, 16, (1, 4000), (1, 1), 1),
        # prompts of odd lengths enter a quantised cache in one call
        _case("write_prompts_e4m3", "write", "e4m3", 6, 8, 128, 64, (1500, 9000), (1500, 5200), 2),
        # a short bf16 cache is copied out of its pages, heads of 64
        _case("read_short_bf16", "read", "bf16", 3, 4, 64, 32, (1, 700), (1, 1), 3),
        # a ragged quantised batch is read back to bf16 rows, for the calls that take those
        _case("read_ragged_e4m3", "read", "e4m3", 16, 8, 128, 64, (100, 16384), (1, 1), 4),
        # a decode step of a few short sequences, one K/V head per query head: latency
        _case("step_short_d64", "attn", "bf16", 4, 16, 64, 16, (1, 500), (1, 1), 5),
        # the decode benchmark's shape (B=16 H=32 H_kv=8, 16384 keys) over pages
        _case("step_16k", "attn", "bf16", 16, 8, 128, 64, (16384, 16384), (1, 1), 6, G=4),
        # a ragged decode batch over a quantised cache
        _case("step_ragged_e4m3", "attn", "e4m3", 32, 8, 128, 64, (1, 32000), (1, 1), 7, G=4),
        # one user with a very long context: the keys of a head are spread over the GPU
        _case("step_long_one", "attn", "bf16", 1, 8, 128, 128, (131001, 131001), (1, 1), 8, G=4),
        # verification of drafted tokens: 5 new tokens of each sequence, heads of 64
        _case("draft_d64", "attn", "bf16", 24, 8, 64, 32, (300, 8192), (5, 5), 9, G=4),
        # prompts in chunks of 512 over what was cached before
        _case("chunk_512", "attn", "bf16", 4, 8, 128, 64, (2000, 8192), (512, 512), 10, G=4),
        # steps and chunks in one batch, quantised cache, sliding window
        _case("mixed_window_e4m3", "attn", "e4m3", 12, 8, 128, 16, (1, 12000), (1, 700), 11, G=4,
              window=4095),
        # the last chunk of long prompts
        _case("chunk_4096_long", "attn", "bf16", 2, 8, 128, 64, (16384, 16384), (4096, 4096), 12,
              G=4),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("write", "read", "attn", "attn"))
        kind = rng.choice(("bf16", "e4m3"))
        d = rng.choice((64, 128, 128))
        page = rng.choice((16, 32, 48, 64, 128, 256))
        Hkv = rng.choice((1, 2, 4, 8, 8, 16))
        G = rng.choice((1, 2, 3, 4, 4, 7, 8)) if op == "attn" else 1
        B = _log_uniform(rng, 1, 64)
        kv_max = _log_uniform(rng, 32, 65536)
        kv_min = rng.choice((1, kv_max // 2 + 1, kv_max))
        q_max = 1
        if op == "write" or (op == "attn" and rng.random() < 0.5):
            q_max = _log_uniform(rng, 1, min(kv_max, 4096))
        q_min = rng.choice((1, q_max))
        causal = rng.random() < 0.85
        window = _log_uniform(rng, 16, 8192) if op == "attn" and rng.random() < 0.25 else -1
        c = _case("", op, kind, B, Hkv, d, page, (kv_min, kv_max), (q_min, q_max),
                  rng.randrange(1 << 30), G, causal, window)
        del c["name"]
        if _cost(c) <= most and _pool_bytes(c) <= 6e9 and _scores(c) <= 4e9:
            return c


# ------------------------------------------------------------- the batch of a case

def _lengths(c):
    """New tokens and whole lengths (the new ones included) of the case's sequences."""
    r = random.Random(c["lens"])
    kv = [r.randint(c["kv_min"], c["kv_max"]) for _ in range(c["B"])]
    kv[r.randrange(c["B"])] = c["kv_max"]
    q = [min(r.randint(c["q_min"], c["q_max"]), n) for n in kv]
    return q, kv


def _pages(c):
    return [-(-n // c["page"]) for n in _lengths(c)[1]]


def _pool_bytes(c):
    one = 2 if c["type"] == "bf16" else 1
    return 2.0 * sum(_pages(c)) * c["page"] * c["Hkv"] * c["d"] * one


def _scores(c):
    q, kv = _lengths(c)
    return 1.0 * c["B"] * c["Hkv"] * c["G"] * max(q) * max(kv) if c["op"] == "attn" else 0.0


def _visible(c, n, L):
    """(keys that any of the n last positions sees, pairs of query and key it makes)."""
    pos = np.arange(L - n, L, dtype=np.int64)
    hi = pos + 1 if c["causal"] else np.full(n, L, dtype=np.int64)
    lo = np.maximum(0, pos - c["window"]) if c["window"] >= 0 else np.zeros(n, dtype=np.int64)
    return int(hi.max() - lo.min()), int(np.maximum(0, hi - lo).sum())


def work(case):
    c = case
    q, kv = _lengths(c)
    row = c["d"] * (2 if c["type"] == "bf16" else 1) + (c["type"] == "e4m3")  # a cached row
    T, new = sum(q), c["d"] * 2
    if c["op"] == "write":
        return {"bytes": 2 * T * c["Hkv"] * (new + row), "flops": 0}
    if c["op"] == "read":
        return {"bytes": 2 * c["Hkv"] * (sum(kv) * row + c["B"] * max(kv) * new), "flops": 0}
    keys, pairs = zip(*(_visible(c, n, L) for n, L in zip(q, kv)))
    H = c["Hkv"] * c["G"]
    return {"bytes": 2 * sum(keys) * c["Hkv"] * row + T * H * (2 * new + 4),
            "flops": 4 * c["d"] * H * sum(pairs)}


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


# ------------------------------------------------------------- inputs

def _power(e):
    """2^e in fp32 for whole e of -126 .. 127, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """e4m3 codes and scale bytes of rows [..., d]: the scale of a row is the smallest
    power of two, 2^E_MIN .. 2^E_MAX, that brings its largest magnitude to 448 or less
    (1 for a row of zeros), stored as exponent + 127."""
    x = x.float()
    top = x.abs().amax(-1)
    m, x2 = torch.frexp(top)
    e = (x2 - 9 + (m > 0.875).to(x2.dtype)).clamp(E_MIN, E_MAX)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    y = (x * _power(-e).unsqueeze(-1)).clamp(-448, 448)
    return y.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _rows(g, *shape):
    """Key or value rows: normal, with channels of unlike size."""
    x = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16)
    return x * torch.rand(shape[-1], generator=g, device=DEVICE).add(0.5).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))
    q, kv = _lengths(c)
    count = _pages(c)
    P, T = sum(count) + SPARE_PAGES, sum(q)
    s = {"case": c, "T": T, "q_max": max(q), "N": max(kv)}
    order = torch.randperm(P, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((c["B"], max(count)), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for b, n in enumerate(count):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=DEVICE)
    s["cu"] = torch.tensor([0] + list(np.cumsum(q)), dtype=torch.int32, device=DEVICE)
    shape = (P, c["Hkv"], c["page"], c["d"])
    for name in ("k", "v"):
        pages, scale = _rows(g, *shape), None
        if c["type"] == "e4m3":
            pages, scale = _quantise(pages)
        s[name], s[name + "_scale"] = pages, scale
    if c["op"] == "write":
        s["k_new"], s["v_new"] = (_rows(g, T, c["Hkv"], c["d"]) for _ in range(2))
    if c["op"] == "attn":
        s["q"] = torch.randn((T, c["Hkv"] * c["G"], c["d"]), generator=g, device=DEVICE,
                             dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------- plain forms

def _token_places(s):
    """Sequence, and position in it, of each new token: the last ones of the sequence."""
    t = torch.arange(s["T"], device=s["cu"].device)
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    b = torch.searchsorted(cu[1:], t, right=True)
    return b, kv[b] - (cu[b + 1] - t)


def _plain_write(s):
    page = s["case"]["page"]
    b, pos = _token_places(s)
    at = s["table"][b, pos // page].long()
    for name in ("k", "v"):
        x = s[name + "_new"]
        if s["case"]["type"] == "e4m3":
            x, scale = _quantise(x)
            s[name + "_scale"][at, :, pos % page] = scale
        s[name][at, :, pos % page] = x


def _plain_rows(s, name):
    """Cached rows [B, H_kv, positions, d] in fp32; what lies behind a sequence is zero."""
    pages = s["table"].clamp(min=0).long()
    x = s[name][pages]
    if s["case"]["type"] == "e4m3":
        e = s[name + "_scale"][pages].to(torch.int32) - 127
        x = x.view(torch.float8_e4m3fn).float() * _power(e).unsqueeze(-1)
    x = x.float().transpose(1, 2).flatten(2, 3)[:, :, :s["N"]]
    there = torch.arange(s["N"], device=x.device) < s["kv_lens"][:, None]
    return torch.where(there[:, None, :, None], x, torch.zeros((), device=x.device))


def _plain_attn(s):
    c = s["case"]
    B, Hkv, G, d, n = c["B"], c["Hkv"], c["G"], c["d"], s["q_max"]
    k, v = _plain_rows(s, "k"), _plain_rows(s, "v")
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    i = torch.arange(n, device=k.device)
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["T"] - 1)].float()  # [B, n, H, d]
    q = q.view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    pos = (kv - (cu[1:] - cu[:-1]))[:, None] + i  # [B, n]
    j = torch.arange(s["N"], device=k.device)
    seen = (j < kv[:, None])[:, None, :].expand(B, n, s["N"])
    if c["causal"]:
        seen = seen & (j <= pos[..., None])
    if c["window"] >= 0:
        seen = seen & (j >= pos[..., None] - c["window"])
    z = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(B, Hkv, n, G, s["N"])
    z.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, n * G, s["N"]) @ v).view(B, Hkv, n, G, d)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + l.log())[..., 0]
    b, at = _token_places(s)
    at = at - pos[b, 0]
    o = o.permute(0, 2, 1, 3, 4)[b, at].reshape(s["T"], Hkv * G, d)
    return o.to(torch.bfloat16), lse.permute(0, 2, 1, 3)[b, at].reshape(s["T"], Hkv * G)


# ------------------------------------------------------------- one pass

def _cache_outputs(s):
    if s["case"]["type"] == "bf16":
        return {"k": s["k"], "v": s["v"]}
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def run(state):
    s, c = state, state["case"]
    if own:
        import io_aware_exact_07_gb300 as fa
        scales = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
        if c["op"] == "write":
            fa.paged_write(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["kv_lens"],
                           cu_seqlens_q=s["cu"], **scales)
            return _cache_outputs(s)
        if c["op"] == "read":
            k, v = fa.paged_read(s["k"], s["v"], s["table"], s["kv_lens"], s["N"], **scales)
            return {"k": k, "v": v}
        o, lse = fa.paged_attn(s["q"], s["k"], s["v"], s["table"], s["kv_lens"],
                               cu_seqlens_q=s["cu"], max_q=s["q_max"], causal=c["causal"],
                               window_left=c["window"], **scales)
        return {"o": o, "lse": lse}
    if c["op"] == "write":
        _plain_write(s)
        return _cache_outputs(s)
    if c["op"] == "read":
        return {n: _plain_rows(s, n).to(torch.bfloat16) for n in ("k", "v")}
    o, lse = _plain_attn(s)
    return {"o": o, "lse": lse}


# ------------------------------------------------------------- the definition in 64 bits

def _exact_codes(x):
    """The e4m3 values of rows [..., d] and their scales' exponents, in 64 bits: steps of
    2^(floor(log2 |y|) - 3), at least 2^-9, halves to even, 448 at most."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 448).clamp(-2000, 2000)).clamp(E_MIN, E_MAX)
    e = torch.where((top <= 448 * torch.exp2(e - 1)) & (e > E_MIN), e - 1, e)
    e = torch.where((top > 448 * torch.exp2(e)) & (e < E_MAX), e + 1, e)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448), e[..., 0]


def _exact_table():
    """The values of the 256 e4m3 codes."""
    v = []
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        a = math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        v.append(math.nan if b & 127 == 127 else -a if b & 128 else a)
    return torch.tensor(v, dtype=torch.float64, device=DEVICE)


def _exact_sequence(s, name, b, L):
    """Row by row of the definition: position p of sequence b is slot p % page of the page
    that entry p // page of its table names. [L, H_kv, d]"""
    p = torch.arange(L, device=DEVICE)
    at, slot = s["table"][b].long()[p // s["case"]["page"]], p % s["case"]["page"]
    x = s[name][at, :, slot]
    if s["case"]["type"] == "bf16":
        return x.double()
    scale = s[name + "_scale"][at, :, slot].double() - 127
    return _exact_table()[x.long()] * torch.exp2(scale)[..., None]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    q, kv = _lengths(c)
    out = {}
    if c["op"] == "write":
        for name in ("k", "v"):
            e4m3 = c["type"] == "e4m3"
            pages = _exact_table()[s[name].long()] if e4m3 else s[name].double()
            t = 0
            for b, (n, L) in enumerate(zip(q, kv)):
                p = torch.arange(L - n, L, device=DEVICE)
                x = s[name + "_new"][t:t + n]
                x = _exact_codes(x)[0] if e4m3 else x.double()
                pages[s["table"][b].long()[p // c["page"]], :, p % c["page"]] = x
                t += n
            out[name] = pages
            if e4m3:
                out[name + "_scale"] = None
        return out
    if c["op"] == "read":
        for name in ("k", "v"):
            x = torch.zeros((c["B"], c["Hkv"], max(kv), c["d"]), dtype=torch.float64,
                            device=DEVICE)
            for b, L in enumerate(kv):
                x[b, :, :L] = _exact_sequence(s, name, b, L).transpose(0, 1)
            out[name] = x
        return out
    H = c["Hkv"] * c["G"]
    o = torch.zeros((s["T"], H, c["d"]), dtype=torch.float64, device=DEVICE)
    lse = torch.full((s["T"], H), -math.inf, dtype=torch.float64, device=DEVICE)
    t = 0
    for b, (n, L) in enumerate(zip(q, kv)):
        k, v = (_exact_sequence(s, name, b, L) for name in ("k", "v"))
        pos = torch.arange(L - n, L, device=DEVICE)[:, None]
        j = torch.arange(L, device=DEVICE)[None]
        seen = torch.ones((n, L), dtype=torch.bool, device=DEVICE)
        if c["causal"]:
            seen &= j <= pos
        if c["window"] >= 0:
            seen &= pos - j <= c["window"]
        for h in range(H):
            z = s["q"][t:t + n, h].double() @ k[:, h // c["G"]].T / math.sqrt(c["d"])
            z = torch.where(seen, z, -math.inf)
            lse[t:t + n, h] = torch.logsumexp(z, 1)
            o[t:t + n, h] = torch.nan_to_num(torch.softmax(z, 1)) @ v[:, h // c["G"]]
        t += n
    return {"o": o, "lse": lse}
