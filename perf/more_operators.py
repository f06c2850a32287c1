"""Attention of queries over keys of another length, with a learned bias by relative
position: cross attention (an encoder's states, a memory in front of a chunk) with its
backward pass, self or cross attention whose scores get a bias by distance buckets with
the gradient of the bias table, and a decode step with that bias over a K/V cache.

``run`` computes them in plain torch operations, or with this package's calls where
``own`` is true. Query i sits at position i + q_offset of the key axis (at the last
positions of its sequence in a step); the bias of key j is that of the distance
j - position, looked up in a map from clamped distances to rows of the table.
``lens`` seeds the key lengths of the batch, which belong to the case.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
SCORES = 1 << 30  # scores that a plain form holds at once


def _case(name, op, B, H, Hkv, Nq, Nk, d, grad=False, k_min=None, causal=False, q_offset=0,
          lens=0, buckets="", num_buckets=0, distance=0, both=True, table="fp32"):
    return {"name": name, "op": op, "B": B, "H": H, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "d": d,
            "grad": grad, "k_min": Nk if k_min is None else k_min, "causal": causal,
            "q_offset": q_offset, "lens": lens, "buckets": buckets, "num_buckets": num_buckets,
            "distance": distance, "both": both, "table": table}


def listed():
    log = {"buckets": "log", "num_buckets": 32, "distance": 128}
    return [
        # a few target tokens look at a short source: latency
        _case("cross_short", "cross", 2, 8, 8, 33, 100, 64, k_min=40, lens=1),
        # a batch of targets over padded encoder states of odd length
        _case("cross_padded", "cross", 16, 16, 16, 448, 1500, 64, k_min=300, lens=2),
        # the same in training
        _case("cross_train", "cross", 16, 16, 16, 448, 1500, 64, grad=True, k_min=300, lens=2),
        # training on the last 2048 positions over a memory of 6000 in front of them, grouped heads
        _case("memory_train_d128", "cross", 1, 32, 8, 2048, 8048, 128, grad=True, causal=True,
              q_offset=6000),
        # an encoder on a batch of short inputs: nearly every tile is near the diagonal
        _case("rel_short", "rel", 8, 12, 12, 200, 200, 64, k_min=20, lens=3, **log),
        # an encoder layer in training
        _case("rel_train", "rel", 16, 16, 16, 1024, 1024, 64, grad=True, k_min=512, lens=4, **log),
        # a decoder layer in training, table in bf16
        _case("rel_train_causal_d128", "rel", 2, 16, 16, 4096, 4096, 128, grad=True, causal=True,
              both=False, table="bf16", **log),
        # a long document (B=1 H=16 N=16384) in training
        _case("rel_train_long", "rel", 1, 16, 16, 16384, 16384, 64, grad=True, **log),
        # one entry per distance up to 1000, heads of 128
        _case("rel_clip_train", "rel", 4, 8, 8, 2000, 2000, 128, grad=True, buckets="clip",
              distance=1000),
        # a step of a few short answers: latency
        _case("step_short", "step", 4, 16, 16, 1, 500, 64, k_min=1, causal=True, lens=5,
              both=False, **log),
        # a decode batch of ragged lengths
        _case("step_ragged", "step", 32, 16, 16, 1, 4096, 64, k_min=1, causal=True, lens=6,
              both=False, **log),
        # drafted tokens of one long context, grouped heads of 128, table in bf16
        _case("step_long_draft", "step", 1, 32, 8, 5, 131001, 128, causal=True, both=False,
              table="bf16", **log),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("cross", "cross", "rel", "rel", "rel", "step"))
        d = rng.choice((64, 128))
        Hkv = rng.choice((1, 2, 4, 8, 12, 16))
        H = Hkv * rng.choice((1, 1, 1, 2, 4))
        B = _log_uniform(rng, 1, 64)
        c = {"op": op, "B": B, "H": H, "Hkv": Hkv, "d": d, "grad": False, "causal": True,
             "q_offset": 0, "lens": rng.randrange(1 << 30), "buckets": "", "num_buckets": 0,
             "distance": 0, "both": True, "table": rng.choice(("fp32", "bf16"))}
        if op == "step":
            c["Nq"], c["Nk"] = rng.choice((1, 1, 1, 2, 5, 8)), _log_uniform(rng, 16, 131072)
        else:
            c["Nq"] = _log_uniform(rng, 1, 16384)
            same = op == "rel" and rng.random() < 0.7
            c["Nk"] = c["Nq"] if same else _log_uniform(rng, 1, 16384)
            c["grad"] = rng.random() < 0.6
            if c["grad"] and c["Nk"] == 1:  # the weight is 1 whatever the score: no gradients
                continue
            c["causal"] = rng.random() < 0.4
            if c["causal"] and c["Nk"] > c["Nq"]:
                c["q_offset"] = rng.choice((c["Nk"] - c["Nq"], rng.randrange(c["Nk"] - c["Nq"])))
        c["k_min"] = rng.choice((c["Nk"], c["Nk"] // 2 + 1, 1))
        if op == "step":
            c["k_min"] = max(c["k_min"], c["Nq"])
        if op != "cross":
            c["buckets"] = rng.choice(("log", "log", "clip"))
            c["both"] = rng.random() < 0.5
            if c["buckets"] == "log":
                c["num_buckets"] = rng.choice((8, 16, 32, 32, 64))
                c["distance"] = _log_uniform(rng, 64, 1000)
            else:
                c["distance"] = _log_uniform(rng, 4, 1500)
        if _cost(c) <= most and 4.0 * B * Hkv * c["Nk"] * d <= 6e9:
            return c


# ------------------------------------------------------------- the batch of a case

def _lengths(c):
    """Key lengths of the batch."""
    r = random.Random(c["lens"])
    n = [r.randint(c["k_min"], c["Nk"]) for _ in range(c["B"])]
    n[r.randrange(c["B"])] = c["Nk"]
    return n


def _starts(c):
    """Position of the first query of each sequence on the key axis."""
    if c["op"] == "step":
        return [n - c["Nq"] for n in _lengths(c)]
    return [c["q_offset"]] * c["B"]


def _pairs(c):
    """Visible pairs of query and key over the batch, for one head."""
    total = 0
    for n, p in zip(_lengths(c), _starts(c)):
        if not c["causal"]:
            total += n * c["Nq"]
            continue
        i0 = min(c["Nq"], max(0, -p))        # rows before the first key see none
        i1 = min(c["Nq"], max(i0, n - p))    # rows i0 .. i1 - 1 see p + i + 1 keys, the rest n
        total += (i1 - i0) * (p + 1) + (i0 + i1 - 1) * (i1 - i0) // 2 + (c["Nq"] - i1) * n
    return total


def _bucket_map(c):
    """Rows of the table by distance -left .. right, and left. Distances beyond are clamped."""
    if c["buckets"] == "clip":
        return list(range(c["distance"] + 1 + c["distance"] * c["both"])), c["distance"]
    half = c["num_buckets"] // 2 if c["both"] else c["num_buckets"]
    exact = half // 2  # distances below it have a bucket each, the others share by their logarithm
    steps = half - exact
    side, n = [], 0
    while not side or side[-1] < half - 1:
        t = 0
        if n >= exact:  # the largest t < steps with (n / exact)^steps >= (distance / exact)^t
            while t + 1 < steps and n ** steps >= c["distance"] ** (t + 1) * exact ** (steps - t - 1):
                t += 1
            side.append(exact + t)
        else:
            side.append(n)
        n += 1
    right = [half + b for b in side[1:]] if c["both"] else []
    return side[::-1] + right, len(side) - 1


def _table_rows(c):
    if c["buckets"] == "clip":
        return c["distance"] + 1 + c["distance"] * c["both"]
    return c["num_buckets"]


def work(case):
    c = case
    pairs, rows, keys = _pairs(c), c["B"] * c["Nq"], sum(_lengths(c))
    table = _table_rows(c) * c["H"] * (4 if c["table"] == "fp32" else 2) if c["buckets"] else 0
    q, kv = rows * c["H"] * c["d"] * 2, keys * c["Hkv"] * c["d"] * 2
    lse = rows * c["H"] * 4
    w = {"bytes": 2 * q + 2 * kv + lse + table, "flops": 4 * c["d"] * c["H"] * pairs}
    if c["grad"]:  # dO read; dQ, and dK and dV over all rows, written
        w["bytes"] += 2 * q + 2 * c["B"] * c["Nk"] * c["Hkv"] * c["d"] * 2
        w["bytes"] += _table_rows(c) * c["H"] * 4 if c["buckets"] else 0
        w["flops"] += 10 * c["d"] * c["H"] * pairs
    return w


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


# ------------------------------------------------------------- inputs

def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))

    def rows(H, N):
        x = torch.randn((c["B"], H, N, c["d"]), generator=g, device=DEVICE, dtype=torch.bfloat16)
        # channels of unlike size
        return x * torch.rand(c["d"], generator=g, device=DEVICE).add(0.5).to(torch.bfloat16)

    s = {"case": c, "q": rows(c["H"], c["Nq"]), "k": rows(c["Hkv"], c["Nk"]),
         "v": rows(c["Hkv"], c["Nk"])}
    s["lens"] = None
    if c["k_min"] < c["Nk"]:
        s["lens"] = torch.tensor(_lengths(c), dtype=torch.int32, device=DEVICE)
    if c["grad"]:
        s["do"] = rows(c["H"], c["Nq"])
    if c["buckets"]:
        rule, s["left"] = _bucket_map(c)
        s["map"] = torch.tensor(rule, dtype=torch.int32, device=DEVICE)
        t = torch.randn((_table_rows(c), c["H"]), generator=g, device=DEVICE)
        s["table"] = t if c["table"] == "fp32" else t.to(torch.bfloat16)
        if own:
            import io_aware_exact_07_gb300 as fa
            if c["buckets"] == "log":
                s["buckets"] = fa.rel_buckets(c["num_buckets"], c["distance"], c["both"],
                                              device=DEVICE)
            else:
                s["buckets"] = fa.RelBuckets(s["map"], s["left"], _table_rows(c))
            if c["op"] == "step":  # a server lays the bias out once
                s["rel"] = fa.rel_bias(s["table"], s["buckets"])
    return s


# ------------------------------------------------------------- plain forms

def _plain_block(s, b0, b1, g0, g1, out):
    """Batch rows b0 .. b1 and K/V heads g0 .. g1 of the case, in fp32."""
    c = s["case"]
    nb, ng, G, Nq, Nk, d = b1 - b0, g1 - g0, c["H"] // c["Hkv"], c["Nq"], c["Nk"], c["d"]
    heads = slice(g0 * G, g1 * G)
    k, v = (s[n][b0:b1, g0:g1].float() for n in ("k", "v"))
    q = s["q"][b0:b1, heads].reshape(nb, ng, G * Nq, d).float()
    z = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(nb, ng * G, Nq, Nk)
    dev = z.device
    kv = (torch.full((nb,), Nk, device=dev) if s["lens"] is None else s["lens"][b0:b1]).long()
    start = kv - Nq if c["op"] == "step" else torch.full_like(kv[:1], c["q_offset"])
    pos = start[:, None, None] + torch.arange(Nq, device=dev)[:, None]  # [nb or 1, Nq, 1]
    j = torch.arange(Nk, device=dev)
    if c["buckets"]:
        away = (j - pos).clamp(-s["left"], s["map"].numel() - 1 - s["left"]) + s["left"]
        row = s["map"].long()[away]  # [nb or 1, Nq, Nk]
        table = s["table"].float()[:, heads]
        for h in range(ng * G):
            z[:, h] += table[:, h][row]
    seen = j < kv[:, None, None]
    if c["causal"]:
        seen = seen & (j <= pos)
    z.masked_fill_(~seen[:, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.mul_(torch.where(l > 0, 1.0 / l, torch.zeros_like(l)))
    o = (p.view(nb, ng, G * Nq, Nk) @ v).view(nb, ng * G, Nq, d)
    out["o"][b0:b1, heads] = o.to(torch.bfloat16)
    out["lse"][b0:b1, heads] = (m + l.log())[..., 0]
    if not c["grad"]:
        return
    do = s["do"][b0:b1, heads].float()
    dg = do.reshape(nb, ng, G * Nq, d)
    out["dv"][b0:b1, g0:g1] = (p.view(nb, ng, G * Nq, Nk).transpose(2, 3) @ dg).to(torch.bfloat16)
    ds = (dg @ v.transpose(2, 3)).view(nb, ng * G, Nq, Nk)
    ds = ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    if c["buckets"]:
        # rows in reverse order, each shifted by one more: column Nq - 1 + j - i holds the
        # scores of distance j - i
        away = torch.arange(1 - Nq, Nk, device=dev) - c["q_offset"]
        away = away.clamp(-s["left"], s["map"].numel() - 1 - s["left"]) + s["left"]
        for h in range(ng * G):
            x = torch.zeros((Nq, Nk + Nq), device=dev)
            x[:, :Nk] = ds[:, h].sum(0).flip(0)
            x = x.flatten()[:Nq * (Nk + Nq - 1)].view(Nq, Nk + Nq - 1)
            out["dtable"][:, g0 * G + h].index_add_(0, s["map"].long()[away],
                                                    x.sum(0, dtype=torch.float64))
    ds = ds.view(nb, ng, G * Nq, Nk)
    scale = 1.0 / math.sqrt(d)
    out["dq"][b0:b1, heads] = (ds @ k).mul_(scale).view(nb, ng * G, Nq, d).to(torch.bfloat16)
    out["dk"][b0:b1, g0:g1] = (ds.transpose(2, 3) @ q).mul_(scale).to(torch.bfloat16)


def _plain(s):
    c = s["case"]
    out = {"o": torch.empty_like(s["q"]),
           "lse": torch.empty(s["q"].shape[:3], dtype=torch.float32, device=DEVICE)}
    if c["grad"]:
        out.update(dq=torch.empty_like(s["q"]), dk=torch.empty_like(s["k"]),
                   dv=torch.empty_like(s["v"]))
        if c["buckets"]:
            out["dtable"] = torch.zeros(s["table"].shape, dtype=torch.float64, device=DEVICE)
    one = c["Nq"] * c["Nk"] * (c["H"] // c["Hkv"])  # scores of a K/V head
    ng = max(1, min(c["Hkv"], SCORES // one))
    nb = max(1, min(c["B"], SCORES // (one * c["Hkv"])))
    for b in range(0, c["B"], nb):
        for g in range(0, c["Hkv"], ng):
            _plain_block(s, b, min(b + nb, c["B"]), g, min(g + ng, c["Hkv"]), out)
    if "dtable" in out:
        out["dtable"] = out["dtable"].float()
    return out


# ------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain(s)
    import io_aware_exact_07_gb300 as fa
    if c["op"] == "step":
        o, lse = fa.decode(s["q"], s["k"], s["v"], causal=c["causal"], seqlens_k=s["lens"],
                           rel_bias=s["rel"])
        return {"o": o, "lse": lse}
    how = {"causal": c["causal"], "seqlens_k": s["lens"], "q_offset": c["q_offset"]}
    if c["buckets"]:  # a training step's table is new
        how["rel_bias"] = fa.rel_bias(s["table"], s["buckets"])
    o, lse = fa.fwd(s["q"], s["k"], s["v"], **how)
    out = {"o": o, "lse": lse}
    if c["grad"]:
        grads = fa.bwd(s["q"], s["k"], s["v"], o, s["do"], lse, **how)
        out.update(zip(("dq", "dk", "dv", "dtable"), grads))
    return out


# ------------------------------------------------------------- the definition in 64 bits

def _exact_bucket(c, away):
    """The row of the table of distance `away` (key minus query), from the rule itself."""
    if c["buckets"] == "clip":
        return max(-c["distance"], min(away, c["distance"] if c["both"] else 0)) + c["distance"]
    half = c["num_buckets"] // 2 if c["both"] else c["num_buckets"]
    n = abs(away) if c["both"] else max(0, -away)
    exact = half // 2
    b = n
    if n >= exact:
        b, E = half - 1, half - exact
        while b > exact and n ** E < c["distance"] ** (b - exact) * exact ** (E - (b - exact)):
            b -= 1
    return b + half if c["both"] and away > 0 else b


def exact(case, seed):
    c = case
    if work(c)["flops"] > 5e12:
        return None
    s = prepare(c, seed)
    G, d, Nq, Nk = c["H"] // c["Hkv"], c["d"], c["Nq"], c["Nk"]
    f64 = {"dtype": torch.float64, "device": DEVICE}
    out = {"o": torch.zeros(s["q"].shape, **f64),
           "lse": torch.full(s["q"].shape[:3], -math.inf, **f64)}
    if c["grad"]:
        out.update({"d" + n: torch.zeros(s[n].shape, **f64) for n in ("q", "k", "v")})
    if c["buckets"]:
        reach = c["distance"]  # the rule is constant beyond
        rule = [_exact_bucket(c, a) for a in range(-reach, reach + 1)]
        # runs of distances with one bucket: where each begins, and their buckets
        at = [0] + [i for i in range(1, len(rule)) if rule[i] != rule[i - 1]]
        runs = torch.tensor([rule[i] for i in at], device=DEVICE)
        first = torch.tensor([i - reach for i in at[1:]], dtype=torch.long, device=DEVICE)
        rule = torch.tensor(rule, device=DEVICE)
        if c["grad"]:
            out["dtable"] = torch.zeros(s["table"].shape, **f64)
    for b, (n, p0) in enumerate(zip(_lengths(c), _starts(c))):
        pos = torch.arange(p0, p0 + Nq, device=DEVICE)[:, None]
        j = torch.arange(n, device=DEVICE)[None]
        hidden = (j > pos) if c["causal"] else None
        if c["buckets"]:
            row = rule[(j - pos).clamp(-reach, reach) + reach]
        for h in range(c["H"]):
            k, v = (s[x][b, h // G, :n].double() for x in ("k", "v"))
            q = s["q"][b, h].double()
            z = q @ k.T / math.sqrt(d)
            if c["buckets"]:
                z += s["table"].double()[:, h][row]
            if hidden is not None:
                z[hidden] = -math.inf
            out["lse"][b, h] = torch.logsumexp(z, 1)
            p = torch.nan_to_num(torch.softmax(z, 1))
            out["o"][b, h] = p @ v
            if not c["grad"]:
                continue
            do = s["do"][b, h].double()
            out["dv"][b, h // G, :n] += p.T @ do
            dp = do @ v.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            out["dq"][b, h] = ds @ k / math.sqrt(d)
            out["dk"][b, h // G, :n] += ds.T @ q / math.sqrt(d)
            if c["buckets"]:  # what a run holds of a row is a difference of two running sums
                upto = torch.cat((torch.zeros((Nq, 1), **f64), ds.cumsum(1)), 1)
                ends = upto.gather(1, (pos + first).clamp(0, n))
                ends = torch.cat((upto[:, :1], ends, upto[:, -1:]), 1)
                out["dtable"][:, h].index_add_(0, runs, ends.diff(dim=1).sum(0))
    return out
