"""The measured cases of the recurrent block's operators: layer norm, gated scan along a
space-filling curve, and dropout into the residual stream.

A block of voxel tokens that mixes them along a curve (the order of ``vg_encode_seq``'s codes)
is a layer norm of the residual stream (``vg_layer_norm_*``), a projection to gates and inputs, a
gated linear recurrence along each sample's curve (``vg_gated_scan_*``), and a dropout of its
result on the way back into the stream (``vg_dropout_add_*``).  With ``own`` false, ``run``
computes them from elementary torch operations in 32 bits; with ``own`` true it calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
LOW = 0xFFFFFFFF            # the low 32 bits of an int64


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one readout token per sample while serving: latency
        {"name": "norm_token_f16", "op": "norm", "train": False, "dtype": "f16", "n": 2, "c": 1024, "affine": True,
         "skip": False},
        # training in fp32, a narrow odd width, odd row count, norm without weights
        {"name": "norm_train_f32", "op": "norm", "train": True, "dtype": "f32", "n": 25179, "c": 72, "affine": False,
         "skip": False},
        # training, the 256^3 scene pair's 319,057 voxels of 128 channels, the residual stream's gradient added
        {"name": "norm_train_bf16", "op": "norm", "train": True, "dtype": "bf16", "n": 319057, "c": 128,
         "affine": True, "skip": True},
        # training at the widest level of the 512^3 scene: 602,492 voxels of 1024 channels
        {"name": "norm_train_large_bf16", "op": "norm", "train": True, "dtype": "bf16", "n": 602492, "c": 1024,
         "affine": True, "skip": False},
        # one token more of each of four sequences, from the states kept between calls: latency
        {"name": "scan_token_bf16", "op": "step", "dtype": "bf16", "n": 4, "c": 512, "free": False},
        # the same for two thousand sequences served together
        {"name": "scan_tokens_f32", "op": "step", "dtype": "f32", "n": 2013, "c": 1024, "free": True},
        # inference along the curve of the 1024^3 scene, 4,915,386 voxels of 64 channels, tokens gathered on the way
        {"name": "scan_long_f16", "op": "scan", "train": False, "dtype": "f16", "n": 4915386, "c": 64, "batch": 1,
         "order": True, "reverse": False, "free": False, "empty": False, "state": False},
        # training at the 64^3 batch of four, rows already in the curve's order, against it
        {"name": "scan_train_bf16", "op": "scan", "train": True, "dtype": "bf16", "n": 25179, "c": 256, "batch": 4,
         "order": False, "reverse": True, "free": False, "empty": False, "state": False},
        # training at the 512^3 scene, 512 channels, tokens gathered along the curve
        {"name": "scan_train_large_bf16", "op": "scan", "train": True, "dtype": "bf16", "n": 602492, "c": 512,
         "batch": 1, "order": True, "reverse": False, "free": False, "empty": False, "state": False},
        # training in fp32: ragged sequences, one without tokens, states handed in and out, unscaled inputs
        {"name": "scan_train_f32", "op": "scan", "train": True, "dtype": "f32", "n": 5001, "c": 40, "batch": 7,
         "order": True, "reverse": True, "free": True, "empty": True, "state": True},
        # the 16^3 sphere's 312 voxels of 32 channels, a projection's output alone: latency
        {"name": "drop_small_f32", "op": "drop", "dtype": "f32", "n": 312 * 32, "p": 0.25, "residual": False},
        # training, 602,492 voxels of 512 channels into the residual stream
        {"name": "drop_train_large_bf16", "op": "drop", "dtype": "bf16", "n": 602492 * 512, "p": 0.1,
         "residual": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng: random.Random):
    op = rng.choice(["norm", "scan", "scan", "scan", "step", "drop"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm":
        c = 8 * _log(rng, 1, 512)
        return {"op": op, "train": rng.random() < 0.7, "dtype": dtype, "n": _log(rng, 1, min(2_000_000, 200_000_000 // c)),
                "c": c, "affine": rng.random() < 0.7, "skip": rng.random() < 0.4}
    if op == "step":
        return {"op": op, "dtype": dtype, "n": _log(rng, 1, 2000), "c": 8 * _log(rng, 1, 256),
                "free": rng.random() < 0.3}
    if op == "drop":
        return {"op": op, "dtype": dtype, "n": _log(rng, 1, 200_000_000), "p": rng.choice([0.05, 0.1, 0.25, 0.5]),
                "residual": rng.random() < 0.6}
    c = 8 * _log(rng, 1, 128)
    n = _log(rng, 1, min(5_000_000, 120_000_000 // c))
    batch = min(n, _log(rng, 1, 64))
    return {"op": op, "train": rng.random() < 0.7, "dtype": dtype, "n": n, "c": c, "batch": batch,
            "order": rng.random() < 0.5, "reverse": rng.random() < 0.5, "free": rng.random() < 0.3,
            "empty": batch > 2 and rng.random() < 0.3, "state": rng.random() < 0.4}


# ------------------------------------------------------------------ shapes of a case
def _lengths(c):
    """Tokens of each sequence, mildly uneven, the same for every seed."""
    w = [1.0 + 0.25 * ((3 * i) % 5) for i in range(c["batch"])]
    cuts = [int(round(c["n"] * sum(w[:i]) / sum(w))) for i in range(c["batch"] + 1)]
    lens = [cuts[i + 1] - cuts[i] for i in range(c["batch"])]
    if c["empty"]:                           # the second sequence's tokens go to the first
        lens[0], lens[1] = lens[0] + lens[1], 0
    return lens


def work(c):
    es = ES[c["dtype"]]
    if c["op"] == "norm":
        x = c["n"] * c["c"]
        passes = (4 if c["train"] else 2) + (1 if c["train"] and c["skip"] else 0)
        return {"bytes": passes * x * es + 8 * c["n"], "flops": (20 if c["train"] else 8) * x}
    if c["op"] == "step":
        x = c["n"] * c["c"]
        return {"bytes": x * (3 * es + 8), "flops": 8 * x}
    if c["op"] == "scan":
        x = c["n"] * c["c"]
        states = c["batch"] * c["c"] * 4 * (1 + c["state"]) * (2 if c["train"] else 1)
        return {"bytes": (6 if c["train"] else 3) * x * es + states + 4 * c["n"] * c["order"],
                "flops": (24 if c["train"] else 8) * x}
    return {"bytes": (5 if c["residual"] else 4) * c["n"] * es, "flops": 30 * c["n"]}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def prepare(c, seed):
    g = _gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt, op, n = DT[c["dtype"]], c["op"], c["n"]
    st = {"case": c}
    if op == "norm":
        w = c["c"]
        # the residual stream: channels of unlike means and spreads
        st["x"] = (rnd(n, w) * (0.5 + rnd(w).abs()) + 0.5 * rnd(w)).to(dt)
        st["weight"] = (1 + 0.2 * rnd(w)).to(dt) if c["affine"] else None
        st["bias"] = (0.1 * rnd(w)).to(dt) if c["affine"] else None
        st["y"], st["stats"] = torch.empty_like(st["x"]), torch.empty(n, 2, device="cuda")
        if c["train"]:
            st["grad_y"] = rnd(n, w).to(dt)
            st["grad_skip"] = rnd(n, w).to(dt) if c["skip"] else None
            st["grad_x"] = torch.empty_like(st["x"])
            st["gw"], st["gb"] = (torch.empty_like(st["weight"]) if c["affine"] else None for _ in range(2))
            if own:
                from voxel_gemm_gb300 import ops
                st["ws"] = ops.layer_norm_workspace(n, w) if c["affine"] else None
    elif op == "drop":
        st["x"] = rnd(n).to(dt)
        st["residual"] = rnd(n).to(dt) if c["residual"] else None
        st["grad_out"] = rnd(n).to(dt)
        st["rng"] = torch.randint(0, 2 ** 62, (2,), generator=g, device="cuda")
        st["out"], st["grad_x"] = torch.empty_like(st["x"]), torch.empty_like(st["x"])
    else:
        w = c["c"]
        # gates that forget over a few up to some hundreds of tokens, from channel to channel
        memory = torch.linspace(0.5, 5.5, w, device="cuda")
        packed = torch.cat([rnd(n, w) + memory, rnd(n, w)], 1).to(dt)      # one projection gives gates and inputs
        st["gate"], st["x"] = packed[:, :w], packed[:, w:]
        st["out"] = torch.empty(n, w, dtype=dt, device="cuda")
        if op == "step":
            st["state"] = rnd(n, w)
            return st
        lens = _lengths(c)
        st["lengths"] = lens
        off = torch.zeros(len(lens) + 1, dtype=torch.int32)
        off[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
        st["offsets"] = off.cuda()
        st["order"] = None
        if c["order"]:                       # each sequence's tokens in an order of their own
            key = torch.randint(0, 2 ** 40, (n,), generator=g, device="cuda")
            seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"))
            st["order"] = torch.argsort(key + (seq << 41)).int()
        st["first"] = rnd(len(lens), w) if c["state"] else None
        st["last"] = torch.empty(len(lens), w, device="cuda")
        if c["train"]:
            st["grad_out"] = rnd(n, w).to(dt)
            st["grad_last"] = rnd(len(lens), w) if c["state"] else None
            st["grad_packed"] = torch.empty(n, 2 * w, dtype=dt, device="cuda")
            st["grad_first"] = torch.empty(len(lens), w, device="cuda") if c["state"] else None
        if own:
            from voxel_gemm_gb300 import ops
            flags = (ops.VG_SCAN_REVERSE if c["reverse"] else 0) | (ops.VG_SCAN_FREE_INPUT if c["free"] else 0)
            st["flags"] = flags
            st["ws"] = ops.gated_scan_workspace(n, w, len(lens), dt)
            st["carries"] = ops.gated_scan_carries(n, w) if c["train"] else None
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    return {"norm": (_norm_plain, _norm_own), "scan": (_scan_plain, _scan_own), "step": (_step_plain, _step_own),
            "drop": (_drop_plain, _drop_own)}[op][bool(own)](st)


def _norm_own(st):
    from voxel_gemm_gb300 import ops
    ops.vg_layer_norm_fwd(st["x"], st["weight"], st["bias"], st["y"], st["stats"], eps=EPS)
    res = {"y": st["y"], "stats": st["stats"]}
    if not st["case"]["train"]:
        return res
    ops.vg_layer_norm_bwd(st["x"], st["weight"], st["stats"], st["grad_y"], st["grad_skip"], st["grad_x"], st["gw"],
                          st["gb"], st["ws"])
    res["grad_x"] = st["grad_x"]
    if st["gw"] is not None:
        res["grad_weight"], res["grad_bias"] = st["gw"], st["gb"]
    return res


def _scan_own(st):
    from voxel_gemm_gb300 import ops
    c, flags = st["case"], st["flags"]
    ops.vg_gated_scan_fwd(st["gate"], st["x"], st["offsets"], st["order"], st["first"], st["out"], st["last"],
                          st["carries"], st["ws"], flags=flags)
    res = {"out": st["out"], "last": st["last"]}
    if not c["train"]:
        return res
    w = c["c"]
    ops.vg_gated_scan_bwd(st["gate"], st["x"], st["offsets"], st["order"], st["first"], st["carries"], st["grad_out"],
                          st["grad_last"], st["grad_packed"][:, :w], st["grad_packed"][:, w:], st["grad_first"],
                          st["ws"], flags=flags)
    res["grad_packed"] = st["grad_packed"]
    if st["grad_first"] is not None:
        res["grad_first"] = st["grad_first"]
    return res


def _step_own(st):
    from voxel_gemm_gb300 import ops
    ops.vg_gated_scan_step(st["gate"], st["x"], st["state"], st["out"],
                           flags=ops.VG_SCAN_FREE_INPUT if st["case"]["free"] else 0)
    return {"out": st["out"], "state": st["state"]}


def _drop_own(st):
    from voxel_gemm_gb300 import ops
    p = st["case"]["p"]
    ops.vg_dropout_add_fwd(st["x"], st["residual"], p, st["rng"], 3, st["out"])
    ops.vg_dropout_add_bwd(st["grad_out"], p, st["rng"], 3, st["grad_x"])
    return {"out": st["out"], "grad_x": st["grad_x"]}


# ------------------------------------------------------------------ plain forms (32 bits)
def _norm_plain(st):
    c, dt = st["case"], st["x"].dtype
    x = st["x"].float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = ((x * x).mean(1, keepdim=True) + EPS).rsqrt()
    x *= rstd
    y = x * st["weight"].float() + st["bias"].float() if c["affine"] else x
    res = {"y": y.to(dt), "stats": torch.cat([mean, rstd], 1)}
    del y
    if not c["train"]:
        return res
    g = st["grad_y"].float()
    if c["affine"]:
        res["grad_weight"], res["grad_bias"] = (g * x).sum(0).to(dt), g.sum(0).to(dt)
        g = g * st["weight"].float()
    along = (g * x).mean(1, keepdim=True)
    gx = (g - g.mean(1, keepdim=True) - x * along) * rstd
    if c["skip"]:
        gx += st["grad_skip"].float()
    res["grad_x"] = gx.to(dt)
    return res


def _visits(st):
    """Row of each visited position [n], the positions in their sequences [n, 1], and the visits' sequences."""
    c, lens = st["case"], st["lengths"]
    n = c["n"]
    rows = st["order"].long() if c["order"] else torch.arange(n, device="cuda")
    seqs = torch.arange(len(lens), device="cuda")
    sizes = torch.tensor(lens, device="cuda")
    starts = st["offsets"][:-1].long()
    if c["reverse"]:                         # from the end: the sequences too are met in the other order
        rows, seqs, sizes = rows.flip(0), seqs.flip(0), sizes.flip(0)
        starts = n - st["offsets"][1:].long().flip(0)
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), sizes)
    pos = torch.arange(n, device="cuda") - starts[seq]
    return rows, pos[:, None], seqs, sizes


def _chain(a, b, pos):
    """h[i] = a[i] h[i - 1] + b[i] with h = 0 before position 0, by doubling the distance looked back."""
    far = int(pos.max()) + 1 if pos.numel() else 0
    d = 1
    while d < far:
        have = pos[d:] >= d
        nb = torch.where(have, a[d:] * b[:-d], 0.0) + b[d:]
        na = a[d:] * torch.where(have, a[:-d], 1.0)
        b, a = torch.cat([b[:d], nb]), torch.cat([a[:d], na])
        d *= 2
    return b


def _scan_plain(st):
    c, w, dt = st["case"], st["case"]["c"], st["out"].dtype
    n, bsz = c["n"], c["batch"]
    rows, pos, seqs, sizes = _visits(st)
    gate, x = st["gate"][rows].float(), st["x"][rows].float()
    a, s = torch.sigmoid(gate), torch.sigmoid(-gate)
    b = x if c["free"] else s * x
    ends = sizes.cumsum(0) - 1
    filled = sizes > 0
    begin = (ends - sizes + 1)[filled]       # visits at which a sequence begins
    first = st["first"][seqs] if c["state"] else torch.zeros(bsz, w, device="cuda")
    b0 = b.clone()
    b0[begin] += a[begin] * first[filled]
    h = _chain(a, b0, pos)
    out = torch.empty(n, w, dtype=dt, device="cuda")
    out[rows] = h.to(dt)
    last = torch.empty(bsz, w, device="cuda")
    last[seqs] = torch.where(filled[:, None], h[ends.clamp(min=0)], first) if n else first
    res = {"out": out, "last": last}
    if not c["train"]:
        return res
    del b0
    before = torch.cat([h[:1], h[:-1]])
    before[begin] = first[filled]
    del h
    up = st["grad_out"][rows].float()
    g_last = st["grad_last"][seqs] if c["state"] else torch.zeros(bsz, w, device="cuda")
    up[ends[filled]] += g_last[filled]
    after = torch.cat([a[1:], a[:1]])        # the gate through which the next state reads this one
    left = (sizes[torch.repeat_interleave(torch.arange(bsz, device="cuda"), sizes)][:, None] - 1 - pos)
    lam = _chain(after.flip(0), up.flip(0), left.flip(0)).flip(0)
    del after, up
    gp = torch.empty(n, 2 * w, dtype=dt, device="cuda")
    slope = a * s
    gp[rows, :w] = (lam * (before if c["free"] else before - x) * slope).to(dt)
    gp[rows, w:] = (lam if c["free"] else lam * s).to(dt)
    res["grad_packed"] = gp
    if c["state"]:
        gf = g_last.clone()
        gf[filled] = a[begin] * lam[begin]
        res["grad_first"] = torch.empty_like(gf)
        res["grad_first"][seqs] = gf
    return res


def _step_plain(st):
    gate, x, h = st["gate"].float(), st["x"].float(), st["state"]
    s = torch.sigmoid(-gate)
    h = torch.sigmoid(gate) * h + (x if st["case"]["free"] else s * x)
    st["state"].copy_(h)
    return {"out": h.to(st["out"].dtype), "state": st["state"]}


def _words(rng, call, n):
    """Random words of elements 0 .. n - 1 as int64 in [0, 2^32): ten rounds of Philox 4x32 (Salmon, Moraes, Dror and
    Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), key rng[0], counter (group of 4, rng[1], call)."""
    i = torch.arange((n + 3) // 4, device="cuda")
    c0, c1, c2, c3 = i & LOW, i >> 32, (rng[1] & LOW).expand_as(i), torch.full_like(i, call)
    k0, k1 = rng[0] & LOW, (rng[0] >> 32) & LOW
    for _ in range(10):
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((q >> 32) & LOW) ^ c1 ^ k0, q & LOW, ((p >> 32) & LOW) ^ c3 ^ k1, p & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return torch.stack([c0, c1, c2, c3], 1).view(-1)[:n]


def _drop_plain(st):
    c, dt = st["case"], st["x"].dtype
    keep = _words(st["rng"], 3, c["n"]) >= round(c["p"] * 2 ** 32)
    scale = 1 / (1 - c["p"])
    y = torch.where(keep, st["x"].float() * scale, 0.0)
    if c["residual"]:
        y += st["residual"].float()
    return {"out": y.to(dt), "grad_x": torch.where(keep, st["grad_out"].float() * scale, 0.0).to(dt)}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(c, seed):
    st = prepare(c, seed)
    return {"norm": _norm_exact, "scan": _scan_exact, "step": _step_exact, "drop": _drop_exact}[c["op"]](st)


def _norm_exact(st):
    """By the derivative of each row's standard form, a range of rows at a time."""
    c = st["case"]
    n, w = c["n"], c["c"]
    one = torch.ones(w, dtype=torch.float64, device="cuda")
    weight = st["weight"].double() if c["affine"] else one
    y, stats = torch.empty(n, w, dtype=torch.float64, device="cuda"), torch.empty(n, 2, dtype=torch.float64, device="cuda")
    gx = torch.empty_like(y) if c["train"] else None
    gw, gb = torch.zeros_like(one), torch.zeros_like(one)
    step = max(1, 40_000_000 // w)
    for lo in range(0, n, step):
        x = st["x"][lo:lo + step].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        sd = (var + EPS).sqrt()
        stats[lo:lo + step] = torch.cat([mean, 1 / sd], 1)
        z = (x - mean) / sd
        y[lo:lo + step] = torch.addcmul(st["bias"].double(), z, weight) if c["affine"] else z
        if c["train"]:
            g = st["grad_y"][lo:lo + step].double()
            gw += torch.einsum("ij,ij->j", g, z)
            gb += g.sum(0)
            g = g * weight
            inner = torch.einsum("ij,ij->i", g, z)[:, None] / w
            gx[lo:lo + step] = (g - g.mean(1, keepdim=True)) / sd - z * inner / sd
            if c["skip"]:
                gx[lo:lo + step] += st["grad_skip"][lo:lo + step].double()
    res = {"y": y, "stats": stats}
    if c["train"]:
        res["grad_x"] = gx
        if c["affine"]:
            res["grad_weight"], res["grad_bias"] = gw, gb
    return res


def _walk(a, b, start):
    """States of h <- a[t] h + b[t] from `start`, one sequence [t, w]: runs of about sqrt(t) side by side."""
    t, w = b.shape
    run = max(1, math.isqrt(t))
    k = -(-t // run)
    pa, pb = (torch.cat([v, v.new_zeros(k * run - t, w)]).view(k, run, w) for v in (a, b))
    grow, local = torch.ones(k, w, dtype=a.dtype, device="cuda"), torch.zeros(k, w, dtype=a.dtype, device="cuda")
    for j in range(run):
        local = torch.addcmul(pb[:, j], pa[:, j], local)
        grow = grow * pa[:, j]
    enter = torch.empty(k, w, dtype=a.dtype, device="cuda")
    h = start
    for i in range(k):
        enter[i] = h
        h = torch.addcmul(local[i], grow[i], h)
    out = torch.empty(k, run, w, dtype=a.dtype, device="cuda")
    for j in range(run):
        enter = torch.addcmul(pb[:, j], pa[:, j], enter)
        out[:, j] = enter
    return out.view(k * run, w)[:t]


def _scan_exact(st):
    c = st["case"]
    n, w = c["n"], c["c"]
    new = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    out, gp = new(n, w), new(n, 2 * w) if c["train"] else None
    last, gfirst = new(c["batch"], w), new(c["batch"], w)
    at = 0
    for i, t in enumerate(st["lengths"]):
        h0 = st["first"][i].double() if c["state"] else new(w)
        gl = st["grad_last"][i].double() if c["train"] and c["state"] else new(w)
        if t == 0:
            last[i], gfirst[i] = h0, gl
            continue
        rows = st["order"][at:at + t].long() if c["order"] else torch.arange(at, at + t, device="cuda")
        if c["reverse"]:
            rows = rows.flip(0)
        at += t
        gate, x = st["gate"][rows].double(), st["x"][rows].double()
        a = 1 / (1 + torch.exp(-gate))
        put = 1 / (1 + torch.exp(gate))
        h = _walk(a, x if c["free"] else put * x, h0)
        out[rows], last[i] = h, h[-1]
        if not c["train"]:
            continue
        prior = torch.cat([h0[None], h[:-1]])
        del h
        # the gradient of the state after each token, walked backwards from the last one's
        up = st["grad_out"][rows].double()
        up[-1] += gl
        through = torch.cat([new(1, w), a[1:].flip(0)])
        lam = _walk(through, up.flip(0), new(w)).flip(0)
        del up, through
        gp[rows, w:] = lam if c["free"] else lam * put
        gp[rows, :w] = lam * (prior if c["free"] else prior - x) * a * put
        gfirst[i] = a[0] * lam[0]
    res = {"out": out, "last": last}
    if c["train"]:
        res["grad_packed"] = gp
        if c["state"]:
            res["grad_first"] = gfirst
    return res


def _step_exact(st):
    gate, x = st["gate"].double(), st["x"].double()
    keep = 1 / (1 + torch.exp(-gate))
    put = 1.0 if st["case"]["free"] else 1 / (1 + torch.exp(gate))
    h = keep * st["state"].double() + put * x
    return {"out": h, "state": h}


def _times(m, v):
    """High and low words of m v for 32-bit m and v held in int64, from the halves of v."""
    low, high = m * (v & 0xFFFF), m * (v >> 16)
    mid = (low >> 16) + (high & 0xFFFF)
    return (high >> 16) + (mid >> 16), ((mid & 0xFFFF) << 16) | (low & 0xFFFF)


def _drop_exact(st):
    c = st["case"]
    n, p = c["n"], c["p"]
    seed, step = (v % 2 ** 64 for v in st["rng"].tolist())
    out, gx = (torch.empty(n, dtype=torch.float64, device="cuda") for _ in range(2))
    share = 1 << 26
    for lo in range(0, n, share):
        hi = min(n, lo + share)
        group = torch.arange(lo // 4, (hi + 3) // 4, device="cuda")
        x = [group % 2 ** 32, group // 2 ** 32, torch.full_like(group, step % 2 ** 32), torch.full_like(group, 3)]
        for turn in range(10):
            ka, kb = (seed + turn * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + turn * 0xBB67AE85) % 2 ** 32
            (ha, la), (hb, lb) = _times(0xD2511F53, x[0]), _times(0xCD9E8D57, x[2])
            x = [torch.bitwise_xor(torch.bitwise_xor(hb, x[1]), ka), lb,
                 torch.bitwise_xor(torch.bitwise_xor(ha, x[3]), kb), la]
        word = torch.stack(x, 1).flatten()[:hi - lo].double()
        stay = (word >= round(p * 2.0 ** 32)).double() / (1 - p)
        out[lo:hi] = st["x"][lo:hi].double() * stay
        if c["residual"]:
            out[lo:hi] += st["residual"][lo:hi].double()
        gx[lo:hi] = st["grad_out"][lo:hi].double() * stay
    return {"out": out, "grad_x": gx}
