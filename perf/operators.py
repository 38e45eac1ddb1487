"""The measured cases of the attention-block operators: query/key norm with rotary
positions, cross attention, and the AdamW step.

Three operators stand side by side in a voxel model's attention block: the
per-head norm and rotation of queries and keys by voxel position
(``vg_qk_norm_rope_*``), the attention of the voxel tokens to an encoder's states
(``vg_cross_attn_*``), and the optimizer step over the block's and the
convolutions' weights (``vg_adamw_step``).  With ``own`` false, ``run`` computes
them from elementary torch operations in 32 bits; with ``own`` true it calls the
library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 256                 # elements per scale of an 8-bit optimizer state
THETA = 10000.0


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one readout token per sample over a short text encoding: the smallest call, latency
        {"name": "attn_token_bf16", "op": "attn", "train": False, "dtype": "bf16", "n_q": 2, "n_k": 154, "batch": 2,
         "hq": 8, "hk": 8, "d": 64, "padded": False, "empty": False},
        # one readout token per sample over all voxels of a 256^3 scene pair (319,057 tokens), shared heads
        {"name": "attn_pool_long_bf16", "op": "attn", "train": False, "dtype": "bf16", "n_q": 2, "n_k": 319057,
         "batch": 2, "hq": 16, "hk": 8, "d": 64, "padded": False, "empty": False},
        # inference: 25,179 voxels (64^3, batch 4) reading padded encoder states, 128-wide heads, shared heads
        {"name": "attn_fwd_f16_d128", "op": "attn", "train": False, "dtype": "f16", "n_q": 25179, "n_k": 4096,
         "batch": 4, "hq": 16, "hk": 4, "d": 128, "padded": True, "empty": False},
        # training at the same voxel count, ragged encoder lengths, one sample without any states, shared heads
        {"name": "attn_train_bf16", "op": "attn", "train": True, "dtype": "bf16", "n_q": 25179, "n_k": 5001,
         "batch": 4, "hq": 16, "hk": 8, "d": 64, "padded": False, "empty": True},
        # training on large scenes: 100k voxel tokens, 1370 image patches a sample
        {"name": "attn_train_large_bf16", "op": "attn", "train": True, "dtype": "bf16", "n_q": 100003, "n_k": 2740,
         "batch": 2, "hq": 16, "hk": 16, "d": 64, "padded": False, "empty": False},
        # training in fp32 with an odd token count and a narrow head (the exact path)
        {"name": "attn_train_f32", "op": "attn", "train": True, "dtype": "f32", "n_q": 2013, "n_k": 1001, "batch": 2,
         "hq": 4, "hk": 2, "d": 40, "padded": False, "empty": False},
        # one token's norm and rotation while serving: latency
        {"name": "rope_token_f16", "op": "rope", "train": False, "dtype": "f16", "n": 1, "hq": 16, "hk": 4, "d": 128,
         "halves": False, "shared": True},
        # training, 319,057 voxels, 16 heads of 64: bandwidth
        {"name": "rope_train_bf16", "op": "rope", "train": True, "dtype": "bf16", "n": 319057, "hq": 16, "hk": 16,
         "d": 64, "halves": False, "shared": False},
        # training in fp32, 48-wide heads, pairs across the halves, unequal head counts
        {"name": "rope_train_f32", "op": "rope", "train": True, "dtype": "f32", "n": 25179, "hq": 6, "hk": 2, "d": 48,
         "halves": True, "shared": True},
        # optimizer step of the smallest layer set (32 channels, fp32)
        {"name": "adamw_small_f32", "op": "adamw", "dtype": "f32", "bits": 32, "master": False, "width": 32,
         "blocks": 1},
        # bf16 weights with fp32 masters and 8-bit states, four 512-channel blocks
        {"name": "adamw_8bit_bf16", "op": "adamw", "dtype": "bf16", "bits": 8, "master": True, "width": 512,
         "blocks": 4},
        # bf16 weights with fp32 masters and 32-bit states, two 1024-channel blocks
        {"name": "adamw_large_bf16", "op": "adamw", "dtype": "bf16", "bits": 32, "master": True, "width": 1024,
         "blocks": 2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["attn", "attn", "rope", "adamw"])
    if op == "attn":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 4])
        d = rng.choice([32, 40, 64, 64, 72, 96, 128])
        batch = rng.choice([1, 2, 3, 4, 7])
        padded = rng.random() < 0.3
        n_q = max(batch, _log(rng, 1, 100000))
        cap = 100003 * 1370 * 16 * 64 // (8 if dtype == "f32" else 1)   # query-key-channel products
        n_k = max(batch, min(_log(rng, 17, 300000), cap // (n_q * hq * d) * batch // 4))
        return {"op": "attn", "train": rng.random() < 0.6, "dtype": dtype, "n_q": n_q, "n_k": n_k, "batch": batch,
                "hq": hq, "hk": hk, "d": d, "padded": padded, "empty": batch > 2 and not padded and rng.random() < 0.5}
    if op == "rope":
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 3])
        d = rng.choice([32, 48, 64, 80, 96, 128])
        n = _log(rng, 1, max(2, 319057 * 2048 // ((hq + hk) * d) // 4))
        return {"op": "rope", "train": rng.random() < 0.7, "dtype": rng.choice(["bf16", "f16", "f32"]), "n": n,
                "hq": hq, "hk": hk, "d": d, "halves": rng.random() < 0.5, "shared": rng.random() < 0.5}
    width = 8 * _log(rng, 4, 100)
    blocks = rng.randint(1, 6)
    while _sizes({"width": width, "blocks": blocks})[1] > 60_000_000:
        blocks -= 1
    dtype = rng.choice(["bf16", "f16", "f32"])
    return {"op": "adamw", "dtype": dtype, "bits": rng.choice([8, 32]), "master": dtype != "f32" and rng.random() < 0.7,
            "width": width, "blocks": blocks}


# ------------------------------------------------------------------ shapes of a case
def _split(total, parts):
    """`total` rows over `parts` samples, mildly uneven, the same for every seed."""
    w = [1.0 + 0.25 * ((3 * i) % 5) for i in range(parts)]
    cuts = [int(round(total * sum(w[:i]) / sum(w))) for i in range(parts + 1)]
    return [cuts[i + 1] - cuts[i] for i in range(parts)]


def _lengths(c):
    """Queries of each sample, key rows of each sample, and how many of those rows are valid."""
    lq = _split(c["n_q"], c["batch"])
    if c["padded"]:
        rows = [c["n_k"] // c["batch"]] * c["batch"]
        valid = [r - (r * ((2 * i + 1) % 4)) // 7 for i, r in enumerate(rows)]
    else:
        rows = _split(c["n_k"], c["batch"])
        if c["empty"]:                       # the second sample's states go to the first
            rows[0], rows[1] = rows[0] + rows[1], 0
        valid = list(rows)
    return lq, rows, valid


def _sizes(c):
    """Element counts of the optimizer's tensors, and their padded total."""
    w = c["width"]
    sizes = [n for _ in range(c["blocks"]) for n in (27 * w * w, w, w * w, w * w, w * w, w * w, 2 * w)] + [7 * w + 3]
    return sizes, sum(-(-n // BLOCK) * BLOCK for n in sizes)


def work(c):
    if c["op"] == "attn":
        lq, rows, valid = _lengths(c)
        es, hq, hk, d = ES[c["dtype"]], c["hq"], c["hk"], c["d"]
        pairs = sum(a * b for a, b in zip(lq, valid)) * hq * d
        nq, nk = sum(lq), sum(valid)
        nbytes = es * d * (2 * nq * hq + 2 * nk * hk) + 4 * nq * hq
        if c["train"]:
            nbytes += es * d * (2 * nq * hq + 2 * sum(rows) * hk)
        return {"bytes": nbytes, "flops": (14 if c["train"] else 4) * pairs}
    if c["op"] == "rope":
        x = c["n"] * (c["hq"] + c["hk"]) * c["d"]
        passes = 4 if c["train"] else 2      # x and dy read, y and dx written
        return {"bytes": passes * x * ES[c["dtype"]] + 16 * c["n"], "flops": (20 if c["train"] else 8) * x}
    sizes, _ = _sizes(c)
    n = sum(sizes)
    per = 3 * ES[c["dtype"]] + (8 if c["master"] else 0)
    per += 16 if c["bits"] == 32 else 4 + 16 / BLOCK + 8        # 8-bit states come back as values
    return {"bytes": per * n, "flops": 16 * n}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _offsets(lengths):
    t = torch.zeros(len(lengths) + 1, dtype=torch.int32)
    t[1:] = torch.tensor(lengths, dtype=torch.int32).cumsum(0)
    return t.cuda()


def prepare(c, seed):
    g = _gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    st = {"case": c}
    if c["op"] == "attn":
        dt = DT[c["dtype"]]
        lq, rows, valid = _lengths(c)
        nq, nk = sum(lq), sum(rows)
        st["lq"], st["rows"], st["valid"] = lq, rows, valid
        st["q"] = rnd(nq, c["hq"], c["d"]).to(dt)
        kv = rnd(nk, 2, c["hk"], c["d"]).to(dt)                  # one projection gives keys and values
        st["k"], st["v"] = kv[:, 0], kv[:, 1]
        st["q_offsets"], st["k_offsets"] = _offsets(lq), _offsets(rows)
        st["k_lens"] = torch.tensor(valid, dtype=torch.int32).cuda() if c["padded"] else None
        st["scale"] = c["d"] ** -0.5
        st["out"], st["lse"] = torch.empty_like(st["q"]), torch.empty(c["hq"], nq, device="cuda")
        if c["train"]:
            st["grad_out"] = rnd(nq, c["hq"], c["d"]).to(dt)
            st["grad_q"] = torch.empty_like(st["q"])
            st["grad_kv"] = torch.empty(nk, 2, c["hk"], c["d"], dtype=dt, device="cuda")
            st["grad_k"], st["grad_v"] = st["grad_kv"][:, 0], st["grad_kv"][:, 1]
        if own:
            from voxel_gemm_gb300 import ops
            st["ws"] = ops.cross_attn_workspace(nq, nk, c["batch"], c["hq"], c["hk"], c["d"], dt, backward=c["train"])
    elif c["op"] == "rope":
        dt, n, d = DT[c["dtype"]], c["n"], c["d"]
        h = c["hq"] + c["hk"]
        qkv = (rnd(n, h + c["hk"], d) * 1.5).to(dt)              # the projection's packed output
        st["q"], st["k"] = qkv[:, :c["hq"]], qkv[:, c["hq"]:h]
        shape = (lambda m: (d,)) if c["shared"] else (lambda m: (m, d))
        st["q_weight"] = (1 + 0.2 * rnd(*shape(c["hq"]))).to(dt)
        st["k_weight"] = (1 + 0.2 * rnd(*shape(c["hk"]))).to(dt)
        st["coords"] = torch.randint(0, 256, (n, 4), generator=g, device="cuda", dtype=torch.int32)
        p = d // 6
        st["axis_pairs"] = (p, p, p)
        one = THETA ** (-torch.arange(p, dtype=torch.float64) / p)
        st["freqs"] = one.repeat(3).float().cuda()
        st["q_out"], st["k_out"] = (torch.empty(n, m, d, dtype=dt, device="cuda") for m in (c["hq"], c["hk"]))
        if c["train"]:
            st["gq_out"], st["gk_out"] = (rnd(n, m, d).to(dt) for m in (c["hq"], c["hk"]))
            st["gq"], st["gk"] = torch.empty_like(st["q_out"]), torch.empty_like(st["k_out"])
            st["gqw"], st["gkw"] = torch.empty_like(st["q_weight"]), torch.empty_like(st["k_weight"])
        if own and c["train"]:
            from voxel_gemm_gb300 import ops
            st["ws"] = ops.qk_norm_rope_workspace(n, c["hq"], c["hk"], d)
    else:
        dt = DT[c["dtype"]]
        sizes, total = _sizes(c)
        real = torch.zeros(total, device="cuda")                 # 1 where the arena holds a parameter
        views, at, wd, decays = [], 0, [], []
        for i, n in enumerate(sizes):
            real[at:at + n] = 1
            views.append((at, n))
            decays.append(0.0 if n <= 2 * c["width"] else 0.01)  # biases and norm weights decay by nothing
            nb = -(-n // BLOCK)
            wd += [torch.full((nb,), decays[-1], dtype=torch.float64)]
            at += nb * BLOCK
        p = rnd(total) * 0.05 * real
        st["param"] = p.to(dt)
        spikes = 1 + 9 * (torch.rand(total, generator=g, device="cuda") < 0.01)
        st["grad"] = (rnd(total) * 1e-3 * spikes * real).to(dt)
        st["master"] = p if c["master"] else None
        m = rnd(total) * 3e-4 * real
        v = (rnd(total) * 1e-3 * real) ** 2 + 1e-9 * real
        st["wd"] = torch.cat(wd).cuda()[:, None]
        st["hyper"] = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "step": 101}
        st["m"], st["v"], st["m_scale"], st["v_scale"] = m, v, None, None
        if c["bits"] == 8:
            st["m"], st["m_scale"] = _encode_m(m)
            st["v"], st["v_scale"] = _encode_u(v.sqrt())
            st["m_value"], st["v_value"] = torch.empty(total, device="cuda"), torch.empty(total, device="cuda")
        if own:
            from voxel_gemm_gb300 import ops
            cut = lambda t: None if t is None else [t[a:a + n] for a, n in views]  # noqa: E731
            st["opt"] = ops.AdamWState(cut(st["param"]), cut(st["grad"]), masters=cut(st["master"]), bits=c["bits"],
                                       weight_decay=decays, m=st["m"], v=st["v"], m_scale=st["m_scale"],
                                       v_scale=st["v_scale"])
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if op == "attn":
        return _attn_own(st) if own else _attn_plain(st)
    if op == "rope":
        return _rope_own(st) if own else _rope_plain(st)
    return _adamw_own(st) if own else _adamw_plain(st)


def _attn_own(st):
    from voxel_gemm_gb300 import ops
    ops.vg_cross_attn_fwd(st["q"], st["k"], st["v"], st["q_offsets"], st["k_offsets"], st["k_lens"], st["out"],
                          st["lse"], st["ws"], scale=st["scale"])
    if not st["case"]["train"]:
        return {"out": st["out"], "lse": st["lse"]}
    ops.vg_cross_attn_bwd(st["q"], st["k"], st["v"], st["q_offsets"], st["k_offsets"], st["k_lens"], st["out"],
                          st["lse"], st["grad_out"], st["grad_q"], st["grad_k"], st["grad_v"], st["ws"],
                          scale=st["scale"])
    return {"out": st["out"], "lse": st["lse"], "grad_q": st["grad_q"], "grad_kv": st["grad_kv"]}


def _rope_own(st):
    from voxel_gemm_gb300 import ops
    flags = ops.VG_ROPE_HALVES if st["case"]["halves"] else 0
    pos = (st["q_weight"], st["k_weight"], st["coords"], st["freqs"], st["axis_pairs"])
    ops.vg_qk_norm_rope_fwd(st["q"], st["k"], *pos, st["q_out"], st["k_out"], eps=1e-6, flags=flags)
    if not st["case"]["train"]:
        return {"q": st["q_out"], "k": st["k_out"]}
    ops.vg_qk_norm_rope_bwd(st["q"], st["k"], *pos, st["gq_out"], st["gk_out"], st["gq"], st["gk"], st["gqw"],
                            st["gkw"], st["ws"], eps=1e-6, flags=flags)
    return {"q": st["q_out"], "k": st["k_out"], "grad_q": st["gq"], "grad_k": st["gk"], "grad_q_weight": st["gqw"],
            "grad_k_weight": st["gkw"]}


def _adamw_own(st):
    from voxel_gemm_gb300 import ops
    h = st["hyper"]
    ops.vg_adamw_step(st["opt"], h["step"], h["lr"], h["beta1"], h["beta2"], h["eps"])
    out = {"param": st["param"]}
    if st["master"] is not None:
        out["master"] = st["master"]
    if st["case"]["bits"] == 32:
        return {**out, "m": st["m"], "v": st["v"]}
    ops.vg_adamw_decode(st["m"], st["m_scale"], st["m_value"], second=False)
    ops.vg_adamw_decode(st["v"], st["v_scale"], st["v_value"], second=True)
    return {**out, "m": st["m_value"], "v": st["v_value"]}


# ------------------------------------------------------------------ plain forms (32 bits)
def _rows(lengths, offsets, total):
    """Row index [B, longest] of every (sample, position) and whether there is such a position."""
    pos = torch.arange(max(1, max(lengths)), device="cuda")
    have = pos[None, :] < torch.tensor(lengths, device="cuda")[:, None]
    return (offsets[:-1, None].long() + pos[None, :]).clamp_(max=max(0, total - 1)), have


def _attn_plain(st):
    c, scale = st["case"], st["scale"]
    hq, hk, d, b = c["hq"], c["hk"], c["d"], c["batch"]
    nq, nk = sum(st["lq"]), sum(st["rows"])
    iq, hq_ok = _rows(st["lq"], st["q_offsets"], nq)
    ik, hk_ok = _rows(st["valid"], st["k_offsets"], nk)
    lq, lk, gr = iq.shape[1], ik.shape[1], hq // hk

    def queries(t):                              # [nq, hq, d] -> [b, hk, gr * lq, d], absent rows zero
        x = t.float()[iq] * hq_ok[:, :, None, None]
        return x.view(b, lq, hk, gr, d).permute(0, 2, 3, 1, 4).reshape(b, hk, gr * lq, d)

    def keys(t):                                 # [nk, hk, d] -> [b, hk, lk, d], absent rows zero
        return torch.where(hk_ok[:, :, None, None], t.float()[ik], 0.0).permute(0, 2, 1, 3).contiguous()

    def back(x):                                 # the reverse of queries()
        y = x.view(b, hk, gr, lq, d).permute(0, 3, 1, 2, 4).reshape(b, lq, hq, d)
        return y[hq_ok]

    q, k, v = queries(st["q"]), keys(st["k"]), keys(st["v"])
    dead = ~hk_ok[:, None, None, :]
    s = (q @ k.transpose(2, 3)).mul_(scale).masked_fill_(dead, -math.inf)
    top = s.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    p.div_(torch.where(total == 0, 1.0, total))
    out = p @ v
    lse = (total.log() + top).view(b, hk, gr, lq).permute(1, 2, 0, 3).reshape(hq, b, lq)[:, hq_ok]
    res = {"out": back(out).to(st["q"].dtype), "lse": lse}
    if not c["train"]:
        return res
    do = queries(st["grad_out"])
    dv = p.transpose(2, 3) @ do
    dp = do @ v.transpose(2, 3)
    ds = dp.sub_((do * out).sum(3, keepdim=True)).mul_(p).mul_(scale)
    dq, dk = ds @ k, ds.transpose(2, 3) @ q
    res["grad_q"] = back(dq).to(st["q"].dtype)
    gkv = torch.zeros(nk, 2, hk, d, device="cuda")
    gkv[ik[hk_ok]] = torch.stack([dk, dv], 1).permute(0, 3, 1, 2, 4)[hk_ok]
    res["grad_kv"] = gkv.to(st["q"].dtype)
    return res


def _pairs(x, halves):
    """The two members of every rotated pair, [..., d / 2] each."""
    d = x.shape[-1]
    return (x[..., :d // 2], x[..., d // 2:]) if halves else (x[..., 0::2], x[..., 1::2])


def _joined(a, b, halves):
    return torch.cat([a, b], -1) if halves else torch.stack([a, b], -1).flatten(-2)


def _angles(st):
    """cos and sin [n, 1, d / 2]; pairs without a frequency are not turned."""
    pos = st["coords"][:, 1:].float().repeat_interleave(torch.tensor(st["axis_pairs"], device="cuda"), 1)
    ang = pos * st["freqs"]
    ang = torch.cat([ang, ang.new_zeros(ang.shape[0], st["case"]["d"] // 2 - ang.shape[1])], 1)[:, None]
    return ang.cos(), ang.sin()


def _rope_plain(st):
    c = st["case"]
    halves, dt = c["halves"], st["q"].dtype
    cos, sin = _angles(st)

    def forward(x, w):
        x = x.float()
        n = x * torch.rsqrt((x * x).mean(2, keepdim=True) + 1e-6) * w.float()
        a, b = _pairs(n, halves)
        return _joined(a * cos - b * sin, a * sin + b * cos, halves).to(dt)

    def backward(x, w, gy):
        x, w = x.float(), w.float()
        r = torch.rsqrt((x * x).mean(2, keepdim=True) + 1e-6)
        a, b = _pairs(gy.float(), halves)
        g = _joined(a * cos + b * sin, b * cos - a * sin, halves)
        xh = x * r
        gw = (g * xh).sum(0)
        gx = r * (g * w - xh * (g * w * xh).mean(2, keepdim=True))
        return gx.to(dt), (gw.sum(0) if w.dim() == 1 else gw).to(dt)

    res = {"q": forward(st["q"], st["q_weight"]), "k": forward(st["k"], st["k_weight"])}
    if c["train"]:
        res["grad_q"], res["grad_q_weight"] = backward(st["q"], st["q_weight"], st["gq_out"])
        res["grad_k"], res["grad_k_weight"] = backward(st["k"], st["k_weight"], st["gk_out"])
    return res


def _scale_of(x, top):
    """Power-of-two scale [blocks, 1] that puts each block's largest finite value into [2^top, 2^(top + 1))."""
    big = torch.where(x.isfinite(), x.abs(), 0.0).amax(1, keepdim=True)
    e = (torch.frexp(big)[1] - 1 - top).clamp(-100, 120)
    return torch.where(big > 0, torch.ldexp(torch.ones_like(big), e), 1.0)


def _encode_m(m):
    """First moments as 8-bit floats (sign, 4 exponent, 3 mantissa bits) times a block's scale; not finite: NaN."""
    x = m.view(-1, BLOCK)
    s = _scale_of(x, 7)
    y = (x * (1 / s)).abs()
    bits = y.clamp(min=2.0 ** -6).view(torch.int32)
    t = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - (120 << 3)
    t = torch.where(y < 2.0 ** -6, (y * 512).round(), t)         # steps of 2^-9 below the normal range
    t = torch.where(x.isfinite(), t, 127) + 128 * torch.signbit(x)
    return t.to(torch.uint8).view(-1), s.view(-1).contiguous()


def _decode_m(code, scale):
    return code.view(torch.float8_e4m3fn).float().view(-1, BLOCK) * scale[:, None]


def _encode_u(u):
    """Square roots of second moments: code 0 is zero, codes 1 to 254 are (1 + j / 16) 2^i, 255 is NaN."""
    x = u.view(-1, BLOCK)
    s = _scale_of(x, 14)
    y = x * (1 / s)
    bits = y.clamp(min=1.0).view(torch.int32)
    t = ((bits + 0x3FFFF + ((bits >> 19) & 1)) >> 19) - (127 << 4) + 1
    t = torch.where(x.isfinite(), torch.where(y > 0, t, 0), 255)
    return t.to(torch.uint8).view(-1), s.view(-1).contiguous()


def _decode_u(code, scale):
    c = code.view(-1, BLOCK).int()
    x = (((c - 1) + (127 << 4)) << 19).view(torch.float32)
    x = torch.where(c == 0, 0.0, torch.where(c == 255, math.nan, x))
    return x * scale[:, None]


def _adamw_plain(st):
    h, c = st["hyper"], st["case"]
    b1, b2, lr, t = h["beta1"], h["beta2"], h["lr"], h["step"]
    small = c["bits"] == 8
    m = _decode_m(st["m"], st["m_scale"]) if small else st["m"].view(-1, BLOCK)
    v = _decode_u(st["v"], st["v_scale"]).square() if small else st["v"].view(-1, BLOCK)
    p = (st["master"] if c["master"] else st["param"].float()).view(-1, BLOCK)
    g = st["grad"].float().view(-1, BLOCK)
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    u = v.sqrt()
    decay = (1 - lr * st["wd"]).float()
    p = p * decay - (m / (u * (1 / math.sqrt(1 - b2 ** t)) + h["eps"])) * (lr / (1 - b1 ** t))
    st["param"].copy_(p.view(-1))
    res = {"param": st["param"]}
    if c["master"]:
        st["master"].copy_(p.view(-1))
        res["master"] = st["master"]
    if not small:
        st["m"].copy_(m.view(-1))
        st["v"].copy_(v.view(-1))
        return {**res, "m": st["m"], "v": st["v"]}
    st["m"], st["m_scale"] = _encode_m(m)
    st["v"], st["v_scale"] = _encode_u(u)
    return {**res, "m": _decode_m(st["m"], st["m_scale"]).view(-1),
            "v": _decode_u(st["v"], st["v_scale"]).square().view(-1)}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "attn":
        return _attn_exact(st)
    return _rope_exact(st) if c["op"] == "rope" else _adamw_exact(st)


def _attn_exact(st):
    c = st["case"]
    q, k, v = (st[x].double() for x in ("q", "k", "v"))
    nq, hq, d = q.shape
    gr = hq // c["hk"]
    out, lse = torch.zeros_like(q), torch.full((hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(q)
    dkv = torch.zeros(k.shape[0], 2, *k.shape[1:], dtype=torch.float64, device="cuda")
    do = st["grad_out"].double() if c["train"] else None
    a = o = 0
    for n, rows, keys in zip(st["lq"], st["rows"], st["valid"]):
        for h in range(hq if n and keys else 0):
            qs, ks, vs = q[a:a + n, h], k[o:o + keys, h // gr], v[o:o + keys, h // gr]
            prob = torch.einsum("id,jd->ij", qs, ks).mul_(st["scale"])
            lse[h, a:a + n] = torch.logsumexp(prob, 1)
            prob.sub_(lse[h, a:a + n, None]).exp_()
            out[a:a + n, h] = prob @ vs
            if c["train"]:
                gs = do[a:a + n, h]
                dkv[o:o + keys, 1, h // gr] += prob.t() @ gs
                prob.mul_(gs @ vs.t() - (gs * out[a:a + n, h]).sum(1, keepdim=True))
                dq[a:a + n, h] = prob @ ks * st["scale"]
                dkv[o:o + keys, 0, h // gr] += prob.t() @ qs * st["scale"]
        a, o = a + n, o + rows
    return {"out": out, "lse": lse, "grad_q": dq, "grad_kv": dkv} if c["train"] else {"out": out, "lse": lse}


def _rope_exact(st):
    """Each pair as a complex number; its rotation is a product with exp(i angle)."""
    c = st["case"]
    d, n = c["d"], c["n"]
    turn = torch.zeros(n, d // 2, dtype=torch.float64, device="cuda")
    at = 0
    for axis, count in enumerate(st["axis_pairs"]):
        turn[:, at:at + count] = st["coords"][:, 1 + axis, None].double() * st["freqs"][at:at + count].double()
        at += count
    rot = torch.polar(torch.ones_like(turn), turn)
    order = torch.arange(d, device="cuda")
    order = torch.stack([order[:d // 2], order[d // 2:]], 1) if c["halves"] else order.view(-1, 2)

    def turned(x, by):
        y = torch.view_as_real(torch.view_as_complex(x[:, order].contiguous()) * by)
        z = torch.empty_like(x)
        z[:, order] = y
        return z

    res = {}
    for name in ("q", "k"):
        x, w = st[name].double(), st[name + "_weight"].double()
        gw = torch.zeros_like(w)
        y, gx = torch.empty_like(x), torch.empty_like(x)
        for h in range(x.shape[1]):
            xs, ws = x[:, h], w if w.dim() == 1 else w[h]
            rms = (xs.square().mean(1, keepdim=True) + 1e-6).sqrt()
            y[:, h] = turned(xs / rms * ws, rot)
            if c["train"]:
                gn = turned(st["g%s_out" % name][:, h].double(), rot.conj())
                (gw if w.dim() == 1 else gw[h]).add_((gn * xs / rms).sum(0))
                gn = gn * ws
                gx[:, h] = gn / rms - xs * (gn * xs).mean(1, keepdim=True) / rms ** 3
        res[name] = y
        if c["train"]:
            res["grad_" + name], res["grad_%s_weight" % name] = gx, gw
    return res


def _adamw_exact(st):
    h, c = st["hyper"], st["case"]
    t = h["step"]
    if c["bits"] == 8:
        m = st["m"].view(torch.float8_e4m3fn).double() * st["m_scale"].double().repeat_interleave(BLOCK)
        code = st["v"].long()
        u = 2.0 ** ((code - 1) // 16).double() * (1 + ((code - 1) % 16).double() / 16)
        v = (torch.where(code == 0, 0.0, u) * st["v_scale"].double().repeat_interleave(BLOCK)) ** 2
    else:
        m, v = st["m"].double(), st["v"].double()
    g = st["grad"].double()
    p = st["master"].double() if c["master"] else st["param"].double()
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
    step = (m / (1 - h["beta1"] ** t)) / ((v / (1 - h["beta2"] ** t)).sqrt() + h["eps"])
    p = p - h["lr"] * st["wd"].repeat_interleave(BLOCK, 1).view(-1) * p - h["lr"] * step
    if c["bits"] == 8:
        # 0.9 m + 0.1 g of a coarse m and a 16-bit g often falls half-way between two values: 32 and 64 bits then
        # round to different sides (about 1 % of the first moments at a bf16 gradient)
        m = _near(m, 7, 3, -6)
        v = _near(v.sqrt(), 14, 4, 0) ** 2
    res = {"param": p, "m": m, "v": v}
    if c["master"]:
        res["master"] = p
    return res


def _near(x, top, bits, low):
    """x in blocks, each value at the nearest one with `bits` mantissa bits and exponents from `low` on, where the
    block's largest has the exponent `top`; with low = 0 nothing but zero goes to zero."""
    x = x.view(-1, BLOCK)
    lead = torch.frexp(x.abs().amax(1, keepdim=True))[1].double() - 1
    scale = 2.0 ** (lead - top)
    y = x / scale
    e = (torch.frexp(y)[1].double() - 1).clamp(min=low)
    unit = 2.0 ** (e - bits)
    z = torch.round(y / unit) * unit
    if low == 0:
        z = torch.where((y > 0) & (y < 1), 1.0, z)
    return (z * scale).view(-1)
