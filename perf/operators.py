"""The operators around the layer step that are measured: the norm and rotation
of queries and keys, dropout with bias and residual, and the log probability
of given tokens, each in both directions.

`run` computes them from elementary torch operations in 32 bits (angles in 64)
where `own` is false, and calls the library where it is true.
"""
import functools
import math

import numpy as np
import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------- cases
def _qk(op, dtype, tokens, groups, q, k, v, hd, rot, inter=False, axes=1, seq=0, far=4096):
    """seq > 0: positions are the token index modulo seq; else they are given, up to `far`."""
    return dict(op=op, dtype=dtype, tokens=tokens, groups=groups, q_heads=q, k_heads=k, v_heads=v,
                head_dim=hd, rot_dim=rot, interleaved=inter, axes=axes, seq=seq, far=far)


def _drop(op, dtype, rows, h, p, f32, bias):
    """f32: the residual stream (forward: resid and y; backward: dy) is held in 32 bits."""
    return dict(op=op, dtype=dtype, rows=rows, h=h, p=p, f32=f32, bias=bias)


def _lp(op, dtype, rows, vocab, ld, top_k=0, mask="none", entropy=True):
    return dict(op=op, dtype=dtype, rows=rows, vocab=vocab, ld=ld, top_k=top_k, mask=mask,
                entropy=entropy)


def listed():
    named = [
        # one generation step of 16 sequences deep in long contexts: latency
        ("qk step of 16 tokens", _qk("qk_fwd", "bf16", 16, 1, 32, 8, 0, 128, 128, far=131072)),
        # the 345M layer's forward, all four shards, V carried along to attention's buffer
        ("qk fwd 8192 x 1024", _qk("qk_fwd", "fp16", 8192, 4, 4, 4, 4, 64, 64, seq=1024)),
        # video tokens with (time, height, width), a ragged count, part of each head rotated
        ("qk bwd 5003 video", _qk("qk_bwd", "bf16", 5003, 1, 32, 8, 8, 80, 64, inter=True, axes=3)),
        # the hidden-10240 layer's backward
        ("qk bwd 2048 x 10240", _qk("qk_bwd", "bf16", 2048, 4, 20, 20, 0, 128, 128, seq=2048)),
        # the tiny layer: latency
        ("dropout fwd 128 x 128", _drop("drop_fwd", "fp16", 128, 128, 0.1, True, True)),
        # the hidden-10240 layer's residual stream
        ("dropout fwd 2048 x 10240", _drop("drop_fwd", "bf16", 2048, 10240, 0.1, True, True)),
        # the 2.4B layer's row-split products in the backward, with their bias gradient
        ("dropout bwd 8192 x 2560", _drop("drop_bwd", "fp16", 8192, 2560, 0.1, False, True)),
        # odd sizes, gradients of a 32-bit residual stream
        ("dropout bwd 777 x 1096", _drop("drop_bwd", "bf16", 777, 1096, 0.25, True, True)),
        # a generation step of 5 sequences: top alternatives among an odd vocabulary
        ("logprob step of 5 tokens", _lp("lp_fwd", "bf16", 5, 50257, 50257, 20, "inf")),
        # scoring a prompt from 32-bit logits
        ("logprob fwd 1000 x 32000", _lp("lp_fwd", "fp32", 1000, 32000, 32000, 5)),
        # the loss of a whole batch of the 117M and 345M configurations, columns padded
        ("logprob fwd 8192 x 50257", _lp("lp_fwd", "bf16", 8192, 50257, 50304)),
        # its gradient over rows of odd length, with an entropy term
        ("logprob bwd 4096 x 50257", _lp("lp_bwd", "bf16", 4096, 50257, 50257)),
    ]
    return [dict(case, name=name) for name, case in named]


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["qk_fwd", "qk_bwd", "drop_fwd", "drop_bwd", "lp_fwd", "lp_bwd"])
    dtype = rng.choice(["fp16", "bf16"])
    if op.startswith("qk"):
        hd = 16 * rng.randint(1, 16)
        q = _log(rng, 1, 48)
        k = rng.choice([q, max(1, q // 4), 1])
        groups = rng.choice([1, 1, 2, 4])
        v = rng.choice([0, k])
        most = 40_000_000 // (groups * (q + k + v) * hd)
        return _qk(op, dtype, _log(rng, 1, max(1, min(8192, most))), groups, q, k, v, hd,
                   16 * rng.randint(0 if rng.random() < 0.2 else 1, hd // 16), rng.random() < 0.5,
                   rng.choice([1, 1, 2, 3, 4]), rng.choice([0, 0, 128, 1024]),
                   rng.choice([4096, 131072, 1 << 20]))
    if op.startswith("drop"):
        rows = _log(rng, 1, 16384)
        return _drop(op, dtype, rows, 8 * _log(rng, 1, min(1280, 20_000_000 // (8 * rows))),
                     rng.choice([0.0, 0.1, round(rng.uniform(0.01, 0.6), 3)]), rng.random() < 0.5,
                     rng.random() < 0.7)
    dtype = rng.choice(["fp16", "bf16", "fp32"])
    vocab = _log(rng, 2, 152_000)
    most = (400_000_000 if op == "lp_fwd" else 200_000_000) // vocab // (2 if dtype == "fp32" else 1)
    rows = _log(rng, 1, min(8192, most))
    top_k = rng.randint(0, min(32, vocab // 2)) if op == "lp_fwd" and rows <= 2048 else 0
    return _lp(op, dtype, rows, vocab, rng.choice([vocab, vocab + rng.randint(0, 64)]), top_k,
               rng.choice(["none", "inf", "low"]), rng.random() < 0.7)


def work(case):
    c, es = case, SIZE[case["dtype"]]
    if c["op"].startswith("qk"):
        rows = c["tokens"] * c["groups"]
        qk, v = rows * (c["q_heads"] + c["k_heads"]) * c["head_dim"], rows * c["v_heads"] * c["head_dim"]
        n = 2 if c["op"] == "qk_fwd" else 3
        return {"bytes": es * (n * qk + 2 * v), "flops": (8 if n == 2 else 18) * qk}
    if c["op"].startswith("drop"):
        n, stream = c["rows"] * c["h"], 4 if c["f32"] else es
        return {"bytes": n * (es + (2 if c["op"] == "drop_fwd" else 1) * stream), "flops": 4 * n}
    n = c["rows"] * c["vocab"]
    if c["op"] == "lp_fwd":
        return {"bytes": n * es + c["rows"] * (20 + 8 * c["top_k"]), "flops": 6 * n}
    return {"bytes": 2 * n * es + 24 * c["rows"], "flops": 6 * n}


# ------------------------------------------------------------------ inputs
def _sections(rot_dim, axes):
    """Pairs of each axis: time gets the smallest share where there are several."""
    pairs, rest = rot_dim // 2, []
    for a in range(axes - 1, 0, -1):
        rest.append(-(-(pairs - sum(rest)) // (a + 1)))
    return [pairs - sum(rest)] + rest[::-1]


def _prepare_qk(c, g):
    dev, dt = "cuda", DT[c["dtype"]]
    T, G, hd = c["tokens"], c["groups"], c["head_dim"]
    heads = c["q_heads"] + c["k_heads"] + c["v_heads"]
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    s = {"case": c, "x": (rand(G, T, heads * hd) * 1.5).to(dt)}
    s["gq"], s["gk"] = (1 + 0.2 * rand(hd)).to(dt), (1 + 0.2 * rand(hd)).to(dt)
    pairs = c["rot_dim"] // 2
    # a pair's turns for each position, base 10000, and its axis, 16 bytes for each pair
    table = torch.zeros(max(pairs, 1), 2, dtype=torch.float64, device=dev)
    j = torch.arange(pairs, dtype=torch.float64, device=dev)
    table[:pairs, 0] = torch.pow(10000.0, -j / max(pairs, 1)) / (2 * math.pi)
    axis = [a for a, n in enumerate(_sections(c["rot_dim"], c["axes"])) for _ in range(n)]
    table.view(torch.int32)[:pairs, 2] = torch.tensor(axis, dtype=torch.int32, device=dev)
    s["table"] = table
    s["axis"] = torch.tensor(axis, dtype=torch.int64, device=dev)
    s["pos"] = None
    if not c["seq"]:
        s["pos"] = torch.randint(0, c["far"], (c["axes"], T), generator=g, device=dev, dtype=torch.int32)
    s["out"] = torch.empty_like(s["x"])
    if c["op"] == "qk_bwd":
        s["dy"] = rand(G, T, heads * hd).to(dt)
        s["dgq"] = torch.empty(hd, device=dev)
        s["dgk"] = torch.empty(hd, device=dev)
    if own:
        from transformer_layer_step_b200 import gptlayer as G_
        s["G"] = G_
        s["desc"] = G_.make_qk_desc(tokens=T, groups=G, q_heads=c["q_heads"], k_heads=c["k_heads"],
                                    v_heads=c["v_heads"], head_dim=hd, rot_dim=c["rot_dim"],
                                    interleaved=c["interleaved"], axes=c["axes"], seq=c["seq"],
                                    eps=1e-6)
        if c["op"] == "qk_bwd":
            s["scratch"] = torch.empty(G_.qk_norm_rope_scratch_bytes(s["desc"]), dtype=torch.uint8,
                                       device=dev)
    return s


def _prepare_drop(c, g):
    dev, dt = "cuda", DT[c["dtype"]]
    st = torch.float32 if c["f32"] else dt
    rows, h = c["rows"], c["h"]
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    s = {"case": c, "site": 5}
    s["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device=dev, dtype=torch.int64)
    if c["op"] == "drop_fwd":
        s["x"], s["resid"] = rand(rows, h).to(dt), (2 * rand(rows, h)).to(st)
        s["bias"] = (0.1 * rand(h)).to(dt) if c["bias"] else None
        s["y"] = torch.empty(rows, h, dtype=st, device=dev)
    else:
        s["dy"] = rand(rows, h).to(st)
        s["dx"] = torch.empty(rows, h, dtype=dt, device=dev)
        s["dbias"] = torch.empty(h, device=dev) if c["bias"] else None
    if own:
        from transformer_layer_step_b200 import gptlayer as G_
        s["G"] = G_
        if c["op"] == "drop_bwd":
            s["scratch"] = torch.empty(G_.dropout_scratch_bytes(rows, h), dtype=torch.uint8, device=dev)
    return s


def _prepare_lp(c, g):
    dev, dt = "cuda", DT[c["dtype"]]
    rows, V = c["rows"], c["vocab"]
    col = torch.arange(V, device=dev)
    target = torch.randint(0, V, (rows,), generator=g, device=dev, dtype=torch.int32)
    target -= (target % 3 == 1).int()                       # never a masked column
    logits = torch.full((rows, c["ld"]), 1e4, dtype=dt, device=dev)
    step = max(1, 200_000_000 // V)
    for r in range(0, rows, step):
        x = 2.5 * torch.randn(min(step, rows - r), V, generator=g, device=dev)
        t = target[r:r + step, None].long()
        x.scatter_add_(1, t, 5 * (t % 2).float())           # half of the targets are likely ones
        if c["mask"] != "none":
            x[:, col % 3 == 1] = -math.inf if c["mask"] == "inf" else torch.finfo(dt).min
        logits[r:r + step, :V] = x.to(dt)
    target[torch.arange(rows, device=dev) % 29 == 7] = -1   # rows without a target
    s = {"case": c, "logits": logits, "target": target}
    if c["op"] == "lp_fwd":
        s["logp"], s["stats"] = torch.empty(rows, device=dev), torch.empty(rows, 2, device=dev)
        s["entropy"] = torch.empty(rows, device=dev) if c["entropy"] else None
        s["top_logp"] = s["top_id"] = None
        if c["top_k"]:
            s["top_logp"] = torch.empty(rows, c["top_k"], device=dev)
            s["top_id"] = torch.empty(rows, c["top_k"], dtype=torch.int32, device=dev)
    else:
        # what the forward left: the maximum, the log of the sum, the entropy
        m = logits[:, :V].amax(1).double()
        z, e = torch.empty_like(m), torch.empty_like(m)
        for r in range(0, rows, step):
            d = (logits[r:r + step, :V].double() - m[r:r + step, None]).clamp(min=-1e4)
            w = d.exp()
            z[r:r + step] = w.sum(1)
            e[r:r + step] = z[r:r + step].log() - (w * d).sum(1) / z[r:r + step]
        s["stats"] = torch.stack([m, z.log()], 1).float()
        s["entropy"] = e.float()
        s["dlogp"] = 16 * torch.randn(rows, generator=g, device=dev)
        s["dentropy"] = torch.randn(rows, generator=g, device=dev) if c["entropy"] else None
        s["dlogits"] = torch.empty_like(logits)
    if own:
        from transformer_layer_step_b200 import gptlayer as G_
        s["G"] = G_
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["op"].split("_")[0]
    return {"qk": _prepare_qk, "drop": _prepare_drop, "lp": _prepare_lp}[kind](case, g)


# ------------------------------------------------- queries and keys, plain
def _rotation(s):
    """cos and sin of every token's pairs, [tokens, pairs] in 32 bits."""
    c = s["case"]
    if s["pos"] is None:
        at = torch.arange(c["tokens"], device="cuda")[:, None] % c["seq"]
    else:
        at = s["pos"][s["axis"]].T
    turn = at.double() * s["table"][:c["rot_dim"] // 2, 0]
    angle = 2 * math.pi * (turn - turn.round())
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _rotate(n, cos, sin, c):
    """Rotates the leading rot_dim elements of each head by (cos, sin)."""
    R = c["rot_dim"]
    lead, rest = n[..., :R], n[..., R:]
    if c["interleaved"]:
        a, b = lead[..., 0::2], lead[..., 1::2]
        lead = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = lead[..., :R // 2], lead[..., R // 2:]
        lead = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([lead, rest], -1)


def _split(s, t):
    """A packed buffer's queries and keys, [groups, tokens, heads, head_dim] in 32 bits, and its V columns."""
    c = s["case"]
    t = t.unflatten(-1, (-1, c["head_dim"]))
    n = c["q_heads"] + c["k_heads"]
    return t[:, :, :n].float(), t[:, :, n:]


def _gains(s):
    c = s["case"]
    return torch.cat([s["gq"].float().expand(c["q_heads"], -1), s["gk"].float().expand(c["k_heads"], -1)])


def _plain_qk(s):
    c = s["case"]
    x, v = _split(s, s["x"])
    xh = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    cos, sin = _rotation(s)
    if c["op"] == "qk_fwd":
        y = _rotate(xh * _gains(s), cos, sin, c)
        return torch.cat([y.to(v.dtype), v], 2).flatten(-2)
    dy, dv = _split(s, s["dy"])
    dn = _rotate(dy, cos, -sin, c)
    dg = (dn * xh).sum((0, 1))
    dh = dn * _gains(s)
    dx = (dh - xh * (dh * xh).mean(-1, keepdim=True)) * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    q = c["q_heads"]
    return torch.cat([dx.to(dv.dtype), dv], 2).flatten(-2), dg[:q].sum(0), dg[q:].sum(0)


# ----------------------------------------------------------- dropout, plain
def _philox_round(at, _):
    """One round of Philox4x32 (Salmon et al., SC 2011) on int64 words below 2^32."""
    c0, c1, c2, c3, k0, k1 = at
    p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
    return ((p1 >> 32 & M32) ^ c1 ^ k0, p1 & M32, (p0 >> 32 & M32) ^ c3 ^ k1, p0 & M32,
            k0 + 0x9E3779B9 & M32, k1 + 0xBB67AE85 & M32)


def _kept(s):
    """Which of [rows, h] are kept, and what a kept one is multiplied by."""
    c = s["case"]
    drop = int(np.float32(c["p"]) * 65536 + 0.5)
    block = torch.arange(c["rows"] * c["h"] // 8, device="cuda")
    seed, offset = s["rng"][0], s["rng"][1]
    at = (block, torch.full_like(block, s["site"]), (offset & M32).expand_as(block),
          (offset >> 32 & M32).expand_as(block), seed & M32, seed >> 32 & M32)
    w = torch.stack(functools.reduce(_philox_round, range(10), at)[:4], -1)
    u = torch.stack([w & 0xFFFF, w >> 16], -1)
    return (u >= drop).view(c["rows"], c["h"]), 65536 / (65536 - drop)


def _plain_drop(s):
    keep, scale = _kept(s)
    if s["case"]["op"] == "drop_fwd":
        z = s["x"].float() if s["bias"] is None else s["x"].float() + s["bias"].float()
        return (s["resid"].float() + torch.where(keep, z * scale, 0.0)).to(s["y"].dtype)
    dx = torch.where(keep, s["dy"].float() * scale, 0.0)
    return dx.to(s["dx"].dtype), dx.sum(0) if s["case"]["bias"] else None


# ------------------------------------------------- log probabilities, plain
def _plain_lp(s):
    c = s["case"]
    x, t = s["logits"][:, :c["vocab"]].float(), s["target"].long()[:, None]
    given = t >= 0
    if c["op"] == "lp_fwd":
        m = x.amax(1, keepdim=True)
        d = x - m
        w = d.exp()
        z = w.sum(1, keepdim=True)
        lz = z.log()
        out = {"logp": torch.where(given, d.gather(1, t.clamp(min=0)) - lz, 0.0)[:, 0],
               "stats": torch.cat([m, lz], 1)}
        if c["entropy"]:
            out["entropy"] = (lz - torch.where(w > 0, w * d, 0.0).sum(1, keepdim=True) / z)[:, 0]
        if c["top_k"]:
            # order by value, then by lowest id: both in one whole number
            bits = x.view(torch.int32).long()
            bits = torch.where(x == 0, 0, bits)             # -0 equals 0
            key = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits) << 32
            key -= torch.arange(c["vocab"], device="cuda")
            top = key.topk(c["top_k"], 1).values
            out["top_id"] = (-top & M32).int()
            out["top_logp"] = d.gather(1, -top & M32) - lz
        return out
    m, lz = s["stats"][:, :1], s["stats"][:, 1:]
    lp = x - m - lz
    p = lp.exp()
    dlogp = torch.where(given, s["dlogp"][:, None], 0.0)
    g = -p * dlogp
    if c["entropy"]:
        g -= torch.where(p > 0, p * (lp + s["entropy"][:, None]), 0.0) * s["dentropy"][:, None]
    g.scatter_add_(1, t.clamp(min=0), dlogp)
    return g.to(s["logits"].dtype)


# --------------------------------------------------- the framework's calls
def _own_qk(s, st):
    G, c = s["G"], s["case"]
    if c["op"] == "qk_fwd":
        G.qk_norm_rope_fwd(s["desc"], c["dtype"], s["x"], s["out"], s["gq"], s["gk"], s["pos"],
                           s["table"], st)
        return s["out"]
    G.qk_norm_rope_bwd(s["desc"], c["dtype"], s["x"], s["dy"], s["out"], s["gq"], s["gk"], s["pos"],
                       s["table"], s["dgq"], s["dgk"], s["scratch"], st)
    return s["out"], s["dgq"], s["dgk"]


def _own_drop(s, st):
    G, c = s["G"], s["case"]
    if c["op"] == "drop_fwd":
        G.dropout_add_fwd(c["rows"], c["h"], c["dtype"], s["x"], s["bias"], s["resid"], c["f32"],
                          c["p"], s["rng"], s["site"], s["y"], c["f32"], st)
        return s["y"]
    G.dropout_add_bwd(c["rows"], c["h"], c["dtype"], s["dy"], c["f32"], c["p"], s["rng"], s["site"],
                      s["dx"], s["dbias"], s["scratch"], st)
    return s["dx"], s["dbias"]


def _own_lp(s, st):
    G, c = s["G"], s["case"]
    if c["op"] == "lp_fwd":
        G.token_logprob_fwd(c["rows"], c["vocab"], c["ld"], c["dtype"], s["logits"], s["target"],
                            s["logp"], s["entropy"], s["stats"], c["top_k"], s["top_logp"],
                            s["top_id"], st)
        out = {"logp": s["logp"], "stats": s["stats"]}
        if c["entropy"]:
            out["entropy"] = s["entropy"]
        if c["top_k"]:
            out["top_id"], out["top_logp"] = s["top_id"], s["top_logp"]
        return out
    G.token_logprob_bwd(c["rows"], c["vocab"], c["ld"], c["dtype"], s["logits"], s["target"],
                        s["stats"], s["entropy"], s["dlogp"], s["dentropy"], s["dlogits"], st)
    return s["dlogits"][:, :c["vocab"]]


def run(state):
    kind = state["case"]["op"].split("_")[0]
    if own:
        call = {"qk": _own_qk, "drop": _own_drop, "lp": _own_lp}[kind]
        return call(state, torch.cuda.current_stream().cuda_stream)
    return {"qk": _plain_qk, "drop": _plain_drop, "lp": _plain_lp}[kind](state)


# ----------------------------------------------------------- from 64 bits
def _exact_qk(s):
    """Rotation as the product with e^(i phi), group by group."""
    c = s["case"]
    hd, R, q = c["head_dim"], c["rot_dim"], c["q_heads"]
    n = q + c["k_heads"]
    rows = torch.arange(c["tokens"], dtype=torch.float64, device="cuda")
    place = [rows % c["seq"] if s["pos"] is None else s["pos"][a].double() for a in range(c["axes"])]
    phi = [2 * math.pi * ((place[a] * f) % 1.0) for a, f in zip(s["axis"].tolist(), s["table"][:, 0].tolist())]
    unit = torch.polar(torch.ones(c["tokens"], R // 2, dtype=torch.float64, device="cuda"),
                       torch.stack(phi, 1) if phi else torch.zeros(c["tokens"], 0, dtype=torch.float64, device="cuda"))

    def turned(v, u):
        T = c["tokens"]
        lead = v[:, :R].reshape(T, R // 2, 2) if c["interleaved"] else v[:, :R].reshape(T, 2, R // 2).mT
        w = torch.view_as_real(torch.view_as_complex(lead.contiguous()) * u)
        w = w.reshape(T, R) if c["interleaved"] else w.mT.reshape(T, R)
        return torch.cat([w, v[:, R:]], 1)

    out = s["x" if c["op"] == "qk_fwd" else "dy"].double()
    dg = [torch.zeros(hd, dtype=torch.float64, device="cuda") for _ in range(2)]
    for g in range(c["groups"]):
        for a in range(n):
            cols = slice(a * hd, (a + 1) * hd)
            x, gain = s["x"][g, :, cols].double(), (s["gq"] if a < q else s["gk"]).double()
            r = 1 / torch.sqrt((x * x).sum(1, keepdim=True) / hd + 1e-6)
            if c["op"] == "qk_fwd":
                out[g, :, cols] = turned(x * r * gain, unit)
                continue
            d = turned(out[g, :, cols].clone(), unit.conj())
            dg[a >= q] += (d * x * r).sum(0)
            d = d * gain
            out[g, :, cols] = r * d - x * r ** 3 * (d * x).sum(1, keepdim=True) / hd
    return out if c["op"] == "qk_fwd" else (out, dg[0], dg[1])


def _exact_keep(s):
    """The kept elements, from the generator's definition on unsigned words on the host."""
    c = s["case"]
    seed, offset = (int(v) for v in s["rng"].tolist())
    i = np.arange(c["rows"] * c["h"] // 8, dtype=np.uint64)
    low, cut = np.uint64(M32), np.uint64(32)
    x = [i, np.full_like(i, s["site"]), np.full_like(i, offset & M32), np.full_like(i, offset >> 32)]
    key = [seed & M32, seed >> 32]
    for _ in range(10):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> cut) ^ x[1] ^ np.uint64(key[0]), b & low, (a >> cut) ^ x[3] ^ np.uint64(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) & M32, (key[1] + 0xBB67AE85) & M32]
    u = np.stack([(w >> np.uint64(16 * half)) & np.uint64(0xFFFF) for w in x for half in (0, 1)], 1)
    drop = int(math.floor(float(np.float32(c["p"])) * 65536 + 0.5))
    return torch.from_numpy((u >= drop).reshape(c["rows"], c["h"])).cuda(), 1 / (1 - drop / 65536)


def _exact_drop(s):
    keep, scale = _exact_keep(s)
    if s["case"]["op"] == "drop_fwd":
        z = s["x"].double()
        if s["bias"] is not None:
            z = z + s["bias"].double()
        return s["resid"].double() + keep * z * scale
    dx = keep * s["dy"].double() * scale
    return dx, dx.sum(0) if s["case"]["bias"] else None


def _exact_lp(s):
    c, parts = s["case"], []
    V = c["vocab"]
    step = max(1, 60_000_000 // V)
    for r in range(0, c["rows"], step):
        x = s["logits"][r:r + step, :V].double()
        t = s["target"][r:r + step].long()
        at = torch.arange(len(t), device="cuda")
        lp = torch.log_softmax(x, 1)
        p = lp.exp()
        h = -torch.special.xlogy(p, p).sum(1)
        if c["op"] == "lp_fwd":
            part = {"logp": torch.where(t < 0, 0.0, lp[at, t.clamp(min=0)]),
                    "stats": torch.stack([x.max(1).values, torch.logsumexp(x, 1) - x.max(1).values], 1)}
            if c["entropy"]:
                part["entropy"] = h
            if c["top_k"]:
                order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
                part["top_id"], part["top_logp"] = order.int(), lp.gather(1, order)
        else:
            up = torch.where(t < 0, 0.0, s["dlogp"][r:r + step].double())
            part = torch.zeros_like(x)
            part[at, t.clamp(min=0)] = up
            part -= p * up[:, None]
            if c["entropy"]:
                part -= s["dentropy"][r:r + step].double()[:, None] * (torch.special.xlogy(p, p) + p * h[:, None])
            part = {"dlogits": part}
        parts.append(part)
    out = {k: torch.cat([q[k] for q in parts]) for k in parts[0]}
    return out if c["op"] == "lp_fwd" else out["dlogits"]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["op"].split("_")[0]
    return {"qk": _exact_qk, "drop": _exact_drop, "lp": _exact_lp}[kind](s)
