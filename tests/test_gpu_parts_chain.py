"""The parts in a row, as a training step uses them around attention: QKV product,
norm and rotation of queries and keys, causal attention, out-projection, dropout
with bias and residual, LayerNorm, logits product, token log probability; then
the whole backward, every gradient against torch's in float64 for the same mask.

Both passes hold their activations in fp16 between steps, as the layer does, so
the bar is the layer's own: 2e-2 of the reference's RMS at the worst element.
"""
import numpy as np
import pytest
import torch

from oracle import parts
from transformer_layer_step_b200 import gptlayer as G
from gpu_util import need_gpu, dev_tensor, host_values, rounded, stream, check_device_error, rel_max_err

pytestmark = pytest.mark.gpu

B, S, HID, HEADS, TP, VOCAB, VPAD = 2, 64, 128, 4, 2, 257, 272
T, HD, P, SEED, OFFSET, SITE, LOSS = B * S, HID // HEADS, 0.2, 77, 5, 3, 1024.0
DT, EPS = "fp16", 1e-5


def _gemm(out, M, N, K, a, b, ldo, out_f32=False, k_shards=1):
    d = G.GemmDesc()
    d.M, d.N, d.K, d.groups, d.k_shards = M, N, K, 1, k_shards
    d.a, d.b = a, b
    d.out, d.out_f32, d.ldo, d.o_mod, d.o_str_div = out.data_ptr(), int(out_f32), ldo, 1, M * ldo
    G.gemm(d, DT, stream())


def _rows(t, rows, k, pitch=None, **kw):                     # K-major: element (row, k)
    return G.operand(t, k, rows, 1, pitch or k, 0, 0, **kw)


def _cols(t, k, cols, pitch=None, **kw):                     # MN-major: element (k, column)
    return G.operand(t, cols, k, 1, pitch or cols, 0, 1, **kw)


def _inputs():
    rng = np.random.default_rng(4)
    w = lambda *s, std=0.1: rounded(std * rng.standard_normal(s), DT)  # noqa: E731
    return dict(x=w(T, HID, std=1.0), w_qkv=w(TP, 3 * HID // TP, HID), gq=1 + w(HD), gk=1 + w(HD),
                w_o=w(HID, HID), b_o=w(HID), ln_g=1 + w(HID), ln_b=w(HID), w_v=w(VPAD, HID),
                target=rng.integers(-2, VOCAB, T).astype(np.int32),
                dlogp=(-LOSS / T * np.ones(T)).astype(np.float32),
                dent=(0.2 * LOSS / T * rng.standard_normal(T)).astype(np.float32))


def _reference(i, table):
    """Outputs and gradients of the chain in float64."""
    v = {k: torch.tensor(a, dtype=torch.float64, requires_grad=True) for k, a in i.items()
         if k not in ("target", "dlogp", "dent")}
    hs = HID // TP
    qkv = torch.einsum("th,gnh->gtn", v["x"], v["w_qkv"]).reshape(TP, B, S, 3, HEADS // TP, HD)
    phi = torch.from_numpy(parts.rope_angles(np.arange(S)[None], np.array([e.axis for e in table]),
                                             np.array([e.turns for e in table])))
    c, s = phi.cos()[:, None], phi.sin()[:, None]

    def turned(x, g):
        n = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * g
        a, b = n[..., :HD // 2], n[..., HD // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    q, k = turned(qkv[:, :, :, 0], v["gq"]), turned(qkv[:, :, :, 1], v["gk"])
    sc = torch.einsum("gbphd,gbqhd->gbhpq", q, k) / HD ** 0.5
    sc = sc.masked_fill(torch.ones(S, S).triu(1).bool(), -np.inf).softmax(-1)
    o = torch.einsum("gbhpq,gbqhd->gbphd", sc, qkv[:, :, :, 2]).reshape(TP, T, hs)
    z = torch.cat(list(o), 1) @ v["w_o"].T
    kept, factor = parts.dropout_mask(T, HID, P, SEED, OFFSET, SITE)
    r = v["x"] + (z + v["b_o"]) * torch.from_numpy(kept * factor)
    n = torch.nn.functional.layer_norm(r, (HID,), v["ln_g"], v["ln_b"], EPS)
    lp = (n @ v["w_v"].T)[:, :VOCAB].log_softmax(1)
    t = torch.from_numpy(i["target"]).long()
    logp = torch.where(t < 0, 0.0, lp.gather(1, t.clamp(min=0)[:, None])[:, 0])
    ent = -(lp.exp() * lp).sum(1)
    (logp @ torch.from_numpy(i["dlogp"]).double() + ent @ torch.from_numpy(i["dent"]).double()).backward()
    return dict(logp=logp, entropy=ent), {k: a.grad.numpy() for k, a in v.items()}


def test_chain_against_float64():
    need_gpu()
    i = _inputs()
    rope = G.rope_table(HD, base=1000.0)
    out, grads = _reference(i, rope)
    table = torch.frombuffer(bytearray(bytes(rope)), dtype=torch.uint8).cuda()
    d = {k: dev_tensor(a, DT) for k, a in i.items() if k not in ("target", "dlogp", "dent")}
    target, dlogp, dent = (torch.from_numpy(i[k]).cuda() for k in ("target", "dlogp", "dent"))
    rng = torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda")
    h16 = lambda *s: torch.empty(s, dtype=torch.float16, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.empty(s, dtype=torch.float32, device="cuda")  # noqa: E731
    hs, st = HID // TP, stream()
    qk = G.make_qk_desc(T, TP, HEADS // TP, HEADS // TP, HEADS // TP, HD, HD, seq=S, eps=EPS)

    # forward
    raw, qkv, o, z, r, n = h16(TP, T, 3 * hs), h16(TP, T, 3 * hs), h16(TP, T, hs), h16(T, HID), h16(T, HID), h16(T, HID)
    lse, mu, rstd = f32(TP * B * HEADS // TP, S), f32(T), f32(T)
    for g in range(TP):
        _gemm(raw[g], T, 3 * hs, HID, _rows(d["x"], T, HID), _rows(d["w_qkv"][g], 3 * hs, HID), 3 * hs)
    G.qk_norm_rope_fwd(qk, DT, raw, qkv, d["gq"], d["gk"], None, table, st)
    G.attention_fwd(B, S, HID, HEADS, TP, DT, qkv, o, lse, st)
    cat = torch.cat(list(o), 1)                              # [T, HID]: the shards' heads side by side
    _gemm(z, T, HID, HID, _rows(cat, T, HID), _rows(d["w_o"], HID, HID), HID)
    G.dropout_add_fwd(T, HID, DT, z, d["b_o"], d["x"], 0, P, rng, SITE, r, 0, st)
    G.layernorm_fwd(T, HID, DT, r, d["ln_g"], d["ln_b"], EPS, n, mu, rstd, st)
    logits = f32(T, VPAD)
    _gemm(logits, T, VPAD, HID, _rows(n, T, HID), _rows(d["w_v"], VPAD, HID), VPAD, out_f32=True)
    logp, ent, stats = f32(T), f32(T), f32(T, 2)
    G.token_logprob_fwd(T, VOCAB, VPAD, "fp32", logits, target, logp, ent, stats, stream=st)

    # backward
    dl = torch.zeros(T, VPAD, device="cuda")
    G.token_logprob_bwd(T, VOCAB, VPAD, "fp32", logits, target, stats, ent, dlogp, dent, dl, st)
    dl16 = dl.half()
    dn, dr, dz, do_cat, dqkv, dx = h16(T, HID), h16(T, HID), h16(T, HID), h16(T, HID), h16(TP, T, 3 * hs), f32(T, HID)
    g_wv, g_wo, g_wqkv = f32(VPAD, HID), f32(HID, HID), f32(TP, 3 * hs, HID)
    g_lng, g_lnb, g_bo, g_gq, g_gk = f32(HID), f32(HID), f32(HID), f32(HD), f32(HD)
    _gemm(dn, T, HID, VPAD, _rows(dl16, T, VPAD), _cols(d["w_v"], VPAD, HID), HID)
    _gemm(g_wv, VPAD, HID, T, _cols(dl16, T, VPAD), _cols(n, T, HID), HID, out_f32=True)
    ws = torch.empty(G.layernorm_bwd_scratch_bytes(T, HID), dtype=torch.uint8, device="cuda")
    G.layernorm_bwd(T, HID, DT, dn, r, mu, rstd, d["ln_g"], torch.zeros_like(dn), dr, g_lng, g_lnb, None, ws, st)
    ws2 = torch.empty(G.dropout_scratch_bytes(T, HID), dtype=torch.uint8, device="cuda")
    G.dropout_add_bwd(T, HID, DT, dr, 0, P, rng, SITE, dz, g_bo, ws2, st)
    _gemm(do_cat, T, HID, HID, _rows(dz, T, HID), _cols(d["w_o"], HID, HID), HID)
    _gemm(g_wo, HID, HID, T, _cols(dz, T, HID), _cols(cat, T, HID), HID, out_f32=True)
    do = torch.stack(do_cat.split(hs, 1)).contiguous()
    dvec = torch.empty_like(lse)
    G.attention_bwd(B, S, HID, HEADS, TP, DT, qkv, o, do, lse, dvec, dqkv, stream=st)
    ws3 = torch.empty(G.qk_norm_rope_scratch_bytes(qk), dtype=torch.uint8, device="cuda")
    G.qk_norm_rope_bwd(qk, DT, raw, dqkv, dqkv, d["gq"], d["gk"], None, table, g_gq, g_gk, ws3, st)
    dxp = f32(TP, T, HID)
    for g in range(TP):
        _gemm(dxp[g], T, HID, 3 * hs, _rows(dqkv[g], T, 3 * hs), _cols(d["w_qkv"][g], 3 * hs, HID), HID, out_f32=True)
        _gemm(g_wqkv[g], 3 * hs, HID, T, _cols(dqkv[g], T, 3 * hs), _cols(d["x"], T, HID), HID, out_f32=True)
    dx = dxp.sum(0) + dr.float()
    check_device_error()

    for got, key in ((logp, "logp"), (ent, "entropy")):
        assert rel_max_err(got.cpu().numpy(), out[key].detach().numpy()) < 2e-2, key
    assert (logp[target < 0] == 0).all() and (target < 0).any()
    for got, key in ((g_wv, "w_v"), (g_lng, "ln_g"), (g_lnb, "ln_b"), (g_bo, "b_o"), (g_wo, "w_o"),
                     (g_gq, "gq"), (g_gk, "gk"), (g_wqkv, "w_qkv"), (dx, "x")):
        assert rel_max_err(got.cpu().numpy(), grads[key]) < 2e-2, key
