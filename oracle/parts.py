"""The parts around the layer, from their definitions: norm and rotation of
queries and keys, dropout, token log probabilities.  Test infrastructure only.

The Megatron-LM pages have no counterpart; the definitions are those of
include/gptlayer_parts.h.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------- norm and rotation of a head
def rope_angles(pos: np.ndarray, axis: np.ndarray, turns: np.ndarray) -> np.ndarray:
    """[tokens, pairs] angles: pos [axes, tokens], axis and turns [pairs]."""
    t = pos[axis].T.astype(np.float64) * turns
    return 2 * np.pi * (t - np.rint(t))


def rotate(n: np.ndarray, phi: np.ndarray, interleaved: bool) -> np.ndarray:
    """Turns the leading 2*pairs elements of n [tokens, head_dim] by phi."""
    out = n.copy()
    r = 2 * phi.shape[1]
    ia = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    ib = ia + (1 if interleaved else r // 2)
    a, b = n[:, ia], n[:, ib]
    out[:, ia] = a * np.cos(phi) - b * np.sin(phi)
    out[:, ib] = b * np.cos(phi) + a * np.sin(phi)
    return out


def qk_head_fwd(x, g, phi, interleaved, eps):
    """One head over its tokens [tokens, head_dim]; g None for no norm."""
    n = x if g is None else x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * g
    return rotate(n, phi, interleaved)


def qk_head_bwd(x, g, phi, interleaved, eps, dy):
    """(dx, dg) of qk_head_fwd; dg is None for no norm."""
    dn = rotate(dy, -phi, interleaved)
    if g is None:
        return dn, None
    r = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    d = dn * g
    return r * d - x * r ** 3 * (d * x).mean(1, keepdims=True), (dn * x * r).sum(0)


# ---------------------------------------------------------------- dropout
def philox4x32_10(counter, key):
    """Philox4x32-10 (Salmon et al., SC 2011): counter [..., 4] and key (2
    words) to [..., 4] words, all held as Python-sized unsigned integers."""
    c = [np.asarray(counter)[..., i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low, cut = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> cut) ^ c[1] ^ np.uint64(k[0]), p1 & low,
             (p0 >> cut) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1)


def dropout_mask(rows, h, p, seed, offset, site):
    """(kept [rows, h], factor of a kept element)."""
    drop = int(np.floor(float(np.float32(p)) * 65536 + 0.5))
    n = rows * h // 8
    ctr = np.zeros((n, 4), np.uint64)
    ctr[:, 0] = np.arange(n)
    ctr[:, 1], ctr[:, 2], ctr[:, 3] = site, offset & 0xFFFFFFFF, offset >> 32
    w = philox4x32_10(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    u = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(rows, h)
    return u >= drop, 65536.0 / (65536 - drop)


def dropout_add_fwd(x, bias, resid, kept, factor):
    z = x if bias is None else x + bias
    y = np.where(kept, z * factor, 0.0)
    return y if resid is None else y + resid


def dropout_add_bwd(dy, kept, factor):
    """(dx, dbias)."""
    dx = np.where(kept, dy * factor, 0.0)
    return dx, dx.sum(0)


# ------------------------------------------------ token log probabilities
def token_logprob_fwd(x, target, top_k=0):
    """dict of logp, entropy, stats [rows, 2], top_logp and top_id of the rows of
    x [rows, vocab]; target [rows], negative for none, or None."""
    rows, vocab = x.shape
    out = {"logp": np.zeros(rows), "entropy": np.zeros(rows), "stats": np.zeros((rows, 2)),
           "top_logp": np.zeros((rows, top_k)), "top_id": np.zeros((rows, top_k), np.int64)}
    for r in range(rows):
        v = x[r]
        t = -1 if target is None else int(target[r])
        if np.isnan(v).any() or (v == np.inf).any():
            fin = v[~np.isnan(v)]
            out["stats"][r] = fin.max() if fin.size else -np.inf, np.nan
            out["logp"][r] = np.nan if t >= 0 else 0.0
            out["entropy"][r] = np.nan
            out["top_logp"][r], out["top_id"][r] = np.nan, -1
            continue
        order = np.lexsort((np.arange(vocab), -v))[:top_k]
        out["top_id"][r] = order
        if (v == -np.inf).all():
            out["stats"][r] = -np.inf
            out["logp"][r] = -np.inf if 0 <= t < vocab else (np.nan if t >= vocab else 0.0)
            out["top_logp"][r] = -np.inf
            continue
        m = v.max()
        e = np.exp(v - m)
        z = e.sum()
        lz = np.log(z)
        d = np.where(e > 0, v - m, 0.0)
        out["stats"][r] = m, lz
        out["entropy"][r] = lz - (e * d).sum() / z
        out["logp"][r] = 0.0 if t < 0 else (np.nan if t >= vocab else v[t] - m - lz)
        out["top_logp"][r] = v[order] - m - lz
    return out


def token_logprob_bwd(x, target, dlogp, dentropy):
    """dlogits; dlogp or dentropy may be None."""
    rows, vocab = x.shape
    out = np.zeros_like(x)
    f = token_logprob_fwd(x, None)
    for r in range(rows):
        t = -1 if target is None else int(target[r])
        up = float(dlogp[r]) if dlogp is not None and 0 <= t < vocab else 0.0
        de = float(dentropy[r]) if dentropy is not None else 0.0
        m, lz = f["stats"][r]
        if (up == 0 and de == 0) or lz == -np.inf:
            continue
        if np.isnan(lz):
            out[r] = np.nan
            continue
        l = x[r] - m - lz
        p = np.exp(l)
        lp = np.where(p > 0, l, 0.0)
        out[r] = -p * (up + de * (lp + f["entropy"][r]))
        if up:
            out[r, t] += up
    return out
