"""Arguments of the parts around the layer: everything that the header rules out
is refused before any launch, without a device."""
import ctypes as C
import math

import numpy as np
import pytest

from transformer_layer_step_b200 import gptlayer as G

A = 1 << 20                              # stands for aligned device pointers
FAR = 1 << 40


def _code(fn, *args, **kw):
    before = G.launch_count()
    with pytest.raises(G.GptlError) as e:
        fn(*args, **kw)
    assert G.launch_count() == before
    return e.value.code


def test_launch_kinds_have_names():
    import os
    import re
    text = open(os.path.join(G.INCLUDE, "gptlayer_profile.h")).read()
    assert int(re.search(r"GPTL_KIND_COUNT = (\d+)", text).group(1)) == len(G.KIND_NAMES)


# ------------------------------------------------------ queries and keys
def _qk(**kw):
    return G.make_qk_desc(**{**dict(tokens=4, groups=2, q_heads=4, k_heads=2, v_heads=2, head_dim=64,
                                    rot_dim=32, seq=4), **kw})


@pytest.mark.parametrize("bad", [
    dict(tokens=0), dict(tokens=-1), dict(groups=0), dict(q_heads=0), dict(k_heads=0), dict(v_heads=-1),
    dict(head_dim=0), dict(head_dim=72), dict(head_dim=272), dict(rot_dim=8), dict(rot_dim=80),
    dict(rot_dim=-16), dict(axes=0), dict(axes=5), dict(seq=0), dict(x_ld=504), dict(y_ld=516),
    dict(x_gstride=-8), dict(x_ld=1024, x_gstride=2048), dict(tokens=1 << 30, groups=4),
    dict(y_ld=512, y_gstride=504),
])
def test_qk_shapes_refused(bad):
    assert _code(G.qk_norm_rope_fwd, _qk(**bad), "bf16", A, FAR, A, A, None, A) == G.E_SHAPE
    assert _code(G.qk_norm_rope_bwd, _qk(**bad), "bf16", A, FAR, FAR, A, A, None, A, A, A, A) == G.E_SHAPE


def test_qk_arguments_refused():
    d = _qk()
    fwd = lambda *a, dt="fp16", desc=d: _code(G.qk_norm_rope_fwd, desc, dt, *a)  # noqa: E731
    assert fwd(None, FAR, A, A, None, A) == G.E_NULL
    assert fwd(A, FAR, A, None, None, A) == G.E_NULL              # one gain
    assert fwd(A, FAR, A, A, None, None) == G.E_NULL              # rot_dim without a table
    assert fwd(A + 8, FAR, A, A, None, A) == G.E_ALIGN
    assert fwd(A, FAR, A, A + 2, None, A) == G.E_ALIGN
    assert fwd(A, FAR, A, A, A + 2, A) == G.E_ALIGN
    assert fwd(A, FAR, A, A, None, A, dt=7) == G.E_DTYPE
    assert fwd(A, A + 16, A, A, None, A) == G.E_ARG               # partial overlap
    assert fwd(A, A, A, A, None, A, desc=_qk(y_ld=1024)) == G.E_ARG   # in place, other strides
    assert fwd(A, FAR, A, A, None, A, desc=_qk(interleaved=2)) == G.E_ARG
    for eps in (0.0, -1.0, math.nan, math.inf):
        assert fwd(A, FAR, A, A, None, A, desc=_qk(eps=eps)) == G.E_ARG
    bwd = lambda *a: _code(G.qk_norm_rope_bwd, d, "bf16", *a)  # noqa: E731
    assert bwd(A, FAR, FAR, A, A, None, A, A, A, None) == G.E_NULL    # gains without scratch
    assert bwd(A, FAR, FAR, A, A, None, A, A, None, A) == G.E_NULL
    assert bwd(A, FAR, FAR, None, None, None, A, A, A, A) == G.E_NULL  # gradients without gains
    assert bwd(A, FAR, A, A, A, None, A, A, A, A) == G.E_ARG          # dx over x
    assert bwd(A, FAR, FAR + 64, A, A, None, A, A, A, A) == G.E_ARG   # dx partly over dy
    assert G.qk_norm_rope_scratch_bytes(d) > 0
    assert G.qk_norm_rope_scratch_bytes(_qk(head_dim=8)) == 0


def test_rope_table_ladders():
    t = G.rope_table(64, base=500.0)
    want = [500.0 ** (-j / 32) / (2 * math.pi) for j in range(32)]
    np.testing.assert_allclose([e.turns for e in t], want, rtol=1e-15)
    assert {e.axis for e in t} == {0}
    t = G.rope_table(64, axis_pairs=[8, 12, 12])
    assert [e.axis for e in t] == [0] * 8 + [1] * 12 + [2] * 12
    np.testing.assert_allclose([e.turns for e in t],
                               [1e4 ** (-j / 32) / (2 * math.pi) for j in range(32)], rtol=1e-15)
    t = G.rope_table(32, axis_pairs=[8, 8], per_axis=True)
    np.testing.assert_allclose([e.turns for e in t],
                               2 * [1e4 ** (-j / 8) / (2 * math.pi) for j in range(8)], rtol=1e-15)
    assert C.sizeof(G.RopePair) == 16
    for kw in (dict(rot_dim=24), dict(rot_dim=64, axis_pairs=[16, 8]), dict(rot_dim=64, axis_pairs=[40, -8]),
               dict(rot_dim=64, axis_pairs=[8, 8, 8, 4, 4])):
        assert _code(G.rope_table, **kw) == G.E_SHAPE
    for base in (0.0, -1.0, math.nan, math.inf):
        assert _code(G.rope_table, 64, base) == G.E_ARG


# ---------------------------------------------------------------- dropout
def test_dropout_arguments_refused():
    def fwd(rows=4, h=64, dt="bf16", x=A, bias=A, resid=A, rf=1, p=0.1, rng=A, y=FAR, yf=1):
        return _code(G.dropout_add_fwd, rows, h, dt, x, bias, resid, rf, p, rng, 0, y, yf)

    for kw in (dict(rows=0), dict(h=0), dict(h=60), dict(rows=-3), dict(rows=1 << 30, h=64)):
        assert fwd(**kw) == G.E_SHAPE, kw
    for p in (-0.1, 1.0, math.nan, math.inf, 1 - 2.0 ** -20):
        assert fwd(p=p) == G.E_ARG, p
    assert fwd(dt=5) == G.E_DTYPE
    assert fwd(x=None) == G.E_NULL and fwd(y=None) == G.E_NULL and fwd(rng=None) == G.E_NULL
    assert fwd(x=A + 8) == G.E_ALIGN and fwd(bias=A + 2) == G.E_ALIGN and fwd(rng=A + 4) == G.E_ALIGN
    assert fwd(y=A, resid=FAR) == G.E_ARG                  # y over x, another type
    assert fwd(y=FAR, resid=FAR, rf=0) == G.E_ARG          # y over resid, another type
    assert fwd(y=A + 16, yf=0, resid=FAR) == G.E_ARG       # partial overlap
    assert fwd(y=FAR, bias=FAR) == G.E_ARG
    assert fwd(rf=2) == G.E_ARG and fwd(yf=-1) == G.E_ARG

    def bwd(rows=4, h=64, dy=A, f32=0, p=0.1, rng=A, dx=FAR, dbias=A, scratch=A):
        return _code(G.dropout_add_bwd, rows, h, "fp16", dy, f32, p, rng, 0, dx, dbias, scratch)

    assert bwd(h=4) == G.E_SHAPE and bwd(p=1.5) == G.E_ARG and bwd(f32=3) == G.E_ARG
    assert bwd(dy=None) == G.E_NULL and bwd(scratch=None) == G.E_NULL and bwd(rng=None) == G.E_NULL
    assert bwd(dbias=A + 4) == G.E_ALIGN and bwd(scratch=A + 8) == G.E_ALIGN
    assert bwd(dx=A, f32=1) == G.E_ARG and bwd(dx=A + 32) == G.E_ARG
    assert _code(G.rng_advance, None, 1) == G.E_NULL
    assert _code(G.rng_advance, A + 4, 1) == G.E_ALIGN


@pytest.mark.parametrize("rows,h", [(1, 8), (7, 1096), (8192, 2560), (2048, 10240), (1 << 20, 64)])
def test_dropout_scratch_stays_small(rows, h):
    """Partial rows are at most a tenth of the data, beyond a few blocks' worth."""
    n = G.dropout_scratch_bytes(rows, h)
    assert 0 < n <= max(2 * rows * h // 10, 4 * h * 8 + 4 * 8 * 1200 * 32)
    assert G.dropout_scratch_bytes(rows, 4) == 0 and G.dropout_scratch_bytes(0, h) == 0


# ------------------------------------------------- token log probabilities
def test_logprob_arguments_refused():
    def fwd(rows=2, vocab=100, ld=100, dt="bf16", x=A, target=A, logp=A, ent=A, stats=A, k=0, tv=None,
            ti=None):
        return _code(G.token_logprob_fwd, rows, vocab, ld, dt, x, target, logp, ent, stats, k, tv, ti)

    for kw in (dict(rows=0), dict(vocab=0), dict(ld=99), dict(vocab=1 << 30, ld=1 << 30), dict(ld=1 << 40)):
        assert fwd(**kw) == G.E_SHAPE, kw
    assert fwd(x=None) == G.E_NULL and fwd(target=None) == G.E_NULL and fwd(logp=None) == G.E_NULL
    assert fwd(target=None, logp=None, ent=None, stats=None) == G.E_NULL      # no output
    assert fwd(k=3) == G.E_NULL and fwd(k=3, tv=A) == G.E_NULL
    for kw in (dict(k=-1), dict(k=33), dict(k=8, vocab=7)):
        assert fwd(**kw, tv=A, ti=A) == G.E_ARG, kw
    assert fwd(k=1, vocab=(1 << 20) + 1, ld=1 << 21, tv=A, ti=A) == G.E_SHAPE
    assert fwd(x=A + 2) == G.E_ALIGN and fwd(target=A + 2) == G.E_ALIGN and fwd(ent=A + 1) == G.E_ALIGN

    def bwd(rows=2, vocab=100, ld=100, x=A, target=A, stats=A, ent=A, up=A, de=A, dx=FAR):
        return _code(G.token_logprob_bwd, rows, vocab, ld, "fp32", x, target, stats, ent, up, de, dx)

    assert bwd(ld=10) == G.E_SHAPE
    assert bwd(stats=None) == G.E_NULL and bwd(up=None, de=None) == G.E_NULL
    assert bwd(target=None) == G.E_NULL and bwd(ent=None) == G.E_NULL and bwd(dx=None) == G.E_NULL
    assert bwd(dx=FAR + 4) == G.E_ALIGN
    assert bwd(dx=A + 16) == G.E_ARG                       # partial overlap
    rc = G.lib().gptl_token_logprob_fwd(2, 100, 100, 5, 0, A, A, A, A, A, 0, None, None, None)
    assert rc == G.E_DTYPE
    rc = G.lib().gptl_token_logprob_fwd(2, 100, 100, 0, 2, A, A, A, A, A, 0, None, None, None)
    assert rc == G.E_ARG
