"""Sizes whose offsets would leave 64 bits are refused before any launch.  (No
device is needed: the pointers are made up.)"""
import pytest

from transformer_layer_step_b200 import gptlayer as G

A, FAR = 1 << 20, 1 << 50                # stand for aligned device pointers
LD = (1 << 40) - 8                       # the largest stride by itself


def _refused(fn, *args):
    before = G.launch_count()
    with pytest.raises(G.GptlError) as e:
        fn(*args)
    assert G.launch_count() == before
    return e.value.code == G.E_SHAPE


@pytest.mark.parametrize("kw", [dict(tokens=(1 << 30) - 1, x_ld=LD), dict(tokens=(1 << 30) - 1, y_ld=LD),
                                dict(groups=1 << 19, tokens=3, x_ld=32, x_gstride=LD),
                                dict(groups=1 << 17, tokens=2, y_ld=32, y_gstride=LD)], ids=str)
def test_query_key_strides(kw):
    d = G.make_qk_desc(**{**dict(tokens=1, groups=1, q_heads=1, k_heads=1, v_heads=0, head_dim=16, rot_dim=0), **kw})
    assert _refused(G.qk_norm_rope_fwd, d, "bf16", A, FAR, None, None, None, None)
    assert _refused(G.qk_norm_rope_bwd, d, "bf16", A, FAR, FAR, None, None, None, None, None, None, None)
    assert G.qk_norm_rope_scratch_bytes(d) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logit_rows(dtype):
    rows = (1 << 31) - 1
    assert _refused(G.token_logprob_fwd, rows, 100, LD, dtype, A, A, A)
    assert _refused(G.token_logprob_bwd, rows, 100, LD, dtype, A, A, A, None, A, None, FAR)
