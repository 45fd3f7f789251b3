"""The scratch size of a call that the library refuses is 0, as its header says."""
import pytest

from transformer_layer_step_b200 import gptlayer as G

A, FAR = 1 << 20, 1 << 50                # stand for aligned device pointers


@pytest.mark.parametrize("rows,h", [(1 << 30, 64), ((1 << 31) - 1, 24), (1 << 24, 1 << 20), (0, 8), (4, 12)])
def test_dropout(rows, h):
    assert G.dropout_scratch_bytes(rows, h) == 0
    with pytest.raises(G.GptlError) as e:
        G.dropout_add_bwd(rows, h, "bf16", A, 0, 0.1, A, 0, FAR, A, A)
    assert e.value.code == G.E_SHAPE
