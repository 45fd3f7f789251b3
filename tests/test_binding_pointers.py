"""What the binding takes for a pointer: None, an integer, or an object with
data_ptr().  Anything else is refused before the library is called: a host
array's address must never reach a kernel."""
import ctypes as C

import numpy as np
import pytest

from transformer_layer_step_b200 import gptlayer as G

A, FAR = 1 << 20, 1 << 40                # stand for aligned device pointers


class Tensor:
    def data_ptr(self):
        return A


HOST = [G.rope_table(32), (C.c_float * 8)(), b"0123456789abcdef", "0123456789abcdef", C.c_void_p(A),
        C.pointer(C.c_int(0)), np.zeros(16), np.int64(A), 1.0, [A]]


@pytest.mark.parametrize("x", HOST, ids=lambda x: type(x).__name__)
def test_other_objects_are_refused(x):
    with pytest.raises(AttributeError):
        G._ptr(x)
    calls = [
        lambda: G.qk_norm_rope_fwd(G.make_qk_desc(4, 1, 1, 1, 0, 32, 32, seq=4), "bf16", A, FAR, None, None, None, x),
        lambda: G.dropout_add_fwd(4, 64, "bf16", x, None, None, 0, 0.0, None, 0, FAR, 0),
        lambda: G.token_logprob_fwd(2, 100, 100, "fp32", x, None, None, A),
        lambda: G.layernorm_fwd(4, 128, "bf16", x, A, A, 1e-5, FAR, A, A),
    ]
    before = G.launch_count()
    for call in calls:
        with pytest.raises(AttributeError):
            call()
    assert G.launch_count() == before


def test_pointers_that_are_taken():
    assert G._ptr(None) is None and G._ptr(A) == A and G._ptr(Tensor()) == A and G._ptr(0) == 0
