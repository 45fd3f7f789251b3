"""Token log probabilities where a warp takes a row: many rows of up to 2048
16-byte vectors, on both sides of that border, with every row's end checked.

Tolerance, f = 2^-24, from the path that a warp's row takes.  V = ceil(vectors / 32)
vectors of N elements a lane, in batches of 2 and at most one single each after
the last: b <= V / 2 + 2 steps.
* A term's exponential is off by 4 f (ex2.approx, 2^-22) and 3 f |t| (the roundings of
  x - m, of its product with log2 e, and of log2 e itself).  Each later growth of the
  maximum multiplies it by another such exponential: 4 f, one rounding, and 3 f of the
  part of |t| that it brings.  The maximum grows at most once a step, once each for
  the head's and the tail's element, and in the 5 joins over the lanes: K = b + 7.
  Together 4 f + 5 K f + 3 f |t|, with |t| at most log2(vocab) + 2 in a row's mean.
* Additions of positive terms in the longest chain: V N / 2 in a lane's pair of sums,
  one a step where the pair is folded, head, tail and 5 joins: V N / 2 + b + 7.
  R = f (4 + 3 (log2 vocab + 2) + 5 K + V N / 2 + b + 7).
The bounds on the outputs follow from R as in test_gpu_logprob.py, whose checks are
used with this R.  The gradient's kernel adds nothing up: it takes R through ln Z
and the entropy only.
"""
import numpy as np
import pytest
import torch

import test_gpu_logprob as L
from transformer_layer_step_b200 import gptlayer as G
from gpu_util import need_gpu, stream, check_device_error

pytestmark = pytest.mark.gpu

ROWS = 1187                                                  # 8 a multiprocessor and 3


def _r_warp(n):
    def r(vocab):
        v = -(-(vocab // n) // 32)
        b = v // 2 + 2
        return L.F * (4 + 3 * (np.log2(vocab) + 2) + 5 * (b + 7) + v * n / 2 + b + 7)
    return r


# dtype, vocab, ld - vocab, kind; the last two are a block's rows, which R covers too
# (shorter chains; 5 + 4 joins instead of 5 and fewer steps)
CASES = [("bf16", 4096, 0, "random"), ("fp16", 9001, 3, "inf"), ("bf16", 16391, 0, "random"),
         ("fp16", 16384, 8, "rising"), ("fp32", 4099, 1, "low"), ("fp32", 8195, 0, "random"),
         ("fp32", 8192, 0, "rising"), ("bf16", 12001, 0, "large"), ("bf16", 16392, 0, "random"),
         ("fp32", 8196, 0, "rising")]


@pytest.mark.parametrize("dtype,vocab,pad,kind", CASES)
def test_rows_of_a_warp(dtype, vocab, pad, kind, monkeypatch):
    need_gpu()
    monkeypatch.setattr(L, "_r", _r_warp(4 if dtype == "fp32" else 8))
    ld = vocab + pad
    rng = np.random.default_rng(vocab)
    x_t, x = L._logits(ROWS, vocab, ld, dtype, vocab, "random" if kind == "rising" else kind)
    if kind == "rising":                                     # the maximum grows at every step
        ramp = (8 * torch.arange(vocab) / vocab).to(x_t.dtype)
        x_t[:ROWS, :vocab] = ramp.cuda()
        x[:] = ramp.double().numpy()
    x_t[3, 5], x_t[4, vocab - 1], x_t[5, :vocab] = float("nan"), float("inf"), float("-inf")
    x[3, 5], x[4, vocab - 1], x[5] = np.nan, np.inf, -np.inf
    target = rng.integers(0, vocab, ROWS).astype(np.int32)
    target[rng.random(ROWS) < 0.1] = -1
    t_t = torch.from_numpy(target).cuda()
    o = L._fwd(x_t, ROWS, vocab, ld, dtype, t_t, 0)
    check_device_error()
    some = np.r_[0:40, ROWS // 2 - 10:ROWS // 2 + 10, ROWS - 40:ROWS]
    at = torch.from_numpy(some).cuda()
    want = L._check_fwd({k: None if v is None else v[at] for k, v in o.items()}, x[some], target[some], 0)
    # every row got its answer: the maximum is exact, the rest in the range of one
    m = np.where(np.isnan(x), -np.inf, x).max(1)
    assert np.array_equal(o["stats"][:, 0].double().cpu().numpy(), m)
    ok = np.r_[0:3, 6:ROWS]
    assert torch.isfinite(o["entropy"][ok]).all() and (o["entropy"][ok] <= np.log(vocab) + 1e-3).all()
    up = rng.standard_normal(ROWS).astype(np.float32)
    de = (0.3 * rng.standard_normal(ROWS)).astype(np.float32)
    d_t = torch.full_like(x_t, 9.0)
    G.token_logprob_bwd(ROWS, vocab, ld, dtype, x_t, t_t, o["stats"], o["entropy"], torch.from_numpy(up).cuda(),
                        torch.from_numpy(de).cuda(), d_t, stream())
    check_device_error()
    L._check_bwd(d_t[at, :vocab].double().cpu().numpy(), x[some], target[some], up[some], de[some], want, dtype)
    assert (d_t[ROWS] == 9.0).all() and (d_t[:, vocab:] == 9.0).all()


def test_outputs_filled_on_the_streams_that_write_them():
    """Two streams at once, each filling its outputs and then calling."""
    need_gpu()
    rows, vocab = 4, 50001
    sides = []
    for k in range(2):
        x_t, x = L._logits(rows, vocab, vocab, "bf16", 20 + k)
        sides.append((x_t, x, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for x_t, x, st in sides:
            with torch.cuda.stream(st):
                outs.append((L._fwd(x_t, rows, vocab, vocab, "bf16", None, 8, st.cuda_stream), x))
    check_device_error()
    for o, x in outs:
        L._check_fwd(o, x, None, 8)
