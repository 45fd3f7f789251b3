"""GPU parity of bias + dropout + residual, forward and backward, against the
float64 oracle with the generator's own mask.

Tolerances: z = x + bias, its product with the factor and the sum with resid are
each rounded to fp32 (3 f of the absolute terms, f = 2^-24), and the result once
to its type (u of its size; fp16 below its normal range 2^-25).  The mask is
exact: every dropped element is resid to the last bit.  dbias sums at most
rows / 8 terms in a thread, 256 teams of a block and 4 * 148 partial rows after that:
under (rows + 1200) f of the sum of the absolute terms.
"""
import numpy as np
import pytest
import torch

from oracle import parts
from transformer_layer_step_b200 import gptlayer as G
from gpu_util import need_gpu, dev_tensor, host_values, rounded, stream, check_device_error

pytestmark = pytest.mark.gpu

F = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": F}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# dtype, rows, h, p, resid (None or its type), y type, bias
CASES = [
    ("bf16", 1, 8, 0.5, "bf16", "bf16", True),
    ("fp16", 3, 24, 0.1, "fp32", "fp32", True),
    ("bf16", 129, 264, 0.3, "fp32", "bf16", False),
    ("fp16", 777, 1096, 0.25, "fp16", "fp32", True),
    ("bf16", 40, 8192, 0.9, None, "bf16", True),
    ("fp16", 2500, 64, 0.1, "fp16", "fp16", True),
    ("bf16", 2048, 2560, 0.1, "fp32", "fp32", True),
    ("fp16", 65, 40, 0.0, "fp32", "fp16", True),             # nothing is dropped
    ("bf16", 9, 16, 65535 / 65536, "bf16", "bf16", False),   # the largest p
]


def _rng_state(seed, offset):
    words = np.array([seed, offset], np.uint64).view(np.int64)
    return torch.from_numpy(words).cuda()


def _f32(t):
    return torch.from_numpy(t.astype(np.float32)).cuda()


def _dev(a, ty):
    return None if a is None else (_f32(a) if ty == "fp32" else dev_tensor(a, ty))


def _host(t, ty):
    return t.double().cpu().numpy() if ty == "fp32" else host_values(t, ty)


def _round(a, ty):
    return a.astype(np.float32).astype(np.float64) if ty == "fp32" else rounded(a, ty)


SEED, OFFSET, SITE = (1 << 63) + 12345, (7 << 32) + 99, 0xFFFFFFFE


@pytest.mark.parametrize("dtype,rows,h,p,rt,yt,bias", CASES)
def test_fwd(dtype, rows, h, p, rt, yt, bias):
    need_gpu()
    rng = np.random.default_rng(rows + h)
    x = rounded(rng.standard_normal((rows, h)), dtype)
    b = rounded(0.3 * rng.standard_normal(h), dtype) if bias else None
    r = _round(2 * rng.standard_normal((rows, h)), rt) if rt else None
    x_t, b_t, r_t = dev_tensor(x, dtype), _dev(b, dtype), _dev(r, rt)
    full = torch.full((rows + 2, h), 7.0, dtype=TORCH[yt], device="cuda")   # rows behind stay
    y_t = full[:rows]
    st = _rng_state(SEED, OFFSET)
    G.dropout_add_fwd(rows, h, dtype, x_t, b_t, r_t, rt == "fp32", p, st if p else None, SITE, y_t,
                      yt == "fp32", stream())
    check_device_error()
    kept, factor = parts.dropout_mask(rows, h, p, SEED, OFFSET, SITE)
    want = parts.dropout_add_fwd(x, b, r, kept, factor)
    got = _host(y_t, yt)
    z = np.abs(x) + (0 if b is None else np.abs(b))
    size = np.where(kept, z * factor, 0) + (0 if r is None else np.abs(r))
    assert (np.abs(got - want) <= U[yt] * np.abs(want) + 3 * F * size + TINY[yt]).all()
    base = np.zeros((rows, h)) if r is None else _round(r, yt)
    assert np.array_equal(got[~kept], base[~kept])
    assert (full[rows:] == 7.0).all()
    assert st.cpu().numpy().view(np.uint64).tolist() == [SEED, OFFSET]


@pytest.mark.parametrize("dtype,rows,h,p,rt,yt,bias", CASES)
def test_bwd(dtype, rows, h, p, rt, yt, bias):
    need_gpu()
    dt = "fp32" if yt == "fp32" else dtype                    # dy has y's type
    rng = np.random.default_rng(rows * 3 + h)
    dy = _round(rng.standard_normal((rows, h)), dt)
    dy_t = _dev(dy, dt)
    full = torch.full((rows + 2, h), 7.0, dtype=TORCH[dtype], device="cuda")
    dx_t = full[:rows]
    db = scratch = None
    if bias:
        db = torch.full((h,), float("nan"), device="cuda")
        scratch = torch.full((G.dropout_scratch_bytes(rows, h),), 255, dtype=torch.uint8, device="cuda")
    st = _rng_state(SEED, OFFSET) if p else None
    args = (rows, h, dtype, dy_t, dt == "fp32", p, st, SITE, dx_t, db, scratch)
    G.dropout_add_bwd(*args, stream())
    check_device_error()
    kept, factor = parts.dropout_mask(rows, h, p, SEED, OFFSET, SITE)
    dx, dbias = parts.dropout_add_bwd(dy, kept, factor)
    got = host_values(dx_t, dtype)
    assert (np.abs(got - dx) <= U[dtype] * np.abs(dx) + 2 * F * np.abs(dx) + TINY[dtype]).all()
    assert (got[~kept] == 0).all() and (full[rows:] == 7.0).all()
    if bias:
        first = db.clone()
        assert (np.abs(db.double().cpu().numpy() - dbias) <= (rows + 1200) * F * np.abs(dx).sum(0)).all()
        db.fill_(float("nan"))
        G.dropout_add_bwd(*args, stream())
        assert torch.equal(db, first)                        # the same bits again


def test_in_place_forms():
    need_gpu()
    rows, h, dtype = 37, 200, "bf16"
    rng = np.random.default_rng(0)
    x = dev_tensor(rng.standard_normal((rows, h)), dtype)
    r16 = dev_tensor(rng.standard_normal((rows, h)), dtype)
    r32 = torch.randn(rows, h, device="cuda")
    st = _rng_state(5, 6)
    run = lambda x, r, y, rf, yf: G.dropout_add_fwd(rows, h, dtype, x, None, r, rf, 0.4, st, 1, y, yf, stream())  # noqa: E731
    y16, y32 = torch.empty_like(x), torch.empty_like(r32)
    run(x, r16, y16, 0, 0)
    a, b = x.clone(), r16.clone()
    run(a, r16, a, 0, 0)
    run(x, b, b, 0, 0)
    assert torch.equal(a, y16) and torch.equal(b, y16)
    run(x, r32, y32, 1, 1)
    c = r32.clone()
    run(x, c, c, 1, 1)
    assert torch.equal(c, y32)
    d = x.clone()
    G.dropout_add_bwd(rows, h, dtype, x, 0, 0.4, st, 1, y16, None, None, stream())
    G.dropout_add_bwd(rows, h, dtype, d, 0, 0.4, st, 1, d, None, None, stream())
    check_device_error()
    assert torch.equal(d, y16)


def test_dropped_infinities_are_gone():
    need_gpu()
    rows, h = 16, 64
    kept, _ = parts.dropout_mask(rows, h, 0.5, 3, 4, 9)
    x = np.where(kept, 1.0, np.nan)
    x[~kept] = np.where(np.arange((~kept).sum()) % 2, np.inf, np.nan)
    x_t = torch.from_numpy(x).to(torch.bfloat16).cuda()
    y = torch.empty_like(x_t)
    G.dropout_add_fwd(rows, h, "bf16", x_t, None, None, 0, 0.5, _rng_state(3, 4), 9, y, 0, stream())
    check_device_error()
    assert np.array_equal(y.float().cpu().numpy(), np.where(kept, 2.0, 0.0))


def test_forward_and_backward_share_the_mask_across_replays():
    """A captured step that advances the state draws new masks at each replay,
    and its backward makes its forward's mask again."""
    need_gpu()
    rows, h, p = 64, 128, 0.3
    one = torch.ones(rows, h, dtype=torch.float16, device="cuda")
    y, dx = torch.empty_like(one), torch.empty_like(one)
    db = torch.empty(h, device="cuda")
    scratch = torch.empty(G.dropout_scratch_bytes(rows, h), dtype=torch.uint8, device="cuda")
    st = _rng_state(11, (1 << 32) - 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        s = torch.cuda.current_stream().cuda_stream
        G.dropout_add_fwd(rows, h, "fp16", one, None, None, 0, p, st, 2, y, 0, s)
        G.dropout_add_bwd(rows, h, "fp16", one, 0, p, st, 2, dx, db, scratch, s)
        G.rng_advance(st, 1, s)
    seen = []
    for step in range(3):
        graph.replay()
        check_device_error()
        kept, factor = parts.dropout_mask(rows, h, p, 11, (1 << 32) - 1 + step, 2)
        assert np.array_equal(y.cpu().numpy() != 0, kept) and torch.equal(y, dx)
        seen.append(kept)
    assert not np.array_equal(seen[0], seen[1]) and not np.array_equal(seen[1], seen[2])
