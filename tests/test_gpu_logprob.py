"""GPU parity of the token log probabilities, their entropy, top alternatives
and gradient against the float64 oracle on the same logits.

Tolerances, f = 2^-24: an exponential's argument t = (x - m) log2 e is rounded
twice and ex2.approx is good to 2^-22, so a term is off by 4 f + 3 f |t| of itself;
p-weighted, |t| is at most log2(vocab) + 2 in a row's mean.  A sum of positive terms
is off by at most one f for each addition in its longest chain: with 128 threads and
pairs of sums vocab / 256, and 16 in the trees and the remainder.  Z is good to
R = f (4 + 3 (log2 vocab + 2) + vocab / 256 + 16) of itself.  (Not counted: the factor
of a maximum that grows, and the longer chains of a warp's row, vocab / 64 beyond 512
elements in 1200 rows here; test_gpu_logprob_many_rows.py counts both.)
* logp, top_logp: R + 3 f (|x - m| + ln Z).
* entropy: R on ln Z, and on S / Z = sum p t twice R of sum p |t|, which is at
  most entropy + ln Z + 1: R (1 + 3 (ln Z + entropy + 1)).
* gradient: with l = (x - m) - ln Z, the first difference is off by f |x - m|, the
  second by f |l|, ln Z by R, and l log2 e by f of itself, so p is off by
  R + 4 f + f (|x - m| + 2 |l|) <= 2 R + 3 f (|l| + ln Z) of itself.  l + H is off
  by 2 R + f (...) absolutely (R for ln Z, R for H, more where H is large: 3 R H),
  which is why 1 stands beside |l| + H.  With
  A = p (|dlogp| + |dentropy| (|l| + H + 1)): (4 R + 6 f (|l| + ln Z)) A + u |dx|; the
  target's own entry adds dlogp - p dlogp in fp32 (2 f |dlogp|); fp16 2^-25 absolute.
Whole numbers are exact.
"""
import numpy as np
import pytest
import torch

from oracle import parts
from transformer_layer_step_b200 import gptlayer as G
from gpu_util import need_gpu, stream, check_device_error

pytestmark = pytest.mark.gpu

F = 2.0 ** -24


def _r(vocab):
    return F * (4 + 3 * (np.log2(vocab) + 2) + vocab / 256 + 16)


U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": F}
TINY = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -25, "fp32": 2.0 ** -126}
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _logits(rows, vocab, ld, dtype, seed, kind="random"):
    """(device [rows + 1, ld] with garbage around, float64 values [rows, vocab])."""
    g = torch.Generator().manual_seed(seed)
    x = 3 * torch.randn(rows, vocab, generator=g)
    if kind == "ties":
        x = x.round()
    elif kind == "inf":
        x[torch.rand(rows, vocab, generator=g) < 0.7] = -np.inf
        x[:, 0] = 0.0
    elif kind == "low":
        x[torch.rand(rows, vocab, generator=g) < 0.7] = torch.finfo(TORCH[dtype]).min
    elif kind == "sharp":
        x[:, vocab // 2] = 60.0
    elif kind == "large":
        x = x + 20000.0
    full = torch.full((rows + 1, ld), 3e4, dtype=TORCH[dtype])
    full[:rows, :vocab] = x.to(TORCH[dtype])
    return full.cuda(), full[:rows, :vocab].double().numpy()


def _fwd(x_t, rows, vocab, ld, dtype, target, top_k, st=None):
    new = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    o = dict(logp=new(rows) if target is not None else None, entropy=new(rows), stats=new(rows, 2),
             top_logp=new(rows, top_k) if top_k else None,
             top_id=torch.full((rows, top_k), -7, dtype=torch.int32, device="cuda") if top_k else None)
    G.token_logprob_fwd(rows, vocab, ld, dtype, x_t, target, o["logp"], o["entropy"], o["stats"], top_k,
                        o["top_logp"], o["top_id"], stream() if st is None else st)
    return o


def _close(got, want, tol):
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    tol = np.broadcast_to(tol, want.shape)[fin]
    off = np.abs(got[fin] - want[fin])
    assert (off <= tol).all(), float((off - tol).max())


def _check_fwd(o, x, target, top_k):
    R = _r(x.shape[1])
    want = parts.token_logprob_fwd(x, target, top_k)
    host = {k: None if v is None else v.double().cpu().numpy() for k, v in o.items()}
    lz = np.where(np.isfinite(want["stats"][:, 1]), want["stats"][:, 1], 0)
    h = np.where(np.isfinite(want["entropy"]), want["entropy"], 0)
    assert np.array_equal(host["stats"][:, 0], want["stats"][:, 0])
    _close(host["stats"][:, 1], want["stats"][:, 1], R + 3 * F * lz)
    if target is not None:
        lp = np.where(np.isfinite(want["logp"]), np.abs(want["logp"]), 0)
        _close(host["logp"], want["logp"], R + 3 * F * (lp + 2 * lz))
    _close(host["entropy"], want["entropy"], R * (1 + 3 * (lz + h + 1)))
    if top_k:
        assert np.array_equal(host["top_id"], want["top_id"])
        lp = np.where(np.isfinite(want["top_logp"]), np.abs(want["top_logp"]), 0)
        _close(host["top_logp"], want["top_logp"], R + 3 * F * (lp + 2 * lz[:, None]))
    return want


def _check_bwd(dx, x, target, up, de, want, dtype):
    R = _r(x.shape[1])
    g = parts.token_logprob_bwd(x, target, up, de)
    m, lz = want["stats"][:, :1], want["stats"][:, 1:]
    with np.errstate(invalid="ignore"):
        l = x - m - lz
    p = np.where(np.isfinite(l), np.exp(np.where(np.isfinite(l), l, -1e9)), 0)
    al = np.where(p > 0, np.abs(np.where(np.isfinite(l), l, 0)), 0)
    a = p * (np.abs(up)[:, None] * (0 if target is None else 1) +
             np.abs(de)[:, None] * (al + np.nan_to_num(want["entropy"])[:, None] + 1))
    tol = (4 * R + 6 * F * (al + np.abs(np.nan_to_num(lz, neginf=0)))) * a + U[dtype] * np.abs(np.nan_to_num(g)) + TINY[dtype]
    if target is not None:
        t = np.asarray(target)
        ok = (t >= 0) & (t < x.shape[1])
        tol[np.flatnonzero(ok), t[ok]] += 2 * F * np.abs(up)[ok]
    _close(dx, g, tol)


# dtype, rows, vocab, ld - vocab, top_k, kind: every alignment of a row, one
# block to eight a row, thread counts, heads and tails without a body
CASES = [
    ("bf16", 3, 1, 0, 1, "random"), ("fp32", 4, 2, 1, 2, "random"), ("fp16", 5, 7, 0, 7, "ties"),
    ("bf16", 9, 8, 5, 3, "random"), ("fp32", 6, 33, 0, 32, "ties"), ("fp16", 17, 100, 0, 32, "ties"),
    ("bf16", 300, 501, 2, 5, "inf"), ("fp32", 40, 1003, 0, 20, "low"), ("fp16", 11, 4099, 0, 20, "ties"),
    ("bf16", 2, 8209, 3, 32, "inf"), ("fp32", 5, 16411, 0, 20, "random"), ("bf16", 1, 50257, 0, 20, "random"),
    ("fp16", 30, 20011, 1, 10, "low"), ("bf16", 70, 12345, 0, 20, "ties"), ("fp32", 180, 9001, 2, 3, "sharp"),
    ("fp32", 3, 5000, 0, 8, "large"), ("bf16", 1200, 3001, 0, 0, "random"), ("fp16", 600, 700, 4, 1, "inf"),
    ("bf16", 1, 152000, 0, 32, "ties"),
]


@pytest.mark.parametrize("dtype,rows,vocab,pad,top_k,kind", CASES)
def test_fwd_bwd(dtype, rows, vocab, pad, top_k, kind):
    need_gpu()
    ld = vocab + pad
    rng = np.random.default_rng(vocab)
    x_t, x = _logits(rows, vocab, ld, dtype, vocab, kind)
    target = rng.integers(0, vocab, rows).astype(np.int32)
    target[rng.random(rows) < 0.15] = -100
    t_t = torch.from_numpy(target).cuda()
    o = _fwd(x_t, rows, vocab, ld, dtype, t_t, top_k)
    check_device_error()
    want = _check_fwd(o, x, target, top_k)
    up = rng.standard_normal(rows).astype(np.float32)
    de = (0.3 * rng.standard_normal(rows)).astype(np.float32)
    up_t, de_t = torch.from_numpy(up).cuda(), torch.from_numpy(de).cuda()
    d_t = torch.full_like(x_t, 9.0)
    G.token_logprob_bwd(rows, vocab, ld, dtype, x_t, t_t, o["stats"], o["entropy"], up_t, de_t, d_t, stream())
    check_device_error()
    _check_bwd(d_t[:rows, :vocab].double().cpu().numpy(), x, target, up, de, want, dtype)
    assert (d_t[rows] == 9.0).all() and (d_t[:, vocab:] == 9.0).all()
    # in place, each gradient alone
    e_t = x_t.clone()
    G.token_logprob_bwd(rows, vocab, ld, dtype, e_t, t_t, o["stats"], o["entropy"], up_t, de_t, e_t, stream())
    assert torch.equal(e_t[:rows, :vocab], d_t[:rows, :vocab]) and torch.equal(e_t[rows], x_t[rows])
    zero = np.zeros(rows, np.float32)
    G.token_logprob_bwd(rows, vocab, ld, dtype, x_t, t_t, o["stats"], None, up_t, None, d_t, stream())
    check_device_error()
    _check_bwd(d_t[:rows, :vocab].double().cpu().numpy(), x, target, up, zero, want, dtype)
    G.token_logprob_bwd(rows, vocab, ld, dtype, x_t, None, o["stats"], o["entropy"], None, de_t, d_t, stream())
    check_device_error()
    _check_bwd(d_t[:rows, :vocab].double().cpu().numpy(), x, None, zero, de, want, dtype)


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 149])
@pytest.mark.parametrize("dtype,vocab", [("bf16", 511), ("bf16", 527), ("bf16", 4096), ("fp32", 4200), ("fp16", 8192),
                                         ("fp32", 2051), ("bf16", 16390)])
def test_between_the_splits(rows, dtype, vocab):
    """Sizes at which the work goes over from a warp to a block, and to clusters."""
    need_gpu()
    x_t, x = _logits(rows, vocab, vocab + 1, dtype, rows)
    t = np.arange(rows, dtype=np.int32)
    o = _fwd(x_t, rows, vocab, vocab + 1, dtype, torch.from_numpy(t).cuda(), 0)
    check_device_error()
    _check_fwd(o, x, t, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab", [37, 9003])
def test_rows_that_masks_and_infinities_leave(dtype, vocab):
    """All -inf; all the type's lowest; two tokens left; +inf; NaN; one value
    everywhere; a NaN beside -inf alone; the mask in all but the last place."""
    need_gpu()
    rows, k = 8, 20
    x = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(1))
    low = torch.finfo(TORCH[dtype]).min
    x[0] = -np.inf
    x[1] = low
    x[2] = -np.inf
    x[2, [5, vocab - 1]] = torch.tensor([1.0, 2.0])
    x[3, 17] = np.inf
    x[4, 30] = np.nan
    x[5] = 1.5
    x[6] = -np.inf
    x[6, 3] = np.nan
    x[7, :-1] = -np.inf
    x_t = x.to(TORCH[dtype]).cuda()
    xd = x.to(TORCH[dtype]).double().numpy()
    target = np.array([2, 3, 5, 4, 4, 6, 7, vocab - 1], np.int32)
    t_t = torch.from_numpy(target).cuda()
    o = _fwd(x_t, rows, vocab, vocab, dtype, t_t, k)
    check_device_error()
    want = parts.token_logprob_fwd(xd, target, k)
    _check_fwd(o, xd, target, k)
    up, de = np.ones(rows, np.float32), np.full(rows, 0.5, np.float32)
    d_t = torch.empty_like(x_t)
    G.token_logprob_bwd(rows, vocab, vocab, dtype, x_t, t_t, o["stats"], o["entropy"],
                        torch.from_numpy(up).cuda(), torch.from_numpy(de).cuda(), d_t, stream())
    check_device_error()
    _check_bwd(d_t.double().cpu().numpy(), xd, target, up, de, want, dtype)
    assert (d_t[0] == 0).all()
    # rows without any gradient are exact zeros whatever their logits
    none = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    G.token_logprob_bwd(rows, vocab, vocab, dtype, x_t, none, o["stats"], None,
                        torch.ones(rows, device="cuda"), None, d_t, stream())
    check_device_error()
    assert (d_t == 0).all()


def test_target_beyond_the_vocabulary_is_reported():
    need_gpu()
    x_t, x = _logits(3, 100, 100, "bf16", 0)
    target = torch.tensor([5, 100, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    o = _fwd(x_t, 3, 100, 100, "bf16", target, 0)
    torch.cuda.synchronize()
    assert G.read_device_error(clear=True) == 2
    assert torch.isnan(o["logp"]).tolist() == [False, True, True]
    d_t = torch.empty_like(x_t)
    G.token_logprob_bwd(3, 100, 100, "bf16", x_t, target, o["stats"], None, torch.ones(3, device="cuda"),
                        None, d_t, stream())
    torch.cuda.synchronize()
    assert G.read_device_error(clear=True) == 2
    assert (d_t[0] != 0).any() and (d_t[1:3] == 0).all()


def test_optional_outputs_and_repeatability():
    need_gpu()
    rows, vocab = 12, 9999
    x_t, x = _logits(rows, vocab, vocab, "bf16", 5, "ties")
    a = _fwd(x_t, rows, vocab, vocab, "bf16", None, 16)
    b = _fwd(x_t, rows, vocab, vocab, "bf16", None, 16)
    for k in ("entropy", "stats", "top_logp", "top_id"):
        assert torch.equal(a[k], b[k])
    only = torch.empty(rows, device="cuda")
    t = torch.arange(rows, dtype=torch.int32, device="cuda")
    G.token_logprob_fwd(rows, vocab, vocab, "bf16", x_t, t, only, stream=stream())
    check_device_error()
    full = _fwd(x_t, rows, vocab, vocab, "bf16", t, 0)
    assert torch.allclose(only, full["logp"], rtol=0, atol=4 * _r(vocab))


def test_graph_replay_and_side_stream():
    need_gpu()
    rows, vocab = 6, 30000
    x_t, x = _logits(rows, vocab, vocab, "bf16", 8)
    t_t = torch.arange(rows, dtype=torch.int32, device="cuda") * 1000
    o = _fwd(x_t, rows, vocab, vocab, "bf16", t_t, 12)
    d_t, up = torch.empty_like(x_t), torch.ones(rows, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        s = torch.cuda.current_stream().cuda_stream
        G.token_logprob_fwd(rows, vocab, vocab, "bf16", x_t, t_t, o["logp"], o["entropy"], o["stats"], 12,
                            o["top_logp"], o["top_id"], s)
        G.token_logprob_bwd(rows, vocab, vocab, "bf16", x_t, t_t, o["stats"], o["entropy"], up, up, d_t, s)
    y_t, y = _logits(rows, vocab, vocab, "bf16", 9, "ties")
    x_t.copy_(y_t)
    graph.replay()
    check_device_error()
    want = _check_fwd(o, y, t_t.cpu().numpy(), 12)
    one = np.ones(rows, np.float32)
    _check_bwd(d_t[:rows].double().cpu().numpy(), y, t_t.cpu().numpy(), one, one, want, "bf16")


def _ordered_rows(kind, rows, vocab, dtype):
    """Rows that crowd the search for the top: far more elements than are kept in
    the vectors of a few threads, slopes, plateaus and one repeated value."""
    i = torch.arange(vocab, dtype=torch.float64)
    if kind == "crowd":                     # 20 of every 256 vectors hold everything large
        x = torch.where((i // (16 // TORCH[dtype].itemsize)) % 256 < 20, 5 + i / vocab, -i / vocab)
    elif kind == "rising":
        x = i / 64
    elif kind == "falling":
        x = -i / 64
    elif kind == "plateau":                 # half of the row shares the largest value
        x = torch.where(i % 2 == 1, 3.0, 1.0)
    else:                                   # "same"
        x = torch.full((vocab,), -7.0, dtype=torch.float64)
    return x.expand(rows, -1).to(TORCH[dtype]).contiguous()


@pytest.mark.parametrize("kind", ["crowd", "rising", "falling", "plateau", "same"])
@pytest.mark.parametrize("dtype,rows,vocab,pad,top_k", [
    ("bf16", 150, 40000, 0, 32), ("fp32", 150, 21001, 0, 20), ("fp16", 1200, 12001, 1, 32),
    ("bf16", 2, 70003, 0, 32), ("fp32", 3, 9000, 1, 1), ("fp16", 2, 1030, 0, 32), ("fp32", 150, 1 << 20, 0, 32)])
def test_top_of_ordered_rows(kind, dtype, rows, vocab, pad, top_k):
    """One block a row, and a cluster, where candidates overflow what is kept, tie
    over half of the row, or lie in one thread's vectors."""
    need_gpu()
    x = _ordered_rows(kind, rows, vocab, dtype)
    x_t = torch.full((rows, vocab + pad), 1e4, dtype=x.dtype, device="cuda")
    x_t[:, :vocab] = x.cuda()
    o = _fwd(x_t, rows, vocab, vocab + pad, dtype, None, top_k)
    check_device_error()
    want = parts.token_logprob_fwd(x[:1].double().numpy(), None, top_k)
    ids = o["top_id"].cpu().numpy()
    assert (ids == want["top_id"]).all(), ids[(ids != want["top_id"]).any(1)][:1]
    _check_fwd({k: None if v is None else v[:1] for k, v in o.items()}, x[:1].double().numpy(), None, top_k)


def test_two_streams_at_once():
    need_gpu()
    rows, vocab = 4, 50001
    sides = []
    for k in range(2):
        x_t, x = _logits(rows, vocab, vocab, "bf16", 20 + k)
        sides.append((x_t, x, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[_fwd(x_t, rows, vocab, vocab, "bf16", None, 8, st.cuda_stream) for x_t, _, st in sides] for _ in range(20)]
    check_device_error()
    for pair in outs:
        for o, (_, x, _) in zip(pair, sides):
            _check_fwd(o, x, None, 8)
