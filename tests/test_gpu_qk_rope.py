"""GPU parity of the norm and rotation of queries and keys, forward and
backward, against the float64 oracle on the same 16-bit inputs.

Tolerances, with u the 16-bit type's half step (2^-8, 2^-11) and f = 2^-24:
* y = n_a cos - n_b sin is rounded once (u |y|) after fp32 arithmetic on terms
  of at most N = max |n| of its head.  Each of these at its worst, with |a cos| +
  |b sin| <= 1.42 N: the fast cosine and sine, 2^-21.19 and 2^-21.41 absolute as
  documented, 7 f N and 6 f N; the angle's three roundings (its fixed-point turns to
  fp32, the constant 2 pi / 2^32, their product), pi f each, 13.4 f N; the products'
  roundings 2.4 f N: 29 f N for a rotation alone.  With gains, r (a chain of 14
  additions of squares halved by the root, mean and eps 1, rsqrtf's 2 ulp: 12 f), x r
  and the gain, 14 f of each term: 20 f N more.  The bar is 32 f N in both: above the
  rotation's worst, and for the norm 0.65 of the sum of all worsts, which do not
  meet in one element.
* dx likewise, on terms of at most D = r max|d| + r^3 |x| mean|d x|, whose mean
  has a relative error of 24 f in its absolute sum: 64 f D.
* dg sums dn x r over rows in fp32: at most 1024 additions in a lane's chain at
  these sizes, then 64 in trees: 1100 f of the sum of the absolute terms.  Each
  dn is itself a rotation, off by 29 f of the head's largest |dy| as y is of N
  (not of |dn|, which may cancel): 32 f of the sum of max |dy| |x| r besides.
* fp16 results below its normal range are rounded to multiples of 2^-24:
  2^-25 absolute.
"""
import numpy as np
import pytest
import torch

from oracle import parts
from transformer_layer_step_b200 import gptlayer as G
from gpu_util import need_gpu, dev_tensor, host_values, rounded, stream, check_device_error

pytestmark = pytest.mark.gpu

F = 2.0 ** -24
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25}

# tokens, groups, q, k, v heads, head_dim, rot_dim, interleaved, axes, positions ("seq" or the farthest)
CASES = [
    ("bf16", 1, 1, 1, 1, 0, 16, 16, 0, 1, 5),                # the smallest head
    ("fp16", 1, 1, 32, 8, 8, 128, 128, 0, 1, 2 ** 31 - 1),   # one token, the farthest positions
    ("bf16", 7, 1, 5, 3, 1, 48, 32, 1, 2, 4096),             # odd counts, part of the head
    ("fp16", 33, 2, 3, 1, 2, 80, 64, 0, 3, 100000),          # head_dim 80, lanes left over
    ("bf16", 130, 4, 4, 4, 4, 64, 64, 1, 1, "seq"),          # the layer's packed rows
    ("fp16", 65, 1, 2, 2, 0, 256, 256, 0, 4, 1 << 20),       # the largest head
    ("bf16", 19, 3, 7, 2, 2, 112, 0, 0, 1, 9),               # no rotation
    ("bf16", 700, 1, 9, 1, 1, 96, 48, 1, 1, "seq"),          # shared key head, many tokens
    ("fp16", 3000, 2, 2, 2, 2, 32, 32, 0, 2, 50),            # every resident warp has tokens
    ("bf16", 41, 3, 5, 2, 0, 144, 96, 0, 1, 70),             # nine lanes a head
    ("fp16", 90, 2, 4, 3, 1, 160, 160, 1, 2, 70),            # ten
    ("bf16", 23, 1, 6, 2, 1, 176, 176, 0, 1, 5000),          # eleven of sixteen
]


def _table(rot, axes, seed):
    """A table whose axes come in no order; (device bytes, turns, axis)."""
    rng = np.random.default_rng(seed)
    pairs = rot // 2
    turns = 10000.0 ** (-np.arange(pairs) / max(pairs, 1)) / (2 * np.pi)
    axis = rng.integers(0, axes, pairs)
    raw = np.zeros(max(pairs, 1), dtype=[("turns", "f8"), ("axis", "i4"), ("reserved", "i4")])
    raw["turns"][:pairs], raw["axis"][:pairs] = turns, axis
    return torch.from_numpy(raw.view(np.uint8)).cuda(), turns, axis


class Case:
    def __init__(self, dtype, tokens, groups, q, k, v, hd, rot, inter, axes, far, norm=True, pad=0, scale=1.5):
        need_gpu()
        self.dtype, self.norm, self.hd, self.q, self.k, self.v = dtype, norm, hd, q, k, v
        self.inter, self.groups, self.tokens = bool(inter), groups, tokens
        rng = np.random.default_rng(tokens * 1000 + hd)
        self.width = (q + k + v) * hd
        self.x = rounded(rng.standard_normal((groups, tokens, self.width)) * scale, dtype)
        self.dy = rounded(rng.standard_normal((groups, tokens, self.width)), dtype)
        self.g = [rounded(1 + 0.3 * rng.standard_normal(hd), dtype) if norm else None for _ in range(2)]
        seq = 50 if far == "seq" else 0
        self.pos = None if seq else rng.integers(0, far, (axes, tokens), dtype=np.int32, endpoint=True)
        if not seq:
            self.pos[:, -1] = far                           # the farthest one is there
        self.table, turns, axis = _table(rot, axes, hd)
        at = np.tile(np.arange(tokens) % max(seq, 1), (axes, 1)) if seq else self.pos
        self.phi = parts.rope_angles(at, axis, turns)
        self.eps = 1e-5
        self.ld = self.width + pad
        self.desc = G.make_qk_desc(tokens, groups, q, k, v, hd, rot, inter, axes, seq, self.eps,
                                   self.ld if pad else 0, 0, self.ld if pad else 0, 0)
        self.pos_t = None if seq else torch.from_numpy(self.pos).cuda()
        self.g_t = [dev_tensor(g, dtype) if norm else None for g in self.g]

    def buffer(self, values, fill=7.0):
        """[groups, tokens, ld] on the device, padding columns at `fill`."""
        b = np.full((self.groups, self.tokens, self.ld), fill)
        if values is not None:
            b[:, :, :self.width] = values
        return dev_tensor(b, self.dtype)

    def heads(self):
        for gr in range(self.groups):
            for h in range(self.q + self.k):
                yield gr, slice(h * self.hd, (h + 1) * self.hd), int(h >= self.q)

    def fwd(self, x_t, y_t, st=None):
        G.qk_norm_rope_fwd(self.desc, self.dtype, x_t, y_t, *self.g_t, self.pos_t, self.table,
                           stream() if st is None else st)

    def bwd(self, x_t, dy_t, dx_t, st=None):
        n = self.hd if self.norm else 0
        dg = [torch.full((n,), float("nan"), device="cuda") if n else None for _ in range(2)]
        scratch = torch.full((G.qk_norm_rope_scratch_bytes(self.desc),), 255, dtype=torch.uint8,
                             device="cuda") if n else None
        G.qk_norm_rope_bwd(self.desc, self.dtype, x_t, dy_t, dx_t, *self.g_t, self.pos_t, self.table,
                           *dg, scratch, stream() if st is None else st)
        return dg

    def check_fwd(self, y_t, v_too=True):
        got = host_values(y_t, self.dtype)
        assert (got[:, :, self.width:] == 7.0).all()        # padding columns left alone
        if v_too:
            lo = (self.q + self.k) * self.hd
            assert np.array_equal(got[:, :, lo:self.width], self.x[:, :, lo:])
        for gr, col, kind in self.heads():
            x = self.x[gr, :, col]
            y = parts.qk_head_fwd(x, self.g[kind], self.phi, self.inter, self.eps)
            n = np.abs(x if not self.norm else parts.qk_head_fwd(x, self.g[kind], self.phi[:, :0], False, self.eps))
            tol = U[self.dtype] * np.abs(y) + 32 * F * n.max(1, keepdims=True) + TINY[self.dtype]
            assert (np.abs(got[gr, :, col] - y) <= tol).all()

    def check_bwd(self, dx_t, dg, v_too=True):
        got = host_values(dx_t, self.dtype)
        assert (got[:, :, self.width:] == 7.0).all()
        if v_too:
            lo = (self.q + self.k) * self.hd
            assert np.array_equal(got[:, :, lo:self.width], self.dy[:, :, lo:])
        want, size, turned = np.zeros((2, self.hd)), np.zeros((2, self.hd)), np.zeros((2, self.hd))
        for gr, col, kind in self.heads():
            x, dy, g = self.x[gr, :, col], self.dy[gr, :, col], self.g[kind]
            dx, dgh = parts.qk_head_bwd(x, g, self.phi, self.inter, self.eps, dy)
            dn = parts.rotate(dy, -self.phi, self.inter)
            if self.norm:
                r = 1 / np.sqrt((x * x).mean(1, keepdims=True) + self.eps)
                d = np.abs(dn * g)
                D = r * d.max(1, keepdims=True) + r ** 3 * np.abs(x) * (d * np.abs(x)).mean(1, keepdims=True)
                want[kind] += dgh
                size[kind] += np.abs(dn * x * r).sum(0)
                turned[kind] += (np.abs(dy).max(1, keepdims=True) * np.abs(x) * r).sum(0)
            else:
                D = np.abs(dn).max(1, keepdims=True)
            assert (np.abs(got[gr, :, col] - dx) <= U[self.dtype] * np.abs(dx) + 64 * F * D + TINY[self.dtype]).all()
        if self.norm:
            for kind in (0, 1):
                assert (np.abs(dg[kind].cpu().numpy() - want[kind]) <= 1100 * F * size[kind] + 32 * F * turned[kind]).all()


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("norm", [True, False])
def test_fwd_bwd(case, norm):
    c = Case(*case, norm=norm, pad=8)
    x_t, y_t = c.buffer(c.x), c.buffer(None)
    c.fwd(x_t, y_t)
    check_device_error()
    c.check_fwd(y_t)
    assert torch.equal(x_t, c.buffer(c.x))
    dx_t = c.buffer(None)
    dg = c.bwd(x_t, c.buffer(c.dy), dx_t)
    check_device_error()
    c.check_bwd(dx_t, dg)


@pytest.mark.parametrize("case", CASES[2:6], ids=str)
def test_in_place_is_the_same(case):
    """In place, V columns and padding are left alone, and the bits are those of
    the call with an output of its own; calls repeat bit for bit."""
    c = Case(*case, pad=16)
    x_t, y_t = c.buffer(c.x), c.buffer(None)
    c.fwd(x_t, y_t)
    z_t = x_t.clone()
    c.fwd(z_t, z_t)
    assert torch.equal(z_t, y_t)
    dy_t, dx_t = c.buffer(c.dy), c.buffer(None)
    dg = c.bwd(x_t, dy_t, dx_t)
    dz_t = dy_t.clone()
    dh = c.bwd(x_t, dz_t, dz_t)
    check_device_error()
    assert torch.equal(dz_t, dx_t) and all(torch.equal(a, b) for a, b in zip(dg, dh))


def test_groups_inside_tokens():
    """Strides with the groups side by side in a token's row: [tokens][groups][width]."""
    c = Case(*CASES[4])
    dense_x, dense_y = c.buffer(c.x), c.buffer(None)
    c.fwd(dense_x, dense_y)
    w = c.width
    c.desc = G.make_qk_desc(c.tokens, c.groups, c.q, c.k, c.v, c.hd, 64, 1, 1, 50, c.eps,
                            c.groups * w, w, c.groups * w, w)
    x_t = dense_x.transpose(0, 1).contiguous()
    y_t = torch.zeros_like(x_t)
    c.fwd(x_t, y_t)
    check_device_error()
    assert torch.equal(y_t.transpose(0, 1), dense_y)


def test_zero_and_infinite_heads():
    """A head of zeros stays zero and sends back r g dn; an infinite element
    makes its own head's results NaN or 0 and no other head's."""
    c = Case("bf16", 6, 1, 2, 2, 0, 64, 64, 0, 1, 100)
    c.x[0, 1] = 0.0
    x_t, y_t = c.buffer(c.x), c.buffer(None)
    c.fwd(x_t, y_t)
    dx_t = c.buffer(None)
    dg = c.bwd(x_t, c.buffer(c.dy), dx_t)
    check_device_error()
    c.check_fwd(y_t)
    c.check_bwd(dx_t, dg)
    assert (y_t[0, 1, :c.width] == 0).all()
    clean = y_t.clone()
    x_t[0, 3, 64] = float("inf")                             # query head 1 of token 3
    c.fwd(x_t, y_t)
    check_device_error()
    same = y_t == clean
    same[0, 3, 64:128] = True
    assert same.all()


@pytest.mark.parametrize("eps,scale", [(1e-30, 1.5), (1e-30, 1e-12), (1e-5, 1e15), (1e30, 1.5)])
def test_far_scales(eps, scale):
    """r from 1e-15 to 1e15, whose cube is outside fp32, and a head of zeros."""
    c = Case("bf16", 5, 1, 2, 1, 0, 64, 64, 0, 1, 100, scale=scale)
    c.x[0, 2] = 0.0
    c.eps = c.desc.eps = float(np.float32(eps))
    x_t, y_t, dx_t = c.buffer(c.x), c.buffer(None), c.buffer(None)
    c.fwd(x_t, y_t)
    dg = c.bwd(x_t, c.buffer(c.dy), dx_t)
    check_device_error()
    c.check_fwd(y_t)
    c.check_bwd(dx_t, dg)


def test_bad_axis_is_reported():
    """An axis outside the descriptor's sets bit 2 of the error word and counts
    as axis 0; the table is read within its bounds all the same."""
    c = Case("fp16", 5, 1, 2, 2, 0, 32, 32, 0, 1, 1000)
    x_t, y_t, z_t = c.buffer(c.x), c.buffer(None), c.buffer(None)
    c.fwd(x_t, y_t)
    check_device_error()
    c.table.view(torch.int32)[2::4] = torch.tensor([1, -1] * 8, dtype=torch.int32, device="cuda")
    c.fwd(x_t, z_t)
    torch.cuda.synchronize()
    assert G.read_device_error(clear=True) == 2
    assert torch.equal(y_t, z_t)


def test_streams_and_graph_replay():
    """Forward and backward captured into a graph on a side stream replay with
    the buffers' new values; a call in another stream has its own workspace."""
    c = Case(*CASES[7])
    x_t, dy_t = c.buffer(c.x), c.buffer(c.dy)
    y_t, dx_t = c.buffer(None), c.buffer(None)
    n = G.qk_norm_rope_scratch_bytes(c.desc)
    dg = [torch.zeros(c.hd, device="cuda") for _ in range(2)]
    scratch = torch.zeros(n, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        st = torch.cuda.current_stream().cuda_stream
        c.fwd(x_t, y_t, st)
        G.qk_norm_rope_bwd(c.desc, c.dtype, x_t, dy_t, dx_t, *c.g_t, c.pos_t, c.table, *dg, scratch, st)
    c.x = np.roll(c.x, 1, axis=1)
    x_t.copy_(c.buffer(c.x))
    graph.replay()
    check_device_error()
    c.check_fwd(y_t)
    c.check_bwd(dx_t, dg)


def test_two_streams_with_their_own_scratch():
    cases = [Case(*CASES[7]), Case(*CASES[4])]
    streams = [torch.cuda.Stream() for _ in cases]
    held = [(c, c.buffer(c.x), c.buffer(c.dy), c.buffer(None), c.buffer(None)) for c in cases]
    torch.cuda.synchronize()
    dgs = []
    for _ in range(10):
        dgs = []
        for (c, x_t, dy_t, y_t, dx_t), st in zip(held, streams):
            with torch.cuda.stream(st):
                c.fwd(x_t, y_t, st.cuda_stream)
                dgs.append(c.bwd(x_t, dy_t, dx_t, st.cuda_stream))
    check_device_error()
    for (c, _, _, y_t, dx_t), dg in zip(held, dgs):
        c.check_fwd(y_t)
        c.check_bwd(dx_t, dg)


def test_single_heads_of_every_lane_count():
    """One query and one key head of each head_dim, one token: every lane layout."""
    for hd in range(16, 257, 16):
        for inter in (0, 1):
            c = Case("fp16", 1, 1, 1, 1, 0, hd, hd, inter, 1, 12345)
            x_t, y_t, dx_t = c.buffer(c.x), c.buffer(None), c.buffer(None)
            c.fwd(x_t, y_t)
            dg = c.bwd(x_t, c.buffer(c.dy), dx_t)
            check_device_error()
            c.check_fwd(y_t)
            c.check_bwd(dx_t, dg)
