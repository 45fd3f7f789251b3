"""Offsets beyond 2^31 elements: the last rows of large buffers give what the same
rows give in a small call (the log probabilities and the gradient, bit for bit; the
query/key rows likewise), or what the oracle says (dropout's mask)."""
import numpy as np
import pytest
import torch

from oracle import parts
from transformer_layer_step_b200 import gptlayer as G
from gpu_util import need_gpu, stream, check_device_error

pytestmark = pytest.mark.gpu


def _free():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_logprob_rows_behind_2_31():
    need_gpu()
    rows, vocab, few = 43000, 50257, 3
    assert (rows - few) * vocab > 2 ** 31
    x = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    x[-few:] = 3 * torch.randn(few, vocab, device="cuda")
    x[:-few] = 0
    t = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    t[-few:] = torch.tensor([50256, 0, 777], dtype=torch.int32)
    new = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    def run(x, t):
        n = len(t)
        o = dict(logp=new(n), entropy=new(n), stats=new(n, 2))
        G.token_logprob_fwd(n, vocab, vocab, "bf16", x, t, *o.values(), stream=stream())
        return o
    # enough rows for the small call to split the work as the large one does
    small = 1200
    xs, ts = x[-small:].clone(), t[-small:].clone()
    # the row's distance from a 16-byte boundary decides the order of its sums
    assert x[-small].data_ptr() % 16 == xs.data_ptr() % 16
    big, ref = run(x, t), run(xs, ts)
    check_device_error()
    for k in big:
        assert torch.equal(big[k][-small:], ref[k]), k
    up = torch.ones(rows, device="cuda")
    d = torch.empty(small, vocab, dtype=torch.bfloat16, device="cuda")
    G.token_logprob_bwd(small, vocab, vocab, "bf16", xs, ts, ref["stats"], None, up[:small], None, d, stream())
    G.token_logprob_bwd(rows, vocab, vocab, "bf16", x, t, big["stats"], None, up, None, x, stream())
    check_device_error()
    assert torch.equal(x[-small:], d) and (x[:-few] == 0).all()
    del x, xs, d
    _free()


def test_dropout_rows_behind_2_31():
    need_gpu()
    rows, h, p = (1 << 31) // 8192 + 5, 8192, 0.25
    x = torch.ones(rows, h, dtype=torch.bfloat16, device="cuda")
    state = torch.tensor([9, 10], dtype=torch.int64, device="cuda")
    G.dropout_add_fwd(rows, h, "bf16", x, None, None, 0, p, state, 3, x, 0, stream())
    check_device_error()
    n = h // 8
    ctr = np.zeros((n, 4), np.uint64)
    for r in (0, rows - 1):
        ctr[:, 0] = r * n + np.arange(n)
        ctr[:, 1], ctr[:, 2] = 3, 10
        w = parts.philox4x32_10(ctr, (9, 0))
        u = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(h)
        assert np.array_equal(x[r].float().cpu().numpy() != 0, u >= 16384)
    del x
    _free()


def test_query_key_tokens_behind_2_31():
    need_gpu()
    tokens, heads, hd = 270000, 64, 128
    width = heads * hd
    assert (tokens - 7) * width > 2 ** 31
    x = torch.zeros(tokens, width, dtype=torch.float16, device="cuda")
    x[-7:] = torch.randn(7, width, device="cuda").half()
    tail = x[-7:].clone()
    table = torch.frombuffer(bytearray(bytes(G.rope_table(hd))), dtype=torch.uint8).cuda()
    gain = torch.ones(hd, dtype=torch.float16, device="cuda")
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda") - 135000       # negative ones among them
    for n, buf, at in ((tokens, x, pos), (7, tail, pos[-7:].clone())):
        d = G.make_qk_desc(n, 1, 48, 16, 0, hd, hd)
        G.qk_norm_rope_fwd(d, "fp16", buf, buf, gain, gain, at, table, stream())
    check_device_error()
    assert torch.equal(x[-7:], tail) and (x[:-7] == 0).all()
    del x
    _free()


def test_negative_positions_turn_back():
    need_gpu()
    hd = 64
    table = torch.frombuffer(bytearray(bytes(G.rope_table(hd))), dtype=torch.uint8).cuda()
    x = torch.randn(9, 2 * hd, device="cuda").half()
    pos = torch.tensor([1, -1, 5, -5, 40000, -40000, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    d = G.make_qk_desc(9, 1, 1, 1, 0, hd, hd)
    G.qk_norm_rope_fwd(d, "fp16", x, y, None, None, pos, table, stream())
    G.qk_norm_rope_bwd(d, "fp16", x, x, z, None, None, -pos, table, None, None, None, stream())
    check_device_error()
    # a turn by -phi is the turn back by phi (-2^31 has no opposite: it is its own)
    assert torch.equal(y[:7], z[:7]) and torch.equal(y[8], z[8])
    turns = np.array([e.turns for e in G.rope_table(hd)])
    phi = parts.rope_angles(pos.cpu().numpy()[None].astype(np.int64), np.zeros(32, int), turns)
    want = parts.rotate(x[:, :hd].double().cpu().numpy(), phi, False)
    n = np.abs(x.double().cpu().numpy()).max()
    # one rounding to fp16, and 32 fp32 roundings of the head's largest element
    assert (np.abs(y[:, :hd].double().cpu().numpy() - want) <= 2.0 ** -11 * np.abs(want) + 32 * 2.0 ** -24 * n + 2.0 ** -25).all()
