"""Which outputs count as overlapping their input: rows do, the columns between
rows do not.  Without a device, every placement of two small sets of rows is
checked against the elements themselves; on a GPU, column ranges of one buffer
give what buffers of their own give.
"""
import numpy as np
import pytest
import torch

from transformer_layer_step_b200 import gptlayer as G
from gpu_util import need_gpu, stream, check_device_error

A = 1 << 20                              # stands for an aligned device pointer
W = 32                                   # one query and one key head of 16


def _code(fn, *args):
    try:
        fn(*args)
    except G.GptlError as e:
        return e.code
    return 0


def _elements(tokens, groups, ld, gs):
    return {g * gs + t * ld + c for g in range(groups) for t in range(tokens) for c in range(W)}


def _placements():
    for tokens, groups, ld, gs in [(1, 1, 32, 32), (3, 1, 32, 96), (3, 1, 64, 192), (4, 1, 104, 416),
                                   (2, 2, 72, 144), (3, 2, 128, 512), (1, 3, 32, 80), (2, 3, 200, 40),
                                   (3, 4, 320, 80), (5, 2, 96, 48 * 11)]:
        for off in range(-8 * 130, 8 * 130, 8):
            yield tokens, groups, ld, gs, off


@pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls would launch on made-up pointers")
def test_rows_count_and_columns_between_them_do_not():
    for tokens, groups, ld, gs, off in _placements():
        if off == 0:
            continue                                          # in place
        d = G.make_qk_desc(tokens, groups, 1, 1, 0, 16, 0, x_ld=ld, x_gstride=gs, y_ld=ld, y_gstride=gs)
        at = _elements(tokens, groups, ld, gs)
        want = any(e + off in at for e in at)
        far = A + (1 << 30)
        for code in (_code(G.qk_norm_rope_fwd, d, "bf16", A, A + 2 * off, None, None, None, None),
                     _code(G.qk_norm_rope_bwd, d, "bf16", A, far, A + 2 * off, None, None, None, None, None, None, None),
                     _code(G.qk_norm_rope_bwd, d, "bf16", far, A, A + 2 * off, None, None, None, None, None, None, None)):
            assert (code == G.E_ARG) == want, (tokens, groups, ld, gs, off)
        if groups == 1:
            code = _code(G.token_logprob_bwd, tokens, W, ld, "fp16", A, A, A, None, A, None, A + 2 * off)
            assert (code == G.E_ARG) == want, (tokens, ld, off)


def test_other_strides_are_kept_apart_as_ranges():
    d = G.make_qk_desc(3, 1, 1, 1, 0, 16, 0, x_ld=64, y_ld=128)
    assert _code(G.qk_norm_rope_fwd, d, "bf16", A, A + 64, None, None, None, None) == G.E_ARG


@pytest.mark.gpu
def test_column_ranges_of_one_buffer():
    need_gpu()
    tokens, groups, hd = 37, 2, 64
    w = 5 * hd
    g = torch.Generator(device="cuda").manual_seed(3)
    both = torch.randn(groups, tokens, 2 * w + 8, generator=g, device="cuda").bfloat16()
    gain = [(1 + 0.2 * torch.randn(hd, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    table = torch.frombuffer(bytearray(bytes(G.rope_table(hd))), dtype=torch.uint8).cuda()
    x, dy = both[..., :w].contiguous(), both[..., w:2 * w].contiguous()
    y, dx, dg = torch.empty_like(x), torch.empty_like(x), [torch.empty(hd, device="cuda") for _ in range(2)]
    d = G.make_qk_desc(tokens, groups, 2, 2, 1, hd, hd, seq=20)
    scratch = torch.empty(G.qk_norm_rope_scratch_bytes(d), dtype=torch.uint8, device="cuda")
    G.qk_norm_rope_fwd(d, "bf16", x, y, *gain, None, table, stream())
    G.qk_norm_rope_bwd(d, "bf16", x, dy, dx, *gain, None, table, *dg, scratch, stream())
    ld = 2 * w + 8
    s = G.make_qk_desc(tokens, groups, 2, 2, 1, hd, hd, seq=20, x_ld=ld, y_ld=ld)
    two = both.clone()
    left, right = two.data_ptr(), two.data_ptr() + 2 * w
    dh = [torch.empty_like(t) for t in dg]
    # dy -> dx in place beside x, then x -> y over the columns of dy
    G.qk_norm_rope_bwd(s, "bf16", left, right, right, *gain, None, table, *dh, scratch, stream())
    check_device_error()
    assert torch.equal(two[..., w:w + 4 * hd], dx[..., :4 * hd]) and all(torch.equal(a, b) for a, b in zip(dg, dh))
    G.qk_norm_rope_fwd(s, "bf16", left, right, *gain, None, table, stream())
    check_device_error()
    assert torch.equal(two[..., w:2 * w], y) and torch.equal(two[..., :w], x)
    assert torch.equal(two[..., 2 * w:], both[..., 2 * w:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,pad", [("fp32", 4), ("bf16", 8), ("fp16", 3)])
def test_gradient_beside_the_logits(dtype, pad):
    need_gpu()
    ty = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    rows, vocab = 23, 1000
    ld = 2 * vocab + pad
    two = torch.randn(rows, ld, device="cuda").to(ty)
    x = two[:, :vocab].clone()
    t = torch.arange(rows, dtype=torch.int32, device="cuda")
    new = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    logp, ent, stats, up = new(rows), new(rows), new(rows, 2), torch.randn(rows, device="cuda")
    keep = two.clone()
    G.token_logprob_fwd(rows, vocab, ld, dtype, two, t, logp, ent, stats, stream=stream())
    apart = torch.empty_like(two)
    G.token_logprob_bwd(rows, vocab, ld, dtype, two, t, stats, ent, up, up, apart, stream())
    G.token_logprob_bwd(rows, vocab, ld, dtype, two, t, stats, ent, up, up,
                        two.data_ptr() + vocab * two.element_size(), stream())
    check_device_error()
    assert torch.equal(two[:, vocab:2 * vocab], apart[:, :vocab])
    assert torch.equal(two[:, :vocab], x) and torch.equal(two[:, 2 * vocab:], keep[:, 2 * vocab:])
