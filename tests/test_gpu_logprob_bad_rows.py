"""Top alternatives of rows that hold NaN or +inf in any number, with one block to
eight a row: every place of such a row is written (top_id -1, NaN), whatever the
outputs held before, the rows between them are not disturbed, and the error word
stays clear.  NaNs of either sign: a negative one sorts below -inf as bits.
"""
import numpy as np
import pytest
import torch

from transformer_layer_step_b200 import gptlayer as G
from gpu_util import need_gpu, stream, check_device_error
from test_gpu_logprob import TORCH, _check_fwd

pytestmark = pytest.mark.gpu

INT = {"bf16": torch.int16, "fp16": torch.int16, "fp32": torch.int32}
NAN = {"bf16": (0x7FC0, 0xFFC0 - 0x10000), "fp16": (0x7E00, 0xFE00 - 0x10000),
       "fp32": (0x7FC00000, 0xFFC00000 - (1 << 32))}


def _bad_rows(vocab, dtype):
    """[rows, vocab] on the host, and which rows hold NaN or +inf (a short row lacks some parts)."""
    g = torch.Generator().manual_seed(vocab)
    eighth, n = vocab // 8, 16
    x = (3 * torch.randn(n, vocab, generator=g)).to(TORCH[dtype])
    b = x.view(INT[dtype])
    pos, neg = NAN[dtype]
    b[0] = pos                                               # nothing else
    b[2] = neg
    b[4, :vocab // 2] = pos                                  # half of the row, either half
    b[5, vocab // 2:] = neg
    b[6, -eighth:] = pos                                     # the last block's part
    b[7, 3 * eighth:4 * eighth] = neg                        # one in the middle
    b[8, eighth:] = neg                                      # all but the first part
    b[10, 64:] = neg                                         # every thread's later vectors
    b[11, torch.arange(vocab) % 64 >= 8] = pos               # most vectors, among finite ones
    x[12] = -np.inf
    b[12, vocab // 3:] = neg
    x[13, ::2] = np.inf
    x[14] = np.inf
    b[15, 2048:] = neg                                       # more NaN vectors than a search keeps
    return x, (x.isnan() | (x == np.inf)).any(1).numpy()


@pytest.mark.parametrize("top_k", [1, 20, 32])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("copies,vocab", [(1, 37), (1, 2000), (1, 5000), (1, 9003), (1, 20011), (10, 20011), (1, 50257)])
def test_every_place_of_a_bad_row_is_written(copies, vocab, dtype, top_k):
    need_gpu()
    x, bad = _bad_rows(vocab, dtype)
    x, bad = x.repeat(copies, 1), np.tile(bad, copies)
    rows, x_t = len(bad), x.cuda()
    target = np.where(np.arange(rows) % 3 == 2, -1, np.arange(rows) % vocab).astype(np.int32)
    o = dict(logp=torch.full((rows,), 5.0, device="cuda"), entropy=torch.full((rows,), 5.0, device="cuda"),
             stats=torch.full((rows, 2), 5.0, device="cuda"),
             top_logp=torch.full((rows, top_k), 5.0, device="cuda"),
             top_id=torch.full((rows, top_k), 7, dtype=torch.int32, device="cuda"))
    G.token_logprob_fwd(rows, vocab, vocab, dtype, x_t, torch.from_numpy(target).cuda(), o["logp"], o["entropy"],
                        o["stats"], top_k, o["top_logp"], o["top_id"], stream())
    check_device_error()
    ids, lps = o["top_id"].cpu().numpy(), o["top_logp"].cpu().numpy()
    assert (ids[bad] == -1).all() and np.isnan(lps[bad]).all()
    assert (ids[~bad] >= 0).all() and np.isfinite(lps[~bad]).all()
    _check_fwd(o, x.double().numpy(), target, top_k)
