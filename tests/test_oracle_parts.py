"""Pins for the oracle of the parts around the layer.

* Rotation keeps a pair's length, is undone by the opposite angle, and makes
  the product of a query and a key depend on the difference of positions.
* Philox4x32-10 gives the words of the known-answer vectors of its authors'
  reference implementation.
* Backward passes equal central differences of the forward.
* Log probabilities equal torch's log_softmax in float64; the entropy of a
  uniform row is ln vocab.
"""
import numpy as np
import pytest
import torch

from oracle import parts


def _diff(f, x, dy, h=1e-6):
    g = np.zeros_like(x)
    flat, gf = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + h
        up = float((f(x) * dy).sum())
        flat[i] = keep - h
        gf[i] = (up - float((f(x) * dy).sum())) / (2 * h)
        flat[i] = keep
    return g


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_relative(interleaved):
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 16))
    turns, axis = np.array([0.1, 0.01, 0.003, 0.2]), np.zeros(4, int)
    at = lambda p: parts.rope_angles(np.array([[p]]), axis, turns)  # noqa: E731
    rot = lambda v, p: parts.rotate(v, at(p), interleaved)  # noqa: E731
    assert np.allclose((rot(q, 1007) * rot(k, 1000)).sum(), (rot(q, 7) * rot(k, 0)).sum(), atol=1e-12)
    assert np.allclose(np.linalg.norm(rot(q, 5)), np.linalg.norm(q))
    assert np.allclose(parts.rotate(rot(q, 5), -at(5), interleaved), q)
    assert np.array_equal(rot(q, 9)[:, 8:], q[:, 8:])          # beyond rot_dim


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_head_backward_is_the_difference(interleaved, norm):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((2, 3, 16))
    g = 1 + 0.3 * rng.standard_normal(16) if norm else None
    phi = rng.uniform(-3, 3, (3, 6))
    dx, dg = parts.qk_head_bwd(x, g, phi, interleaved, 1e-3, dy)
    fwd = lambda v: parts.qk_head_fwd(v, g, phi, interleaved, 1e-3)  # noqa: E731
    np.testing.assert_allclose(dx, _diff(fwd, x, dy), atol=1e-8)
    if norm:
        np.testing.assert_allclose(
            dg, _diff(lambda v: parts.qk_head_fwd(x, v, phi, interleaved, 1e-3), g, dy), atol=1e-8)


@pytest.mark.parametrize("counter,key,words", [
    ([0] * 4, [0] * 2, [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
    ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
     [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]),
])
def test_philox_known_answers(counter, key, words):
    assert parts.philox4x32_10(np.array(counter, np.uint64), key).tolist() == words


def test_dropout_mask_statistics_and_independence():
    kept, factor = parts.dropout_mask(512, 512, 0.25, 123, 7, 3)
    n = kept.size
    assert factor == 65536 / (65536 - 16384)
    # five standard deviations of a binomial share
    assert abs(kept.mean() - 0.75) < 5 * np.sqrt(0.25 * 0.75 / n)
    for other in [(124, 7, 3), (123, 8, 3), (123, 7, 4)]:
        k2, _ = parts.dropout_mask(512, 512, 0.25, *other)
        assert abs((kept & k2).mean() - 0.75 ** 2) < 5 * np.sqrt(0.25 / n)
    assert parts.dropout_mask(4, 8, 0.0, 1, 1, 1)[0].all()


def test_logprob_against_torch_and_closed_forms():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 40)) * 3
    t = np.array([3, 39, -1, 0, 17])
    f = parts.token_logprob_fwd(x, t, 4)
    lp = torch.log_softmax(torch.from_numpy(x), 1).numpy()
    np.testing.assert_allclose(f["logp"], np.where(t < 0, 0, lp[np.arange(5), t]), atol=1e-13)
    np.testing.assert_allclose(f["entropy"], -(np.exp(lp) * lp).sum(1), atol=1e-13)
    for r in range(5):
        assert sorted(f["top_logp"][r], reverse=True) == list(f["top_logp"][r])
        np.testing.assert_allclose(f["top_logp"][r], lp[r, f["top_id"][r]])
    u = parts.token_logprob_fwd(np.full((1, 64), -2.5), np.array([9]), 3)
    np.testing.assert_allclose([u["entropy"][0], -u["logp"][0]], np.log(64))
    assert u["top_id"][0].tolist() == [0, 1, 2]                # ties by index


def test_logprob_backward_is_the_difference():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 9)) * 2
    x[1, 4] = -np.inf
    t, up, de = np.array([2, -1]), np.array([1.5, 7.0]), np.array([-0.4, 0.8])
    got = parts.token_logprob_bwd(x, t, up, de)

    def loss(v):
        f = parts.token_logprob_fwd(v, t)
        return np.stack([f["logp"], f["entropy"]], 1)

    x0 = x.copy()
    x0[1, 4] = -50.0
    want = _diff(loss, x0, np.stack([up, de], 1))
    np.testing.assert_allclose(got, want, atol=1e-7)
    assert got[1, 4] == 0
