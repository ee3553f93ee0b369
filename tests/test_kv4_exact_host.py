"""The inputs of kv4_exact.py tell apart what they are made to tell apart: a
model that keeps every bit is within their tolerances, one that leaves out a
piece of the queries or of the weights is far outside."""

import numpy as np
import pytest

import kv4_exact as ke
import kv4_ref as ref


def test_pieces_hold_a_query():
    rng = np.random.default_rng(1)
    q = (rng.standard_normal((200, 64)) * np.exp(3 * rng.standard_normal((200, 64)))).astype(np.float32)
    q[0] = 0
    top = np.repeat(np.abs(q.reshape(200, 2, 32)).max(-1), 32, 1)
    for n, left in zip(range(1, 7), (-4, -9, -14, -19, -24, -29)):
        assert (np.abs(ke.cut_query(q, n) - q) <= 2.0 ** left * np.maximum(top, 1e-30) * 1.07).all(), n


def test_weights_are_cut_to_their_upper_bits():
    w = np.array([1.0, 1 - 2.0 ** -24, 2.0 ** -100 * (1 + 2.0 ** -15 + 2.0 ** -23)])
    assert np.array_equal(ke.cut_weight(w), w)
    assert np.array_equal(ke.cut_weight(w, 16), [1.0, 1 - 2.0 ** -16, 2.0 ** -100 * (1 + 2.0 ** -15)])


@pytest.mark.parametrize("heads,dim", [(6, 64), (12, 96)])
def test_each_piece_is_needed(heads, dim):
    q, k, v, scale, want, tol = ke.piece_case(heads, dim)
    assert np.array_equal(ref.hold(k), k) and np.array_equal(ref.hold(v), v)
    assert (np.abs(ke.model(q, k, v, scale) - want) <= tol).all()
    for pieces in range(6):
        far = np.abs(ke.model(q, k, v, scale, pieces) - want) > 1e4 * tol
        assert far[np.arange(heads) % 6 >= pieces].all(), pieces


@pytest.mark.parametrize("heads,dim", [(8, 64), (16, 96)])
def test_each_weight_piece_is_needed(heads, dim):
    q, k, v, scale, want, tol = ke.weight_case(heads, dim)
    assert np.array_equal(ref.hold(k), k) and np.array_equal(ref.hold(v), v)
    assert (np.abs(ke.model(q, k, v, scale) - want) <= tol).all()
    for bits, times in ((16, 4), (8, 1000)):
        assert (np.abs(ke.model(q, k, v, scale, bits=bits) - want) / tol).max() > times, bits


@pytest.mark.parametrize("dim,length", [(64, 300), (128, 1200)])
def test_the_norm_tells_weights_of_16_bits(dim, length):
    rng = np.random.default_rng(dim)
    q = rng.standard_normal((16, dim)).astype(np.float32)
    k = ref.hold(rng.standard_normal((length, dim)).astype(np.float32))
    v = ref.hold(rng.standard_normal((length, dim)).astype(np.float32))

    def error(**kw):
        d = ke.model(q, k, v, dim ** -0.5, **kw) - want
        return np.sqrt((d ** 2).sum() / (want ** 2).sum())
    s = dim ** -0.5 * q.astype(np.float64) @ k.T
    w = np.exp(s - s.max(-1, keepdims=True))
    want = w @ v / w.sum(-1, keepdims=True)
    assert error() <= ke.NORM / 4
    for kw in (dict(bits=16), dict(bits=8), dict(pieces=3), dict(pieces=2)):
        assert error(**kw) > 4 * ke.NORM, kw
