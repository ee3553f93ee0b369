"""The attention's arithmetic: results that depend on every piece of the queries
and of the softmax weights, within the roundings that kv4_exact.py counts."""

import numpy as np
import pytest
import torch

import kv4_exact as ke
from gpu_util import q8 as _q8
from test_gpu_kv4 import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    assert _q8().q8_device_supported(), "device is not gfx950"
    yield
    torch.cuda.synchronize()


@pytest.fixture(scope="module")
def q8():
    return _q8()


# kv heads, group, dim: 8 rows a tile (folded) and 16, blocks in one operand and two
SHAPES = [(2, 6, 64), (1, 12, 64), (3, 8, 96), (1, 16, 128), (1, 7, 160), (1, 13, 256)]
# a window of two positions that lie in one lane's word, in two lanes, on both
# sides of a tile, of a step and of a page
LENGTHS = [2, 4, 18, 33, 64, 97, 101]


@pytest.mark.parametrize("kv,group,dim", SHAPES)
@pytest.mark.parametrize("case", [ke.piece_case, ke.weight_case])
def test_two_positions(q8, case, kv, group, dim):
    q, k, v, scale, want, tol = case(group, dim)
    s = Step(q8, dim, kv, group, 1, 32, LENGTHS, window=2, scale=scale)
    for i, n in enumerate(LENGTHS):
        s.put(i, np.arange(n - 2, n), np.repeat(k[:, None], kv, 1), np.repeat(v[:, None], kv, 1))
    s.q[:] = np.tile(q, (kv, 1)).reshape(-1)
    err = np.abs(s.run().reshape(len(LENGTHS), kv, group, dim) - want)
    assert (err <= tol).all(), f"worst error / tolerance {(err / np.maximum(tol, 1e-300)).max():.3g}"


@pytest.mark.parametrize("dim,kv,group,tokens,lens", [
    (64, 3, 4, 1, [77, 600, 1500]),
    (128, 2, 5, 1, [65, 512, 1100]),
    (128, 2, 5, 4, [35, 515, 1200]),
    (96, 1, 2, 17, [64, 900]),
    (160, 2, 4, 1, [555, 31]),
    (256, 1, 16, 1, [700]),
])
def test_norm_of_the_error(q8, dim, kv, group, tokens, lens):
    s = Step(q8, dim, kv, group, tokens, 32, lens)
    want, _ = s.want()
    d = (s.run() - want).reshape(len(lens), -1)
    error = np.sqrt((d ** 2).sum(1) / (want.reshape(len(lens), -1) ** 2).sum(1))
    assert (error <= ke.NORM).all(), error
