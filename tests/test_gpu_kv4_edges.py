"""The attention over the 4-bit cache where its inputs are at an edge: slots
outside the block table, scores beyond fp32's range, more sequences than a
wave has lanes."""

import numpy as np
import pytest
import torch

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


@pytest.mark.parametrize("tokens,group", [(1, 5), (4, 5)])
@pytest.mark.parametrize("slot", ["n_slots", 2 ** 31 - 1, -2 ** 31])
def test_slots_outside_the_table(q8, tokens, group, slot):
    """A sequence whose slot lies outside the table gives NaN, however far
    outside, and leaves its neighbours alone; idle rows give zeros even there."""
    s = Step(q8, 64, 2, group, tokens, 64, [300, 40, 600, 90])
    bad = s.cache.n_slots if slot == "n_slots" else slot
    t = tokens
    s.seq[1 * t:2 * t] = bad
    s.seq[3 * t:4 * t] = bad
    s.pos[3] = -1
    got = s.run()
    want, tol = s.want()
    assert np.isnan(got[t:2 * t]).all()
    assert (got[3 * t:] == 0).all()
    for i in (0, 2):
        rows = slice(i * t, (i + 1) * t)
        assert (np.abs(got[rows] - want[rows]) <= tol[rows]).all()
    assert not s.ws[:1 << 20].any()
    assert np.array_equal(s.run(), got, equal_nan=True)
