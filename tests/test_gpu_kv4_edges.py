"""The attention over the 4-bit cache where its inputs are at an edge: slots
outside the block table, scores beyond fp32's range, more sequences than a
wave has lanes."""

import numpy as np
import pytest
import torch

import kv4_ref as ref
from gpu_util import q8 as _q8, to_dev
from test_gpu_kv4 import Step, host, i32, rotated_within

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


# positions whose score overflows to -inf, of how many, window, query heads
LOST = [
    (np.arange(32), 200, 0, 1),               # the first step of one wave
    (np.arange(32), 200, 0, 9),               # the same with 16 rows a tile
    (np.r_[0:32, 128:160], 200, 0, 3),        # all that one wave sees
    (np.array([31]), 190, 159, 2),            # the one position a window leaves of its first step
    (np.arange(1300), 3000, 0, 2),            # whole parts of a cut sequence
    (np.r_[0:700, 1500:3000], 3000, 0, 12),
    (np.arange(1, 90), 90, 0, 4),             # all but the first position
]


@pytest.mark.parametrize("lost,length,window,group", LOST)
def test_scores_of_minus_infinity_only_lose_their_positions(q8, lost, length, window, group):
    """A row with positions whose scores overflow to -inf is the attention
    over its other positions, wherever a wave's steps and a sequence's parts
    begin.  Those have score zero here: their weights are equal."""
    s = Step(q8, 32, 1, group, 1, 32, [length], window=window)
    k = np.zeros((length, 1, 32), np.float32)
    k[lost, 0, 0] = 3e38
    s.put(0, np.arange(length), k, s.v[0])
    s.q[:] = 0
    s.q[0, ::32] = -1e10
    seen = np.setdiff1d(np.arange(max(0, length - window) if window else 0, length), lost)
    v = ref.hold(s.v[0])[seen, 0]
    want, tol = ref.attend(np.zeros((1, 32)), np.zeros_like(v), v, [len(seen) - 1], s.scale)
    got = s.run()[0]
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all()


# sequences, tokens, kv heads, group, longest; with workgroups that share a
# compute unit: 3 with up to 8 rows a head, else 2
MANY = [(150, 1, 4, 4, 1200, 3), (70, 5, 2, 4, 1300, 2), (300, 1, 4, 2, 600, 3), (129, 3, 1, 2, 4000, 3)]


@pytest.mark.parametrize("n,tokens,kv,group,longest,on_cu", MANY)
def test_many_sequences_end_to_end(q8, n, tokens, kv, group, longest, on_cu):
    """More sequences than a wave has lanes, and more steps than shares run at
    once: they are measured 64 at a time while the shares are walked.  Some
    are idle, one has no slot."""
    rng = np.random.default_rng(n)
    lens = rng.integers(tokens, longest, n).tolist()
    lens[64] = tokens
    row_blocks = 1 if on_cu == 3 else -(-tokens * group // 16)
    least = sum(-(-L // 256) * 8 for L in lens) * row_blocks   # steps, a unit's rounded up to 8
    assert least > 8 * (256 * on_cu // kv)
    s = Step(q8, 64, kv, group, tokens, 32, lens, slots=n)
    s.pos[[1, 63, 65]] = -1
    s.seq[66 * tokens:67 * tokens] = n
    got = s.run()
    want, tol = s.want()
    off = slice(66 * tokens, 67 * tokens)
    assert np.isnan(got[off]).all()
    got[off] = want[off]
    assert (np.abs(got - want) <= tol).all()
    again = s.run()
    again[off] = want[off]
    assert np.array_equal(again, got)
    assert not s.ws[:1 << 20].any()


def test_plan_of_a_models_own_frequencies(q8):
    """A YaRN whose ramp is linear in the pair's index, which is not "yarn":
    its frequencies and amplitude make a plan of their own."""
    rot, base, factor, context = 128, 1e6, 4.0, 32768.0
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)

    def index(turns):
        return rot * np.log(context / (2 * np.pi * turns)) / (2 * np.log(base))
    first, last = np.floor(index(32.0)), np.ceil(index(1.0))
    kept = 1 - np.clip((i - first) / (last - first), 0, 1)
    own = (1 - kept) * f / factor + kept * f
    by_turns, amplitude = q8.rotary_frequencies(rot, base, "yarn", factor, context)
    ratio = own / by_turns.numpy()
    assert 1.7 < ratio.max() < 1.72 and (np.abs(ratio[np.r_[0:24, 40:64]] - 1) < 1e-12).all()
    rng = np.random.default_rng(9)
    x = rng.standard_normal((17, 3, rot), dtype=np.float32)
    pos = rng.integers(0, 131072, 17)
    plan = q8.Rotary(to_dev(own), amplitude=amplitude)
    y = torch.empty(17, 3 * rot, device="cuda")
    q8.q8_rotary(to_dev(x.reshape(17, -1)), y, 17, 3 * rot, i32(pos), 3, rot, plan)
    assert rotated_within(host(y).reshape(17, 3, rot), x, pos, own, False, amplitude)
