"""The feed-forward side's operators on the GPU against their 64-bit
definitions (tests/ffn_ref.py): microscaled blocks, products with 4-bit
weights, the gated block, and the norms around a block, at the shapes, slots and
values where they can go wrong.

Tolerances.  What a block holds: exact.  Sums of products that fit 24 bits in
the unit of their products: exact; others: ffn_ref.product and gated.  Norms are
computed in double and rounded once: half a step of fp32 and 2^-40 of the
largest term for the double arithmetic."""

import numpy as np
import pytest
import torch

import ffn_ref as ref
from gpu_util import q8 as _q8, to_dev

pytestmark = pytest.mark.gpu

FORMS = ("mx4", "mx6", "mx8")
PIECES = {"mx4": 1, "mx6": 1, "mx8": 2}


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


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def i32(a):
    return to_dev(np.asarray(a, dtype=np.int32))


def rows(seed, n, k, spread=1.0):
    r = np.random.default_rng(seed)
    x = r.standard_normal((n, k)) * np.exp(spread * r.standard_normal((n, k)))
    return x.astype(np.float32)


def acts_of(q8, x, form, n_slots=None):
    a = q8.Acts(n_slots or x.shape[0], x.shape[1], form)
    q8.q8_mx_quantize_acts(to_dev(x), x.shape[0], a)
    return a


def values(q8, acts, index=None, n=None):
    n = n or (acts.n_slots if index is None else len(index))
    out = torch.empty(n, acts.K, device="cuda")
    q8.q8_mx_read_acts(acts, None if index is None else i32(index), n, out)
    return host(out).astype(np.float64)


def same(a, b):
    """Equal, NaN to NaN, zeros of either sign."""
    return np.array_equal(a, b, equal_nan=True)


# ------------------------------------------------------------------- blocks

def edge_rows(form, k=256):
    """Values on, next to and between the codes, at many scales; the borders of
    the scale rule; blocks of zeros, denormals, the largest values."""
    g = ref.GRIDS[form]
    mid = (g[1:] + g[:-1]) / 2
    pts = np.concatenate([g, mid, mid * (1 - 2.0 ** -23), mid * (1 + 2.0 ** -23)])
    r = np.random.default_rng(7)
    out = []
    for e in (0, 1, -7, 30, -118, 118, -126, 122):
        b = np.resize(pts, (-(-pts.size // 31), 31))
        b = np.concatenate([np.full((b.shape[0], 1), g[-1]), b], 1) * r.choice([-1, 1], (b.shape[0], 32))
        out.append(b * 2.0 ** e)
        tops = np.array([1, 1 - 2.0 ** -23, 1 + 2.0 ** -23]) * ref.BORDER[form]
        out.append(np.concatenate([tops[:, None], np.tile(r.choice(pts, (1, 31)), (3, 1))], 1) * 2.0 ** e)
    out.append(np.zeros((2, 32)))
    out.append(np.full((1, 32), -0.0))
    out.append(np.resize([2.0 ** -149, -2.0 ** -140, 2.0 ** -126, 2.0 ** -122], (1, 32)))
    out.append(np.resize([3.4028234663852886e38, -3.4e38, 1e38, 1e-38], (1, 32)))
    with np.errstate(over="ignore"):
        x = np.concatenate(out).astype(np.float32)
    x[~np.isfinite(x)] = 3e38
    x = np.resize(x, (-(-x.size // k), k))
    return np.ascontiguousarray(x)


@pytest.mark.parametrize("form", FORMS)
def test_blocks_hold_the_nearest_codes(q8, form):
    for x in (edge_rows(form), rows(1, 37, 96, 3.0), rows(2, 3, 32), rows(3, 130, 1056, 0.5)):
        got = values(q8, acts_of(q8, x, form))
        want = ref.hold(x, form)
        assert same(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("form", FORMS)
def test_blocks_that_are_not_finite_read_as_nan(q8, form):
    x = rows(4, 5, 160)
    x[1, 33] = np.nan
    x[2, 159] = np.inf
    x[4, 0] = -np.inf
    got = values(q8, acts_of(q8, x, form))
    assert same(got, ref.hold(x, form))
    assert np.isnan(got[1, 32:64]).all() and not np.isnan(got[1, 64:]).any()


@pytest.mark.parametrize("form", FORMS)
def test_other_slots_stay_as_they_are(q8, form):
    x = rows(5, 19, 96)
    a = q8.Acts(40, 96, form)
    a.data.fill_(0xA5)
    before = values(q8, a)
    q8.q8_mx_quantize_acts(to_dev(x), 19, a)
    got = values(q8, a)
    assert same(got[:19], ref.hold(x, form)) and same(got[19:], before[19:])


@pytest.mark.parametrize("form", FORMS)
def test_quantise_rows_at_any_stride_and_alignment(q8, form):
    big = to_dev(rows(6, 1, 9 * 203 + 64)[0])
    for off, stride in ((0, 128), (1, 203), (4, 132), (3, 97)):
        x = torch.as_strided(big, (9, 96), (stride, 1), off)
        a = q8.Acts(16, 96, form)
        q8.q8_mx_quantize_acts(big[off:], 9, a, x_stride=stride)
        assert same(values(q8, a, n=9), ref.hold(host(x.contiguous()), form))


def test_read_by_index(q8):
    x = rows(7, 20, 64)
    a = acts_of(q8, x, "mx6")
    index = [3, 3, 19, 0, -1, 20, 1 << 30, -(1 << 31)]
    got = values(q8, a, index)
    assert same(got[:4], ref.hold(x[[3, 3, 19, 0]], "mx6")) and np.isnan(got[4:]).all()


@pytest.mark.parametrize("n,k", [(1, 32), (17, 96), (16, 128), (100, 544), (33, 2080)])
def test_weights_pack_import_and_export(q8, n, k):
    x = rows(8, n, k, 2.0)
    x[0, 5] = np.nan if n > 1 else 1.0
    w = q8.MX4Weights(n, k)
    w.data.fill_(0xFF)
    q8.q8_mx4_pack_weights(to_dev(x), w)
    codes = torch.full((n, k // 2), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, k // 32), 0x55, dtype=torch.uint8, device="cuda")
    q8.q8_mx4_unpack_weights(w, codes, scales)
    i, neg, e = ref.codes(x, "mx4")
    good = np.repeat(e != 128, 16, axis=1)
    assert np.array_equal(host(scales), (e + 127).astype(np.uint8))
    assert np.array_equal(host(codes)[good], ref.mx4_bytes(i, neg)[good])
    again = q8.MX4Weights(n, k)
    again.data.fill_(0x3C)
    q8.q8_mx4_pack_weights_q(codes, scales, again)
    q8.q8_mx4_unpack_weights(again, *(back := [torch.empty_like(codes), torch.empty_like(scales)]))
    assert torch.equal(back[0], codes) and torch.equal(back[1], scales)
    # any bytes come back as they were put in
    r = np.random.default_rng(9)
    c, s = (to_dev(r.integers(0, 256, (n, k // d), dtype=np.uint8)) for d in (2, 32))
    q8.q8_mx4_pack_weights_q(c, s, again)
    q8.q8_mx4_unpack_weights(again, codes, scales)
    assert torch.equal(c, codes) and torch.equal(s, scales)


# ------------------------------------------------------------------ product

def integer_case(seed, form, n, k, slots):
    """Weights and activations whose products are whole multiples of one unit and
    whose sums stay below 2^24 of them: (codes, scales, weights, x, x held)."""
    r = np.random.default_rng(seed)
    idx, neg = r.integers(0, 8, (n, k)), r.integers(0, 2, (n, k))
    scales = np.full((n, k // 32), 127, np.uint8)
    g = ref.GRIDS[form]
    x = g[r.integers(0, len(g), (slots, k))] * r.choice([-1, 1], (slots, k))
    x[:, ::32] = g[-1]  # the scale of every block is 1
    x = x.astype(np.float32)
    assert same(ref.hold(x, form), x)
    codes = ref.mx4_bytes(idx, neg)
    return codes, scales, ref.mx4_values(codes, scales), x


def weights_of(q8, codes, scales):
    w = q8.MX4Weights(codes.shape[0], codes.shape[1] * 2)
    w.data.fill_(0xEE)
    q8.q8_mx4_pack_weights_q(to_dev(codes), to_dev(scales), w)
    return w


SHAPES = [(1, 32, 1), (1, 32, 70), (16, 128, 16), (17, 160, 5), (130, 544, 17), (48, 5120, 33), (33, 1056, 49),
          (40, 2080, 64), (100, 8736, 3), (520, 640, 65), (257, 512, 300), (300, 96, 513), (64, 1280, 1000)]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,k,live", SHAPES)
def test_product_is_exact_where_the_sums_fit(q8, form, n, k, live):
    codes, scales, w, x = integer_case(n + k, form, n, k, live + 3)
    index = np.random.default_rng(live).integers(0, live + 3, live)
    y = torch.full((live, n), 7.0, device="cuda")
    q8.q8_mx4_matmul(weights_of(q8, codes, scales), acts_of(q8, x, form), i32(index), live, y)
    assert np.array_equal(host(y).astype(np.float64), x[index].astype(np.float64) @ w.T)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,k,live", [(37, 96, 4), (200, 1184, 16), (65, 5120, 61), (130, 800, 200), (513, 17408, 16)])
def test_product_of_real_weights(q8, form, n, k, live):
    wf, x = rows(11, n, k, 0.7) * np.float32(0.02), rows(12, live, k, 1.0)
    w = q8.MX4Weights(n, k)
    q8.q8_mx4_pack_weights(to_dev(wf), w)
    y = torch.empty(live, n, device="cuda")
    q8.q8_mx4_matmul(w, acts_of(q8, x, form), None, live, y)
    want, tol = ref.product(ref.hold(wf, "mx4"), ref.hold(x, form), PIECES[form])
    assert (np.abs(host(y) - want) <= tol).all()


def test_product_with_scales_far_apart(q8):
    """Every scale byte that a block can have, as long as the sums stay in range."""
    r = np.random.default_rng(13)
    n, k = 24, 512
    codes = r.integers(0, 256, (n, k // 2), dtype=np.uint8)
    scales = r.integers(67, 187, (n, k // 32), dtype=np.uint8)
    x = (rows(14, 16, k) * np.repeat(2.0 ** r.integers(-60, 60, (16, k // 32)), 32, axis=1)).astype(np.float32)
    for form in FORMS:
        y = torch.empty(16, n, device="cuda")
        q8.q8_mx4_matmul(weights_of(q8, codes, scales), acts_of(q8, x, form), None, 16, y)
        want, tol = ref.product(ref.mx4_values(codes, scales), ref.hold(x, form), PIECES[form])
        assert (np.abs(host(y) - want) <= tol).all(), form


@pytest.mark.parametrize("live", [16, 100, 300])
def test_nan_stays_in_its_row_and_column(q8, live):
    codes, scales, w, x = integer_case(15, "mx8", 40, 256, live)
    scales = scales.copy()
    scales[7, 3] = 255
    x[5, 70] = np.nan
    x[live - 1, 0] = np.inf
    for form in FORMS:
        y = torch.empty(live, 40, device="cuda")
        xf = x if form == "mx8" else np.where(np.isfinite(x), ref.hold(x, form), x).astype(np.float32)
        q8.q8_mx4_matmul(weights_of(q8, codes, scales), acts_of(q8, xf, form), None, live, y)
        got = host(y)
        assert np.isnan(got[5]).all() and np.isnan(got[live - 1]).all() and np.isnan(got[:, 7]).all()
        got = np.delete(np.delete(got, [5, live - 1], 0), 7, 1)
        held = ref.hold(np.delete(xf, [5, live - 1], 0), form)
        assert np.array_equal(got.astype(np.float64), held @ np.delete(w, 7, 0).T), form


@pytest.mark.parametrize("live", [6, 70, 400])
def test_slots_outside_the_buffer_give_nan_rows(q8, live):
    codes, scales, w, x = integer_case(16, "mx6", 50, 96, 9)
    index = np.random.default_rng(live).integers(0, 9, live)
    index[[1, 4, live - 1]] = [-1, 9, 1 << 30]
    y = torch.empty(live, 50, device="cuda")
    q8.q8_mx4_matmul(weights_of(q8, codes, scales), acts_of(q8, x, "mx6"), i32(index), live, y)
    bad = (index < 0) | (index >= 9)
    got = host(y)
    assert np.isnan(got[bad]).all()
    assert np.array_equal(got[~bad].astype(np.float64), x[index[~bad]].astype(np.float64) @ w.T)


def test_output_rows_at_a_stride(q8):
    codes, scales, w, x = integer_case(17, "mx4", 45, 160, 200)
    for live in (3, 200):
        for stride, off in ((45, 0), (61, 1), (64, 0), (48, 2)):
            y = torch.full((live * stride + 8,), 7.0, device="cuda")
            q8.q8_mx4_matmul(weights_of(q8, codes, scales), acts_of(q8, x, "mx4"), None, live, y[off:], y_stride=stride)
            got = host(y)[off:off + live * stride].reshape(live, stride)
            assert np.array_equal(got[:, :45].astype(np.float64), x[:live].astype(np.float64) @ w.T)
            assert (got[:-1, 45:] == 7).all() and (host(y)[off + live * stride - stride + 45:] == 7).all()


# Large tiles (enough of them that blocks of 64 tokens take longer), small and large, with
# ends in both directions: by cost, not by these sizes.
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,k,live", [(2077, 544, 1290), (4093, 160, 3701), (2080, 96, 3700), (7001, 1184, 515)])
def test_product_in_large_tiles(q8, form, n, k, live):
    codes, scales, w, x = integer_case(n + live, form, n, k, 700)
    index = np.random.default_rng(live).integers(0, 700, live)
    index[[3, live - 1]] = [-1, 700]
    y = torch.full((live + 1, n), 7.0, device="cuda")
    q8.q8_mx4_matmul(weights_of(q8, codes, scales), acts_of(q8, x, form), i32(index), live, y)
    got = host(y)
    good = np.ones(live + 1, bool)
    good[[3, live - 1, live]] = False
    assert np.isnan(got[[3, live - 1]]).all() and (got[live] == 7).all()
    want = (x.astype(np.float64) @ w.T)[index[good[:live]]]
    assert np.array_equal(got[good].astype(np.float64), want)


# Super-chunks of 512 columns: 13 and 16 (two a wave, kept), 18 and 34 (fetched again), odd ones.
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,k", [(53, 6176), (53, 6432), (40, 8192), (53, 8736), (33, 17408), (530, 6688)])
def test_product_and_gated_of_wide_rows(q8, form, n, k):
    codes, scales, w, x = integer_case(k, form, n, k, 21)
    for live in (1, 16, 21):
        y = torch.empty(live, n, device="cuda")
        q8.q8_mx4_matmul(weights_of(q8, codes, scales), acts_of(q8, x, form), None, live, y)
        assert np.array_equal(host(y).astype(np.float64), x[:live].astype(np.float64) @ w.T)
        h = torch.empty(live, n, device="cuda")
        one = weights_of(q8, codes, scales)
        q8.q8_mx4_gated(one, one, acts_of(q8, x, form), None, live, H=h, activation="identity")
        v = (x[:live].astype(np.float64) @ w.T).astype(np.float32)
        assert np.array_equal(host(h), v * v)


# Long rows, the most tokens, 2^20 rows.  Signs are random, so that a partial sum of 2^17
# products of at most 12 x 127 units has a deviation of at most 2^8.5 x 1524 = 5.6e5: 2^24 are 30.
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,k,live", [(17, 1 << 17, 3), (17, 1 << 17, 40), (16, 32, 1 << 20), (1 << 20, 32, 3),
                                      (1 << 20, 32, 33)])
def test_product_at_the_ends_of_its_ranges(q8, form, n, k, live):
    codes, scales, w, x = integer_case(n + live, form, n, k, 50)
    index = np.random.default_rng(live).integers(0, 50, live)
    y = torch.empty(live, n, device="cuda")
    q8.q8_mx4_matmul(weights_of(q8, codes, scales), acts_of(q8, x, form), i32(index), live, y)
    want = (x.astype(np.float64) @ w.T).astype(np.float32)
    assert torch.equal(y, to_dev(want)[torch.from_numpy(index).cuda()])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("slots", [64, 65, 700])
def test_the_same_rows_in_buffers_of_any_size(q8, form, slots):
    codes, scales, w, x = integer_case(slots, form, 97, 1312, slots)
    a, m = acts_of(q8, x, form), weights_of(q8, codes, scales)
    assert same(values(q8, a), x)
    want = x.astype(np.float64) @ w.T
    for live in (1, 9, 16, 17, 33, 64, 80):
        for index in (np.random.default_rng(live).integers(0, slots, live), np.full(live, slots - 1),
                      np.arange(live)[::-1] % slots):
            y = torch.empty(live, 97, device="cuda")
            q8.q8_mx4_matmul(m, a, i32(index), live, y)
            assert np.array_equal(host(y).astype(np.float64), want[index]), live
            h, held = torch.empty(live, 97, device="cuda"), q8.Acts(slots, 96, form)
            q8.q8_mx4_gated(m, m, a, i32(index), live, H=h, activation="identity")
            v = want[index].astype(np.float32)
            assert np.array_equal(host(h), v * v), live
    few = q8.MX4Weights(96, 1312)
    q8.q8_mx4_pack_weights_q(to_dev(codes[:96]), to_dev(scales[:96]), few)
    for live in (9, 40):
        held, want_held = (q8.Acts(slots, 96, form) for _ in range(2))
        for b in (held, want_held):
            b.data.fill_(0x29)
        h = torch.empty(live, 96, device="cuda")
        q8.q8_mx4_gated(few, few, a, None, live, H=h, h_acts=held)
        q8.q8_mx_quantize_acts(h, live, want_held)
        assert torch.equal(held.data, want_held.data)


# The order of a row's sums is one up to 16 tokens, another in blocks of 64.
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("most,lives", [(16, (1, 5, 15)), (130, (17, 33, 40, 63, 64, 100))])
def test_a_row_does_not_depend_on_the_others(q8, form, most, lives):
    n, k = 70, 2592
    x, wf = rows(18, most, k, 3.0), rows(19, n, k, 3.0)
    w, a = q8.MX4Weights(n, k), acts_of(q8, x, form)
    q8.q8_mx4_pack_weights(to_dev(wf), w)
    full = torch.empty(most, n, device="cuda")
    q8.q8_mx4_matmul(w, a, None, most, full)
    for live in lives:
        index = np.random.default_rng(live).permutation(most)[:live]
        y = torch.empty(live, n, device="cuda")
        q8.q8_mx4_matmul(w, a, i32(index), live, y)
        assert torch.equal(y, full[torch.from_numpy(index).cuda()])


# -------------------------------------------------------------------- gated

ACTIVATIONS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid", "identity")


@pytest.mark.parametrize("kind", ACTIVATIONS)
@pytest.mark.parametrize("n,k,live,form", [(1, 32, 1, "mx8"), (33, 160, 5, "mx6"), (96, 1184, 16, "mx8"),
                                           (50, 640, 61, "mx4"), (160, 544, 70, "mx8"), (250, 512, 300, "mx6")])
def test_gated(q8, kind, n, k, live, form):
    r = np.random.default_rng(n)
    wf = [(rows(20 + i, n, k, 0.3) * np.float32(3 / k ** 0.5)) for i in range(2)]
    x = rows(22, live + 2, k, 0.3)
    x[0] *= 8  # far into the activation's tails
    w = [q8.MX4Weights(n, k) for _ in wf]
    for a, b in zip(wf, w):
        q8.q8_mx4_pack_weights(to_dev(a), b)
    index = r.integers(0, live + 2, live)
    index[0] = 0
    h = torch.empty(live, n, device="cuda")
    q8.q8_mx4_gated(*w, acts_of(q8, x, form), i32(index), live, H=h, activation=kind)
    want, tol = ref.gated(*(ref.hold(a, "mx4") for a in wf), ref.hold(x, form)[index], PIECES[form], kind)
    assert (np.abs(host(h) - want) <= tol).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("out", FORMS)
@pytest.mark.parametrize("n,k,live", [(32, 96, 1), (160, 640, 16), (96, 5152, 40), (544, 256, 64), (416, 160, 90),
                                      (288, 512, 261)])
def test_gated_quantised_rows_are_the_quantised_fp32_rows(q8, form, out, n, k, live):
    w = [q8.MX4Weights(n, k) for _ in range(2)]
    for i, b in enumerate(w):
        q8.q8_mx4_pack_weights(to_dev(rows(30 + i, n, k) * np.float32(2 / k ** 0.5)), b)
    a = acts_of(q8, rows(32, live, k), form)
    h, alone = torch.empty(live, n, device="cuda"), q8.Acts(live + 20, n, out)
    both = q8.Acts(live + 20, n, out)
    want = q8.Acts(live + 20, n, out)
    for b in (alone, both, want):
        b.data.fill_(0x41)
    q8.q8_mx4_gated(*w, a, None, live, H=h, h_acts=both)
    q8.q8_mx4_gated(*w, a, None, live, h_acts=alone)
    q8.q8_mx_quantize_acts(h, live, want)
    assert torch.equal(both.data, want.data) and torch.equal(alone.data, want.data)


@pytest.mark.parametrize("kind", ACTIVATIONS)
@pytest.mark.parametrize("n,k,live,form", [(1050, 288, 1300, "mx8"), (4095, 96, 1900, "mx4"), (4095, 96, 1900, "mx8")])
def test_gated_in_large_tiles(q8, kind, n, k, live, form):
    wf = [(rows(24 + i, n, k, 0.3) * np.float32(3 / k ** 0.5)) for i in range(2)]
    x = rows(26, 90, k, 0.3)
    x[0] *= 8
    w = [q8.MX4Weights(n, k) for _ in wf]
    for a, b in zip(wf, w):
        q8.q8_mx4_pack_weights(to_dev(a), b)
    index = np.random.default_rng(n).integers(0, 90, live)
    h = torch.empty(live, n, device="cuda")
    q8.q8_mx4_gated(*w, acts_of(q8, x, form), i32(index), live, H=h, activation=kind)
    want, tol = ref.gated(*(ref.hold(a, "mx4") for a in wf), ref.hold(x, form), PIECES[form], kind)
    assert (np.abs(host(h) - want[index]) <= tol[index]).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,k,live", [(4096, 96, 1900), (1056, 160, 1300)])
def test_gated_quantised_rows_in_large_tiles(q8, form, n, k, live):
    w = [q8.MX4Weights(n, k) for _ in range(2)]
    for i, b in enumerate(w):
        q8.q8_mx4_pack_weights(to_dev(rows(36 + i, n, k) * np.float32(2 / k ** 0.5)), b)
    a = acts_of(q8, rows(38, live, k), form)
    for out in FORMS:
        h, both, want = torch.empty(live, n, device="cuda"), q8.Acts(live + 20, n, out), q8.Acts(live + 20, n, out)
        both.data.fill_(0x41), want.data.fill_(0x41)
        q8.q8_mx4_gated(*w, a, None, live, H=h, h_acts=both)
        q8.q8_mx_quantize_acts(h, live, want)
        assert torch.equal(both.data, want.data)


@pytest.mark.parametrize("live", [9, 150])
def test_gated_nan(q8, live):
    w = [q8.MX4Weights(64, 96) for _ in range(2)]
    wf = [rows(33 + i, 64, 96) for i in range(2)]
    wf[0][3, 0], wf[1][40, 95] = np.inf, np.nan
    for a, b in zip(wf, w):
        q8.q8_mx4_pack_weights(to_dev(a), b)
    x = rows(35, live, 96)
    x[4, 1] = np.nan
    index = np.arange(live)
    index[2] = live
    h, m = torch.empty(live, 64, device="cuda"), q8.Acts(live, 64, "mx8")
    for kind in ACTIVATIONS:
        q8.q8_mx4_gated(*w, acts_of(q8, x, "mx8"), i32(index), live, H=h, h_acts=m, activation=kind)
        got, held = host(h), values(q8, m)
        assert np.isnan(got[[2, 4]]).all() and np.isnan(got[:, [3, 40]]).all() and np.isnan(held[[2, 4]]).all()
        rest = np.delete(np.delete(got, [2, 4], 0), [3, 40], 1)
        assert np.isfinite(rest).all() and np.isnan(held).all()  # each block of 32 features has one of the two


# -------------------------------------------------------------------- norms

def norm_tensors(seed, n, k, per_row):
    r = np.random.default_rng(seed)
    shape = (n, k) if per_row else (k,)
    return [(1 + 0.3 * r.standard_normal(shape)).astype(np.float32), r.standard_normal(shape).astype(np.float32)]


def check_norm(q8, n, k, post, pre, gate, residual, per_row=False, scale=0.37, offset=1.0, seed=0, bias=None,
               in_place=False):
    x, r = rows(seed, n, k), rows(seed + 1, n, k)
    g = None if gate is None else rows(seed + 2, n, k)[:n if gate == "rows" else 1]
    norms, args = [], []
    for i, kind in enumerate((post, pre)):
        if kind is None:
            norms.append(None), args.append((None, None, None))
            continue
        w, b = norm_tensors(seed + 3 + i, n, k, per_row)
        if not (bias if bias is not None else kind == "layer"):
            b = None
        norms.append(q8.Norm(k, kind, to_dev(w), None if b is None else to_dev(b), eps=1e-5, offset=offset))
        args.append((kind, w, b))
    xd, rd = to_dev(x), to_dev(r)
    ro, y = (rd, xd) if in_place else (torch.empty_like(xd), torch.empty_like(xd))
    q8.q8_norm_step(xd, n, k, post=norms[0], gate=None if g is None else to_dev(g if gate == "rows" else g[0]),
                    scale=scale, residual=rd if residual else None, residual_out=ro, pre=norms[1], Y=y)
    b = ref.norm(x.astype(np.float64), *args[0], 1e-5, offset)
    t = float(np.float32(scale)) * b * (1.0 if g is None else g.astype(np.float64))
    big = np.abs(t) + np.abs(t).max(-1, keepdims=True) + np.abs(r)
    t = t + (r.astype(np.float64) if residual else 0.0)
    got = host(ro).astype(np.float64)
    assert (np.abs(got - t) <= ref.U * np.abs(t) + 2.0 ** -40 * big + 2.0 ** -149).all()
    want = ref.norm(got, *args[1], 1e-5, offset)
    tol = ref.U * np.abs(want) + 2.0 ** -40 * (np.abs(want).max(-1, keepdims=True) + 4) + 2.0 ** -149
    assert (np.abs(host(y) - want) <= tol).all()


@pytest.mark.parametrize("n,k", [(1, 1), (3, 2), (2, 31), (5, 64), (7, 255), (16, 768), (3, 1000), (4, 2049), (16, 5120),
                                 (2, 8192), (2, 16383), (1, 32768), (600, 320)])
def test_norm_widths(q8, n, k):
    check_norm(q8, n, k, None, "rms", None, True)
    check_norm(q8, n, k, "layer", "layer", "rows", True, per_row=True, offset=0.0)
    check_norm(q8, n, k, "rms", None, "shared", False)


@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("pre", [None, "rms", "layer"])
@pytest.mark.parametrize("gate", [None, "shared", "rows"])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_forms(q8, post, pre, gate, residual):
    check_norm(q8, 9, 416, post, pre, gate, residual, seed=50)
    check_norm(q8, 4, 99, post, pre, gate, residual, per_row=True, bias=True, scale=-2.0, offset=0.0, seed=60)


def test_norm_in_place(q8):
    check_norm(q8, 33, 1504, "rms", "rms", "shared", True, in_place=True)


def test_norm_without_weights(q8):
    x = rows(70, 6, 200)
    y = torch.empty(6, 200, device="cuda")
    for kind in ("rms", "layer"):
        q8.q8_norm_step(to_dev(x), 6, 200, pre=q8.Norm(200, kind, eps=1e-3), Y=y)
        want = ref.norm(x.astype(np.float64), kind, None, None, 1e-3, 0.0)
        assert (np.abs(host(y) - want) <= ref.U * np.abs(want) + 2.0 ** -40 * 20).all()


def test_norm_rows_at_strides(q8):
    n, k = 5, 130
    for stride, off in ((131, 1), (132, 4), (200, 0), (130, 3)):
        big = to_dev(rows(71, 1, n * stride + 64)[0])
        out = torch.full((n * stride + 64,), 7.0, device="cuda")
        y = torch.full((n * stride + 64,), 7.0, device="cuda")
        x = host(torch.as_strided(big, (n, k), (stride, 1), off).contiguous())
        q8.q8_norm_step(big[off:], n, k, residual=big[off:], residual_out=out[off:], pre=q8.Norm(k), Y=y[off:],
                        x_stride=stride, residual_stride=stride, residual_out_stride=stride, y_stride=stride)
        got = host(torch.as_strided(out, (n, k), (stride, 1), off).contiguous())
        assert np.array_equal(got, x + x)
        got = host(torch.as_strided(y, (n, k), (stride, 1), off).contiguous())
        want = ref.norm((x + x).astype(np.float64), "rms", None, None, 1e-6, 0.0)
        assert (np.abs(got - want) <= ref.U * np.abs(want) + 2.0 ** -40 * 20).all()
        for t in (out, y):
            keep = np.ones(n * stride + 64, bool)
            for i in range(n):
                keep[off + i * stride:off + i * stride + k] = False
            assert (host(t)[keep] == 7).all()


def test_norm_far_offsets_and_tiny_rows(q8):
    """A layer norm of values that differ in their last bits only, values whose squares
    leave the range of fp32, and denormals."""
    r = np.random.default_rng(72)
    base = (1e4 + np.ldexp(r.integers(-8, 8, (4, 512)), -10)).astype(np.float32)
    for x in (base, rows(73, 4, 512) * np.float32(1e30), rows(74, 4, 512) * np.float32(1e-41)):
        for kind in ("layer", "rms"):
            y = torch.empty(4, 512, device="cuda")
            q8.q8_norm_step(to_dev(x), 4, 512, pre=q8.Norm(512, kind, eps=0.0), Y=y)
            want = ref.norm(x.astype(np.float64), kind, None, None, 0.0, 0.0)
            assert (np.abs(host(y) - want) <= ref.U * np.abs(want) + 2.0 ** -30).all()


def test_norm_values_that_are_not_finite_stay_in_their_row(q8):
    x = rows(75, 4, 96)
    x[1, 5], x[2, 90] = np.nan, np.inf
    a, y = q8.Acts(4, 96, "mx8"), torch.empty(4, 96, device="cuda")
    q8.q8_norm_step(to_dev(x), 4, 96, pre=q8.Norm(96), Y=y, acts=a)
    got, held = host(y), values(q8, a)
    assert np.isnan(got[1]).all() and np.isnan(got[2, 90]) and np.isnan(held[1]).all() and np.isnan(held[2, 64:]).all()
    assert np.isfinite(got[[0, 3]]).all() and np.isfinite(held[[0, 3]]).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,k,slots", [(1, 32, 1), (5, 160, 33), (16, 5120, 16), (40, 1056, 64), (3, 32768, 5), (70, 768, 70)])
def test_norm_quantises_as_the_quantiser_does(q8, form, n, k, slots):
    x, r = to_dev(rows(76, n, k)), to_dev(rows(77, n, k))
    y, both, alone, want = torch.empty(n, k, device="cuda"), *(q8.Acts(slots, k, form) for _ in range(3))
    for b in (both, alone, want):
        b.data.fill_(0x17)
    norm = q8.Norm(k, "rms", to_dev(rows(78, 1, k)[0]))
    q8.q8_norm_step(x, n, k, residual=r, pre=norm, Y=y, acts=both)
    q8.q8_norm_step(x, n, k, residual=r, pre=norm, acts=alone)
    q8.q8_mx_quantize_acts(y, n, want)
    assert torch.equal(both.data, want.data) and torch.equal(alone.data, want.data)


@pytest.mark.parametrize("n,k,slots", [(1, 32, 16), (16, 768, 16), (16, 5120, 16), (33, 1120, 48), (64, 288, 64)])
def test_norm_fills_q8_0_slots_as_their_quantiser_does(q8, n, k, slots):
    x = to_dev(rows(79, n, k))
    y, acts = torch.empty(n, k, device="cuda"), q8.Acts(slots, k, "q8_0")
    want = torch.full_like(acts.data, 0x17)
    acts.data.fill_(0x17)
    q8.q8_norm_step(x, n, k, pre=q8.Norm(k, "layer"), Y=y, acts=acts)
    q8.q8_quantize_acts_n(y, n, k, want, slots)
    assert torch.equal(acts.data, want)


# ------------------------------------------------------- a run of them together

class Block:
    """norm -> gated block -> down projection -> the next norm, on buffers of its own."""

    def __init__(self, q8, width, inner, live, form, seed=90):
        self.q8, self.width, self.inner, self.live = q8, width, inner, live
        self.f = [rows(seed + i, *s, 0.3) * np.float32(s[1] ** -0.5)
                  for i, s in enumerate(((inner, width), (inner, width), (width, inner)))]
        self.w = [q8.MX4Weights(*a.shape) for a in self.f]
        for a, b in zip(self.f, self.w):
            q8.q8_mx4_pack_weights(to_dev(a), b)
        self.nw = [to_dev(1 + 0.1 * rows(seed + 3 + i, 1, width)[0]) for i in range(2)]
        self.norms = [q8.Norm(width, "rms", w) for w in self.nw]
        self.x, self.h, self.next = q8.Acts(live, width, form), q8.Acts(live, inner, form), q8.Acts(live, width, form)
        self.stream = to_dev(rows(seed + 5, live, width))
        self.branch = to_dev(rows(seed + 6, live, width))
        self.y = torch.empty(live, width, device="cuda")

    def step(self):
        q8, n, w = self.q8, self.live, self.width
        q8.q8_norm_step(self.branch, n, w, residual=self.stream, residual_out=self.stream, pre=self.norms[0], acts=self.x)
        q8.q8_mx4_gated(self.w[0], self.w[1], self.x, None, n, h_acts=self.h)
        q8.q8_mx4_matmul(self.w[2], self.h, None, n, self.y)
        q8.q8_norm_step(self.y, n, w, residual=self.stream, residual_out=self.stream, scale=0.5, pre=self.norms[1],
                        acts=self.next)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("live", [1, 16, 130])
def test_feed_forward_half_of_a_layer(q8, form, live):
    b = Block(q8, 320, 864, live, form)
    s0 = host(b.stream).astype(np.float64) + host(b.branch)
    b.step()
    # each step from what the one before really held
    s1 = s0.astype(np.float32).astype(np.float64)
    x = values(q8, b.x)
    y = ref.norm(s1, "rms", host(b.nw[0]), None, 1e-6, 0.0).astype(np.float32)
    differ = (x != ref.hold(y, form)).mean()
    assert differ <= 1e-5, differ  # double arithmetic apart, the same blocks
    w = [ref.hold(a, "mx4") for a in b.f]
    h, tol = ref.gated(w[0], w[1], x, PIECES[form], "silu")
    held = values(q8, b.h)
    # a value within its tolerance of a border may fall to either side of it: one
    # code further in its block, whose steps are at most this part of the largest
    edge = np.abs(h).reshape(live, -1, 32).max(-1).repeat(32, -1) / {"mx4": 2, "mx6": 8, "mx8": 60}[form]
    assert (np.abs(held - ref.hold(h.astype(np.float32), form)) <= edge).all()
    assert (held != ref.hold(h.astype(np.float32), form)).mean() <= 1e-3
    y, tol = ref.product(w[2], held, PIECES[form])
    got = host(b.y)
    assert (np.abs(got - y) <= tol).all()
    s2 = s1 + 0.5 * got.astype(np.float64)
    assert (np.abs(host(b.stream) - s2) <= ref.U * np.abs(s2) + 2.0 ** -40).all()
    y = ref.norm(host(b.stream).astype(np.float64), "rms", host(b.nw[1]), None, 1e-6, 0.0).astype(np.float32)
    assert (values(q8, b.next) != ref.hold(y, form)).mean() <= 1e-5


@pytest.mark.parametrize("live", [16, 130])
def test_captured_and_replayed(q8, live):
    b, e = (Block(q8, 352, 1056, live, "mx8") for _ in range(2))
    b.step(), e.step()  # warm up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for i in range(4):
        fresh = to_dev(rows(100 + i, live, 352))
        b.branch.copy_(fresh), e.branch.copy_(fresh)
        graph.replay()
        e.step()
        torch.cuda.synchronize()
        for a, c in ((b.stream, e.stream), (b.y, e.y), (b.h.data, e.h.data), (b.next.data, e.next.data)):
            assert torch.equal(a, c), i


def test_two_streams_at_once(q8):
    blocks = [Block(q8, 352, 1056, live, "mx6", seed=110) for live in (16, 90, 16, 90)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in (2, 3):
        blocks[i].step()
    torch.cuda.synchronize()
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                blocks[i].step()
    for _ in range(2):
        for i in (2, 3):
            blocks[i].step()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert torch.equal(blocks[i].stream, blocks[i + 2].stream)
        assert torch.equal(blocks[i].next.data, blocks[i + 2].next.data)


def test_decode_feed_forward_example():
    """The example runs and stays finite."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decode_feed_forward.py")
    spec = importlib.util.spec_from_file_location("decode_feed_forward", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for form in FORMS:
        out = mod.main(["--live", "3", "--steps", "5", "--format", form])
        assert out["finite"] and out["format"] == form
