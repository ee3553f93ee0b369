"""The feed-forward side's operators on the GPU at the values, sizes and forms
that each choice of a kernel has an end at.  Tolerances as in test_gpu_ffn.py;
U is half a step of fp32 relative to a value, a rounding."""

import numpy as np
import pytest
import torch

import ffn_ref as ref
import ffn_shapes as shapes
import test_gpu_ffn as base
from gpu_util import q8 as _q8, to_dev

pytestmark = pytest.mark.gpu

U = ref.U


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


# -------------------------------------------------------------- activations

def gate_values(n, seed):
    """fp32 numbers over the activations' ranges, their ends and borders, with all 24 bits in use."""
    r = np.random.default_rng(seed)
    edges = [0.0, 1e-30, 1.0, 9.49, 9.5, 9.51, 12.0, 16.1, 79.9, 80.0, 80.1, 86.6, 87.4, 88.8, 95.0, 103.9, 104.5, 126.0,
             129.0, 174.0, 259.0, 261.0, 1e4, 1e18, 3e38]
    x = np.concatenate([edges, -np.array(edges), r.uniform(-4, 4, n // 4), r.uniform(-12, 12, n // 4), r.uniform(-110, 0, n // 4)])
    x = np.concatenate([x, r.uniform(-110, 110, n)])[:n] if n > len(edges) * 2 else r.permutation(x)[:n]
    return x.astype(np.float32)


def gates(q8, x, shifts):
    """([weights of the gate, of the up projection], activations, x as they hold it): token t's gate is x[t] / 2^shifts[f]
    at feature f without an error, its up projection 1.  x[t] comes in four pieces of 7 bits, each in a block of its
    own, the first of which saturates for x beyond a block's largest value."""
    acts = np.zeros((len(x), 160), np.float32)
    rest = x.astype(np.float64)
    unit = 2.0 ** (np.floor(np.log2(np.where(x == 0, 1, np.abs(rest)))) - 6)
    for i in range(4):
        q = np.trunc(rest / unit)
        acts[:, 32 * i] = q * unit
        rest, unit = rest - q * unit, unit / 128
    assert not rest.any()
    acts[:, 128] = 1.0
    n = len(shifts)
    codes, scales = np.zeros((2, n, 80), np.uint8), np.full((2, n, 5), 127, np.uint8)
    codes[0][:, [0, 16, 32, 48]] = 2  # 1.0 in the even column
    codes[1][:, 64] = 2
    scales[0] -= np.asarray(shifts, np.uint8)[:, None]
    w = [q8.MX4Weights(n, 160) for _ in range(2)]
    for c, s, to in zip(codes, scales, w):
        q8.q8_mx4_pack_weights_q(to_dev(c), to_dev(s), to)
    a = q8.Acts(len(x), 160, "mx8")
    q8.q8_mx_quantize_acts(to_dev(acts), len(x), a)
    return w, a, ref.hold(acts, "mx8")[:, :128].sum(-1)


def activation_and_bound(g, kind):
    """The activation of 64-bit numbers and the error of its fp32 form, in roundings.  exp(-y) is 2^t (1 + r): 2^t is
    good to a unit in the last place, 2; 1 + r is 1; log 2 in r's computation is off by 1.905e-9, which times y log2 e
    is 0.0462 |y|.  The sum with 1 is 1, its inverse 2, the product with x 1.  The tanh form's argument has errors of 3
    (x^2, the polynomial, its constants), each of which is |y| of exp(-y).  GELU's argument has 2, of which erfc makes
    2 v^2 + 1 each, and erfc itself 16 units.  A sigmoid below 2^-126 may be 0."""
    if kind in ("silu", "sigmoid", "gelu_tanh"):
        y = 2 * (2 / np.pi) ** 0.5 * (g + 0.044715 * g ** 3) if kind == "gelu_tanh" else g
        sig = torch.sigmoid(y)
        v = sig if kind == "sigmoid" else g * sig
        bound = 7 + (3 * y.abs() * torch.sigmoid(-y) if kind == "gelu_tanh" else 0.0462 * y.abs())
        bound = torch.where(sig <= 2.0 ** -126 * 1.001, 2.0 ** 25, bound.clamp(max=2.0 ** 23))
    elif kind == "gelu":
        v, bound = 0.5 * g * torch.special.erfc(-g * 0.5 ** 0.5), 36 + 2 * (g.clamp(max=0) ** 2 + 1)
    elif kind == "relu":
        v, bound = g.clamp(min=0), 0
    else:
        v, bound = g, 0
    v = torch.where(v.isnan(), torch.zeros_like(v), v)
    return v, bound * U * v.abs() + 2.0 ** -149 * (g.abs() if kind == "gelu" else 1)


# One tile, blocks of 64 and large tiles.
@pytest.mark.parametrize("kind", ["identity", "silu", "sigmoid", "gelu_tanh", "gelu", "relu"])
@pytest.mark.parametrize("live,n", [(1, 16), (16, 160), (48, 160), (320, 160), (1900, 4096)])
def test_activations_to_a_few_roundings(q8, kind, live, n):
    for seed in range(4 if live < 64 else 1):
        x = gate_values(live, seed)
        shifts = np.arange(n) % 8
        w, a, held = gates(q8, x, shifts)
        h = torch.full((live, n), 7.0, device="cuda")
        q8.q8_mx4_gated(*w, a, None, live, H=h, activation=kind)
        g = to_dev(held)[:, None] / to_dev(2.0 ** shifts[:8])
        want, tol = activation_and_bound(g, kind)
        err = (h[:, :n // 8 * 8].unflatten(1, (-1, 8)).double() - want[:, None]).abs()
        part = (err / tol.clamp(min=1e-60)[:, None]).amax(1).flatten()
        worst = torch.argmax(part).item()
        print(f"{kind}: {part[worst].item():.3f} of the bound at {g.flatten()[worst].item():.6g}")
        assert bool((err <= tol[:, None]).all()), (g.flatten()[worst].item(), want.flatten()[worst].item())


@pytest.mark.parametrize("live", [3, 40, 300])
def test_activations_of_numbers_that_are_not_finite(q8, live):
    """Infinities as sums that leave fp32's range: formulas as they stand, so x sigmoid(y) of -infinity is NaN."""
    n, inf = 48, np.inf
    codes, scales = np.zeros((2, n, 80), np.uint8), np.full((2, n, 5), 127, np.uint8)
    codes[0][:, 0], codes[1][:, 64] = 7, 2  # 6 and 1
    scales[0] = 140
    w = [q8.MX4Weights(n, 160) for _ in range(2)]
    for c, s, to in zip(codes, scales, w):
        q8.q8_mx4_pack_weights_q(to_dev(c), to_dev(s), to)
    x = np.zeros((live, 160), np.float32)
    x[:, 0], x[:, 128] = np.resize([3e37, -3e37, 0.0], live), 1.0
    a = q8.Acts(live, 160, "mx8")
    q8.q8_mx_quantize_acts(to_dev(x), live, a)
    want = {"silu": (inf, np.nan, 0), "sigmoid": (1, 0, 0.5), "gelu_tanh": (inf, np.nan, 0), "gelu": (inf, np.nan, 0),
            "relu": (inf, 0, 0), "identity": (inf, -inf, 0)}
    for kind, values in want.items():
        h = torch.full((live, n), 7.0, device="cuda")
        q8.q8_mx4_gated(*w, a, None, live, H=h, activation=kind)
        expect = np.resize(values, live)[:, None].repeat(n, 1)
        assert np.array_equal(h.cpu().numpy(), expect, equal_nan=True), kind


# ---------------------------------------------------------- every tile of a product

def whole_case(seed, form, n, k, slots):
    """Weights and activations whose products are whole multiples of one unit and whose sums stay below 2^24 of them
    (a product has at most 12 x 127 units): (weights, their values, activations, theirs), values in 64 bits."""
    assert k * 12 * 127 < 2 ** 24
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q8 = _q8()
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    w = q8.MX4Weights(n, k)
    w.data.fill_(0xEE)
    q8.q8_mx4_pack_weights_q(codes, torch.full((n, k // 32), 127, dtype=torch.uint8, device="cuda"), w)
    one = to_dev(ref.GRIDS["mx4"])
    one = torch.cat((one, -one))
    values = torch.stack((one[(codes & 15).int()], one[(codes >> 4).int()]), -1).flatten(-2)
    grid = to_dev(ref.GRIDS[form])
    x = grid[torch.randint(0, len(grid), (slots, k), generator=g, device="cuda")]
    x *= 1.0 - 2.0 * torch.randint(0, 2, (slots, k), generator=g, device="cuda")
    x[:, ::32] = grid[-1]  # the scale of every block is 1
    a = q8.Acts(slots, k, form)
    q8.q8_mx_quantize_acts(x.float(), slots, a)
    return w, values, a, x


def index_of(live, slots, seed):
    """Slots in any order, two of them outside the buffer: (on the GPU, which are inside, those)."""
    index = np.random.default_rng(seed).integers(0, slots, live)
    index[[1, live - 1]] = [-1, slots]
    good = torch.from_numpy((index >= 0) & (index < slots)).cuda()
    index = to_dev(index.astype(np.int32))
    return index, good, index[good].long()


@pytest.mark.parametrize("form", ["mx4", "mx6", "mx8"])
@pytest.mark.parametrize("shape,tile,several", shapes.PRODUCTS)
def test_products_in_every_tile(q8, form, shape, tile, several):
    n, k, live = shape
    slots = min(live, 700)
    w, values, a, x = whole_case(n + live, form, n, k, slots)
    index, good, inside = index_of(live, slots, n)
    y = torch.full((live + 1, n), 7.0, device="cuda")
    q8.q8_mx4_matmul(w, a, index, live, y)
    assert bool((y[live] == 7).all()) and bool(y[:live][~good].isnan().all())
    assert torch.equal(y[:live][good], (x @ values.T).float()[inside]), tile


@pytest.mark.parametrize("form", ["mx4", "mx6", "mx8"])
@pytest.mark.parametrize("shape,tile,several", shapes.GATED)
def test_gated_blocks_in_every_tile(q8, form, shape, tile, several):
    n, k, live = shape
    slots = min(live, 700)
    wg, vg, a, x = whole_case(n + live, form, n, k, slots)
    wu, vu, _, _ = whole_case(n + live + 1, form, n, k, 1)
    index, good, inside = index_of(live, slots, n)
    h = torch.full((live + 1, n), 7.0, device="cuda")
    q8.q8_mx4_gated(wg, wu, a, index, live, H=h, activation="identity")
    assert bool((h[live] == 7).all()) and bool(h[:live][~good].isnan().all())
    assert torch.equal(h[:live][good], ((x @ vg.T).float() * (x @ vu.T).float())[inside]), tile


@pytest.mark.parametrize("form,out", [("mx4", "mx8"), ("mx6", "mx4"), ("mx8", "mx8"), ("mx8", "mx6")])
@pytest.mark.parametrize("shape,tile,several", shapes.QUANTISED)
def test_quantised_rows_in_every_tile(q8, form, out, shape, tile, several):
    n, k, live = shape
    slots = min(live, 700)
    wg, vg, a, x = whole_case(n + live, form, n, k, slots)
    wu, vu, _, _ = whole_case(n + live + 1, form, n, k, 1)
    index, good, inside = index_of(live, slots, n)
    h, alone, both, want = torch.empty(live, n, device="cuda"), *(q8.Acts(live + 3, n, out) for _ in range(3))
    for b in (alone, both, want):
        b.data.fill_(0x41)
    q8.q8_mx4_gated(wg, wu, a, index, live, H=h, h_acts=both, activation="identity")
    q8.q8_mx4_gated(wg, wu, a, index, live, h_acts=alone, activation="identity")
    q8.q8_mx_quantize_acts(h, live, want)
    assert torch.equal(both.data, want.data) and torch.equal(alone.data, want.data), tile
    assert torch.equal(h[good], ((x @ vg.T).float() * (x @ vu.T).float())[inside]), tile


@pytest.mark.parametrize("n,k,live", [(45, 160, 5), (45, 160, 40), (4093, 96, 1900)])
def test_gated_rows_at_a_stride(q8, n, k, live):
    """h_stride beyond the row, at every alignment: the rows and nothing between them."""
    wg, vg, a, x = whole_case(n, "mx8", n, k, live)
    wu, vu, _, _ = whole_case(n + 1, "mx8", n, k, 1)
    want = (x @ vg.T).float() * (x @ vu.T).float()
    for stride, off in ((n, 0), (n + 16, 1), (n + 19, 0), (n + 3, 2)):
        h = torch.full((live * stride + 8,), 7.0, device="cuda")
        q8.q8_mx4_gated(wg, wu, a, None, live, H=h[off:], h_stride=stride, activation="identity")
        rows = h[off:off + live * stride].view(live, stride)
        assert torch.equal(rows[:, :n], want), (stride, off)
        assert bool((rows[:, n:] == 7).all()) and bool((h[:off] == 7).all()) and bool((h[off + live * stride:] == 7).all())


# ------------------------------------------------------ rows past the caches, wide rows

@pytest.mark.parametrize("form", ["mx4", "mx6", "mx8"])
def test_large_quantisation_is_that_of_its_parts(q8, form):
    """From 32 MB on fp32 rows go past the caches, read and written; aligned or not."""
    n, k = 1640, 5152
    big = torch.randn(n * (k + 3) + 4, device="cuda")
    big *= torch.exp(torch.randn(big.numel(), device="cuda"))
    for stride, off in ((k, 0), (k + 3, 1)):
        x = torch.as_strided(big, (n, k), (stride, 1), off).contiguous()
        a, out = q8.Acts(n, k, form), torch.empty(n * k + 1, device="cuda")
        q8.q8_mx_quantize_acts(big[off:], n, a, x_stride=stride)
        for at in (0, 1):  # 16-byte stores or single ones
            q8.q8_mx_read_acts(a, None, n, out[at:])
            got = out[at:at + n * k].view(n, k)
            for first in range(0, n, 410):
                part, small = q8.Acts(410, k, form), torch.empty(410, k, device="cuda")
                q8.q8_mx_quantize_acts(x[first:first + 410], 410, part)
                q8.q8_mx_read_acts(part, None, 410, small)
                assert torch.equal(got[first:first + 410], small)
        some = np.array([0, 1, 819, n - 1])
        assert np.array_equal(got[to_dev(some)].cpu().numpy().astype(np.float64), ref.hold(x[to_dev(some)].cpu().numpy(), form))


def test_large_weights_are_packed_as_their_parts(q8):
    n, k = 2064, 5120
    x = torch.randn(n, k, device="cuda") * 0.02
    w = q8.MX4Weights(n, k)
    q8.q8_mx4_pack_weights(x, w)
    codes, scales = (torch.empty(n, k // d, dtype=torch.uint8, device="cuda") for d in (2, 32))
    q8.q8_mx4_unpack_weights(w, codes, scales)
    for first in range(0, n, 688):
        part = q8.MX4Weights(688, k)
        q8.q8_mx4_pack_weights(x[first:first + 688], part)
        c, s = (torch.empty(688, k // d, dtype=torch.uint8, device="cuda") for d in (2, 32))
        q8.q8_mx4_unpack_weights(part, c, s)
        assert torch.equal(c, codes[first:first + 688]) and torch.equal(s, scales[first:first + 688])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("stride", [5120, 5123])
def test_large_norm_is_that_of_its_parts(q8, in_place, stride):
    """From 32 MB on stores go past the caches."""
    n, k = 1640, 5120
    x, r = (torch.randn(n, stride, device="cuda") for _ in range(2))
    g = torch.randn(n, k, device="cuda")
    post, pre = (q8.Norm(k, kind, torch.randn(k, device="cuda"), torch.randn(k, device="cuda")) for kind in ("rms", "layer"))
    args = dict(post=post, gate=g, scale=0.5, residual=r.clone(), pre=pre, x_stride=stride, residual_stride=stride,
                residual_out_stride=stride, y_stride=stride)
    out, y = (args["residual"], x.clone()) if in_place else (torch.full_like(r, 7.0) for _ in range(2))
    acts = q8.Acts(n, k, "mx8")
    q8.q8_norm_step(y if in_place else x, n, k, residual_out=out, Y=y, acts=acts, **args)
    held = torch.empty(n, k, device="cuda")
    q8.q8_mx_read_acts(acts, None, n, held)
    for first in range(0, n, 205):
        s = slice(first, first + 205)
        o, t = (torch.full((205, stride), 7.0, device="cuda") for _ in range(2))
        a, b = q8.Acts(205, k, "mx8"), torch.empty(205, k, device="cuda")
        q8.q8_norm_step(x[s], 205, k, residual_out=o, Y=t, acts=a, **dict(args, gate=g[s], residual=r[s]))
        q8.q8_mx_read_acts(a, None, 205, b)
        assert torch.equal(out[s, :k], o[:, :k]) and torch.equal(y[s, :k], t[:, :k]) and torch.equal(held[s], b)
    if not in_place:
        assert bool((out[:, k:] == 7).all()) and bool((y[:, k:] == 7).all())


@pytest.mark.parametrize("k", [8196, 8224, 12288, 12290, 16416, 20480, 20483, 24576, 24581, 28672, 28676, 32737])
def test_norms_of_wide_rows(q8, k):
    """Every number of units that a thread of 16 waves holds, at its ends; aligned or not."""
    base.check_norm(q8, 3, k, None, "rms", None, True)
    base.check_norm(q8, 2, k, "layer", "layer", "rows", True, per_row=True, offset=0.0)
    base.check_norm(q8, 2, k, "rms", "rms", "shared", True, in_place=True)
    if k % 32 == 0:
        base.test_norm_quantises_as_the_quantiser_does(q8, "mx8", 3, k, 5)
        base.test_norm_fills_q8_0_slots_as_their_quantiser_does(q8, 3, k, 16)


# ---------------------------------------------------------------- ends of the scales

@pytest.mark.parametrize("form", ["mx4", "mx6", "mx8"])
@pytest.mark.parametrize("live", [8, 40, 400])
def test_products_at_the_ends_of_the_scales(q8, form, live):
    """Single products of every code at the smallest and largest scale bytes: exact down to fp32's denormals, infinite
    beyond its largest number."""
    held = [(c, s) for s in (0, 1, 2, 3, 10, 60, 120, 200, 250, 252, 253, 254) for c in range(16)]
    codes, scales = np.zeros((len(held), 16), np.uint8), np.zeros((len(held), 1), np.uint8)
    codes[:, 0], scales[:, 0] = [c for c, _ in held], [s for _, s in held]
    w = q8.MX4Weights(len(held), 32)
    q8.q8_mx4_pack_weights_q(to_dev(codes), to_dev(scales), w)
    x = np.zeros((live, 32), np.float32)
    x[:, 0] = np.resize([1.5 * 2.0 ** e for e in (-120, -100, -22, -1, 0, 3, 60, 118)], live)
    a, y = q8.Acts(live, 32, form), torch.empty(live, len(held), device="cuda")
    q8.q8_mx_quantize_acts(to_dev(x), live, a)
    q8.q8_mx4_matmul(w, a, None, live, y)
    with np.errstate(over="ignore"):
        want = (ref.hold(x, form) @ ref.mx4_values(codes, scales).T).astype(np.float32)
    assert np.array_equal(y.cpu().numpy(), want) and np.isinf(want).any() and (np.abs(want[want != 0]) < 2.0 ** -126).any()
