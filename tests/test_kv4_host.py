"""The attention-side entry points (include/q8kv4.h) on the host: the header
and the binding agree, sizes follow the layout, frequencies follow their
formulas, and every invalid argument is refused before any HIP call."""

import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import kv4_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "q8kv4.h")
P = 0x10000  # an aligned address that no call may read


@pytest.fixture(scope="module")
def q8():
    import quantized_weight_streaming_q8_amd as q8
    return q8


def test_header_and_binding_agree(q8):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(q8_\w+)\s*\(", text, flags=re.M))
    assert names == set(q8._KV4_SIGNATURES)
    lib = ctypes.CDLL(q8.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    for n in ("Q8_KV4_MAX_HEAD_DIM", "Q8_KV4_MAX_PAGE", "Q8_KV4_MAX_TOKENS", "Q8_KV4_MAX_SEQS"):
        assert int(re.search(rf"#define {n} (\d+)", text).group(1)) == getattr(q8, n)
    for name, v in q8.Q8_ROTARY_SCALINGS.items():
        assert int(re.search(rf"Q8_ROTARY_{name.upper()} = (\d+)", text).group(1)) == v


def test_page_bytes(q8):
    # 17 bytes per 32 values
    for kv, d, t in ((8, 128, 64), (12, 64, 32), (1, 256, 4096), (3, 32, 32)):
        assert q8.q8_kv4_page_bytes(kv, d, t) == kv * t * 2 * (d // 2 + d // 32)
    assert q8.q8_kv4_page_bytes(5, 96, 96) == 5 * 96 * 2 * 3 * 17
    for bad in ((0, 128, 64), (1025, 128, 64), (8, 0, 64), (8, 48, 64), (8, 288, 64), (8, 128, 0),
                (8, 128, 48), (8, 128, 4128), (-1, 128, 64)):
        assert q8.q8_kv4_page_bytes(*bad) == 0, bad


@pytest.mark.parametrize("rot", [2, 6, 64, 128])
def test_frequencies(q8, rot):
    i = np.arange(rot // 2)
    base, f, ctx = 5e5, 4.0, 8192.0
    w = base ** (-2.0 * i / rot)
    turns = ctx * w / (2 * math.pi)

    def get(*a, **k):
        t, amp = q8.rotary_frequencies(rot, base, *a, **k)
        return t.numpy(), amp

    def near(got, want):
        assert np.allclose(got, want, rtol=2.0 ** -48, atol=0)

    got, amp = get()
    near(got, w)
    assert amp == 1.0
    near(get("linear", f)[0], w / f)
    near(get("ntk", f)[0], w if rot == 2 else (base * f ** (rot / (rot - 2))) ** (-2.0 * i / rot))
    if rot > 2:  # the slowest pair of "ntk" is exactly interpolated
        assert math.isclose(get("ntk", f)[0][-1], w[-1] / f, rel_tol=1e-12)
    g = np.clip((turns - 1) / 3, 0, 1)
    near(get("bands", f, ctx)[0], (1 - g) * w / f + g * w)
    g = np.clip((turns - 1) / 31, 0, 1)
    got, amp = get("yarn", f, ctx)
    near(got, (1 - g) * w / f + g * w)
    assert math.isclose(amp, 0.1 * math.log(f) + 1, rel_tol=1e-15)
    g = np.clip((turns - 2) / 6, 0, 1)
    near(get("yarn", f, ctx, low=2.0, high=8.0)[0], (1 - g) * w / f + g * w)


def test_frequencies_refuse(q8):
    nan, inf = float("nan"), float("inf")
    for a in ((0,), (3,), (1026,), (-2,), (64, 1.0), (64, nan), (64, 1e30), (64, 1e4, "linear", 0.5),
              (64, 1e4, "ntk", nan), (64, 1e4, "linear", inf), (64, 1e4, "bands", 2.0, 0.0),
              (64, 1e4, "yarn", 2.0, nan), (64, 1e4, "yarn", 2.0, 4096.0, 4.0, 4.0),
              (64, 1e4, "bands", 2.0, 4096.0, -1.0, 4.0), (64, 1e4, "bands", 2.0, 4096.0, 1.0, nan)):
        with pytest.raises(q8.Q8Error):
            q8.rotary_frequencies(*a)
    with pytest.raises(ValueError, match="scaling"):
        q8.rotary_frequencies(64, 1e4, "other")
    fn, buf = q8.library().q8_rotary_frequencies, torch.empty(32, dtype=torch.float64)
    amp = ctypes.c_double()
    ok = [64, 1e4, 0, 1.0, 0.0, 1.0, 4.0, buf.data_ptr(), ctypes.addressof(amp)]
    assert fn(*ok) == 0
    for i, v in ((2, 5), (2, -1), (7, None), (8, None)):
        a = list(ok)
        a[i] = v
        assert fn(*a) == q8.Q8_ERR_INVALID_ARG, (i, v)


def _plan(q8, **k):
    f = dict(inv_freq=P, amplitude=1.0, rot_dim=128, interleaved=0, **{})
    f.update(k)
    return q8._RotaryPlan(f["inv_freq"], f["amplitude"], f["rot_dim"], f["interleaved"])


def _cache(q8, **k):
    f = dict(pages=P, block_table=P, n_pages=100, n_slots=16, max_pages=10, page_tokens=64,
             n_kv_heads=8, head_dim=128)
    f.update(k)
    return q8._KV4Cache(*[f[n] for n, _ in q8._KV4Cache._fields_])


BAD_CACHES = [dict(pages=None), dict(pages=P + 128), dict(block_table=None), dict(block_table=P + 2),
              dict(n_pages=0), dict(n_pages=-1), dict(n_pages=1 << 40), dict(n_slots=0),
              dict(max_pages=0), dict(max_pages=1 << 25), dict(n_slots=1 << 20, max_pages=1 << 12),
              dict(page_tokens=0), dict(page_tokens=40), dict(page_tokens=8192), dict(n_kv_heads=0),
              dict(n_kv_heads=1025), dict(head_dim=0), dict(head_dim=80), dict(head_dim=512)]
BAD_PLANS = [dict(inv_freq=None), dict(inv_freq=P + 4), dict(rot_dim=0), dict(rot_dim=130),
             dict(rot_dim=63), dict(interleaved=2), dict(interleaved=-1), dict(amplitude=0.0),
             dict(amplitude=-1.0), dict(amplitude=float("nan")), dict(amplitude=float("inf"))]


def _refuses(fn, ok, changes):
    for i, v in changes:
        a = list(ok)
        a[i] = v
        assert fn(*a) == 1, (i, v)


def test_rotary_refuses(q8):
    fn = q8.library().q8_rotary
    ok = [P, 7168, P, 6144, 16, P, 48, 128, ctypes.addressof(_plan(q8)), None]
    keep = [_plan(q8)] + [_plan(q8, **b) for b in BAD_PLANS]
    ok[8] = ctypes.addressof(keep[0])
    _refuses(fn, ok, [(0, None), (0, P + 2), (2, None), (2, P + 1), (1, 6143), (3, 6143),
                      (1, 1 << 37), (3, 1 << 37), (4, 0), (4, -1), (4, (1 << 20) + 1), (5, None),
                      (5, P + 2), (6, 0), (6, 1 << 18), (7, 0), (7, 127), (7, 1026), (7, 64), (8, None)])
    _refuses(fn, ok, [(8, ctypes.addressof(p)) for p in keep[1:]])


def test_append_refuses(q8):
    fn = q8.library().q8_kv4_append
    c, plan = _cache(q8), _plan(q8)
    bad_caches = [_cache(q8, **b) for b in BAD_CACHES]
    bad_plans = [_plan(q8, **b) for b in BAD_PLANS]
    A = ctypes.addressof
    ok = [A(c), P, P, P, 7168, 16, P, P, A(plan), 40, P, 5120, None]
    _refuses(fn, ok, [(0, None), (1, None), (1, P + 2), (2, None), (2, P + 1), (3, None), (3, P + 2),
                      (4, 5119), (4, 1 << 37), (5, 0), (5, (1 << 20) + 1), (6, None), (6, P + 2),
                      (7, None), (7, P + 1), (9, -1), (9, 8193), (10, None), (10, P + 2),
                      (11, 5119), (11, 1 << 37)])
    _refuses(fn, ok, [(0, A(b)) for b in bad_caches])
    _refuses(fn, ok, [(8, A(b)) for b in bad_plans])
    ok[9] = 0  # keys and values alone: a row of at least one of them
    _refuses(fn, ok, [(4, 1023)])


def test_read_refuses(q8):
    fn = q8.library().q8_kv4_read
    c = _cache(q8)
    bad_caches = [_cache(q8, **b) for b in BAD_CACHES]
    A = ctypes.addressof
    ok = [A(c), P, P, 16, P, P, None]
    _refuses(fn, ok, [(0, None), (1, None), (1, P + 2), (2, None), (2, P + 2), (3, 0),
                      (3, (1 << 20) + 1), (4, P + 2), (5, P + 1)])
    _refuses(fn, ok, [(0, A(b)) for b in bad_caches])
    assert fn(A(c), P, P, 16, None, None, None) == 1


def test_attend_refuses(q8):
    lib = q8.library()
    c = _cache(q8)
    bad_caches = [_cache(q8, **b) for b in BAD_CACHES]
    A = ctypes.addressof
    need = lib.q8_kv4_attend_workspace_bytes(A(c), 16, 1, 40)
    assert need > 0
    ok = [A(c), P, 5120, 16, 1, 40, P, P, 0.1, 0, P, 5120, P, need, None]
    nan, inf = float("nan"), float("inf")
    _refuses(lib.q8_kv4_attend, ok,
             [(0, None), (1, None), (1, P + 2), (2, 5119), (2, 1 << 37), (3, 0), (3, 4097), (4, 0),
              (4, 65), (5, 0), (5, 41), (5, -8), (5, 8200), (6, None), (6, P + 2), (7, None),
              (7, P + 2), (8, 0.0), (8, -1.0), (8, nan), (8, inf), (8, 1.2e12), (9, -1), (10, None), (10, P + 2),
              (11, 5119), (11, 1 << 37), (12, None), (12, P + 128), (13, need - 1), (13, 0)])
    _refuses(lib.q8_kv4_attend, ok, [(0, A(b)) for b in bad_caches])
    ws = lib.q8_kv4_attend_workspace_bytes
    assert ws(None, 16, 1, 40) == 0
    for n, t, h in ((0, 1, 40), (16, 0, 40), (16, 65, 40), (16, 1, 39), (16, 1, 0), (4097, 1, 40)):
        assert ws(A(c), n, t, h) == 0, (n, t, h)
    # more than 2^18 row blocks
    many = _cache(q8, n_kv_heads=1024, n_pages=1)
    assert ws(A(many), 4096, 64, 8192) == 0


def test_attend_workspace_is_bounded(q8):
    """It grows with the context up to two records for each share that runs at
    once, whatever the context."""
    ws = q8.library().q8_kv4_attend_workspace_bytes
    A = ctypes.addressof
    sizes = [ws(A(_cache(q8, max_pages=n)), 16, 1, 40) for n in (1, 8, 9, 100, 1000, 100000)]
    assert sizes == sorted(sizes) and sizes[0] < sizes[-1] == sizes[-2]
    assert sizes[-1] <= (1 << 20) + 2 * 768 * 5 * 130 * 4


# --------------------------------------------------------- binding checks

def test_binding_refuses(q8):
    def t(n, dtype=torch.float32):
        return torch.zeros(n, dtype=dtype)

    i4 = t(4, torch.int32)
    table = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="inv_freq: expected float64"):
        q8.Rotary(t(32))
    with pytest.raises(ValueError, match="inv_freq: expected a device tensor"):
        q8.Rotary(t(32, torch.float64))
    with pytest.raises(ValueError, match="block_table: expected int32"):
        q8.KV4Cache(4, 64, 8, 128, table.long())
    with pytest.raises(ValueError, match="block_table: expected .n_slots."):
        q8.KV4Cache(4, 64, 8, 128, table.flatten())
    with pytest.raises(ValueError, match="block_table: expected a contiguous"):
        q8.KV4Cache(4, 64, 8, 128, table.t())
    with pytest.raises(ValueError, match="invalid cache shape"):
        q8.KV4Cache(4, 48, 8, 128, table)
    with pytest.raises(ValueError, match="pages: holds"):
        q8.KV4Cache(4, 64, 8, 128, table, pages=t(4 * q8.q8_kv4_page_bytes(8, 128, 64) - 1, torch.uint8))
    with pytest.raises(ValueError, match="pages: expected a device tensor"):
        q8.KV4Cache(4, 64, 8, 128, table)
    with pytest.raises(ValueError, match="X: holds"):
        q8.q8_rotary(t(4 * 256 - 1), t(4 * 256), 4, 256, i4, 2, 128, None, stream=0)
    with pytest.raises(ValueError, match="Y: holds"):
        q8.q8_rotary(t(4 * 256), t(4 * 256 - 1), 4, 256, i4, 2, 128, None, stream=0)
    with pytest.raises(ValueError, match="pos: expected int32"):
        q8.q8_rotary(t(4 * 256), t(4 * 256), 4, 256, i4.long(), 2, 128, None, stream=0)
    with pytest.raises(TypeError, match="rotary: expected a Rotary"):
        q8.q8_rotary(P, P, 4, 256, P, 2, 128, None, stream=0)

    class Shape:  # the fields a call's size checks read
        head_dim, n_kv_heads = 128, 2
    with pytest.raises(ValueError, match="row_stride: 511"):
        q8.q8_kv4_append(Shape, t(4 * 512), 4, 511, i4, i4)
    with pytest.raises(ValueError, match="QKV: holds"):
        q8.q8_kv4_append(Shape, t(4 * 512 - 1), 4, 512, i4, i4)
    with pytest.raises(ValueError, match="batch_index: holds"):
        q8.q8_kv4_append(Shape, t(5 * 512), 5, 512, i4, t(5, torch.int32))
    with pytest.raises(TypeError, match="cache: expected a KV4Cache"):
        q8.q8_kv4_append(Shape, P, 4, 512, P, P)
    with pytest.raises(ValueError, match="K: holds"):
        q8.q8_kv4_read(Shape, i4, i4, 4, t(4 * 256 - 1), t(4 * 256))
    with pytest.raises(ValueError, match="Q: expected float32"):
        q8.q8_kv4_attend(Shape, t(4 * 256, torch.float16), 4, 1, 2, i4, i4, t(4 * 256), None)
    with pytest.raises(ValueError, match="O: holds"):
        q8.q8_kv4_attend(Shape, t(4 * 256), 4, 1, 2, i4, i4, t(4 * 256 - 1), None)
    with pytest.raises(ValueError, match="O: expected a contiguous"):
        q8.q8_kv4_attend(Shape, t(4 * 256), 4, 1, 2, i4, i4, t(4 * 512).reshape(4, 512)[:, :256], None)


# ------------------------------------------------------ the oracle itself

def test_reference_blocks_closed_forms():
    """Blocks worked by hand: the scale rule on both sides of 7, ties to the
    even code, saturation, subnormal and largest blocks, NaN."""
    def block(*vals):
        x = np.zeros(32, dtype=np.float32)
        x[:len(vals)] = vals
        return ref.hold(x)[:len(vals)].tolist()
    assert block(6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.3) == [6, 4, 4, 2, 2, 1, 1, 0, -0.5]
    assert block(7, 5.01, -7) == [6, 6, -6]              # 7 keeps the scale and saturates
    assert block(7.001, 5, 2.9, 0.5) == [8, 4, 3, 0]     # above it the scale doubles
    assert block(0.0, -0.0) == [0, 0]
    assert block(2.0 ** -130, 2.0 ** -126) == [0, 2.0 ** -126]  # smallest scale 2^-125
    assert block(3.4e38) == [6 * 2.0 ** 125]
    assert np.isnan(ref.hold(np.r_[np.inf, np.ones(31)].astype(np.float32))).all()


def test_reference_attention_closed_forms():
    v = np.arange(12.0).reshape(3, 4)
    k = np.zeros((3, 4))
    q = np.ones((3, 4))
    O, _ = ref.attend(q, k, v, [0, 2, -1], 0.5)
    assert np.allclose(O, [v[0], v.mean(0), 0 * v[0]])
    O, _ = ref.attend(q, k, v, [0, 2, 2], 0.5, window=2)
    assert np.allclose(O[1], v[1:].mean(0))
    x = np.array([[[1.0, 0.0, 5.0, 7.0]]])
    assert np.allclose(ref.rotate(x, [1], [math.pi / 2]), [[[0, 1, 5, 7]]])
    assert np.allclose(ref.rotate(x, [2], [math.pi / 4, math.pi], True), [[[0, 1, 5, 7]]])
    assert np.allclose(ref.rotate(x, [2], [math.pi / 4, math.pi]), [[[-5, 0, 1, 7]]])
