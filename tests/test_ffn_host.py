"""The feed-forward side's entry points (include/q8ffn.h) on the host: the
header and the binding agree, sizes follow the layout, and every invalid argument
is refused before any HIP call; the 64-bit definitions in closed forms."""

import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import ffn_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "q8ffn.h")
P = 0x10000  # an aligned address that no call may read
INVALID = 1


@pytest.fixture(scope="module")
def q8():
    import quantized_weight_streaming_q8_amd as q8
    return q8


def test_header_and_binding_agree(q8):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(q8_\w+)\s*\(", text, flags=re.M))
    assert names == set(q8._FFN_SIGNATURES)
    lib = ctypes.CDLL(q8.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    for n in ("Q8_FFN_MAX_ROWS", "Q8_NORM_MAX_WIDTH"):
        a, b = re.search(rf"#define {n} \((\d+) << (\d+)\)", text).groups()
        assert int(a) << int(b) == getattr(q8, n)
    for prefix, table in (("Q8_ACTS_", q8.Q8_ACTS_FORMATS), ("Q8_ACT_", q8.Q8_ACTIVATIONS),
                          ("Q8_NORM_", q8.Q8_NORM_KINDS)):
        for name, v in table.items():
            assert int(re.search(rf"\b{prefix}{name.upper()} = (\d+)", text).group(1)) == v


def test_buffer_sizes(q8):
    # 16 rows x 128 columns: 1024 bytes of 4-bit codes; scales for 4 such chunks: 256
    assert q8.q8_mx4_weight_bytes(16, 128) == 1024 + 256
    assert q8.q8_mx4_weight_bytes(17, 544) == 2 * (5 * 1024 + 2 * 256)
    assert q8.q8_mx4_weight_bytes(7168, 5120) == 7168 * 5120 * 17 // 32
    # up to 64 slots tiles of 16 rows, above that rows of whole super-chunks of 512 values,
    # codes rounded up to 256 bytes; a scale byte for each 32 values (two for MX8,
    # which holds 12 bits a value)
    for n, k in ((1, 32), (40, 672), (64, 5120), (65, 160), (4099, 5120)):
        wide = -(-k // 512) * 512
        for form, bits, pieces in (("mx4", 4, 1), ("mx6", 6, 1), ("mx8", 12, 2)):
            if n <= 64:
                rows, codes = -(-n // 16) * 16, -(-n // 16) * 16 * -(-k // 128) * 128 * bits // 8
            else:
                rows, codes = n, -(-n * wide * bits // 8 // 256) * 256
            assert q8.q8_acts_bytes(n, k, form) == codes + rows * wide // 32 * pieces, (n, k, form)
    for n in (16, 32, 48, 64):
        assert q8.q8_acts_bytes(n, 5120, "q8_0") == q8.q8_act_buffer_bytes_n(5120, n)


def test_invalid_shapes_have_no_size(q8):
    for n, k in ((0, 128), (-1, 128), (16, 0), (16, -32), (16, 48), (16, (1 << 20) + 32), (1 << 30, 128)):
        assert q8.q8_mx4_weight_bytes(n, k) == 0, (n, k)
    assert q8.q8_mx4_weight_bytes(1 << 27, 128) > 0 and q8.q8_mx4_weight_bytes((1 << 27) + 1, 128) == 0
    for n, k in ((0, 128), ((1 << 20) + 1, 128), (16, 100), (1 << 20, 4096)):
        for f in ("mx4", "mx6", "mx8"):
            assert q8.q8_acts_bytes(n, k, f) == 0, (n, k)
    assert q8.q8_acts_bytes(1 << 20, 2048, "mx8") > 0 and q8.q8_acts_bytes(1 << 20, 2049, "mx8") == 0
    assert q8.q8_acts_bytes(17, 128, "q8_0") == 0
    fn = q8.library().q8_acts_bytes
    assert fn(16, 128, 4) == 0 and fn(16, 128, -1) == 0


A = ctypes.addressof


def weights(q8, data=P, N=256, K=512):
    return q8._MX4Weights(data, N, K)


def acts(q8, data=2 * P, K=512, n_slots=64, form="mx8"):
    return q8._Acts(data, K, n_slots, q8.Q8_ACTS_FORMATS[form] if isinstance(form, str) else form)


BAD_WEIGHTS = (dict(data=None), dict(data=P + 128), dict(N=0), dict(N=-5), dict(K=0), dict(K=80), dict(N=1 << 40))
BAD_ACTS = (dict(data=None), dict(data=P + 64), dict(K=0), dict(K=100), dict(n_slots=0), dict(n_slots=(1 << 20) + 1),
            dict(form=4), dict(form=-1))


def refuses(fn, ok, changes):
    for i, v in changes:
        a = list(ok)
        a[i] = v
        assert fn(*a) == INVALID, (i, v)


def test_quantisation_refuses(q8):
    lib = q8.library()
    keep = [weights(q8, **b) for b in BAD_WEIGHTS]
    w = weights(q8)
    refuses(lib.q8_mx4_pack_weights, [P, A(w), None], [(0, None), (0, P + 4), (1, None)] + [(1, A(b)) for b in keep])
    for fn, ok, c, s in ((lib.q8_mx4_pack_weights_q, [P, P, A(w), None], 0, 1),
                         (lib.q8_mx4_unpack_weights, [A(w), P, P, None], 1, 2)):
        at = 3 - c - s
        refuses(fn, ok, [(c, None), (c, P + 8), (s, None), (at, None)] + [(at, A(b)) for b in keep])
    x = acts(q8)
    bad = [acts(q8, **b) for b in BAD_ACTS] + [acts(q8, form="q8_0")]
    refuses(lib.q8_mx_quantize_acts, [P, 512, 64, A(x), None],
            [(0, None), (0, P + 2), (1, 511), (1, 1 << 36), (2, 0), (2, 65), (3, None)] + [(3, A(b)) for b in bad])
    refuses(lib.q8_mx_read_acts, [A(x), P, 64, P, None],
            [(0, None), (1, P + 2), (2, 0), (2, (1 << 20) + 1), (3, None), (3, P + 1)] + [(0, A(b)) for b in bad])
    refuses(lib.q8_mx_read_acts, [A(x), None, 64, P, None], [(2, 65)])
    long = acts(q8, K=1 << 14, n_slots=64)
    refuses(lib.q8_mx_read_acts, [A(long), P, 64, P, None], [(2, 1 << 20)])


def test_product_refuses(q8):
    lib = q8.library()
    w, x = weights(q8), acts(q8)
    ok = [A(w), A(x), P, 64, P, 256, None]
    keep = [weights(q8, **b) for b in BAD_WEIGHTS] + [weights(q8, K=544)]
    bad = [acts(q8, **b) for b in BAD_ACTS] + [acts(q8, form="q8_0"), acts(q8, K=480)]
    changes = [(0, None), (1, None), (2, P + 2), (3, 0), (3, -1), (3, (1 << 20) + 1), (4, None), (4, P + 2), (5, 255),
               (5, 1 << 35)] + [(0, A(b)) for b in keep] + [(1, A(b)) for b in bad]
    refuses(lib.q8_mx4_matmul, ok, changes)
    refuses(lib.q8_mx4_matmul, [A(w), A(x), None, 64, P, 256, None], [(3, 65)])
    big = weights(q8, N=1 << 24, K=32)
    small = acts(q8, K=32)
    refuses(lib.q8_mx4_matmul, [A(big), A(small), P, 64, P, 1 << 24, None], [(3, 4097)])


def test_gated_refuses(q8):
    lib = q8.library()
    w, u, x, h = weights(q8), weights(q8, data=4 * P), acts(q8), acts(q8, data=3 * P, K=256)
    ok = [A(w), A(u), A(x), P, 64, 0, P, 256, A(h), None]
    keep = [weights(q8, **b) for b in BAD_WEIGHTS] + [weights(q8, K=544), weights(q8, N=255)]
    bad = [acts(q8, **b) for b in BAD_ACTS] + [acts(q8, form="q8_0"), acts(q8, K=480)]
    out = [acts(q8, **dict(dict(data=3 * P, K=256), **b)) for b in BAD_ACTS] + [
        acts(q8, data=3 * P, K=256, form="q8_0"), acts(q8, data=3 * P, K=288), acts(q8, data=3 * P, K=256, n_slots=63),
        acts(q8, data=2 * P, K=256)]  # the input's own buffer
    changes = [(0, None), (1, None), (2, None), (3, P + 2), (4, 0), (4, (1 << 20) + 1), (5, -1), (5, 6), (6, P + 2), (7, 255)]
    changes += [(i, A(b)) for i in (0, 1) for b in keep] + [(2, A(b)) for b in bad] + [(8, A(b)) for b in out]
    refuses(lib.q8_mx4_gated, ok, changes)
    refuses(lib.q8_mx4_gated, [A(w), A(u), A(x), P, 64, 0, None, 256, A(h), None], [(8, None)])
    odd = weights(q8, N=250)
    held = acts(q8, data=3 * P, K=250)
    refuses(lib.q8_mx4_gated, [A(odd), A(odd), A(x), P, 64, 0, P, 250, None, None], [(8, A(held))])


def test_norm_refuses(q8):
    lib = q8.library()
    nan, inf = math.nan, math.inf

    def norm(weight=P, bias=P, ws=0, bs=0, eps=1e-6, offset=0.0, kind=0):
        return q8._Norm(weight, bias, ws, bs, eps, offset, kind)

    n, a = norm(), acts(q8)
    # X, x_stride, post, gate, gate_stride, scale, R, r_stride, R_out, stride, pre, Y, y_stride, acts, n_rows, K
    ok = [P, 512, A(n), P, 0, 1.0, P, 512, 3 * P, 512, A(n), 5 * P, 512, A(a), 16, 512, None]
    bad = [norm(weight=P + 2), norm(bias=P + 1), norm(ws=511), norm(bs=1), norm(ws=-512), norm(bs=1 << 38), norm(eps=-1e-6),
           norm(eps=nan), norm(eps=inf), norm(offset=inf), norm(offset=nan), norm(kind=2), norm(kind=-1)]
    bufs = [acts(q8, **b) for b in BAD_ACTS] + [acts(q8, K=480), acts(q8, n_slots=15), acts(q8, form="q8_0", n_slots=17)]
    changes = [(0, None), (0, P + 2), (1, 511), (1, 1 << 38), (3, P + 2), (4, 511), (4, -1), (5, nan), (5, inf), (6, P + 2),
               (7, 511), (8, P + 2), (9, 511), (11, P + 2), (12, 511), (14, 0), (14, -3), (14, (1 << 20) + 1), (15, 0),
               (15, (1 << 15) + 1), (15, 480)]
    changes += [(i, A(b)) for i in (2, 10) for b in bad] + [(13, A(b)) for b in bufs]
    changes += [(11, 3 * P)]  # both outputs the same
    refuses(lib.q8_norm_step, ok, changes)
    # in place with another stride; nothing to write
    refuses(lib.q8_norm_step, [P, 512, None, None, 0, 1.0, None, 0, P, 512, None, None, 0, None, 16, 512, None],
            [(9, 513), (8, None)])
    refuses(lib.q8_norm_step, [P, 512, None, None, 0, 1.0, 3 * P, 512, None, 0, None, 3 * P, 512, None, 16, 512, None],
            [(12, 600)])


def test_norm_in_place_refuses_another_stride_where_both_inputs_are_one(q8):
    """X and R at one address with strides of their own: an output there has the
    stride of both or is refused, since its rows would overlap the other's."""
    lib = q8.library()
    for out, stride in ((8, 9), (11, 12)):
        for x_stride, r_stride, o_stride in ((512, 600, 512), (512, 600, 600), (600, 512, 512), (600, 512, 600), (512, 512, 600)):
            a = [P, x_stride, None, None, 0, 1.0, P, r_stride, None, 0, None, None, 0, None, 16, 512, None]
            a[out], a[stride] = P, o_stride
            assert lib.q8_norm_step(*a) == INVALID, (out, x_stride, r_stride, o_stride)


# --------------------------------------------------------- binding checks

def test_binding_refuses(q8):
    def t(*n, dtype=torch.float32):
        return torch.zeros(*n, dtype=dtype)

    with pytest.raises(ValueError, match="invalid shape"):
        q8.MX4Weights(16, 100)
    with pytest.raises(ValueError, match="data: holds"):
        q8.MX4Weights(16, 128, data=t(1279, dtype=torch.uint8))
    with pytest.raises(ValueError, match="data: expected a device tensor"):
        q8.MX4Weights(16, 128, data=t(1280, dtype=torch.uint8))
    with pytest.raises(ValueError, match="format: expected one of"):
        q8.Acts(16, 128, "mx5")
    with pytest.raises(ValueError, match="invalid buffer shape"):
        q8.Acts(17, 128, "q8_0")
    with pytest.raises(ValueError, match="data: holds"):
        q8.Acts(16, 128, "mx6", data=t(1536, dtype=torch.uint8))
    with pytest.raises(ValueError, match="kind: expected one of"):
        q8.Norm(64, "batch")
    with pytest.raises(ValueError, match="weight: expected a tensor of"):
        q8.Norm(64, weight=t(65))
    with pytest.raises(ValueError, match="bias: expected a tensor of"):
        q8.Norm(64, bias=t(2, 3, 64))
    with pytest.raises(ValueError, match="weight: expected float32"):
        q8.Norm(64, weight=t(64, dtype=torch.float16))
    with pytest.raises(ValueError, match="weight: expected a device tensor"):
        q8.Norm(64, weight=t(64))

    class W:  # the fields a call's size checks read
        N, K = 64, 128

    class X:
        K, n_slots = 128, 16
    i4 = t(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="W: holds"):
        q8.q8_mx4_pack_weights(t(64 * 128 - 1), W)
    with pytest.raises(ValueError, match="codes: expected uint8"):
        q8.q8_mx4_pack_weights_q(t(64, 64, dtype=torch.int8), t(64, 4, dtype=torch.uint8), W)
    with pytest.raises(ValueError, match="scales: holds"):
        q8.q8_mx4_unpack_weights(W, t(64, 64, dtype=torch.uint8), t(255, dtype=torch.uint8))
    with pytest.raises(ValueError, match="X: holds"):
        q8.q8_mx_quantize_acts(t(4 * 128 - 1), 4, X)
    with pytest.raises(ValueError, match="X: expected a contiguous"):
        q8.q8_mx_quantize_acts(t(4, 256)[:, :128], 4, X)
    with pytest.raises(TypeError, match="acts: expected a Acts"):
        q8.q8_mx_quantize_acts(P, 4, X)
    with pytest.raises(ValueError, match="batch_index: expected int32"):
        q8.q8_mx_read_acts(X, i4.long(), 4, t(4, 128))
    with pytest.raises(ValueError, match="Y: holds"):
        q8.q8_mx4_matmul(W, X, i4, 4, t(255))
    with pytest.raises(TypeError, match="weights: expected a MX4Weights"):
        q8.q8_mx4_matmul(W, X, P, 4, P)
    with pytest.raises(ValueError, match="activation: expected one of"):
        q8.q8_mx4_gated(W, W, X, i4, 4, H=t(256), activation="tanh")
    with pytest.raises(ValueError, match="H: holds"):
        q8.q8_mx4_gated(W, W, X, i4, 4, H=t(255))
    with pytest.raises(ValueError, match="residual: holds"):
        q8.q8_norm_step(t(4 * 128), 4, 128, residual=t(4 * 128 - 1), Y=t(4 * 128))
    with pytest.raises(ValueError, match="gate: holds"):
        q8.q8_norm_step(t(4 * 128), 4, 128, gate=t(2, 128), Y=t(4 * 128))
    with pytest.raises(ValueError, match="pre: a norm of 64 values"):
        q8.q8_norm_step(P, 4, 128, pre=q8.Norm(64), Y=P)
    with pytest.raises(TypeError, match="post: expected a Norm"):
        q8.q8_norm_step(P, 4, 128, post="rms", Y=P)


# ------------------------------------------------------ the oracle itself

def test_reference_blocks_closed_forms():
    """Blocks worked by hand: the scale rule on both sides of its border, ties to
    the even code, saturation, smallest and largest scales, NaN."""
    def block(form, *vals):
        x = np.zeros(32, dtype=np.float32)
        x[:len(vals)] = vals
        return ref.hold(x, form)[:len(vals)].tolist()
    assert block("mx4", 6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.3) == [6, 4, 4, 2, 2, 1, 1, 0, -0.5]
    assert block("mx4", 7, 5.01, -7) == [6, 6, -6]
    assert block("mx4", 7.001, 5, 2.9, 0.5) == [8, 4, 3, 0]
    assert block("mx6", 7.5, 7.75, 7.25, 5.25, 3.125, 1.0625, 0.1875, 0.0625, -0.07) == [7.5, 7.5, 7, 5, 3, 1, 0.25, 0, -0.125]
    assert block("mx6", 7.76, 1.1, 0.125) == [8, 1, 0]
    assert block("mx8", 127, 126.5, 125.5, 0.5, 1.5, -3.4) == [127, 126, 126, 0, 2, -3]
    assert block("mx8", 127.5, -127.5, 1) == [127, -127, 1]
    assert block("mx8", 127.6, 1, 3, 5) == [128, 0, 4, 4]
    assert block("mx8", 0.0, -0.0) == [0, 0]
    # the smallest scale is 2^-120: a quarter of it is a tie between 0 and 0.5, or two steps
    for form, top, low in (("mx4", 6, 0), ("mx6", 7.5, 2.0 ** -122)):
        assert block(form, 2.0 ** -122, 2.0 ** -149) == [low, 0]
        assert block(form, 3.4028234663852886e38) == [top * 2.0 ** 125]
        assert np.isnan(ref.hold(np.r_[np.inf, np.ones(31)].astype(np.float32), form)).all()
    assert block("mx8", 3.4028234663852886e38)[0] == 127 / 64 * 2.0 ** 125


def test_reference_products_and_norms_closed_forms():
    c = np.array([[0x21, 0xF9] + [0] * 14], np.uint8)
    assert ref.mx4_values(c, np.array([[128]], np.uint8))[0, :4].tolist() == [1, 2, -1, -12]
    y, tol = ref.product(np.array([[1.0, 2, 3]]), np.array([[1.0, 0, -1], [2, 2, 2]]), 1)
    assert y.tolist() == [[-2], [12]] and (tol > 0).all()
    for kind, at in (("silu", 1 / (1 + math.exp(-1))), ("gelu", 0.8413447460685429), ("gelu_tanh", 0.8411919906082768),
                     ("relu", 1), ("sigmoid", 1 / (1 + math.exp(-1))), ("identity", 1)):
        assert abs(ref.activation(np.array([1.0]), kind)[0] - at) < 1e-12, kind
    x = np.array([[3.0, 4.0]])
    assert np.allclose(ref.norm(x, "rms", np.array([1.0, 2.0]), None, 0.0, 0.0), [[3 / 12.5 ** .5, 8 / 12.5 ** .5]])
    assert np.allclose(ref.norm(x, "layer", None, np.array([10.0, 20.0]), 0.0, 1.0), [[9, 21]])


def test_imports_where_torch_has_no_device():
    """A torch built without one lacks the names of the current device and stream:
    sizes and host checks need neither."""
    import subprocess
    import sys
    code = ("import torch\n"
            "del torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream\n"
            "import quantized_weight_streaming_q8_amd as q8\n"
            "assert q8.q8_mx4_weight_bytes(16, 128) == 1280 and q8.q8_act_buffer_bytes(128) > 0\n"
            "try:\n"
            "    q8.q8_norm_step(65536, 0, 128, Y=65536, stream=0)\n"
            "except q8.Q8Error as e:\n"
            "    assert e.status == q8.Q8_ERR_INVALID_ARG\n"
            "else:\n"
            "    raise AssertionError('no rows accepted')\n")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, timeout=300)


def test_counts_beyond_32_bits_are_refused(q8):
    """ctypes keeps the low 32 bits of a larger number, which would be a count of rows again."""
    for n in ((1 << 32) + 4, -(1 << 32) + 4, 1 << 31, (1 << 20) + 1, 0):
        for form in ("mx4", "mx6", "mx8", "q8_0"):
            assert q8.q8_acts_bytes(n * 4, 128, form) == 0
        with pytest.raises(ValueError, match="invalid buffer shape"):
            q8.Acts(n * 4, 128, "mx8")
        for call in (lambda: q8.q8_norm_step(P, n, 128, Y=P, stream=0), lambda: q8.q8_mx_quantize_acts(P, n, X, stream=0),
                     lambda: q8.q8_mx_read_acts(X, None, n, P, stream=0), lambda: q8.q8_mx4_matmul(W, X, P, n, P, stream=0),
                     lambda: q8.q8_mx4_gated(W, W, X, P, n, H=P, stream=0)):
            with pytest.raises(q8.Q8Error) as e:
                call()
            assert e.value.status == INVALID


class W:  # the fields a call's size checks read
    N, K = 64, 128


class X:
    K, n_slots = 128, 16
