"""Python binding of libq8narrow.so, the narrow-batch q8_0 decode matmul for
MI355X (gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in ``include/q8narrow.h``; torch supplies
device memory and the current stream.  The functions keep the C names and
raise ``Q8Error`` on a non-OK status.  There is no fallback: if the library
is not built, importing this package raises.

With the environment variable Q8_LIBRARY=timeline set before the first
import, the package loads the timeline build, libq8narrow_timeline.so, instead
(same entry points and results, plus ``q8_timeline_set`` of
``include/q8timeline.h``: per-wave real-time counter records for profiling).

The attention side (``include/q8kv4.h``: rotary positions, the paged 4-bit
cache, its append, read-back and attention) takes two handles that a program
makes once: ``Rotary`` (a plan, from ``rotary_plan``) and ``KV4Cache``.  Their
tensors are checked when they are made, so that a step's calls check only
what changes from step to step.

The feed-forward side (``include/q8ffn.h``: norms around a block, microscaled
blocks, products with 4-bit weights, the gated block) has handles of the same
kind: ``MX4Weights``, ``Acts`` (a buffer of quantised activation rows) and
``Norm``.
"""

from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

_VARIANT = os.environ.get("Q8_LIBRARY", "")
if _VARIANT not in ("", "timeline"):
    raise ImportError(f"Q8_LIBRARY={_VARIANT!r}: only 'timeline' (or unset) is known")
TIMELINE = _VARIANT == "timeline"
LIB_PATH = _build.TIMELINE_LIB_PATH if TIMELINE else _build.LIB_PATH

Q8_BLOCK = 32
Q8_MAX_SLOTS = 16
Q8_MAX_COLUMNS = 64

Q8_OK = 0
Q8_ERR_INVALID_ARG = 1
Q8_ERR_UNSUPPORTED = 2
Q8_ERR_HIP = 3
Q8_ERR_TOO_LARGE = 4
Q8_NOALLOC_SCRATCH_BYTES = 8 << 20
Q8_FUSED_TIMEOUTS_OFFSET = 256

Q8_PATH_AUTO = 0
Q8_PATH_MFMA = 1
Q8_PATH_DOT4 = 2

# Every symbol the header declares, with its ctypes signature.
_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_SIGNATURES = {
    "q8_packed_weight_bytes": ([_i64, _i64], ctypes.c_size_t),
    "q8_act_buffer_bytes": ([_i64], ctypes.c_size_t),
    "q8_pack_weights": ([_vp, _i64, _i64, _vp, _vp], _i32),
    "q8_pack_weights_q": ([_vp, _vp, _i64, _i64, _vp, _vp], _i32),
    "q8_unpack_weights": ([_vp, _i64, _i64, _vp, _vp, _vp], _i32),
    "q8_quantize_acts": ([_vp, _i32, _i64, _vp, _vp], _i32),
    "q8_matmul_narrow": ([_vp, _vp, _vp, _i32, _i64, _i64, _vp, _vp], _i32),
    "q8_matmul_narrow_path": ([_vp, _vp, _vp, _i32, _i64, _i64, _vp, _vp, _i32], _i32),
    "q8_matmul_workspace_bytes": ([_i64, _i64], ctypes.c_size_t),
    "q8_matmul_launch_info": ([_i64, _i64, _i32, _i32, _vp], _i32),
    "q8_matmul_narrow_ws": ([_vp, _vp, _vp, _i32, _i64, _i64, _vp, _vp, ctypes.c_size_t, _vp], _i32),
    "q8_matmul_narrow_noalloc": ([_vp, _vp, _vp, _i32, _i64, _i64, _vp, _vp], _i32),
    "q8_matmul_fused_workspace_bytes": ([_i64, _i64], ctypes.c_size_t),
    "q8_matmul_narrow_fused": ([_vp, _vp, _i32, _vp, _vp, _i32, _i64, _i64, _vp, _vp,
                                ctypes.c_size_t, _vp], _i32),
    "q8_matmul_narrow_fused_bounded": ([_vp, _vp, _i32, _vp, _vp, _i32, _i64, _i64, _vp, _vp,
                                        ctypes.c_size_t, _i32, _i32, _vp], _i32),
    "q8_act_buffer_bytes_n": ([_i64, _i32], ctypes.c_size_t),
    "q8_quantize_acts_n": ([_vp, _i32, _i64, _vp, _i32, _vp], _i32),
    "q8_matmul_multi": ([_vp, _vp, _i32, _vp, _i32, _i64, _i64, _vp, _vp], _i32),
    "q8_rope_multi": ([_vp, _i32, _i64, _vp, _i32, _i32, ctypes.c_double, _vp], _i32),
    "q8_stream_read": ([_vp, ctypes.c_size_t, _vp, _vp], _i32),
    "q8_device_supported": ([], _i32),
    "q8_status_str": ([_i32], ctypes.c_char_p),
}


class _RotaryPlan(ctypes.Structure):
    _fields_ = [("inv_freq", _vp), ("amplitude", ctypes.c_double), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32)]


class _KV4Cache(ctypes.Structure):
    _fields_ = [("pages", _vp), ("block_table", _vp), ("n_pages", _i64),
                ("n_slots", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


# include/q8kv4.h.
_f64, _f32, _size = ctypes.c_double, ctypes.c_float, ctypes.c_size_t
_KV4_SIGNATURES = {
    "q8_rotary_frequencies": ([_i32, _f64, _i32, _f64, _f64, _f64, _f64, _vp, _vp], _i32),
    "q8_rotary": ([_vp, _i64, _vp, _i64, _i32, _vp, _i32, _i32, _vp, _vp], _i32),
    "q8_kv4_page_bytes": ([_i32, _i32, _i32], _size),
    "q8_kv4_append": ([_vp, _vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _i32, _vp, _i64, _vp], _i32),
    "q8_kv4_read": ([_vp, _vp, _vp, _i32, _vp, _vp, _vp], _i32),
    "q8_kv4_attend_workspace_bytes": ([_vp, _i32, _i32, _i32], _size),
    "q8_kv4_attend": ([_vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _f32, _i32, _vp, _i64, _vp,
                       _size, _vp], _i32),
}


class _MX4Weights(ctypes.Structure):
    _fields_ = [("data", _vp), ("N", _i64), ("K", _i64)]


class _Acts(ctypes.Structure):
    _fields_ = [("data", _vp), ("K", _i64), ("n_slots", ctypes.c_int32), ("format", ctypes.c_int32)]


class _Norm(ctypes.Structure):
    _fields_ = [("weight", _vp), ("bias", _vp), ("weight_stride", _i64), ("bias_stride", _i64),
                ("eps", ctypes.c_float), ("offset", ctypes.c_float), ("kind", ctypes.c_int32)]


# include/q8ffn.h.
_FFN_SIGNATURES = {
    "q8_acts_bytes": ([ctypes.c_int32, _i64, ctypes.c_int32], _size),
    "q8_mx4_weight_bytes": ([_i64, _i64], _size),
    "q8_mx4_pack_weights": ([_vp, _vp, _vp], _i32),
    "q8_mx4_pack_weights_q": ([_vp, _vp, _vp, _vp], _i32),
    "q8_mx4_unpack_weights": ([_vp, _vp, _vp, _vp], _i32),
    "q8_mx_quantize_acts": ([_vp, _i64, _i32, _vp, _vp], _i32),
    "q8_mx_read_acts": ([_vp, _vp, _i32, _vp, _vp], _i32),
    "q8_mx4_matmul": ([_vp, _vp, _vp, _i32, _vp, _i64, _vp], _i32),
    "q8_mx4_gated": ([_vp, _vp, _vp, _vp, _i32, _i32, _vp, _i64, _vp, _vp], _i32),
    "q8_norm_step": ([_vp, _i64, _vp, _vp, _i64, _f32, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i32, _i64, _vp],
                     _i32),
}
# The timeline build's own symbol (include/q8timeline.h).
_TIMELINE_SIGNATURES = {
    "q8_timeline_set": ([_vp, _i64], _i32),
}
Q8_STAMP_WORDS = 8


class Q8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)}")


def _load_library():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
            "or `python quantized_weight_streaming_q8_amd/build.py` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    sigs = dict(_SIGNATURES, **_KV4_SIGNATURES, **_FFN_SIGNATURES,
                **(_TIMELINE_SIGNATURES if TIMELINE else {}))
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load_library()


def library() -> ctypes.CDLL:
    return _lib


# ------------------------------------------------------------------ helpers

_F32 = (torch.float32,)
_I32 = (torch.int32,)
_I8 = (torch.int8,)
_H16 = (torch.int16, torch.float16)  # binary16 bits
_ANY = None


def _arg(x, name: str, dtypes=_ANY, need_bytes: int = 0):
    """First check of argument `name` for the C ABI: a tensor's dtype (when
    the argument has one), that it holds at least `need_bytes` bytes (0: no
    size check, e.g. when the shape itself is invalid and the library will
    reject the call) and that it is contiguous.  An int is a raw device
    address and None is NULL; both pass unchecked (the library's own host
    checks still apply).  Returns (name, x) for _dev."""
    if x is None or isinstance(x, int):
        return name, x
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: cannot pass {type(x).__name__} as a device pointer")
    if dtypes is not None and x.dtype not in dtypes:
        want = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name}: expected {want}, got {str(x.dtype).replace('torch.', '')}")
    have = x.numel() * x.element_size()
    if have < need_bytes:
        raise ValueError(f"{name}: holds {have} bytes, the call needs at least {need_bytes}")
    if not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return name, x


def _dev(*checked):
    """Second check, once every argument has passed _arg: each tensor lives
    on the current device.  Returns the device addresses, in order."""
    out = []
    for name, x in checked:
        if isinstance(x, torch.Tensor):
            if not x.is_cuda:
                raise ValueError(f"{name}: expected a device tensor, got one on {x.device}")
            if x.device.index != torch.cuda.current_device():
                raise ValueError(f"{name}: on {x.device}, but the current device is "
                                 f"cuda:{torch.cuda.current_device()}")
            x = x.data_ptr()
        out.append(x)
    return out


def _ptr(x) -> int | None:
    """Device address of a tensor (or an int address, or None for NULL)."""
    return _dev(_arg(x, "argument"))[0]


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(rc: int, where: str) -> None:
    if rc != Q8_OK:
        raise Q8Error(rc, where)


def status_str(status: int) -> str:
    return _lib.q8_status_str(int(status)).decode()


def _n(count: int, size: int) -> int:
    """Bytes of `count` elements of `size` bytes (0 for a non-positive count,
    which the library rejects itself)."""
    return count * size if count > 0 else 0


# ----------------------------------------------------------------- the ABI

def q8_packed_weight_bytes(N: int, K: int) -> int:
    return int(_lib.q8_packed_weight_bytes(N, K))


def q8_act_buffer_bytes(K: int) -> int:
    return int(_lib.q8_act_buffer_bytes(K))


def q8_pack_weights(W, N: int, K: int, Wq, stream=None) -> None:
    w, wq = _dev(_arg(W, "W", _F32, _n(N * K, 4)),
                 _arg(Wq, "Wq", _ANY, q8_packed_weight_bytes(N, K)))
    _check(_lib.q8_pack_weights(w, N, K, wq, _stream(stream)), "q8_pack_weights")


def q8_pack_weights_q(q, d16, N: int, K: int, Wq, stream=None) -> None:
    qq, dd, wq = _dev(_arg(q, "q", _I8, _n(N * K, 1)),
                      _arg(d16, "d16", _H16, _n(N * (K // Q8_BLOCK), 2)),
                      _arg(Wq, "Wq", _ANY, q8_packed_weight_bytes(N, K)))
    _check(_lib.q8_pack_weights_q(qq, dd, N, K, wq, _stream(stream)), "q8_pack_weights_q")


def q8_unpack_weights(Wq, N: int, K: int, q, d16, stream=None) -> None:
    wq, qq, dd = _dev(_arg(Wq, "Wq", _ANY, q8_packed_weight_bytes(N, K)),
                      _arg(q, "q", _I8, _n(N * K, 1)),
                      _arg(d16, "d16", _H16, _n(N * (K // Q8_BLOCK), 2)))
    _check(_lib.q8_unpack_weights(wq, N, K, qq, dd, _stream(stream)), "q8_unpack_weights")


def q8_quantize_acts(X, n_rows: int, K: int, Xq, stream=None) -> None:
    x, xq = _dev(_arg(X, "X", _F32, _n(n_rows * K, 4)),
                 _arg(Xq, "Xq", _ANY, q8_act_buffer_bytes(K)))
    _check(_lib.q8_quantize_acts(x, n_rows, K, xq, _stream(stream)), "q8_quantize_acts")


def _mm_checked(Wq, Xq, batch_index, n_live: int, N: int, K: int, Y, xq_bytes: int | None = None):
    return [_arg(Wq, "Wq", _ANY, q8_packed_weight_bytes(N, K)),
            _arg(Xq, "Xq", _ANY, q8_act_buffer_bytes(K) if xq_bytes is None else xq_bytes),
            _arg(batch_index, "batch_index", _I32, _n(n_live, 4)),
            _arg(Y, "Y", _F32, _n(n_live * N, 4))]


def q8_matmul_narrow(Wq, Xq, batch_index, n_live: int, N: int, K: int, Y,
                     stream=None) -> None:
    wq, xq, bi, y = _dev(*_mm_checked(Wq, Xq, batch_index, n_live, N, K, Y))
    _check(_lib.q8_matmul_narrow(wq, xq, bi, n_live, N, K, y, _stream(stream)), "q8_matmul_narrow")


def q8_matmul_narrow_path(Wq, Xq, batch_index, n_live: int, N: int, K: int, Y,
                          path: int, stream=None) -> None:
    wq, xq, bi, y = _dev(*_mm_checked(Wq, Xq, batch_index, n_live, N, K, Y))
    _check(_lib.q8_matmul_narrow_path(wq, xq, bi, n_live, N, K, y, _stream(stream), int(path)),
           "q8_matmul_narrow_path")


def q8_matmul_workspace_bytes(N: int, K: int) -> int:
    return int(_lib.q8_matmul_workspace_bytes(N, K))


class _LaunchInfo(ctypes.Structure):
    _fields_ = [("row_groups_per_wave", ctypes.c_int32), ("column_tiles", ctypes.c_int32),
                ("chunks_in_flight", ctypes.c_int32), ("k_splits", ctypes.c_int32),
                ("slices_per_split", ctypes.c_int32), ("split_workgroups", ctypes.c_int32),
                ("whole_row_workgroups", ctypes.c_int32), ("waves_per_workgroup", ctypes.c_int32),
                ("workgroups", ctypes.c_int64), ("lds_bytes", ctypes.c_int64)]


def q8_matmul_launch_info(N: int, K: int, n_slots: int = Q8_MAX_SLOTS,
                          with_workspace: bool = False) -> dict:
    """The MFMA engine's launch for an N x K matrix (host only)."""
    info = _LaunchInfo()
    _check(_lib.q8_matmul_launch_info(N, K, n_slots, int(with_workspace), ctypes.byref(info)),
           "q8_matmul_launch_info")
    return {name: int(getattr(info, name)) for name, _ in _LaunchInfo._fields_}


def _ws_bytes(workspace, workspace_bytes):
    if workspace_bytes is not None:
        return workspace_bytes
    if isinstance(workspace, torch.Tensor):
        return workspace.numel() * workspace.element_size()
    return 0


def q8_matmul_narrow_ws(Wq, Xq, batch_index, n_live: int, N: int, K: int, Y,
                        workspace, workspace_bytes: int | None = None,
                        stream=None) -> None:
    wq, xq, bi, y, ws = _dev(*_mm_checked(Wq, Xq, batch_index, n_live, N, K, Y),
                             _arg(workspace, "workspace", _ANY, q8_matmul_workspace_bytes(N, K)))
    _check(_lib.q8_matmul_narrow_ws(wq, xq, bi, n_live, N, K, y, ws,
                                    _ws_bytes(workspace, workspace_bytes), _stream(stream)),
           "q8_matmul_narrow_ws")


def q8_matmul_narrow_noalloc(Wq, Xq, batch_index, n_live: int, N: int, K: int, Y,
                             stream=None) -> None:
    wq, xq, bi, y = _dev(*_mm_checked(Wq, Xq, batch_index, n_live, N, K, Y))
    _check(_lib.q8_matmul_narrow_noalloc(wq, xq, bi, n_live, N, K, y, _stream(stream)),
           "q8_matmul_narrow_noalloc")


def q8_matmul_fused_workspace_bytes(N: int, K: int) -> int:
    return int(_lib.q8_matmul_fused_workspace_bytes(N, K))


def _fused_ptrs(Wq, X, n_rows, Xq, batch_index, n_live, N, K, Y, workspace):
    mm = _mm_checked(Wq, Xq, batch_index, n_live, N, K, Y)
    return _dev(mm[0], _arg(X, "X", _F32, _n(n_rows * K, 4)), mm[1], mm[2], mm[3],
                _arg(workspace, "workspace", _ANY, q8_matmul_fused_workspace_bytes(N, K)))


def q8_matmul_narrow_fused(Wq, X, n_rows: int, Xq, batch_index, n_live: int, N: int, K: int,
                           Y, workspace, workspace_bytes: int | None = None,
                           stream=None) -> None:
    wq, x, xq, bi, y, ws = _fused_ptrs(Wq, X, n_rows, Xq, batch_index, n_live, N, K, Y, workspace)
    _check(_lib.q8_matmul_narrow_fused(wq, x, n_rows, xq, bi, n_live, N, K, y, ws,
                                       _ws_bytes(workspace, workspace_bytes), _stream(stream)),
           "q8_matmul_narrow_fused")


def q8_matmul_narrow_fused_bounded(Wq, X, n_rows: int, Xq, batch_index, n_live: int, N: int,
                                   K: int, Y, workspace, max_spins: int, quantize: int,
                                   workspace_bytes: int | None = None, stream=None) -> None:
    wq, x, xq, bi, y, ws = _fused_ptrs(Wq, X, n_rows, Xq, batch_index, n_live, N, K, Y, workspace)
    _check(_lib.q8_matmul_narrow_fused_bounded(wq, x, n_rows, xq, bi, n_live, N, K, y, ws,
                                               _ws_bytes(workspace, workspace_bytes),
                                               int(max_spins), int(quantize), _stream(stream)),
           "q8_matmul_narrow_fused_bounded")


def fused_timeouts(workspace) -> int:
    """The fused workspace's count of matmul workgroups whose wait ran out
    (reads 4 bytes back from the device; synchronises)."""
    w = workspace[Q8_FUSED_TIMEOUTS_OFFSET:Q8_FUSED_TIMEOUTS_OFFSET + 4]
    return int.from_bytes(bytes(w.cpu().numpy().tobytes()), "little")


def q8_act_buffer_bytes_n(K: int, n_slots: int) -> int:
    return int(_lib.q8_act_buffer_bytes_n(K, n_slots))


def q8_quantize_acts_n(X, n_rows: int, K: int, Xq, n_slots: int, stream=None) -> None:
    x, xq = _dev(_arg(X, "X", _F32, _n(n_rows * K, 4)),
                 _arg(Xq, "Xq", _ANY, q8_act_buffer_bytes_n(K, n_slots)))
    _check(_lib.q8_quantize_acts_n(x, n_rows, K, xq, n_slots, _stream(stream)),
           "q8_quantize_acts_n")


def q8_matmul_multi(Wq, Xq, n_slots: int, batch_index, n_live: int, N: int, K: int, Y,
                    stream=None) -> None:
    wq, xq, bi, y = _dev(*_mm_checked(Wq, Xq, batch_index, n_live, N, K, Y,
                                      xq_bytes=q8_act_buffer_bytes_n(K, n_slots)))
    _check(_lib.q8_matmul_multi(wq, xq, n_slots, bi, n_live, N, K, y, _stream(stream)),
           "q8_matmul_multi")


def q8_rope_multi(Y, n_rows: int, row_stride: int, pos, n_heads: int, head_dim: int,
                  base: float, stream=None) -> None:
    need = _n((n_rows - 1) * row_stride + n_heads * head_dim, 4) if n_rows > 0 else 0
    y, p = _dev(_arg(Y, "Y", _F32, need), _arg(pos, "pos", _I32, _n(n_rows, 4)))
    _check(_lib.q8_rope_multi(y, n_rows, row_stride, p, n_heads, head_dim, float(base),
                              _stream(stream)), "q8_rope_multi")


def q8_stream_read(buf, nbytes: int, sink, stream=None) -> None:
    b, sk = _dev(_arg(buf, "buf", _ANY, max(nbytes, 0)), _arg(sink, "sink", _I32, 4 * 1024))
    _check(_lib.q8_stream_read(b, nbytes, sk, _stream(stream)), "q8_stream_read")


def q8_device_supported() -> bool:
    return bool(_lib.q8_device_supported())


def q8_timeline_set(records, max_waves: int) -> None:
    """Timeline build only: the record buffer (int64, Q8_STAMP_WORDS per
    wave) of the following matmul launches; None or max_waves 0 switches
    recording off."""
    if not TIMELINE:
        raise Q8Error(Q8_ERR_UNSUPPORTED, "q8_timeline_set (set Q8_LIBRARY=timeline before the "
                      "first import to load the timeline build)")
    (r,) = _dev(_arg(records, "records", (torch.int64,), 8 * Q8_STAMP_WORDS * max(max_waves, 0)))
    _check(_lib.q8_timeline_set(r, max_waves), "q8_timeline_set")


# ------------------------------------- the attention side (include/q8kv4.h)

Q8_ROTARY_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}
Q8_KV4_MAX_HEAD_DIM = 256
Q8_KV4_MAX_PAGE = 4096
Q8_KV4_MAX_TOKENS = 64
Q8_KV4_MAX_SEQS = 4096
_F64 = (torch.float64,)


class Rotary:
    """A rotary plan: the frequencies of a model's position rotation on the
    device (float64, one for each pair), how values pair up, and the amplitude
    of the rotated values."""

    def __init__(self, inv_freq: torch.Tensor, interleaved: bool = False, amplitude: float = 1.0):
        (addr,) = _dev(_arg(inv_freq, "inv_freq", _F64, 8))
        self.inv_freq = inv_freq
        self.rot_dim = 2 * inv_freq.numel()
        self.interleaved = bool(interleaved)
        self.amplitude = float(amplitude)
        self.device = inv_freq.device
        self._device_index = inv_freq.get_device()
        self._c = _RotaryPlan(addr, self.amplitude, self.rot_dim, int(self.interleaved))
        self._ref = ctypes.addressof(self._c)


def rotary_frequencies(rot_dim: int, base: float = 1e4, scaling: str = "none",
                       factor: float = 1.0, original_context: float = 0.0,
                       low: float = 1.0, high: float | None = None):
    """(frequencies float64 on the host, amplitude) of q8_rotary_frequencies.
    ``low`` and ``high`` bound the ramp of "bands" (default 1..4 turns) and
    "yarn" (1..32).  Both ramps are linear in the turns; a model whose YaRN ramp is
    linear in the pair's index has other frequencies: make its plan from them,
    ``Rotary(frequencies on the device, amplitude=...)``."""
    if scaling not in Q8_ROTARY_SCALINGS:
        raise ValueError(f"scaling: expected one of {sorted(Q8_ROTARY_SCALINGS)}, got {scaling!r}")
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    out = torch.empty(max(rot_dim, 2) // 2, dtype=torch.float64)
    amplitude = ctypes.c_double()
    _check(_lib.q8_rotary_frequencies(rot_dim, base, Q8_ROTARY_SCALINGS[scaling], factor,
                                      original_context, low, high, out.data_ptr(),
                                      ctypes.addressof(amplitude)), "q8_rotary_frequencies")
    return out, amplitude.value


def rotary_plan(rot_dim: int, base: float = 1e4, interleaved: bool = False, scaling: str = "none",
                factor: float = 1.0, original_context: float = 0.0, low: float = 1.0,
                high: float | None = None, device="cuda") -> Rotary:
    """A rotary plan on the device (rotary_frequencies for the scalings)."""
    f, amplitude = rotary_frequencies(rot_dim, base, scaling, factor, original_context, low, high)
    return Rotary(f.to(device), interleaved, amplitude)


class KV4Cache:
    """A paged 4-bit cache: ``n_pages`` pages of ``page_tokens`` positions for
    ``n_kv_heads`` heads of ``head_dim``, and the block table (int32
    [n_slots][max_pages], kept and read by every call) that names the pages of
    each slot.  ``pages`` is allocated unless given (uint8, any contents)."""

    def __init__(self, n_pages: int, page_tokens: int, n_kv_heads: int, head_dim: int,
                 block_table: torch.Tensor, pages: torch.Tensor | None = None):
        nbytes = q8_kv4_page_bytes(n_kv_heads, head_dim, page_tokens)
        if nbytes == 0 or n_pages < 1:
            raise ValueError(f"invalid cache shape: {n_pages} pages of {page_tokens} positions, "
                             f"{n_kv_heads} heads of {head_dim}")
        _arg(block_table, "block_table", _I32, 4)
        if block_table.dim() != 2:
            raise ValueError(f"block_table: expected [n_slots][max_pages], got {list(block_table.shape)}")
        if pages is None:
            pages = torch.empty(n_pages * nbytes, dtype=torch.uint8, device=block_table.device)
        addr, table = _dev(_arg(pages, "pages", _ANY, n_pages * nbytes), ("block_table", block_table))
        self.pages, self.block_table = pages, block_table
        self.n_pages, self.page_tokens = n_pages, page_tokens
        self.n_kv_heads, self.head_dim = n_kv_heads, head_dim
        self.n_slots, self.max_pages = block_table.shape
        self.page_bytes = nbytes
        self.device = block_table.device
        self._device_index = block_table.get_device()
        self._c = _KV4Cache(addr, table, n_pages, self.n_slots, self.max_pages, page_tokens,
                            n_kv_heads, head_dim)
        self._ref = ctypes.addressof(self._c)


def _handle(h, kind, name: str):
    """Address of a handle's C struct, its device checked."""
    if not isinstance(h, kind):
        raise TypeError(f"{name}: expected a {kind.__name__}, got {type(h).__name__}")
    if h._device_index != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: on {h.device}, but the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return h._ref


def _fast(x, name: str, dtype, need_bytes: int, device: int):
    """_dev(_arg(x, name, (dtype,), need_bytes)) for one argument, in a
    fraction of the time where x passes (a decode step's calls take a few
    microseconds on the GPU); anything else goes the long way, which says what
    is wrong with it."""
    if x is None or type(x) is int:
        return x
    if type(x) is torch.Tensor and (x.dtype is dtype or dtype is None) and x.is_cuda and x.get_device() == device \
            and x.is_contiguous() and x.nbytes >= need_bytes:
        return x.data_ptr()
    return _arg(x, name, None if dtype is None else (dtype,), need_bytes)


def _fast_all(*addresses):
    """The device check of the arguments that _fast left to _dev."""
    for a in addresses:
        if type(a) is tuple:
            return _dev(*(a if type(a) is tuple else ("argument", a) for a in addresses))
    return addresses


def _current_device() -> int:
    """The current device, -1 without one."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -1


def _raw_stream(stream, device: int):
    if stream is None and device >= 0:
        return torch._C._cuda_getCurrentRawStream(device)
    return _stream(stream)


def _span(rows: int, stride: int, width: int) -> int:
    """Bytes of `rows` fp32 rows of `width` values, `stride` apart."""
    return _n((rows - 1) * stride + width, 4) if rows > 0 else 0


def q8_rotary(X, Y, n_rows: int, x_stride: int, pos, n_heads: int, head_dim: int,
              rotary: Rotary, y_stride: int | None = None, stream=None) -> None:
    """Y (default stride n_heads * head_dim) = X rotated at pos; X itself may
    be Y, with y_stride = x_stride."""
    w = n_heads * head_dim
    if y_stride is None:
        y_stride = w
    dev = _current_device()
    x, y, p = _fast_all(_fast(X, "X", torch.float32, _span(n_rows, x_stride, w), dev),
                        _fast(Y, "Y", torch.float32, _span(n_rows, y_stride, w), dev),
                        _fast(pos, "pos", torch.int32, _n(n_rows, 4), dev))
    _check(_lib.q8_rotary(x, x_stride, y, y_stride, n_rows, p, n_heads, head_dim,
                          _handle(rotary, Rotary, "rotary"), _raw_stream(stream, dev)), "q8_rotary")


def q8_kv4_page_bytes(n_kv_heads: int, head_dim: int, page_tokens: int) -> int:
    return int(_lib.q8_kv4_page_bytes(n_kv_heads, head_dim, page_tokens))


def q8_kv4_append(cache: KV4Cache, QKV, n_rows: int, row_stride: int, batch_index, pos,
                  rotary: Rotary | None = None, n_q_heads: int = 0, Q=None,
                  q_stride: int | None = None, stream=None) -> None:
    """Append the rows of a QKV projection: QKV fp32 [n_rows][row_stride],
    n_q_heads query heads, then n_kv_heads key heads, then as many value
    heads.  With a Q, the rotated queries go there (rows q_stride apart,
    default n_q_heads * head_dim); without one the queries are skipped."""
    d, kv = cache.head_dim, cache.n_kv_heads
    wq = n_q_heads * d
    width = wq + 2 * kv * d
    if row_stride < width:
        raise ValueError(f"row_stride: {row_stride} is less than the {width} values of a row")
    if q_stride is None:
        q_stride = wq
    dev = _current_device()
    rows, bi, p, out = _fast_all(
        _fast(QKV, "QKV", torch.float32, _span(n_rows, row_stride, width), dev),
        _fast(batch_index, "batch_index", torch.int32, _n(n_rows, 4), dev),
        _fast(pos, "pos", torch.int32, _n(n_rows, 4), dev),
        _fast(Q, "Q", torch.float32, _span(n_rows, q_stride, wq), dev))
    _check(_lib.q8_kv4_append(_handle(cache, KV4Cache, "cache"), rows, rows and rows + 4 * wq,
                              rows and rows + 4 * (wq + kv * d), row_stride, n_rows, bi, p,
                              None if rotary is None else _handle(rotary, Rotary, "rotary"),
                              0 if Q is None else n_q_heads, out, q_stride, _raw_stream(stream, dev)),
           "q8_kv4_append")


def q8_kv4_read(cache: KV4Cache, batch_index, pos, n_rows: int, K, V, stream=None) -> None:
    need = _n(n_rows * cache.n_kv_heads * cache.head_dim, 4)
    dev = _current_device()
    bi, p, k, v = _fast_all(_fast(batch_index, "batch_index", torch.int32, _n(n_rows, 4), dev),
                            _fast(pos, "pos", torch.int32, _n(n_rows, 4), dev),
                            _fast(K, "K", torch.float32, need, dev), _fast(V, "V", torch.float32, need, dev))
    _check(_lib.q8_kv4_read(_handle(cache, KV4Cache, "cache"), bi, p, n_rows, k, v,
                            _raw_stream(stream, dev)),
           "q8_kv4_read")


def q8_kv4_attend_workspace_bytes(cache: KV4Cache, n_seq: int, tokens_per_seq: int,
                                  n_q_heads: int) -> int:
    return int(_lib.q8_kv4_attend_workspace_bytes(cache._ref, n_seq, tokens_per_seq, n_q_heads))


def q8_kv4_attend(cache: KV4Cache, Q, n_seq: int, tokens_per_seq: int, n_q_heads: int,
                  batch_index, pos, O, workspace, scale: float | None = None, window: int = 0,
                  q_stride: int | None = None, o_stride: int | None = None,
                  workspace_bytes: int | None = None, stream=None) -> None:
    """Attention of n_seq * tokens_per_seq query rows over the cache.  scale
    defaults to head_dim ** -0.5, the strides to n_q_heads * head_dim."""
    w, rows = n_q_heads * cache.head_dim, n_seq * tokens_per_seq
    q_stride = w if q_stride is None else q_stride
    o_stride = w if o_stride is None else o_stride
    dev = _current_device()
    q, bi, p, o, ws = _fast_all(_fast(Q, "Q", torch.float32, _span(rows, q_stride, w), dev),
                                _fast(batch_index, "batch_index", torch.int32, _n(rows, 4), dev),
                                _fast(pos, "pos", torch.int32, _n(rows, 4), dev),
                                _fast(O, "O", torch.float32, _span(rows, o_stride, w), dev),
                                _fast(workspace, "workspace", None, 0, dev))
    _check(_lib.q8_kv4_attend(_handle(cache, KV4Cache, "cache"), q, q_stride, n_seq, tokens_per_seq,
                              n_q_heads, bi, p, cache.head_dim ** -0.5 if scale is None else scale,
                              window, o, o_stride, ws, _ws_bytes(workspace, workspace_bytes),
                              _raw_stream(stream, dev)), "q8_kv4_attend")


def kv4_attend_workspace(cache: KV4Cache, n_seq: int, tokens_per_seq: int,
                         n_q_heads: int) -> torch.Tensor:
    """A zero-filled workspace for q8_kv4_attend."""
    nbytes = q8_kv4_attend_workspace_bytes(cache, n_seq, tokens_per_seq, n_q_heads)
    if nbytes == 0:
        raise ValueError(f"invalid attention shape: {n_seq} sequences of {tokens_per_seq} tokens, "
                         f"{n_q_heads} query heads over {cache.n_kv_heads}")
    return torch.zeros(nbytes, dtype=torch.uint8, device=cache.device)


# --------------------------------- the feed-forward side (include/q8ffn.h)

Q8_ACTS_FORMATS = {"q8_0": 0, "mx4": 1, "mx6": 2, "mx8": 3}
Q8_ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4, "identity": 5}
Q8_NORM_KINDS = {"rms": 0, "layer": 1}
Q8_FFN_MAX_ROWS = 1 << 20
Q8_NORM_MAX_WIDTH = 1 << 15
_U8 = (torch.uint8,)


def q8_acts_bytes(n_slots: int, K: int, format: str) -> int:
    kind = Q8_ACTS_FORMATS[format]
    return int(_lib.q8_acts_bytes(n_slots, K, kind)) if 0 < n_slots <= Q8_FFN_MAX_ROWS else 0


def q8_mx4_weight_bytes(N: int, K: int) -> int:
    return int(_lib.q8_mx4_weight_bytes(N, K))


class MX4Weights:
    """An N x K weight matrix in 4-bit microscaled blocks (``data``: uint8,
    allocated unless given; fill it with q8_mx4_pack_weights or
    q8_mx4_pack_weights_q)."""

    def __init__(self, N: int, K: int, data: torch.Tensor | None = None, device="cuda"):
        nbytes = q8_mx4_weight_bytes(N, K)
        if nbytes == 0:
            raise ValueError(f"invalid shape N={N} K={K}")
        if data is None:
            data = torch.empty(nbytes, dtype=torch.uint8, device=device)
        (addr,) = _dev(_arg(data, "data", _ANY, nbytes))
        self.data, self.N, self.K, self.nbytes = data, N, K, nbytes
        self.device = data.device
        self._device_index = data.get_device()
        self._c = _MX4Weights(addr, N, K)
        self._ref = ctypes.addressof(self._c)


class Acts:
    """A buffer of ``n_slots`` quantised activation rows of K values: "mx4",
    "mx6" or "mx8", or "q8_0" for the slot buffer that q8_matmul_narrow takes
    (as ``data``).  ``data`` is allocated, all zeros, unless given."""

    def __init__(self, n_slots: int, K: int, format: str = "mx8", data: torch.Tensor | None = None,
                 device="cuda"):
        if format not in Q8_ACTS_FORMATS:
            raise ValueError(f"format: expected one of {sorted(Q8_ACTS_FORMATS)}, got {format!r}")
        nbytes = q8_acts_bytes(n_slots, K, format)
        if nbytes == 0:
            raise ValueError(f"invalid buffer shape: {n_slots} slots of {K} values in {format}")
        if data is None:
            data = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        (addr,) = _dev(_arg(data, "data", _ANY, nbytes))
        self.data, self.n_slots, self.K, self.format, self.nbytes = data, n_slots, K, format, nbytes
        self.device = data.device
        self._device_index = data.get_device()
        self._c = _Acts(addr, K, n_slots, Q8_ACTS_FORMATS[format])
        self._ref = ctypes.addressof(self._c)


class Norm:
    """A norm of rows of ``width`` values: kind "rms" or "layer", weight and
    bias fp32 [width] or, one row of them for each row of a call,
    [rows][width] (None: none).  ``offset`` is added to the weight."""

    def __init__(self, width: int, kind: str = "rms", weight: torch.Tensor | None = None,
                 bias: torch.Tensor | None = None, eps: float = 1e-6, offset: float = 0.0):
        if kind not in Q8_NORM_KINDS:
            raise ValueError(f"kind: expected one of {sorted(Q8_NORM_KINDS)}, got {kind!r}")
        for name, t in (("weight", weight), ("bias", bias)):
            if t is not None and (not isinstance(t, torch.Tensor) or t.dim() not in (1, 2) or t.shape[-1] != width):
                raise ValueError(f"{name}: expected a tensor of [{width}] or [rows][{width}]")
        w, b = _dev(_arg(weight, "weight", _F32), _arg(bias, "bias", _F32))
        self.width, self.kind, self.weight, self.bias = width, kind, weight, bias
        self.eps, self.offset = float(eps), float(offset)
        given = [t for t in (weight, bias) if t is not None]
        if len({t.device for t in given}) > 1:
            raise ValueError(f"bias: on {bias.device}, but the weight is on {weight.device}")
        # rows that the tensors hold, where there is one for each row of a call
        self.rows = min((t.shape[0] for t in given if t.dim() == 2), default=None)
        self.device = given[0].device if given else None
        self._device_index = given[0].get_device() if given else None
        stride = [0 if t is None or t.dim() == 1 else width for t in (weight, bias)]
        self._c = _Norm(w, b, *stride, self.eps, self.offset, Q8_NORM_KINDS[kind])
        self._ref = ctypes.addressof(self._c)


def _norm_ref(n, name: str, width: int, n_rows: int):
    if n is None:
        return None
    if isinstance(n, Norm):
        if n.width != width:
            raise ValueError(f"{name}: a norm of {n.width} values for rows of {width}")
        if n.rows is not None and n.rows < n_rows:
            raise ValueError(f"{name}: weights of {n.rows} rows for {n_rows}")
        if n._device_index is None:
            return n._ref
    return _handle(n, Norm, name)


def q8_mx4_pack_weights(W, weights: MX4Weights, stream=None) -> None:
    (w,) = _dev(_arg(W, "W", _F32, _n(weights.N * weights.K, 4)))
    _check(_lib.q8_mx4_pack_weights(w, _handle(weights, MX4Weights, "weights"), _stream(stream)),
           "q8_mx4_pack_weights")


def _codes(codes, scales, weights):
    return _dev(_arg(codes, "codes", _U8, weights.N * weights.K // 2),
                _arg(scales, "scales", _U8, weights.N * weights.K // 32))


def q8_mx4_pack_weights_q(codes, scales, weights: MX4Weights, stream=None) -> None:
    """codes uint8 [N][K/2] (two to a byte, the even column low) and scale
    bytes uint8 [N][K/32]."""
    c, s = _codes(codes, scales, weights)
    _check(_lib.q8_mx4_pack_weights_q(c, s, _handle(weights, MX4Weights, "weights"), _stream(stream)),
           "q8_mx4_pack_weights_q")


def q8_mx4_unpack_weights(weights: MX4Weights, codes, scales, stream=None) -> None:
    c, s = _codes(codes, scales, weights)
    _check(_lib.q8_mx4_unpack_weights(_handle(weights, MX4Weights, "weights"), c, s, _stream(stream)),
           "q8_mx4_unpack_weights")


# A call's count of rows is checked here too: ctypes keeps the low 32 bits of a larger number.
_Tensor, _float32, _int32 = torch.Tensor, torch.float32, torch.int32
# None in a torch without a device, where no handle or tensor leads to a call of them.
_get_device = getattr(torch._C, "_cuda_getDevice", None)
_get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _address(x, name: str, dtype, need_bytes: int, dev: int):
    """_fast, without its test for a device that get_device() answers too."""
    if type(x) is _Tensor and x.get_device() == dev and x.dtype is dtype and x.nbytes >= need_bytes \
            and x.is_contiguous() and dev >= 0:
        return x.data_ptr()
    return _fast(x, name, dtype, need_bytes, dev)


def _short(h, kind, name: str, dev: int):
    """_handle(h, kind, name) where the current device is known."""
    return h._ref if type(h) is kind and h._device_index == dev else _handle(h, kind, name)


def q8_mx_quantize_acts(X, n_rows: int, acts: Acts, x_stride: int | None = None, stream=None) -> None:
    """Rows of X (x_stride apart, default K) into slots 0 .. n_rows - 1."""
    if not 0 < n_rows <= Q8_FFN_MAX_ROWS:
        _check(Q8_ERR_INVALID_ARG, "q8_mx_quantize_acts")
    K = acts.K
    if x_stride is None:
        x_stride = K
    dev = _get_device() if type(acts) is Acts else _current_device()
    x = _address(X, "X", _float32, 4 * ((n_rows - 1) * x_stride + K), dev)
    if type(x) is tuple:
        (x,) = _fast_all(x)
    rc = _lib.q8_mx_quantize_acts(x, x_stride, n_rows, _short(acts, Acts, "acts", dev), _get_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _check(rc, "q8_mx_quantize_acts")


def q8_mx_read_acts(acts: Acts, batch_index, n_rows: int, X, stream=None) -> None:
    """The values of slots batch_index[0 .. n_rows - 1] (None: slots 0 ..)."""
    if not 0 < n_rows <= Q8_FFN_MAX_ROWS:
        _check(Q8_ERR_INVALID_ARG, "q8_mx_read_acts")
    dev = _get_device() if type(acts) is Acts else _current_device()
    bi = None if batch_index is None else _address(batch_index, "batch_index", _int32, 4 * n_rows, dev)
    x = _address(X, "X", _float32, 4 * n_rows * acts.K, dev)
    if type(bi) is tuple or type(x) is tuple:
        bi, x = _fast_all(bi, x)
    rc = _lib.q8_mx_read_acts(_short(acts, Acts, "acts", dev), bi, n_rows, x, _get_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _check(rc, "q8_mx_read_acts")


def q8_mx4_matmul(weights: MX4Weights, acts: Acts, batch_index, n_live: int, Y, y_stride: int | None = None,
                  stream=None) -> None:
    """Y [n_live][N] (rows y_stride apart, default N); token t takes slot
    batch_index[t] (None: slot t)."""
    if not 0 < n_live <= Q8_FFN_MAX_ROWS:
        _check(Q8_ERR_INVALID_ARG, "q8_mx4_matmul")
    N = weights.N
    if y_stride is None:
        y_stride = N
    dev = _get_device() if type(weights) is MX4Weights else _current_device()
    bi = None if batch_index is None else _address(batch_index, "batch_index", _int32, 4 * n_live, dev)
    y = _address(Y, "Y", _float32, 4 * ((n_live - 1) * y_stride + N), dev)
    if type(bi) is tuple or type(y) is tuple:
        bi, y = _fast_all(bi, y)
    rc = _lib.q8_mx4_matmul(_short(weights, MX4Weights, "weights", dev), _short(acts, Acts, "acts", dev), bi, n_live, y,
                            y_stride, _get_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _check(rc, "q8_mx4_matmul")


def q8_mx4_gated(gate: MX4Weights, up: MX4Weights, acts: Acts, batch_index, n_live: int, H=None,
                 h_acts: Acts | None = None, activation: str = "silu", h_stride: int | None = None,
                 stream=None) -> None:
    """activation(gate x) * (up x) for each token: fp32 rows to H, quantised
    ones to slots 0 .. n_live - 1 of h_acts, or both."""
    kind = Q8_ACTIVATIONS.get(activation)
    if kind is None:
        raise ValueError(f"activation: expected one of {sorted(Q8_ACTIVATIONS)}, got {activation!r}")
    if not 0 < n_live <= Q8_FFN_MAX_ROWS:
        _check(Q8_ERR_INVALID_ARG, "q8_mx4_gated")
    N = gate.N
    if h_stride is None:
        h_stride = N
    dev = _get_device() if type(gate) is MX4Weights else _current_device()
    bi = None if batch_index is None else _address(batch_index, "batch_index", _int32, 4 * n_live, dev)
    h = None if H is None else _address(H, "H", _float32, 4 * ((n_live - 1) * h_stride + N), dev)
    if type(bi) is tuple or type(h) is tuple:
        bi, h = _fast_all(bi, h)
    rc = _lib.q8_mx4_gated(_short(gate, MX4Weights, "gate", dev), _short(up, MX4Weights, "up", dev),
                           _short(acts, Acts, "acts", dev), bi, n_live, kind, h, h_stride,
                           None if h_acts is None else _short(h_acts, Acts, "h_acts", dev), _get_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _check(rc, "q8_mx4_gated")


def q8_norm_step(X, n_rows: int, K: int, post: Norm | None = None, gate=None, scale: float = 1.0, residual=None,
                 residual_out=None, pre: Norm | None = None, Y=None, acts: Acts | None = None,
                 x_stride: int | None = None, gate_stride: int | None = None, residual_stride: int | None = None,
                 residual_out_stride: int | None = None, y_stride: int | None = None, stream=None) -> None:
    """residual_out = residual + scale * gate * post(X); y = pre(residual_out)
    goes to Y, to acts, or both.  Strides default to K, gate_stride to 0 (one
    gate for all rows) unless the gate is a tensor of two dimensions."""
    if not 0 < n_rows <= Q8_FFN_MAX_ROWS:
        _check(Q8_ERR_INVALID_ARG, "q8_norm_step")
    xs = K if x_stride is None else x_stride
    rs = K if residual_stride is None else residual_stride
    os = K if residual_out_stride is None else residual_out_stride
    ys = K if y_stride is None else y_stride
    if gate_stride is None:
        gate_stride = K if isinstance(gate, torch.Tensor) and gate.dim() == 2 else 0
    dev = _get_device() if type(X) is _Tensor and X.is_cuda else _current_device()
    f32 = _float32
    x = _address(X, "X", f32, 4 * ((n_rows - 1) * xs + K), dev)
    g = None if gate is None else _address(gate, "gate", f32, 4 * ((n_rows - 1) * gate_stride + K), dev)
    r = None if residual is None else _address(residual, "residual", f32, 4 * ((n_rows - 1) * rs + K), dev)
    o = None if residual_out is None else _address(residual_out, "residual_out", f32, 4 * ((n_rows - 1) * os + K), dev)
    y = None if Y is None else _address(Y, "Y", f32, 4 * ((n_rows - 1) * ys + K), dev)
    if type(x) is tuple or type(g) is tuple or type(r) is tuple or type(o) is tuple or type(y) is tuple:
        x, g, r, o, y = _fast_all(x, g, r, o, y)
    rc = _lib.q8_norm_step(x, xs, None if post is None else _norm_ref(post, "post", K, n_rows), g, gate_stride, scale,
                           r, rs, o, os, None if pre is None else _norm_ref(pre, "pre", K, n_rows), y, ys,
                           None if acts is None else _short(acts, Acts, "acts", dev), n_rows, K,
                           _get_stream(dev) if stream is None and dev >= 0 else _stream(stream))
    if rc:
        _check(rc, "q8_norm_step")


# ------------------------------------------------- torch allocation helpers

def empty_packed_weights(N: int, K: int, device="cuda") -> torch.Tensor:
    nbytes = q8_packed_weight_bytes(N, K)
    if nbytes == 0:
        raise ValueError(f"invalid shape N={N} K={K}")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def zeroed_workspace(N: int, K: int, device="cuda") -> torch.Tensor | None:
    """A zero-filled workspace for q8_matmul_narrow_ws (None if the shape
    needs none)."""
    nbytes = q8_matmul_workspace_bytes(N, K)
    if nbytes == 0:
        return None
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def zeroed_fused_workspace(N: int, K: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for q8_matmul_narrow_fused."""
    nbytes = q8_matmul_fused_workspace_bytes(N, K)
    if nbytes == 0:
        raise ValueError(f"invalid shape N={N} K={K}")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def empty_act_slots(K: int, device="cuda", n_slots: int = Q8_MAX_SLOTS) -> torch.Tensor:
    nbytes = q8_act_buffer_bytes_n(K, n_slots)
    if nbytes == 0:
        raise ValueError(f"invalid K={K} or n_slots={n_slots}")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def read_act_slots(Xq: torch.Tensor, K: int, stream=None, n_slots: int = Q8_MAX_SLOTS):
    """All slots of a slot buffer in canonical q8_0 form:
    (q int8 [n_slots][K], d16 int16 [n_slots][K/32]) device tensors."""
    q = torch.empty((n_slots, K), dtype=torch.int8, device=Xq.device)
    d = torch.empty((n_slots, K // Q8_BLOCK), dtype=torch.int16, device=Xq.device)
    q8_unpack_weights(Xq, n_slots, K, q, d, stream)
    return q, d


def write_act_slots(Xq: torch.Tensor, K: int, q: torch.Tensor, d16: torch.Tensor,
                    stream=None, n_slots: int = Q8_MAX_SLOTS) -> None:
    """Write all slots from canonical q8_0 (q int8 [n_slots][K], d16 int16
    [n_slots][K/32] binary16 bits)."""
    q8_pack_weights_q(q, d16, n_slots, K, Xq, stream)
