"""Thin ctypes binding of libfp8bs (C ABI declared in ``include/fp8bs.h``).

Each ``fp8bs_*`` function has the name and argument order of the C entry
point; tensors (PyTorch, on the GPU) stand for the device pointers and their
row strides are taken from the tensor.  Nothing here computes: every step
runs in the library's HIP kernels.  The ``quant_*`` / ``gemm`` helpers at the
bottom only allocate output tensors and call the entry points.

The library must have been built (``python -m fp8_fine_grained_fp8bs_amd.build``);
loading fails loudly otherwise.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfp8bs.so")
# the compiled short way into the operators of small calls, of this Python
MARSHAL_PATH = os.path.join(PKG, "_marshal" + importlib.machinery.EXTENSION_SUFFIXES[0])

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED_SHAPE = 2
ERR_MISALIGNED = 3
ERR_NO_DEVICE = 4
ERR_LAUNCH = 5

OUT_BF16 = 0
OUT_F32 = 1
BSCALE_BLOCK_128x128 = 0
BSCALE_ROW_1x128 = 1
SRC_FP8_1x128 = 0
SRC_BF16 = 1
SRC_E5M6 = 2
ROPE_HALF = 0
ROPE_INTERLEAVED = 1
INDEX_I32 = 0
INDEX_I64 = 1

ENTRY_POINTS = ("fp8bs_quant_act_1x128", "fp8bs_quant_w_128x128", "fp8bs_quant_act_w",
                "fp8bs_swiglu_quant_1x128",
                "fp8bs_quant_per_tensor",
                "fp8bs_cast_e4m3",
                "fp8bs_encode_e5m6", "fp8bs_decode_e5m6", "fp8bs_requant_T_128x1",
                "fp8bs_transpose_w_128x128", "fp8bs_gemm", "fp8bs_gemm_quant_1x128", "fp8bs_gemm_bf16a",
                "fp8bs_grouped_gemm",
                "fp8bs_rope_table", "fp8bs_rope", "fp8bs_kv_append", "fp8bs_attn_paged",
                "fp8bs_attn_paged_ws",
                "fp8bs_rmsnorm_quant_1x128", "fp8bs_rmsnorm_bwd", "fp8bs_rmsnorm_bwd_ws",
                "fp8bs_moe_sort", "fp8bs_moe_sort_ws", "fp8bs_moe_gather", "fp8bs_moe_dispatch",
                "fp8bs_moe_combine", "fp8bs_moe_combine_bwd", "fp8bs_swiglu_bwd_quant_1x128",
                "fp8bs_status_string", "fp8bs_version")

_lib = None
_lib_path = LIB_PATH
_functions = {}      # the loaded library's entry points by name
_addresses = {}      # and their addresses
_marshal = None      # the compiled short way into the operators of small calls
_ways = {}           # its functions with the loaded library's entry points


class _Names(dict):
    """Names of dtypes (str() of one costs more than a call's other checks)."""

    def __missing__(self, dtype):
        name = self[dtype] = str(dtype).replace("torch.", "")
        return name


_dtype_names = _Names()


def use_library(path: str) -> str:
    """Route every later call through another build of the library (the
    tests use the LDS-poisoning debug build, ``libfp8bs_poison.so``);
    returns the path in use before."""
    global _lib, _lib_path
    prev = _lib_path
    _lib_path, _lib = path, None
    _functions.clear()
    _addresses.clear()
    _ways.clear()
    for sizes in (_ws_bytes, _norm_ws_bytes, _sort_ws_bytes):
        sizes.cache_clear()
    return prev


class Fp8bsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def load() -> ctypes.CDLL:
    """Load libfp8bs.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_lib_path):
        raise RuntimeError(f"{_lib_path} is missing: build it with "
                           "`python -m fp8_fine_grained_fp8bs_amd.build` (hipcc, gfx950)")
    lib = ctypes.CDLL(_lib_path)
    P, I64, I32, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    F, F64 = ctypes.c_float, ctypes.c_double
    sigs = {
        "fp8bs_quant_act_1x128": [P, I64, I64, I64, P, I64, P, I64, P],
        "fp8bs_swiglu_quant_1x128": [P, I64, P, I64, I64, I64, P, I64, P, I64, P, I64, P],
        "fp8bs_quant_w_128x128": [P, I64, I64, I64, P, I64, P, I64, P],
        "fp8bs_quant_act_w": [P, I64, I64, P, I64, P, I64, P, I64, I64, P, I64, P, I64, I64, P],
        "fp8bs_quant_per_tensor": [P, I64, P, P, P],
        "fp8bs_cast_e4m3": [P, I64, P, P],
        "fp8bs_encode_e5m6": [P, I64, I64, I64, P, I64, P],
        "fp8bs_decode_e5m6": [P, I64, I64, I64, P, I64, P],
        "fp8bs_requant_T_128x1": [I, P, P, I64, I64, I64, I64, P, I64, P, I64, P],
        "fp8bs_transpose_w_128x128": [P, I64, I64, I64, P, I64, P, I64, P, I64, P],
        "fp8bs_gemm": [P, P, I64, I64, P, P, I64, I64, I, P, I64, I, I64, I64, I64, P],
        "fp8bs_gemm_quant_1x128": [P, P, I64, I64, P, P, I64, I64, I, P, I64, P, I64, I64, I64, I64, P],
        "fp8bs_grouped_gemm": [P, P, I64, P, P, P, I32, I64, P, I, I64, I64, P],
        "fp8bs_gemm_bf16a": [P, I64, P, I64, P, I64, P, P, I64, I64, P, I64, I, I64, I64, I64, P],
        "fp8bs_rope_table": [P, I64, I64, F64, F64, F64, F64, F64, F64, P],
        "fp8bs_rope": [P, I64, P, I64, P, I64, I64, I64, I64, I64, I, I, P, I64, P],
        "fp8bs_kv_append": [P, I64, P, I64, I64, P, I64, P, I64, I64, I64, P, I64, I64, I64, I, P, P, I64, I64,
                            I64, P, I64, I64, I64, P, P, P, P, I64, P],
        "fp8bs_attn_paged": [P, I64, P, I64, P, I64, P, P, I64, I64, I64, I64, I64, I64, P, I64, I64, I64, P, P,
                             P, P, I64, F, I, I64, P, I64, P],
        "fp8bs_rmsnorm_quant_1x128": [P, I64, P, I64, P, I, F, I64, I64, P, I64, P, I64, P, I64, P, I64, P, P],
        "fp8bs_rmsnorm_bwd": [P, I64, P, I64, P, I64, P, I, P, I64, I64, P, I64, P, P, I64, P],
        "fp8bs_moe_sort": [P, I, I64, I64, I64, I64, I64, I64, P, P, P, I64, P],
        "fp8bs_moe_gather": [I, P, I64, P, I64, I64, I64, P, I64, P, I64, P, I64, P, I64, I64, P],
        "fp8bs_moe_dispatch": [I, P, I64, P, I64, I64, I64, P, I, I64, I64, I64, I64, P, P, P, I64, P, I64, P, I64,
                               I64, P, I64, P],
        "fp8bs_moe_combine": [P, I, I64, I64, P, P, I64, I64, I64, I64, P, I64, P, I64, P],
        "fp8bs_moe_combine_bwd": [P, I64, P, I, I64, P, P, I64, I64, I64, I64, P, I64, P, I64, P, I64, I64, P, I64, P],
        "fp8bs_swiglu_bwd_quant_1x128": [P, I64, P, I64, P, I64, I64, I64, P, I64, P, I64, P, I64, P, I64, P],
    }
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.fp8bs_attn_paged_ws.argtypes = [I64] * 8
    lib.fp8bs_attn_paged_ws.restype = I64
    lib.fp8bs_rmsnorm_bwd_ws.argtypes = [I64] * 2
    lib.fp8bs_rmsnorm_bwd_ws.restype = I64
    lib.fp8bs_moe_sort_ws.argtypes = [I64] * 3
    lib.fp8bs_moe_sort_ws.restype = I64
    lib.fp8bs_status_string.argtypes = [ctypes.c_int]
    lib.fp8bs_status_string.restype = ctypes.c_char_p
    lib.fp8bs_version.argtypes = []
    lib.fp8bs_version.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(st: int) -> str:
    return load().fp8bs_status_string(int(st)).decode()


def _ptr(t):
    """Device pointer of a GPU tensor (or an int address, or None for NULL).
    A host tensor is refused here: its address would reach the kernels as a
    device pointer."""
    if t is None or isinstance(t, int):
        return t
    if t.is_cuda:
        return t.data_ptr()
    raise ValueError("libfp8bs takes device tensors; got a tensor on " + str(t.device))


def _ld(t):
    """Row stride (elements) of a row-major 2-D tensor view."""
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"expected a 2-D tensor with contiguous rows, got shape {tuple(t.shape)} "
                         f"strides {tuple(t.stride())}")
    return t.stride(0)


_CODES = ("uint8", "float8_e4m3fn")


def _check(t, what, shape, dtypes, contiguous=False):
    """Refuse a tensor whose shape or dtype does not fit what the kernels
    will read or write (a short output would be written past its end).
    shape entries: an int (exact), (">=", n) (at least n) or None (any)."""
    if t is None:
        raise ValueError(f"{what}: missing tensor")
    if _dtype_names[t.dtype] not in dtypes:
        raise ValueError(f"{what}: dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != len(shape):
        raise ValueError(f"{what}: {t.dim()}-D tensor, expected {len(shape)}-D")
    for i, want in enumerate(shape):
        got = t.shape[i]
        if want is None:
            continue
        if isinstance(want, tuple):
            if got < want[1]:
                raise ValueError(f"{what}: dimension {i} is {got}, needs at least {want[1]}")
        elif got != want:
            raise ValueError(f"{what}: dimension {i} is {got}, expected {want}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if t.dim() == 2:
        _ld(t)


def _groups(K):
    return K // 128


_raw_stream = None


def _current_stream():
    """Handle of the current device's current stream (without the stream
    object, whose making costs as much as a launch)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream = (lambda: get(torch.cuda.current_device())) if get is not None else \
            (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _call(name, *args):
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(load(), name)
    st = fn(*args)
    if st != OK:
        raise Fp8bsError(st, name)


# ---------------------------------------------------------------------------
# entry points (same names and argument order as the C ABI)
# ---------------------------------------------------------------------------

def fp8bs_quant_act_1x128(x, q, s, stream=None):
    """x bf16 [M][K] -> q u8 [M][K], s f32 [M][K/128]."""
    M, K = x.shape
    _check(x, "x", (M, K), ("bfloat16",))
    _check(q, "q", (M, K), _CODES)
    _check(s, "s", (M, (">=", _groups(K))), ("float32",))
    _call("fp8bs_quant_act_1x128", _ptr(x), M, K, _ld(x), _ptr(q), _ld(q), _ptr(s), _ld(s),
          _stream(stream))


def fp8bs_quant_w_128x128(w, q, s, stream=None):
    """w bf16 [N][K] -> q u8 [N][K], s f32 [ceil(N/128)][K/128]."""
    N, K = w.shape
    _check(w, "w", (N, K), ("bfloat16",))
    _check(q, "q", (N, K), _CODES)
    _check(s, "s", ((N + 127) // 128, (">=", _groups(K))), ("float32",))
    _call("fp8bs_quant_w_128x128", _ptr(w), N, K, _ld(w), _ptr(q), _ld(q), _ptr(s), _ld(s),
          _stream(stream))


def fp8bs_quant_per_tensor(x, q, s, stream=None):
    """x bf16 (contiguous, n % 128 == 0) -> q u8 (same shape), s f32 [1]."""
    if not (x.is_contiguous() and q.is_contiguous()) or q.numel() != x.numel():
        raise ValueError("x and q must be contiguous with the same number of elements")
    if str(x.dtype) != "torch.bfloat16" or str(q.dtype).replace("torch.", "") not in _CODES:
        raise ValueError("x must be bfloat16 and q uint8 codes")
    if s is None or s.numel() < 1 or str(s.dtype) != "torch.float32":
        raise ValueError("s must hold one float32")
    _call("fp8bs_quant_per_tensor", _ptr(x), x.numel(), _ptr(q), _ptr(s), _stream(stream))


def fp8bs_cast_e4m3(x, q, stream=None):
    """x f32 (contiguous) -> q u8 (same number of elements): nearest-even
    E4M3 codes, saturated to +-448."""
    if not (x.is_contiguous() and q.is_contiguous()) or q.numel() != x.numel():
        raise ValueError("x and q must be contiguous with the same number of elements")
    if str(x.dtype) != "torch.float32" or str(q.dtype).replace("torch.", "") not in _CODES:
        raise ValueError("x must be float32 and q uint8 codes")
    _call("fp8bs_cast_e4m3", _ptr(x), x.numel(), _ptr(q), _stream(stream))


def fp8bs_encode_e5m6(x, y, stream=None):
    """bf16 x [T][C] -> packed E5M6 y u8 [T][>= 1.5 C]."""
    T, C = x.shape
    _check(x, "x", (T, C), ("bfloat16",))
    _check(y, "y", (T, (">=", (3 * C + 1) // 2)), ("uint8",))
    _call("fp8bs_encode_e5m6", _ptr(x), T, C, _ld(x), _ptr(y), _ld(y), _stream(stream))


def fp8bs_decode_e5m6(y, x, stream=None):
    """packed E5M6 y u8 [T][>= 1.5 C] -> bf16 x [T][C] (exact)."""
    T, C = x.shape
    _check(x, "x", (T, C), ("bfloat16",))
    _check(y, "y", (T, (">=", (3 * C + 1) // 2)), ("uint8",))
    _call("fp8bs_decode_e5m6", _ptr(y), T, C, _ld(y), _ptr(x), _ld(x), _stream(stream))


def fp8bs_requant_T_128x1(src, x, s_in, q_out, s_out, stream=None):
    """x [T][C] (codes with s_in [T][C/128], or bf16), or packed E5M6
    x u8 [T][1.5 C] -> q_out [C][T], s_out [C][ceil(T/128)]."""
    if int(src) == SRC_E5M6:
        T, C = x.shape[0], q_out.shape[0]
        _check(x, "x", (T, C // 2 * 3), _CODES)
    else:
        T, C = x.shape
    if int(src) == SRC_FP8_1x128:
        _check(x, "x", (T, C), _CODES)
        _check(s_in, "s_in", (T, (">=", _groups(C))), ("float32",))
    elif int(src) == SRC_BF16:
        _check(x, "x", (T, C), ("bfloat16",))
    _check(q_out, "q_out", (C, T), _CODES)
    _check(s_out, "s_out", (C, (">=", (T + 127) // 128)), ("float32",))
    lds_in = _ld(s_in) if s_in is not None else 0
    _call("fp8bs_requant_T_128x1", int(src), _ptr(x), _ptr(s_in), T, C, _ld(x), lds_in,
          _ptr(q_out), _ld(q_out), _ptr(s_out), _ld(s_out), _stream(stream))


def fp8bs_transpose_w_128x128(q, s, qt, st, stream=None):
    """Codes q [N][K] with 128x128 block scales s [N/128][K/128] -> their
    transpose qt [K][N], st [K/128][N/128]."""
    N, K = q.shape
    _check(q, "q", (N, K), _CODES)
    _check(s, "s", ((N + 127) // 128, (">=", _groups(K))), ("float32",))
    _check(qt, "qt", (K, N), _CODES)
    _check(st, "st", (_groups(K), (">=", (N + 127) // 128)), ("float32",))
    _call("fp8bs_transpose_w_128x128", _ptr(q), N, K, _ld(q), _ptr(s), _ld(s), _ptr(qt), _ld(qt),
          _ptr(st), _ld(st), _stream(stream))


def _check_gemm_operands(a, sa, b, sb, bmode):
    M, K = a.shape
    N = b.shape[0]
    _check(a, "a", (M, K), _CODES)
    _check(sa, "sa", (M, (">=", _groups(K))), ("float32",))
    _check(b, "b", (N, K), _CODES)
    rows_sb = N if int(bmode) == BSCALE_ROW_1x128 else (N + 127) // 128
    _check(sb, "sb", (rows_sb, (">=", _groups(K))), ("float32",))


def fp8bs_gemm(a, sa, b, sb, bmode, d, dt, stream=None):
    """D [M][N] = A [M][K] * B [N][K]^T with block scales."""
    M, K = a.shape
    N = b.shape[0]
    _check_gemm_operands(a, sa, b, sb, bmode)
    _check(d, "d", (M, N), ("float32",) if int(dt) == OUT_F32 else ("bfloat16",))
    _call("fp8bs_gemm", _ptr(a), _ptr(sa), _ld(a), _ld(sa), _ptr(b), _ptr(sb), _ld(b), _ld(sb),
          int(bmode), _ptr(d), _ld(d), int(dt), M, N, K, _stream(stream))


def fp8bs_gemm_quant_1x128(a, sa, b, sb, bmode, q, s, stream=None):
    """D = A [M][K] * B [N][K]^T, quantized in 1x128 tiles along N:
    q u8 [M][N], s f32 [M][N/128]."""
    M, K = a.shape
    N = b.shape[0]
    _check_gemm_operands(a, sa, b, sb, bmode)
    _check(q, "q", (M, N), _CODES)
    _check(s, "s", (M, (">=", N // 128)), ("float32",))
    _call("fp8bs_gemm_quant_1x128", _ptr(a), _ptr(sa), _ld(a), _ld(sa), _ptr(b), _ptr(sb), _ld(b),
          _ld(sb), int(bmode), _ptr(q), _ld(q), _ptr(s), _ld(s), M, N, K, _stream(stream))


def fp8bs_gemm_bf16a(x, qx, sx, b, sb, d, dt, stream=None):
    """D [M][N] = quant_1x128(x bf16 [M][K]) * B [N][K]^T with 128x128 B
    scales; qx u8 [M][K] and sx f32 [M][K/128] receive the codes of x when
    given (both or neither)."""
    M, K = x.shape
    N = b.shape[0]
    _check(x, "x", (M, K), ("bfloat16",))
    if (qx is None) != (sx is None):
        raise ValueError("qx and sx: both or neither")
    if qx is not None:
        _check(qx, "qx", (M, K), _CODES)
        _check(sx, "sx", (M, (">=", _groups(K))), ("float32",))
    _check(b, "b", (N, K), _CODES)
    _check(sb, "sb", ((N + 127) // 128, (">=", _groups(K))), ("float32",))
    _check(d, "d", (M, N), ("float32",) if int(dt) == OUT_F32 else ("bfloat16",))
    _call("fp8bs_gemm_bf16a", _ptr(x), _ld(x), _ptr(qx), _ld(qx) if qx is not None else 0, _ptr(sx),
          _ld(sx) if sx is not None else 0, _ptr(b), _ptr(sb), _ld(b), _ld(sb), _ptr(d), _ld(d), int(dt),
          M, N, K, _stream(stream))


def fp8bs_grouped_gemm(a, sa, b, sb, offsets, d, dt, stream=None):
    """Per-expert D rows = A rows * B[e]^T; offsets int32 [E+1] on the device."""
    M_total, K = a.shape
    E, N, _ = b.shape
    _check(a, "a", (M_total, K), _CODES, contiguous=True)
    _check(sa, "sa", (M_total, (">=", _groups(K))), ("float32",))
    _check(b, "b", (E, N, K), _CODES, contiguous=True)
    _check(sb, "sb", (E, (N + 127) // 128, _groups(K)), ("float32",), contiguous=True)
    _check(offsets, "offsets", (E + 1,), ("int32",), contiguous=True)
    _check(d, "d", (M_total, N), ("float32",) if int(dt) == OUT_F32 else ("bfloat16",), contiguous=True)
    _call("fp8bs_grouped_gemm", _ptr(a), _ptr(sa), _ld(sa), _ptr(b), _ptr(sb), _ptr(offsets),
          int(E), M_total, _ptr(d), int(dt), N, K, _stream(stream))


def _load_marshal():
    """The short way's functions by entry point: none where it has not been built, or,
    with a warning, was built for another torch."""
    if not os.path.exists(MARSHAL_PATH):
        return {}
    import torch  # its libraries are the module's
    try:
        from . import _marshal as module
        if module.torch_version != torch.__version__:
            raise ImportError(f"built for torch {module.torch_version}, this is {torch.__version__}")
        return {"fp8bs_" + f: getattr(module, f) for f in (
            "rope", "kv_append", "attn_paged", "rmsnorm_quant_1x128", "rmsnorm_bwd", "moe_dispatch", "moe_combine",
            "moe_combine_bwd", "swiglu_bwd_quant_1x128")}
    except (ImportError, AttributeError) as e:
        import warnings
        warnings.warn(f"{MARSHAL_PATH}: {e}; the short helpers go through ctypes")
        return {}


def _short(name, *args):
    """The named operator by the compiled short way (csrc/marshal.cpp): its
    result, or None where an argument is not as it should be (the checks below then
    say which) or there is no short way (the library is then called through ctypes)."""
    global _marshal
    if _marshal is None:
        _marshal = _load_marshal()
    way = _marshal.get(name)
    if way is None:
        return None
    result = way(_address(name), *args)
    if type(result) is int:
        raise Fp8bsError(result, name)
    return result


def _way(name, *sizes):
    """The named operator by the compiled short way, as a function of what follows its
    entry points (the operator's and those of the sizes it needs): like _short for
    helpers whose own time counts, a status is left to them."""
    global _marshal
    if _marshal is None:
        _marshal = _load_marshal()
    way = _marshal.get(name)
    way = _no_way if way is None else functools.partial(way, *map(_address, (name,) + sizes))
    _ways[name] = way
    return way


def _no_way(*args):
    return None


def _address(name):
    address = _addresses.get(name)
    if address is None:
        address = _addresses[name] = ctypes.cast(getattr(load(), name), ctypes.c_void_p).value
    return address


def _stream_later(stream):
    """A stream's handle, or for the current one the function that gives it."""
    return _current_stream if stream is None else _stream(stream)


def _heads(t, what):
    """Row stride (elements) of a [T][H][D] view whose heads are contiguous in a row, and its shape."""
    shape = t.shape
    if len(shape) != 3 or _dtype_names[t.dtype] != "bfloat16":
        raise ValueError(f"{what}: expected a 3-D bfloat16 tensor [T][H][D], got {len(shape)}-D {t.dtype}")
    T, H, D = shape
    row, head, one = t.stride()
    if one != 1 or (H > 1 and head != D):
        raise ValueError(f"{what}: heads must be contiguous in a row, got strides {(row, head, one)}")
    return (row if T > 1 else max(row, H * D)), shape


def _layout(layout):
    if layout in ("half", ROPE_HALF):
        return ROPE_HALF
    if layout in ("interleaved", ROPE_INTERLEAVED):
        return ROPE_INTERLEAVED
    raise ValueError(f"layout: {layout!r}, expected 'half' or 'interleaved'")


def _int32s(t, what, n):
    if t.shape != (n,) or _dtype_names[t.dtype] != "int32" or not t.is_contiguous():
        raise ValueError(f"{what}: expected {n} contiguous int32, got {t.dtype} {tuple(t.shape)}")


def _check_angles(cs):
    """(n_pos, rot) of a table of angles."""
    if _dtype_names[cs.dtype] != "float32" or cs.dim() != 2 or not cs.is_contiguous():
        raise ValueError(f"cs: expected a contiguous float32 table [n_pos][rot], got {cs.dtype} {tuple(cs.shape)}")
    return cs.shape


def _check_cache(kc, ks, vc, vs, table, kv_len, q_off, T):
    """Shapes of a paged cache and its packing; returns
    (B, Hkv, D, page, n_pages, ldt, max_pages)."""
    shape, name = kc.shape, _dtype_names[kc.dtype]
    if len(shape) != 4 or name not in _CODES or not kc.is_contiguous():
        raise ValueError(f"kc: expected contiguous codes [n_pages][Hkv][page][D], got {kc.dtype} {tuple(shape)}")
    if vc.shape != shape or _dtype_names[vc.dtype] != name or not vc.is_contiguous():
        raise ValueError("vc: must have kc's shape and dtype, contiguous")
    n_pages, Hkv, page, D = shape
    blocks = (n_pages, Hkv)
    if ks.shape != blocks or _dtype_names[ks.dtype] != "float32" or not ks.is_contiguous():
        raise ValueError(f"ks: expected contiguous float32 {blocks}, got {ks.dtype} {tuple(ks.shape)}")
    if vs.shape != blocks or _dtype_names[vs.dtype] != "float32" or not vs.is_contiguous():
        raise ValueError(f"vs: expected contiguous float32 {blocks}, got {vs.dtype} {tuple(vs.shape)}")
    listed = table.shape
    if len(listed) != 2 or _dtype_names[table.dtype] != "int32":
        raise ValueError(f"table: expected int32 [B][max_pages], got {table.dtype} {tuple(listed)}")
    B, max_pages = listed
    ldt, one = table.stride()
    if one != 1 and max_pages > 1:
        raise ValueError(f"table: rows must be contiguous, got strides {(ldt, one)}")
    _int32s(kv_len, "kv_len", B)
    if q_off is not None:
        _int32s(q_off, "q_off", B + 1)
    elif T != B:
        raise ValueError(f"q_off: without it every sequence has one row, but T = {T} and B = {B}")
    return B, Hkv, D, page, n_pages, (ldt if B > 1 else max(ldt, max_pages)), max_pages


def fp8bs_rope_table(cs, base, factor, orig_len, turns_lo, turns_hi, mscale, stream=None):
    """cs f32 [n_pos][rot]: cos and sin of every position's angles."""
    _check_angles(cs)
    _call("fp8bs_rope_table", _ptr(cs), cs.shape[0], cs.shape[1], base, factor, orig_len, turns_lo, turns_hi,
          mscale, _stream(stream))


def fp8bs_rope(x, y, pos, rot_off, layout, inverse, cs, stream=None):
    """x bf16 [T][H][D] -> y (same shape; may be x), rotated by the angles
    cs f32 [n_pos][rot] of positions pos i32 [T]."""
    ldx, shape = _heads(x, "x")
    ldy, shape_y = _heads(y, "y")
    T, H, D = shape
    if shape_y != shape:
        raise ValueError(f"y: shape {tuple(shape_y)}, expected {tuple(shape)}")
    _int32s(pos, "pos", T)
    n_pos, rot = _check_angles(cs)
    _call("fp8bs_rope", _ptr(x), ldx, _ptr(y), ldy, _ptr(pos), T, H, D, rot, rot_off, _layout(layout),
          1 if inverse else 0, _ptr(cs), n_pos, _stream(stream))


def fp8bs_kv_append(q, q_out, k, v, cs, rot_off, layout, q_off, kv_len, max_q, table, kc, ks, vc, vs, stream=None):
    """k, v bf16 [T][Hkv][D] into the paged cache kc, vc u8 [n_pages][Hkv][page][D],
    ks, vs f32 [n_pages][Hkv]; q bf16 [T][Hq][D] rotated into q_out (both or neither)."""
    ldk, shape = _heads(k, "k")
    ldv, shape_v = _heads(v, "v")
    T = shape[0]
    B, Hkv, D, page, n_pages, ldt, max_pages = _check_cache(kc, ks, vc, vs, table, kv_len, q_off, T)
    if shape != (T, Hkv, D) or shape_v != shape:
        raise ValueError(f"k, v: shapes {tuple(shape)}, {tuple(shape_v)}, expected {(T, Hkv, D)}")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out: both or neither")
    Hq = ldq = ldqo = n_pos = rot = 0
    if q is not None:
        ldq, shape_q = _heads(q, "q")
        ldqo, shape_o = _heads(q_out, "q_out")
        Hq = shape_q[1]
        if shape_q != (T, Hq, D) or shape_o != shape_q:
            raise ValueError(f"q, q_out: shapes {tuple(shape_q)}, {tuple(shape_o)}, expected {(T, Hq, D)}")
    if cs is not None:
        n_pos, rot = _check_angles(cs)
    _call("fp8bs_kv_append", _ptr(q), ldq, _ptr(q_out), ldqo, Hq, _ptr(k), ldk, _ptr(v), ldv, Hkv, D, _ptr(cs),
          n_pos, rot, rot_off, _layout(layout), _ptr(q_off), _ptr(kv_len), B, T, max_q, _ptr(table), ldt,
          max_pages, page, _ptr(kc), _ptr(ks), _ptr(vc), _ptr(vs), n_pages, _stream(stream))


@functools.lru_cache(maxsize=4096)
def _ws_bytes(*sizes):
    return load().fp8bs_attn_paged_ws(*sizes)


def fp8bs_attn_paged_ws(B, T, max_q, Hq, Hkv, D, max_pages, page):
    """Bytes of working memory fp8bs_attn_paged needs (-1: invalid sizes)."""
    return _ws_bytes(B, T, max_q, Hq, Hkv, D, max_pages, page)


def fp8bs_attn_paged(q, out, lse, q_off, kv_len, max_q, table, kc, ks, vc, vs, scale, causal, window, ws,
                     stream=None):
    """q bf16 [T][Hq][D] -> out (same shape) and lse f32 [T][Hq] (or None):
    attention over the paged cache; ws uint8 [>= fp8bs_attn_paged_ws(...)]."""
    ldq, shape = _heads(q, "q")
    ldo, shape_o = _heads(out, "out")
    T, Hq, D = shape
    B, Hkv, Dc, page, n_pages, ldt, max_pages = _check_cache(kc, ks, vc, vs, table, kv_len, q_off, T)
    if Dc != D or shape_o != shape:
        raise ValueError(f"q, out: shapes {tuple(shape)}, {tuple(shape_o)}, expected heads of {Dc}")
    ldl = ws_bytes = 0
    if lse is not None:
        _check(lse, "lse", (T, Hq), ("float32",))
        ldl = _ld(lse) if T > 1 else max(lse.stride(0), Hq)
    if ws is not None:
        if not ws.is_contiguous():
            raise ValueError("ws: must be contiguous")
        ws_bytes = ws.numel() * ws.element_size()
    _call("fp8bs_attn_paged", _ptr(q), ldq, _ptr(out), ldo, _ptr(lse), ldl, _ptr(q_off), _ptr(kv_len), B, T, max_q,
          Hq, Hkv, D, _ptr(table), ldt, max_pages, page, _ptr(kc), _ptr(ks), _ptr(vc), _ptr(vs), n_pages,
          scale, 1 if causal else 0, window, _ptr(ws), ws_bytes, _stream(stream))


def _row_ld(t, cols):
    """Row stride of a checked 2-D tensor (a single row's does not matter), or 0 for None."""
    if t is None:
        return 0
    return t.stride(0) if t.shape[0] > 1 else cols


def _optional(t, what, shape, dtypes):
    if t is not None:
        _check(t, what, shape, dtypes)


def _dtype(t, what):
    """OUT_BF16 or OUT_F32 by the tensor's type."""
    name = _dtype_names[t.dtype]
    if name not in ("bfloat16", "float32"):
        raise ValueError(f"{what}: dtype {t.dtype}, expected bfloat16 or float32")
    return OUT_F32 if name == "float32" else OUT_BF16


def _vector(t, what, n, dtypes):
    if t is None or t.shape != (n,) or _dtype_names[t.dtype] not in dtypes or not t.is_contiguous():
        got = None if t is None else (t.dtype, tuple(t.shape))
        raise ValueError(f"{what}: expected {n} contiguous values of {dtypes}, got {got}")


def _here(*tensors):
    """Refuse tensors that are not on the current device, on which the kernels run."""
    import torch
    device = None
    for t in tensors:
        if t is None:
            continue
        _ptr(t)
        if device is None:
            device = torch.cuda.current_device()
        if t.get_device() != device:
            raise ValueError(f"tensors have to be on the current device {device}; got one on {t.device}")


def _workspace(ws):
    """Bytes of a workspace tensor."""
    if ws is None:
        return 0
    if not ws.is_contiguous():
        raise ValueError("ws: must be contiguous")
    return ws.numel() * ws.element_size()


def _check_rows(q, s, y, C, rows=None):
    """Row outputs (codes with scales, BF16): both of q and s or neither, all with
    the same number of rows, which is returned (`rows` where there are none)."""
    if (q is None) != (s is None):
        raise ValueError("q and s: both or neither")
    if rows is None:
        rows = q.shape[0] if q is not None else y.shape[0] if y is not None else 0
    _optional(q, "q", (rows, C), _CODES)
    _optional(s, "s", (rows, (">=", _groups(C))), ("float32",))
    _optional(y, "y", (rows, C), ("bfloat16",))
    return rows


def _row_count(q, s, y, C):
    """Rows of a dispatch's or a gather's outputs, of which there has to be one."""
    if q is None and y is None:
        raise ValueError("no output")
    return _check_rows(q, s, y, C)


def fp8bs_rmsnorm_quant_1x128(x, r, gamma, eps, h, q, s, y, rstd, stream=None):
    """x (and r) bf16 [T][C], gamma bf16 or f32 [C] -> h = x + r bf16 [T][C] (with
    r), its norm as q u8 [T][C] with s f32 [T][C/128] and/or y bf16 [T][C], and
    rstd f32 [T] (or None)."""
    _check(x, "x", (None, None), ("bfloat16",))
    T, C = x.shape
    if (r is None) != (h is None):
        raise ValueError("r and h: both or neither")
    _optional(r, "r", (T, C), ("bfloat16",))
    _optional(h, "h", (T, C), ("bfloat16",))
    _vector(gamma, "gamma", C, ("bfloat16", "float32"))
    if q is None and y is None:
        raise ValueError("no output")
    _check_rows(q, s, y, C, T)
    if rstd is not None:
        _vector(rstd, "rstd", T, ("float32",))
    _here(x, r, gamma, h, q, s, y, rstd)
    _call("fp8bs_rmsnorm_quant_1x128", _ptr(x), _row_ld(x, C), _ptr(r), _row_ld(r, C), _ptr(gamma),
          _dtype(gamma, "gamma"), eps, T, C, _ptr(h), _row_ld(h, C), _ptr(q), _row_ld(q, C), _ptr(s),
          _row_ld(s, _groups(C)), _ptr(y), _row_ld(y, C), _ptr(rstd), _stream(stream))


@functools.lru_cache(maxsize=4096)
def _norm_ws_bytes(T, C):
    return load().fp8bs_rmsnorm_bwd_ws(T, C)


def fp8bs_rmsnorm_bwd_ws(T, C):
    """Bytes of working memory fp8bs_rmsnorm_bwd needs (-1: invalid sizes)."""
    return _norm_ws_bytes(T, C)


def fp8bs_rmsnorm_bwd(dn, dres, h, gamma, rstd, dx, dgamma, ws, stream=None):
    """Gradient of the norm of h bf16 [T][C]: dn (and dres or None) bf16 [T][C] ->
    dx bf16 [T][C] and dgamma f32 [C] (or None; with it ws uint8
    [>= fp8bs_rmsnorm_bwd_ws(T, C)])."""
    _check(h, "h", (None, None), ("bfloat16",))
    T, C = h.shape
    _check(dn, "dn", (T, C), ("bfloat16",))
    _optional(dres, "dres", (T, C), ("bfloat16",))
    _check(dx, "dx", (T, C), ("bfloat16",))
    _vector(gamma, "gamma", C, ("bfloat16", "float32"))
    _vector(rstd, "rstd", T, ("float32",))
    if dgamma is not None:
        _vector(dgamma, "dgamma", C, ("float32",))
    _here(dn, dres, h, gamma, rstd, dx, dgamma, ws)
    _call("fp8bs_rmsnorm_bwd", _ptr(dn), _row_ld(dn, C), _ptr(dres), _row_ld(dres, C), _ptr(h), _row_ld(h, C),
          _ptr(gamma), _dtype(gamma, "gamma"), _ptr(rstd), T, C, _ptr(dx), _row_ld(dx, C), _ptr(dgamma), _ptr(ws),
          _workspace(ws), _stream(stream))


@functools.lru_cache(maxsize=4096)
def _sort_ws_bytes(T, k, E):
    return load().fp8bs_moe_sort_ws(T, k, E)


def fp8bs_moe_sort_ws(T, k, E):
    """Bytes of working memory fp8bs_moe_sort and fp8bs_moe_dispatch need (-1: invalid sizes)."""
    return _sort_ws_bytes(T, k, E)


def _overlap(at, rows, width, step, begin, nbytes):
    """Whether nbytes from address begin lie on rows of width bytes, step bytes apart, from address at."""
    if begin >= at + (rows - 1) * step + width or begin + nbytes <= at or width == 0 or nbytes == 0:
        return False
    first = max(0, (begin - at - width) // step + 1) if rows > 1 else 0   # of the rows that end behind begin
    return first < rows and at + first * step < begin + nbytes


def _check_apart(ids, offsets, slot, ws):
    """Refuse a caller's outputs and working memory that lie on the ids [T][k] of a sort."""
    if ids.dim() != 2:
        return      # refused with the ids
    (T, k), item, at = ids.shape, ids.element_size(), ids.data_ptr()
    for name, t in (("offsets", offsets), ("slot", slot), ("ws", ws)):
        if t is not None and _overlap(at, T, k * item, max(ids.stride(0), 1) * item, t.data_ptr(),
                                      t.numel() * t.element_size()):
            raise ValueError(f"{name}: must not overlap ids")


def _check_ids(ids, offsets, slot):
    """(index type, row stride, T, k, E) of a sort."""
    if _dtype_names[ids.dtype] not in ("int32", "int64") or ids.dim() != 2:
        raise ValueError(f"ids: expected int32 or int64 [T][k], got {ids.dtype} {tuple(ids.shape)}")
    T, k = ids.shape
    row, one = ids.stride()
    if one != 1 and k > 1:
        raise ValueError(f"ids: rows must be contiguous, got strides {(row, one)}")
    _check(offsets, "offsets", ((">=", 2),), ("int32",), contiguous=True)
    _check(slot, "slot", (T, k), ("int32",), contiguous=True)
    return (INDEX_I64 if _dtype_names[ids.dtype] == "int64" else INDEX_I32), _row_ld(ids, k), T, k, offsets.shape[0] - 1


def fp8bs_moe_sort(ids, first, M, offsets, slot, ws, stream=None):
    """ids i32 or i64 [T][k] -> offsets i32 [E+1] and slot i32 [T][k] of the
    assignments to experts first .. first + E - 1; ws uint8
    [>= fp8bs_moe_sort_ws(T, k, E)] (or None where that is 0)."""
    _check_apart(ids, offsets, slot, ws)
    _moe_sort(ids, first, M, offsets, slot, ws, stream)


def _moe_sort(ids, first, M, offsets, slot, ws, stream):
    it, ldi, T, k, E = _check_ids(ids, offsets, slot)
    _here(ids, offsets, slot, ws)
    _call("fp8bs_moe_sort", _ptr(ids), it, ldi, T, k, first, E, M, _ptr(offsets), _ptr(slot), _ptr(ws), _workspace(ws),
          _stream(stream))


def _check_source(src, x, s_in):
    """(T, C) of rows given as codes with scales or in BF16."""
    codes = int(src) == SRC_FP8_1x128
    _check(x, "x", (None, None), _CODES if codes else ("bfloat16",))
    if codes:
        _check(s_in, "s_in", (x.shape[0], (">=", _groups(x.shape[1]))), ("float32",))
    return x.shape


def fp8bs_moe_gather(src, x, s_in, slot, q, s, y, stream=None):
    """Token t's row of x (bf16 [T][C], or codes with s_in f32 [T][C/128]) to the
    rows slot i32 [T][k] of q u8 [M][C] with s f32 [M][C/128] and/or y bf16 [M][C]."""
    T, C = _check_source(src, x, s_in)
    _check(slot, "slot", (T, None), ("int32",), contiguous=True)
    M = _row_count(q, s, y, C)
    _here(x, s_in, slot, q, s, y)
    _call("fp8bs_moe_gather", int(src), _ptr(x), _row_ld(x, C), _ptr(s_in), _row_ld(s_in, _groups(C)), T, C,
          _ptr(slot), slot.shape[1], _ptr(q), _row_ld(q, C), _ptr(s), _row_ld(s, _groups(C)), _ptr(y),
          _row_ld(y, C), M, _stream(stream))


def fp8bs_moe_dispatch(src, x, s_in, ids, first, offsets, slot, q, s, y, ws, stream=None):
    """fp8bs_moe_sort of ids and fp8bs_moe_gather of x in one call."""
    _check_apart(ids, offsets, slot, ws)
    _moe_dispatch(src, x, s_in, ids, first, offsets, slot, q, s, y, ws, stream)


def _moe_dispatch(src, x, s_in, ids, first, offsets, slot, q, s, y, ws, stream):
    T, C = _check_source(src, x, s_in)
    it, ldi, n, k, E = _check_ids(ids, offsets, slot)
    if n != T:
        raise ValueError(f"ids: {n} tokens, x has {T}")
    M = _row_count(q, s, y, C)
    _here(x, s_in, ids, offsets, slot, q, s, y, ws)
    _call("fp8bs_moe_dispatch", int(src), _ptr(x), _row_ld(x, C), _ptr(s_in), _row_ld(s_in, _groups(C)), T, C, _ptr(ids),
          it, ldi, k, first, E, _ptr(offsets), _ptr(slot), _ptr(q), _row_ld(q, C), _ptr(s), _row_ld(s, _groups(C)),
          _ptr(y), _row_ld(y, C), M, _ptr(ws), _workspace(ws), _stream(stream))


def fp8bs_moe_combine(y, slot, w, add, out, stream=None):
    """out bf16 [T][N] = add (or None) + the sum of w (or 1) times rows slot
    i32 [T][k] of y bf16 or f32 [M][N]; w f32 [T][k] or None."""
    _check(y, "y", (None, None), ("bfloat16", "float32"))
    M, N = y.shape
    _check(slot, "slot", (None, None), ("int32",), contiguous=True)
    T, k = slot.shape
    _optional(w, "w", (T, k), ("float32",))
    _optional(add, "add", (T, N), ("bfloat16",))
    _check(out, "out", (T, N), ("bfloat16",))
    _here(y, slot, w, add, out)
    _call("fp8bs_moe_combine", _ptr(y), _dtype(y, "y"), _row_ld(y, N), M, _ptr(slot), _ptr(w), _row_ld(w, k), T, k, N,
          _ptr(add), _row_ld(add, N), _ptr(out), _row_ld(out, N), _stream(stream))


def fp8bs_moe_combine_bwd(dout, y, slot, w, q, s, dy, dw, stream=None):
    """Gradient of fp8bs_moe_combine: dout bf16 [T][N], w f32 [T][k] -> rows slot
    of q u8 [M][N] with s f32 [M][N/128] and/or dy bf16 [M][N], and dw f32 [T][k]
    (or None; with it y [M][N])."""
    _check(dout, "dout", (None, None), ("bfloat16",))
    T, N = dout.shape
    _check(slot, "slot", (T, None), ("int32",), contiguous=True)
    k = slot.shape[1]
    _check(w, "w", (T, k), ("float32",))
    if dw is not None:
        _check(dw, "dw", (T, k), ("float32",))
        _check(y, "y", (None, N), ("bfloat16", "float32"))
    elif q is None and dy is None:
        raise ValueError("no output")
    M = _check_rows(q, s, dy, N, None if q is not None or dy is not None else y.shape[0])
    if dw is not None and y.shape[0] != M:
        raise ValueError(f"y: {y.shape[0]} rows, the outputs have {M}")
    _here(dout, y, slot, w, q, s, dy, dw)
    _call("fp8bs_moe_combine_bwd", _ptr(dout), _row_ld(dout, N), _ptr(y), OUT_BF16 if y is None else _dtype(y, "y"),
          _row_ld(y, N), _ptr(slot), _ptr(w), _row_ld(w, k), T, k, N, _ptr(q), _row_ld(q, N), _ptr(s),
          _row_ld(s, _groups(N)), _ptr(dy), _row_ld(dy, N), M, _ptr(dw), _row_ld(dw, k), _stream(stream))


def fp8bs_swiglu_bwd_quant_1x128(dh, g, u, q, s, d, h, stream=None):
    """Gradient of h = silu(g) u: dh, g, u bf16 [T][I] -> dg and du side by side as
    q u8 [T][2I] with s f32 [T][2I/128] and/or d bf16 [T][2I], and h bf16 [T][I] (or None)."""
    _check(g, "g", (None, None), ("bfloat16",))
    T, I = g.shape
    _check(dh, "dh", (T, I), ("bfloat16",))
    _check(u, "u", (T, I), ("bfloat16",))
    _check_rows(q, s, d, 2 * I, T)
    _optional(h, "h", (T, I), ("bfloat16",))
    if q is None and d is None and h is None:
        raise ValueError("no output")
    _here(dh, g, u, q, s, d, h)
    _call("fp8bs_swiglu_bwd_quant_1x128", _ptr(dh), _row_ld(dh, I), _ptr(g), _row_ld(g, I), _ptr(u), _row_ld(u, I), T, I,
          _ptr(q), _row_ld(q, 2 * I), _ptr(s), _row_ld(s, _groups(2 * I)), _ptr(d), _row_ld(d, 2 * I), _ptr(h),
          _row_ld(h, I), _stream(stream))


# ---------------------------------------------------------------------------
# allocating helpers (torch tensors on the current device)
# ---------------------------------------------------------------------------

def quant_act_1x128(x, stream=None):
    import torch
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    s = torch.empty((M, K // 128), dtype=torch.float32, device=x.device)
    fp8bs_quant_act_1x128(x, q, s, stream)
    return q, s


def quant_w_128x128(w, stream=None):
    import torch
    N, K = w.shape
    q = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    s = torch.empty(((N + 127) // 128, K // 128), dtype=torch.float32, device=w.device)
    fp8bs_quant_w_128x128(w, q, s, stream)
    return q, s


def fp8bs_quant_act_w(x, qx, sx, w, qw, sw, stream=None):
    """x bf16 [M][K] -> qx, sx (1x128 tiles) and w bf16 [N][K] -> qw, sw
    (128x128 blocks), in one launch."""
    M, K = x.shape
    N = w.shape[0]
    _check(x, "x", (M, K), ("bfloat16",))
    _check(qx, "qx", (M, K), _CODES)
    _check(sx, "sx", (M, (">=", _groups(K))), ("float32",))
    _check(w, "w", (N, K), ("bfloat16",))
    _check(qw, "qw", (N, K), _CODES)
    _check(sw, "sw", ((N + 127) // 128, (">=", _groups(K))), ("float32",))
    _call("fp8bs_quant_act_w", _ptr(x), M, _ld(x), _ptr(qx), _ld(qx), _ptr(sx), _ld(sx),
          _ptr(w), N, _ld(w), _ptr(qw), _ld(qw), _ptr(sw), _ld(sw), K, _stream(stream))


def fp8bs_swiglu_quant_1x128(g, u, q, s, h, stream=None):
    """h = silu(g) u of bf16 [T][I] halves -> q u8 [T][I] + s f32 [T][I/128]
    (1x128 tiles; both or neither) and/or h bf16 [T][I]."""
    T, I = g.shape
    _check(g, "g", (T, I), ("bfloat16",))
    _check(u, "u", (T, I), ("bfloat16",))
    if (q is None) != (s is None):
        raise ValueError("q and s: both or neither")
    if q is None and h is None:
        raise ValueError("no output")
    if q is not None:
        _check(q, "q", (T, I), _CODES)
        _check(s, "s", (T, (">=", _groups(I))), ("float32",))
    if h is not None:
        _check(h, "h", (T, I), ("bfloat16",))
    _call("fp8bs_swiglu_quant_1x128", _ptr(g), _ld(g), _ptr(u), _ld(u), T, I, _ptr(q),
          _ld(q) if q is not None else 0, _ptr(s), _ld(s) if s is not None else 0, _ptr(h),
          _ld(h) if h is not None else 0, _stream(stream))


def swiglu_quant_1x128(g, u, with_h=False, stream=None):
    import torch
    T, I = g.shape
    q = torch.empty((T, I), dtype=torch.uint8, device=g.device)
    s = torch.empty((T, I // 128), dtype=torch.float32, device=g.device)
    h = torch.empty((T, I), dtype=torch.bfloat16, device=g.device) if with_h else None
    fp8bs_swiglu_quant_1x128(g, u, q, s, h, stream)
    return (q, s, h) if with_h else (q, s)


def quant_act_w(x, w, stream=None):
    import torch
    M, K = x.shape
    N = w.shape[0]
    qx = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    sx = torch.empty((M, K // 128), dtype=torch.float32, device=x.device)
    qw = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    sw = torch.empty(((N + 127) // 128, K // 128), dtype=torch.float32, device=w.device)
    fp8bs_quant_act_w(x, qx, sx, w, qw, sw, stream)
    return qx, sx, qw, sw


def quant_per_tensor(x, stream=None):
    import torch
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    s = torch.empty((1,), dtype=torch.float32, device=x.device)
    fp8bs_quant_per_tensor(x, q, s, stream)
    return q, s


def encode_e5m6(x, stream=None):
    import torch
    T, C = x.shape
    y = torch.empty((T, C // 2 * 3), dtype=torch.uint8, device=x.device)
    fp8bs_encode_e5m6(x, y, stream)
    return y


def decode_e5m6(y, C, stream=None):
    import torch
    x = torch.empty((y.shape[0], C), dtype=torch.bfloat16, device=y.device)
    fp8bs_decode_e5m6(y, x, stream)
    return x


def requant_T_128x1(x, s_in=None, stream=None):
    """FP8 source when s_in is given (x u8 codes), bf16 source otherwise."""
    import torch
    T, C = x.shape
    Tp = (T + 15) // 16 * 16  # 16-byte aligned output rows
    q = torch.empty((C, Tp), dtype=torch.uint8, device=x.device)[:, :T]
    s = torch.empty((C, (T + 127) // 128), dtype=torch.float32, device=x.device)
    src = SRC_FP8_1x128 if s_in is not None else SRC_BF16
    fp8bs_requant_T_128x1(src, x, s_in, q, s, stream)
    return q, s


def requant_T_128x1_e5m6(y, C, stream=None):
    """Packed E5M6 rows y u8 [T][1.5 C] -> (q [C][T], s [C][ceil(T/128)])."""
    import torch
    T = y.shape[0]
    Tp = (T + 15) // 16 * 16  # 16-byte aligned output rows
    q = torch.empty((C, Tp), dtype=torch.uint8, device=y.device)[:, :T]
    s = torch.empty((C, (T + 127) // 128), dtype=torch.float32, device=y.device)
    fp8bs_requant_T_128x1(SRC_E5M6, y, None, q, s, stream)
    return q, s


def transpose_w_128x128(q, s, stream=None):
    import torch
    N, K = q.shape
    qt = torch.empty((K, N), dtype=torch.uint8, device=q.device)
    st = torch.empty((K // 128, N // 128), dtype=torch.float32, device=q.device)
    fp8bs_transpose_w_128x128(q, s, qt, st, stream)
    return qt, st


def gemm(a, sa, b, sb, bmode=BSCALE_BLOCK_128x128, out_f32=False, stream=None):
    import torch
    M, N = a.shape[0], b.shape[0]
    d = torch.empty((M, N), dtype=torch.float32 if out_f32 else torch.bfloat16, device=a.device)
    fp8bs_gemm(a, sa, b, sb, bmode, d, OUT_F32 if out_f32 else OUT_BF16, stream)
    return d


def gemm_quant_1x128(a, sa, b, sb, bmode=BSCALE_BLOCK_128x128, stream=None):
    import torch
    M, N = a.shape[0], b.shape[0]
    q = torch.empty((M, N), dtype=torch.uint8, device=a.device)
    s = torch.empty((M, N // 128), dtype=torch.float32, device=a.device)
    fp8bs_gemm_quant_1x128(a, sa, b, sb, bmode, q, s, stream)
    return q, s


def gemm_bf16a(x, b, sb, out_f32=False, with_codes=False, stream=None):
    import torch
    M, K = x.shape
    N = b.shape[0]
    d = torch.empty((M, N), dtype=torch.float32 if out_f32 else torch.bfloat16, device=x.device)
    qx = sx = None
    if with_codes:
        qx = torch.empty((M, K), dtype=torch.uint8, device=x.device)
        sx = torch.empty((M, K // 128), dtype=torch.float32, device=x.device)
    fp8bs_gemm_bf16a(x, qx, sx, b, sb, d, OUT_F32 if out_f32 else OUT_BF16, stream)
    return (d, qx, sx) if with_codes else d


def grouped_gemm(a, sa, b, sb, offsets, out_f32=False, stream=None):
    import torch
    M, N = a.shape[0], b.shape[1]
    d = torch.empty((M, N), dtype=torch.float32 if out_f32 else torch.bfloat16, device=a.device)
    fp8bs_grouped_gemm(a, sa, b, sb, offsets, d, OUT_F32 if out_f32 else OUT_BF16, stream)
    return d


def rope_table(n_pos, rot, base=10000.0, factor=1.0, orig_len=0, turns_lo=1.0, turns_hi=32.0, mscale=1.0,
               device="cuda", stream=None):
    """Angles of positions 0 .. n_pos-1 for heads with `rot` rotated dims:
    factor stretches positions (orig_len = 0) or, with orig_len the trained
    length, only the slow pairs (by parts)."""
    import torch
    cs = torch.empty((n_pos, rot), dtype=torch.float32, device=device)
    fp8bs_rope_table(cs, base, factor, orig_len, turns_lo, turns_hi, mscale, stream)
    return cs


def rope(x, pos, cs, rot_offset=0, layout="half", inverse=False, stream=None):
    """x bf16 [T][H][D] rotated.  Not recorded by autograd: y is detached, and the
    gradient of x is rope(dy, ..., inverse=True)."""
    y = _short("fp8bs_rope", x, pos, cs, rot_offset, _layout(layout), bool(inverse), _stream_later(stream))
    if y is not None:
        return y
    import torch
    y = torch.empty_like(x)
    fp8bs_rope(x, y, pos, rot_offset, layout, inverse, cs, stream)
    return y


def paged_cache(n_pages, heads, page, dim, device="cuda"):
    """An empty cache: (kc, ks, vc, vs) for n_pages pages of `page` tokens."""
    import torch
    kc = torch.zeros((n_pages, heads, page, dim), dtype=torch.uint8, device=device)
    ks = torch.zeros((n_pages, heads), dtype=torch.float32, device=device)
    return kc, ks, torch.zeros_like(kc), torch.zeros_like(ks)


def kv_append(k, v, kc, ks, vc, vs, table, kv_len, q_off, max_q, q=None, cs=None, rot_offset=0, layout="half",
              stream=None):
    """Appends k, v [T][Hkv][D] to the cache (keys rotated when cs is given);
    returns the rotated queries when q is given."""
    if q is not None and cs is not None:
        q_out = _short("fp8bs_kv_append", kc, ks, vc, vs, table, kv_len, q_off, k, v, q, cs, rot_offset, _layout(layout),
                       max_q, _stream_later(stream))
        if q_out is not None:
            return q_out
    import torch
    q_out = None if q is None else torch.empty_like(q)
    fp8bs_kv_append(q, q_out, k, v, cs, rot_offset, layout, q_off, kv_len, max_q, table, kc, ks, vc, vs, stream)
    return q_out


def _scratch(nbytes, device, stream):
    """Working memory that belongs to the given stream, so that it is not
    handed out again before that stream is done with it."""
    import torch
    on = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    with torch.cuda.stream(on):
        return torch.empty((nbytes,), dtype=torch.uint8, device=device)


def attn_paged(q, kc, ks, vc, vs, table, kv_len, q_off=None, max_q=1, scale=None, causal=True, window=0,
               with_lse=False, ws=None, stream=None):
    """Attention of q bf16 [T][Hq][D] over the cache; scale None: D^-1/2.
    The working memory is allocated unless given.  A table no wider than the longest
    context needs, and single tokens in a call of their own, are faster."""
    if ws is None and stream is None and not with_lse:
        out = _short("fp8bs_attn_paged", kc, ks, vc, vs, table, kv_len, q_off, _address("fp8bs_attn_paged_ws"), q, max_q,
                     scale, bool(causal), window, _current_stream)
        if out is not None:
            return out
    import torch
    T, Hq, D = q.shape
    out = torch.empty_like(q)
    lse = ks.new_empty((T, Hq)) if with_lse else None
    if ws is None:
        B, max_pages = table.shape
        _, Hkv, page, _ = kc.shape
        need = _ws_bytes(B, T, max_q, Hq, Hkv, D, max_pages, page)
        if need > 0:
            ws = ks.new_empty(need // 4) if stream is None else _scratch(need, q.device, stream)
    fp8bs_attn_paged(q, out, lse, q_off, kv_len, max_q, table, kc, ks, vc, vs,
                     D ** -0.5 if scale is None else scale, causal, window, ws, stream)
    return (out, lse) if with_lse else out


def _code_rows(rows, C, device):
    import torch
    return (torch.empty((rows, C), dtype=torch.uint8, device=device),
            torch.empty((rows, _groups(C)), dtype=torch.float32, device=device))


def _ws(nbytes, device, stream):
    """Working memory of the given stream, or None where none is needed."""
    import torch
    if nbytes <= 0:
        return None
    if stream is None:
        return torch.empty((nbytes,), dtype=torch.uint8, device=device)
    return _scratch(nbytes, device, stream)


def rmsnorm_quant_1x128(x, gamma, residual=None, eps=1e-6, codes=True, with_y=False, with_rstd=False, stream=None):
    """Root-mean-square norm of x bf16 [T][C] (plus a residual) times gamma:
    (q, s, h, y, rstd), where codes q and scales s, the sum h, the norm y in
    BF16 and the row factors rstd are None unless asked for (h: without a
    residual).  Not recorded by autograd; the gradient is rmsnorm_bwd."""
    if stream is None:
        way = _ways.get("fp8bs_rmsnorm_quant_1x128") or _way("fp8bs_rmsnorm_quant_1x128")
        outputs = way(x, gamma, residual, eps, codes, with_y, with_rstd, None)
        if outputs.__class__ is tuple:
            return outputs
        if outputs is not None:
            raise Fp8bsError(outputs, "fp8bs_rmsnorm_quant_1x128")
    import torch
    T, C = x.shape
    q, s = _code_rows(T, C, x.device) if codes else (None, None)
    h = None if residual is None else torch.empty((T, C), dtype=torch.bfloat16, device=x.device)
    y = torch.empty((T, C), dtype=torch.bfloat16, device=x.device) if with_y else None
    rstd = torch.empty((T,), dtype=torch.float32, device=x.device) if with_rstd else None
    fp8bs_rmsnorm_quant_1x128(x, residual, gamma, eps, h, q, s, y, rstd, stream)
    return q, s, h, y, rstd


def rmsnorm_bwd(dn, h, gamma, rstd, dres=None, with_dgamma=True, stream=None):
    """Gradient of the norm of h (the x + residual that rmsnorm_quant_1x128
    gave, or x): (dx, dgamma), dx that of x and of the residual, dgamma f32
    or None.  dres: the gradient of h's other uses.  Not recorded by autograd."""
    if stream is None:
        way = _ways.get("fp8bs_rmsnorm_bwd") or _way("fp8bs_rmsnorm_bwd", "fp8bs_rmsnorm_bwd_ws")
        outputs = way(dn, h, gamma, rstd, dres, with_dgamma, None)
        if outputs.__class__ is tuple:
            return outputs
        if outputs is not None:
            raise Fp8bsError(outputs, "fp8bs_rmsnorm_bwd")
    import torch
    T, C = h.shape
    dx = torch.empty((T, C), dtype=torch.bfloat16, device=h.device)
    dgamma = torch.empty((C,), dtype=torch.float32, device=h.device) if with_dgamma else None
    ws = _ws(_norm_ws_bytes(T, C), h.device, stream) if with_dgamma else None
    fp8bs_rmsnorm_bwd(dn, dres, h, gamma, rstd, dx, dgamma, ws, stream)
    return dx, dgamma


def moe_sort(ids, E, first=0, rows=None, stream=None):
    """Assignments ids [T][k] (int32 or int64) to experts first .. first + E - 1
    sorted by expert: (offsets i32 [E+1], slot i32 [T][k]).  rows: how many
    the sorted arrays will hold (default T k)."""
    import torch
    T, k = ids.shape
    offsets = torch.empty((E + 1,), dtype=torch.int32, device=ids.device)
    slot = torch.empty((T, k), dtype=torch.int32, device=ids.device)
    _moe_sort(ids, first, T * k if rows is None else rows, offsets, slot,
              _ws(_sort_ws_bytes(T, k, E), ids.device, stream), stream)
    return offsets, slot


def _row_outputs(out, rows, C, codes, with_y, device):
    """(q, s, y): those given, or new ones."""
    import torch
    if out is not None:
        return out
    q, s = _code_rows(rows, C, device) if codes else (None, None)
    return q, s, torch.empty((rows, C), dtype=torch.bfloat16, device=device) if with_y else None


def moe_gather(x, slot, s_in=None, rows=None, codes=True, with_y=False, out=None, stream=None):
    """Tokens' rows (bf16, or codes x with scales s_in) to their places: (q, s, y)
    with codes and scales, and BF16 rows where asked for (None otherwise).  out:
    such a triple to write into; rows that no slot names are not written.  Not
    recorded by autograd; the gradient is moe_combine without weights."""
    T, C = x.shape
    q, s, y = _row_outputs(out, slot.numel() if rows is None else rows, C, codes, with_y, x.device)
    fp8bs_moe_gather(SRC_BF16 if s_in is None else SRC_FP8_1x128, x, s_in, slot, q, s, y, stream)
    return q, s, y


def moe_dispatch(x, ids, E, first=0, s_in=None, rows=None, codes=True, with_y=False, out=None, stream=None):
    """moe_sort and moe_gather in one call: (q, s, y, offsets, slot).  Not recorded by
    autograd; the gradient of x is moe_combine without weights."""
    if stream is None:
        way = _ways.get("fp8bs_moe_dispatch") or _way("fp8bs_moe_dispatch", "fp8bs_moe_sort_ws")
        outputs = way(x, s_in, ids, E, first, rows, codes, with_y, out, None)
        if outputs.__class__ is tuple:
            return outputs
        if outputs is not None:
            raise Fp8bsError(outputs, "fp8bs_moe_dispatch")
    import torch
    (T, C), k = x.shape, ids.shape[1]
    q, s, y = _row_outputs(out, T * k if rows is None else rows, C, codes, with_y, x.device)
    offsets = torch.empty((E + 1,), dtype=torch.int32, device=x.device)
    slot = torch.empty((T, k), dtype=torch.int32, device=x.device)
    _moe_dispatch(SRC_BF16 if s_in is None else SRC_FP8_1x128, x, s_in, ids, first, offsets, slot, q, s, y,
                  _ws(_sort_ws_bytes(T, k, E), x.device, stream), stream)
    return q, s, y, offsets, slot


def moe_combine(y, slot, w=None, add=None, stream=None):
    """Rows of y (bf16 or f32) back to their tokens, weighted by w f32 [T][k] (or
    summed plainly: the gradient of moe_gather), onto add.  Not recorded by
    autograd; the gradient is moe_combine_bwd (add's is the output's)."""
    if stream is None:
        way = _ways.get("fp8bs_moe_combine") or _way("fp8bs_moe_combine")
        out = way(y, slot, w, add, None)
        if out.__class__ is int:
            raise Fp8bsError(out, "fp8bs_moe_combine")
        if out is not None:
            return out
    import torch
    out = torch.empty((slot.shape[0], y.shape[1]), dtype=torch.bfloat16, device=y.device)
    fp8bs_moe_combine(y, slot, w, add, out, stream)
    return out


def moe_combine_bwd(dout, slot, w, y=None, rows=None, codes=True, with_dy=False, out=None, stream=None):
    """Gradient of moe_combine: (q, s, dy, dw), the rows' gradient as codes with
    scales and in BF16 where asked for, and the weights' (with y) or None.  out:
    (q, s, dy) to write into; rows that no slot names are not written.  Not recorded
    by autograd."""
    if stream is None:
        way = _ways.get("fp8bs_moe_combine_bwd") or _way("fp8bs_moe_combine_bwd")
        outputs = way(dout, slot, w, y, rows, codes, with_dy, out, None)
        if outputs.__class__ is tuple:
            return outputs
        if outputs is not None:
            raise Fp8bsError(outputs, "fp8bs_moe_combine_bwd")
    import torch
    if rows is None:
        rows = slot.numel() if y is None else y.shape[0]
    q, s, dy = _row_outputs(out, rows, dout.shape[1], codes, with_dy, dout.device)
    dw = None if y is None else torch.empty(slot.shape, dtype=torch.float32, device=dout.device)
    fp8bs_moe_combine_bwd(dout, y, slot, w, q, s, dy, dw, stream)
    return q, s, dy, dw


def swiglu_bwd_quant_1x128(dh, g, u, codes=True, with_d=False, with_h=False, stream=None):
    """Gradient of h = silu(g) u: (q, s, d, h), the gradients of g and u side by
    side [T][2I] as codes with scales and in BF16, and h itself, where asked for
    (None otherwise).  Not recorded by autograd."""
    if stream is None:
        way = _ways.get("fp8bs_swiglu_bwd_quant_1x128") or _way("fp8bs_swiglu_bwd_quant_1x128")
        outputs = way(dh, g, u, codes, with_d, with_h, None)
        if outputs.__class__ is tuple:
            return outputs
        if outputs is not None:
            raise Fp8bsError(outputs, "fp8bs_swiglu_bwd_quant_1x128")
    import torch
    T, I = g.shape
    q, s = _code_rows(T, 2 * I, g.device) if codes else (None, None)
    d = torch.empty((T, 2 * I), dtype=torch.bfloat16, device=g.device) if with_d else None
    h = torch.empty((T, I), dtype=torch.bfloat16, device=g.device) if with_h else None
    fp8bs_swiglu_bwd_quant_1x128(dh, g, u, q, s, d, h, stream)
    return q, s, d, h
