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
# the compiled short way into the attention operators, of this Python
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

ENTRY_POINTS = ("fp8bs_quant_act_1x128", "fp8bs_quant_w_128x128", "fp8bs_quant_act_w",
                "fp8bs_swiglu_quant_1x128",
                "fp8bs_quant_per_tensor",
                "fp8bs_cast_e4m3",
                "fp8bs_encode_e5m6", "fp8bs_decode_e5m6", "fp8bs_requant_T_128x1",
                "fp8bs_transpose_w_128x128", "fp8bs_gemm", "fp8bs_gemm_quant_1x128", "fp8bs_gemm_bf16a",
                "fp8bs_grouped_gemm",
                "fp8bs_rope_table", "fp8bs_rope", "fp8bs_kv_append", "fp8bs_attn_paged",
                "fp8bs_attn_paged_ws",
                "fp8bs_status_string", "fp8bs_version")

_lib = None
_lib_path = LIB_PATH
_functions = {}      # the loaded library's entry points by name
_addresses = {}      # and their addresses
_marshal = None      # the compiled short way into the attention operators


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
    _ws_bytes.cache_clear()
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
    }
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.fp8bs_attn_paged_ws.argtypes = [I64] * 8
    lib.fp8bs_attn_paged_ws.restype = I64
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
        return {"fp8bs_" + f: getattr(module, f) for f in ("rope", "kv_append", "attn_paged")}
    except (ImportError, AttributeError) as e:
        import warnings
        warnings.warn(f"{MARSHAL_PATH}: {e}; the attention helpers go through ctypes")
        return {}


def _short(name, *args):
    """The named attention operator by the compiled short way (csrc/marshal.cpp): its
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
