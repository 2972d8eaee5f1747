"""ctypes binding of the C ABI in include/moe.h (same names, argument
marshalling only: every step runs in the HIP library).

Tensors are torch tensors on the GPU (device pointers are taken with
``data_ptr()``); streams default to torch's current stream. A non-zero status
raises ``MoEError`` carrying the library's message.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_gfx950.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_CAPACITY = -2
MOE_ERR_SLOT_STATE = -3
MOE_ERR_WORKSPACE = -4
MOE_ERR_HIP = -5
MOE_ERR_UNSUPPORTED = -6
MOE_DT_F32 = 0
MOE_DT_BF16 = 1
MOE_DT_BF16_FP8W = 2   # bf16 activations, fp8 e4m3 weights with fp32 row scales
MOE_DT_BF16_FP4W = 3   # bf16 activations, MXFP4 weights (E2M1 codes, E8M0 scale per 32)
_DTYPE_CODE = {"f32": MOE_DT_F32, "bf16": MOE_DT_BF16, "bf16_fp8w": MOE_DT_BF16_FP8W,
               "bf16_fp4w": MOE_DT_BF16_FP4W, MOE_DT_F32: MOE_DT_F32, MOE_DT_BF16: MOE_DT_BF16,
               MOE_DT_BF16_FP8W: MOE_DT_BF16_FP8W, MOE_DT_BF16_FP4W: MOE_DT_BF16_FP4W}


def fp4_slice_bytes(N: int, K: int) -> int:
    """Bytes of a packed MXFP4 slice [N][K]: per 256-row block and 32-wide K
    piece, 16 code bytes a row plus the rows' scale bytes padded to 16."""
    piece = lambda rows: rows * 16 + (rows + 15) // 16 * 16
    full, rem = divmod(N, 256)
    return (K // 32) * (full * piece(256) + (piece(rem) if rem else 0))


def fp8_scale_bytes(K: int) -> int:
    """Bytes between the scale rows of rows of K values quantised to fp8: one
    for each 128, in whole 16-byte pieces."""
    return (K + 2047) // 2048 * 16


MOE_DEVERR_EXPERT_ID = 1
MOE_ROUTE_RESET = 1
MOE_FFN_EXPERTS = 1
MOE_FFN_FINALIZE = 2
MOE_FFN_SIMPLE_KERNEL = 4
MOE_FFN_FUSED = 8
MOE_FFN_ACT_MXFP4 = 16
MOE_SLOT_AVAILABLE, MOE_SLOT_FILLING, MOE_SLOT_READY, MOE_SLOT_IN_USE = 0, 1, 2, 3
MOE_MAX_EXPERTS = 512
MOE_DECODE_MAX_T = 64
MOE_DECODE_MAX_ROUTES = 1024
MOE_DECODE_MAX_D = 131072
MOE_FP8_MAX_K = 1048576
MOE_COMBINE_MAX_D = 1048576


class MoEError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"moe status {status}: {msg}")
        self.status = status


class moe_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("f", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("P", ctypes.c_int32), ("capacity", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ldy", ctypes.c_int64)]


class moe_routes(ctypes.Structure):
    _fields_ = [("topk_idx", ctypes.c_void_p), ("topk_w", ctypes.c_void_p),
                ("slot_count", ctypes.c_void_p), ("slot_offset", ctypes.c_void_p),
                ("rec_token", ctypes.c_void_p), ("rec_route", ctypes.c_void_p),
                ("route_pos", ctypes.c_void_p)]


_lib = None

_VP, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_SIGS = {
    "moe_version": ([], ctypes.c_char_p),
    "moe_last_error": ([ctypes.c_char_p, _SZ], _I32),
    "moe_workspace_bytes": ([_VP], _SZ),
    "moe_workspace_init": ([_VP, _VP, _SZ, _VP], _I32),
    "moe_device_errors": ([_VP, _VP, _SZ, _VP, _VP], _I32),
    "moe_router_logits": ([_VP, _VP, _VP, _VP, _VP, _VP], _I32),
    "moe_route_build": ([_VP, _I32, _I32, _VP, _VP, _I32, _VP, _VP, _SZ, _VP], _I32),
    "moe_expert_ffn": ([_VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, _SZ, _VP], _I32),
    "moe_layer_prefill": ([_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP, _VP], _I32),
    "moe_layer_prefill_noalloc": ([_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP], _I32),
    "moe_quantize_mxfp4": ([_VP, _I32, _I64, _I32, _I64, _VP, _VP, _VP], _I32),
    "moe_dequantize_mxfp4": ([_VP, _VP, _I64, _I32, _VP, _I32, _I64, _VP], _I32),
    "moe_matmul_mxfp4": ([_I32, _I32, _I32, _VP, _VP, _I32, _VP, _VP, _I32, _VP, _I64, _VP, _I32, _I64, _VP], _I32),
    "moe_quantize_fp8": ([_VP, _I32, _I64, _I32, _I64, _I32, _VP, _VP, _VP], _I32),
    "moe_dequantize_fp8": ([_VP, _VP, _I64, _I32, _I32, _VP, _I32, _I64, _VP], _I32),
    "moe_matmul_fp8": ([_I32, _I32, _I32, _VP, _VP, _I32, _VP, _VP, _I32, _VP, _VP, _I64, _I64, _VP, _I32, _I64, _VP], _I32),
    "moe_gate_up_fp8_workspace_bytes": ([_I32, _I32, _I32, _I32], _SZ),
    "moe_gate_up_fp8": ([_I32, _I32, _I32, _VP, _VP, _I32, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _I64, _I64, _VP, _VP, _VP,
                         _SZ, _VP], _I32),
    "moe_combine": ([_I32, _I32, _I32, _I32, _VP, _I32, _I64, _VP, _VP, _VP, _I64, _VP], _I32),
    "moe_combine_backward": ([_I32, _I32, _I32, _I32, _VP, _I32, _I64, _VP, _VP, _VP, _I64, _VP, _I64, _VP, _VP], _I32),
    "moe_balance_workspace_bytes": ([_VP, _I32], _SZ),
    "moe_balance_loss": ([_VP, _VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP], _I32),
    "moe_router_backward": ([_VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP], _I32),
    "moe_decode_workspace_bytes": ([_VP], _SZ),
    "moe_decode_workspace_init": ([_VP, _VP, _SZ, _VP], _I32),
    "moe_layer_decode": ([_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP], _I32),
    "moe_pack_gate_up": ([_VP, _VP, _VP, _VP, _I32, _I64, _I64, _VP], _I32),
    "moe_pack_gate_up_host": ([_VP, _VP, _VP, _VP], _I32),
    "moe_pack_down": ([_VP, _VP, _VP, _I32, _I64, _I64, _VP], _I32),
    "moe_pack_down_host": ([_VP, _VP, _VP], _I32),
    "moe_arena_create": ([_VP, _VP, _VP, _VP, _I64, _I64, _I32], _I32),
    "moe_arena_destroy": ([_VP], None),
    "arena_bind_slot": ([_VP, _I32, _I32, _VP, _VP, _VP], _I32),
    "arena_reserve_slot": ([_VP, _I32, _I32], _I32),
    "arena_publish_slot": ([_VP, _I32, _I32, _VP], _I32),
    "arena_release_slot": ([_VP, _I32], _I32),
    "arena_phi": ([_VP, _VP, _I32], _I32),
    "arena_slot_info": ([_VP, _I32, _VP, _VP], _I32),
    "moe_selftest_mfma_layout": ([_VP, _VP], _I32),
    "moe_profile_begin": ([_I32, _I32], _I32),
    "moe_profile_end": ([_I32, _VP, _I32, _VP], _I32),
}

MOE_KERNEL = {"router": 1, "topk": 2, "route_count": 3, "route_place": 4, "gate_up": 5, "down": 6,
              "combine": 7, "h2d": 8, "fused": 9}


def lib_path() -> str:
    return LIB_PATH


def load() -> ctypes.CDLL:
    """Load the HIP library, building it first only if it was never built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        from . import build as _build
        _build.build()
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"HIP library missing: {LIB_PATH} (run __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != MOE_OK:
        buf = ctypes.create_string_buffer(512)
        load().moe_last_error(buf, 512)
        raise MoEError(status, buf.value.decode())


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(s) -> Optional[int]:
    if s is None:
        if torch.cuda.is_initialized():   # the current stream without a Stream object: 0.3 us instead of 3.6
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _stream_of(t, s) -> Optional[int]:
    """_stream(s) for work on t, whose GPU has to be the current one: a launch
    goes to the current device, wherever its pointers lead."""
    if t is not None and not isinstance(t, int):
        if t.get_device() < 0:
            raise ValueError("the tensors must be on the GPU")
        here = torch.cuda.current_device()
        if t.get_device() != here or getattr(s, "device_index", here) != here:
            raise ValueError(f"the tensors and the stream must be on the current device, cuda:{here}")
        if s is None:
            return _raw_stream(here)
    return _stream(s)


def _stream_of_all(tensors, s) -> Optional[int]:
    """_stream_of for work on several tensors (handles and None pass), which have
    to be on one GPU."""
    first = dev = None
    for t in tensors:
        get_device = getattr(t, "get_device", None)
        if get_device is None:
            continue
        if first is None:
            first, dev = t, get_device()
        elif get_device() != dev:
            raise ValueError("the operands must be on one device")
    return _stream_of(first, s)


@contextlib.contextmanager
def on_stream(stream):
    """``stream`` (None: as it is) is torch's current stream within, behind what
    the current one holds so far: temporaries of calls on a stream come from its
    own pool, so that their memory is neither used by another stream's work
    before nor given to it while these calls are queued."""
    if stream is None:
        yield
        return
    if isinstance(stream, int):   # a handle; 0 and 1 (the legacy one) are the default stream's
        if stream == 2:           # this thread's: torch takes a handle for an address, and would use another stream
            raise ValueError("the per-thread stream has no torch stream: give one of torch's, or its handle")
        stream = torch.cuda.ExternalStream(stream) if stream > 2 else torch.cuda.default_stream()
    stream.wait_stream(torch.cuda.current_stream(stream.device))
    with torch.cuda.stream(stream):
        yield


def make_shape(T, d, f, E, k, n_shared=0, P=None, capacity=None, dtype="bf16", renorm=True,
               ldx=None, ldy=None) -> moe_shape:
    kp = k + n_shared
    return moe_shape(T=T, d=d, f=f, E=E, k=k, n_shared=n_shared,
                     P=(E + n_shared) if P is None else P,
                     capacity=max(1, T * kp) if capacity is None else capacity,
                     dtype=_DTYPE_CODE[dtype],
                     renorm=int(bool(renorm)), ldx=d if ldx is None else ldx,
                     ldy=d if ldy is None else ldy)


def routes_struct(r: dict) -> moe_routes:
    return moe_routes(*[_ptr(r.get(k)) for k in ("topk_idx", "topk_w", "slot_count", "slot_offset",
                                              "rec_token", "rec_route", "route_pos")])


# ----------------------------------------------------------------- calls --
def moe_version() -> str:
    return load().moe_version().decode()


def moe_last_error():
    buf = ctypes.create_string_buffer(512)
    st = load().moe_last_error(buf, 512)
    return st, buf.value.decode()


def moe_workspace_bytes(shape: moe_shape) -> int:
    return int(load().moe_workspace_bytes(ctypes.byref(shape)))


def moe_workspace_init(shape, ws, stream=None):
    _check(load().moe_workspace_init(ctypes.byref(shape), _ptr(ws), ws.numel() * ws.element_size(),
                                     _stream(stream)))


def moe_device_errors(shape, ws, stream=None) -> int:
    v = ctypes.c_int32(0)
    st = load().moe_device_errors(ctypes.byref(shape), _ptr(ws), ws.numel() * ws.element_size(),
                                  ctypes.byref(v), _stream(stream))
    if st not in (MOE_OK, MOE_ERR_INVALID_ARG):
        _check(st)
    return int(v.value)


def moe_router_logits(shape, X, W_r, bias, logits, stream=None):
    _check(load().moe_router_logits(ctypes.byref(shape), _ptr(X), _ptr(W_r), _ptr(bias),
                                    _ptr(logits), _stream(stream)))


def _phi_arr(phi):
    if phi is None:
        return None
    vals = [int(x) for x in phi]
    return (ctypes.c_int32 * len(vals))(*vals)


def moe_route_build(shape, t0, nt, logits, phi, flags, routes: dict, ws, stream=None):
    rs = routes_struct(routes)
    _check(load().moe_route_build(ctypes.byref(shape), t0, nt, _ptr(logits), _phi_arr(phi), flags,
                                  ctypes.byref(rs), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream)))


def moe_expert_ffn(shape, X, Y, routes: dict, arena, phi, flags, ws, stream=None):
    rs = routes_struct(routes)
    _check(load().moe_expert_ffn(ctypes.byref(shape), _ptr(X), _ptr(Y), ctypes.byref(rs),
                                 arena.handle if arena is not None else None, _phi_arr(phi), flags,
                                 _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_layer_prefill(shape, X, W_r, bias, logits, Y, arena, host_gu, host_d, routes: dict, ws,
                      compute=None, copy=None):
    rs = routes_struct(routes)
    gu = d = None
    if host_gu is not None:
        n = len(host_gu)
        gu = (ctypes.c_void_p * n)(*[_ptr(t) for t in host_gu])
        d = (ctypes.c_void_p * n)(*[_ptr(t) for t in host_d])
    _check(load().moe_layer_prefill(ctypes.byref(shape), _ptr(X), _ptr(W_r), _ptr(bias), _ptr(logits),
                                    _ptr(Y), arena.handle, gu, d, ctypes.byref(rs), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(compute),
                                    _stream(copy) if copy is not None else None))


def moe_layer_prefill_noalloc(shape, X, W_r, bias, logits, Y, arena, routes: dict, stream=None):
    rs = routes_struct(routes)
    _check(load().moe_layer_prefill_noalloc(ctypes.byref(shape), _ptr(X), _ptr(W_r), _ptr(bias), _ptr(logits),
                                            _ptr(Y), arena.handle, ctypes.byref(rs), _stream(stream)))


def moe_decode_workspace_bytes(shape: moe_shape) -> int:
    return int(load().moe_decode_workspace_bytes(ctypes.byref(shape)))


def moe_decode_workspace_init(shape, ws, stream=None):
    _check(load().moe_decode_workspace_init(ctypes.byref(shape), _ptr(ws), ws.numel() * ws.element_size(),
                                            _stream_of_all((ws,), stream)))


def moe_layer_decode(shape, X, W_r, bias, logits, Y, arena, routes: dict, ws, stream=None):
    rs = routes_struct(routes)
    st = _stream_of_all((X, W_r, bias, logits, Y, ws, routes.get("topk_idx"), routes.get("topk_w"),
                         getattr(arena, "plane_gu", None)), stream)
    _check(load().moe_layer_decode(ctypes.byref(shape), _ptr(X), _ptr(W_r), _ptr(bias), _ptr(logits), _ptr(Y),
                                   arena.handle, ctypes.byref(rs), _ptr(ws), ws.numel() * ws.element_size(), st))


_VAL_DTYPE = {torch.float32: MOE_DT_F32, torch.bfloat16: MOE_DT_BF16}


def _mx_views(values, codes, scales):
    """Type code, rows, K and row stride of [..., K] values and their blocks;
    leading dimensions that one row stride covers count as rows."""
    # one row's calls are as long as what the host does: each attribute is asked for once
    dtype = _VAL_DTYPE.get(values.dtype)
    if dtype is None:
        raise ValueError("values must be float32 or bfloat16")
    shape, n, dev = values.shape, values.numel(), values.get_device()
    K = shape[-1]
    if (codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8 or K % 32 or codes.numel() * 2 != n
            or scales.numel() * 32 != n or not codes.is_contiguous() or not scales.is_contiguous()):
        raise ValueError("need contiguous uint8 codes [rows][K/2] and scales [rows][K/32], K a multiple of 32")
    if codes.get_device() != dev or scales.get_device() != dev:
        raise ValueError("values, codes and scales must be on one device")
    if values.is_contiguous():
        ld = K
    elif len(shape) != 2:
        raise ValueError("values: only a matrix may have a row stride")
    else:
        ld, step = values.stride()
        if step != 1:
            raise ValueError("values: rows must be contiguous")
    return dtype, n // K if K else 0, K, ld


def moe_quantize_mxfp4(values, codes, scales, stream=None):
    dtype, rows, K, ld = _mx_views(values, codes, scales)
    _check(load().moe_quantize_mxfp4(values.data_ptr(), dtype, rows, K, ld, codes.data_ptr(), scales.data_ptr(),
                                     _stream_of(values, stream)))


def moe_dequantize_mxfp4(codes, scales, values, stream=None):
    dtype, rows, K, ld = _mx_views(values, codes, scales)
    _check(load().moe_dequantize_mxfp4(codes.data_ptr(), scales.data_ptr(), rows, K, values.data_ptr(), dtype, ld,
                                       _stream_of(values, stream)))


def moe_matmul_mxfp4(A_codes, A_scales, B, C, slot_offset=None, row_index=None, stream=None):
    """C [M][N] = rows of A times the packed slices B [P][bytes] (or one slice
    [bytes]); A_codes uint8 [A_rows][K/2], A_scales uint8 [A_rows][K/32]."""
    u8 = torch.uint8
    A_rows, half = A_codes.shape
    M, N = C.shape
    K = 2 * half
    dtype, dev = _VAL_DTYPE.get(C.dtype), C.get_device()
    b_shape, b_stride = B.shape, B.stride()
    P = 1 if len(b_shape) == 1 else b_shape[0]
    if A_codes.dtype is not u8 or A_scales.dtype is not u8 or B.dtype is not u8:
        raise ValueError("A_codes, A_scales and B must be uint8")
    if not A_codes.is_contiguous() or not A_scales.is_contiguous() or A_scales.shape != (A_rows, K // 32):
        raise ValueError("A_codes [A_rows][K/2] and A_scales [A_rows][K/32] must be contiguous")
    ldc, step = C.stride()
    if M <= 1:
        ldc = (N + 7) // 8 * 8   # one row: any aligned stride does
    if dtype is None or (step != 1 and N > 1) or ldc < N:
        raise ValueError("C must be float32 or bfloat16 with contiguous rows")
    if b_shape[-1] < fp4_slice_bytes(N, K) or b_stride[-1] != 1:
        raise ValueError("B: a slice is smaller than [N][K]")
    if A_codes.get_device() != dev or A_scales.get_device() != dev or B.get_device() != dev:
        raise ValueError("the operands must be on one device")
    for t, n, name in ((slot_offset, P + 1, "slot_offset"), (row_index, M, "row_index")):
        if t is not None and (t.dtype != torch.int32 or t.numel() < n or not t.is_contiguous() or t.get_device() != dev):
            raise ValueError(f"{name}: need int32 [{n}]")
    _check(load().moe_matmul_mxfp4(M, N, K, A_codes.data_ptr(), A_scales.data_ptr(), A_rows, _ptr(row_index),
                                   _ptr(slot_offset), P, B.data_ptr(), b_stride[0] if len(b_shape) > 1 else b_shape[0],
                                   C.data_ptr(), dtype, ldc, _stream_of(C, stream)))


def _fp8_views(values, codes, scales, block_rows):
    """Type code, rows, K and row stride of [..., K] values and their fp8
    blocks; leading dimensions that one row stride covers count as rows."""
    dtype = _VAL_DTYPE.get(values.dtype)
    if dtype is None:
        raise ValueError("values must be float32 or bfloat16")
    shape, n, dev = values.shape, values.numel(), values.get_device()
    K = shape[-1]
    rows = n // K if K else 0
    if codes.dtype is not torch.uint8 or codes.numel() != n or not codes.is_contiguous():
        raise ValueError("need contiguous uint8 codes [rows][K]")
    if block_rows == 1:
        if scales.dtype is not torch.uint8 or scales.numel() != rows * fp8_scale_bytes(K) or not scales.is_contiguous():
            raise ValueError("need contiguous uint8 scales [rows][fp8_scale_bytes(K)]")
    elif (scales.dtype is not torch.float32 or scales.numel() != -(-rows // 128) * -(-K // 128)
          or not scales.is_contiguous()):
        raise ValueError("need contiguous float32 scales [ceil(rows / 128)][ceil(K / 128)]")
    if codes.get_device() != dev or scales.get_device() != dev:
        raise ValueError("values, codes and scales must be on one device")
    if values.is_contiguous():
        ld = K
    elif len(shape) != 2:
        raise ValueError("values: only a matrix may have a row stride")
    else:
        ld, step = values.stride()
        if step != 1:
            raise ValueError("values: rows must be contiguous")
        if rows == 1:
            ld = (K + 7) // 8 * 8   # one row: any aligned stride does
    return dtype, rows, K, ld


def moe_quantize_fp8(values, codes, scales, block_rows=1, stream=None):
    """block_rows 1: scales uint8 [rows][fp8_scale_bytes(K)]; 128: float32 [ceil(rows/128)][ceil(K/128)]."""
    dtype, rows, K, ld = _fp8_views(values, codes, scales, block_rows)
    _check(load().moe_quantize_fp8(values.data_ptr(), dtype, rows, K, ld, block_rows, codes.data_ptr(), scales.data_ptr(),
                                   _stream_of(values, stream)))


def moe_dequantize_fp8(codes, scales, values, block_rows=1, stream=None):
    dtype, rows, K, ld = _fp8_views(values, codes, scales, block_rows)
    _check(load().moe_dequantize_fp8(codes.data_ptr(), scales.data_ptr(), rows, K, block_rows, values.data_ptr(), dtype, ld,
                                     _stream_of(values, stream)))


def _fp8_rows(codes, scales, name):
    rows, K = codes.shape
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise ValueError(f"{name}: codes and scales must be uint8")
    if not codes.is_contiguous() or not scales.is_contiguous() or scales.numel() != rows * fp8_scale_bytes(K):
        raise ValueError(f"{name}: need contiguous codes [rows][K] and scales [rows][fp8_scale_bytes(K)]")
    return rows, K


def _fp8_slices(codes, scales, K, name):
    """P, N and the strides of weight slices [P][N][K] (or one [N][K]) with
    their scales; a slice is contiguous, its distance to the next free."""
    shape, stride = codes.shape, codes.stride()
    if len(shape) not in (2, 3) or codes.dtype is not torch.uint8 or shape[-1] != K or stride[-1] != 1 or stride[-2] != K:
        raise ValueError(f"{name}: need uint8 codes [P][N][{K}], a slice contiguous")
    N, KB, P = shape[-2], -(-K // 128), shape[0] if len(shape) == 3 else 1
    NB, s_stride = -(-N // 128), scales.stride()
    if (scales.dtype is not torch.float32 or scales.shape != ((P, NB, KB) if len(shape) == 3 else (NB, KB))
            or KB > 1 and s_stride[-1] != 1 or NB > 1 and s_stride[-2] != KB):
        raise ValueError(f"{name}: need float32 scales [P][ceil(N / 128)][ceil(K / 128)], a slice's contiguous")
    return P, N, stride[0] if P > 1 else N * K, s_stride[0] if P > 1 else 0


def _list_of(t, n, dev, name):
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.numel() < n or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: need int32 [{n}]")
    return t.data_ptr()


def _one_device(dev, *tensors):
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("the operands must be on one device")


def moe_matmul_fp8(A_codes, A_scales, B_codes, B_scales, C, slot_offset=None, row_index=None, stream=None):
    """C [M][N] = rows of A times the slices B_codes [P][N][K] (or one [N][K])
    with their scales; A_codes uint8 [A_rows][K]."""
    A_rows, K = _fp8_rows(A_codes, A_scales, "A")
    P, N, b_stride, s_stride = _fp8_slices(B_codes, B_scales, K, "B")
    M, dtype, dev = C.shape[0], _VAL_DTYPE.get(C.dtype), C.get_device()
    ldc, step = C.stride()
    if M <= 1:
        ldc = (N + 7) // 8 * 8   # one row: any aligned stride does
    if dtype is None or C.shape[1] != N or step != 1 or ldc < N:
        raise ValueError(f"C must be float32 or bfloat16 [M][{N}] with contiguous rows")
    _one_device(dev, A_codes, A_scales, B_codes, B_scales)
    take, offset = _list_of(row_index, M, dev, "row_index"), _list_of(slot_offset, P + 1, dev, "slot_offset")
    _check(load().moe_matmul_fp8(M, N, K, A_codes.data_ptr(), A_scales.data_ptr(), A_rows, take, offset, P, B_codes.data_ptr(), B_scales.data_ptr(), b_stride, s_stride,
                                 C.data_ptr(), dtype, ldc, _stream_of(C, stream)))


def moe_gate_up_fp8_workspace_bytes(M: int, f: int, K: int, P: int = 1) -> int:
    return load().moe_gate_up_fp8_workspace_bytes(M, f, K, P)


def moe_gate_up_fp8(A_codes, A_scales, Wg_codes, Wg_scales, Wu_codes, Wu_scales, H_codes, H_scales, slot_offset=None,
                    row_index=None, ws=None, stream=None):
    """H [M][f] = fp8 rows of SiLU(A Wg^T) * (A Wu^T); Wg_codes and Wu_codes
    uint8 [P][f][K] (or one [f][K]), of the same strides. ws: see
    ``moe_gate_up_fp8_workspace_bytes``; without it torch's allocator gives the
    call one of its own, on its stream."""
    A_rows, K = _fp8_rows(A_codes, A_scales, "A")
    M, f = _fp8_rows(H_codes, H_scales, "H")
    gate = _fp8_slices(Wg_codes, Wg_scales, K, "Wg")
    if gate[1] != f or gate != _fp8_slices(Wu_codes, Wu_scales, K, "Wu"):
        raise ValueError(f"Wg and Wu need the same shapes and strides, {f} rows a slice")
    P, _, w_stride, s_stride = gate
    dev = H_codes.get_device()
    _one_device(dev, A_codes, A_scales, Wg_codes, Wg_scales, Wu_codes, Wu_scales, H_scales)
    take, offset = _list_of(row_index, M, dev, "row_index"), _list_of(slot_offset, P + 1, dev, "slot_offset")
    st, n = _stream_of(H_codes, stream), 0
    if ws is not None:
        _one_device(dev, ws)
        n = ws.numel() * ws.element_size()
    else:
        n = load().moe_gate_up_fp8_workspace_bytes(M, f, K, P)
        if n and stream is None:
            ws = H_codes.new_empty(n)
        elif n:
            with on_stream(stream):   # its memory goes back to the pool of the stream that uses it
                ws = H_codes.new_empty(n)
    _check(load().moe_gate_up_fp8(M, f, K, A_codes.data_ptr(), A_scales.data_ptr(), A_rows, take, offset, P, Wg_codes.data_ptr(), Wg_scales.data_ptr(), Wu_codes.data_ptr(),
                                  Wu_scales.data_ptr(), w_stride, s_stride, H_codes.data_ptr(), H_scales.data_ptr(),
                                  _ptr(ws), n, st))


def _strided(t, name, cols):
    """Row stride of a matrix with contiguous rows that do not overlap."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[1] != cols:
        raise ValueError(f"{name}: need a matrix of {cols} columns")
    if cols > 1 and stride[1] != 1 or shape[0] > 1 and stride[0] < cols:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    return stride[0] if shape[0] > 1 else (cols + 7) // 8 * 8   # one row: any aligned stride does


def _combine_args(C, route_pos, topk_w, Y, name):
    T, d = Y.shape
    dtype, kp, dev = _VAL_DTYPE.get(C.dtype), topk_w.shape[-1], Y.get_device()
    if dtype is None or Y.dtype is not torch.float32:
        raise ValueError(f"C must be float32 or bfloat16 and {name} float32")
    ldc, ldy = _strided(C, "C", d), _strided(Y, name, d)
    if topk_w.dtype is not torch.float32 or topk_w.shape != (T, kp) or not topk_w.is_contiguous():
        raise ValueError(f"topk_w: need contiguous float32 [{T}][K']")
    if route_pos.dtype is not torch.int32 or route_pos.numel() != T * kp or not route_pos.is_contiguous():
        raise ValueError(f"route_pos: need contiguous int32 [{T * kp}]")
    if C.get_device() != dev or route_pos.get_device() != dev or topk_w.get_device() != dev:
        raise ValueError("the operands must be on one device")
    return T, d, kp, C.shape[0], C.data_ptr(), dtype, ldc, route_pos.data_ptr(), topk_w.data_ptr(), Y.data_ptr(), ldy


def moe_combine(C, route_pos, topk_w, Y, stream=None):
    """Y [T][d] += the rows of C [M][d] at route_pos [T*K'], times topk_w [T][K']."""
    _check(load().moe_combine(*_combine_args(C, route_pos, topk_w, Y, "Y"), _stream_of(Y, stream)))


def moe_combine_backward(C, route_pos, topk_w, dY, dC, d_topk_w, stream=None):
    """dC [M][d] (or None) and d_topk_w [T][K'] of moe_combine."""
    args = _combine_args(C, route_pos, topk_w, dY, "dY")
    lddc = 0
    if dC is not None:
        if dC.dtype is not C.dtype or dC.shape != C.shape:
            raise ValueError("dC: need C's shape and type")
        lddc = _strided(dC, "dC", args[1])
        _one_device(dY.get_device(), dC)
    if d_topk_w.dtype is not torch.float32 or d_topk_w.shape != topk_w.shape or not d_topk_w.is_contiguous():
        raise ValueError("d_topk_w: need topk_w's shape, contiguous float32")
    _one_device(dY.get_device(), d_topk_w)
    _check(load().moe_combine_backward(*args, _ptr(dC), lddc, d_topk_w.data_ptr(), _stream_of(dY, stream)))


def moe_balance_workspace_bytes(shape: moe_shape, S: int = 1) -> int:
    return int(load().moe_balance_workspace_bytes(ctypes.byref(shape), S))


def _whole(t, dtype, shape, name, dev):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: need contiguous {dtype} {list(shape)} on the operands' device")


def _sequences(shape, seq_offset, mask, dev):
    S = 1
    if seq_offset is not None:
        S = seq_offset.numel() - 1
        _whole(seq_offset, torch.int32, (S + 1,), "seq_offset", dev)
    if mask is not None:
        if mask.dtype not in (torch.uint8, torch.bool):
            raise ValueError("mask: need uint8 or bool")
        _whole(mask, mask.dtype, (shape.T,), "mask", dev)
    return S


def moe_balance_loss(shape, logits, topk_idx, loss, counts, prob, slope, ws, seq_offset=None, mask=None, stream=None):
    """loss [1], counts (int32), prob and slope [S][E] of the routing topk_idx
    [T][K'] of logits [T][E]; seq_offset int32 [S+1], mask uint8 or bool [T]."""
    dev, f32, i32 = logits.get_device(), torch.float32, torch.int32
    S = _sequences(shape, seq_offset, mask, dev)
    _whole(logits, f32, (shape.T, shape.E), "logits", dev)
    _whole(topk_idx, i32, (shape.T, shape.k + shape.n_shared), "topk_idx", dev)
    _whole(loss, f32, (1,), "loss", dev)
    for t, dt, name in ((counts, i32, "counts"), (prob, f32, "prob"), (slope, f32, "slope")):
        _whole(t, dt, (S, shape.E), name, dev)
    _one_device(dev, ws)
    _check(load().moe_balance_loss(ctypes.byref(shape), logits.data_ptr(), topk_idx.data_ptr(), _ptr(seq_offset), S,
                                   _ptr(mask), loss.data_ptr(), counts.data_ptr(), prob.data_ptr(), slope.data_ptr(),
                                   ws.data_ptr(), ws.numel() * ws.element_size(), _stream_of(logits, stream)))


def moe_router_backward(shape, logits, topk_idx, d_logits, slope=None, d_loss=None, d_topk_w=None, seq_offset=None,
                        mask=None, stream=None):
    """d_logits [T][E] of d_loss [1] (None: 1) times the balance loss whose
    slope is given, plus that of d_topk_w [T][K']."""
    dev, f32 = logits.get_device(), torch.float32
    S = _sequences(shape, seq_offset, mask, dev)
    kp = shape.k + shape.n_shared
    _whole(logits, f32, (shape.T, shape.E), "logits", dev)
    _whole(d_logits, f32, (shape.T, shape.E), "d_logits", dev)
    if topk_idx is not None:
        _whole(topk_idx, torch.int32, (shape.T, kp), "topk_idx", dev)
    for t, want, name in ((slope, (S, shape.E), "slope"), (d_loss, (1,), "d_loss"), (d_topk_w, (shape.T, kp), "d_topk_w")):
        if t is not None:
            _whole(t, f32, want, name, dev)
    _check(load().moe_router_backward(ctypes.byref(shape), logits.data_ptr(), _ptr(topk_idx), _ptr(slope), _ptr(d_loss),
                                      _ptr(seq_offset), S, _ptr(mask), _ptr(d_topk_w), d_logits.data_ptr(),
                                      _stream_of(logits, stream)))


def moe_pack_gate_up(shape, Wg, Wu, dst, n, src_stride, dst_stride, stream=None):
    _check(load().moe_pack_gate_up(ctypes.byref(shape), _ptr(Wg), _ptr(Wu), _ptr(dst), n,
                                   src_stride, dst_stride, _stream(stream)))


def moe_pack_gate_up_host(shape, Wg, Wu, dst):
    _check(load().moe_pack_gate_up_host(ctypes.byref(shape), _ptr(Wg), _ptr(Wu), _ptr(dst)))


def moe_pack_down(shape, Wd, dst, n, src_stride, dst_stride, stream=None):
    _check(load().moe_pack_down(ctypes.byref(shape), _ptr(Wd), _ptr(dst), n, src_stride, dst_stride,
                                _stream(stream)))


def moe_pack_down_host(shape, Wd, dst):
    _check(load().moe_pack_down_host(ctypes.byref(shape), _ptr(Wd), _ptr(dst)))


def moe_arena_create(shape, plane_gu, plane_d, stride_gu, stride_d, G) -> int:
    h = ctypes.c_void_p(0)
    _check(load().moe_arena_create(ctypes.byref(h), ctypes.byref(shape), _ptr(plane_gu), _ptr(plane_d),
                                   stride_gu, stride_d, G))
    return h.value


def moe_arena_destroy(handle) -> None:
    load().moe_arena_destroy(handle)


def arena_bind_slot(arena, slot, expert, src_gu, src_d, copy_stream=None):
    _check(load().arena_bind_slot(arena.handle, slot, expert, _ptr(src_gu), _ptr(src_d),
                                  _stream(copy_stream)))


def arena_reserve_slot(arena, slot, expert):
    _check(load().arena_reserve_slot(arena.handle, slot, expert))


def arena_publish_slot(arena, slot, expert, stream=None):
    _check(load().arena_publish_slot(arena.handle, slot, expert, _stream(stream)))


def arena_release_slot(arena, slot):
    _check(load().arena_release_slot(arena.handle, slot))


def arena_phi(arena, n) -> list:
    buf = (ctypes.c_int32 * n)()
    _check(load().arena_phi(arena.handle, buf, n))
    return list(buf)


def arena_slot_info(arena, slot):
    st, ex = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load().arena_slot_info(arena.handle, slot, ctypes.byref(st), ctypes.byref(ex)))
    return int(st.value), int(ex.value)


def moe_selftest_mfma_layout(out, stream=None):
    _check(load().moe_selftest_mfma_layout(_ptr(out), _stream(stream)))


# ------------------------------------------------------- buffer helpers --
def row_stride(t: torch.Tensor) -> int:
    """Elements between rows; a single row's stride says nothing, any aligned one does."""
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 7) // 8 * 8


def check_rows(t: torch.Tensor, dtype, cols: int, name: str) -> None:
    """A matrix on the GPU whose rows are contiguous and do not overlap."""
    if t.dim() != 2 or t.dtype != dtype or t.shape[1] != cols or not t.is_cuda:
        raise ValueError(f"{name}: need a GPU matrix [rows][{cols}] of {dtype}")
    if cols > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < cols:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")


def check_device(tensors, stream=None) -> None:
    """The tensors and the stream are on the current GPU."""
    _stream_of_all(tensors, stream)


def alloc_routes(shape: moe_shape, device="cuda") -> dict:
    kp = shape.k + shape.n_shared
    i32 = dict(dtype=torch.int32, device=device)
    return dict(topk_idx=torch.zeros((shape.T, kp), **i32),
                topk_w=torch.zeros((shape.T, kp), dtype=torch.float32, device=device),
                slot_count=torch.zeros(shape.P, **i32),
                slot_offset=torch.zeros(shape.P + 1, **i32),
                rec_token=torch.full((shape.capacity,), -1, **i32),
                rec_route=torch.full((shape.capacity,), -1, **i32),
                route_pos=torch.full((shape.T * kp,), -1, **i32))


def alloc_workspace(shape: moe_shape, device="cuda") -> torch.Tensor:
    n = moe_workspace_bytes(shape)
    if n == 0:
        _check(MOE_ERR_INVALID_ARG)
    buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    ws = buf[off:off + n]
    moe_workspace_init(shape, ws)
    return ws


def alloc_decode_workspace(shape: moe_shape, device="cuda") -> torch.Tensor:
    n = moe_decode_workspace_bytes(shape)
    if n == 0:
        _check(MOE_ERR_INVALID_ARG)
    buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    ws = buf[off:off + n]
    moe_decode_workspace_init(shape, ws)
    return ws


def alloc_balance_workspace(shape: moe_shape, S: int = 1, device="cuda") -> torch.Tensor:
    n = moe_balance_workspace_bytes(shape, S)
    if n == 0:
        _check(MOE_ERR_INVALID_ARG)
    buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + n]


class Arena:
    """Device planes of P slots (Eq. 3) plus the library's residency table."""

    def __init__(self, shape: moe_shape, G: Optional[int] = None, device="cuda"):
        self.shape = shape
        if shape.dtype in (MOE_DT_BF16_FP8W, MOE_DT_BF16_FP4W):
            # a slice is its codes then its scales; strides in bytes
            if shape.dtype == MOE_DT_BF16_FP8W:
                self.stride_gu = 2 * shape.f * shape.d + 8 * shape.f
                self.stride_d = shape.d * shape.f + 4 * shape.d
            else:
                self.stride_gu = fp4_slice_bytes(2 * shape.f, shape.d)
                self.stride_d = fp4_slice_bytes(shape.d, shape.f)
            self.plane_gu = torch.empty((shape.P, self.stride_gu), dtype=torch.uint8, device=device)
            self.plane_d = torch.empty((shape.P, self.stride_d), dtype=torch.uint8, device=device)
        else:
            dt = torch.bfloat16 if shape.dtype == MOE_DT_BF16 else torch.float32
            self.stride_gu = 2 * shape.f * shape.d
            self.stride_d = shape.d * shape.f
            self.plane_gu = torch.empty((shape.P, 2 * shape.f, shape.d), dtype=dt, device=device)
            self.plane_d = torch.empty((shape.P, shape.d, shape.f), dtype=dt, device=device)
        self.G = shape.P if G is None else G
        self.handle = moe_arena_create(shape, self.plane_gu, self.plane_d, self.stride_gu,
                                       self.stride_d, self.G)

    def close(self):
        if self.handle:
            moe_arena_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def load_resident(self, Wg, Wu, Wd, phi: Sequence[int], stream=None, scales=None):
        """Pack and publish every expert e with phi[e] >= 0 into slot phi[e].
        scales: (Sg, Su, Sd) row scales (fp8 codes) or block scales (MXFP4).
        An MXFP4 arena takes fp32 or bf16 weights too, without scales: they
        are quantised on the way (moe_quantize_mxfp4). With a stream, the work
        is queued there, behind the current stream's; the weights are the
        caller's to keep until it is done."""
        quantise = self.shape.dtype == MOE_DT_BF16_FP4W and scales is None and Wg.dtype in _VAL_DTYPE
        if quantise:   # the packing reads as much as the arena's shape says
            f, d = self.shape.f, self.shape.d
            if tuple(Wg.shape[1:]) != (f, d) or tuple(Wu.shape[1:]) != (f, d) or tuple(Wd.shape[1:]) != (d, f):
                raise ValueError(f"load_resident: need Wg and Wu [experts][{f}][{d}] and Wd [experts][{d}][{f}]")
        with on_stream(stream):
            for e, s in enumerate(phi):
                if s < 0:
                    continue
                if quantise:
                    g, u, dn = (mxfp4_slice(W[e]) for W in (Wg, Wu, Wd))
                else:
                    g, u, dn = expert_slices(Wg, Wu, Wd, scales, e)
                moe_pack_gate_up(self.shape, g, u, self.plane_gu[s], 1, 0, 0)
                moe_pack_down(self.shape, dn, self.plane_d[s], 1, 0, 0)
                arena_publish_slot(self, s, e)


def mxfp4_slice(W, stream=None) -> torch.Tensor:
    """W [N][K] (fp32 or bf16) as a source slice of the packing calls: MXFP4
    codes [N][K/2], then scale bytes [N][K/32]. With a stream, the slice
    belongs to it: it is written, to be read and may be dropped there."""
    N, K = W.shape
    with on_stream(stream):
        out = torch.empty(N * K // 2 + N * K // 32, dtype=torch.uint8, device=W.device)
        moe_quantize_mxfp4(W, out[: N * K // 2], out[N * K // 2:])
    return out


def expert_slices(Wg, Wu, Wd, scales, e):
    """Expert e's gate, up and down slices in the layout the C ABI takes:
    the weight rows, then (fp8 codes) the rows' fp32 scales as bytes or
    (MXFP4: packed code bytes [N][K/2]) the E8M0 scale bytes [N][K/32]."""
    if scales is None:
        return Wg[e], Wu[e], Wd[e]
    Sg, Su, Sd = scales
    cat = lambda q, sc: torch.cat([q[e].reshape(-1), sc[e].contiguous().view(torch.uint8).reshape(-1)])
    return cat(Wg, Sg), cat(Wu, Su), cat(Wd, Sd)


def moe_profile_begin(kernel: str, max_launches: int):
    _check(load().moe_profile_begin(MOE_KERNEL[kernel], max_launches))


def moe_profile_end(kernel: str, n: int) -> list:
    buf = (ctypes.c_float * n)()
    rec = ctypes.c_int32(0)
    _check(load().moe_profile_end(MOE_KERNEL[kernel], buf, n, ctypes.byref(rec)))
    return [float(buf[i]) for i in range(min(n, rec.value))]
