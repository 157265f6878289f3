"""Thin ctypes binding of libexl3_gfx950.so (names follow include/exl3.h).

Only argument marshalling happens here: torch tensors give device pointers and
the current HIP stream; every step of the encoder runs in the library's
kernels.  There is no CPU fallback -- if the library or a GPU is missing, the
calls raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

from . import build as _build

EXL3_OK = 0
EXL3_EINVAL = -1
EXL3_ENOMEM = -2
EXL3_ENONFINITE = -3
EXL3_EHIP = -4
EXL3_EUNSUPPORTED = -5
EXL3_F32 = 0
EXL3_BF16 = 1
EXL3_F16 = 2
EXL3_ROW_MAJOR = 0
EXL3_TILE_MAJOR = 1

EXPORTED = [
    "exl3_version", "exl3_ctx_create", "exl3_ctx_destroy", "exl3_last_error",
    "exl3_ctx_set_stream", "exl3_set_codebook", "exl3_get_codebook", "exl3_set_codebook_kind",
    "exl3_set_tile_order",
    "exl3_regularize", "exl3_unregularize",
    "exl3_channel_normalize", "exl3_encode_tiles", "exl3_encode_tiles_noalloc",
    "exl3_encode_tiles_f16", "exl3_decode_tiles", "exl3_quantize_matrix",
    "exl3_quantize_matrix_ldlq", "exl3_quantize_matrix_grid", "exl3_quantize_matrix_f16", "exl3_scratch_per_tile",
    "exl3_ctx_set_timing", "exl3_ctx_read_timing",
    "exl3_linear", "exl3_grouped_linear", "exl3_adapter_linear", "exl3_adapter_linear_backward",
    "exl3_block_quantize", "exl3_block_quantize_weight", "exl3_rms_norm", "exl3_rms_norm_backward",
    "exl3_block_linear", "exl3_block_grouped_linear",
]
CODEBOOK_KINDS = {"mul1": 0, "mcg": 1, "3inst": 2}
KERNEL_KINDS = {"fwd1": 0, "fwd2": 1, "tb1": 2, "tb2": 3, "regularize": 4, "fwd_side": 5,
                "fwd_cost": 6, "channel": 7, "decode": 8, "product": 9, "block": 10, "norm": 11}


class Exl3Error(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("exl3 error %d: %s" % (code, msg))
        self.code = code
        self.msg = msg


class GSS(ctypes.Structure):
    _fields_ = [("iters", ctypes.c_int), ("lo", ctypes.c_double), ("hi", ctypes.c_double)]


class Grid(ctypes.Structure):
    _fields_ = [("coarse_lo", ctypes.c_double), ("coarse_hi", ctypes.c_double),
                ("coarse_step", ctypes.c_double), ("stride", ctypes.c_int),
                ("fine_radius", ctypes.c_double), ("fine_step", ctypes.c_double),
                ("floor", ctypes.c_double)]


class _Weight(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("su", ctypes.c_void_p),
                ("sv", ctypes.c_void_p), ("groups", ctypes.c_int), ("rows", ctypes.c_int),
                ("cols", ctypes.c_int), ("K", ctypes.c_int), ("had_block", ctypes.c_int)]


class _Adapters(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("alpha", ctypes.c_void_p),
                ("count", ctypes.c_int), ("rank", ctypes.c_int)]


class _BlockRows(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ldq", ctypes.c_int64),
                ("lds", ctypes.c_int64)]


class _BlockWeight(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("groups", ctypes.c_int),
                ("rows", ctypes.c_int), ("cols", ctypes.c_int), ("ldq", ctypes.c_int64)]


GRID_PAGES = (0.1, 1.9, 0.1, 2, 0.075, 0.025, 0.01)


_lib = None


def library_path() -> str:
    return _build.LIB


def load_library():
    """Load the built library (never builds; raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        raise FileNotFoundError(
            "libexl3_gfx950.so is not built; run __graft_entry__.build() or "
            "python trellis_coded_weight_amd/build.py")
    lib = ctypes.CDLL(_build.LIB)
    vp, i32, i64, f32, f64, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                  ctypes.c_float, ctypes.c_double, ctypes.c_size_t)
    lib.exl3_version.restype = ctypes.c_char_p
    lib.exl3_version.argtypes = []
    lib.exl3_ctx_create.restype = i32
    lib.exl3_ctx_create.argtypes = [ctypes.POINTER(vp), i32, vp, sz]
    lib.exl3_ctx_destroy.restype = None
    lib.exl3_ctx_destroy.argtypes = [vp]
    lib.exl3_last_error.restype = ctypes.c_char_p
    lib.exl3_last_error.argtypes = [vp]
    lib.exl3_ctx_set_stream.restype = i32
    lib.exl3_ctx_set_stream.argtypes = [vp, vp]
    lib.exl3_set_codebook.restype = i32
    lib.exl3_set_codebook.argtypes = [vp, vp]
    lib.exl3_get_codebook.restype = i32
    lib.exl3_set_codebook_kind.restype = i32
    lib.exl3_set_codebook_kind.argtypes = [vp, i32]
    lib.exl3_get_codebook.argtypes = [vp, vp]
    lib.exl3_set_tile_order.restype = i32
    lib.exl3_set_tile_order.argtypes = [vp, vp]
    lib.exl3_regularize.restype = i32
    lib.exl3_regularize.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, i32, vp, vp]
    lib.exl3_unregularize.restype = i32
    lib.exl3_unregularize.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp]
    lib.exl3_channel_normalize.restype = i32
    lib.exl3_channel_normalize.argtypes = [vp, vp, i32, i32, i32, vp, f64, vp, vp, vp]
    lib.exl3_encode_tiles.restype = i32
    lib.exl3_encode_tiles.argtypes = [vp, vp, i64, i32, f32, vp, vp, vp]
    lib.exl3_encode_tiles_noalloc.restype = i32
    lib.exl3_encode_tiles_noalloc.argtypes = [vp, vp, i64, i32, f32, vp, vp, vp]
    lib.exl3_encode_tiles_f16.restype = i32
    lib.exl3_encode_tiles_f16.argtypes = [vp, vp, i64, i32, vp, vp, vp]
    lib.exl3_decode_tiles.restype = i32
    lib.exl3_decode_tiles.argtypes = [vp, vp, i64, i32, f32, vp]
    lib.exl3_quantize_matrix.restype = i32
    lib.exl3_quantize_matrix.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp,
                                         ctypes.POINTER(GSS), f32, vp, ctypes.POINTER(f32),
                                         ctypes.POINTER(f64), vp, vp]
    lib.exl3_quantize_matrix_ldlq.restype = i32
    lib.exl3_quantize_matrix_ldlq.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp,
                                              ctypes.POINTER(GSS), f32, vp, vp,
                                              ctypes.POINTER(f32), ctypes.POINTER(f64), vp, vp]
    lib.exl3_quantize_matrix_f16.restype = i32
    lib.exl3_quantize_matrix_f16.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp,
                                             ctypes.POINTER(GSS), f32, vp, ctypes.POINTER(f32),
                                             ctypes.POINTER(f64), vp, vp]
    lib.exl3_quantize_matrix_grid.restype = i32
    lib.exl3_quantize_matrix_grid.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp,
                                              ctypes.POINTER(Grid), vp, ctypes.POINTER(f32),
                                              ctypes.POINTER(f64), vp, vp]
    lib.exl3_scratch_per_tile.restype = sz
    lib.exl3_scratch_per_tile.argtypes = [i32]
    lib.exl3_ctx_set_timing.restype = i32
    lib.exl3_ctx_set_timing.argtypes = [vp, i32]
    lib.exl3_ctx_read_timing.restype = i32
    lib.exl3_ctx_read_timing.argtypes = [vp, i32, ctypes.POINTER(f64), ctypes.POINTER(i64),
                                         ctypes.POINTER(i64)]
    wp, ap = ctypes.POINTER(_Weight), ctypes.POINTER(_Adapters)
    lib.exl3_linear.restype = i32
    lib.exl3_linear.argtypes = [vp, wp, i32, vp, i64, i64, i32, vp, i64]
    lib.exl3_grouped_linear.restype = i32
    lib.exl3_grouped_linear.argtypes = [vp, wp, vp, i32, vp, i64, i64, i32, vp, i64]
    lib.exl3_adapter_linear.restype = i32
    lib.exl3_adapter_linear.argtypes = [vp, wp, ap, vp, vp, i64, i64, i32, vp, i64]
    lib.exl3_adapter_linear_backward.restype = i32
    lib.exl3_adapter_linear_backward.argtypes = [vp, wp, ap, vp, vp, i64, vp, i64, i64, i32, vp,
                                                 i64, vp, vp]
    bp, wb = ctypes.POINTER(_BlockRows), ctypes.POINTER(_BlockWeight)
    lib.exl3_block_quantize.restype = i32
    lib.exl3_block_quantize.argtypes = [vp, vp, i64, i64, i32, i32, bp]
    lib.exl3_block_quantize_weight.restype = i32
    lib.exl3_block_quantize_weight.argtypes = [vp, vp, i64, i32, i32, i32, vp, i64, vp]
    lib.exl3_rms_norm.restype = i32
    lib.exl3_rms_norm.argtypes = [vp, vp, i64, vp, i64, vp, i32, f32, i64, i32, i32, vp, i64, bp,
                                  vp, i64]
    lib.exl3_rms_norm_backward.restype = i32
    lib.exl3_rms_norm_backward.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp, i32, f32, i64, i32,
                                           i32, vp, i64, vp]
    lib.exl3_block_linear.restype = i32
    lib.exl3_block_linear.argtypes = [vp, wb, i32, vp, i64, bp, i64, i32, vp, i64]
    lib.exl3_block_grouped_linear.restype = i32
    lib.exl3_block_grouped_linear.argtypes = [vp, wb, vp, i32, vp, i64, bp, i64, i32, vp, i64]
    _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without building a Stream object, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, dtype, shape, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


class CodedWeight:
    """A coded matrix, or one per group (expert), as the products take it: the container of
    quantize_matrix, its scale and the vectors su [rows] and sv [cols] (signs, or folded).
    W = diag(su) H (scale * levels) H diag(sv), rows the output channels.

    packed  int16 [rows/16, cols/16, 16K], or [groups, ...]
    scale   a number, or float32 [groups] on the device
    su, sv  float32 [rows] and [cols], or [groups, ...]

    The tensors are kept, not copied: in-place changes to them show in later products."""

    def __init__(self, packed: torch.Tensor, K: int, scale, su: torch.Tensor, sv: torch.Tensor,
                 had_block: int = 128):
        if not isinstance(packed, torch.Tensor) or packed.dim() not in (3, 4):
            raise ValueError("packed must be a tensor [rows/16, cols/16, 16K] or [groups, ...]")
        self.grouped = packed.dim() == 4
        lead = tuple(packed.shape[:-3])
        groups = packed.shape[0] if self.grouped else 1
        rows, cols = 16 * packed.shape[-3], 16 * packed.shape[-2]
        _need(packed, torch.int16, lead + (rows // 16, cols // 16, 16 * int(K)), "packed")
        if not isinstance(scale, torch.Tensor):
            scale = torch.full((groups,), float(scale), dtype=torch.float32, device=packed.device)
        scale = scale.reshape(-1)
        if su.numel() == groups * rows:
            su = su.reshape(lead + (rows,))
        if sv.numel() == groups * cols:
            sv = sv.reshape(lead + (cols,))
        _need(scale, torch.float32, (groups,), "scale")
        _need(su, torch.float32, lead + (rows,), "su")
        _need(sv, torch.float32, lead + (cols,), "sv")
        self.packed, self.scale, self.su, self.sv = packed, scale, su, sv
        self.groups, self.rows, self.cols = groups, rows, cols
        self.K, self.had_block, self.device = int(K), int(had_block), packed.device
        self._c = _Weight(packed.data_ptr(), scale.data_ptr(), su.data_ptr(), sv.data_ptr(),
                          groups, rows, cols, self.K, self.had_block)
        self._ref = ctypes.byref(self._c)


class Adapters:
    """Low-rank adapters of one rank beside a coded matrix: A [count, rank, cols] and
    B [count, rows, rank] in the activations' type, alpha float32 [count]."""

    def __init__(self, A: torch.Tensor, B: torch.Tensor, alpha: torch.Tensor):
        if A.dim() != 3 or B.dim() != 3:
            raise ValueError("A must be [count, rank, cols] and B [count, rows, rank]")
        count, rank, cols = A.shape
        if A.dtype not in _ACT:
            raise ValueError("A must be bfloat16 or float16, got %s" % A.dtype)
        _need(A, A.dtype, (count, rank, cols), "A")
        _need(B, A.dtype, (count, B.shape[1], rank), "B")
        _need(alpha, torch.float32, (count,), "alpha")
        self.A, self.B, self.alpha = A, B, alpha
        self.count, self.rank, self.cols, self.rows = count, rank, cols, B.shape[1]
        self.dtype, self.device = A.dtype, A.device
        self._c = _Adapters(A.data_ptr(), B.data_ptr(), alpha.data_ptr(), count, rank)
        self._ref = ctypes.byref(self._c)


BLOCK = 128                        # elements along a row that share a scale in 8-bit blocks
_E4M3 = torch.float8_e4m3fn


def _blocks(width: int) -> int:
    return -(-width // BLOCK)


class BlockRows:
    """Rows of activations in 8-bit blocks: a code (e4m3) for each element and a scale for every
    128 consecutive ones of a row; a code stands for scale * q.

    q      float8_e4m3fn [n, cols]
    scale  float32 [n, cols/128 rounded up]

    Both attributes are views of the storage that products read: rows padded with zeros to whole
    blocks, scales of one block of consecutive rows side by side.  Tensors that lie so already
    (cols a multiple of 128, scale transposed) are kept, others copied."""

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        if not isinstance(q, torch.Tensor) or q.dim() != 2 or q.shape[1] < 1:
            raise ValueError("q must be a tensor [n, cols]")
        _need_e4m3(q, "q")
        n, cols = q.shape
        if not isinstance(scale, torch.Tensor) or scale.device != q.device:
            raise ValueError("scale must be a tensor on q's device")
        if scale.dtype != torch.float32 or tuple(scale.shape) != (n, _blocks(cols)):
            raise ValueError("scale must be float32 %s, got %s %s" %
                             ((n, _blocks(cols)), scale.dtype, tuple(scale.shape)))
        if (cols % BLOCK or q.stride(1) != 1 or q.data_ptr() % 16 or
                (n > 1 and (q.stride(0) < cols or q.stride(0) % BLOCK))):
            q = _pad_codes(q)
        ldq = q.stride(0) if n > 1 else BLOCK * _blocks(cols)
        by_block = scale.t()
        if (n > 1 and by_block.stride(1) != 1) or (by_block.shape[0] > 1 and
                                                   by_block.stride(0) < n):
            by_block = by_block.contiguous()
        lds = by_block.stride(0) if by_block.shape[0] > 1 else max(n, 1)
        self._set(q, by_block, n, cols, ldq, lds)

    def _set(self, codes, by_block, n, cols, ldq, lds):
        self._codes, self._by_block = codes, by_block
        self.n, self.cols, self.device = n, cols, codes.device
        self._c = _BlockRows(codes.data_ptr(), by_block.data_ptr(), ldq, lds)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def _empty(cls, n: int, cols: int, device) -> "BlockRows":
        rows = cls.__new__(cls)
        blocks = _blocks(cols)
        rows._set(torch.empty(n, BLOCK * blocks, dtype=_E4M3, device=device),
                  torch.empty(blocks, n, dtype=torch.float32, device=device), n, cols,
                  BLOCK * blocks, n or 1)
        return rows

    @property
    def q(self) -> torch.Tensor:
        codes = self._codes
        return codes if codes.shape[1] == self.cols else codes[:, :self.cols]

    @property
    def scale(self) -> torch.Tensor:
        return self._by_block.t()

    def dequantize(self) -> torch.Tensor:
        """The values [n, cols] in float32."""
        return self.q.float() * self.scale.repeat_interleave(BLOCK, dim=1)[:, :self.cols]


class BlockWeight:
    """A matrix in 8-bit blocks, or one per group (expert): a code (e4m3) for each element and a
    scale for every 128 x 128.

    q      float8_e4m3fn [rows, cols], or [groups, rows, cols]
    scale  float32 [rows/128, cols/128] rounded up, or [groups, ...]

    Contiguous tensors with cols a multiple of 128 are kept, others copied once (q padded with
    zeros to whole blocks); in-place changes to kept tensors show in later products."""

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        if not isinstance(q, torch.Tensor) or q.dim() not in (2, 3) or not q.numel():
            raise ValueError("q must be a tensor [rows, cols] or [groups, rows, cols]")
        _need_e4m3(q, "q")
        lead = tuple(q.shape[:-2])
        rows, cols = q.shape[-2:]
        _need(scale.contiguous() if isinstance(scale, torch.Tensor) else scale, torch.float32,
              lead + (_blocks(rows), _blocks(cols)), "scale")
        if scale.device != q.device:
            raise ValueError("scale must be on q's device")
        if cols % BLOCK or not q.is_contiguous() or q.data_ptr() % 16:
            q = _pad_codes(q)
        scale = scale.contiguous()
        self._set(q, scale, cols)

    def _set(self, q, scale, cols):
        self.grouped = q.dim() == 3
        self.q, self.scale, self.device = q[..., :cols], scale, q.device
        self.groups, self.rows, self.cols = q.shape[0] if self.grouped else 1, q.shape[-2], cols
        self._c = _BlockWeight(q.data_ptr(), scale.data_ptr(), self.groups, self.rows, cols,
                               q.shape[-1])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def _of(cls, q, scale, cols) -> "BlockWeight":
        """From codes in whole blocks of columns and their scales, both contiguous."""
        weight = cls.__new__(cls)
        weight._set(q, scale, cols)
        return weight

    def dequantize(self) -> torch.Tensor:
        """The matrices in float32."""
        s = self.scale.repeat_interleave(BLOCK, dim=-1).repeat_interleave(BLOCK, dim=-2)
        return self.q.float() * s[..., :self.rows, :self.cols]


def _need_e4m3(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dtype != _E4M3:
        raise ValueError("%s must be %s, got %s" % (name, _E4M3, t.dtype))


def _pad_codes(q):
    """q [..., cols] in whole blocks of columns, zeros behind the last."""
    wide = torch.zeros(q.shape[:-1] + (BLOCK * _blocks(q.shape[-1]),), dtype=torch.uint8,
                       device=q.device)
    wide[..., :q.shape[-1]] = q.view(torch.uint8) if q.stride(-1) == 1 else \
        q.contiguous().view(torch.uint8)
    return wide.view(_E4M3)


_ACT = {torch.bfloat16: EXL3_BF16, torch.float16: EXL3_F16}
_FLOAT = {torch.float32: EXL3_F32, **_ACT}


def _act_rows(t: torch.Tensor, width: int, name: str):
    """(tensor, row pitch) of activations [n, width]; a tensor whose rows are not of
    consecutive elements is copied."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    if t.dtype not in _ACT:
        raise ValueError("%s must be bfloat16 or float16, got %s" % (name, t.dtype))
    if t.dim() != 2 or t.shape[1] != width:
        raise ValueError("%s must have shape (n, %d), got %s" % (name, width, tuple(t.shape)))
    if t.stride(1) != 1 or (t.shape[0] > 1 and t.stride(0) < width):
        t = t.contiguous()
    return t, t.stride(0) if t.shape[0] > 1 else width


def _out_rows(out: Optional[torch.Tensor], n: int, width: int, like: torch.Tensor, name: str):
    """(tensor, row pitch) of the output: `out` if given, else a new one."""
    if out is None:
        return torch.empty(n, width, dtype=like.dtype, device=like.device), width
    if not isinstance(out, torch.Tensor) or out.device != like.device or out.dtype != like.dtype:
        raise ValueError("%s must be a %s tensor on %s" % (name, like.dtype, like.device))
    if tuple(out.shape) != (n, width) or out.stride(1) != 1 or (n > 1 and out.stride(0) < width):
        raise ValueError("%s must have shape %s and rows of consecutive elements" %
                         (name, (n, width)))
    return out, out.stride(0) if n > 1 else width


class Context:
    """One library context (scratch, level table) bound to a device."""

    def __init__(self, device: int = 0, scratch_bytes: int = 0):
        if not torch.cuda.is_available():
            raise RuntimeError("the EXL3 encoder needs a GPU; none is visible")
        self.lib = load_library()
        self.device = torch.device("cuda", device)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            rc = self.lib.exl3_ctx_create(ctypes.byref(h), device,
                                          ctypes.c_void_p(_stream_handle(self.device)),
                                          scratch_bytes)
        if rc != EXL3_OK:
            raise Exl3Error(rc, "context creation failed")
        self.handle = h
        # what the level table and the within-tile order were set to
        self._levels, self._order = "mul1", None

    def close(self):
        if getattr(self, "handle", None):
            self.lib.exl3_ctx_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    # -- helpers --
    def _sync_stream(self):
        rc = self.lib.exl3_ctx_set_stream(self.handle,
                                          ctypes.c_void_p(_stream_handle(self.device)))
        self._check(rc)

    def _check(self, rc):
        if rc != EXL3_OK:
            raise Exl3Error(rc, self.lib.exl3_last_error(self.handle).decode())

    def last_error(self) -> str:
        return self.lib.exl3_last_error(self.handle).decode()

    def set_timing(self, enable: bool):
        self._sync_stream()
        self._check(self.lib.exl3_ctx_set_timing(self.handle, 1 if enable else 0))

    def read_timing(self, kind: str):
        """(total_ms, launches, tiles) of the recorded launches of one kernel kind."""
        ms = ctypes.c_double()
        nl = ctypes.c_int64()
        nt = ctypes.c_int64()
        self._check(self.lib.exl3_ctx_read_timing(self.handle, KERNEL_KINDS[kind],
                                                  ctypes.byref(ms), ctypes.byref(nl),
                                                  ctypes.byref(nt)))
        return ms.value, nl.value, nt.value

    # -- API --
    def set_codebook(self, levels_fp16: Optional[torch.Tensor]):
        """levels_fp16: host tensor of 65536 float16 values (None restores mul1)."""
        self._sync_stream()
        if levels_fp16 is None:
            self._check(self.lib.exl3_set_codebook(self.handle, None))
            self._levels = "mul1"
            return
        lv = levels_fp16.detach().cpu().contiguous().view(torch.int16)
        if lv.numel() != 65536:
            raise ValueError("need 65536 levels")
        self._check(self.lib.exl3_set_codebook(self.handle, ctypes.c_void_p(lv.data_ptr())))
        self._levels = lv.numpy().tobytes()

    def set_codebook_kind(self, name: str):
        """Select a procedural codebook by name: "mul1", "mcg" or "3inst"."""
        self._sync_stream()
        self._check(self.lib.exl3_set_codebook_kind(self.handle, CODEBOOK_KINDS[name]))
        self._levels = name

    def set_tile_order(self, order):
        """Within-tile order of tile-major arrays: position t of a tile holds its
        element order[t] (16 * row + col); None restores the natural order."""
        self._sync_stream()
        if order is None:
            self._check(self.lib.exl3_set_tile_order(self.handle, None))
            self._order = None
            return
        o = torch.as_tensor(order, dtype=torch.int64).cpu()
        if o.numel() != 256 or int(o.min()) < 0 or int(o.max()) > 255:
            raise ValueError("a within-tile order has 256 entries in 0..255")
        buf = o.to(torch.uint8).contiguous()
        self._check(self.lib.exl3_set_tile_order(self.handle, ctypes.c_void_p(buf.data_ptr())))
        order = buf.numpy().tobytes()
        self._order = None if order == bytes(range(256)) else order

    def _decoder(self):
        """What codes mean to this context now, for comparison with a later time."""
        return self._levels, self._order

    def get_codebook(self) -> torch.Tensor:
        out = torch.empty(65536, dtype=torch.int16)
        self._sync_stream()
        self._check(self.lib.exl3_get_codebook(self.handle, ctypes.c_void_p(out.data_ptr())))
        return out.view(torch.float16)

    def regularize(self, w: torch.Tensor, su: torch.Tensor, sv: torch.Tensor,
                   had_block: int = 128, tile_major: bool = True):
        """Returns (w_reg float32, tile_sumsq float32 [tiles], nonfinite int32 [1])."""
        rows, cols = w.shape
        dt = {torch.float32: EXL3_F32, torch.bfloat16: EXL3_BF16}.get(w.dtype)
        if dt is None:
            raise ValueError("w must be float32 or bfloat16")
        w = w.contiguous()
        if tile_major:
            out = torch.empty((rows // 16) * (cols // 16), 256, dtype=torch.float32,
                              device=w.device)
        else:
            out = torch.empty(rows, cols, dtype=torch.float32, device=w.device)
        sums = torch.empty((rows // 16) * (cols // 16), dtype=torch.float32, device=w.device)
        flag = torch.zeros(1, dtype=torch.int32, device=w.device)
        self._sync_stream()
        self._check(self.lib.exl3_regularize(
            self.handle, _ptr(w), dt, rows, cols, had_block, _ptr(su.contiguous()),
            _ptr(sv.contiguous()), _ptr(out), EXL3_TILE_MAJOR if tile_major else EXL3_ROW_MAJOR,
            _ptr(sums), _ptr(flag)))
        return out, sums, flag

    def unregularize(self, w_reg: torch.Tensor, rows: int, cols: int, su: torch.Tensor,
                     sv: torch.Tensor, had_block: int = 128, tile_major: bool = True):
        """Inverse regularization of float32 weights (tile-major [tiles, 256] or row-major
        [rows, cols]) -> row-major float32 [rows, cols]."""
        _need(w_reg, torch.float32, tuple(w_reg.shape), "w_reg")
        if w_reg.numel() != rows * cols:
            raise ValueError("w_reg has %d elements, not %d" % (w_reg.numel(), rows * cols))
        out = torch.empty(rows, cols, dtype=torch.float32, device=w_reg.device)
        self._sync_stream()
        self._check(self.lib.exl3_unregularize(
            self.handle, _ptr(w_reg.contiguous()), EXL3_TILE_MAJOR if tile_major else EXL3_ROW_MAJOR,
            rows, cols, had_block, _ptr(su.contiguous()), _ptr(sv.contiguous()), _ptr(out)))
        return out

    def channel_normalize(self, w: torch.Tensor, su: torch.Tensor, floor: float = 0.1):
        """Out-channel RMS normalization: returns (w_norm float32 [rows, cols],
        su_folded float32 [rows], row_rms float64 [rows])."""
        rows, cols = w.shape
        dt = {torch.float32: EXL3_F32, torch.bfloat16: EXL3_BF16}.get(w.dtype)
        if dt is None:
            raise ValueError("w must be float32 or bfloat16")
        w = w.contiguous()
        out = torch.empty(rows, cols, dtype=torch.float32, device=w.device)
        su_f = torch.empty(rows, dtype=torch.float32, device=w.device)
        rms = torch.empty(rows, dtype=torch.float64, device=w.device)
        self._sync_stream()
        self._check(self.lib.exl3_channel_normalize(
            self.handle, _ptr(w), dt, rows, cols, _ptr(su.contiguous()), float(floor), _ptr(out),
            _ptr(su_f), _ptr(rms)))
        return out, su_f, rms

    def encode_tiles(self, x: torch.Tensor, K: int, scale: float, want_states: bool = True,
                     want_sse: bool = True):
        """x float32 [n, 256] -> (packed int16 [n, 16K], states int16 [n, 256] | None,
        sse float32 [n] | None)."""
        n = x.shape[0]
        _need(x, torch.float32, (n, 256), "x")
        packed = torch.empty(n, 16 * K, dtype=torch.int16, device=x.device)
        states = torch.empty(n, 256, dtype=torch.int16, device=x.device) if want_states else None
        sse = torch.empty(n, dtype=torch.float32, device=x.device) if want_sse else None
        self._sync_stream()
        self._check(self.lib.exl3_encode_tiles(self.handle, _ptr(x), n, K, float(scale),
                                               _ptr(packed), _ptr(states), _ptr(sse)))
        return packed, states, sse

    def encode_tiles_noalloc(self, x: torch.Tensor, K: int, scale: float, packed: torch.Tensor,
                             states: Optional[torch.Tensor] = None,
                             sse: Optional[torch.Tensor] = None) -> None:
        """encode_tiles into caller-allocated outputs through the entry point that
        allocates no device memory (at most 256 tiles per call, 512 at K = 4)."""
        n = x.shape[0]
        _need(x, torch.float32, (n, 256), "x")
        _need(packed, torch.int16, (n, 16 * K), "packed")
        if states is not None:
            _need(states, torch.int16, (n, 256), "states")
        if sse is not None:
            _need(sse, torch.float32, (n,), "sse")
        self._sync_stream()
        self._check(self.lib.exl3_encode_tiles_noalloc(self.handle, _ptr(x), n, K, float(scale),
                                                       _ptr(packed), _ptr(states), _ptr(sse)))

    def encode_tiles_f16(self, x: torch.Tensor, K: int, want_states: bool = True,
                         want_cost: bool = True):
        """x float16 [n, 256] -> (packed int16 [n, 16K], states int16 [n, 256] | None,
        cost float16 [n] | None); binary16 arithmetic throughout."""
        n = x.shape[0]
        _need(x, torch.float16, (n, 256), "x")
        packed = torch.empty(n, 16 * K, dtype=torch.int16, device=x.device)
        states = torch.empty(n, 256, dtype=torch.int16, device=x.device) if want_states else None
        cost = torch.empty(n, dtype=torch.float16, device=x.device) if want_cost else None
        self._sync_stream()
        self._check(self.lib.exl3_encode_tiles_f16(self.handle, _ptr(x), n, K, _ptr(packed),
                                                   _ptr(states), _ptr(cost)))
        return packed, states, cost

    def decode_tiles(self, packed: torch.Tensor, K: int, scale: float) -> torch.Tensor:
        n = packed.shape[0]
        _need(packed, torch.int16, (n, 16 * K), "packed")
        out = torch.empty(n, 256, dtype=torch.float32, device=packed.device)
        self._sync_stream()
        self._check(self.lib.exl3_decode_tiles(self.handle, _ptr(packed), n, K, float(scale),
                                               _ptr(out)))
        return out

    # -- products with coded weights --
    def linear(self, x: torch.Tensor, weight: CodedWeight, transpose: bool = False,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x [n, cols] -> x W^T [n, rows]; transpose: x [n, rows] -> x W [n, cols] (the input
        gradient of the former).  bfloat16 or float16, rows of any pitch; out: a tensor to
        write instead of a new one."""
        if weight.grouped and weight.groups != 1:
            raise ValueError("a weight of %d groups: use grouped_linear" % weight.groups)
        wide, tall = (weight.rows, weight.cols) if transpose else (weight.cols, weight.rows)
        x, ldx = _act_rows(x, wide, "x")
        y, ldy = _out_rows(out, x.shape[0], tall, x, "out")
        self._sync_stream()
        self._check(self.lib.exl3_linear(self.handle, weight._ref, int(transpose), x.data_ptr(),
                                         ldx, x.shape[0], _ACT[x.dtype], y.data_ptr(), ldy))
        return y

    def grouped_linear(self, x: torch.Tensor, weight: CodedWeight, offsets: torch.Tensor,
                       transpose: bool = False,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """linear with a matrix per group (expert): rows offsets[e] .. offsets[e + 1] - 1 of x
        are multiplied by matrix e; offsets int32 [groups + 1] on the device.  Rows of no group
        give zeros."""
        _need(offsets, torch.int32, (weight.groups + 1,), "offsets")
        wide, tall = (weight.rows, weight.cols) if transpose else (weight.cols, weight.rows)
        x, ldx = _act_rows(x, wide, "x")
        y, ldy = _out_rows(out, x.shape[0], tall, x, "out")
        self._sync_stream()
        self._check(self.lib.exl3_grouped_linear(
            self.handle, weight._ref, offsets.data_ptr(), int(transpose), x.data_ptr(), ldx,
            x.shape[0], _ACT[x.dtype], y.data_ptr(), ldy))
        return y

    def _adapter_args(self, x, weight, adapters, ids):
        if (adapters.rows, adapters.cols) != (weight.rows, weight.cols):
            raise ValueError("adapters of a %d x %d matrix beside one of %d x %d" %
                             (adapters.rows, adapters.cols, weight.rows, weight.cols))
        if adapters.dtype != x.dtype:
            raise ValueError("adapters must be %s, got %s" % (x.dtype, adapters.dtype))
        _need(ids, torch.int32, (x.shape[0],), "ids")

    def adapter_linear(self, x: torch.Tensor, weight: CodedWeight, adapters: Adapters,
                       ids: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x W^T + alpha_a (x A_a^T) B_a^T, a = ids[t] for row t (int32 [n] on the device, -1:
        no adapter)."""
        x, ldx = _act_rows(x, weight.cols, "x")
        self._adapter_args(x, weight, adapters, ids)
        y, ldy = _out_rows(out, x.shape[0], weight.rows, x, "out")
        self._sync_stream()
        self._check(self.lib.exl3_adapter_linear(
            self.handle, weight._ref, adapters._ref, ids.data_ptr(), x.data_ptr(), ldx,
            x.shape[0], _ACT[x.dtype], y.data_ptr(), ldy))
        return y

    def adapter_linear_backward(self, dy: torch.Tensor, x: torch.Tensor, weight: CodedWeight,
                                adapters: Adapters, ids: torch.Tensor, want_dx: bool = True,
                                want_adapters: bool = True):
        """Gradients (dx, dA, dB) of adapter_linear at x for dy [n, rows]; None for what is
        not wanted.  The coded matrix is frozen."""
        dy, lddy = _act_rows(dy, weight.rows, "dy")
        x, ldx = _act_rows(x, weight.cols, "x")
        if x.shape[0] != dy.shape[0] or x.dtype != dy.dtype:
            raise ValueError("x and dy differ in rows or type")
        self._adapter_args(x, weight, adapters, ids)
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if want_dx else None
        dA = torch.empty_like(adapters.A) if want_adapters else None
        dB = torch.empty_like(adapters.B) if want_adapters else None
        self._sync_stream()
        self._check(self.lib.exl3_adapter_linear_backward(
            self.handle, weight._ref, adapters._ref, ids.data_ptr(), dy.data_ptr(), lddy,
            x.data_ptr(), ldx, x.shape[0], _ACT[x.dtype],
            None if dx is None else dx.data_ptr(), weight.cols,
            None if dA is None else dA.data_ptr(), None if dB is None else dB.data_ptr()))
        return dx, dA, dB

    # -- 8-bit blocks --
    def block_quantize(self, x: torch.Tensor) -> BlockRows:
        """x [n, cols] bfloat16 or float16, rows of any pitch, as 8-bit blocks."""
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x must be a tensor [n, cols]")
        x, ldx = _act_rows(x, x.shape[1], "x")
        out = BlockRows._empty(x.shape[0], x.shape[1], x.device)
        self._sync_stream()
        self._check(self.lib.exl3_block_quantize(self.handle, x.data_ptr(), ldx, x.shape[0],
                                                 x.shape[1], _ACT[x.dtype], out._ref))
        return out

    def block_quantize_weight(self, w: torch.Tensor) -> BlockWeight:
        """w [rows, cols] float32, bfloat16 or float16 as 8-bit blocks of 128 x 128; [groups, rows,
        cols]: matrix by matrix."""
        if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3) or not w.numel():
            raise ValueError("w must be a tensor [rows, cols] or [groups, rows, cols]")
        if not w.is_cuda:
            raise ValueError("w must be a device tensor")
        if w.dtype not in _FLOAT:
            raise ValueError("w must be float32, bfloat16 or float16, got %s" % w.dtype)
        rows, cols = w.shape[-2:]
        lead = tuple(w.shape[:-2])
        q = torch.empty(lead + (rows, BLOCK * _blocks(cols)), dtype=_E4M3, device=w.device)
        scale = torch.empty(lead + (_blocks(rows), _blocks(cols)), dtype=torch.float32,
                            device=w.device)
        self._sync_stream()
        for g in range(w.shape[0] if lead else 1):
            one = w[g] if lead else w
            if one.stride(1) != 1 or (rows > 1 and one.stride(0) < cols):
                one = one.contiguous()
            self._check(self.lib.exl3_block_quantize_weight(
                self.handle, one.data_ptr(), one.stride(0) if rows > 1 else cols, rows, cols,
                _FLOAT[w.dtype], (q[g] if lead else q).data_ptr(), q.shape[-1],
                (scale[g] if lead else scale).data_ptr()))
        return BlockWeight._of(q, scale, cols)

    def block_weight(self, weight: CodedWeight) -> BlockWeight:
        """A coded matrix (or one per group) decoded and written as 8-bit blocks: twice the bytes of
        K = 4, and products at the 8-bit rate.  Reads the scales on the host."""
        n = weight.rows // 16 * (weight.cols // 16)
        parts = []
        for g, scale in enumerate(weight.scale.tolist()):
            def of(t):
                return t[g] if weight.grouped else t
            tiles = self.decode_tiles(of(weight.packed).reshape(n, 16 * weight.K), weight.K, scale)
            parts.append(self.block_quantize_weight(
                self.unregularize(tiles, weight.rows, weight.cols, of(weight.su), of(weight.sv),
                                  weight.had_block)))
        if not weight.grouped:
            return parts[0]
        return BlockWeight(torch.stack([p.q for p in parts]), torch.stack([p.scale for p in parts]))

    def _gain(self, gain, x):
        if not isinstance(gain, torch.Tensor) or gain.dtype not in (x.dtype, torch.float32):
            raise ValueError("gain must be a %s or float32 tensor" % x.dtype)
        _need(gain, gain.dtype, (x.shape[1],), "gain")
        return _FLOAT[gain.dtype]

    def rms_norm(self, x: torch.Tensor, gain: torch.Tensor, eps: float = 1e-6,
                 residual: Optional[torch.Tensor] = None, blocks: bool = False,
                 out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None):
        """Root-mean-square norm of s = x + residual: s / sqrt(mean(s^2) + eps) * gain over the
        columns of x [n, cols] (bfloat16 or float16, rows of any pitch), as a tensor of the same
        type or, with blocks, as BlockRows.  gain [cols], of x's type or float32.
        Without a residual returns y, with one (y, s); s is rounded to x's type after the norm has
        used it.  out, sum_out: tensors to write; each may be x or residual itself."""
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            raise ValueError("x must be a tensor [n, cols]")
        x, ldx = _act_rows(x, x.shape[1], "x")
        n, cols = x.shape
        gain_dtype = self._gain(gain, x)
        ldr = ldsum = ldy = 0
        total = None
        if residual is not None:
            residual, ldr = _act_rows(residual, cols, "residual")
            if residual.shape != x.shape or residual.dtype != x.dtype:
                raise ValueError("residual must be %s %s" % (x.dtype, tuple(x.shape)))
            total, ldsum = _out_rows(sum_out, n, cols, x, "sum_out")
        elif sum_out is not None:
            raise ValueError("sum_out without a residual")
        if blocks:
            if out is not None:
                raise ValueError("out with blocks")
            y = BlockRows._empty(n, cols, x.device)
        else:
            y, ldy = _out_rows(out, n, cols, x, "out")
        self._sync_stream()
        self._check(self.lib.exl3_rms_norm(
            self.handle, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr,
            gain.data_ptr(), gain_dtype, float(eps), n, cols, _ACT[x.dtype],
            None if blocks else y.data_ptr(), ldy, y._ref if blocks else None,
            None if total is None else total.data_ptr(), ldsum))
        return y if residual is None else (y, total)

    def rms_norm_backward(self, dy: torch.Tensor, s: torch.Tensor, gain: torch.Tensor,
                          eps: float = 1e-6, ds: Optional[torch.Tensor] = None,
                          want_dx: bool = True, want_dgain: bool = True):
        """Gradients (dx, dgain) of rms_norm at s, what was normalised (its second result, or x),
        for dy and, where the sum is used further, its gradient ds.  dx is the gradient of x and
        of the residual alike; dgain is of gain's type.  None for what is not wanted."""
        if not isinstance(s, torch.Tensor) or s.dim() != 2:
            raise ValueError("s must be a tensor [n, cols]")
        s, lds = _act_rows(s, s.shape[1], "s")
        n, cols = s.shape
        dy, lddy = _act_rows(dy, cols, "dy")
        gain_dtype = self._gain(gain, s)
        ldds = 0
        if ds is not None:
            ds, ldds = _act_rows(ds, cols, "ds")
        for t, name in ((dy, "dy"), (ds, "ds")):
            if t is not None and (t.shape != s.shape or t.dtype != s.dtype):
                raise ValueError("%s must be %s %s" % (name, s.dtype, tuple(s.shape)))
        dx = torch.empty(n, cols, dtype=s.dtype, device=s.device) if want_dx else None
        dgain = torch.empty_like(gain) if want_dgain else None
        self._sync_stream()
        self._check(self.lib.exl3_rms_norm_backward(
            self.handle, dy.data_ptr(), lddy, None if ds is None else ds.data_ptr(), ldds,
            s.data_ptr(), lds, gain.data_ptr(), gain_dtype, float(eps), n, cols, _ACT[s.dtype],
            None if dx is None else dx.data_ptr(), cols,
            None if dgain is None else dgain.data_ptr()))
        return dx, dgain

    def _block_input(self, x, width, out, dtype):
        """(x or None, its pitch, blocks or None, n, type of the result)."""
        if isinstance(x, BlockRows):
            if x.cols != width:
                raise ValueError("x must have %d columns, got %d" % (width, x.cols))
            if dtype is None:
                dtype = out.dtype if isinstance(out, torch.Tensor) else torch.bfloat16
            if dtype not in _ACT:
                raise ValueError("dtype must be bfloat16 or float16, got %s" % dtype)
            return None, 0, x, x.n, dtype
        x, ldx = _act_rows(x, width, "x")
        if dtype is not None and dtype != x.dtype:
            raise ValueError("dtype must be that of x, %s" % x.dtype)
        return x, ldx, None, x.shape[0], x.dtype

    def block_linear(self, x, weight: BlockWeight, transpose: bool = False,
                     out: Optional[torch.Tensor] = None, dtype=None) -> torch.Tensor:
        """x [n, cols] -> x W^T [n, rows]; transpose: x [n, rows] -> x W [n, cols] (the input
        gradient of the former).  x: bfloat16 or float16, rows of any pitch, which the call writes
        as 8-bit blocks first; or BlockRows, with dtype the type of the result (that of out, or
        bfloat16)."""
        if weight.grouped and weight.groups != 1:
            raise ValueError("a weight of %d groups: use block_grouped_linear" % weight.groups)
        return self._block_product(x, weight, None, transpose, out, dtype)

    def block_grouped_linear(self, x, weight: BlockWeight, offsets: torch.Tensor,
                             transpose: bool = False, out: Optional[torch.Tensor] = None,
                             dtype=None) -> torch.Tensor:
        """block_linear with a matrix per group (expert): rows offsets[e] .. offsets[e + 1] - 1 of
        x are multiplied by matrix e; offsets int32 [groups + 1] on the device.  Rows of no group
        give zeros."""
        _need(offsets, torch.int32, (weight.groups + 1,), "offsets")
        return self._block_product(x, weight, offsets, transpose, out, dtype)

    def _block_product(self, x, weight, offsets, transpose, out, dtype):
        wide, tall = (weight.rows, weight.cols) if transpose else (weight.cols, weight.rows)
        x, ldx, blocks, n, dtype = self._block_input(x, wide, out, dtype)
        device = blocks.device if x is None else x.device
        if out is None:
            y, ldy = torch.empty(n, tall, dtype=dtype, device=device), tall
        else:
            y, ldy = _out_rows(out, n, tall, torch.empty(0, dtype=dtype, device=device), "out")
        ptr = None if x is None else x.data_ptr()
        ref = None if blocks is None else blocks._ref
        self._sync_stream()
        if offsets is None:
            rc = self.lib.exl3_block_linear(self.handle, weight._ref, int(transpose), ptr, ldx, ref,
                                            n, _ACT[dtype], y.data_ptr(), ldy)
        else:
            rc = self.lib.exl3_block_grouped_linear(
                self.handle, weight._ref, offsets.data_ptr(), int(transpose), ptr, ldx, ref, n,
                _ACT[dtype], y.data_ptr(), ldy)
        self._check(rc)
        return y

    def quantize_matrix(self, w: torch.Tensor, K: int, su: torch.Tensor, sv: torch.Tensor,
                        had_block: int = 128,
                        gss: Optional[Tuple[int, float, float]] = (12, 0.5, 2.0),
                        scale: float = 1.0, want_w_hat: bool = False,
                        want_tile_sse: bool = False):
        """Returns dict(packed int16 [R/16, C/16, 16K], scale, mse, w_hat?, tile_sse?)."""
        rows, cols = w.shape
        dt = {torch.float32: EXL3_F32, torch.bfloat16: EXL3_BF16}.get(w.dtype)
        if dt is None:
            raise ValueError("w must be float32 or bfloat16")
        w = w.contiguous()
        dev = w.device
        packed = torch.empty(rows // 16, cols // 16, 16 * K, dtype=torch.int16, device=dev)
        w_hat = (torch.empty((rows // 16) * (cols // 16), 256, dtype=torch.float32, device=dev)
                 if want_w_hat else None)
        tsse = (torch.empty((rows // 16) * (cols // 16), dtype=torch.float32, device=dev)
                if want_tile_sse else None)
        g = None if gss is None else ctypes.byref(GSS(int(gss[0]), float(gss[1]), float(gss[2])))
        s_out = ctypes.c_float(0.0)
        mse = ctypes.c_double(0.0)
        self._sync_stream()
        self._check(self.lib.exl3_quantize_matrix(
            self.handle, _ptr(w), dt, rows, cols, K, had_block, _ptr(su.contiguous()),
            _ptr(sv.contiguous()), g, float(scale), _ptr(packed), ctypes.byref(s_out),
            ctypes.byref(mse), _ptr(w_hat), _ptr(tsse)))
        return {"packed": packed, "scale": s_out.value, "mse": mse.value, "w_hat": w_hat,
                "tile_sse": tsse}

    def quantize_matrix_f16(self, w: torch.Tensor, K: int, su: torch.Tensor, sv: torch.Tensor,
                            had_block: int = 128,
                            gss: Optional[Tuple[int, float, float]] = (12, 0.5, 2.0),
                            scale: float = 1.0, want_w_hat: bool = False,
                            want_tile_sse: bool = False):
        """Whole-matrix path with the binary16 encoder inside the scale search.
        Returns dict(packed int16 [R/16, C/16, 16K], scale, mse, w_hat?, tile_sse?)."""
        rows, cols = w.shape
        dt = {torch.float32: EXL3_F32, torch.bfloat16: EXL3_BF16}.get(w.dtype)
        if dt is None:
            raise ValueError("w must be float32 or bfloat16")
        w = w.contiguous()
        dev = w.device
        packed = torch.empty(rows // 16, cols // 16, 16 * K, dtype=torch.int16, device=dev)
        w_hat = (torch.empty((rows // 16) * (cols // 16), 256, dtype=torch.float32, device=dev)
                 if want_w_hat else None)
        tsse = (torch.empty((rows // 16) * (cols // 16), dtype=torch.float32, device=dev)
                if want_tile_sse else None)
        g = None if gss is None else ctypes.byref(GSS(int(gss[0]), float(gss[1]), float(gss[2])))
        s_out = ctypes.c_float(0.0)
        mse = ctypes.c_double(0.0)
        self._sync_stream()
        self._check(self.lib.exl3_quantize_matrix_f16(
            self.handle, _ptr(w), dt, rows, cols, K, had_block, _ptr(su.contiguous()),
            _ptr(sv.contiguous()), g, float(scale), _ptr(packed), ctypes.byref(s_out),
            ctypes.byref(mse), _ptr(w_hat), _ptr(tsse)))
        return {"packed": packed, "scale": s_out.value, "mse": mse.value, "w_hat": w_hat,
                "tile_sse": tsse}

    def quantize_matrix_grid(self, w: torch.Tensor, K: int, su: torch.Tensor, sv: torch.Tensor,
                             had_block: int = 128, grid: Tuple = GRID_PAGES,
                             want_w_hat: bool = False, want_tile_sse: bool = False):
        """Whole-matrix path with the grid + parabolic scale search.
        Returns dict(packed int16 [R/16, C/16, 16K], scale, mse, w_hat?, tile_sse?)."""
        rows, cols = w.shape
        dt = {torch.float32: EXL3_F32, torch.bfloat16: EXL3_BF16}.get(w.dtype)
        if dt is None:
            raise ValueError("w must be float32 or bfloat16")
        w = w.contiguous()
        dev = w.device
        packed = torch.empty(rows // 16, cols // 16, 16 * K, dtype=torch.int16, device=dev)
        w_hat = (torch.empty((rows // 16) * (cols // 16), 256, dtype=torch.float32, device=dev)
                 if want_w_hat else None)
        tsse = (torch.empty((rows // 16) * (cols // 16), dtype=torch.float32, device=dev)
                if want_tile_sse else None)
        g = Grid(float(grid[0]), float(grid[1]), float(grid[2]), int(grid[3]), float(grid[4]),
                 float(grid[5]), float(grid[6]))
        s_out = ctypes.c_float(0.0)
        mse = ctypes.c_double(0.0)
        self._sync_stream()
        self._check(self.lib.exl3_quantize_matrix_grid(
            self.handle, _ptr(w), dt, rows, cols, K, had_block, _ptr(su.contiguous()),
            _ptr(sv.contiguous()), ctypes.byref(g), _ptr(packed), ctypes.byref(s_out),
            ctypes.byref(mse), _ptr(w_hat), _ptr(tsse)))
        return {"packed": packed, "scale": s_out.value, "mse": mse.value, "w_hat": w_hat,
                "tile_sse": tsse}

    def quantize_matrix_ldlq(self, w: torch.Tensor, K: int, su: torch.Tensor, sv: torch.Tensor,
                             L: torch.Tensor, had_block: int = 128,
                             gss: Optional[Tuple[int, float, float]] = (12, 0.5, 2.0),
                             scale: float = 1.0, want_w_hat: bool = False,
                             want_tile_err: bool = False):
        """LDLQ whole-matrix path; L float32 [cols, cols] on the device.
        Returns dict(packed int16 [R/16, C/16, 16K], scale, mse, w_hat?, tile_err?)."""
        rows, cols = w.shape
        dt = {torch.float32: EXL3_F32, torch.bfloat16: EXL3_BF16}.get(w.dtype)
        if dt is None:
            raise ValueError("w must be float32 or bfloat16")
        _need(L, torch.float32, (cols, cols), "L")
        w = w.contiguous()
        dev = w.device
        packed = torch.empty(rows // 16, cols // 16, 16 * K, dtype=torch.int16, device=dev)
        w_hat = (torch.empty((rows // 16) * (cols // 16), 256, dtype=torch.float32, device=dev)
                 if want_w_hat else None)
        terr = (torch.empty((rows // 16) * (cols // 16), dtype=torch.float32, device=dev)
                if want_tile_err else None)
        g = None if gss is None else ctypes.byref(GSS(int(gss[0]), float(gss[1]), float(gss[2])))
        s_out = ctypes.c_float(0.0)
        mse = ctypes.c_double(0.0)
        self._sync_stream()
        self._check(self.lib.exl3_quantize_matrix_ldlq(
            self.handle, _ptr(w), dt, rows, cols, K, had_block, _ptr(su.contiguous()),
            _ptr(sv.contiguous()), g, float(scale), _ptr(L), _ptr(packed), ctypes.byref(s_out),
            ctypes.byref(mse), _ptr(w_hat), _ptr(terr)))
        return {"packed": packed, "scale": s_out.value, "mse": mse.value, "w_hat": w_hat,
                "tile_err": terr}


def scratch_per_tile(K: int) -> int:
    return int(load_library().exl3_scratch_per_tile(K))


def version() -> str:
    return load_library().exl3_version().decode()


_DEFAULT_CTX = {}


def quantize_matrix(w: torch.Tensor, K: int, su: torch.Tensor, sv: torch.Tensor,
                    had_block: int = 128,
                    gss: Optional[Tuple[int, float, float]] = (12, 0.5, 2.0),
                    scale: float = 1.0):
    """The whole-matrix path as a tuple: (packed int16 [R/16, C/16, 16K], scale,
    mse), on a context per device kept for the process (its scratch is the
    library's default bound).  Context.quantize_matrix takes the same arguments
    and also returns the optional outputs."""
    dev = w.device.index if w.device.index is not None else torch.cuda.current_device()
    ctx = _DEFAULT_CTX.get(dev)
    if ctx is None:
        ctx = _DEFAULT_CTX[dev] = Context(dev)
    out = ctx.quantize_matrix(w, K, su, sv, had_block=had_block, gss=gss, scale=scale)
    return out["packed"], out["scale"], out["mse"]
