"""The 4-bit operators of the rest of a decoder block: INT4 projections, a
paged 4-bit cache of keys and values with the attention that reads it, and the
plan of the pages and slots that a step's tokens take.

    plan = plan_pages(lens, delta, table, free_pages, free_count, page_size, max_new=64)
    qkv = Linear4(w_qkv).forward(x)                    # x: [B, d], B <= 16
    cache.append(k, v, plan.slots)
    o = cache.attend(q, table, plan.lens)              # [B, Hq, D]

Argument checks and marshalling only; the arithmetic runs in libprox.so.
"""

from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from ._lib import DTYPE_BF16, DTYPE_F16, DTYPE_F32, check, lib

DTYPES = {torch.float32: DTYPE_F32, torch.float16: DTYPE_F16, torch.bfloat16: DTYPE_BF16}


def _raw_stream(stream, device: torch.device) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A result tensor that belongs to the stream that writes it."""
    if isinstance(stream, torch.cuda.Stream):
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def _act(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return code


def _ints(t: torch.Tensor, dtype: torch.dtype, numel: int, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    if t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name} must hold {numel} contiguous values")
    return t


def _same_device(device: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


class Linear4:
    """INT4 weights of one [d_in, d_out] matrix on the current CUDA device:
    y = x W for 1 to 16 tokens.

    w: bf16 [d_in, d_out], quantised by pack_proxy's rule; or codes and scales
    as pack_proxy returns them.  The library keeps its own copy, so the tensors
    may be freed afterwards.
    """

    def __init__(self, w: torch.Tensor | None = None, *, codes: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, stream=None):
        h = ctypes.c_void_p(0)
        if w is not None:
            if codes is not None or scales is not None:
                raise ValueError("give either w or codes and scales")
            if not isinstance(w, torch.Tensor) or not w.is_cuda or w.dtype != torch.bfloat16:
                raise TypeError("w must be a bfloat16 CUDA tensor")
            if w.dim() != 2 or not w.is_contiguous():
                raise ValueError("w must be a contiguous [d_in, d_out] matrix")
            self._on_device(w)
            d_in, d_out = w.shape
            check(lib.prox_linear4_create_bf16(w.data_ptr(), d_in, d_out, _raw_stream(stream, w.device),
                                               ctypes.byref(h)))
            self.device = w.device
        else:
            if codes is None or scales is None:
                raise ValueError("give either w or codes and scales")
            for t, dt, name in ((codes, torch.uint8, "codes"), (scales, torch.float16, "scales")):
                if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dt:
                    raise TypeError(f"{name} must be a CUDA tensor of {dt}")
                if t.dim() != 2 or not t.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous matrix")
                self._on_device(t)
            d_in, d_out = codes.shape[0], 2 * codes.shape[1]
            if d_in % 128 or tuple(scales.shape) != (d_in // 128, d_out):
                raise ValueError(f"scales must be [{d_in} / 128, {d_out}], got {tuple(scales.shape)}")
            check(lib.prox_linear4_create(codes.data_ptr(), scales.data_ptr(), d_in, d_out,
                                          _raw_stream(stream, codes.device), ctypes.byref(h)))
            self.device = codes.device
        self.d_in, self.d_out = d_in, d_out
        self._h = h

    @staticmethod
    def _on_device(t: torch.Tensor) -> None:
        cur = torch.cuda.current_device()
        if t.device.index != cur:
            raise ValueError(f"the tensor is on {t.device}, not on the current CUDA device cuda:{cur}")

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib.prox_linear4_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise RuntimeError("the weights are closed")
        return self._h

    def forward(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x [B, d_in] or [d_in] (rows may be strided) -> [B, d_out] or [d_out] of x's type."""
        dt = _act(x, "x")
        dim = x.dim()
        if dim not in (1, 2) or x.shape[-1] != self.d_in or x.stride(-1) != 1:
            raise ValueError(f"x must be [B, {self.d_in}] or [{self.d_in}] with contiguous rows, "
                             f"got {tuple(x.shape)}")
        B = x.shape[0] if dim == 2 else 1
        if out is None:
            if x.device != self.device:
                raise ValueError(f"x is on {x.device}, not on {self.device}")
            out = _empty((B, self.d_out) if dim == 2 else (self.d_out,), x.dtype, x.device, stream)
            out_stride = self.d_out
        else:
            _same_device(self.device, x=x, out=out)
            if out.dtype != x.dtype or out.dim() != dim or out.shape[-1] != self.d_out \
                    or out.stride(-1) != 1 or (dim == 2 and out.shape[0] != B):
                raise ValueError(f"out must be {x.dtype} of {B} rows of {self.d_out} contiguous values")
            out_stride = out.stride(0) if dim == 2 else self.d_out
        check(lib.prox_linear4_forward(self.handle, x.data_ptr(), x.stride(0) if dim == 2 else self.d_in,
                                       out.data_ptr(), out_stride, B, dt, _raw_stream(stream, x.device)))
        return out

    __call__ = forward


class KVCache4:
    """A paged cache of keys and values in 4 bits, on the caller's tensors:
    codes uint8 [pages, heads, page_size, head_dim / 2], scales fp16 [pages,
    heads, page_size].  One stream at a time uses a cache."""

    def __init__(self, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor,
                 v_scales: torch.Tensor):
        for t, dt, name in ((k_codes, torch.uint8, "k_codes"), (v_codes, torch.uint8, "v_codes"),
                            (k_scales, torch.float16, "k_scales"), (v_scales, torch.float16, "v_scales")):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dt:
                raise TypeError(f"{name} must be a CUDA tensor of {dt}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            Linear4._on_device(t)
        if k_codes.dim() != 4 or v_codes.shape != k_codes.shape \
                or k_scales.shape != k_codes.shape[:3] or v_scales.shape != k_codes.shape[:3]:
            raise ValueError("codes must be [pages, heads, page_size, head_dim / 2] and scales "
                             "[pages, heads, page_size]")
        self.num_pages, self.n_heads, self.page_size = k_codes.shape[:3]
        self.head_dim = 2 * k_codes.shape[3]
        self.device = k_codes.device
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        h = ctypes.c_void_p(0)
        check(lib.prox_kv4_create(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                                  v_scales.data_ptr(), self.num_pages, self.n_heads, self.page_size,
                                  self.head_dim, ctypes.byref(h)))
        self._h = h

    @classmethod
    def zeros(cls, num_pages: int, n_heads: int, page_size: int, head_dim: int,
              device="cuda") -> "KVCache4":
        """A cache whose rows all read as zero."""
        shape = (num_pages, n_heads, page_size)
        codes = [torch.full(shape + (head_dim // 2,), 0x88, dtype=torch.uint8, device=device)
                 for _ in range(2)]
        scales = [torch.zeros(shape, dtype=torch.float16, device=device) for _ in range(2)]
        return cls(codes[0], scales[0], codes[1], scales[1])

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib.prox_kv4_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise RuntimeError("the cache is closed")
        return self._h

    def error_word(self, stream=None) -> int:
        """DEVERR_SLOT / DEVERR_PAGE / DEVERR_LEN bits since the last call (synchronises)."""
        v = ctypes.c_int32(0)
        check(lib.prox_kv4_error(self.handle, ctypes.byref(v), _raw_stream(stream, self.device)))
        return int(v.value)

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
        """Quantises rows k, v [T, heads, head_dim] (any strides, values
        contiguous) into slots (int64 [T]; negative: skipped)."""
        dt = _act(k, "k")
        shape = k.shape
        if len(shape) != 3 or shape[1] != self.n_heads or shape[2] != self.head_dim or v.shape != shape \
                or k.stride(2) != 1 or v.stride(2) != 1:
            raise ValueError(f"k and v must be [T, {self.n_heads}, {self.head_dim}] with contiguous rows")
        if v.dtype != k.dtype:
            raise TypeError(f"k and v must have one type, got {k.dtype} and {v.dtype}")
        _ints(slots, torch.int64, shape[0], "slots")
        _same_device(self.device, k=k, v=v, slots=slots)
        check(lib.prox_kv4_append(self.handle, k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1),
                                  v.stride(0), v.stride(1), slots.data_ptr(), shape[0], dt,
                                  _raw_stream(stream, self.device)))

    def read(self, slots: torch.Tensor, dtype: torch.dtype = torch.float32,
             stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        """The values held at slots (int64 [T]): k and v [T, heads, head_dim],
        zeros for negative slots."""
        if dtype not in DTYPES:
            raise TypeError(f"dtype must be float32, float16 or bfloat16, got {dtype}")
        T = slots.numel()
        _ints(slots, torch.int64, T, "slots")
        _same_device(self.device, slots=slots)
        k, v = _empty((2, T, self.n_heads, self.head_dim), dtype, self.device, stream).unbind(0)
        check(lib.prox_kv4_read(self.handle, slots.data_ptr(), T, k.data_ptr(), v.data_ptr(), DTYPES[dtype],
                                _raw_stream(stream, self.device)))
        return k, v

    def attend(self, q: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, scale: float | None = None,
               out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of the newest tokens, causal: q [B, Tq, Hq, head_dim] or
        [B, Hq, head_dim] for one token each; table int32 [B, cols] of pages;
        lens int32 [B], the cached tokens with the new ones among them.  scale
        defaults to head_dim ** -0.5.  lse: optional fp32 [B, Tq, Hq]."""
        dt = _act(q, "q")
        dim = q.dim()
        if dim not in (3, 4) or q.shape[-1] != self.head_dim or q.stride(-1) != 1:
            raise ValueError(f"q must be [B, Tq, Hq, {self.head_dim}] or [B, Hq, {self.head_dim}] with "
                             f"contiguous rows, got {tuple(q.shape)}")
        B, Hq = q.shape[0], q.shape[-2]
        Tq = q.shape[1] if dim == 4 else 1
        if not isinstance(table, torch.Tensor) or table.dtype != torch.int32 or table.dim() != 2 \
                or table.shape[0] != B or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError(f"table must be int32 [{B}, cols] with contiguous rows")
        _ints(lens, torch.int32, B, "lens")
        _same_device(self.device, q=q, table=table, lens=lens, out=out, lse=lse)
        if out is None:
            out = _empty(q.shape, q.dtype, self.device, stream)
        elif out.dtype != q.dtype or out.shape != q.shape or not out.is_contiguous():
            raise ValueError("out must be a contiguous tensor of q's shape and type")
        if lse is not None and (lse.dtype != torch.float32 or lse.numel() != B * Tq * Hq
                                or not lse.is_contiguous()):
            raise ValueError(f"lse must hold {B * Tq * Hq} contiguous float32 values")
        cols = table.shape[1]
        check(lib.prox_kv4_attend(self.handle, q.data_ptr(), q.stride(0), q.stride(1) if dim == 4 else 0,
                                  q.stride(-2), Hq, B, Tq, table.data_ptr(), max(table.stride(0), cols), cols,
                                  lens.data_ptr(), 1.0 / math.sqrt(self.head_dim) if scale is None else scale,
                                  out.data_ptr(), None if lse is None else lse.data_ptr(), dt,
                                  _raw_stream(stream, self.device)))
        return out


class PagePlan(NamedTuple):
    """What plan_pages returns (device tensors): lens int32 [B] and count int32
    [1] after the step, cu int32 [B + 1], slots int64 and positions int32
    [max_new], status int32 [1] (1: the plan did not fit, nothing changed)."""
    lens: torch.Tensor
    count: torch.Tensor
    cu: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    status: torch.Tensor


def plan_pages(lens: torch.Tensor, delta: torch.Tensor, table: torch.Tensor, free_pages: torch.Tensor,
               free_count: torch.Tensor, page_size: int, max_new: int, commit: bool = False,
               stream=None) -> PagePlan:
    """Pages, slots and positions of the tokens that B requests gain (delta >
    0) or drop (delta < 0) in a step, on the GPU.  lens, delta: int32 [B];
    table: int32 [B, cols], updated in place; free_pages: int32, updated in
    place beyond what is in use; free_count: int32 [1].  commit: lens and
    free_count are updated in place too (and returned); otherwise the new ones
    are new tensors and the same plan may be made again."""
    B = lens.numel()
    _ints(lens, torch.int32, B, "lens")
    _ints(delta, torch.int32, B, "delta")
    _ints(free_count, torch.int32, 1, "free_count")
    _ints(free_pages, torch.int32, free_pages.numel(), "free_pages")
    if not isinstance(table, torch.Tensor) or table.dtype != torch.int32 or table.dim() != 2 \
            or table.shape[0] != B or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"table must be int32 [{B}, cols] with contiguous rows")
    if max_new < 0:
        raise ValueError(f"max_new={max_new} must be >= 0")
    dev = lens.device
    _same_device(dev, delta=delta, table=table, free_pages=free_pages, free_count=free_count)
    Linear4._on_device(lens)
    buf = _empty((2 * B + 3 + max_new,), torch.int32, dev, stream)
    new_lens, cu, count, status, positions = buf.split_with_sizes([B, B + 1, 1, 1, max_new])
    slots = _empty((max_new,), torch.int64, dev, stream)
    if commit:
        new_lens, count = lens, free_count
    cols = table.shape[1]
    check(lib.prox_plan_pages(lens.data_ptr(), delta.data_ptr(), B, int(page_size), table.data_ptr(),
                              max(table.stride(0), cols), cols, free_pages.data_ptr(), free_pages.numel(),
                              free_count.data_ptr(), new_lens.data_ptr(), count.data_ptr(), cu.data_ptr(),
                              slots.data_ptr(), positions.data_ptr(), max_new, status.data_ptr(),
                              _raw_stream(stream, dev)))
    return PagePlan(new_lens, count, cu, slots, positions, status)
