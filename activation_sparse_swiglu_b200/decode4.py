"""The 4-bit operators of the rest of a decoder block: INT4 projections, a
paged 4-bit cache of keys and values with the attention that reads it, and the
plan of the pages and slots that a step's tokens take.

    plan = plan_pages(lens, delta, table, free_pages, free_count, page_size, max_new=64)
    qkv = Linear4(w_qkv).forward(x)                    # x: [B, d], B <= 16
    cache.append(k, v, plan.slots)
    o = cache.attend(q, table, plan.lens)              # [B, Hq, D]

No call gives gradients: one whose inputs carry them (outside torch.no_grad())
is refused.

Argument checks and marshalling only, most of it in the native module _decode4
(csrc/decode4_py.cpp); the arithmetic runs in libprox.so.
"""

from __future__ import annotations

import ctypes
import math
import sys
from typing import NamedTuple

import torch

from ._lib import PKG, check, lib

class _Missing:
    """In the native module's place where it cannot be loaded: the rest of the
    package does without it, every 4-bit operator raises."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"{PKG}/_decode4.so cannot be loaded: build it with `python {PKG}/build.py` (the 4-bit "
                          f"operators need it; there is no fallback): {self._why}")


try:
    from . import _decode4
    _tag = f"torch {torch.__version__}, {sys.implementation.cache_tag}"
    if _decode4.built_for != _tag:
        raise ImportError(f"it was built for {_decode4.built_for}, this is {_tag}")
except ImportError as e:
    _decode4 = _Missing(str(e))


def _raw_stream(stream, index: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def on_stream(stream, device: torch.device):
    """Context in which `stream` (a torch stream or a raw handle) is current."""
    if not isinstance(stream, torch.cuda.Stream):
        # 0 and 1 (cudaStreamLegacy) are handles of the default stream.  As an
        # ExternalStream torch would take 0 for "none given" and make one of its
        # pool, which nothing orders behind the caller's work, and 1 (its own
        # streams have odd ids) for one of its own.
        handle = int(stream)
        stream = (torch.cuda.default_stream(device) if handle in (0, 1)
                  else torch.cuda.ExternalStream(handle, device=device))
    return torch.cuda.stream(stream)


def _empty(device: torch.device, shape, dtype, stream) -> torch.Tensor:
    """A result tensor that belongs to the stream that writes it."""
    with on_stream(stream, device):
        return torch.empty(shape, dtype=dtype, device=device)


class Linear4:
    """INT4 weights of one [d_in, d_out] matrix on the current CUDA device:
    y = x W for 1 to 16 tokens.

    w: bf16 [d_in, d_out], quantised by pack_proxy's rule; or codes and scales
    as pack_proxy returns them.  The library keeps its own copy, so the tensors
    may be freed afterwards.
    """

    def __init__(self, w: torch.Tensor | None = None, *, codes: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, stream=None):
        _decode4.linear4_forward  # raises here if the module is missing
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
            check(lib.prox_linear4_create_bf16(w.data_ptr(), d_in, d_out, _raw_stream(stream, w.device.index),
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
                                          _raw_stream(stream, codes.device.index), ctypes.byref(h)))
            self.device = codes.device
        self.d_in, self.d_out = d_in, d_out
        self._index = self.device.index
        self._h, self._raw = h, h.value

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
        if self._h is None:
            raise RuntimeError("the weights are closed")
        if stream is not None:
            if out is None and isinstance(x, torch.Tensor):
                out = _empty(self.device, x.shape[:-1] + (self.d_out,), x.dtype, stream)
            stream = _raw_stream(stream, self._index)
        return _decode4.linear4_forward(self._raw, self._index, self.d_in, self.d_out, x, out, stream)

    __call__ = forward


class KVCache4:
    """A paged cache of keys and values in 4 bits, on the caller's tensors:
    codes uint8 [pages, heads, page_size, head_dim / 2], scales fp16 [pages,
    heads, page_size].  One stream at a time uses a cache."""

    def __init__(self, k_codes: torch.Tensor, k_scales: torch.Tensor, v_codes: torch.Tensor,
                 v_scales: torch.Tensor):
        _decode4.kv4_attend  # raises here if the module is missing
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
        self._index = self.device.index
        self._scale = 1.0 / math.sqrt(self.head_dim)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        h = ctypes.c_void_p(0)
        check(lib.prox_kv4_create(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                                  v_scales.data_ptr(), self.num_pages, self.n_heads, self.page_size,
                                  self.head_dim, ctypes.byref(h)))
        self._h, self._raw = h, h.value

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
        check(lib.prox_kv4_error(self.handle, ctypes.byref(v), _raw_stream(stream, self._index)))
        return int(v.value)

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
        """Quantises rows k, v [T, heads, head_dim] (any strides, values
        contiguous) into slots (int64 [T]; negative: skipped)."""
        if self._h is None:
            raise RuntimeError("the cache is closed")
        _decode4.kv4_append(self._raw, self._index, self.n_heads, self.head_dim, k, v, slots,
                            None if stream is None else _raw_stream(stream, self._index))

    def read(self, slots: torch.Tensor, dtype: torch.dtype = torch.float32,
             stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        """The values held at slots (int64 [T]): k and v [T, heads, head_dim],
        zeros for negative slots."""
        if self._h is None:
            raise RuntimeError("the cache is closed")
        kv = None
        if stream is not None and isinstance(slots, torch.Tensor) and slots.is_cuda:
            shape = (slots.numel(), self.n_heads, self.head_dim)
            kv = tuple(_empty(self.device, shape, dtype, stream) for _ in range(2))
            stream = _raw_stream(stream, self._index)
        return _decode4.kv4_read(self._raw, self._index, self.n_heads, self.head_dim, slots, dtype, kv, stream)

    def attend(self, q: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, scale: float | None = None,
               out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Attention of the newest tokens, causal: q [B, Tq, Hq, head_dim] or
        [B, Hq, head_dim] for one token each; table int32 [B, cols] of pages;
        lens int32 [B], the cached tokens with the new ones among them.  scale
        defaults to head_dim ** -0.5.  lse: optional fp32 [B, Tq, Hq]."""
        if self._h is None:
            raise RuntimeError("the cache is closed")
        if stream is not None:
            if out is None and isinstance(q, torch.Tensor):
                out = _empty(self.device, q.shape, q.dtype, stream)
            stream = _raw_stream(stream, self._index)
        return _decode4.kv4_attend(self._raw, self._index, self.head_dim, q, table, lens,
                                   self._scale if scale is None else scale, out, lse, stream)


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

    def per_request(self) -> "PagePlan":
        """This plan of a step in which a request gains at most one token, with a
        slot and a position for each request (cu None) in place of each new
        token: slot -1 where a request gains none (idle, finished, rolled back;
        all of them where the plan did not fit), position that of its newest
        token.  On the current stream."""
        if self.cu is None:
            return self
        positions = (self.lens - 1).clamp_(min=0)
        if self.slots.numel() == 0:
            return self._replace(cu=None, slots=torch.full_like(self.lens, -1, dtype=torch.int64), positions=positions)
        at = self.cu[:-1].clamp(max=self.slots.numel() - 1).long()
        slots = torch.where(self.cu[1:] > self.cu[:-1], self.slots.gather(0, at), -1)
        return self._replace(cu=None, slots=slots, positions=positions)


def plan_pages(lens: torch.Tensor, delta: torch.Tensor, table: torch.Tensor, free_pages: torch.Tensor,
               free_count: torch.Tensor, page_size: int, max_new: int, commit: bool = False,
               stream=None) -> PagePlan:
    """Pages, slots and positions of the tokens that B requests gain (delta >
    0) or drop (delta < 0) in a step, on the GPU.  lens, delta: int32 [B];
    table: int32 [B, cols], updated in place; free_pages: int32, updated in
    place beyond what is in use; free_count: int32 [1].  commit: lens and
    free_count are updated in place too (and returned); otherwise the new ones
    are new tensors and the same plan may be made again."""
    made = None
    if stream is not None and isinstance(lens, torch.Tensor) and lens.is_cuda:
        made = (_empty(lens.device, (2 * lens.numel() + 3 + max(0, max_new),), torch.int32, stream),
                _empty(lens.device, (max(0, max_new),), torch.int64, stream))
        stream = _raw_stream(stream, lens.device.index)
    return PagePlan._make(_decode4.plan_pages(lens, delta, table, free_pages, free_count, page_size, max_new,
                                              commit, made, stream))


class Attention4:
    """One attention sub-layer of a decoder block in 4 bits, for tokens of a
    decode step: the query, key and value projections, the new rows into a
    cache of its own, the attention over it and the output projection.

    w_qkv: bf16 [d, (n_heads + 2 n_kv_heads) head_dim] (queries, then keys, then
    values), w_o: bf16 [n_heads head_dim, d]; quantised by pack_proxy's rule.
    rotate: optional callable (q, k, positions) -> (q, k) that applies the
    model's position encoding to q [n, n_heads, head_dim] and k [n, n_kv_heads,
    head_dim] (on the step's stream).  The cache has num_pages pages of page_size tokens; which rows a
    step's tokens take is the caller's plan (plan_pages), shared by all layers.
    """

    def __init__(self, w_qkv: torch.Tensor, w_o: torch.Tensor, n_heads: int, n_kv_heads: int,
                 head_dim: int, num_pages: int, page_size: int = 64, rotate=None, stream=None):
        if n_heads < 1 or n_kv_heads < 1 or n_heads % n_kv_heads:
            raise ValueError(f"n_heads={n_heads} must be a multiple of n_kv_heads={n_kv_heads}")
        if w_qkv.dim() != 2 or w_qkv.shape[1] != (n_heads + 2 * n_kv_heads) * head_dim \
                or tuple(w_o.shape) != (n_heads * head_dim, w_qkv.shape[0]):
            raise ValueError("inconsistent weight shapes")
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, n_kv_heads, head_dim
        self.qkv, self.out = Linear4(w_qkv, stream=stream), Linear4(w_o, stream=stream)
        self.cache = KVCache4.zeros(num_pages, n_kv_heads, page_size, head_dim, device=w_qkv.device)
        self.rotate = rotate

    def step(self, x: torch.Tensor, plan: PagePlan, table: torch.Tensor, stream=None) -> torch.Tensor:
        """x [B, d], the new token of each request (B <= 16) -> [B, d].  A request
        may gain none in the plan (idle, finished): its row of x is not cached
        and attends to what it has (zeros if that is nothing).  More than one
        is not looked for (the plan is on the device): verify drafted tokens
        with the operators themselves.  A plan whose status is 1 caches
        nothing.  Calls for several layers share plan.per_request(), which each
        would work out again."""
        if stream is not None:  # what the step makes on the way belongs to its stream
            with on_stream(stream, self.qkv.device):
                return self.step(x, plan, table)
        plan = plan.per_request()
        B, D = x.shape[0], self.head_dim
        # (what attend would refuse must not have cached rows)
        if x.dim() != 2 or plan.lens.numel() != B or plan.slots.numel() < B or table.dim() != 2 or table.shape[0] != B:
            raise ValueError(f"x {tuple(x.shape)}, a plan of {plan.lens.numel()} requests and a table "
                             f"{tuple(table.shape)} do not belong together")
        heads = self.qkv.forward(x).view(B, self.n_heads + 2 * self.n_kv_heads, D)
        q, k, v = heads.split_with_sizes([self.n_heads, self.n_kv_heads, self.n_kv_heads], 1)
        if self.rotate is not None:
            q, k = self.rotate(q, k, plan.positions[:B])
        self.cache.append(k, v, plan.slots[:B])
        o = self.cache.attend(q, table, plan.lens)
        return self.out.forward(o.view(B, self.n_heads * D))

    def close(self):
        self.qkv.close()
        self.out.close()
        self.cache.close()
