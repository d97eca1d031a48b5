"""Python binding of the prompt side of the cache (``include/hkv_prompt.h``).

Page plans, per-head norms with the position rotation, the attention of a chunk
of new tokens over the paged cache, and the tiers filled from finished prompts.
Argument checks and marshalling only, as in ``hkv``; lengths stay on the device.
"""
from __future__ import annotations

import ctypes as C
import struct
from contextlib import nullcontext
from dataclasses import dataclass
from functools import lru_cache
from typing import Optional

import torch

from .hkv import HkvError, Problem, Tier, _check, lib

DEV_PAGES_FULL = 0x40
MAX_REQUESTS, MAX_TOKENS = 8192, 1 << 22


class _Pages(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("stride_p", C.c_int64), ("stride_h", C.c_int64),
                ("stride_t", C.c_int64), ("pages", C.c_int32), ("page", C.c_int32), ("table", C.c_void_p),
                ("table_stride", C.c_int64), ("table_cols", C.c_int32)]


class _State(C.Structure):
    _fields_ = [("free", C.c_void_p), ("free_count", C.c_void_p), ("held", C.c_void_p)]


class _Chunk(C.Structure):
    _fields_ = [("tokens", C.c_int32), ("q_start", C.c_void_p), ("kv_len", C.c_void_p), ("pos", C.c_void_p),
                ("slot", C.c_void_p)]


class _Rope(C.Structure):
    _fields_ = [("inv_freq", C.c_void_p), ("rot", C.c_int32), ("interleaved", C.c_int32), ("mscale", C.c_float)]


def _signatures():
    P, i32, i64, sz, f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t, C.c_float
    sig = {
        "hkv_page_plan": [i32, P, P, P, P, P, P, P, P, sz, P],
        "hkv_page_release": [i32, P, P, P, P, P, sz, P],
        "hkv_qk_norm_rope": [P, P, i64, P, i64, P, i64, i32, P, P, P, P, P, f32, P, P, P, P, P, sz, P],
        "hkv_chunk_workspace_size": [P, i32, C.POINTER(C.c_size_t)],
        "hkv_chunk_attention": [P, P, i64, i32, P, P, P, P, P, P, sz, P],
        "hkv_fill_tiers": [P, P, P, P, P, P, P, P, P, sz, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = C.c_int


_signatures()


# A call's checks and marshalling cost more host time than its launch, so the
# checks below ask for plain values (sizes, device numbers) and nothing twice.


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _int32(t: torch.Tensor, n: int, what: str):
    """A contiguous int32 vector of n elements."""
    if t.dtype is not torch.int32:
        raise TypeError(f"{what} must be int32")
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n} elements")


def _together(device: int, *tensors):
    """Every tensor (and workspace) on `device` (a number, as get_device gives it)."""
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"on different devices: {device} and {t.get_device()}")


@lru_cache(maxsize=256)
def _problem_c(B, Hq, Hkv, D, dtype, scale, p, bmin, bmax, layout):
    return Problem(B, Hq, Hkv, D, dtype, p, bmin, bmax, scale, layout).c()


def _problem(prob: Problem):
    """The problem's plain values (these calls use neither its inverse temperatures nor its per-unit p)."""
    return C.byref(_problem_c(prob.B, prob.Hq, prob.Hkv, prob.D, prob.dtype, prob.scale, prob.p, prob.bmin, prob.bmax,
                              prob.layout))


def _call(fn, device: int, stream, *args):
    """Call `fn` on the device of its tensors, with that device's current stream unless one is given."""
    if device < 0:
        raise ValueError("the tensors must be on a CUDA device")
    if device == torch.cuda.current_device():
        # (the raw handle: a Stream object costs as much as a launch)
        code = fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            return _call(fn, device, stream, *args)
    if code:
        _check(code, fn.__name__)


def _keep(obj, **fields):
    """Fields of a frozen object: what its tensors were marshalled to."""
    for name, value in fields.items():
        object.__setattr__(obj, name, value)


class StatusWorkspace:
    """Workspace of the calls that use only its status word (256 bytes)."""

    def __init__(self, device, nbytes: int = 256):
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.nbytes = int(nbytes)
        buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=dev)
        self.tensor = buf[(-buf.data_ptr()) % 256:][:self.nbytes]
        self.device = self.tensor.get_device()
        self.ptr = self.tensor.data_ptr()
        self.init()

    def get_device(self) -> int:
        return self.device

    def init(self, stream=None):
        """Zero the workspace (again after a timeout)."""
        _call(lib.hkv_workspace_init, self.device, stream, self.ptr, self.nbytes)

    def status(self, stream=None) -> int:
        """Read and clear the device status word; returns the HKV_DEV_* bits."""
        flags = C.c_uint32(0)
        try:
            _call(lib.hkv_get_status, self.device, stream, self.ptr, C.byref(flags))
        except HkvError as e:
            if e.code not in (4, 5):
                raise
        return int(flags.value)


def status_workspace(device) -> StatusWorkspace:
    return StatusWorkspace(device)


class ChunkWorkspace(StatusWorkspace):
    """Workspace of ``chunk_attention`` for up to `tokens` rows; serves the other calls too."""

    def __init__(self, prob: Problem, tokens: int, device):
        n = C.c_size_t(0)
        dev = torch.device(device)
        with torch.cuda.device(dev) if dev.type == "cuda" else nullcontext():
            _check(lib.hkv_chunk_workspace_size(C.byref(prob.c()), int(tokens), C.byref(n)),
                   "hkv_chunk_workspace_size")
        super().__init__(dev, n.value)


@dataclass(frozen=True, eq=False)
class Pages:
    """The page pool: k, v of [pages, Hkv, page, D] (D contiguous, any other strides, the same for both) and the
    block tables, int32 [B, columns] (rows contiguous; needed by the calls that read tokens back)."""

    k: torch.Tensor
    v: torch.Tensor
    table: Optional[torch.Tensor] = None

    def __post_init__(self):
        k, v, t = self.k, self.v, self.table
        _need(k.dim() == 4 and k.stride(3) == 1, "pages must be [pages, Hkv, page, D] with D contiguous")
        _need(v.shape == k.shape and v.stride() == k.stride() and v.dtype == k.dtype,
              "K and V must share type, shape and strides")
        _together(k.get_device(), v, t)
        if t is not None:
            if t.dtype != torch.int32:
                raise TypeError("table must be int32")
            _need(t.dim() == 2 and (t.shape[1] <= 1 or t.stride(1) == 1), "table must be [B, columns] with contiguous rows")
        # the pool and its tables stay where they are: checked and marshalled once
        c = _Pages(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2), k.shape[0], k.shape[2], _p(t),
                   0 if t is None else max(t.stride(0), t.shape[1]), 0 if t is None else t.shape[1])
        _keep(self, _c=c, _ref=C.byref(c), _shape=(k.shape[1], k.shape[3], k.dtype), _device=k.get_device(),
              _rows=None if t is None else t.shape[0])

    def c(self) -> _Pages:
        return self._c

    def fits(self, prob: Problem, table: bool = True):
        if self._shape != (prob.Hkv, prob.D, prob.dtype):
            if self._shape[2] != prob.dtype:
                raise TypeError(f"pages of {self._shape[2]} for a problem of {prob.dtype}")
            raise ValueError("pages must be [pages, Hkv, page, D] of the problem")
        if table and self._rows != prob.B:
            raise ValueError("the call needs block tables [B, columns]")


@dataclass(frozen=True, eq=False)
class PageState:
    """Allocation state: block tables int32 [B, columns], the stack of free pages int32 [pages] with its count [1]
    (the top is entry count-1), the pages each request holds [B], and the pool's page size and pages."""

    table: torch.Tensor
    free: torch.Tensor
    free_count: torch.Tensor
    held: torch.Tensor
    page: int
    pages: int

    def __post_init__(self):
        B = self.table.shape[0]
        if self.table.dtype != torch.int32:
            raise TypeError("table must be int32")
        _need(self.table.dim() == 2 and (self.table.shape[1] <= 1 or self.table.stride(1) == 1),
              "table must be [B, columns] with contiguous rows")
        _int32(self.free, self.pages, "free")
        _int32(self.free_count, 1, "free_count")
        _int32(self.held, B, "held")
        _together(self.table.get_device(), self.free, self.free_count, self.held)
        t = self.table
        pages = _Pages(None, None, 0, 0, 0, self.pages, self.page, t.data_ptr(), max(t.stride(0), t.shape[1]), t.shape[1])
        c = _State(self.free.data_ptr(), self.free_count.data_ptr(), self.held.data_ptr())
        _keep(self, _pages=pages, _c=c, _pages_ref=C.byref(pages), _ref=C.byref(c), _device=t.get_device(), _rows=B,
              _pool=(t.data_ptr(), t.shape, t.stride(), self.free.data_ptr(), self.page, self.pages))

    @staticmethod
    def allocate(B: int, columns: int, page: int, pages: int, device) -> "PageState":
        """An empty state: every page free (page 0 is given out first), no request holds any."""
        i32 = dict(dtype=torch.int32, device=device)
        return PageState(torch.full((B, columns), -1, **i32), torch.arange(pages - 1, -1, -1, **i32),
                         torch.full((1,), pages, **i32), torch.zeros(B, **i32), page, pages)

    def _same_pool(self, other: "PageState"):
        if other is not self and (self._pool != other._pool or self._device != other._device):
            raise ValueError("the states before and after must share tables, stack and pool")


@dataclass(frozen=True, eq=False)
class Chunk:
    """The rows of one step: q_start [B+1], kv_len [B], pos and slot [tokens], all int32."""

    q_start: torch.Tensor
    kv_len: torch.Tensor
    pos: torch.Tensor
    slot: torch.Tensor

    def __post_init__(self):
        B, T = self.kv_len.shape[0], self.pos.shape[0]
        _int32(self.kv_len, B, "kv_len")
        _int32(self.q_start, B + 1, "q_start")
        _int32(self.pos, T, "pos")
        _int32(self.slot, T, "slot")
        _together(self.kv_len.get_device(), self.q_start, self.pos, self.slot)
        c = _Chunk(T, self.q_start.data_ptr(), self.kv_len.data_ptr(), self.pos.data_ptr(), self.slot.data_ptr())
        _keep(self, _c=c, _ref=C.byref(c), _rows=B, _device=self.kv_len.get_device())

    @staticmethod
    def allocate(B: int, tokens: int, device) -> "Chunk":
        i32 = dict(dtype=torch.int32, device=device)
        return Chunk(torch.zeros(B + 1, **i32), torch.zeros(B, **i32), torch.full((tokens,), -1, **i32),
                     torch.full((tokens,), -1, **i32))


@dataclass(frozen=True, eq=False)
class Rope:
    """The position rotation: pair i turns by pos * inv_freq[i] (fp64 [rot/2]); mscale multiplies cosine and sine."""

    inv_freq: Optional[torch.Tensor]
    rot: int
    interleaved: bool = False
    mscale: float = 1.0

    def __post_init__(self):
        if self.rot:
            _need(self.inv_freq is not None, "inv_freq is missing")
            if self.inv_freq.dtype != torch.float64:
                raise TypeError("inv_freq must be float64")
            _need(self.inv_freq.shape == (self.rot // 2,) and self.inv_freq.is_contiguous(),
                  "inv_freq must be contiguous [rot/2]")
        c = _Rope(_p(self.inv_freq), int(self.rot), int(bool(self.interleaved)), float(self.mscale))
        _keep(self, _c=c, _ref=C.byref(c))

    @staticmethod
    def of_base(rot: int, base: float, device, interleaved: bool = False) -> "Rope":
        """inv_freq[i] = base^(-2 i / rot)."""
        i = torch.arange(0, rot, 2, dtype=torch.float64)
        return Rope((base ** (-i / max(rot, 1))).to(device), rot, interleaved)


def page_plan(ctx_len: torch.Tensor, new_len: torch.Tensor, state: PageState, after: PageState, chunk: Chunk,
              ws: StatusWorkspace, granted: Optional[torch.Tensor] = None, stream=None):
    """Block tables, slot map and positions for new_len[b] tokens behind the ctx_len[b] cached ones of each request
    (int32 [B]; see hkv_page_plan). `after` receives the state: it shares `state`'s tables and stack, and may be
    `state` itself, as chunk.kv_len may be ctx_len. chunk is written; granted: optional int32 [B], the tokens each
    request was given (0 where it was left out)."""
    B = state._rows
    _int32(ctx_len, B, "ctx_len")
    _int32(new_len, B, "new_len")
    if chunk._rows != B:
        raise ValueError("chunk and state must have the same requests")
    if granted is not None:
        _int32(granted, B, "granted")
    state._same_pool(after)
    dev = state._device
    _together(dev, ctx_len, new_len, granted)
    if chunk._device != dev or ws.device != dev:
        raise ValueError("chunk and workspace must be on the state's device")
    _call(lib.hkv_page_plan, dev, stream, B, ctx_len.data_ptr(), new_len.data_ptr(), state._pages_ref, state._ref,
          after._ref, chunk._ref, _p(granted), ws.ptr, ws.nbytes)


def page_release(done: torch.Tensor, state: PageState, after: PageState, ws: StatusWorkspace, stream=None):
    """The pages of the requests with done[b] != 0 (int32 [B]) go back on the stack, each as often as it stands in their
    tables: a page that several requests share must go back with one of them only. See hkv_page_release."""
    B = state._rows
    _int32(done, B, "done")
    state._same_pool(after)
    dev = state._device
    _together(dev, done, ws)
    _call(lib.hkv_page_release, dev, stream, B, done.data_ptr(), state._pages_ref, state._ref, after._ref, ws.ptr,
          ws.nbytes)


def _rows(t: torch.Tensor, dtype: torch.dtype, shape: tuple, what: str) -> int:
    """Row stride of a [tokens, heads, D] tensor with heads and D contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be of the problem's type")
    if t.shape != shape:
        raise ValueError(f"{what} must be {shape}")
    tokens, heads, D = shape
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != D):
        raise ValueError(f"{what}: heads and D must be contiguous")
    return s[0] if tokens > 1 else heads * D


def _contiguous(t: torch.Tensor, dtype: torch.dtype, shape: tuple, what: str):
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {shape}")


def qk_norm_rope(prob: Problem, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor, rope: Rope,
                 q_out: torch.Tensor, ws: StatusWorkspace, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, k_out: Optional[torch.Tensor] = None,
                 v_out: Optional[torch.Tensor] = None, pages: Optional[Pages] = None,
                 slot: Optional[torch.Tensor] = None, stream=None):
    """Per-head RMS norm (with q_weight and k_weight, [D]; left out without them) and position rotation of the
    projected rows q [tokens, Hq, D], k and v [tokens, Hkv, D] at positions pos (int32 [tokens], -1 = skipped row).
    q goes to q_out; k and v to the slots of the pages (pages and slot) or to k_out and v_out, as hkv.append takes
    them. Contiguous q, k and v may be their own outputs. See hkv_qk_norm_rope."""
    T, D, dtype = q.shape[0], prob.D, prob.dtype
    qs = _rows(q, dtype, (T, prob.Hq, D), "q")
    ks = _rows(k, dtype, (T, prob.Hkv, D), "k")
    vs = _rows(v, dtype, (T, prob.Hkv, D), "v")
    _int32(pos, T, "pos")
    _contiguous(q_out, dtype, (T, prob.Hq, D), "q_out")
    if q_weight is not None:
        _contiguous(q_weight, dtype, (D,), "q_weight")
    if k_weight is not None:
        _contiguous(k_weight, dtype, (D,), "k_weight")
    dev = q.get_device()
    if pages is not None:
        if slot is None or k_out is not None or v_out is not None:
            raise ValueError("pages go with slot, and without k_out and v_out")
        pages.fits(prob, table=False)
        _int32(slot, T, "slot")
        if pages._device != dev:
            raise ValueError("pages on another device")
    else:
        if slot is not None or k_out is None or v_out is None:
            raise ValueError("give pages and slot, or k_out and v_out")
        _contiguous(k_out, dtype, (T, prob.Hkv, D), "k_out")
        _contiguous(v_out, dtype, (T, prob.Hkv, D), "v_out")
    _together(dev, k, v, pos, rope.inv_freq, q_out, q_weight, k_weight, k_out, v_out, slot, ws)
    _call(lib.hkv_qk_norm_rope, dev, stream, _problem(prob), q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T,
          pos.data_ptr(), _p(slot), rope._ref, _p(q_weight), _p(k_weight), eps, q_out.data_ptr(), _p(k_out), _p(v_out),
          None if pages is None else pages._ref, ws.ptr, ws.nbytes)


def chunk_attention(prob: Problem, q: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, pages: Pages,
                    out: torch.Tensor, ws: ChunkWorkspace, lse: Optional[torch.Tensor] = None, stream=None):
    """Attention of a chunk of new tokens over the paged cache: rows q_start[b] .. q_start[b+1]-1 of q are the last
    tokens of request b, whose kv_len[b] tokens (those included) are in the pages; each attends up to its own
    position. q, out: [tokens, Hq, D] (out contiguous, apart from q); lse: optional fp32 [tokens, Hq]. See
    hkv_chunk_attention."""
    T = q.shape[0]
    shape = (T, prob.Hq, prob.D)
    qs = _rows(q, prob.dtype, shape, "q")
    _contiguous(out, prob.dtype, shape, "out")
    _int32(q_start, prob.B + 1, "q_start")
    _int32(kv_len, prob.B, "kv_len")
    pages.fits(prob)
    if lse is not None:
        _contiguous(lse, torch.float32, (T, prob.Hq), "lse")
    dev = pages._device
    _together(dev, q, q_start, kv_len, out, lse, ws)
    _call(lib.hkv_chunk_attention, dev, stream, _problem(prob), q.data_ptr(), qs, T, q_start.data_ptr(),
          kv_len.data_ptr(), pages._ref, out.data_ptr(), _p(lse), ws.ptr, ws.nbytes)


_TIER = struct.Struct("PPqqqiP")  # hkv_tier


def _tier(t: Optional[Tier], prob: Problem, device: int, what: str):
    """hkv_tier of a tier of the problem, as bytes."""
    if t is None:
        return None
    k, v, n = t.k, t.v, t.len
    if v is None or k.dtype is not prob.dtype or v.dtype is not prob.dtype:
        raise TypeError(f"{what}: the tier needs K and V of the problem's type")
    shape, s = k.shape, k.stride()
    if len(shape) != 4 or shape[0] != prob.B or shape[1] != prob.Hkv or shape[3] != prob.D or s[3] != 1:
        raise ValueError(f"{what} must be [B, Hkv, cap, D] of the problem with D contiguous")
    if v.shape != shape or v.stride() != s:
        raise ValueError(f"{what}: K and V must share shape and strides")
    _int32(n, prob.B * prob.Hkv, what)
    if k.get_device() != device or v.get_device() != device or n.get_device() != device:
        raise ValueError(f"{what}: tier on another device")
    return _TIER.pack(k.data_ptr(), v.data_ptr(), s[0], s[1], s[2], shape[2], n.data_ptr())


def fill_tiers(prob: Problem, pages: Pages, kv_len: torch.Tensor, dense: Optional[Tier], head: Optional[torch.Tensor],
               sparse: Optional[Tier], ws: StatusWorkspace, take: Optional[torch.Tensor] = None,
               dropped: Optional[torch.Tensor] = None, stream=None):
    """The dense and sparse tiers of finished prompts (all, or those with take[b] != 0), from their pages: what
    kv_len[b] calls of hkv.append leave, started from empty tiers. head, dropped: int32 [B*Hkv]."""
    pages.fits(prob)
    _int32(kv_len, prob.B, "kv_len")
    if take is not None:
        _int32(take, prob.B, "take")
    if head is not None:
        _int32(head, prob.units, "head")
    if dropped is not None:
        _int32(dropped, prob.units, "dropped")
    dev = pages._device
    _together(dev, kv_len, take, head, dropped, ws)
    _call(lib.hkv_fill_tiers, dev, stream, _problem(prob), pages._ref, kv_len.data_ptr(), _p(take),
          _tier(dense, prob, dev, "dense"), _p(head), _tier(sparse, prob, dev, "sparse"), _p(dropped), ws.ptr, ws.nbytes)
