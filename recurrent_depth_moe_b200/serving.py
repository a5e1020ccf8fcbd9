"""Serving operators over librdt: the paged key / value cache (written, read back, attended by
one new token) and the sampled next token.

As in api.py each function checks placement, dtype and layout of its tensors, allocates outputs
and workspace with torch when none is given, and calls the C entry point of the same name on
the current stream of the tensors' device.  There is no CPU or eager fallback."""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Union

import torch

from . import _native as N

_DT = {"fp32": (0, torch.float32), "bf16": (1, torch.bfloat16)}
_NAME = {torch.float32: "fp32", torch.bfloat16: "bf16"}
E4M3 = torch.float8_e4m3fn
_PARAMS = ("temperature", "top_k", "top_p", "min_p")


def _lib():
    if not torch.cuda.is_available():
        raise RuntimeError("recurrent_depth_moe_b200 needs a CUDA device (B200, sm_100a); no CPU path exists")
    return N.load()


_fns: dict = {}
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda i: torch.cuda.current_stream(i).cuda_stream


def _call(name: str, device: torch.device, *args):
    """The entry point on the device's current stream, with that device current.  (A serving step
    makes these calls every few microseconds: the entry point is looked up once.)"""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_lib(), name)
    i = device.index
    if i == _current_device():
        rc = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(i))
    if rc != N.RDT_OK:
        raise N.RdtError(name, rc)


def _check(t, name: str, dtype, shape, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or t.shape != shape or \
            not t.is_contiguous() or (device is not None and t.device != device):
        got = f"{t.device} {t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()}" if isinstance(t, torch.Tensor) \
            else type(t).__name__
        raise ValueError(f"{name}: expected contiguous {device or 'CUDA'} {dtype} {tuple(shape)}, got {got}")


def _check_rows(t, name: str, dtype, shape, device):
    """A [rows, heads, hd] tensor whose rows are contiguous; the rows may be spaced apart."""
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype != dtype or t.shape != shape:
        got = f"{t.device} {t.dtype} {tuple(t.shape)}" if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: expected {device} {dtype} {tuple(shape)}, got {got}")
    rows, heads, hd = shape
    w = heads * hd
    if t.is_contiguous():
        return w
    st = t.stride()
    if (hd > 1 and st[2] != 1) or (heads > 1 and st[1] != hd) or (rows > 1 and st[0] < w):
        raise ValueError(f"{name}: each row must be contiguous and the rows must not overlap, got strides {st}")
    return st[0] if rows > 1 else w


class PagedKVCache:
    """Paged K/V cache of the recurrent loops (or, with n_loops 1, of one block), GQA.

    k, v [n_loops, n_pages, Hkv, page_size, hd] in the model dtype, or in float8_e4m3fn with
    k_exp, v_exp uint8 [n_loops, n_pages, Hkv, page_size] (a row is q * 2^(exp - 127)); dtype
    ("fp32" | "bf16") is the model dtype, needed for an e4m3 cache.  page_table int32
    [batch, max_pages]: position t of sequence b is slot t % page_size of page
    page_table[b, t // page_size].  The tensors are the caller's; the table may be changed in
    place between calls.  Out-of-range table entries and positions, in these calls and in the
    model's over the cache, are recorded in a status word (read_status)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                 k_exp: Optional[torch.Tensor] = None, v_exp: Optional[torch.Tensor] = None,
                 dtype: Optional[str] = None):
        if not isinstance(k, torch.Tensor) or k.dim() != 5:
            raise ValueError("k: expected a [n_loops, n_pages, Hkv, page_size, hd] tensor")
        quant = k.dtype == E4M3
        if dtype is None:
            if quant:
                raise ValueError("dtype: an e4m3 cache needs the model dtype ('fp32' or 'bf16')")
            dtype = _NAME.get(k.dtype)
        if dtype not in _DT or (not quant and k.dtype != _DT[dtype][1]):
            raise ValueError(f"k: expected float8_e4m3fn or the model dtype ({dtype}), got {k.dtype}")
        dev = k.device
        _check(k, "k", k.dtype, k.shape)
        _check(v, "v", k.dtype, k.shape, dev)
        if quant:
            _check(k_exp, "k_exp", torch.uint8, k.shape[:4], dev)
            _check(v_exp, "v_exp", torch.uint8, k.shape[:4], dev)
        elif k_exp is not None or v_exp is not None:
            raise ValueError("k_exp, v_exp: only an e4m3 cache has exponent bytes")
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table: expected an int32 [batch, max_pages] tensor")
        _check(page_table, "page_table", torch.int32, page_table.shape, dev)
        self._k, self._v, self._k_exp, self._v_exp, self._table = k, v, k_exp, v_exp, page_table
        self.dtype, self.quantised, self.device = dtype, quant, dev
        self.torch_dtype = _DT[dtype][1]
        self.n_loops, self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.batch, self.max_pages = page_table.shape
        s = N.rdt_paged_cache()
        s.k, s.v, s.page_table = k.data_ptr(), v.data_ptr(), page_table.data_ptr()
        s.k_exp, s.v_exp = (k_exp.data_ptr(), v_exp.data_ptr()) if quant else (None, None)
        s.dtype, s.kv_type = _DT[dtype][0], int(quant)
        s.n_loops, s.n_pages, s.page_size = self.n_loops, self.n_pages, self.page_size
        s.n_kv_heads, s.head_dim, s.batch, s.max_pages = self.n_kv_heads, self.head_dim, self.batch, self.max_pages
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)
        self._status = s.status = self.status.data_ptr()
        self._struct = s
        self._ref = ctypes.byref(s)

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_exp = property(lambda self: self._k_exp)
    v_exp = property(lambda self: self._v_exp)
    page_table = property(lambda self: self._table)

    @property
    def t_max(self) -> int:
        """Positions one sequence's table row can hold."""
        return self.max_pages * self.page_size

    def struct(self) -> N.rdt_paged_cache:
        return self._struct

    @staticmethod
    def alloc(cfg, n_loops: int, batch: int, t_max: int, page_size: int = 64, quantised: bool = False,
              n_pages: Optional[int] = None, page_table: Optional[torch.Tensor] = None, device=None) -> "PagedKVCache":
        """Zeroed pages for `batch` sequences of up to t_max positions.  Without a page_table
        every sequence gets its own pages, one after another (n_pages, if given, may hold more); with
        one (int32 [batch, max_pages]) n_pages says how many pages to hold."""
        if cfg.attn_type != "gqa":
            raise ValueError("a paged cache holds GQA keys and values")
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if page_table is None:
            per = -(-t_max // page_size)
            if n_pages is not None and n_pages < batch * per:
                raise ValueError(f"n_pages: {batch} sequences of {t_max} positions need {batch * per}, got {n_pages}")
            page_table = torch.arange(batch * per, dtype=torch.int32, device=device).reshape(batch, per)
            n_pages = batch * per if n_pages is None else n_pages
        elif n_pages is None:
            raise ValueError("n_pages: needed with a page_table")
        shape = (n_loops, n_pages, cfg.n_kv_heads, page_size, cfg.dim // cfg.n_heads)
        dt = E4M3 if quantised else _DT[cfg.dtype][1]
        k, v = torch.zeros(shape, dtype=dt, device=device), torch.zeros(shape, dtype=dt, device=device)
        ke = torch.zeros(shape[:4], dtype=torch.uint8, device=device) if quantised else None
        ve = torch.zeros_like(ke) if quantised else None
        return PagedKVCache(k, v, page_table, ke, ve, dtype=cfg.dtype)

    def read_status(self) -> int:
        """Synchronise, read and clear the cache's device status word."""
        with torch.cuda.device(self.device):
            return _lib().rdt_read_device_status(self.status.data_ptr(),
                                                 torch.cuda.current_stream(self.device).cuda_stream)


def paged_kv_write(k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, cache: PagedKVCache, seq: int = 1,
                   loop: int = 0) -> None:
    """rdt_paged_kv_write: rows k, v [N, Hkv, hd] (model dtype; rows may be slices of wider
    rows) into loop `loop`, row i at position positions[i] (int32 [N]; negative: a padding row)
    of sequence i // seq."""
    n, c = positions.numel(), cache
    ld = _check_rows(k, "k", c.torch_dtype, (n, c.n_kv_heads, c.head_dim), c.device)
    if _check_rows(v, "v", c.torch_dtype, (n, c.n_kv_heads, c.head_dim), c.device) != ld:
        raise ValueError("k and v must have the same row stride")
    _check(positions, "positions", torch.int32, (n,), c.device)
    _call("rdt_paged_kv_write", c.device, c._ref, loop, k.data_ptr(), v.data_ptr(), ld, positions.data_ptr(), n, seq,
          c._status)


def paged_kv_read(lens: torch.Tensor, cache: PagedKVCache, t_out: Optional[int] = None, loop: int = 0,
                  out: Optional[tuple] = None) -> tuple:
    """rdt_paged_kv_read: positions 0 .. lens[b] - 1 of loop `loop` as (k, v)
    [B, Hkv, t_out, hd] in the model dtype.  Rows past a sequence's length keep what `out`
    holds, zeros without it; t_out is out's or, without it, the table's capacity."""
    c = cache
    B = lens.numel()
    _check(lens, "lens", torch.int32, (B,), c.device)
    if out is None:
        t_out = c.t_max if t_out is None else t_out
        out = tuple(torch.zeros(B, c.n_kv_heads, t_out, c.head_dim, dtype=c.torch_dtype, device=c.device)
                    for _ in range(2))
    else:
        t_out = out[0].shape[2] if t_out is None and out[0].dim() == 4 else t_out
        for o, name in zip(out, ("out[0]", "out[1]")):
            _check(o, name, c.torch_dtype, (B, c.n_kv_heads, t_out, c.head_dim), c.device)
    _call("rdt_paged_kv_read", c.device, c._ref, loop, lens.data_ptr(), B, t_out, out[0].data_ptr(),
          out[1].data_ptr(), c._status)
    return out


def paged_attention_workspace(cache: PagedKVCache, n_heads: int, batch: Optional[int] = None) -> torch.Tensor:
    """Workspace of paged_attention calls with up to `batch` sequences (the table's rows without
    it), for one call at a time."""
    with torch.cuda.device(cache.device):
        need = int(_lib().rdt_paged_attention_workspace_size(cache._ref, cache.batch if batch is None else batch, n_heads))
    if need == 0:
        raise N.RdtError("rdt_paged_attention_workspace_size", N.RDT_ERR_INVALID_ARG)
    return torch.empty(need, dtype=torch.uint8, device=cache.device)


def paged_attention(q: torch.Tensor, lens: torch.Tensor, cache: PagedKVCache, loop: int = 0,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """rdt_paged_attention: one query token per sequence, q [B, H, hd] (model dtype), over its
    lens[b] cached positions of loop `loop`; scale defaults to 1 / sqrt(hd).  Returns [B, H, hd]."""
    c = cache
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q: expected a [B, H, hd] tensor")
    B, H = q.shape[:2]
    q_ld = _check_rows(q, "q", c.torch_dtype, (B, H, c.head_dim), c.device)
    _check(lens, "lens", torch.int32, (B,), c.device)
    if out is None:
        out = torch.empty(B, H, c.head_dim, dtype=c.torch_dtype, device=c.device)
    o_ld = _check_rows(out, "out", c.torch_dtype, (B, H, c.head_dim), c.device)
    if B == 0:
        return out
    if workspace is None:
        workspace = paged_attention_workspace(c, H, B)
    elif workspace.device != c.device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {c.device}")
    _call("rdt_paged_attention", c.device, c._ref, loop, q.data_ptr(), q_ld, lens.data_ptr(), B, H,
          1.0 / math.sqrt(c.head_dim) if scale is None else float(scale), out.data_ptr(), o_ld, workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), c._status)
    return out


def sample_tokens(logits: torch.Tensor, u: torch.Tensor, temperature: Union[float, torch.Tensor] = 1.0,
                  top_k: Union[int, torch.Tensor] = 0, top_p: Union[float, torch.Tensor] = 1.0,
                  min_p: Union[float, torch.Tensor] = 0.0, out: Optional[torch.Tensor] = None,
                  return_logprob: bool = False):
    """rdt_sample_tokens: one token per row of fp32 logits [n, V] (rows may be spaced apart)
    from one uniform number u[row] in [0, 1).  Each parameter is a number for all rows or a
    tensor with one per row (fp32 [n]; top_k int32 [n]); temperature 0 takes the most likely
    token.  Returns int32 [n], with return_logprob also the drawn tokens' log-probabilities
    among the kept tokens (fp32 [n])."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dtype != torch.float32 or \
            logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError("logits: expected a CUDA float32 [n, vocab] tensor with contiguous rows")
    n, V = logits.shape
    dev = logits.device
    ld = V
    if not logits.is_contiguous():
        if V > 1 and logits.stride(1) != 1:
            raise ValueError("logits: expected a CUDA float32 [n, vocab] tensor with contiguous rows")
        ld = logits.stride(0) if n > 1 else V
        if ld < V:
            raise ValueError("logits: the rows must not overlap")
    shape = (n,)
    _check(u, "u", torch.float32, shape, dev)
    scalars, rows = [1.0, 0, 1.0, 0.0], [None] * 4
    for i, (val, name) in enumerate(zip((temperature, top_k, top_p, min_p), _PARAMS)):
        if isinstance(val, torch.Tensor):
            _check(val, name, torch.int32 if i == 1 else torch.float32, shape, dev)
            rows[i] = val.data_ptr()
        else:
            # (a top_k beyond 32 bits is beyond every vocabulary; below 0 it is refused)
            scalars[i] = max(-1, min(val, 2 ** 31 - 1)) if i == 1 else val
    a = N.rdt_sampling(*scalars, *rows)
    if out is None:
        out = torch.empty(n, dtype=torch.int32, device=dev)
    elif not isinstance(out, torch.Tensor) or out.device != dev or out.dtype != torch.int32 or out.shape != shape or \
            (n > 1 and out.stride(0) < 1):
        raise ValueError(f"out: expected int32 ({n},) on {dev}")
    lp = torch.empty(n, dtype=torch.float32, device=dev) if return_logprob else None
    _call("rdt_sample_tokens", dev, logits.data_ptr(), ld, n, V, u.data_ptr(), ctypes.byref(a), out.data_ptr(),
          out.stride(0) if n > 1 else 1, None if lp is None else lp.data_ptr())
    return (out, lp) if return_logprob else out
