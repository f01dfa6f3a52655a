"""The operators around a ragged verification step: norm and rotation of heads, the append to a paged
key/value cache held in 4 bits, attention over it, and the penalties, biases and masks of the logits.

All take the ragged rows of the scheduler and the verification: request r owns rows row_off[r] ..
row_off[r+1]-1 (``tgt_off``), the last of its kv_len[r] tokens.  The functions here name the arguments;
csrc/binding.cpp checks them, allocates outputs and workspaces with torch and calls the C ABI on the
current stream (a kernel may take 3 us: the same checks in Python took 13 us a call), or on ``stream``,
where it is given: what the call allocates belongs to that stream then, and its inputs have to be ready
there and stay until it is done with them.  Nothing is synchronised.  Pass ``status`` (one int32 on the device, see ``check``) to share the error word
of a step; without it each call makes its own.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import numpy as np
import torch

import speculative_decoding_draft_gb300 as _ds

class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Rope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("gain", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


class _ByteCache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32)]


class _Ragged(ctypes.Structure):
    _fields_ = [("row_off", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("B", ctypes.c_int64), ("rows", ctypes.c_int64), ("max_pages", ctypes.c_int64)]


class _Penalties(ctypes.Structure):
    _fields_ = [("hist", ctypes.c_void_p), ("hist_len", ctypes.c_void_p), ("prompt_len", ctypes.c_void_p),
                ("draft_tok", ctypes.c_void_p), ("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("bias_tok", ctypes.c_void_p), ("bias_val", ctypes.c_void_p),
                ("mask", ctypes.c_void_p), ("hist_cap", ctypes.c_int64), ("draft_cap", ctypes.c_int64),
                ("bias_cap", ctypes.c_int64)]


def declare(L) -> None:
    """Argument types of the library's entry points (called by ``lib()``)."""
    P, i64, i32, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    H, R, C, W, C8 = (ctypes.POINTER(t) for t in (_Heads, _Rope, _Cache, _Ragged, _ByteCache))
    for name, args in (
            ("dspark_attn_norm_rope", [H, H, i64, i32, i32, i32, i32, P, R, P, P, f, P, P, P, P]),
            ("dspark_attn_append", [H, H, H, i32, i32, C, W, P, R, P, P, f, P, P, P]),
            ("dspark_attn_cache_read", [C, W, P, P, P, P, P, P]),
            ("dspark_attn_paged", [H, i32, i32, C, W, i64, f, i32, i64, P, P, P, ctypes.c_size_t, P, P]),
            ("dspark_logits_penalize", [P, i32, i64, i64, i64, P, ctypes.POINTER(_Penalties), P, P, P]),
            ("dspark_attn_prompt", [H, H, H, i64, i64, i64, i32, i32, i32, i32, P, P, f, i32, i64, P, P, P,
                                    ctypes.c_size_t, P, P]),
            ("dspark_attn_append_byte", [H, H, H, i32, i32, C8, W, P, R, P, P, f, P, P, P]),
            ("dspark_attn_cache_read_byte", [C8, W, i32, P, P, P, P]),
            ("dspark_attn_paged_byte", [H, i32, i32, C8, W, i64, f, i32, i64, P, P, P, ctypes.c_size_t, P, P])):
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    L.dspark_attn_paged_workspace_bytes.argtypes = [i32, C, W, i64]
    L.dspark_attn_paged_workspace_bytes.restype = ctypes.c_size_t
    L.dspark_attn_paged_byte_workspace_bytes.argtypes = [i32, C8, W, i64]
    L.dspark_attn_paged_byte_workspace_bytes.restype = ctypes.c_size_t
    L.dspark_attn_prompt_workspace_bytes.argtypes = [i64, i64, i64, i32, i32, i32]
    L.dspark_attn_prompt_workspace_bytes.restype = ctypes.c_size_t


_binding = None


def _native():
    """The native binding (csrc/binding.cpp), which checks the arguments and calls the loaded library."""
    global _binding
    if _binding is None:
        L = _ds.lib()
        try:
            from . import _binding as native
        except ImportError as e:
            raise _ds.DsparkUnavailable(f"the native binding is not built ({e}); run "
                                        "`python -c 'import __graft_entry__ as g; g.build()'`") from None
        native.init(*(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in (
            "dspark_attn_norm_rope", "dspark_attn_append", "dspark_attn_cache_read",
            "dspark_attn_paged_workspace_bytes", "dspark_attn_paged", "dspark_logits_penalize",
            "dspark_attn_prompt_workspace_bytes", "dspark_attn_prompt", "dspark_attn_append_byte",
            "dspark_attn_cache_read_byte", "dspark_attn_paged_byte_workspace_bytes", "dspark_attn_paged_byte")))
        _binding = native
    return _binding


def _done(result, where):
    """The dict of a call, or the entry point's error."""
    if type(result) is int:
        raise _ds.DsparkError(result, where)
    return result


def _raw(stream):
    if stream is None:
        return None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
class Rope:
    """Rotary positions of the first ``rotary_dim`` dimensions of a head (a multiple of 16).

    layout: "half" turns dimensions (i, i + rotary_dim/2), "interleaved" (2i, 2i + 1).
    scaling, for contexts past the ``original_len`` that a model was trained on, by ``factor``:
      "none"; "linear": frequencies / factor; "ntk": base * factor^(d / (d - 2));
      "yarn": pairs with over ``beta_fast`` turns in original_len stay, those under ``beta_slow`` are divided
      by factor, a linear ramp lies between, and cos and sin are multiplied by 0.1 ln(factor) + 1
      (or by ``gain``, where it is given).
    ``inv_freq`` (float64) in place of base and scaling takes any other schedule of frequencies.
    """

    def __init__(self, rotary_dim: int, *, base: float = 10000.0, layout: str = "half", scaling: str = "none",
                 factor: float = 1.0, original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 gain: Optional[float] = None, inv_freq: Optional[torch.Tensor] = None, device="cuda"):
        if rotary_dim < 16 or rotary_dim % 16:
            raise ValueError(f"rotary_dim must be a multiple of 16, got {rotary_dim}")
        if layout not in ("half", "interleaved"):
            raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
        if scaling not in ("none", "linear", "ntk", "yarn"):
            raise ValueError(f"scaling must be 'none', 'linear', 'ntk' or 'yarn', got {scaling!r}")
        if not base > 1 or not factor > 0:
            raise ValueError("base must be above 1 and factor above 0")
        if scaling == "yarn" and original_len < 1:
            raise ValueError("scaling 'yarn' needs original_len")
        n = rotary_dim // 2
        own_gain = 1.0
        if inv_freq is None:
            i = np.arange(n, dtype=np.float64)
            if scaling == "ntk":
                base = base * factor ** (rotary_dim / (rotary_dim - 2))
            inv = base ** (-2 * i / rotary_dim)
            if scaling == "linear":
                inv = inv / factor
            elif scaling == "yarn":
                def pair_of(turns):   # the pair that makes so many turns in original_len positions
                    return rotary_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))

                low, high = max(math.floor(pair_of(beta_fast)), 0), min(math.ceil(pair_of(beta_slow)), rotary_dim - 1)
                ramp = ((i - low) / max(high - low, 0.001)).clip(0, 1)
                inv = inv * (1 - ramp) + inv / factor * ramp
                own_gain = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
        else:
            inv = inv_freq.detach().to("cpu", torch.float64).numpy()
            if inv.shape != (n,):
                raise ValueError(f"inv_freq must have shape ({n},)")
        self.inv_freq, self.rotary_dim, self.layout = torch.from_numpy(inv), rotary_dim, layout
        self.gain = own_gain if gain is None else float(gain)
        # turns per position in 64-bit fixed point, wrapped: whole turns say nothing
        turn = inv / (2 * math.pi)
        turn = np.minimum((turn - np.rint(turn)) * 2.0 ** 64, 2.0 ** 63 - 1024)   # [-1/2, 1/2): a signed fraction
        self.turns = torch.from_numpy(np.rint(turn).astype(np.int64)).to(device)
        self._c = _Rope(self.turns.data_ptr(), rotary_dim, layout == "interleaved", self.gain)
        self._at, self.device = ctypes.addressof(self._c), self.turns.get_device()


def norm_rope(q, k=None, positions=None, rope: Optional[Rope] = None, *, q_weight=None, k_weight=None,
              eps: float = 1e-6, out: Optional[dict] = None, status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Norm and rotation of query and key heads in one pass (C ABI dspark_attn_norm_rope).

    q [rows, Hq, D], k [rows, Hkv, D] or None (float32, bfloat16 or float16; D a multiple of 16 to 256; rows and
    heads may be strided, as in a view of a fused projection), positions [rows] int32 (with a rope), q_weight /
    k_weight [D], on a 16-byte boundary, or None (no norm).  Returns q and k of the inputs' shape, contiguous (``out`` may name the
    inputs themselves where those are contiguous).
    """
    turn = None if rope is None else _of(rope, Rope, "rope")._at
    if turn is not None and isinstance(q, torch.Tensor) and rope.device != q.get_device():
        raise ValueError(f"rope must be on {q.device}, got {rope.turns.device}")
    return _done(_native().norm_rope(q, k, positions, turn, q_weight, k_weight, eps, out, status, _raw(stream)),
                 "dspark_attn_norm_rope")


def _of(x, kind, name):
    if not isinstance(x, kind):
        kinds = kind if isinstance(kind, tuple) else (kind,)
        raise TypeError(f"{name} must be a {' or a '.join(k.__name__ for k in kinds)}")
    return x


# ---------------------------------------------------------------------------
# the paged cache
# ---------------------------------------------------------------------------
class PagedCache:
    """A paged key/value cache in 4 bits: uint8 [pages, kv_heads, page_size/16, 18 D] (see include/dspark.h for a
    tile's layout): e2m1 elements, an e4m3 scale for 16 dimensions, a power of two for the whole cache (k_scale,
    v_scale; scales lie between 2^-9 and 448 times it, so it should lie near the largest magnitudes / 2688 up to
    about their size).  4.5 bits an element."""

    def __init__(self, data: torch.Tensor, page_size: int, *, k_scale: float = 1.0, v_scale: float = 1.0):
        if not isinstance(data, torch.Tensor) or not data.is_cuda or data.dtype != torch.uint8:
            raise TypeError("data must be a uint8 CUDA tensor")
        if data.dim() != 4 or not data.is_contiguous() or data.data_ptr() % 16:
            raise ValueError("data must be contiguous [pages, kv_heads, page_size/16, 18 D], 16-byte aligned")
        if page_size < 16 or page_size % 16 or page_size > 4096 or data.shape[2] != page_size // 16:
            raise ValueError(f"page_size {page_size} does not fit data of shape {tuple(data.shape)}")
        if data.shape[3] not in (18 * 64, 18 * 128):
            raise ValueError("the cache holds heads of 64 or 128 dimensions")
        for name, x in (("k_scale", k_scale), ("v_scale", v_scale)):
            if not (x > 0 and math.isfinite(x) and math.frexp(x)[0] == 0.5):
                raise ValueError(f"{name} must be a power of two, got {x}")
        self.data, self.page_size, self.k_scale, self.v_scale = data, page_size, float(k_scale), float(v_scale)
        self.pages, self.kv_heads, self.head_dim = data.shape[0], data.shape[1], data.shape[3] // 18
        self.device = data.get_device()
        self._c = _Cache(data.data_ptr(), self.pages, self.kv_heads, self.head_dim, page_size, k_scale, v_scale)
        self._at = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, page_size: int = 64, *, k_scale: float = 1.0,
              v_scale: float = 1.0, device="cuda") -> "PagedCache":
        """A cache of zeros."""
        if page_size < 16 or page_size % 16 or page_size > 4096:
            raise ValueError(f"page_size must be a multiple of 16 to 4096, got {page_size}")
        if head_dim not in (64, 128):
            raise ValueError("the cache holds heads of 64 or 128 dimensions")
        return cls(torch.zeros(pages, kv_heads, page_size // 16, 18 * head_dim, dtype=torch.uint8, device=device),
                   page_size, k_scale=k_scale, v_scale=v_scale)


class PagedCache8:
    """A paged key/value cache in 8 bits: data uint8 [pages, kv_heads, 2, page_size, D] (keys, then values; e4m3
    elements) and scales uint8 [pages, kv_heads, 2, page_size/16], a power of two for a block of 16 tokens of a head
    (see include/dspark.h for the places of a token's elements).  No range has to be chosen: a block's scale follows
    its loudest token."""

    def __init__(self, data: torch.Tensor, scales: torch.Tensor):
        for name, x in (("data", data), ("scales", scales)):
            if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype != torch.uint8:
                raise TypeError(f"{name} must be a uint8 CUDA tensor")
        if data.dim() != 5 or data.shape[2] != 2 or not data.is_contiguous() or data.data_ptr() % 16:
            raise ValueError("data must be contiguous [pages, kv_heads, 2, page_size, D], 16-byte aligned")
        pages, heads, _, page_size, dim = data.shape
        if page_size < 16 or page_size % 16 or page_size > 4096:
            raise ValueError(f"page_size must be a multiple of 16 to 4096, got {page_size}")
        if dim not in (64, 128):
            raise ValueError("the cache holds heads of 64 or 128 dimensions")
        if scales.shape != (pages, heads, 2, page_size // 16) or not scales.is_contiguous() or scales.device != data.device:
            raise ValueError(f"scales must be contiguous {(pages, heads, 2, page_size // 16)} on {data.device}")
        self.data, self.scales, self.page_size = data, scales, page_size
        self.pages, self.kv_heads, self.head_dim = pages, heads, dim
        self.device = data.get_device()
        self._c = _ByteCache(data.data_ptr(), scales.data_ptr(), pages, heads, dim, page_size)
        self._at = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, head_dim: int, page_size: int = 64, *, device="cuda") -> "PagedCache8":
        """A cache of zeros."""
        if page_size < 16 or page_size % 16 or page_size > 4096:
            raise ValueError(f"page_size must be a multiple of 16 to 4096, got {page_size}")
        return cls(torch.zeros(pages, kv_heads, 2, page_size, head_dim, dtype=torch.uint8, device=device),
                   torch.zeros(pages, kv_heads, 2, page_size // 16, dtype=torch.uint8, device=device))


_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def cache_append(cache, k, v, row_off, kv_len, page_table, *, positions=None, rope: Optional[Rope] = None,
                 k_weight=None, q=None, q_weight=None, eps: float = 1e-6, out: Optional[dict] = None,
                 status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Append the rows' keys and values to the cache, keys normed and rotated on the way (C ABI dspark_attn_append;
    to a PagedCache8 dspark_attn_append_byte).

    k, v [rows, Hkv, D]; row_off [B+1], kv_len [B] (with these rows among them), page_table [B, max_pages], all
    int32; positions [rows] int32 or None (a row's place in its request); with q [rows, Hq, D] the queries are
    normed and rotated in the same pass and returned as q (contiguous).  Two rows must not name the same place, and in
    a PagedCache8 a block of 16 tokens that is written to belongs to one request.
    """
    _of(cache, (PagedCache, PagedCache8), "cache")
    turn = None if rope is None else _of(rope, Rope, "rope")._at
    if turn is not None and rope.device != cache.device:
        raise ValueError(f"rope must be on {cache.data.device}, got {rope.turns.device}")
    if isinstance(cache, PagedCache8):
        return _done(_native().append_byte(cache._at, cache.device, k, v, row_off, kv_len, page_table, positions, turn,
                                           k_weight, q, q_weight, eps, out, status, _raw(stream)), "dspark_attn_append_byte")
    return _done(_native().append(cache._at, cache.device, k, v, row_off, kv_len, page_table, positions, turn, k_weight, q,
                                  q_weight, eps, out, status, _raw(stream)), "dspark_attn_append")


def cache_read(cache, row_off, kv_len, page_table, rows: int, *, dtype: Optional[torch.dtype] = None,
               out: Optional[dict] = None, status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """What the cache holds of the rows' tokens (C ABI dspark_attn_cache_read): k, v [rows, Hkv, D] and k_scale,
    v_scale [rows, Hkv, D/16], float8_e4m3fn and exact; an element's value is element * scale * the cache's scale.
    A request's whole text: row_off over kv_len rows each.

    Of a PagedCache8 the values themselves (C ABI dspark_attn_cache_read_byte): k, v [rows, Hkv, D] of ``dtype``
    (bfloat16 unless given, or float32: exact; float16: rounded), as attend_prompt takes them."""
    _of(cache, (PagedCache, PagedCache8), "cache")
    if isinstance(cache, PagedCache8):
        code = _DTYPES.get(torch.bfloat16 if dtype is None else dtype)
        if code is None:
            raise TypeError(f"dtype must be torch.bfloat16, torch.float32 or torch.float16, got {dtype}")
        return _done(_native().read_byte(cache._at, cache.device, row_off, kv_len, page_table, rows, code, out, status,
                                         _raw(stream)), "dspark_attn_cache_read_byte")
    if dtype is not None:
        raise TypeError("a cache in 4 bits is read as elements and scales: no dtype")
    return _done(_native().read(cache._at, cache.device, row_off, kv_len, page_table, rows, out, status, _raw(stream)),
                 "dspark_attn_cache_read")


def attend_paged(q, cache, row_off, kv_len, page_table, *, scale: Optional[float] = None,
                 causal: bool = True, window: int = 0, max_rows: Optional[int] = None, want_lse: bool = False,
                 out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Attention of ragged rows over the cache (C ABI dspark_attn_paged; over a PagedCache8 dspark_attn_paged_byte).

    q [rows, Hq, D] bfloat16 or float16 (rows and heads may be strided), Hq a multiple of the cache's heads;
    scale: 1/sqrt(D) unless given.  Row j of request r sees its tokens up to itself (causal) or all kv_len[r], and
    with window > 0 only the last ``window`` of them (pages before every row's window may be gone: their entries in
    page_table are not read); a row that sees nothing gets 0 and lse -inf.  max_rows: the
    most rows of a request (default: what ``rows`` allows; smaller is faster).  Returns out [rows, Hq, D] and,
    with want_lse, lse [rows, Hq] float32.
    """
    _of(cache, (PagedCache, PagedCache8), "cache")
    if isinstance(cache, PagedCache8):
        return _done(_native().paged_byte(q, cache._at, cache.device, row_off, kv_len, page_table, scale, causal, window,
                                          max_rows, want_lse, out, workspace, status, _raw(stream)), "dspark_attn_paged_byte")
    return _done(_native().paged(q, cache._at, cache.device, row_off, kv_len, page_table, scale, causal, window, max_rows,
                                 want_lse, out, workspace, status, _raw(stream)), "dspark_attn_paged")


# ---------------------------------------------------------------------------
# whole prompts
# ---------------------------------------------------------------------------
def attend_prompt(q, k, v, row_off, *, kv_off=None, scale: Optional[float] = None, causal: bool = True, window: int = 0,
                  want_lse: bool = False, out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Attention of whole prompts over keys and values in 16 bits (C ABI dspark_attn_prompt).

    q [rows, Hq, D], k, v [kv_rows, Hkv, D] bfloat16 or float16, D 64 or 128, Hq a multiple of Hkv (rows and heads may
    be strided, as in a view of a fused projection or of [heads, rows, D], but k and v not broadcast); row_off [B+1]
    int32: request r's queries.  kv_off [B+1] int32 (default: row_off): its keys and values, of which the queries are
    the last where there are more (a later piece of a prompt over its earlier ones).  scale: 1/sqrt(D) unless given.
    Row j of n sees its request's m tokens up to m - n + j (causal) or all, and with window > 0 only the last
    ``window`` of them; a row that sees nothing gets 0 and lse -inf, and what masked tokens hold (infinities, NaN)
    changes nothing.  Returns out [rows, Hq, D] (``out`` may name q itself where that is contiguous) and, with want_lse, lse [rows, Hq] float32.  Rows
    at and past row_off[B] are left alone.
    """
    return _done(_native().prompt(q, k, v, row_off, kv_off, scale, causal, window, want_lse, out, workspace, status,
                                  _raw(stream)), "dspark_attn_prompt")


# ---------------------------------------------------------------------------
# the logits
# ---------------------------------------------------------------------------
def penalize_logits(logits, row_off, hist, hist_len, prompt_len, repetition, presence, frequency, *, draft_tok=None,
                    bias_tok=None, bias_val=None, mask=None, out: Optional[dict] = None,
                    status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Penalties, biases and grammar masks of ragged rows of logits (C ABI dspark_logits_penalize).

    logits [rows, V] float32 or bfloat16; row_off [B+1], hist [B, cap], hist_len, prompt_len [B] int32 (token ids:
    the prompt, then the output); repetition, presence, frequency [B] float32; draft_tok [B, K] int32 or None (row j
    of a request counts its first j draft tokens as output); bias_tok [B, n] int32 (-1 pads) with bias_val [B, n]
    float32; mask int32 [rows, ceil(V/32)], bit v%32 of word v//32 allows token v.  Returns logits (``out`` may
    name the input).
    """
    return _done(_native().penalize(logits, row_off, hist, hist_len, prompt_len, repetition, presence, frequency, draft_tok,
                                    bias_tok, bias_val, mask, out, status, _raw(stream)), "dspark_logits_penalize")
