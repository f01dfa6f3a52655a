"""The operators around a ragged verification step: norm and rotation of heads, the append to a paged
key/value cache held in 4 bits, attention over it, and the penalties, biases and masks of the logits.

All take the ragged rows of the scheduler and the verification: request r owns rows row_off[r] ..
row_off[r+1]-1 (``tgt_off``), the last of its kv_len[r] tokens.  As in the rest of the binding, arguments
are checked and marshalled here and the work runs in the library's CUDA kernels on the current stream;
nothing is synchronised.  Pass ``status`` (one int32 on the device, see ``check``) to share the error word
of a step; without it each call makes its own.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

import speculative_decoding_draft_gb300 as _ds

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Rope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("gain", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


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
    H, R, C, W = (ctypes.POINTER(t) for t in (_Heads, _Rope, _Cache, _Ragged))
    for name, args in (
            ("dspark_attn_norm_rope", [H, H, i64, i32, i32, i32, i32, P, R, P, P, f, P, P, P, P]),
            ("dspark_attn_append", [H, H, H, i32, i32, C, W, P, R, P, P, f, P, P, P]),
            ("dspark_attn_cache_read", [C, W, P, P, P, P, P, P]),
            ("dspark_attn_paged", [H, i32, i32, C, W, i64, f, i32, i64, P, P, P, ctypes.c_size_t, P, P]),
            ("dspark_logits_penalize", [P, i32, i64, i64, i64, P, ctypes.POINTER(_Penalties), P, P, P])):
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    L.dspark_attn_paged_workspace_bytes.argtypes = [i32, C, W, i64]
    L.dspark_attn_paged_workspace_bytes.restype = ctypes.c_size_t


# ---------------------------------------------------------------------------
# argument checks.  A call's own time counts where a kernel takes 3 us: the common case is one line of
# comparisons and what is wrong is found out afterwards.  `dev` is a device index.
# ---------------------------------------------------------------------------
def _refuse(t, name, dtype, shape, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


def _like(t, name, dtype, shape, dev) -> int:
    """The address of a contiguous CUDA tensor of this type, shape and device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        _refuse(t, name, dtype, shape, dev)
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _maybe(t, name, dtype, shape, dev):
    return None if t is None else _like(t, name, dtype, shape, dev)


def _heads(t, name, dtype, rows, heads, dim, dev) -> _Heads:
    """A [rows, heads, dim] tensor whose last dimension is dense; rows and heads may be strided."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (rows, heads, dim) and t.get_device() == dev):
        _refuse(t, name, dtype, (rows, heads, dim), dev)
    sr, sh, sd = t.stride()
    unit, at = 4 if dtype is torch.float32 else 8, t.data_ptr()
    if sd != 1 or (rows > 1 and sr % unit) or (heads > 1 and sh % unit) or at % 16:
        raise ValueError(f"{name} must have a dense last dimension and rows and heads on 16-byte boundaries")
    return _Heads(at, sr if rows > 1 else 0, sh if heads > 1 else 0)


def _status(status, dev):
    if status is None:
        return torch.zeros(1, dtype=torch.int32, device=f"cuda:{dev}")
    _like(status, "status", torch.int32, (1,), dev)
    return status


def _dtype(t, name, allowed) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in allowed:
        raise TypeError(f"{name} must be one of {[str(a) for a in allowed]}, got {t.dtype}")
    return _DTYPES[t.dtype]


def _ragged(row_off, kv_len, page_table, rows, dev) -> _Ragged:
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages] int32")
    B, width = page_table.shape
    i32 = torch.int32
    return _Ragged(_like(row_off, "row_off", i32, (B + 1,), dev), _like(kv_len, "kv_len", i32, (B,), dev),
                   _like(page_table, "page_table", i32, (B, width), dev), B, rows, width)


def _result(out, key, shape, dtype, like, dev):
    """out[key], checked, or a new tensor beside `like`."""
    t = None if out is None else out.get(key)
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _like(t, f"out[{key!r}]", dtype, shape, dev)
    return t


def _stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
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
            i = torch.arange(n, dtype=torch.float64)
            if scaling == "ntk":
                base = base * factor ** (rotary_dim / (rotary_dim - 2))
            inv = base ** (-2 * i / rotary_dim)
            if scaling == "linear":
                inv = inv / factor
            elif scaling == "yarn":
                def pair_of(turns):   # the pair that makes so many turns in original_len positions
                    return rotary_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))

                low, high = max(math.floor(pair_of(beta_fast)), 0), min(math.ceil(pair_of(beta_slow)), rotary_dim - 1)
                ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
                inv = inv * (1 - ramp) + inv / factor * ramp
                own_gain = 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
        else:
            inv = inv_freq.detach().to("cpu", torch.float64)
            if inv.shape != (n,):
                raise ValueError(f"inv_freq must have shape ({n},)")
        self.inv_freq, self.rotary_dim, self.layout = inv, rotary_dim, layout
        self.gain = own_gain if gain is None else float(gain)
        # turns per position in 64-bit fixed point, wrapped: whole turns say nothing
        turn = inv / (2 * math.pi)
        turn = turn - turn.round()                     # [-1/2, 1/2]: as a signed 64-bit fraction
        self.turns = (turn * 2.0 ** 64).clamp(max=2.0 ** 63 - 1024).round().to(torch.int64).to(device)
        self._c = _Rope(self.turns.data_ptr(), rotary_dim, layout == "interleaved", self.gain)


def norm_rope(q, k=None, positions=None, rope: Optional[Rope] = None, *, q_weight=None, k_weight=None,
              eps: float = 1e-6, out: Optional[dict] = None, status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Norm and rotation of query and key heads in one pass (C ABI dspark_attn_norm_rope).

    q [rows, Hq, D], k [rows, Hkv, D] or None (float32, bfloat16 or float16; D a multiple of 16 to 256; rows and
    heads may be strided, as in a view of a fused projection), positions [rows] int32 (with a rope), q_weight /
    k_weight [D] or None (no norm).  Returns q and k of the inputs' shape, contiguous (``out`` may name the
    inputs themselves where those are contiguous).
    """
    code = _dtype(q, "q", (torch.float32, torch.bfloat16, torch.float16))
    if q.dim() != 3:
        raise ValueError("q must be [rows, heads, D]")
    rows, hq, d = q.shape
    dev, dt = q.get_device(), q.dtype
    if d < 16 or d > 256 or d % 16:
        raise ValueError(f"head dimension must be a multiple of 16 to 256, got {d}")
    qh, kh, hkv, k_out = _heads(q, "q", dt, rows, hq, d, dev), None, 0, None
    q_out = _result(out, "q", (rows, hq, d), dt, q, dev)
    if k is not None:
        hkv = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 3 else -1
        kh = _heads(k, "k", dt, rows, hkv, d, dev)
        k_out = _result(out, "k", (rows, hkv, d), dt, q, dev)
    turn = _rope_fits(rope, d, dev)
    at = None
    if rope is not None or positions is not None:
        at = _like(positions, "positions", torch.int32, (rows,), dev)
    wq, wk = _maybe(q_weight, "q_weight", dt, (d,), dev), _maybe(k_weight, "k_weight", dt, (d,), dev)
    status = _status(status, dev)
    if rows:
        _ds._raise(_ds.lib().dspark_attn_norm_rope(
            qh, kh, rows, hq, hkv, d, code, at, turn, wq, wk, eps, q_out.data_ptr(),
            None if k_out is None else k_out.data_ptr(), status.data_ptr(), _stream(stream, dev)), "dspark_attn_norm_rope")
    return dict(q=q_out, k=k_out, status=status)


def _rope_fits(rope, d, dev):
    if rope is None:
        return None
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope")
    if rope.rotary_dim > d:
        raise ValueError(f"rope turns {rope.rotary_dim} dimensions of heads with {d}")
    if rope.turns.get_device() != dev:
        raise ValueError(f"rope must be on cuda:{dev}, got {rope.turns.device}")
    return rope._c


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


def _is_cache(cache):
    if not isinstance(cache, PagedCache):
        raise TypeError("cache must be a PagedCache")


def cache_append(cache: PagedCache, k, v, row_off, kv_len, page_table, *, positions=None, rope: Optional[Rope] = None,
                 k_weight=None, q=None, q_weight=None, eps: float = 1e-6, out: Optional[dict] = None,
                 status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Append the rows' keys and values to the cache, keys normed and rotated on the way (C ABI dspark_attn_append).

    k, v [rows, Hkv, D]; row_off [B+1], kv_len [B] (with these rows among them), page_table [B, max_pages], all
    int32; positions [rows] int32 or None (a row's place in its request); with q [rows, Hq, D] the queries are
    normed and rotated in the same pass and returned as q (contiguous).  Two rows must not name the same place.
    """
    _is_cache(cache)
    code = _dtype(k, "k", (torch.float32, torch.bfloat16, torch.float16))
    rows, d, dev, dt = k.shape[0], cache.head_dim, cache.device, k.dtype
    kh, vh = _heads(k, "k", dt, rows, cache.kv_heads, d, dev), _heads(v, "v", dt, rows, cache.kv_heads, d, dev)
    where = _ragged(row_off, kv_len, page_table, rows, dev)
    qh, hq, q_out, q_at = None, 0, None, None
    if q is not None:
        hq = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else -1
        qh = _heads(q, "q", dt, rows, hq, d, dev)
        q_out = _result(out, "q", (rows, hq, d), dt, q, dev)
        q_at = q_out.data_ptr()
    turn, at = _rope_fits(rope, d, dev), _maybe(positions, "positions", torch.int32, (rows,), dev)
    wq, wk = _maybe(q_weight, "q_weight", dt, (d,), dev), _maybe(k_weight, "k_weight", dt, (d,), dev)
    status = _status(status, dev)
    if rows:
        _ds._raise(_ds.lib().dspark_attn_append(kh, vh, qh, hq, code, cache._c, where, at, turn, wq, wk, eps, q_at,
                                                status.data_ptr(), _stream(stream, dev)), "dspark_attn_append")
    return dict(q=q_out, status=status)


def cache_read(cache: PagedCache, row_off, kv_len, page_table, rows: int, *, out: Optional[dict] = None,
               status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """What the cache holds of the rows' tokens (C ABI dspark_attn_cache_read): k, v [rows, Hkv, D] and k_scale,
    v_scale [rows, Hkv, D/16], float8_e4m3fn and exact; an element's value is element * scale * the cache's scale.
    A request's whole text: row_off over kv_len rows each."""
    _is_cache(cache)
    dev, h, d = cache.device, cache.kv_heads, cache.head_dim
    where = _ragged(row_off, kv_len, page_table, rows, dev)
    f8 = torch.float8_e4m3fn
    k, v = (_result(out, key, (rows, h, d), f8, cache.data, dev) for key in ("k", "v"))
    ks, vs = (_result(out, key, (rows, h, d // 16), f8, cache.data, dev) for key in ("k_scale", "v_scale"))
    status = _status(status, dev)
    if rows:
        _ds._raise(_ds.lib().dspark_attn_cache_read(cache._c, where, k.data_ptr(), ks.data_ptr(), v.data_ptr(),
                                                    vs.data_ptr(), status.data_ptr(), _stream(stream, dev)),
                   "dspark_attn_cache_read")
    return dict(k=k, k_scale=ks, v=v, v_scale=vs, status=status)


def attend_paged(q, cache: PagedCache, row_off, kv_len, page_table, *, scale: Optional[float] = None,
                 causal: bool = True, window: int = 0, max_rows: Optional[int] = None, want_lse: bool = False,
                 out: Optional[dict] = None, workspace: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Attention of ragged rows over the cache (C ABI dspark_attn_paged).

    q [rows, Hq, D] bfloat16 or float16 (rows and heads may be strided), Hq a multiple of the cache's heads;
    scale: 1/sqrt(D) unless given.  Row j of request r sees its tokens up to itself (causal) or all kv_len[r], and
    with window > 0 only the last ``window`` of them; a row that sees nothing gets 0 and lse -inf.  max_rows: the
    most rows of a request (default: what ``rows`` allows; smaller is faster).  Returns out [rows, Hq, D] and,
    with want_lse, lse [rows, Hq] float32.
    """
    _is_cache(cache)
    code = _dtype(q, "q", (torch.bfloat16, torch.float16))
    if q.dim() != 3:
        raise ValueError("q must be [rows, heads, D]")
    rows, hq, d = q.shape
    dev = cache.device
    if hq % cache.kv_heads:
        raise ValueError(f"{hq} query heads are no multiple of {cache.kv_heads} key/value heads")
    qh = _heads(q, "q", q.dtype, rows, hq, cache.head_dim, dev)
    where = _ragged(row_off, kv_len, page_table, rows, dev)
    if max_rows is None:
        max_rows = rows
    if max_rows < 1 and rows or window < 0:
        raise ValueError("max_rows must be positive and window not negative")
    o = _result(out, "out", (rows, hq, d), q.dtype, q, dev)
    lse = _result(out, "lse", (rows, hq), torch.float32, q, dev) if want_lse else None
    status = _status(status, dev)
    if rows:
        L = _ds.lib()
        need, at = L.dspark_attn_paged_workspace_bytes(hq, cache._c, where, max_rows), None
        if need:
            workspace = _ds._workspace(need, q.device, workspace)
            at = workspace.data_ptr()
        _ds._raise(L.dspark_attn_paged(
            qh, hq, code, cache._c, where, max_rows, 1 / math.sqrt(d) if scale is None else scale, bool(causal),
            int(window), o.data_ptr(), None if lse is None else lse.data_ptr(), at, workspace.numel() if need else 0,
            status.data_ptr(), _stream(stream, dev)), "dspark_attn_paged")
    return dict(out=o, lse=lse, status=status, workspace=workspace)


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
    code = _dtype(logits, "logits", (torch.float32, torch.bfloat16))
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, V]")
    rows, V = logits.shape
    dev, i32, f32 = logits.get_device(), torch.int32, torch.float32
    at = _like(logits, "logits", logits.dtype, (rows, V), dev)
    if not isinstance(hist, torch.Tensor) or hist.dim() != 2:
        raise ValueError("hist must be [B, cap] int32")
    B, cap = hist.shape
    if (bias_tok is None) != (bias_val is None):
        raise ValueError("bias_tok and bias_val go together")
    n_draft = draft_tok.shape[1] if isinstance(draft_tok, torch.Tensor) and draft_tok.dim() == 2 else 0
    n_bias = bias_tok.shape[1] if isinstance(bias_tok, torch.Tensor) and bias_tok.dim() == 2 else 0
    one = (B,)
    off = _like(row_off, "row_off", i32, (B + 1,), dev)
    p = _Penalties(_like(hist, "hist", i32, (B, cap), dev), _like(hist_len, "hist_len", i32, one, dev),
                   _like(prompt_len, "prompt_len", i32, one, dev), _maybe(draft_tok, "draft_tok", i32, (B, n_draft), dev),
                   _like(repetition, "repetition", f32, one, dev), _like(presence, "presence", f32, one, dev),
                   _like(frequency, "frequency", f32, one, dev), _maybe(bias_tok, "bias_tok", i32, (B, n_bias), dev),
                   _maybe(bias_val, "bias_val", f32, (B, n_bias), dev),
                   _maybe(mask, "mask", i32, (rows, (V + 31) // 32), dev), cap, n_draft, n_bias)
    o = _result(out, "logits", (rows, V), logits.dtype, logits, dev)
    status = _status(status, dev)
    if rows:
        _ds._raise(_ds.lib().dspark_logits_penalize(at, code, rows, V, B, off, p, o.data_ptr(), status.data_ptr(),
                                                    _stream(stream, dev)), "dspark_logits_penalize")
    return dict(logits=o, status=status)
