"""Host-side validation of the operators of prompts and of the cache in 8 bits (no GPU)."""
import ctypes
import math

import pytest
import torch

import speculative_decoding_draft_gb300 as ds
from speculative_decoding_draft_gb300 import serving as sv
from test_serving_host import ONE, heads, lib, name, ragged  # noqa: F401


def cache(**kw):
    a = dict(data=ONE, scales=ONE, pages=4, kv_heads=2, head_dim=64, page_size=16)
    a.update(kw)
    return sv._ByteCache(*[a[f] for f, _ in sv._ByteCache._fields_])


def test_prompt_refusals(lib):  # noqa: F811
    def call(q=heads(), k=heads(), v=heads(), rows=2, kv_rows=2, B=1, hq=4, hkv=2, d=64, dtype=1, off=ONE, kv_off=ONE,
             scale=1.0, window=0, out=ONE, st=ONE):
        return name(lib.dspark_attn_prompt(q, k, v, rows, kv_rows, B, hq, hkv, d, dtype, off, kv_off, scale, 1, window, out,
                                           None, None, 0, st, None))
    assert call(q=None) == call(k=None) == call(v=None) == call(off=None) == call(kv_off=None) == "NULL"
    assert call(out=None) == call(st=None) == call(k=heads(None)) == "NULL"
    assert call(dtype=0) == call(dtype=3) == "DTYPE"
    assert call(rows=0) == call(B=0) == call(hq=3) == call(hkv=0) == call(kv_rows=-1) == call(window=-1) == "DIMS"
    assert call(scale=math.nan) == call(scale=math.inf) == call(scale=3e38) == "DIMS"
    assert call(rows=1 << 30, hq=8) == call(kv_rows=2 ** 31 - 1) == "DIMS"
    assert call(d=96) == call(out=264) == call(q=heads(264)) == call(v=heads(row=1028)) == "UNSUPPORTED"
    # broadcast keys, and rows inside heads whose stride is no multiple of the rows'
    assert call(k=heads(row=0)) == call(v=heads(head=0)) == "UNSUPPORTED"
    assert call(k=heads(row=72, head=328)) == "UNSUPPORTED"


def test_byte_cache_refusals(lib):  # noqa: F811
    def append(k=heads(), v=heads(), q=None, hq=0, dtype=1, c=None, w=None, rope=None, eps=0.0, q_out=None, st=ONE, wk=None):
        return name(lib.dspark_attn_append_byte(k, v, q, hq, dtype, c or cache(), w or ragged(), None, rope, None, wk, eps,
                                                q_out, st, None))
    assert append(k=None) == append(v=None) == append(q=heads()) == append(q_out=ONE) == append(st=None) == "NULL"
    assert append(c=cache(data=None)) == append(c=cache(scales=None)) == append(w=ragged(kv_len=None)) == "NULL"
    for bad in (dict(pages=0), dict(kv_heads=0), dict(page_size=24), dict(page_size=8), dict(page_size=8192)):
        assert append(c=cache(**bad)) == "DIMS", bad
    assert append(c=cache(head_dim=96)) == append(c=cache(data=264)) == append(wk=ONE + 8) == "UNSUPPORTED"
    assert append(rope=sv._Rope(ONE, 80, 0, 1.0)) == append(eps=-1.0) == append(q=heads(), q_out=ONE, hq=0) == "DIMS"
    assert append(dtype=-1) == "DTYPE"

    def read(c=None, w=None, dtype=1, k=ONE, v=ONE):
        return name(lib.dspark_attn_cache_read_byte(c or cache(), w or ragged(), dtype, k, v, ONE, None))
    assert read(k=None) == read(v=None) == read(c=cache(scales=None)) == "NULL"
    assert read(dtype=3) == "DTYPE" and read(k=264) == read(c=cache(head_dim=256)) == "UNSUPPORTED"

    def attend(q=heads(), hq=4, dtype=1, c=None, w=None, most=1, scale=1.0, window=0, out=ONE):
        return name(lib.dspark_attn_paged_byte(q, hq, dtype, c or cache(), w or ragged(), most, scale, 1, window, out, None,
                                               None, 0, ONE, None))
    assert attend(q=None) == attend(out=None) == "NULL"
    assert attend(dtype=0) == "DTYPE"
    assert attend(hq=3) == attend(hq=0) == attend(most=0) == attend(scale=math.nan) == attend(window=-1) == "DIMS"
    assert attend(w=ragged(max_pages=(2 ** 31 - 1) // 16)) == "DIMS" and attend(out=264) == "UNSUPPORTED"


def test_caches_take_cuda_tensors_of_their_shape_only():
    data, scales = torch.zeros(2, 1, 2, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 2, 1, dtype=torch.uint8)
    with pytest.raises(TypeError):
        ds.PagedCache8(data, scales)
    with pytest.raises(ValueError):
        ds.PagedCache8.empty(1, 1, 64, 24, device="cpu")
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for f in (lambda: ds.attend_prompt(x, x, x, None), lambda: ds.cache_append(None, x, x, None, None, None),
              lambda: ds.cache_read(object(), None, None, None, 1), lambda: ds.attend_paged(x, data, None, None, None)):
        with pytest.raises(TypeError):
            f()


def test_the_cache_structure_is_the_header_s():
    assert ctypes.sizeof(sv._ByteCache) == 40
