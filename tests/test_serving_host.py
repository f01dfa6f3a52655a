"""Host-side validation of the operators around a ragged verification step, and the rotary frequencies (no GPU)."""
import ctypes
import math

import pytest
import torch

import speculative_decoding_draft_gb300 as ds
from speculative_decoding_draft_gb300 import serving as sv


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_draft_gb300 import build
    build.build()
    return ds.lib()


ONE = 256          # a non-null, aligned address that is never read: validation comes before any launch


def heads(data=ONE, row=1024, head=64):
    return sv._Heads(data, row, head)


def cache(**kw):
    a = dict(data=ONE, pages=4, kv_heads=2, head_dim=64, page_size=16, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    return sv._Cache(*[a[f] for f, _ in sv._Cache._fields_])


def ragged(**kw):
    a = dict(row_off=ONE, kv_len=ONE, page_table=ONE, B=1, rows=2, max_pages=1)
    a.update(kw)
    return sv._Ragged(*[a[f] for f, _ in sv._Ragged._fields_])


def name(code):
    return ds.STATUS_NAMES[code].replace("DSPARK_ERR_", "")


def test_norm_rope_refusals(lib):
    def call(q=heads(), k=heads(), rows=2, hq=4, hkv=2, d=64, dtype=1, pos=ONE, rope=sv._Rope(ONE, 64, 0, 1.0), eps=1e-6,
             out=ONE, k_out=ONE, st=ONE):
        return name(lib.dspark_attn_norm_rope(q, k, rows, hq, hkv, d, dtype, pos, rope, None, None, eps, out, k_out, st,
                                              None))
    assert call(q=None) == call(out=None) == call(st=None) == call(pos=None) == call(k_out=None) == "NULL"
    assert call(k=None) == "NULL" and call(q=heads(None)) == "NULL"
    assert call(dtype=3) == "DTYPE"
    assert call(rows=0) == call(hq=0) == call(hkv=0) == call(d=72) == call(d=272) == call(eps=-1.0) == "DIMS"
    assert call(eps=math.nan) == call(q=heads(row=-8)) == "DIMS"
    assert call(rope=sv._Rope(ONE, 80, 0, 1.0)) == call(rope=sv._Rope(ONE, 8, 0, 1.0)) == "DIMS"
    assert call(rope=sv._Rope(ONE, 64, 0, math.inf)) == "DIMS" and call(rope=sv._Rope(None, 64, 0, 1.0)) == "NULL"
    assert call(q=heads(264)) == call(q=heads(row=1028)) == call(k=heads(head=4)) == call(out=264) == "UNSUPPORTED"


def test_norm_weights_off_a_boundary_are_refused(lib):
    # refused where the heads are, before the rope and eps of these calls are looked at
    rope = sv._Rope(ONE, 80, 0, 1.0)
    for wq, wk, want in ((ONE, ONE, "DIMS"), (ONE + 8, None, "UNSUPPORTED"), (None, ONE + 2, "UNSUPPORTED"),
                         (ONE, ONE + 4, "UNSUPPORTED")):
        assert name(lib.dspark_attn_norm_rope(heads(), heads(), 2, 4, 2, 64, 1, ONE, rope, wq, wk, 1e-6, ONE, ONE, ONE,
                                              None)) == want
        assert name(lib.dspark_attn_append(heads(), heads(), heads(), 4, 1, cache(), ragged(), None, None, wq, wk, -1.0,
                                           ONE, ONE, None)) == want


def test_cache_refusals(lib):
    def append(k=heads(), v=heads(), q=None, hq=0, dtype=1, c=None, w=None, rope=None, eps=0.0, q_out=None, st=ONE):
        return name(lib.dspark_attn_append(k, v, q, hq, dtype, c or cache(), w or ragged(), None, rope, None, None, eps,
                                           q_out, st, None))
    assert append(k=None) == append(v=None) == append(q=heads()) == append(q_out=ONE) == append(st=None) == "NULL"
    assert append(q=heads(), q_out=ONE, hq=0) == append(q=heads(), q_out=ONE, hq=2000) == "DIMS"
    assert append(c=cache(data=None)) == append(w=ragged(kv_len=None)) == "NULL"
    for bad in (dict(pages=0), dict(kv_heads=0), dict(page_size=24), dict(page_size=8), dict(page_size=8192),
                dict(k_scale=3.0), dict(v_scale=-1.0), dict(k_scale=math.inf), dict(v_scale=0.0)):
        assert append(c=cache(**bad)) == "DIMS", bad
    assert append(c=cache(head_dim=96)) == append(c=cache(data=264)) == "UNSUPPORTED"
    for bad in (dict(B=0), dict(rows=0), dict(max_pages=0), dict(B=1 << 21)):
        assert append(w=ragged(**bad)) == "DIMS", bad
    assert append(rope=sv._Rope(ONE, 80, 0, 1.0)) == "DIMS" and append(dtype=-1) == "DTYPE"

    def read(c=None, w=None, k=ONE, s=ONE):
        return name(lib.dspark_attn_cache_read(c or cache(), w or ragged(), k, s, ONE, ONE, ONE, None))
    assert read(k=None) == read(s=None) == read(c=cache(data=None)) == "NULL"
    assert read(k=264) == read(c=cache(head_dim=256)) == "UNSUPPORTED"

    def attend(q=heads(), hq=4, dtype=1, c=None, w=None, most=1, scale=1.0, window=0, out=ONE):
        return name(lib.dspark_attn_paged(q, hq, dtype, c or cache(), w or ragged(), most, scale, 1, window, out, None, None, 0,
                                          ONE, None))
    assert attend(q=None) == attend(out=None) == "NULL"
    assert attend(dtype=0) == "DTYPE"
    assert attend(hq=3) == attend(hq=0) == attend(most=0) == attend(scale=math.nan) == attend(window=-1) == "DIMS"
    assert attend(w=ragged(max_pages=1 << 28)) == "DIMS" and attend(out=264) == "UNSUPPORTED"


def test_penalize_refusals(lib):
    fields = [f for f, _ in sv._Penalties._fields_]

    def call(logits=ONE, dtype=0, rows=2, V=100, B=1, off=ONE, out=ONE, **kw):
        a = dict({f: ONE for f in fields}, hist_cap=4, draft_cap=2, bias_cap=2)
        a.update(kw)
        return name(lib.dspark_logits_penalize(logits, dtype, rows, V, B, off, sv._Penalties(*[a[f] for f in fields]),
                                               out, ONE, None))
    assert call(logits=None) == call(off=None) == call(out=None) == call(hist=None) == call(frequency=None) == "NULL"
    assert call(bias_tok=None) == call(bias_val=None) == "NULL"
    assert call(dtype=2) == "DTYPE"
    assert call(V=1) == call(rows=0) == call(B=0) == call(hist_cap=0) == call(bias_cap=5000) == call(draft_cap=0) == "DIMS"
    assert call(V=1 << 30, B=1 << 20) == "DIMS"


def test_bindings_take_cuda_tensors_only():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for f in (lambda: ds.norm_rope(x), lambda: ds.PagedCache(torch.zeros(1, 1, 1, 18 * 64, dtype=torch.uint8), 16),
              lambda: ds.attend_paged(x, None, None, None, None),
              lambda: ds.penalize_logits(x[0], None, None, None, None, None, None, None)):
        with pytest.raises(TypeError):
            f()


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_rope_frequencies_and_turns(scaling):
    r = ds.Rope(64, base=1e4, scaling=scaling, factor=8.0, original_len=2048, device="cpu")
    plain = [1e4 ** (-2 * i / 64) for i in range(32)]
    inv = r.inv_freq.tolist()
    if scaling == "none":
        assert inv == pytest.approx(plain, rel=1e-15) and r.gain == 1
    elif scaling == "linear":
        assert inv == pytest.approx([x / 8 for x in plain], rel=1e-15)
    elif scaling == "ntk":      # the first pair stays, the last is divided by the factor
        assert inv[0] == 1 and inv[-1] == pytest.approx(plain[-1] / 8, rel=1e-12)
    else:                       # fast pairs stay, slow ones are divided, the ramp lies between
        assert inv[0] == 1 and inv[-1] == pytest.approx(plain[-1] / 8, rel=1e-12)
        assert all(p / 8 * (1 - 1e-12) <= x <= p * (1 + 1e-12) for x, p in zip(inv, plain))
        assert r.gain == pytest.approx(0.1 * math.log(8) + 1)
    # the fixed-point turn reproduces the angle at a far position (the frequency itself is known to 2^-53)
    for pos in (1, 12345, 2 ** 31 - 1):
        for t, x in zip(r.turns.tolist(), inv):
            frac = (pos * t % 2 ** 64) / 2 ** 64
            want = math.fmod(pos * x / (2 * math.pi), 1.0)
            assert min(abs(frac - want), 1 - abs(frac - want)) < pos * x * 2.0 ** -50 + 2.0 ** -30


def test_rope_takes_frequencies_as_they_are():
    f = torch.linspace(0.1, 9.0, 8)
    assert torch.equal(ds.Rope(16, inv_freq=f, gain=2.0, device="cpu").inv_freq, f.double())
    with pytest.raises(ValueError):
        ds.Rope(16, inv_freq=f[:4], device="cpu")
