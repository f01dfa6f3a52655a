"""Attention over the paged cache in 8 bits against a plain 64-bit implementation on what the cache holds, at the
lengths, masks, pages and values where it can go wrong, and the operators of a prompt and its decoding together.

Tolerances count roundings: half(t) = torch.finfo(t).eps / 2 of a value stored in t; probabilities are fp16 (2^-11), for
bf16 queries then kept to 9 bits (2^-9); a tensor-core step adds 32 products of 25 bits each beside its fp32 sum (2^-20 of
the largest); a product that lies 2^-28 below the largest is rounded away.
"""
import math

import pytest
import torch

import speculative_decoding_draft_gb300 as ds
from test_gpu_serving import gen, half, i32, offsets, ok, paged, randn

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_draft_gb300 import build
    build.build()


def filled(g, kv, hkv, d, page, loud=0.5, stale=True):
    """A cache with texts of kv tokens, what it holds of them [sum kv, hkv, d] in float64, and its page table.  What
    lies behind the texts are NaN elements and scales of any size."""
    table, pages = paged(g, kv, page, spare=1)
    cache = ds.PagedCache8.empty(pages, hkv, d, page)
    if stale:
        cache.data.fill_(0x7f)
        cache.scales.random_(0, 256, generator=g)
    x = randn(g, 2, sum(kv), hkv, d) * torch.exp(loud * randn(g, 2, sum(kv), hkv, 1))
    if sum(kv):
        ok(ds.cache_append(cache, x[0], x[1], offsets(kv), i32(kv), table)["status"])
    got = ds.cache_read(cache, offsets(kv), i32(kv), table, sum(kv), dtype=torch.float32)
    return cache, got["k"].double(), got["v"].double(), table


def plain(q, k, v, n, kv, scale, causal, window):
    rows, hq, d = q.shape
    group = hq // k.shape[1]
    terms = 3 if q.dtype == torch.bfloat16 else 4
    p_off = 2.0 ** -11 + (2.0 ** -9 if terms == 3 else 0)
    out, lse = torch.zeros(rows, hq, d).double().cuda(), torch.full((rows, hq), -math.inf).double().cuda()
    out_bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    a = c = 0
    for nr, mr in zip(n, kv):
        b, e = a + nr, c + mr
        t = torch.arange(mr, device="cuda")
        hi = (mr - nr + torch.arange(nr, device="cuda") + 1 if causal else torch.full((nr,), mr, device="cuda"))[:, None]
        hide = t >= hi
        if window:
            hide |= t < hi - window
        for h in range(hq if nr and mr else 0):
            x, y, z = q[a:b, h].double(), k[c:e, h // group], v[c:e, h // group]
            y, z = (torch.where(hide.all(0)[:, None], 0.0, w) for w in (y, z))
            s = (x @ y.T * scale).masked_fill(hide, -math.inf)
            some = (~hide).any(1)
            lse[a:b, h] = torch.logsumexp(s, 1)
            p = torch.exp(s - torch.where(some, lse[a:b, h], 0)[:, None]).masked_fill(hide, 0.0)
            out[a:b, h] = p @ z
            off = ((x.abs() @ y.abs().T) * abs(scale) * (terms * d // 32) * 2.0 ** -20).masked_fill(hide, 0.0).amax(1) + 2.0 ** -20
            lse_bound[a:b, h] = off + 2.0 ** -20 * lse[a:b, h].abs().nan_to_num(0, 0, 0)
            size = p @ z.abs()
            out_bound[a:b, h] = ((2 * off + p_off + mr / 32 * 2.0 ** -20)[:, None] * size + half(q.dtype) * out[a:b, h].abs()
                                 + mr * 2.0 ** -27 * z.abs().amax())
        a, c = b, e
    return out, lse, out_bound + torch.finfo(q.dtype).smallest_normal, lse_bound


def check(q, cache, k, v, n, kv, table, scale=None, causal=True, window=0, **kw):
    got = ds.attend_paged(q, cache, offsets(n), i32(kv), table, scale=scale, causal=causal, window=window, want_lse=True, **kw)
    ok(got["status"])
    s = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    out, lse, out_bound, lse_bound = plain(q, k, v, n, kv, s, causal, window)
    rows = sum(n)
    far = (got["out"][:rows].double() - out[:rows]).abs() - out_bound[:rows]
    assert far.max() <= 0, f"out is {far.max().item():.3g} past its bound"
    x, y = got["lse"][:rows].double(), lse[:rows]
    assert torch.equal(torch.isinf(x), torch.isinf(y))
    assert ((x - y).abs().nan_to_num(0) <= lse_bound[:rows]).all()
    return got


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,group,page", [(1, 1, 16), (2, 4, 48), (8, 2, 64), (1, 8, 256), (3, 3, 128)])
@pytest.mark.parametrize("n,kv", [([1], [1]), ([1, 1, 1], [127, 128, 129]), ([4, 0, 8, 3], [700, 5, 0, 3]),
                                  ([1, 8, 2], [16, 2049, 300])])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 200), (False, 333)])
def test_attend(dtype, d, hkv, group, page, n, kv, causal, window):
    g = gen(sum(kv) + d + group)
    cache, k, v, table = filled(g, kv, hkv, d, page)
    q = randn(g, sum(n), hkv * group, d).to(DTYPES[dtype])
    check(q, cache, k, v, n, kv, table, causal=causal, window=window, max_rows=max(n))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,kv", [([40, 3], [500, 900]), ([130], [1000])])
def test_many_rows_and_no_bound_on_them(dtype, n, kv):
    g = gen(3)
    cache, k, v, table = filled(g, kv, 2, 128, 64)
    q = randn(g, sum(n), 8, 128).to(DTYPES[dtype])
    check(q, cache, k, v, n, kv, table)


@pytest.mark.parametrize("d,page", [(64, 32), (128, 64)])
def test_one_long_text(d, page):
    g, kv = gen(4), [20011]
    cache, k, v, table = filled(g, kv, 2, d, page)
    q = randn(g, 5, 8, d).bfloat16()
    got = check(q, cache, k, v, [5], kv, table, max_rows=5)
    ws = got["workspace"].fill_(255)                             # what the workspace holds does not matter
    again = ds.attend_paged(q, cache, offsets([5]), i32(kv), table, max_rows=5, want_lse=True, workspace=ws)
    assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])


def test_many_requests():
    g, B = gen(5), 400
    kv = [(37 * i) % 301 for i in range(B)]
    n = [min(1 + i % 3, 3) for i in range(B)]
    cache, k, v, table = filled(g, kv, 2, 64, 16)
    q = randn(g, sum(n), 4, 64).half()
    check(q, cache, k, v, n, kv, table, max_rows=3)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [64, 128])
def test_references_that_rise_and_scales_far_apart(dtype, d):
    g, m = gen(6), 900
    table, pages = paged(g, [m], 64)
    cache = ds.PagedCache8.empty(pages, 1, d, 64)
    sign = randn(g, 1, 1, d).sign()
    k = (sign * torch.linspace(0.05, 6, m, device="cuda")[:, None, None]).expand(m, 1, d).contiguous()
    v = randn(g, m, 1, d) * torch.exp2(torch.randint(-24, 25, (m, 1, 1), generator=g, device="cuda").float())
    ok(ds.cache_append(cache, k, v, offsets([m]), i32([m]), table)["status"])
    got = ds.cache_read(cache, offsets([m]), i32([m]), table, m, dtype=torch.float32)
    q = (sign * (0.5 + randn(g, 4, 4, d).abs())).to(DTYPES[dtype])
    for scale in (0.02, -0.02, 0.0):
        out, lse, bound, lse_bound = plain(q, got["k"].double(), got["v"].double(), [4], [m], scale, True, 0)
        r = ds.attend_paged(q, cache, offsets([4]), i32([m]), table, scale=scale, want_lse=True)
        ok(r["status"])
        assert ((r["lse"].double() - lse).abs() <= lse_bound).all()
        # out may pass fp16's range, where the type's infinity is right
        x = r["out"].double()
        fine = out.abs() + bound < torch.finfo(q.dtype).max
        assert ((x - out).abs() <= bound)[fine].all()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 40])
def test_nans_in_masked_places(dtype, d, window):
    g, n, m = gen(7), 6, 300
    table, pages = paged(g, [m], 32)
    caches = []
    x = randn(g, 2, m, 2, d)
    for bad in (False, True):
        if bad:
            x[1, m - 3, 0, 5] = math.nan                         # a value that the last three rows see
            x[0, m - 2, 1, 9] = math.nan                         # a key that the last two see
        cache = ds.PagedCache8.empty(pages, 2, d, 32)
        ok(ds.cache_append(cache, x[0], x[1], offsets([m]), i32([m]), table)["status"])
        caches.append(cache)
    q = randn(g, n, 4, d).to(DTYPES[dtype])
    clean, got = (ds.attend_paged(q, c, offsets([n]), i32([m]), table, window=window)["out"] for c in caches)
    same = torch.ones_like(got, dtype=torch.bool)
    same[n - 3:, :2, 5] = False
    same[n - 2:, 2:] = False
    # (scales of blocks without a NaN in their place are the same: a NaN counts nothing)
    assert torch.equal(got[same], clean[same])
    assert torch.isnan(got[n - 3:, :2, 5]).all() and torch.isnan(got[n - 2:, 2:]).all()


def test_rows_behind_the_last_strides_and_failed_steps():
    g, n, kv = gen(8), [3, 2], [40, 70]
    cache, k, v, table = filled(g, kv, 2, 64, 16)
    q = randn(g, 9, 6, 64).bfloat16()[:, 1:5]
    out, lse = torch.full((9, 4, 64), 7.0, device="cuda").bfloat16(), torch.full((9, 4), 7.0, device="cuda")
    check(q, cache, k, v, n, kv, table, out=dict(out=out, lse=lse))
    assert (out[5:] == 7).all() and (lse[5:] == 7).all()
    status = ds.new_status("cuda")
    status.fill_(9)
    ds.attend_paged(q, cache, offsets(n), i32(kv), table, want_lse=True, out=dict(out=out.fill_(5), lse=lse), status=status)
    assert (out == 5).all()


@pytest.mark.parametrize("bad,name", [(dict(off=[0, 9, 4]), "OFFSETS"), (dict(kv=[-1, 2]), "LENGTHS"),
                                      (dict(kv=[4, 33]), "LENGTHS"), (dict(max_rows=1), "LENGTHS"),
                                      (dict(table=[[0, 1], [2, 0]]), "PAGES"), (dict(table=[[-1, 1], [0, 0]]), "PAGES")])
def test_inconsistent_arguments(bad, name):
    cache = ds.PagedCache8.empty(2, 1, 64, 16)
    q = torch.ones(4, 1, 64, device="cuda").half()
    off, kv, table = (i32(bad.get(k, v)) for k, v in (("off", [0, 2, 4]), ("kv", [4, 20]), ("table", [[0, 1], [1, 0]])))
    got = ds.attend_paged(q, cache, off, kv, table, max_rows=bad.get("max_rows", 2))
    assert ds.check(got["status"]) == "DSPARK_ERR_" + name


def test_two_streams_and_a_graph():
    g, n, kv = gen(9), [2, 8, 1], [600, 2100, 33]
    cache, k, v, table = filled(g, kv, 2, 128, 64)
    q = randn(g, 11, 8, 128).bfloat16()
    off, length = offsets(n), i32(kv)
    want = ds.attend_paged(q, cache, off, length, table, max_rows=8)["out"]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [ds.attend_paged(q, cache, off, length, table, max_rows=8, stream=s)["out"] for s in streams for _ in range(3)]
    for s in streams:
        s.synchronize()
    assert all(torch.equal(x, want) for x in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = ds.attend_paged(q, cache, off, length, table, max_rows=8)["out"]
    q.copy_(randn(g, 11, 8, 128))
    graph.replay()
    assert torch.equal(held, ds.attend_paged(q, cache, off, length, table, max_rows=8)["out"])


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_a_prompt_in_pieces_then_decoding(dtype):
    """A prompt whose second piece is read over the first one's keys and values as the cache gives them back, then rows
    over the cache: all against one plain attention on what the cache holds."""
    g, dt, hq, hkv, d = gen(10), DTYPES[dtype], 8, 2, 128
    first, second, then = [150, 40], [33, 90], [3, 1]
    lengths = [a + b + c for a, b, c in zip(first, second, then)]
    table, pages = paged(g, lengths, 64)
    cache = ds.PagedCache8.empty(pages, hkv, d, 64)
    rope = ds.Rope(d, base=1e4)
    status = ds.new_status("cuda")
    done = [0, 0]
    for call, n in enumerate((first, second, then)):
        rows = sum(n)
        qkv = randn(g, rows, hq + 2 * hkv, d).to(dt)
        kv = [x + y for x, y in zip(done, n)]
        off, length = offsets(n), i32(kv)
        q = ds.cache_append(cache, qkv[:, hq: hq + hkv], qkv[:, hq + hkv:], off, length, table, rope=rope, q=qkv[:, :hq],
                            status=status)["q"]
        held = ds.cache_read(cache, offsets(kv), length, table, sum(kv), dtype=dt, status=status)
        if call < 2:
            got = ds.attend_prompt(q, held["k"], held["v"], off, kv_off=offsets(kv), status=status)["out"]
        else:
            got = ds.attend_paged(q, cache, off, length, table, max_rows=3, status=status)["out"]
        exact = ds.cache_read(cache, offsets(kv), length, table, sum(kv), dtype=torch.float32, status=status)
        ok(status)
        out, _, bound, _ = plain(q, exact["k"].double(), exact["v"].double(), n, kv, d ** -0.5, True, 0)
        # the prompt's probabilities are rounded to the type itself, fp16 values of the cache to 2^-11
        bound = bound + (half(dt) + 2.0 ** -10) * 4 * math.sqrt(d) * 2.0 ** -3
        assert ((got.double() - out).abs() <= bound).all()
        done = kv


def test_the_example_decodes_over_8_bits():
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import verification_step as example
    finally:
        sys.path.pop(0)
    B, K = 5, 3
    dec = example.Decoder(example.Target(B, bits=8), [[7 + r, 11, 3 * r] + list(range(r)) for r in range(B)])
    for i in range(6):
        dec.step(example.draft_model(B, K, dec.t.V, seed=9 + i), K, 0.0)
    assert ds.check(dec.t.status) == "DSPARK_OK"
    for r in range(B):                                           # the grammar holds along every emitted token
        out = dec.text[r, int(dec.prompt[r]) - 1: int(dec.length[r])]
        assert len(out) > 6 and ((out[1:] + out[:-1]) % 2 == 1).all()
