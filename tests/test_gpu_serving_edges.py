"""The operators around a ragged verification step where they once went wrong: norm weights off their boundary, NaN in
16-bit keys and values, elements and scales at the borders of their codes, windows past every token, pages that a
window has left, calls on a stream of their own, steps that had failed before the call."""
import math

import pytest
import torch

import speculative_decoding_draft_gb300 as ds
from test_gpu_serving import DTYPES, E2M1, attend_check, built, filled, gen, i32, offsets, ok, paged, randn  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------------------------------
# what 4 bits keep
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("turned", [False, True])
def test_append_marks_the_groups_with_a_nan(dtype, d, turned):
    g, dt = gen(41), DTYPES[dtype]
    k, v = randn(g, 3, 2, d).to(dt), randn(g, 3, 2, d).to(dt)
    kw = dict(rope=ds.Rope(d), k_weight=torch.ones(d, device="cuda").to(dt)) if turned else {}
    where = (i32([0, 3]), i32([3]), i32([[0]]))
    kept = []
    for bad in (False, True):
        if bad:
            k[1, 0, 20] = v[2, 1, 37] = math.nan
        cache = ds.PagedCache.empty(1, 2, d, 16)
        ok(ds.cache_append(cache, k, v, *where, **kw)["status"])
        back = ds.cache_read(cache, *where, 3)
        kept.append({h: back[h].float() for h in ("k", "k_scale", "v", "v_scale")})
    lost = {"k_scale": torch.zeros(3, 2, d // 16, dtype=torch.bool, device="cuda")}
    lost["v_scale"] = lost["k_scale"].clone()
    lost["k_scale"][1, 0, slice(None) if turned else 1] = True       # a norm spreads a NaN over its head
    lost["v_scale"][2, 1, 2] = True
    for h in ("k", "v"):
        bad, s = lost[h + "_scale"], kept[1][h + "_scale"]
        assert torch.equal(torch.isnan(s), bad)
        assert torch.equal(s[~bad], kept[0][h + "_scale"][~bad])
        wide = bad.repeat_interleave(16, -1)
        assert not kept[1][h][wide].any() and torch.equal(kept[1][h][~wide], kept[0][h][~wide])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("part", ["k", "v"])
def test_attention_sees_the_nan_of_a_key_or_value_of_any_type(dtype, part):
    # token 37 of 40: of rows 35 .. 39 only 37 on see it
    g, d, n, kv = gen(42), 128, [5], [40]
    table, pages = paged(g, kv, 16)
    cache, held = filled(g, kv, table, pages, 1, d, 16)
    bad = torch.ones(1, 1, d, device="cuda").to(DTYPES[dtype])
    one = bad.clone()
    bad[0, 0, 20] = math.nan
    ds.cache_append(cache, bad if part == "k" else one, bad if part == "v" else one, i32([0, 1]), i32([38]), table)
    q = randn(g, 5, 2, d).bfloat16()
    got = ds.attend_paged(q, cache, offsets(n), i32(kv), table, want_lse=True)
    ok(got["status"])
    assert torch.isnan(got["out"][2:, :, 16:32]).all()
    assert torch.isnan(got["lse"][2:]).all() == (part == "k")
    attend_check(q[:2], got, [tuple(t[:37] for t in held[0])], [2], [37], d ** -0.5, True, 0)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_append_of_infinities_and_of_values_past_the_largest_scale(dtype):
    d, dt = 64, DTYPES[dtype]
    big = 6e4 if dt == torch.float16 else 1e30
    x = torch.ones(1, 1, d, device="cuda").to(dt)
    x[0, 0, 3], x[0, 0, 17], x[0, 0, 18], x[0, 0, 34], x[0, 0, 50] = math.inf, -math.inf, math.inf, -big, 2688
    x[0, 0, 51] = -2240                                    # 5 times the largest scale: a tie, to the even code
    cache = ds.PagedCache.empty(1, 1, d, 16)
    where = (i32([0, 1]), i32([1]), i32([[0]]))
    ok(ds.cache_append(cache, x, x, *where)["status"])
    got = ds.cache_read(cache, *where, 1)
    want = torch.zeros(d, device="cuda")
    want[3], want[17], want[18], want[34], want[50], want[51] = 6, -6, 6, -6, 6, -4
    for h in ("k", "v"):
        assert (got[h + "_scale"].float() == 448).all() and torch.equal(got[h].float().flatten(), want)


EDGES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def nearest(y):
    """Elements and scales of y (64 bits), a tie to the even code.  A quotient that is no border lies further from it
    than 64 bits round."""
    y = y.unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn).double()
    z = torch.where(s[..., None] > 0, y / s[..., None], 0.0)
    code = torch.zeros_like(z, dtype=torch.long)
    for i, e in enumerate(EDGES):
        code += (z.abs() > e) if i % 2 == 0 else (z.abs() >= e)
    return (torch.tensor(E2M1, dtype=torch.float64, device=y.device)[code] * z.sign()).flatten(-2), s


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("unit", [1.0, 2.0 ** -5, 2.0 ** 9])
def test_append_takes_the_nearest_code_at_every_border(dtype, unit):
    # a group for each scale: its largest element gives that scale, the others lie at a border of two codes and one
    # step of the type to either side of it
    dt, d = DTYPES[dtype], 64
    scales = torch.arange(1, 127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).float()
    edges = torch.tensor(EDGES, device="cuda")
    at = (scales[:, None] * edges * unit).to(dt)
    assert torch.equal(at.double(), scales.double()[:, None] * edges.double() * unit) or dt == torch.float16
    rows = []
    for step in (-1, 0, 1):
        x = torch.zeros(126, 16, device="cuda").to(dt)
        x[:, 0] = (scales * 6 * unit).to(dt)
        x[:, 1:8] = (at.view(torch.int32 if dt == torch.float32 else torch.int16) + step).view(dt)
        x[:, 8:15] = -x[:, 1:8]
        rows.append(x)
    x = torch.cat(rows + [torch.zeros(2, 16, device="cuda").to(dt)]).view(-1, 1, d)
    x = torch.where(x.isfinite(), x, 0)
    n = x.shape[0]
    where = (i32([0, n]), i32([n]), i32([list(range(-(-n // 16)))]))
    cache = ds.PagedCache.empty(-(-n // 16), 1, d, 16, k_scale=unit, v_scale=unit)
    ok(ds.cache_append(cache, x, x, *where)["status"])
    got = ds.cache_read(cache, *where, n)
    want, s = nearest(x.double() / unit)
    for h in ("k", "v"):
        assert torch.equal(got[h + "_scale"].double(), s) and torch.equal(got[h].double(), want)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("layout,d", [("half", 128), ("interleaved", 64)])
def test_append_takes_the_nearest_codes_of_normed_and_turned_keys(dtype, layout, d):
    # a normed and turned key has all the bits of fp32, as norm_rope gives them of the same heads in fp32
    g, dt, n, hkv = gen(43), DTYPES[dtype], 8192, 8
    k, w, rope = randn(g, n, hkv, d).to(dt), (1 + 0.1 * randn(g, d)).to(dt), ds.Rope(d, layout=layout)
    where = (i32([0, n]), i32([n]), i32([list(range(n // 64))]))
    cache = ds.PagedCache.empty(n // 64, hkv, d, 64, k_scale=0.5)
    ok(ds.cache_append(cache, k, k, *where, rope=rope, k_weight=w)["status"])
    got = ds.cache_read(cache, *where, n)
    y = ds.norm_rope(k.float(), None, i32(list(range(n))), rope, q_weight=w.float())["q"]
    e, s = nearest(y.double() / 0.5)
    assert torch.equal(got["k_scale"].double(), s) and torch.equal(got["k"].double(), e)


def test_norm_weights_off_a_boundary_are_refused():
    g, d = gen(44), 64
    q, flat = randn(g, 2, 2, d).bfloat16(), torch.ones(2 * d, device="cuda").bfloat16()
    cache, where = ds.PagedCache.empty(1, 2, d, 16), (i32([0, 2]), i32([2]), i32([[0]]))
    good = flat[8: 8 + d]                                     # 16 bytes on
    want = ds.norm_rope(q, q, q_weight=flat[:d], k_weight=flat[:d])
    got = ds.norm_rope(q, q, q_weight=good, k_weight=good)
    assert torch.equal(got["q"], want["q"]) and torch.equal(got["k"], want["k"])
    for at in (1, 4, 7):
        bad = flat[at: at + d]
        for kw in (dict(q_weight=bad), dict(k_weight=bad)):
            with pytest.raises(ValueError, match="16-byte"):
                ds.norm_rope(q, q, **kw)
            with pytest.raises(ValueError, match="16-byte"):
                ds.cache_append(cache, q, q, *where, q=q, **kw)


# ---------------------------------------------------------------------------------------------------------------
# what a row sees
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_a_window_past_every_token_is_none(d, causal):
    g, n, kv = gen(45), [5, 12, 2], [2, 7, 90]               # two requests with rows before their first token
    table, pages = paged(g, kv, 16)
    cache, held = filled(g, kv, table, pages, 1, d, 16)
    q = randn(g, sum(n), 3, d).bfloat16()
    args = (q, cache, offsets(n), i32(kv), table)
    want = ds.attend_paged(*args, causal=causal, want_lse=True)
    attend_check(q, want, held, n, kv, d ** -0.5, causal, 0)
    for window in (90, 2 ** 30, 2 ** 31 - 12, 2 ** 31 - 3, 2 ** 31 - 1):
        got = ds.attend_paged(*args, causal=causal, window=window, want_lse=True)
        ok(got["status"])
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"]), window


@pytest.mark.parametrize("d,page,n,window,causal", [
    (128, 16, 1, 20, True), (64, 16, 3, 33, True), (64, 32, 2, 1, True), (128, 48, 7, 17, True), (64, 48, 5, 40, False),
    (128, 64, 2, 30, True), (128, 16, 30, 9, True)])
def test_pages_that_the_window_has_left_are_not_looked_up(d, page, n, window, causal):
    g, kv = gen(46 + d + page), list(range(40, 300, 13))
    B, rows = len(kv), [n] * len(kv)
    table, pages = paged(g, kv, page)
    cache, held = filled(g, kv, table, pages, 2, d, page)
    q = randn(g, sum(rows), 4, d).half()
    args = dict(causal=causal, window=window, max_rows=n, want_lse=True)
    want = ds.attend_paged(q, cache, offsets(rows), i32(kv), table, **args)
    ok(want["status"])
    freed = table.clone()
    for r in range(B):
        first = max(0, (kv[r] - n + 1 if causal else kv[r]) - window)       # the first token that a row sees
        freed[r, : first // page] = -1
    assert (freed != table).any()
    got = ds.attend_paged(q, cache, offsets(rows), i32(kv), freed, **args)
    ok(got["status"])
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    attend_check(q, got, held, rows, kv, d ** -0.5, causal, window)
    freed[0, (kv[0] - 1) // page] = pages                 # one that a row does see
    bad = ds.attend_paged(q, cache, offsets(rows), i32(kv), freed, **args)["status"]
    assert ds.check(bad) == "DSPARK_ERR_PAGES"


def test_pages_that_the_window_has_left_of_a_request_in_parts():
    g, d, page, kv, window = gen(47), 128, 16, [60007], 39985
    table, pages = paged(g, kv, page)
    cache, held = filled(g, kv, table, pages, 1, d, page)
    q = randn(g, 2, 4, d).bfloat16()
    freed = table.clone()
    freed[0, : (kv[0] - 1 - window) // page] = -1
    got = ds.attend_paged(q, cache, offsets([2]), i32(kv), freed, window=window, want_lse=True)
    ok(got["status"])
    assert got["workspace"] is not None
    attend_check(q, got, held, [2], kv, d ** -0.5, True, window)


# ---------------------------------------------------------------------------------------------------------------
# streams and failed steps
# ---------------------------------------------------------------------------------------------------------------
def each_operator(seed=48, kv=(50, 20)):
    """name -> (call(**kw), its outputs' names) of every operator, on inputs of its own."""
    g, n, d, page = gen(seed), [3, 1], 64, 16
    table, pages = paged(g, list(kv), page)
    cache, _ = filled(g, list(kv), table, pages, 2, d, page)
    x = randn(g, 4, 8, d).bfloat16()
    rope, off, lens = ds.Rope(d), offsets(n), i32(list(kv))
    one, z = torch.full((2,), 1.5, device="cuda"), randn(g, 4, 999)
    hist, two, pos = i32([[1, 2, 3], [4, 5, 998]]), i32([2, 3]), i32([5, 6, 7, 8])
    return {
        "norm_rope": (lambda **kw: ds.norm_rope(x[:, :4], x[:, 4:6], pos, rope, **kw), ("q", "k")),
        "cache_append": (lambda **kw: ds.cache_append(cache, x[:, 4:6], x[:, 6:], off, lens, table, rope=rope,
                                                      q=x[:, :4], **kw), ("q",)),
        "cache_read": (lambda **kw: ds.cache_read(cache, off, lens, table, 4, **kw), ("k", "k_scale", "v", "v_scale")),
        "attend_paged": (lambda **kw: ds.attend_paged(x[:, :4], cache, off, lens, table, max_rows=3, want_lse=True, **kw),
                         ("out", "lse")),
        "penalize_logits": (lambda **kw: ds.penalize_logits(z, off, hist, two, two, one, one, one, **kw), ("logits",)),
    }


def bits(t):
    return t.contiguous().view(torch.uint8).clone()


@pytest.mark.parametrize("name", ["norm_rope", "cache_append", "cache_read", "attend_paged", "penalize_logits"])
def test_a_stream_of_its_own_while_the_current_one_is_busy(name):
    call, outputs = each_operator()[name]
    want = call()
    ok(want["status"])
    words = [torch.full((1,), 8, dtype=torch.int32, device="cuda") for _ in range(256)]   # freed words that hold an error
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    del words[::2]
    torch.cuda._sleep(200_000_000)                          # a tenth of a second that the current stream has to do
    got = call(stream=side)
    with torch.cuda.stream(side):
        kept = {h: bits(got[h]) for h in outputs}
    assert ds.check(got["status"], stream=side) == "DSPARK_OK"
    side.synchronize()
    for h in outputs:
        assert torch.equal(kept[h], bits(want[h]))


def test_a_result_dropped_at_once_keeps_its_memory_until_its_stream_is_done():
    g, d, kv = gen(49), 128, [60000]
    table, pages = paged(g, kv, 64)
    cache, _ = filled(g, kv, table, pages, 1, d, 64)
    q, off, lens = randn(g, 1, 8, d).bfloat16(), offsets([1]), i32(kv)
    want = ds.attend_paged(q, cache, off, lens, table)
    size = want["workspace"].numel()
    side, out = torch.cuda.Stream(), torch.empty_like(want["out"])
    want = want["out"].clone()
    for _ in range(5):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        ds.attend_paged(q, cache, off, lens, table, out=dict(out=out), stream=side)      # its workspace is dropped here
        for _ in range(4000):                                  # the current stream takes what memory is free
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        side.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("name", ["norm_rope", "cache_append", "cache_read", "attend_paged", "penalize_logits"])
def test_a_step_that_failed_leaves_the_outputs_alone(name):
    call, outputs = each_operator()[name]
    good = call()
    out = {h: torch.full_like(good[h], 3.0) for h in outputs}
    st = i32([8])
    call(status=st, out=out)
    assert ds.check(st) == "DSPARK_ERR_LENGTHS"
    assert all((out[h].float() == 3).all() for h in outputs)


def test_a_step_that_failed_leaves_attention_in_parts_alone():
    g, d, kv = gen(50), 64, [40000]
    table, pages = paged(g, kv, 64)
    cache, _ = filled(g, kv, table, pages, 1, d, 64)
    q, out = randn(g, 2, 2, d).half(), dict(out=torch.full((2, 2, d), 3.0, device="cuda").half())
    st = i32([8])
    got = ds.attend_paged(q, cache, offsets([2]), i32(kv), table, out=out, status=st)
    assert got["workspace"] is not None and ds.check(st) == "DSPARK_ERR_LENGTHS" and (out["out"] == 3).all()
