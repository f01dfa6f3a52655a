"""The operators around a ragged verification step against plain 64-bit implementations, at the sizes and masks
where they can go wrong.

Tolerances count roundings: half(t) = torch.finfo(t).eps / 2 relative for a value stored in t, 2^-24 for an fp32
operation on a value of the stated size.
"""
import math

import pytest
import torch

import speculative_decoding_draft_gb300 as ds

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F32 = 2.0 ** -24
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_draft_gb300 import build
    build.build()


def half(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def ok(status):
    assert ds.check(status) == "DSPARK_OK"


def offsets(n):
    return i32([sum(n[:i]) for i in range(len(n) + 1)])


def paged(g, kv, page, spare=0, width=0):
    """A page table over shuffled pages and the number of pages."""
    need = [-(-k // page) for k in kv]
    ids = (torch.randperm(sum(need) + spare, generator=g, device="cuda")).tolist()
    wide = max([1, width] + need)
    table, at = [], 0
    for m in need:
        table.append(ids[at: at + m] + [-7] * (wide - m))     # entries past a request's pages are not read
        at += m
    return i32(table), max(1, sum(need) + spare)


# ---------------------------------------------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------------------------------------------
def rotate64(x, weight, eps, pos, rope):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    if rope is None:
        return x
    r, y = rope.rotary_dim, x.clone()
    ang = pos.double()[:, None] * rope.inv_freq.to(x.device)
    c, s = (torch.cos(ang) * rope.gain)[:, None], (torch.sin(ang) * rope.gain)[:, None]
    a, b = (slice(0, r // 2), slice(r // 2, r)) if rope.layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def rotate_bound(ref, dtype, gain):
    # norm: D/8 + log2 sums, rsqrt, two products; rotation: two products, an addition, cos and sin to 2^-22
    size = ref.abs().amax(-1, keepdim=True) * max(1.0, gain) * math.sqrt(2)
    return half(dtype) * ref.abs() + 64 * F32 * size + torch.finfo(dtype).smallest_normal * half(dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d,rot,layout,scaling", [
    (16, 16, "half", "none"), (64, 64, "half", "linear"), (64, 32, "interleaved", "ntk"), (80, 80, "half", "none"),
    (96, 48, "half", "yarn"), (128, 128, "interleaved", "yarn"), (128, 64, "half", "none"), (256, 256, "half", "ntk"),
    (240, 16, "interleaved", "none")])
@pytest.mark.parametrize("rows,hq,hkv,norm", [(1, 1, 1, True), (7, 5, 2, False), (33, 12, 4, True)])
def test_norm_rope(dtype, d, rot, layout, scaling, rows, hq, hkv, norm):
    g, dt = gen(rows * 1000 + d), DTYPES[dtype]
    rope = ds.Rope(rot, base=5e5, layout=layout, scaling=scaling, factor=4.0, original_len=4096)
    qkv = randn(g, rows, hq + 2 * hkv, d).to(dt)             # heads of a fused projection: strided rows
    q, k = qkv[:, :hq], qkv[:, hq: hq + hkv]
    pos = torch.randint(0, 2 ** 21, (rows,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 0
    pos[-1] = 2 ** 31 - 1                                    # as exact at the last position as at the first
    w = [(1 + 0.2 * randn(g, d)).to(dt) if norm else None for _ in range(2)]
    got = ds.norm_rope(q, k, pos, rope, q_weight=w[0], k_weight=w[1], eps=1e-5)
    ok(got["status"])
    for x, weight, y in ((q, w[0], got["q"]), (k, w[1], got["k"])):
        ref = rotate64(x, weight, 1e-5, pos, rope)
        # the turn is kept to 2^-65 turns a position: at 2^31 positions 2^-34 turns, nothing beside fp32
        assert ((y.double() - ref).abs() <= rotate_bound(ref, dt, rope.gain)).all()


def test_norm_rope_norms_one_of_the_two_and_runs_in_place():
    g = gen(3)
    q, k = randn(g, 9, 6, 128).bfloat16(), randn(g, 9, 2, 128).bfloat16()
    w, pos, rope = (1 + randn(g, 128)).bfloat16(), i32(list(range(9))), ds.Rope(128)
    want_q, want_k = rotate64(q, w, 1e-6, pos, rope), rotate64(k, None, 0, pos, rope)
    got = ds.norm_rope(q, k, pos, rope, q_weight=w, out=dict(q=q, k=k))
    assert got["q"].data_ptr() == q.data_ptr() and got["k"].data_ptr() == k.data_ptr()
    for y, ref in ((q, want_q), (k, want_k)):
        assert ((y.double() - ref).abs() <= rotate_bound(ref, torch.bfloat16, 1.0)).all()
    q, want = randn(g, 9, 6, 128), None                       # a norm alone, queries alone
    want = rotate64(q, w.float(), 1e-6, pos, None)
    got = ds.norm_rope(q, q_weight=w.float())
    assert got["k"] is None and ((got["q"].double() - want).abs() <= rotate_bound(want, torch.float32, 1.0)).all()


def test_norm_rope_heads_of_zeros_and_nans():
    q = torch.zeros(2, 4, 64, device="cuda", dtype=torch.float16)
    q[0, 1, 5] = math.nan
    got = ds.norm_rope(q, None, i32([1, 2]), ds.Rope(64), q_weight=torch.ones(64, device="cuda").half(), eps=0.0)["q"]
    assert torch.isnan(got[0, 1]).all()                      # 0 / 0 elsewhere: eps 0 is the caller's choice
    got = ds.norm_rope(q, None, i32([1, 2]), ds.Rope(64), q_weight=torch.ones(64, device="cuda").half())["q"]
    assert torch.isnan(got[0, 1]).all() and not got[1].any() and not got[0, 2:].any()


# ---------------------------------------------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------------------------------------------
def quantize64(y):
    """Elements, scales and the distance of each quotient to the nearest border of two elements."""
    y = y.unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn).double()
    z = torch.where(s[..., None] > 0, y / s[..., None], 0.0)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=y.device)
    code = torch.zeros_like(z, dtype=torch.long)
    for i, e in enumerate(edges):
        code += (z.abs() > e) if i % 2 == 0 else (z.abs() >= e)      # a tie goes to the even code
    near = (z.abs()[..., None] - edges).abs().amin(-1)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=y.device)
    return (grid[code] * z.sign()).flatten(-2), s, near.flatten(-2)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,ahead,d,hkv,hq,page", [
    ([1], [0], 64, 1, 0, 16), ([1, 0, 3, 0], [15, 4, 14, 0], 128, 2, 4, 16), ([5, 33, 2], [61, 0, 127], 128, 3, 3, 64),
    ([70, 1], [10, 1000], 64, 2, 8, 32), ([2] * 70, list(range(70)), 64, 1, 1, 48)])
@pytest.mark.parametrize("scaled", [False, True])
def test_append_and_read(dtype, n, ahead, d, hkv, hq, page, scaled):
    g, dt = gen(sum(n) + d), DTYPES[dtype]
    kv = [a + b for a, b in zip(n, ahead)]
    table, pages = paged(g, kv, page, spare=3)
    rows, pad = sum(n), 4                                       # rows past row_off[B] are left alone
    off, kv_len = offsets(n), i32(kv)
    ks, vs = (0.25, 8.0) if scaled else (1.0, 1.0)
    data = torch.randint(0, 256, (pages, hkv, page // 16, 18 * d), generator=g, device="cuda", dtype=torch.uint8)
    cache, before = ds.PagedCache(data, page, k_scale=ks, v_scale=vs), data.clone()
    x = randn(g, rows + pad, hq + 2 * hkv, d).to(dt)
    q, k, v = x[:, :hq], x[:, hq: hq + hkv], x[:, hq + hkv:]
    k[0, 0, :16] = 0
    v[0, 0, 16:32] = 0
    rope, w = ds.Rope(d // 2, layout="interleaved"), (1 + 0.1 * randn(g, d)).to(dt)
    got = ds.cache_append(cache, k, v, off, kv_len, table, rope=rope, k_weight=w, q=q if hq else None, q_weight=w)
    ok(got["status"])
    back = ds.cache_read(cache, off, kv_len, table, rows)
    ok(back["status"])
    pos = i32([a + i for a, m in zip(ahead, n) for i in range(m)])
    if hq:
        ref = rotate64(q[:rows], w, 1e-6, pos, rope)
        assert ((got["q"][:rows].double() - ref).abs() <= rotate_bound(ref, dt, 1.0)).all()
    e, s, _ = quantize64(v[:rows].double() / vs)                # values: exact, ties included
    assert torch.equal(back["v"].double(), e) and torch.equal(back["v_scale"].double(), s)
    y = rotate64(k[:rows], w, 1e-6, pos, rope) / ks
    e, s, near = quantize64(y)
    # fp32 norm and rotation move a key by 64 * 2^-24 of its head's largest, a scale where its quotient lies as near
    # to a border (e4m3 steps of 2^-3): then the group counts as one with another scale
    same = back["k_scale"].double() == s
    assert same.double().mean() > 0.999
    wide = same.repeat_interleave(16, -1)
    slack = 64 * F32 * y.abs().amax(-1, keepdim=True) / s.clamp(min=2.0 ** -9).repeat_interleave(16, -1)
    assert ((back["k"].double() == e) | (near <= slack) | ~wide).all()
    # nothing else was written
    touched = torch.zeros_like(data, dtype=torch.bool)
    for r, m in enumerate(n):
        for p in range(ahead[r], kv[r]):
            tile, t, c = touched[table[r, p // page], :, p % page // 16], p % 16, torch.arange(8, device="cuda")
            tile[:, t * d // 2: (t + 1) * d // 2] = True
            tile[:, 16 * d + t * d // 16: 16 * d + (t + 1) * d // 16] = True
            at = 8 * d + d // 16 * (64 * (t // 8) + 8 * c + t % 8)
            tile[:, (at[:, None] + torch.arange(d // 16, device="cuda")).flatten()] = True
            tile[:, 17 * d + t // 8 * d // 2 + 8 * torch.arange(d // 16, device="cuda") + t % 8] = True
    assert torch.equal(data[~touched], before[~touched])


def test_append_of_infinities_nans_and_tiny_values():
    d = 64
    k = torch.full((1, 1, d), 1e-6, device="cuda")
    v = torch.ones(1, 1, d, device="cuda")
    k[0, 0, 16], k[0, 0, 33], k[0, 0, 50] = math.inf, math.nan, 1e9
    v[0, 0, 3] = -math.inf
    cache = ds.PagedCache.empty(1, 1, d, 16)
    args = (cache, k, v, i32([0, 1]), i32([1]), i32([[0]]))
    ok(ds.cache_append(*args)["status"])
    got = ds.cache_read(cache, *args[3:], 1)
    s = got["k_scale"].float().flatten()
    assert s[0] == 0 and s[1] == 448 and math.isnan(s[2]) and s[3] == 448
    e = got["k"].float().flatten()
    assert not e[:16].any() and e[16] == 6 and not e[17:32].any() and not e[32:48].any() and e[50] == 6
    assert got["v_scale"].float()[0, 0, 0] == 448 and got["v"].float()[0, 0, 3] == -6


def test_append_at_explicit_positions():
    g, d = gen(8), 128
    k, v, pos = randn(g, 2, 1, d).bfloat16(), randn(g, 2, 1, d).bfloat16(), i32([70, 900])
    rope, out = ds.Rope(d), []
    for kw in (dict(positions=pos, rope=rope), dict()):
        cache = ds.PagedCache.empty(2, 1, d, 16)
        x = k if kw else rotate64(k, None, 0, pos, rope).float()
        ds.cache_append(cache, x, v if kw else v.float(), i32([0, 2]), i32([3]), i32([[1, 0]]), **kw)
        out.append(ds.cache_read(cache, i32([0, 2]), i32([3]), i32([[1, 0]]), 2)["k"].float())
    assert (out[0] == out[1]).float().mean() > 0.99


# ---------------------------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------------------------
def filled(g, kv, table, pages, hkv, d, page, dtype=torch.bfloat16, std=1.0, data=None):
    """A cache with random tokens of every request and NaN everywhere else, and its values."""
    data = torch.full((pages, hkv, page // 16, 18 * d), 255, dtype=torch.uint8, device="cuda") if data is None else data
    cache = ds.PagedCache(data, page, k_scale=0.5, v_scale=2.0)
    off, total = offsets(kv), sum(kv)
    k, v = (randn(g, max(1, total), hkv, d).mul(std).to(dtype) for _ in range(2))
    if total:
        ok(ds.cache_append(cache, k, v, off, i32(kv), table)["status"])
    c = ds.cache_read(cache, off, i32(kv), table, max(1, total))
    wide = lambda x, s: x.double() * s.double().repeat_interleave(16, -1)  # noqa: E731
    k, v = wide(c["k"], c["k_scale"]) * 0.5, wide(c["v"], c["v_scale"]) * 2.0
    at = off.tolist()
    return cache, [(k[a:b], v[a:b]) for a, b in zip(at, at[1:])]


def attend_check(q, got, held, n, kv, scale, causal, window):
    dt, row = q.dtype, 0
    for r, m in enumerate(n):
        k, v = held[r]
        for j in range(m):
            hi = kv[r] - m + j + 1 if causal else kv[r]
            lo = max(0, hi - window) if window else 0
            y, z = got["out"][row].double(), got["lse"][row].double()
            x = q[row].double()
            row += 1
            if hi <= lo:
                assert not y.any() and (z == -math.inf).all()
                continue
            group = q.shape[1] // k.shape[1]
            kk, vv = (t[lo:hi].repeat_interleave(group, 1).transpose(0, 1) for t in (k, v))   # [Hq, T, D]
            s = (kk @ x[..., None])[..., 0] * scale
            ref_lse = torch.logsumexp(s, -1)
            p = torch.exp(s - ref_lse[:, None])
            ref = (p[:, None] @ vv)[:, 0]
            # scores: 128 fp32 additions; probabilities: rounded to fp16, exponent to 2^-20; tiny ones kept to 2^-31
            ds_ = 128 * F32 * ((kk.abs() @ x.abs()[..., None])[..., 0] * abs(scale)).amax(-1, keepdim=True)
            rel = half(torch.float16) + 2 * ds_ + 2.0 ** -20 + 64 * F32
            bound = half(dt) * ref.abs() + rel * (p[:, None] @ vv.abs())[:, 0] + 2.0 ** -30 * vv.abs().sum(1)
            assert ((y - ref).abs() <= bound + 2.0 ** -25).all()
            assert ((z - ref_lse).abs() <= ds_[:, 0] + 2.0 ** -20 + 8 * F32 * ref_lse.abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,kv,d,hkv,group,page,causal,window", [
    ([1], [1], 128, 1, 1, 16, True, 0),
    ([1], [0], 64, 2, 4, 16, True, 0),                                     # nothing in the cache
    ([1, 1, 1], [15, 16, 17], 128, 2, 4, 16, True, 0),
    ([3, 0, 8, 1], [2, 9, 300, 0], 64, 2, 4, 32, True, 0),                 # a request before its tokens, one without rows
    ([8, 5, 1], [700, 31, 33], 128, 2, 3, 64, True, 0),                    # 24 row-heads, an odd group
    ([7, 2], [513, 2049], 128, 1, 8, 128, True, 100),
    ([4, 9], [40, 4100], 64, 4, 2, 48, True, 33),
    ([8, 8], [257, 64], 128, 1, 2, 32, False, 0),                          # a block that attends to all of itself
    ([6], [90], 64, 1, 1, 16, False, 17),
    ([40, 3], [41, 1000], 128, 2, 4, 64, True, 0),                         # several tiles of rows
    ([16], [5000], 64, 1, 1, 64, True, 0),
    ([1, 2], [9000, 3], 128, 8, 2, 64, True, 0)])
def test_attend(dtype, n, kv, d, hkv, group, page, causal, window):
    g, dt = gen(sum(kv) + d), DTYPES[dtype]
    table, pages = paged(g, kv, page, spare=2)
    cache, held = filled(g, kv, table, pages, hkv, d, page)
    rows = sum(n)
    x = randn(g, rows, hkv * group + 1, d).to(dt)               # a strided view
    q = x[:, : hkv * group]
    got = ds.attend_paged(q, cache, offsets(n), i32(kv), table, causal=causal, window=window, max_rows=max(n),
                          want_lse=True)
    ok(got["status"])
    attend_check(q, got, held, n, kv, 1 / math.sqrt(d), causal, window)


def test_attend_sharp_scores_and_other_scales():
    # scores of hundreds: the running maximum moves all the time, most probabilities vanish
    g, n, kv, d = gen(5), [4, 1], [3000, 77], 128
    table, pages = paged(g, kv, 64)
    cache, held = filled(g, kv, table, pages, 2, d, 64, std=6.0)
    q = randn(g, 5, 4, d).mul(8.0).bfloat16()
    for scale in (1.0, -0.3, 1e-4, 0.0):
        got = ds.attend_paged(q, cache, offsets(n), i32(kv), table, scale=scale, want_lse=True)
        attend_check(q, got, held, n, kv, scale, True, 0)
    big, small = q * 2.0 ** 100, (q.float() * 2.0 ** -120).bfloat16()
    for x, scale in ((big, 2.0 ** -104), (small, 2.0 ** 116)):
        attend_check(x, ds.attend_paged(x, cache, offsets(n), i32(kv), table, scale=scale, want_lse=True), held, n, kv,
                     scale, True, 0)


def test_attend_one_row_is_the_same_with_others_beside_it():
    # default max_rows, and padding rows past row_off[B] that stay as they are
    g, n, kv = gen(6), [2, 1], [130, 50]
    table, pages = paged(g, kv, 32, width=9)
    cache, held = filled(g, kv, table, pages, 2, 64, 32)
    q = randn(g, 8, 4, 64).half()
    out = dict(out=torch.full((8, 4, 64), 7.0, device="cuda").half(), lse=torch.full((8, 4), 7.0, device="cuda"))
    got = ds.attend_paged(q, cache, offsets(n), i32(kv), table, want_lse=True, out=out)
    ok(got["status"])
    attend_check(q[:3], got, held, n, kv, 0.125, True, 0)
    assert (got["out"][3:] == 7).all() and (got["lse"][3:] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
def test_attend_keeps_nans_to_the_rows_that_see_them(d):
    # token 37 of 40 holds NaN (a group of its value, then of its key): of rows 35 .. 39 only 37 on see it
    g, n, kv = gen(7), [5], [40]
    for part in ("v", "k"):
        table, pages = paged(g, kv, 16)
        cache, held = filled(g, kv, table, pages, 1, d, 16)
        k, v = held[0]
        bad = torch.zeros(1, 1, d, device="cuda", dtype=torch.float32)
        bad[0, 0, 20] = math.nan
        zero = torch.ones_like(bad)
        ds.cache_append(cache, bad if part == "k" else zero, bad if part == "v" else zero, i32([0, 1]), i32([38]), table)
        q = randn(g, 5, 2, d).bfloat16()
        got = ds.attend_paged(q, cache, offsets(n), i32(kv), table, want_lse=True)
        out = got["out"].float()
        assert not torch.isnan(out[:2]).any()
        if part == "v":
            assert torch.isnan(out[2:, :, 16:32]).all()
            assert not torch.isnan(out[2:, :, :16]).any() and not torch.isnan(out[2:, :, 32:]).any()
        else:
            assert torch.isnan(out[2:]).all() and torch.isnan(got["lse"][2:]).all()
        # within a window that has passed it again
        out = ds.attend_paged(q, cache, offsets(n), i32(kv), table, window=2)["out"].float()
        assert not torch.isnan(out[:2]).any() and not torch.isnan(out[4:]).any()
        assert torch.isnan(out[2:4]).any(-1).all()
        attend_check(q[:2], dict(out=got["out"], lse=got["lse"]), [(k[:37], v[:37])], [2], [37], d ** -0.5, True, 0)


def test_attend_over_a_cache_past_four_gigabytes():
    g, d, hkv, page, kv = gen(9), 128, 8, 64, [200, 64]
    per = hkv * (page // 16) * 18 * d
    pages = (5 << 30) // per
    data = torch.empty(pages, hkv, page // 16, 18 * d, dtype=torch.uint8, device="cuda")
    table = i32([[pages - 1, 3, pages - 2, pages - 9], [pages - 4, -1, -1, -1]])
    cache, held = filled(g, kv, table, pages, hkv, d, page, data=data)
    q = randn(g, 3, 16, d).bfloat16()
    got = ds.attend_paged(q, cache, offsets([2, 1]), i32(kv), table, want_lse=True)
    ok(got["status"])
    attend_check(q, got, held, [2, 1], kv, d ** -0.5, True, 0)


@pytest.mark.parametrize("n,kv,d,hkv,group,page", [
    ([300], [333], 128, 2, 4, 64),                     # a prompt chunk: many tiles of 32 rows
    ([70, 1, 130], [70, 500, 140], 64, 1, 3, 32),
    ([1] * 300, [3 * i % 97 for i in range(300)], 64, 1, 2, 16),      # more requests than are put in order
    ([8], [40000], 128, 1, 4, 64),                     # one key/value head: split through the workspace
    ([2], [40000], 64, 2, 1, 48)])
def test_attend_shapes_of_the_launch(n, kv, d, hkv, group, page):
    g = gen(len(n) + d)
    table, pages = paged(g, kv, page)
    cache, held = filled(g, kv, table, pages, hkv, d, page)
    q = randn(g, sum(n), hkv * group, d).half()
    got = ds.attend_paged(q, cache, offsets(n), i32(kv), table, max_rows=max(n), want_lse=True)
    ok(got["status"])
    attend_check(q, got, held, n, kv, d ** -0.5, True, 0)
    again = ds.attend_paged(q, cache, offsets(n), i32(kv), table, max_rows=max(n), want_lse=True,
                            workspace=got["workspace"])
    assert torch.equal(again["out"], got["out"]) and torch.equal(again["lse"], got["lse"])       # the order of sums is fixed


def test_heads_with_gaps_between_them():
    g, d, n, kv = gen(21), 64, [5, 2], [25, 40]
    table, pages = paged(g, kv, 16)
    x = randn(g, 7, 9, d + 24).bfloat16()[..., :d]      # a head's rows do not follow one another
    q, k, v = x[:, :5], x[:, 5:7], x[:, 7:]
    pos, rope, w = i32(list(range(7))), ds.Rope(d), (1 + 0.1 * randn(g, d)).bfloat16()
    a, b = (ds.norm_rope(*t, pos, rope, q_weight=w) for t in ((q, k), (q.contiguous(), k.contiguous())))
    assert torch.equal(a["q"], b["q"]) and torch.equal(a["k"], b["k"])
    kept = []
    for t in ((q, k, v), (q.contiguous(), k.contiguous(), v.contiguous())):
        cache = ds.PagedCache.empty(pages, 2, d, 16)
        got = ds.cache_append(cache, t[1], t[2], offsets(n), i32(kv), table, rope=rope, k_weight=w, q=t[0], q_weight=w)
        out = ds.attend_paged(t[0][:, :4], cache, offsets(n), i32(kv), table)
        kept.append((got["q"], cache.data, out["out"]))
    assert all(torch.equal(s, t) for s, t in zip(*kept))


def test_attend_workspace():
    import ctypes
    from speculative_decoding_draft_gb300 import serving as sv
    g, d, kv = gen(22), 128, [40000]              # long enough to be split
    table, pages = paged(g, kv, 64)
    cache, _ = filled(g, kv, table, pages, 1, d, 64)
    q, off, lens = randn(g, 1, 2, d).bfloat16(), offsets([1]), i32(kv)
    st, out = ds.new_status("cuda"), torch.empty(1, 2, d, device="cuda").bfloat16()
    where = sv._Ragged(off.data_ptr(), lens.data_ptr(), table.data_ptr(), 1, 1, table.shape[1])
    heads, L = sv._Heads(q.data_ptr(), 2 * d, d), ds.lib()
    need = L.dspark_attn_paged_workspace_bytes(2, cache._c, where, 1)
    assert need > 0
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")

    def call(at, size):
        return L.dspark_attn_paged(heads, 2, 1, cache._c, where, 1, 0.1, 1, 0, out.data_ptr(), None, at, size,
                                   st.data_ptr(), None)
    assert call(None, 0) == 10 and call(ws.data_ptr(), need - 1) == 10 and call(ws.data_ptr() + 16, need) == 10
    assert call(ws.data_ptr(), need) == 0
    ok(st)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")          # too small a one is replaced
    got = ds.attend_paged(q, cache, off, lens, table, scale=0.1, workspace=small)
    assert torch.equal(got["out"], out) and got["workspace"].numel() >= need


# ---------------------------------------------------------------------------------------------------------------
# penalties
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,V,cap,n_bias,mask,draft", [
    ([1], 2, 1, 0, False, False), ([3, 0, 1], 33, 5, 2, True, True), ([4, 2], 4095, 300, 5, True, True),
    ([2, 8], 4097, 64, 0, True, True), ([1, 1, 5], 10000, 1000, 40, False, True), ([8], 131072, 5000, 3, True, False), ([2, 1], 3000, 7, 4096, False, True)])
def test_penalize(dtype, n, V, cap, n_bias, mask, draft):
    g, dt, B, rows, K = gen(V + cap), DTYPES[dtype], len(n), sum(n), max(n)
    ints = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    z = (randn(g, rows + 2, V) * 3).to(dt)
    z[0, :2] = torch.tensor([0.0, -math.inf], device="cuda").to(dt)
    hist = (ints(0, V, B, cap).float() ** 2 / V).int()                 # tokens that repeat
    hist[0, 0] = V - 1
    hist_len = ints(0, cap + 1, B)
    hist_len[0], hist_len[-1] = cap, 0 if B > 1 else cap
    prompt = torch.minimum(ints(0, cap + 1, B), hist_len)
    rep, pre, fre = (1 + torch.rand(B, generator=g, device="cuda") for _ in range(3))
    rep[-1] = 0.7
    tok = (ints(0, V, B, K).float() ** 2 / V).int()
    bt = bv = words = None
    if n_bias:
        bt, bv = ints(-1, V, B, n_bias), randn(g, B, n_bias)
        bt[0, 0] = bt[0, -1] = V - 1                                 # listed twice
    if mask:
        words = ints(-2 ** 31, 2 ** 31 - 1, rows + 2, (V + 31) // 32)
        words[0] = 0                                               # nothing allowed
    out = dict(logits=torch.full_like(z, 9.0))
    got = ds.penalize_logits(z, offsets(n), hist, hist_len, prompt, rep, pre, fre, draft_tok=tok if draft else None,
                             bias_tok=bt, bias_val=bv, mask=words, out=out)
    ok(got["status"])
    assert (got["logits"][rows:] == 9).all()
    row = 0
    for r in range(B):
        for j in range(n[r]):
            h, m = hist[r, : hist_len[r]].long(), int(prompt[r])
            said = torch.bincount(h[m:], minlength=V)
            if draft:
                said += torch.bincount(tok[r, :j].long(), minlength=V)
            seen = (said > 0) | (torch.bincount(h[:m], minlength=V) > 0)
            x = z[row].double()
            y = torch.where(seen, torch.where(x > 0, x / rep[r].double(), x * rep[r].double()), x)
            size = y.abs()
            y = y - (said > 0) * pre[r].double() - said * fre[r].double()
            size = size + 2 * (said > 0) * pre[r].double() + 3 * said * fre[r].double()
            if bt is not None:
                for b in range(n_bias):
                    if bt[r, b] >= 0:
                        y[bt[r, b]] += bv[r, b].double()
                        size[bt[r, b]] += 2 * bv[r, b].abs().double()
            if words is not None:
                bits = (words[row][:, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
                y[bits.flatten()[:V] == 0] = -math.inf
            have = got["logits"][row].double()
            fine = y != -math.inf
            assert torch.equal(fine, have != -math.inf)
            # division or product, two subtractions, the biases' sums: each 2^-24 of what it works on
            assert ((have - y)[fine].abs() <= half(dt) * y[fine].abs() + (6 * F32 * size + 2.0 ** -140)[fine]).all()
            row += 1
    again = ds.penalize_logits(z, offsets(n), hist, hist_len, prompt, rep, pre, fre, draft_tok=tok if draft else None,
                               bias_tok=bt, bias_val=bv, mask=words, out=dict(logits=z))["logits"]     # in place
    assert again.data_ptr() == z.data_ptr() and torch.equal(again[:rows], got["logits"][:rows])


# ---------------------------------------------------------------------------------------------------------------
# together, on another stream, in a graph; refusals on the device
# ---------------------------------------------------------------------------------------------------------------
def small_step(seed=11):
    g, n, kv, d, page = gen(seed), [3, 1], [50, 20], 64, 16
    table, pages = paged(g, [64, 64], page)
    cache, _ = filled(g, [64, 64], table, pages, 2, d, page)
    x = randn(g, 4, 8, d).bfloat16()
    rope, st = ds.Rope(d), ds.new_status("cuda")
    off, lens, out = offsets(n), i32(kv), torch.empty(4, 4, d, device="cuda").bfloat16()

    def step():
        q = ds.cache_append(cache, x[:, 4:6], x[:, 6:], off, lens, table, rope=rope, q=x[:, :4], status=st)["q"]
        return ds.attend_paged(q, cache, off, lens, table, max_rows=4, out=dict(out=out), status=st)["out"]
    return step, lens, st


def test_another_stream_and_a_graph_give_the_same():
    step, lens, st = small_step()
    want = step().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step().clone()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    lens += 5                                          # the lengths are the device's: the graph follows them
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out, want) and torch.equal(out.clone(), step())
    ok(st)


def test_device_errors_are_reported_and_leave_the_context_usable():
    g, d = gen(12), 64
    cache = ds.PagedCache.empty(4, 1, d, 16)
    x = randn(g, 3, 1, d).bfloat16()
    off, lens, table = i32([0, 2, 3]), i32([20, 5]), i32([[0, 1], [2, -1]])

    def codes(off, lens, table, max_rows=3):
        a = ds.cache_append(cache, x, x, off, lens, table)["status"]
        r = ds.cache_read(cache, off, lens, table, 3)["status"]
        p = ds.attend_paged(x, cache, off, lens, table, max_rows=max_rows)["status"]
        return [ds.check(s) for s in (a, r, p)]

    assert codes(off, lens, table) == ["DSPARK_OK"] * 3
    assert codes(off, lens, i32([[0, 9], [2, -1]])) == ["DSPARK_ERR_PAGES"] * 3
    assert codes(off, lens, i32([[0, -1], [2, -1]])) == ["DSPARK_ERR_PAGES"] * 3
    assert codes(off, i32([33, 5]), table) == ["DSPARK_ERR_LENGTHS"] * 3
    assert codes(off, i32([1, 5]), table)[:2] == ["DSPARK_ERR_LENGTHS"] * 2      # attention: a row that sees nothing
    assert codes(i32([0, 2, 4]), lens, table)[2] == "DSPARK_ERR_OFFSETS"
    assert codes(i32([2, 0, 3]), lens, table)[2] == "DSPARK_ERR_OFFSETS"
    assert codes(off, lens, table, max_rows=1)[2] == "DSPARK_ERR_LENGTHS"
    # a failed step: later kernels leave everything alone
    st = i32([8])
    keep = cache.data.clone()
    ds.cache_append(cache, -x, -x, off, lens, table, status=st)
    out = torch.full((3, 1, d), 5.0, device="cuda").bfloat16()
    ds.norm_rope(x, status=st, out=dict(q=out))
    assert torch.equal(keep, cache.data) and (out == 5).all() and ds.check(st) == "DSPARK_ERR_LENGTHS"

    def pen(**kw):
        one = torch.ones(2, device="cuda")
        a = dict(off=off, hist=i32([[1, 2], [3, 4]]), hist_len=i32([2, 1]), prompt=i32([1, 0]), tok=i32([[5], [6]]))
        a.update(kw)
        z = torch.zeros(3, 64, device="cuda")
        return ds.check(ds.penalize_logits(z, a["off"], a["hist"], a["hist_len"], a["prompt"], one, one, one,
                                           draft_tok=a["tok"])["status"])

    assert pen() == "DSPARK_OK"
    assert pen(off=i32([0, 2, 9])) == "DSPARK_ERR_OFFSETS"
    assert pen(off=i32([0, 3, 3])) == "DSPARK_ERR_OFFSETS"          # three rows, one draft token
    assert pen(hist_len=i32([3, 1])) == "DSPARK_ERR_LENGTHS"
    assert pen(prompt=i32([1, 2])) == "DSPARK_ERR_LENGTHS"
    assert pen(hist=i32([[1, 64], [3, 4]])) == "DSPARK_ERR_TOKEN_RANGE"
    assert pen(tok=i32([[-1], [6]])) == "DSPARK_ERR_TOKEN_RANGE"


def test_bindings_refuse():
    g, d = gen(13), 64
    cache = ds.PagedCache.empty(4, 2, d, 16)
    q, k = randn(g, 2, 4, d).bfloat16(), randn(g, 2, 2, d).bfloat16()
    off, lens, table, rope = i32([0, 2]), i32([2]), i32([[0]]), ds.Rope(d)
    bad = [
        lambda: ds.norm_rope(q.cpu()), lambda: ds.norm_rope(q.double()), lambda: ds.norm_rope(q[..., ::2]),
        lambda: ds.norm_rope(q[..., :40]), lambda: ds.norm_rope(q, None, None, rope), lambda: ds.norm_rope(q, k.half()),
        lambda: ds.norm_rope(q, None, off[:2].long(), rope), lambda: ds.norm_rope(q, None, lens, rope),
        lambda: ds.norm_rope(q, q_weight=torch.ones(d, device="cuda")),
        lambda: ds.norm_rope(q, out=dict(q=q.half())), lambda: ds.norm_rope(q[..., :32], None, off, ds.Rope(d)),
        lambda: ds.Rope(24), lambda: ds.Rope(64, layout="other"), lambda: ds.Rope(64, scaling="yarn"),
        lambda: ds.PagedCache.empty(4, 2, 96), lambda: ds.PagedCache.empty(4, 2, d, 24),
        lambda: ds.PagedCache(cache.data, 32), lambda: ds.PagedCache(cache.data, 16, k_scale=0.3),
        lambda: ds.cache_append(cache, k, q, off, lens, table), lambda: ds.cache_append(cache, k, k, off, lens[:0], table),
        lambda: ds.cache_append(cache, k, k, off.long(), lens, table), lambda: ds.cache_append(None, k, k, off, lens, table),
        lambda: ds.cache_append(cache, k, k, off, lens, table[0]),
        lambda: ds.attend_paged(q.float(), cache, off, lens, table), lambda: ds.attend_paged(q[:, :3], cache, off, lens, table),
        lambda: ds.attend_paged(q, cache, off, lens, table, window=-1),
        lambda: ds.attend_paged(q, cache, off, lens, table, max_rows=0),
        lambda: ds.penalize_logits(q, off, table, lens, lens, lens.float(), lens.float(), lens.float()),
        lambda: ds.penalize_logits(q[0].half(), off, table, lens, lens, lens.float(), lens.float(), lens.float()),
        lambda: ds.penalize_logits(q[0], off, table, lens, lens, lens, lens.float(), lens.float()),
        lambda: ds.penalize_logits(q[0], off, table, lens, lens, *[lens.float()] * 3, bias_tok=table),
        lambda: ds.penalize_logits(q[0], off, table, lens, lens, *[lens.float()] * 3, mask=table),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError, ds.DsparkError)):
            f()
            pytest.fail(f"case {i} was taken")
    empty = ds.attend_paged(q[:0], cache, i32([0, 0]), lens, table)
    assert empty["out"].shape == (0, 4, d)


def guarded(shape, dtype):
    """A tensor inside a larger one whose surroundings hold a pattern, and a check of these."""
    n, pad, size = math.prod(shape), 4096, torch.empty(0, dtype=dtype).element_size()
    whole = torch.full((n * size + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    inside = whole[pad: pad + n * size].view(dtype).view(shape)
    return inside, lambda: bool((whole[:pad] == 0xA5).all() and (whole[pad + n * size:] == 0xA5).all())


@pytest.mark.parametrize("d,hq,hkv,n,kv,page,V", [(128, 12, 4, [3, 1], [90, 33], 16, 1003), (64, 5, 5, [7], [7], 32, 33)])
def test_nothing_is_written_around_the_outputs(d, hq, hkv, n, kv, page, V):
    g, rows, B = gen(31), sum(n), len(n)
    table, pages = paged(g, kv, page)
    off, lens = offsets(n), i32(kv)
    x = randn(g, rows, hq + 2 * hkv, d).bfloat16()
    q, k, v = x[:, :hq], x[:, hq: hq + hkv], x[:, hq + hkv:]
    f8, bf = torch.float8_e4m3fn, torch.bfloat16
    checks = []

    def room(shape, dtype):
        t, check = guarded(shape, dtype)
        checks.append(check)
        return t

    rope = ds.Rope(d)
    ds.norm_rope(q, k, off.new_zeros(rows), rope, out=dict(q=room((rows, hq, d), bf), k=room((rows, hkv, d), bf)))
    data = room((pages, hkv, page // 16, 18 * d), torch.uint8)
    data.zero_()
    cache = ds.PagedCache(data, page)
    ds.cache_append(cache, k, v, off, lens, table, rope=rope, q=q, out=dict(q=room((rows, hq, d), bf)))
    ds.cache_read(cache, off, lens, table, rows, out=dict(
        k=room((rows, hkv, d), f8), v=room((rows, hkv, d), f8), k_scale=room((rows, hkv, d // 16), f8),
        v_scale=room((rows, hkv, d // 16), f8)))
    ds.attend_paged(q, cache, off, lens, table, max_rows=max(n), want_lse=True,
                    out=dict(out=room((rows, hq, d), bf), lse=room((rows, hq), torch.float32)))
    one = torch.ones(B, device="cuda")
    for dtype in (bf, torch.float32):
        z = randn(g, rows, V).to(dtype)
        mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, (V + 31) // 32), generator=g, device="cuda", dtype=torch.int32)
        ds.penalize_logits(z, off, i32([[V - 1, 0]] * B), i32([2] * B), i32([1] * B), one, one, one,
                           draft_tok=i32([[V - 1] * max(n)] * B), mask=mask, out=dict(logits=room((rows, V), dtype)))
    torch.cuda.synchronize()
    assert all(c() for c in checks)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_penalize_where_input_and_output_lie_differently(dtype):
    g, dt, n, V = gen(32), DTYPES[dtype], [2, 1], 517
    flat = randn(g, 3 * V + 1).to(dt)
    z = flat[1:].view(3, V)                                 # one element off a 16-byte boundary
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, (V + 31) // 32), generator=g, device="cuda", dtype=torch.int32)
    one = torch.full((2,), 1.5, device="cuda")
    args = (offsets(n), i32([[5, 9, 5], [516, 0, 1]]), i32([3, 2]), i32([1, 0]), one, one, one)
    for m in (None, mask):
        want = ds.penalize_logits(z.clone(), *args, mask=m)["logits"]
        assert torch.equal(ds.penalize_logits(z, *args, mask=m)["logits"], want)
    assert torch.equal(ds.penalize_logits(z, *args, mask=mask, out=dict(logits=z))["logits"], want)
