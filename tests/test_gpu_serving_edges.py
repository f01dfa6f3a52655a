"""The operators around a ragged verification step where they once went wrong: norm weights off their boundary, NaN in
16-bit keys and values."""
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
