"""Attention of whole prompts against a plain 64-bit implementation, at the lengths, masks, layouts and values where
it can go wrong.

Tolerances count roundings: half(t) = torch.finfo(t).eps / 2 of a value stored in t; a tensor-core product adds 16
terms at a time to an fp32 sum, each step off by 2^-22 of its largest term at most.
"""
import math

import pytest
import torch

import speculative_decoding_draft_gb300 as ds

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
STEP = 2.0 ** -22


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


def offsets(n):
    return torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")


def ok(status):
    assert ds.check(status) == "DSPARK_OK"


def plain(q, k, v, n, m, scale, causal, window):
    """out, lse in 64 bits, and the bounds on both."""
    rows, hq, d = q.shape
    hkv = k.shape[1]
    group = hq // hkv
    out, lse = torch.zeros(rows, hq, d).double().cuda(), torch.full((rows, hq), -math.inf).double().cuda()
    out_bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    a = c = 0
    for nr, mr in zip(n, m):
        b, e = a + nr, c + mr
        i, t = torch.arange(nr, device="cuda")[:, None], torch.arange(mr, device="cuda")
        hi = mr - nr + i + 1 if causal else torch.full_like(i, mr)
        hide = t >= hi
        if window:
            hide |= t < hi - window
        for h in range(hq if nr and mr else 0):
            x, y, z = q[a:b, h].double(), k[c:e, h // group].double(), v[c:e, h // group].double()
            # (what no row sees may be no number)
            y, z = (torch.where(hide.all(0)[:, None], 0.0, w) for w in (y, z))
            s = (x @ y.T * scale).masked_fill(hide, -math.inf)
            some = (~hide).any(1)
            lse[a:b, h] = torch.logsumexp(s, 1)
            p = torch.exp(s - torch.where(some, lse[a:b, h], 0)[:, None]).masked_fill(hide, 0.0)
            out[a:b, h] = p @ z
            # scores: D / 16 steps of their absolute terms; exponentials to 2^-21
            off = ((x.abs() @ y.abs().T) * abs(scale) * (d // 16) * STEP).masked_fill(hide, 0.0).amax(1) + 2.0 ** -21
            lse_bound[a:b, h] = off + 2.0 ** -21 * lse[a:b, h].abs().nan_to_num(0, 0, 0)
            size = p @ z.abs()
            out_bound[a:b, h] = (2 * off + half(q.dtype) + mr / 16 * STEP)[:, None] * size + half(q.dtype) * out[a:b, h].abs()
        a, c = b, e
    return out, lse, out_bound + torch.finfo(q.dtype).smallest_normal, lse_bound


def check(q, k, v, n, m, scale=None, causal=True, window=0, **kw):
    got = ds.attend_prompt(q, k, v, offsets(n), kv_off=None if n == m else offsets(m), scale=scale, causal=causal,
                           window=window, want_lse=True, **kw)
    ok(got["status"])
    s = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    out, lse, out_bound, lse_bound = plain(q, k, v, n, m, s, causal, window)
    rows = sum(n)
    far = ((got["out"][:rows].double() - out[:rows]).abs() - out_bound[:rows])
    assert far.max() <= 0, f"out is {far.max().item():.3g} past its bound"
    x, y = got["lse"][:rows].double(), lse[:rows]
    assert torch.equal(torch.isinf(x), torch.isinf(y))
    assert ((x - y).abs().nan_to_num(0) <= lse_bound[:rows]).all()
    return got


LENGTHS = [([1], [1]), ([37], [37]), ([128, 129, 0, 127, 5], None), ([3, 40, 1], [700, 40, 385]),
           ([300, 7, 64], [20, 0, 64]), ([513, 257], None), ([20, 130], [2200, 1700])]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv,group", [(1, 1), (2, 3), (3, 4), (1, 32)])
@pytest.mark.parametrize("lengths", range(len(LENGTHS)))
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 50), (False, 130), (True, 400)])
def test_prompt(dtype, d, hkv, group, lengths, causal, window):
    n, m = LENGTHS[lengths]
    m = m or n
    g, dt = gen(lengths * 100 + d + group), DTYPES[dtype]
    q = randn(g, sum(n), hkv * group, d).to(dt)
    k, v = randn(g, sum(m), hkv, d).to(dt), randn(g, sum(m), hkv, d).to(dt)
    check(q, k, v, n, m, causal=causal, window=window)


def test_strided_heads_of_a_projection():
    g, n = gen(1), [65, 200]
    qkv = randn(g, sum(n), 8 + 2 * 2, 128).bfloat16()
    check(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], n, n)
    by_head = randn(g, 4, sum(n), 64).half().transpose(0, 1)             # rows inside the heads
    check(by_head, by_head[:, :2], by_head[:, 2:], n, n)
    gaps = randn(g, sum(n), 5, 72).half()[:, :, :64]                     # gaps behind heads and rows
    check(gaps[:, :4], gaps[:, :2], gaps[:, 2:4], n, n)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(scale):
    g, n = gen(2), [150]
    q, k, v = (randn(g, 150, 2, 64).bfloat16() for _ in range(3))
    check(q, k, v, n, n, scale=scale)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [64, 128])
def test_maxima_that_rise_step_by_step(dtype, d):
    # scores that grow along the tokens move the running maximum in every step, those that fall in none
    g, dt, m = gen(3), DTYPES[dtype], 1500
    for up in (True, False):
        along = torch.linspace(0.1, 6.0, m, device="cuda")[:, None, None]
        k = (randn(g, 1, 1, d).sign() * (along if up else along.flip(0))).expand(m, 1, d).to(dt).contiguous()
        q = (k[:1].float().sign() * (0.5 + randn(g, 300, 2, d).abs())).to(dt)
        check(q, k, randn(g, m, 1, d).to(dt), [300], [m], scale=0.05)


def test_large_values():
    g, n = gen(4), [140]
    q, k = (randn(g, 140, 2, 64).half() for _ in range(2))
    v = (randn(g, 140, 2, 64) * 15000).clamp(-65000, 65000).half()
    check(q, k, v, n, n)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 60])
def test_infinities_and_nans_in_masked_places(dtype, d, window):
    g, dt, n = gen(5), DTYPES[dtype], [200, 90]
    q = randn(g, 290, 4, d).to(dt)
    k, v = randn(g, 300, 2, d).to(dt), randn(g, 300, 2, d).to(dt)
    k[290:], v[290:] = math.nan, math.inf                                 # behind the last sequence
    clean = ds.attend_prompt(q, k[:290], v[:290], offsets(n), window=window)["out"]
    bad = [(150, math.inf), (171, math.nan), (289, -math.inf)]
    for t, x in bad:
        v[t, 0, 3] = x
    k[120, 1, :] = math.nan
    got = ds.attend_prompt(q, k, v, offsets(n), kv_off=offsets(n), window=window)
    ok(got["status"])
    out = got["out"]
    row = torch.arange(290, device="cuda")

    def sees(t):
        return (row >= t) & (row < (200 if t < 200 else 290)) & ((row < t + window) if window else True)
    same = torch.ones_like(out, dtype=torch.bool)
    for t, _ in bad:
        same[sees(t), :2, 3] = False
    same[sees(120), 2:] = False                                           # a key that is a NaN: the rows that see it
    assert torch.equal(out[same], clean[same])
    for h in range(2):
        want = sum(torch.where(sees(t), x, 0.0) for t, x in bad)
        x = out[:, h, 3].float()
        told = ~torch.isfinite(want)
        assert torch.equal(torch.isnan(x[told]), torch.isnan(want[told]))
        assert torch.equal(x[told & ~torch.isnan(want)], want[told & ~torch.isnan(want)].float())
    assert torch.isnan(out[sees(120), 2:]).all()


@pytest.mark.parametrize("n,m", [([3], [20000]), ([1, 2], [9000, 12001]), ([17], [6000])])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 5000)])
def test_few_rows_over_many_tokens(n, m, causal, window):
    g = gen(6)
    q, k, v = randn(g, sum(n), 8, 128).bfloat16(), randn(g, sum(m), 2, 128).bfloat16(), randn(g, sum(m), 2, 128).bfloat16()
    got = check(q, k, v, n, m, causal=causal, window=window)
    assert got["workspace"] is not None                                   # the tokens are shared out
    again = ds.attend_prompt(q, k, v, offsets(n), kv_off=offsets(m), causal=causal, window=window, want_lse=True,
                             workspace=got["workspace"].fill_(255))
    assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])


def test_a_long_prompt():
    g, n = gen(7), [6000]
    q, k, v = randn(g, 6000, 4, 128).bfloat16(), randn(g, 6000, 1, 128).bfloat16(), randn(g, 6000, 1, 128).bfloat16()
    got = check(q, k, v, n, n)
    for _ in range(20):                                                   # the same bits every time
        assert torch.equal(got["out"], ds.attend_prompt(q, k, v, offsets(n))["out"])


def test_rows_behind_the_last_and_requests_without_any():
    g = gen(8)
    q, k, v = (randn(g, 100, 2, 64).bfloat16() for _ in range(3))
    out, lse = torch.full_like(q, 7.0), torch.full((100, 2), 7.0, device="cuda")
    off = offsets([0, 30, 0, 40, 0])
    got = ds.attend_prompt(q, k, v, off, kv_off=off, want_lse=True, out=dict(out=out, lse=lse))
    ok(got["status"])
    assert (out[70:] == 7).all() and (lse[70:] == 7).all()
    want = ds.attend_prompt(q[:70], k[:70], v[:70], off)["out"]
    assert torch.equal(out[:70], want)
    none = torch.zeros(0, 2, 64, device="cuda").bfloat16()
    got = ds.attend_prompt(q, none, none, offsets([100]), kv_off=offsets([0]), want_lse=True)
    ok(got["status"])
    assert (got["out"] == 0).all() and (got["lse"] == -math.inf).all()
    assert ds.attend_prompt(none, none, none, offsets([0]))["out"].shape == (0, 2, 64)


def test_offsets_that_fall_or_pass_the_rows():
    g = gen(9)
    q, k, v = (randn(g, 20, 2, 64).bfloat16() for _ in range(3))
    for off in ([0, 21], [5, 2], [-1, 20]):
        bad = torch.tensor(off, dtype=torch.int32, device="cuda")
        assert ds.check(ds.attend_prompt(q, k, v, bad)["status"]) == "DSPARK_ERR_OFFSETS"
        assert ds.check(ds.attend_prompt(q, k, v, offsets([20]), kv_off=bad)["status"]) == "DSPARK_ERR_OFFSETS"
    status = ds.new_status("cuda")
    status.fill_(9)
    out = torch.full_like(q, 7.0)
    ds.attend_prompt(q, k, v, offsets([20]), status=status, out=dict(out=out))
    assert (out == 7).all()                                               # a step that had failed


def test_refusals():
    q = torch.zeros(4, 4, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    off = offsets([4])

    def refused(kind, *args, **kw):
        with pytest.raises(kind):
            ds.attend_prompt(*args, **kw)
    refused(TypeError, q.float(), k.float(), k.float(), off)
    refused(TypeError, q, k.half(), k, off)
    refused(TypeError, q.cpu(), k, k, off)
    refused(TypeError, q, k, k, off.long())
    refused(ValueError, q[:, :3], k, k, off)
    refused(ValueError, q, k, k[:3], off)
    refused(ValueError, q, k[:3], k[:3], off)                             # fewer keys need kv_off
    refused(ValueError, q, k, k, off, kv_off=offsets([2, 2]))
    refused(ValueError, q, k, k, off, window=-1)
    refused(ValueError, q[..., :32], k[..., :32], k[..., :32], off)
    refused(ValueError, q, k[:1].expand(4, 2, 64), k, off)
    refused(ValueError, q, k[:, :1].expand(4, 2, 64), k, off)
    odd = torch.zeros(2 * 328, device="cuda", dtype=torch.bfloat16).as_strided((4, 2, 64), (72, 328, 1))
    refused(ValueError, q, odd, k, off)                                   # rows inside heads, 328 no multiple of 72
    refused(ds.DsparkError, q, k, k, off, scale=math.nan)
    refused(TypeError, q, k, k, off, out=[q])


def test_another_stream_and_a_graph():
    g, n = gen(10), [70, 260]
    q, k, v = randn(g, 330, 4, 128).bfloat16(), randn(g, 330, 2, 128).bfloat16(), randn(g, 330, 2, 128).bfloat16()
    off = offsets(n)
    want = ds.attend_prompt(q, k, v, off, want_lse=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = ds.attend_prompt(q, k, v, off, want_lse=True, stream=s)
    s.synchronize()
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = ds.attend_prompt(q, k, v, off, want_lse=True)
    q.copy_(randn(g, 330, 4, 128))
    graph.replay()
    assert torch.equal(held["out"], ds.attend_prompt(q, k, v, off)["out"])


def test_infinities_where_the_tokens_are_shared_out():
    # few rows over many tokens: a value that only the last row sees, in the last part
    g, m = gen(11), 9000
    q = randn(g, 3, 4, 128).bfloat16()
    k, v = randn(g, m, 1, 128).bfloat16(), randn(g, m, 1, 128).bfloat16()
    clean = ds.attend_prompt(q, k, v, offsets([3]), kv_off=offsets([m]))
    assert clean["workspace"] is not None
    v[m - 1, 0, 7], v[m - 2, 0, 9] = math.inf, math.nan
    got = ds.attend_prompt(q, k, v, offsets([3]), kv_off=offsets([m]))
    ok(got["status"])
    same = torch.ones_like(q, dtype=torch.bool)
    same[2, :, 7] = same[1:, :, 9] = False
    assert torch.equal(got["out"][same], clean["out"][same])
    assert (got["out"][2, :, 7] == math.inf).all() and torch.isnan(got["out"][1:, :, 9]).all()


def test_the_output_may_be_the_queries():
    g, n = gen(12), [300, 20]
    q, k, v = randn(g, 320, 4, 64).half(), randn(g, 320, 2, 64).half(), randn(g, 320, 2, 64).half()
    want = ds.attend_prompt(q, k, v, offsets(n))["out"]
    got = ds.attend_prompt(q, k, v, offsets(n), out=dict(out=q))
    ok(got["status"])
    assert got["out"].data_ptr() == q.data_ptr() and torch.equal(q, want)
