"""The paged cache in 8 bits: append and read-back against a model of the cache in exact arithmetic, call after call.

Values that are kept as they come (no norm, no rotation) have to be held exactly as the model says.  Normed and turned
keys are fp32 values y whose nearest element the kernel keeps: off y by half a step of e4m3 and what fp32 is off.
"""
import math

import pytest
import torch

import speculative_decoding_draft_gb300 as ds
from test_gpu_serving import DTYPES, gen, i32, offsets, ok, paged, randn, rotate64, rotate_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_draft_gb300 import build
    build.build()


def e4m3(x):
    """The nearest e4m3 of float64 x, ties to even, at most 448; a NaN stays."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6, max=8) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exponent(top):
    """The smallest e in -32 .. 31 with top <= 448 * 2^e."""
    m, e = torch.frexp(top.double())                           # top = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    return torch.where(top > 0, (e - 9 + (m > 0.875).int()).double(), -32.0).clamp(-32, 31)


class Model:
    """One request's keys or values [tokens, heads, D], block by block."""

    def __init__(self, heads, d):
        self.x, self.e = torch.zeros(0, heads, d).double().cuda(), torch.zeros(0, heads).double().cuda()

    def append(self, new, end):
        first = end - len(new)
        self.x = torch.cat((self.x[:first], torch.zeros_like(new.double())))
        at = 0
        while at < len(new):
            block, t0 = (first + at) // 16, (first + at) % 16
            m = min(16 - t0, len(new) - at)
            y = new[at: at + m].double()
            fine = torch.where(torch.isfinite(y), y, 0.0)
            e = exponent(fine.abs().amax((0, 2)))
            self.e = self.e[: block + 1]
            if t0:
                e = torch.maximum(e, self.e[block])
                old = slice(16 * block, 16 * block + t0)
                u = torch.exp2(e)[:, None]
                self.x[old] = e4m3(self.x[old] / u) * u
                self.e[block] = e
            else:
                self.e = torch.cat((self.e[:block], e[None]))
            u = torch.exp2(e)[:, None]
            self.x[first + at: first + at + m] = e4m3((y / u).nan_to_num(math.nan, 1e9, -1e9)) * u
            at += m


def equal(x, y):
    return bool((((x == y) | (torch.isnan(x) & torch.isnan(y))).all()))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,page", [(1, 16), (3, 48), (8, 64), (2, 256)])
def test_calls_one_after_another(dtype, d, heads, page):
    g, dt, B = gen(d + heads), DTYPES[dtype], 4
    most = 100
    table, pages = paged(g, [most] * B, page, spare=2)
    cache = ds.PagedCache8.empty(pages, heads, d, page)
    cache.data.fill_(0x7f)                                     # what was there before: NaN elements, any scale
    cache.scales.random_(0, 256, generator=g)
    models = [[Model(heads, d) for _ in range(2)] for _ in range(B)]
    length = [0] * B
    # prompts, steps of a few rows of which some are rejected, single tokens
    for call, rows in enumerate([[17, 1, 40, 0], [5, 3, 1, 33], [1, 1, 1, 1], [8, 2, 16, 7], [0, 31, 3, 8], [1, 1, 0, 1]]):
        n = sum(rows)
        new = randn(g, n, 2 * heads + 1, d) * torch.exp(2 * randn(g, n, 2 * heads + 1, 1))   # some tokens louder
        new = new.clamp(-60000, 60000).to(dt)
        k, v = new[:, :heads], new[:, heads: 2 * heads]
        back = [min(2, length[r]) if call % 2 else 0 for r in range(B)]       # rejected tokens are written over
        kv = [length[r] - back[r] + rows[r] for r in range(B)]
        got = ds.cache_append(cache, k, v, offsets(rows), i32(kv), table)
        ok(got["status"])
        at = 0
        for r in range(B):
            for m, x in zip(models[r], (k, v)):
                if rows[r]:
                    m.append(x[at: at + rows[r]], kv[r])
            at += rows[r]
            length[r] = kv[r] if rows[r] else length[r]
        read = ds.cache_read(cache, offsets(length), i32(length), table, sum(length), dtype=torch.float32)
        ok(read["status"])
        at = 0
        for r in range(B):
            for m, x in zip(models[r], (read["k"], read["v"])):
                assert equal(x[at: at + length[r]].double(), m.x[: length[r]]), (call, r)
            at += length[r]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d,rot,layout", [(64, 64, "half"), (64, 32, "interleaved"), (128, 128, "interleaved"), (128, 64, "half")])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("given", [True, False])
def test_norm_and_rotation_on_the_way(dtype, d, rot, layout, norm, given):
    g, dt, hq, hkv, rows, kv = gen(d + rot), DTYPES[dtype], 6, 3, [9, 1, 40], [9, 33, 71]
    rope = ds.Rope(rot, base=5e5, layout=layout, scaling="yarn", factor=4.0, original_len=64)
    n = sum(rows)
    qkv = randn(g, n, hq + 2 * hkv, d).to(dt)
    q, k, v = qkv[:, :hq], qkv[:, hq: hq + hkv], qkv[:, hq + hkv:]
    w = [(1 + 0.2 * randn(g, d)).to(dt) if norm else None for _ in range(2)]
    table, pages = paged(g, kv, 32)
    cache = ds.PagedCache8.empty(pages, hkv, d, 32)
    first = torch.cat([torch.arange(e - m, e) for m, e in zip(rows, kv)]).int().cuda()
    pos = first * 3 + 1000 if given else None
    got = ds.cache_append(cache, k, v, offsets(rows), i32(kv), table, positions=pos, rope=rope, k_weight=w[1], q=q,
                          q_weight=w[0], eps=1e-5)
    ok(got["status"])
    at = first if pos is None else pos
    ref = rotate64(q, w[0], 1e-5, at, rope)
    assert ((got["q"].double() - ref).abs() <= rotate_bound(ref, dt, rope.gain)).all()
    read = ds.cache_read(cache, offsets(rows), i32(kv), table, n, dtype=torch.float32)
    ok(read["status"])
    y = rotate64(k, w[1], 1e-5, at, rope)
    fp32 = rotate_bound(y, torch.float32, rope.gain)
    # a block of the call lies within 16 rows; its scale is at most twice what its loudest row needs
    top = torch.stack([torch.nn.functional.pad(y.abs().amax(-1), (0, 0, 16, 16))[i: i + 33].amax(0) for i in range(n)])
    floor = torch.exp2(exponent(top * (1 + 1e-5)))[..., None] * 2.0 ** -10
    assert ((read["k"].double() - y).abs() <= 2.0 ** -4 * y.abs() + floor + 2 * fp32).all()


def test_infinities_nans_zeros_and_the_ends_of_the_range():
    d, table = 64, i32([[0, 1, 2]])
    cache = ds.PagedCache8.empty(3, 1, d, 16)
    x = torch.zeros(40, 1, d, device="cuda")
    x[3, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 3.0])
    x[5, 0, 7] = 100.0
    x[16:32] = 1e-30                                            # below the smallest scale: it becomes 0
    x[20, 0, 0] = 2.0 ** -41
    x[33, 0, :3] = torch.tensor([3e38, -3e38, 1.0])             # past the largest: cut to it
    got = ds.cache_append(cache, x, -x, offsets([40]), i32([40]), table)
    ok(got["status"])
    read = ds.cache_read(cache, offsets([40]), i32([40]), table, 40, dtype=torch.float32)
    for m, y in ((read["k"], x), (read["v"], -x)):
        model = Model(1, d)
        model.append(y, 40)
        assert equal(m.double(), model.x)
    k = read["k"][:, 0]
    assert k[3, 0] == 448 * 0.25 and k[3, 1] == -448 * 0.25 and torch.isnan(k[3, 2]) and k[3, 3] == 3.0
    assert k[5, 7] == 96.0 or k[5, 7] == 104.0                  # 100 lies between two elements
    assert k[16].abs().max() == 0 and k[20, 0] == 2.0 ** -41
    assert k[33, 0] == 448 * 2.0 ** 31 and k[33, 1] == -448 * 2.0 ** 31 and k[33, 2] == 0


def test_read_types():
    g, d, table = gen(5), 128, i32([[1, 0]])
    cache = ds.PagedCache8.empty(2, 2, d, 32)
    x = (randn(g, 50, 2, d) * torch.exp(8 * randn(g, 50, 1, 1)))
    ok(ds.cache_append(cache, x, x.flip(0), offsets([50]), i32([50]), table)["status"])
    args = (cache, offsets([50]), i32([50]), table, 50)
    exact = ds.cache_read(*args, dtype=torch.float32)
    assert ds.cache_read(*args)["k"].dtype == torch.bfloat16
    for dt in (torch.bfloat16, torch.float16):
        got = ds.cache_read(*args, dtype=dt)
        for h in "kv":
            assert torch.equal(got[h], exact[h].to(dt)) and (dt == torch.float16 or torch.equal(got[h].float(), exact[h]))
    out = dict(k=torch.empty(50, 2, d, device="cuda"), v=torch.empty(50, 2, d, device="cuda"))
    got = ds.cache_read(*args, dtype=torch.float32, out=out)
    assert got["k"].data_ptr() == out["k"].data_ptr() and torch.equal(out["v"], exact["v"])


def test_rows_behind_the_last_and_a_failed_step():
    g, d = gen(6), 64
    table = i32([[0], [1]])
    cache = ds.PagedCache8.empty(2, 1, d, 16)
    x, q = randn(g, 9, 1, d).bfloat16(), randn(g, 9, 2, d).bfloat16()
    out = torch.full((9, 2, d), 7.0, device="cuda").bfloat16()
    got = ds.cache_append(cache, x, x, offsets([3, 2]), i32([3, 2]), table, q=q, out=dict(q=out))
    ok(got["status"])
    assert torch.equal(out[:5], q[:5]) and (out[5:] == 7).all()
    held = cache.data.clone()
    assert (held[0, 0, :, 3:] == 0).all() and (held[1, 0, :, 2:] == 0).all()      # places that no row names
    status = ds.new_status("cuda")
    status.fill_(9)
    ds.cache_append(cache, -x, -x, offsets([3, 2]), i32([3, 2]), table, q=q, out=dict(q=out.fill_(5)), status=status)
    read = dict(k=torch.full_like(x, 3.0), v=torch.full_like(x, 3.0))
    ds.cache_read(cache, offsets([3, 2]), i32([3, 2]), table, 9, out=read, status=status)
    assert (out == 5).all() and torch.equal(cache.data, held) and (read["k"] == 3).all()
    got = ds.cache_read(cache, offsets([3, 2]), i32([3, 2]), table, 9, out=read)
    ok(got["status"])
    assert (read["k"][5:] == 3).all() and (read["v"][5:] == 3).all()


@pytest.mark.parametrize("bad,name", [(dict(off=[0, 9, 4]), "OFFSETS"), (dict(off=[0, 2, 99]), "OFFSETS"),
                                      (dict(kv=[1, 2]), "LENGTHS"), (dict(kv=[4, 33]), "LENGTHS"),
                                      (dict(table=[[0, 1], [2, 0]]), "PAGES"), (dict(table=[[-1, 1], [0, 0]]), "PAGES")])
def test_inconsistent_arguments(bad, name):
    d = 64
    cache = ds.PagedCache8.empty(2, 1, d, 16)
    x = torch.ones(4, 1, d, device="cuda")
    off, kv, table = (i32(bad.get(k, v)) for k, v in (("off", [0, 2, 4]), ("kv", [4, 20]), ("table", [[0, 1], [1, 0]])))
    if name == "PAGES":
        kv = i32([4, 4])
    got = ds.cache_append(cache, x, x, off, kv, table)
    assert ds.check(got["status"]) == "DSPARK_ERR_" + name
    if name != "OFFSETS":
        assert ds.check(ds.cache_read(cache, off, kv, table, 4)["status"]) == "DSPARK_ERR_" + name


def test_many_requests_of_one_row_and_none():
    g, B, d = gen(7), 700, 64
    rows = [i % 3 % 2 for i in range(B)]
    kv = [1 + (7 * i) % 40 for i in range(B)]
    table, pages = paged(g, kv, 16)
    cache = ds.PagedCache8.empty(pages, 1, d, 16)
    x = randn(g, sum(rows), 1, d).half()
    ok(ds.cache_append(cache, x, -x, offsets(rows), i32(kv), table)["status"])
    got = ds.cache_read(cache, offsets(rows), i32(kv), table, len(x), dtype=torch.float32)
    ok(got["status"])
    u = torch.exp2(exponent(x.float().abs().amax(-1)))[..., None]
    want = e4m3(x.double() / u) * u
    # (a block that goes on has the fresh cache's smallest scale: the row's own counts)
    assert torch.equal(got["k"].double(), want) and torch.equal(got["v"].double(), -want)


def test_another_stream_and_a_graph():
    g, d = gen(8), 128
    table = i32([[0, 1, 2, 3]])
    a, b = (ds.PagedCache8.empty(4, 2, d, 16) for _ in range(2))
    k, v = randn(g, 50, 2, d).bfloat16(), randn(g, 50, 2, d).bfloat16()
    off, kv = offsets([50]), i32([50])
    ds.cache_append(a, k, v, off, kv, table)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ds.cache_append(b, k, v, off, kv, table, stream=s)
    got = ds.cache_read(b, off, kv, table, 50, stream=s)
    s.synchronize()
    assert torch.equal(a.data, b.data) and torch.equal(a.scales, b.scales)
    want = ds.cache_read(a, off, kv, table, 50)
    assert torch.equal(got["k"], want["k"]) and torch.equal(got["v"], want["v"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ds.cache_append(b, k, v, off, kv, table)
        held = ds.cache_read(b, off, kv, table, 50)
    k.mul_(-1)
    graph.replay()
    ds.cache_append(a, k, v, off, kv, table)
    assert torch.equal(held["k"], ds.cache_read(a, off, kv, table, 50)["k"])
