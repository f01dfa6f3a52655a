"""Cases, inputs, plain forms and 64-bit definitions of the operators of prompts and of the cache in 8 bits.

A target model reads a prompt before drafted tokens are verified against it, and keeps what it read.  Per attention
layer, over ragged rows (request r owns rows row_off[r] .. row_off[r+1]-1):

  prompt   attention of whole prompts over their own keys and values (and those of earlier pieces of the same prompt),
           grouped heads, sequences of different lengths packed one after the other;
  append   norm and rotation of queries and keys and the append of keys and values to a paged cache in 8 bits, one
           scale for 16 tokens of a head, then the read-back of what the touched blocks hold;
  attend   attention of few rows a request over that cache.

The cache: data [pages, heads, 2 (keys, values), page tokens, D] e4m3 elements and scales [pages, heads, 2, page / 16],
exponents e + 127 of powers of two 2^e, e in -32 .. 31, one for a block of 16 tokens.  The D elements of token t lie in
pieces of 16, piece c at c ^ (t % 8) where D is 128 and at c ^ (t / 2 % 4) where D is 64.  A block's exponent is the
smallest with 448 * 2^e above every finite magnitude that has been written to it since a call began it at its first
token; elements that are there already are rounded again when it rises.

`run` returns whole outputs; what the cache holds comes back as the values that it stands for."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E_LOW, E_HIGH = -32, 31
MOST_PAIRS = 32 * 16384 * 16384           # scores of one pass


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # a short question of a single user: latency counts
        dict(name="prompt short", op="prompt", dtype="bf16", B=1, most=37, ctx=0, hq=32, hkv=8, d=128, causal=True,
             window=0),
        # sixteen prompts of 128 to 1021 tokens in one pass
        dict(name="prompt batch", op="prompt", dtype="bf16", B=16, most=1021, ctx=0, hq=32, hkv=8, d=128, causal=True,
             window=0),
        # a long document
        dict(name="prompt long", op="prompt", dtype="bf16", B=1, most=16384, ctx=0, hq=32, hkv=8, d=128, causal=True,
             window=0),
        # pieces of three long prompts over what was read before, small heads, a window
        dict(name="prompt pieces window", op="prompt", dtype="fp16", B=3, most=4001, ctx=5000, hq=12, hkv=4, d=64,
             causal=True, window=2048),
        # a block-parallel draft: every row sees the context and the whole block
        dict(name="prompt blocks", op="prompt", dtype="bf16", B=64, most=16, ctx=2000, hq=32, hkv=8, d=128,
             causal=False, window=0),
        # a single user's next token
        dict(name="append one token", op="append", dtype="bf16", B=1, most=1, kv=777, hq=32, hkv=8, d=128, page=16,
             rot=128, layout="half", norm=True),
        # the ragged step: 2048 requests with 1 to 8 rows each
        dict(name="append ragged", op="append", dtype="bf16", B=2048, most=8, kv=2048, hq=32, hkv=8, d=128, page=64,
             rot=128, layout="half", norm=True),
        # a piece of a few prompts, small heads
        dict(name="append piece", op="append", dtype="fp16", B=3, most=2731, kv=9000, hq=12, hkv=4, d=64, page=32,
             rot=32, layout="interleaved", norm=False),
        # a single user, plain decoding
        dict(name="attend one token", op="attend", dtype="bf16", B=1, most=1, kv=1021, hq=32, hkv=8, d=128, page=16,
             causal=True, window=0),
        # a single user with a long document, 8 rows verified
        dict(name="attend long", op="attend", dtype="bf16", B=1, most=8, kv=131071, hq=32, hkv=8, d=128, page=64,
             causal=True, window=0),
        # the 64-request step at contexts of 512 to 4096
        dict(name="attend step", op="attend", dtype="bf16", B=64, most=8, kv=4096, hq=32, hkv=8, d=128, page=64,
             causal=True, window=0),
        # many users, most of them on one row, small heads
        dict(name="attend many", op="attend", dtype="fp16", B=256, most=2, kv=16384, hq=32, hkv=8, d=64, page=32,
             causal=True, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prompt", "append", "attend"))
    d = rng.choice((64, 128))
    hkv, group = rng.choice((1, 2, 3, 4, 8)), rng.choice((1, 2, 3, 4, 6, 8))
    c = dict(op=op, dtype=rng.choice(("bf16", "fp16")), hq=hkv * group, hkv=hkv, d=d)
    if op == "prompt":
        B, most, ctx = _log(rng, 1, 64), _log(rng, 1, 16384), rng.choice((0, 0, _log(rng, 1, 8192)))
        while B * most * (most + ctx) * hkv * group > MOST_PAIRS or B * (2 * most + ctx) > 65536:
            B, most = max(1, B // 2), max(1, most // 2) if B == 1 else most
        return dict(c, B=B, most=most, ctx=ctx, causal=rng.random() < 0.75,
                    window=rng.choice((0, 0, 0, 333, 4096)))
    if op == "attend":
        B, kv, most = _log(rng, 1, 256), _log(rng, 1, 131071), rng.choice((1, 1, 2, 5, 8, rng.randint(9, 40)))
        while B * kv * hkv * d > 256 * 16384 * 8 * 64 or B * kv * hkv * group * most > 256 * 16384 * 32 * 2:
            B, kv = max(1, B // 2), max(1, kv // 2) if B == 1 else kv
        return dict(c, B=B, most=most, kv=kv, page=rng.choice((16, 32, 64, 128, 256)), causal=rng.random() < 0.75,
                    window=rng.choice((0, 0, 0, 333, 4096)))
    B, most = _log(rng, 1, 2048), _log(rng, 1, 3000)
    while B * most > 16384:
        B, most = max(1, B // 2), max(1, most // 2) if B == 1 else most
    return dict(c, dtype=rng.choice(("bf16", "fp16", "fp32")), B=B, most=most, kv=most + _log(rng, 1, 2048),
                page=rng.choice((16, 32, 64, 128, 256)), rot=rng.choice((d, d, d // 2)),
                layout=rng.choice(("half", "interleaved")), norm=rng.random() < 0.6)


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + salt)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _least(case):
    return max(1, case["most"] // 8) if case["B"] < 8 or case["op"] == "prompt" else 1


def _counts(case):
    """Every request's rows: spread evenly over least .. most."""
    i = torch.arange(case["B"], dtype=torch.int64)
    least, most = _least(case), case["most"]
    if case["op"] == "prompt":
        return most - (most - least) * i // max(1, case["B"] - 1)
    return most - i % (most - least + 1)


def _begun(case):
    """How many tokens every request has in the block that it goes on with."""
    return [(5 * i + 8) % 16 if case["kv"] > case["most"] else 0 for i in range(case["B"])]


def _offsets(n):
    off = torch.zeros(len(n) + 1, dtype=torch.int32, device="cuda")
    off[1:] = n.cumsum(0)
    return off


def _pages(case, kv_len, g):
    """A page table over shuffled pages, -1 past a request's last page, and the number of pages."""
    need = (kv_len + case["page"] - 1) // case["page"]
    width, total = max(1, int(need.max())), int(need.sum())
    table = torch.full((case["B"], width), -1, dtype=torch.int32, device="cuda")
    ids = torch.randperm(max(1, total), generator=g, device="cuda").to(torch.int32)
    table[torch.arange(width, device="cuda")[None] < need[:, None]] = ids[:total]
    return table, max(1, total)


def _fill(s, case, pages, g):
    """A cache that holds keys and values of earlier tokens, some tokens louder than others."""
    hkv, page, d = case["hkv"], case["page"], case["d"]
    s["data"] = torch.empty(pages, hkv, 2, page, d, dtype=torch.uint8, device="cuda")
    s["scales"] = torch.empty(pages, hkv, 2, page // 16, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (hkv * page * d))
    for at in range(0, pages, step):
        m = min(step, pages - at)
        x = torch.randn(m, hkv, 2, page, d, generator=g, device="cuda")
        x *= torch.exp(0.4 * torch.randn(m, hkv, 2, page, 1, generator=g, device="cuda"))
        top = x.unflatten(3, (-1, 16)).abs().amax((-2, -1))
        e = _exponent(top)
        x = torch.ldexp(x, -e.repeat_interleave(16, -1)[..., None])
        s["data"][at: at + m] = _swizzle(x.to(torch.float8_e4m3fn).view(torch.uint8), torch.arange(page, device="cuda"))
        s["scales"][at: at + m] = (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = _gen(seed, 1)
    op, s = case["op"], dict(case=case)
    dt = DTYPES[case["dtype"]]
    hq, hkv, d, B = case["hq"], case["hkv"], case["d"], case["B"]
    n = _counts(case).cuda()[torch.randperm(B, generator=g, device="cuda")]
    off = _offsets(n)
    rows = int(off[-1])
    s.update(rows=rows, row_off=off, n=n.int())
    if op == "prompt":
        # earlier tokens: from none up to ctx
        ctx = (torch.rand(B, generator=g, device="cuda") * (case["ctx"] + 1)).to(torch.int64)
        ctx[-1] = case["ctx"]
        s["ctx"] = ctx.int()
        s["kv_off"] = _offsets(n + ctx) if case["ctx"] else off
        if case["ctx"]:
            s["q"] = _normal(g, (rows, hq, d), dt)
            kv = _normal(g, (int(s["kv_off"][-1]), 2 * hkv, d), dt)
            s["k"], s["v"] = kv[:, :hkv], kv[:, hkv:]
        else:   # as one projection leaves them
            qkv = _normal(g, (rows, hq + 2 * hkv, d), dt)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq: hq + hkv], qkv[:, hq + hkv:]
    else:
        if op == "append":           # texts that end at every place of a block
            kv_len = (torch.rand(B, generator=g, device="cuda") * ((case["kv"] - case["most"]) // 16 + 1)).to(torch.int32)
            kv_len = 16 * kv_len + torch.tensor(_begun(case), dtype=torch.int32, device="cuda") + n.int()
        else:
            kv_len = (torch.rand(B, generator=g, device="cuda") * 0.875 + 0.125) * case["kv"]
            kv_len = kv_len.to(torch.int32)
            kv_len[-1] = case["kv"]
            if B > 2:
                kv_len[0] = 0        # a request whose cache is still empty
        s["kv_len"] = kv_len
        s["table"], pages = _pages(case, kv_len, g)
        _fill(s, case, pages, g)
        qkv = _normal(g, (rows, hq + 2 * hkv, d), dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq: hq + hkv], qkv[:, hq + hkv:]
        if op == "attend":
            s["q"], s["k"], s["v"] = s["q"].contiguous(), None, None
        else:
            s["v"] *= torch.exp(0.4 * torch.randn(rows, hkv, 1, generator=g, device="cuda")).to(dt)
            s["inv_freq"] = 1e6 ** (-2 * torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda") / case["rot"])
            s["q_weight"] = s["k_weight"] = None
            if case["norm"]:
                s["q_weight"], s["k_weight"] = ((1 + _normal(g, (d,), torch.float32, 0.1)).to(dt) for _ in range(2))
            # what is read back: the touched blocks up to the requests' ends
            s["read_off"] = _offsets(n + (kv_len - n) % 16)
            s["read_rows"] = int(s["read_off"][-1])
    if own:
        import speculative_decoding_draft_gb300 as ds
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if op != "prompt":
            s["cache"] = ds.PagedCache8(s["data"], s["scales"])
        if op == "append":
            s["rope"] = ds.Rope(case["rot"], base=1e6, layout=case["layout"], device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------
def _exponent(top):
    """The smallest e in range with top <= 448 * 2^e."""
    m, e = torch.frexp(top)                    # top = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    e = torch.where(top > 0, e - 9 + (m > 0.875).int(), E_LOW)
    return e.clamp(E_LOW, E_HIGH).int()


def _swizzle(x, t):
    """Elements [..., tokens, D] to and from their places, t: a token's place in its page."""
    d = x.shape[-1]
    c = torch.arange(d // 16, device="cuda")
    at = c ^ (t[:, None] % 8 if d == 128 else t[:, None] // 2 % 4)
    y = x.unflatten(-1, (-1, 16))
    return torch.gather(y, -2, at[..., None].expand(y.shape)).flatten(-2)


def _element(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _norm_rope(x, weight, positions, inv_freq, case):
    """x [rows, heads, D] in 32 bits: root-mean-square norm of each head where there is a weight, then the rotation of
    its first `rot` dimensions; angles in 64 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = positions.double()[:, None] * inv_freq
    c, s = (f(angle).float()[:, None] for f in (torch.cos, torch.sin))
    rot = case["rot"]
    y = x.clone()
    if case["layout"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def _places(s, off, rows):
    """Of ragged rows at the ends of the requests' texts: the request, the position, the page and the place in it."""
    i = torch.arange(rows, device="cuda", dtype=torch.int32)
    req = torch.searchsorted(off[1:], i, right=True)
    pos = (s["kv_len"] - (off[1:] - off[:-1]))[req] + i - off[req]
    page = s["case"]["page"]
    return req, pos, s["table"][req, (pos // page).long()].long(), (pos % page).long()


def _run_append(s):
    case, data, scales = s["case"], s["data"], s["scales"]
    per = case["page"] // 16
    req, pos, page, t = _places(s, s["row_off"], s["rows"])
    rope = (pos, s["inv_freq"], case)
    q = _norm_rope(s["q"], s["q_weight"], *rope).to(s["q"].dtype)
    new = torch.stack((_norm_rope(s["k"], s["k_weight"], *rope), s["v"].float()), 2)      # [rows, heads, 2, D]
    # the exponents of the touched blocks
    need = _exponent(torch.nan_to_num(new, 0, 0, 0).abs().amax(-1))
    block = page * per + t // 16
    top = torch.full((scales.shape[0] * per, case["hkv"], 2), E_LOW, dtype=torch.int32, device="cuda")
    top.scatter_reduce_(0, block[:, None, None].expand_as(need), need, "amax")
    held = scales.permute(0, 3, 1, 2).flatten(0, 1).int() - 127                            # [blocks, heads, 2]
    first = (s["kv_len"] - s["n"]).long()                                                  # where each request goes on
    old = s["table"].gather(1, first[:, None] // case["page"])[:, 0].long()
    inside = first % 16
    went_on = old * per + first % case["page"] // 16
    went_on, inside = went_on[inside > 0], inside[inside > 0]
    top[went_on] = torch.maximum(top[went_on], held[went_on].clamp(E_LOW, E_HIGH))
    # what the blocks that go on hold already, rounded again where their exponent has risen
    tok = torch.arange(16, device="cuda")
    at = (went_on // per)[:, None], (went_on % per * 16)[:, None] + tok
    keep = tok < inside[:, None]
    at = at[0].expand_as(keep)[keep], at[1][keep]
    was = data[at[0], :, :, at[1]].view(torch.float8_e4m3fn).float()
    by = (held[went_on].clamp(E_LOW, E_HIGH) - top[went_on])[:, None].expand(-1, 16, -1, -1)[keep]
    data[at[0], :, :, at[1]] = _element(torch.ldexp(was, by[..., None])).view(torch.uint8)
    # the new rows
    e = top[block]
    x = _element(torch.ldexp(new, -e[..., None])).view(torch.uint8)
    data[page, :, :, t] = _swizzle(x.permute(1, 2, 0, 3), t).permute(2, 0, 1, 3)
    scales[page, :, :, t // 16] = (e + 127).to(torch.uint8)
    # what is held now
    req, pos, page, t = _places(s, s["read_off"], s["read_rows"])
    x = _swizzle(data[page, :, :, t].permute(1, 2, 0, 3), t).view(torch.float8_e4m3fn).float()
    e = scales[page, :, :, t // 16].int() - 127
    x = torch.ldexp(x.permute(2, 0, 1, 3), e[..., None]).to(torch.bfloat16)
    return dict(q=q, k=x[:, :, 0], v=x[:, :, 1])


def _softmax_v(q, k, v, seen, scale):
    """Attention of q [b, heads, x, D] over k, v [b, heads, t, D] where seen [b, 1, x, t]: out and log-sum-exp."""
    p = (q @ k.transpose(-1, -2)).mul_(scale)
    p.masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = p.sub_(base).exp_()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, torch.ones_like(total), total), (base + torch.log(total)).squeeze(-1)


def _seen(case, n, kv, most, L):
    """[B, most, L]: which of its request's tokens a row sees."""
    end = kv[:, None].expand(-1, most)
    if case["causal"]:
        end = (kv - n)[:, None] + torch.arange(most, device="cuda") + 1
    token = torch.arange(L, device="cuda")
    seen = (token < end[..., None]) & (token < kv[:, None, None])
    if case["window"]:
        seen &= token >= end[..., None] - case["window"]
    return seen


def _run_rows(s, k, v, kv, L):
    """Attention of the ragged rows over padded keys and values [B, heads, L, D] in 32 bits."""
    case = s["case"]
    d, hq, hkv, B, most = case["d"], case["hq"], case["hkv"], case["B"], case["most"]
    group = hq // hkv
    i = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    req = torch.searchsorted(s["row_off"][1:], i, right=True)
    j = (i - s["row_off"][req]).long()
    q = torch.zeros(B, most, hq, d, device="cuda")
    q[req, j] = s["q"].float()
    q = q.view(B, most, hkv, group, d).transpose(1, 2).reshape(B, hkv, most * group, d)
    seen = _seen(case, s["n"], kv, most, L)[:, None, :, None].expand(B, 1, most, group, L).reshape(B, 1, most * group, L)
    out, lse = _softmax_v(q, k, v, seen, 1 / math.sqrt(d))
    shape = lambda x: x.view(B, hkv, most, group, -1).transpose(1, 2).reshape(B, most, hq, -1)[req, j]  # noqa: E731
    return dict(out=shape(out).to(s["q"].dtype), lse=shape(lse).squeeze(-1))


def _run_prompt(s):
    case = s["case"]
    kv = s["kv_off"][1:] - s["kv_off"][:-1]
    L = case["most"] + case["ctx"]
    token = torch.arange(L, device="cuda")
    there = token < kv[:, None]
    at = torch.where(there, s["kv_off"][:-1, None] + token, 0).long()
    pad = lambda x: x[at].float().mul_(there[..., None, None]).transpose(1, 2)  # noqa: E731
    return _run_rows(s, pad(s["k"]), pad(s["v"]), kv, L)


def _run_attend(s):
    case = s["case"]
    L = s["table"].shape[1] * case["page"]
    pages = s["table"].clamp(min=0).long()
    token = torch.arange(case["page"], device="cuda")
    there = torch.arange(L, device="cuda") < s["kv_len"][:, None]
    held = []
    for kind in (0, 1):
        x = _swizzle(s["data"][:, :, kind][pages], token).view(torch.float8_e4m3fn).float()   # [B, pages, heads, page, D]
        e = s["scales"][:, :, kind][pages].int() - 127
        x = torch.ldexp(x, e.repeat_interleave(16, -1)[..., None]).transpose(1, 2).flatten(2, 3)
        held.append(x.mul_(there[:, None, :, None]))
    return _run_rows(s, *held, s["kv_len"], L)


def run(s):
    op, case = s["case"]["op"], s["case"]
    if own:
        import speculative_decoding_draft_gb300 as ds
        if op == "prompt":
            r = ds.attend_prompt(s["q"], s["k"], s["v"], s["row_off"], kv_off=s["kv_off"], causal=case["causal"],
                                 window=case["window"], want_lse=True, status=s["status"])
            return dict(out=r["out"], lse=r["lse"])
        if op == "append":
            r = ds.cache_append(s["cache"], s["k"], s["v"], s["row_off"], s["kv_len"], s["table"], rope=s["rope"],
                                k_weight=s["k_weight"], q=s["q"], q_weight=s["q_weight"], eps=1e-6, status=s["status"])
            c = ds.cache_read(s["cache"], s["read_off"], s["kv_len"], s["table"], s["read_rows"], dtype=torch.bfloat16,
                              status=s["status"])
            return dict(q=r["q"], k=c["k"], v=c["v"])
        r = ds.attend_paged(s["q"], s["cache"], s["row_off"], s["kv_len"], s["table"], causal=case["causal"],
                            window=case["window"], max_rows=case["most"], want_lse=True, status=s["status"])
        return dict(out=r["out"], lse=r["lse"])
    return {"prompt": _run_prompt, "append": _run_append, "attend": _run_attend}[op](s)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    op, B = case["op"], case["B"]
    size = 4 if case["dtype"] == "fp32" else 2
    n = _counts(case).tolist()
    rows = sum(n)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "prompt":
        pairs, tokens = 0.0, 0.0
        for m in n:
            ctx = case["ctx"] / (1 if B == 1 else 2)
            seen = ctx + (m + 1) / 2 if case["causal"] else ctx + m
            if case["window"]:
                seen = min(seen, case["window"])
            pairs += m * seen
            tokens += m + (min(ctx, case["window"]) if case["window"] else ctx)
        return dict(bytes=(2 * rows * hq + 2 * tokens * hkv) * d * size + 4 * rows * hq, flops=4 * pairs * hq * d)
    held = 2 * (d + 1 / 16)                                                   # a token's bytes in one head
    if op == "append":
        # queries in and out, keys and values in, the cache written, read back and returned in 16 bits
        back = rows + sum(_begun(case))
        return dict(bytes=rows * (2 * hq * d * size + 2 * hkv * d * size + hkv * held) + back * hkv * (held + 4 * d),
                    flops=rows * (7 * (hq + hkv) * d + 4 * hkv * d))
    tokens = case["kv"] + (B - 1) * case["kv"] * 0.5625                       # kept lengths are 1/8 to 1 of kv
    if case["window"]:
        span = case["window"] + case["most"] - 1
        tokens = min(tokens, B * span)
    return dict(bytes=tokens * hkv * held + 2 * rows * hq * d * size + 4 * rows * hq,
                flops=4 * tokens * hq * d * rows / B)


# ---------------------------------------------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _exact_heads(x, weight, pos, s):
    """Norm and rotation of [rows, heads, D] as complex products in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * weight.double()
    case, angle = s["case"], torch.outer(pos.double(), s["inv_freq"])
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    part, rest = x[..., : case["rot"]], x[..., case["rot"]:]
    if case["layout"] == "half":
        z = torch.complex(*part.contiguous().chunk(2, -1)) * turn
        return torch.cat((z.real, z.imag, rest), -1)
    z = torch.view_as_complex(part.contiguous().unflatten(-1, (-1, 2))) * turn
    return torch.cat((torch.view_as_real(z).flatten(-2), rest), -1)


def _exact_held(s, r, kind, end):
    """Keys or values [heads, end, D] of request r, element by element from the layout."""
    case = s["case"]
    page, d = case["page"], case["d"]
    tok, i = torch.arange(end, device="cuda"), torch.arange(d, device="cuda")
    at, t = s["table"][r][tok // page].long(), tok % page
    turn = t % 8 if d == 128 else t // 2 % 4
    place = ((i // 16)[None] ^ turn[:, None]) * 16 + i % 16
    x = s["data"][at, :, kind, t].gather(-1, place[:, None].expand(-1, case["hkv"], -1))
    x = x.view(torch.float8_e4m3fn).double() * 2.0 ** (s["scales"][at, :, kind, t // 16].double() - 127)[..., None]
    return x.transpose(0, 1)


def _exact_values(x):
    """e4m3 of x: three bits behind the leading one, steps of 2^-9 at least, to the nearest, ties to even, to 448 at most."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_attend(case, q, k, v, end):
    """q [rows, heads, D] of one request, its keys and values [kv heads, tokens, D]: out and lse in 64 bits."""
    n, (hkv, kv, d), group = len(q), k.shape, case["hq"] // case["hkv"]
    out = torch.zeros(n, case["hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, case["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 28) // max(1, group * kv))
    tok = torch.arange(kv, device="cuda")
    for h in range(hkv):
        heads = slice(h * group, (h + 1) * group)
        for a in range(0, n, step):
            b = min(n, a + step)
            hi = torch.arange(a, b, device="cuda") + end - n + 1 if case["causal"] else torch.full((b - a,), end, device="cuda")
            lo = hi - case["window"] if case["window"] else torch.zeros_like(hi)
            hide = (tok >= hi[:, None]) | (tok < lo[:, None])
            score = torch.einsum("xgd,td->gxt", q[a:b, heads].double(), k[h]).div_(math.sqrt(d)).masked_fill_(hide, -math.inf)
            z = torch.logsumexp(score, -1)
            some = (~hide).any(-1)
            p = score.sub_(torch.where(some, z, 0)[..., None]).exp_()
            out[a:b, heads] = torch.einsum("gxt,td->xgd", p, v[h])
            lse[a:b, heads] = z.T
    return out, lse


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, off = case["op"], s["row_off"].tolist()
    if op == "append":
        kv = s["kv_len"].tolist()
        pos = torch.cat([torch.arange(b - a, device="cuda") + e - (b - a) for a, b, e in zip(off, off[1:], kv)])
        # a key near the border of two elements has no element of its own in 64 bits: the queries and values are held
        raw, back = s["v"].double(), s["read_off"].tolist()
        v = torch.empty(s["read_rows"], case["hkv"], case["d"], dtype=torch.float64, device="cuda")
        if case["B"] > 256 or s["rows"] > 20000:
            return dict(q=_exact_heads(s["q"], s["q_weight"], pos, s), k=None, v=None)
        for r in range(case["B"]):
            first, end = kv[r] - (off[r + 1] - off[r]), kv[r]
            start = first // 16 * 16
            was_e = s["scales"][s["table"][r, start // case["page"]].long(), :, 1, start % case["page"] // 16].double() - 127
            held = _exact_held(s, r, 1, first)[:, start:].transpose(0, 1) if first > start else None
            both = raw[off[r]: off[r + 1]] if held is None else torch.cat((torch.zeros_like(held), raw[off[r]: off[r + 1]]))
            for at in range(0, len(both), 16 * 4096):
                x = both[at: at + 16 * 4096]
                whole = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -len(x) % 16)).unflatten(0, (-1, 16))
                top = whole.abs().amax((1, 3))
                e = torch.ceil(torch.log2(top / 448)).clamp(E_LOW, E_HIGH)
                if at == 0 and held is not None:
                    e[0] = torch.maximum(e[0], was_e)
                    whole[0, : len(held)] = held
                unit = torch.exp2(e)[:, None, :, None]
                v[back[r] + at: back[r] + at + len(x)] = (_exact_values(whole / unit) * unit).flatten(0, 1)[: len(x)]
        return dict(q=_exact_heads(s["q"], s["q_weight"], pos, s), k=None, v=v)
    out = torch.zeros(s["rows"], case["hq"], case["d"], dtype=torch.float64, device="cuda")
    lse = torch.full((s["rows"], case["hq"]), -math.inf, dtype=torch.float64, device="cuda")
    kv_off = s["kv_off"].tolist() if op == "prompt" else None
    for r in range(case["B"]):
        a, b = off[r], off[r + 1]
        if op == "prompt":
            c, e = kv_off[r], kv_off[r + 1]
            end, k, v = e - c, s["k"][c:e].double().transpose(0, 1), s["v"][c:e].double().transpose(0, 1)
        else:
            end = int(s["kv_len"][r])
            if not end:
                continue
            k, v = _exact_held(s, r, 0, end), _exact_held(s, r, 1, end)
        out[a:b], lse[a:b] = _exact_attend(case, s["q"][a:b], k, v, end)
    return dict(out=out, lse=lse)
