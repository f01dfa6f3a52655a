"""Cases, inputs, plain forms and 64-bit definitions of the operators around a ragged verification step.

A target model that verifies drafted tokens runs, per attention layer, over ragged rows (request r owns rows
row_off[r] .. row_off[r+1]-1, the last of its kv_len[r] tokens):

  rotate     norm of every query and key head with the position rotation in the same pass;
  append     the same on the way into a paged key/value cache held in 4 bits (and the rotated queries out);
  attend     attention of the rows over that cache;
  penalize   repetition, presence and frequency penalties, biases and grammar masks on the rows' logits, each row
             counting the draft tokens before it.

The cache: a page of P tokens holds, for one key/value head of D dimensions, P/16 tiles of 16 tokens, 18 D bytes each:
  [0, 8D)     keys: token t at t D/2, two e2m1 codes a byte, the even dimension in the low half;
  [8D, 16D)   values: with w = D/16, chunk g (dimensions 2wg .. 2wg+2w-1) of token t at w (64 (t/8) + 8g + t%8);
  [16D, 17D)  key scales (e4m3, one for 16 dimensions): token t, group c at t D/16 + c;
  [17D, 18D)  value scales: token t, group c at (t/8) D/2 + 8c + t%8.
A stored element is e2m1 * e4m3 * (the cache's power-of-two scale).

`run` returns whole outputs.  What the cache holds comes back as its elements and its scales, both exact in
float8_e4m3fn."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E2M1_EDGES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)   # ties go to the even code


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # one layer of a 64-request step with 8 rows each, normed heads
        dict(name="rotate step", op="rotate", dtype="bf16", rows=512, hq=32, hkv=8, d=128, rot=128, layout="half",
             scaling="none", norm=True, far=4096),
        # a long-context prefill chunk: part of the head rotated, neighbouring pairs, frequencies blended
        dict(name="rotate long partial", op="rotate", dtype="fp16", rows=8191, hq=24, hkv=4, d=96, rot=64,
             layout="interleaved", scaling="yarn", norm=False, far=1000000),
        # a single user's next token
        dict(name="append one token", op="append", dtype="bf16", B=1, most=1, kv=777, hq=32, hkv=8, d=128, page=16,
             rot=128, layout="half", scaling="none", norm=True),
        # the ragged step: 2048 requests with 1 to 8 rows each
        dict(name="append ragged", op="append", dtype="bf16", B=2048, most=8, kv=2048, hq=32, hkv=8, d=128, page=64,
             rot=128, layout="half", scaling="none", norm=True),
        # a prompt chunk of a few requests, small heads
        dict(name="append chunk", op="append", dtype="fp16", B=3, most=2731, kv=9000, hq=12, hkv=4, d=64, page=32,
             rot=32, layout="interleaved", scaling="linear", norm=False),
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
        # a handful of requests over a small vocabulary
        dict(name="penalize tiny", op="penalize", dtype="fp32", B=4, most=8, V=1000, hist=61, bias=3, mask=True),
        # the 64-request step with grammar masks
        dict(name="penalize step", op="penalize", dtype="bf16", B=64, most=8, V=151936, hist=2048, bias=16, mask=True),
        # the ragged step without grammars
        dict(name="penalize ragged", op="penalize", dtype="bf16", B=2048, most=8, V=151936, hist=1024, bias=0,
             mask=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotate", "append", "attend", "penalize"))
    if op == "penalize":
        B, V = _log(rng, 1, 2048), _log(rng, 500, 160000)
        most = rng.randint(1, 9)
        while B * most * V > 2048 * 8 * 151936:
            B = max(1, B // 2)
        return dict(op=op, dtype=rng.choice(("bf16", "fp32")) if B * most * V < 1 << 30 else "bf16", B=B, most=most,
                    V=V, hist=_log(rng, 1, 8192), bias=rng.choice((0, 1, 7, 40)), mask=rng.random() < 0.6)
    d = rng.choice((64, 128))
    hkv, group = rng.choice((1, 2, 3, 4, 8)), rng.choice((1, 2, 3, 4, 6, 8))
    c = dict(op=op, dtype=rng.choice(("bf16", "fp16")), hq=hkv * group, hkv=hkv, d=d)
    if op == "attend":
        B, kv, most = _log(rng, 1, 256), _log(rng, 1, 131071), rng.choice((1, 1, 2, 5, 8, rng.randint(9, 40)))
        while B * kv * hkv * d > 256 * 16384 * 8 * 64 or B * kv * hkv * group * most > 256 * 16384 * 32 * 2:
            B, kv = max(1, B // 2), max(1, kv // 2) if B == 1 else kv
        return dict(c, B=B, most=most, kv=kv, page=rng.choice((16, 32, 64, 128)), causal=rng.random() < 0.75,
                    window=rng.choice((0, 0, 0, 333, 4096)))
    c.update(rot=rng.choice((d, d, d // 2)), layout=rng.choice(("half", "interleaved")),
             scaling=rng.choice(("none", "linear", "ntk", "yarn")), norm=rng.random() < 0.6)
    if op == "rotate":
        c.update(dtype=rng.choice(("bf16", "fp16", "fp32")), d=rng.choice((64, 80, 96, 128, 256)))
        c["rot"] = c["d"] if rng.random() < 0.6 else c["d"] // 32 * 16
        return dict(c, rows=_log(rng, 1, 8192), far=_log(rng, 1000, 2000000))
    B, most = _log(rng, 1, 2048), _log(rng, 1, 3000)
    while B * most > 16384:
        B, most = max(1, B // 2), max(1, most // 2) if B == 1 else most
    return dict(c, B=B, most=most, kv=most + _log(rng, 1, 2048), page=rng.choice((16, 32, 64, 128)))


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + salt)
    return g


def _ints(g, lo, hi, shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _least(case):
    return max(1, case["most"] // 8) if case["B"] < 8 else 1


def _ragged(case, g):
    """row_off [B+1] and each request's rows: spread evenly over least .. most, in an order of the seed's."""
    least, B = _least(case), case["B"]
    n = case["most"] - torch.arange(B, device="cuda", dtype=torch.int32) % (case["most"] - least + 1)
    n = n[torch.randperm(B, generator=g, device="cuda")]
    off = torch.zeros(case["B"] + 1, dtype=torch.int32, device="cuda")
    off[1:] = n.cumsum(0)
    return n, off


def _pages(case, kv_len, g):
    """A page table over shuffled pages, -1 past a request's last page, and the number of pages."""
    need = (kv_len + case["page"] - 1) // case["page"]
    width, total = max(1, int(need.max())), int(need.sum())
    table = torch.full((case["B"], width), -1, dtype=torch.int32, device="cuda")
    ids = torch.randperm(max(1, total), generator=g, device="cuda").to(torch.int32)
    table[torch.arange(width, device="cuda")[None] < need[:, None]] = ids[:total]
    return table, max(1, total)


def _frequencies(case):
    """inv_freq (64-bit, the rotary pairs') and the factor on cos and sin."""
    rot, base, factor, trained = case["rot"], 1e6, 8.0, 32768
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    kind = case["scaling"]
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    inv = base ** (-2 * i / rot)
    if kind == "linear":
        inv = inv / factor
    if kind == "yarn":   # pairs with over 32 turns in the trained length stay, those under 1 are divided, a ramp between
        at = lambda turns: rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        inv = inv * (1 - ramp) + inv / factor * ramp
        return inv, 0.1 * math.log(factor) + 1
    return inv, 1.0


def _rope(case):
    import speculative_decoding_draft_gb300 as ds
    return ds.Rope(case["rot"], base=1e6, layout=case["layout"], scaling=case["scaling"], factor=8.0,
                   original_len=32768, device="cuda")


def _cache(data, case):
    import speculative_decoding_draft_gb300 as ds
    return ds.PagedCache(data, case["page"], k_scale=0.5, v_scale=0.25)


K_SCALE, V_SCALE = 0.5, 0.25


def prepare(case, seed):
    g = _gen(seed, 1)
    op, s = case["op"], dict(case=case)
    dt = DTYPES[case["dtype"]]
    if op == "penalize":
        B, V, most = case["B"], case["V"], case["most"]
        n, off = _ragged(case, g)
        rows = int(off[-1])
        s.update(rows=rows, row_off=off, logits=torch.empty(rows, V, dtype=dt, device="cuda"))
        for at in range(0, rows, 1024):
            s["logits"][at: at + 1024] = _normal(g, (min(1024, rows - at), V), dt, 3.0)
        # a text repeats itself: most tokens come from a few hundred common ones
        u = torch.rand(B, case["hist"], generator=g, device="cuda")
        s["hist"] = ((u ** 4) * (V - 1)).to(torch.int32)
        s["hist_len"] = _ints(g, 0, case["hist"], (B,))
        s["hist_len"][-1] = case["hist"]
        s["prompt_len"] = (s["hist_len"] * torch.rand(B, generator=g, device="cuda")).to(torch.int32)
        s["draft_tok"] = ((torch.rand(B, most, generator=g, device="cuda") ** 4) * (V - 1)).to(torch.int32)
        s["repetition"] = 1.0 + 0.3 * torch.rand(B, generator=g, device="cuda")
        s["presence"] = torch.rand(B, generator=g, device="cuda")
        s["frequency"] = torch.rand(B, generator=g, device="cuda") * 0.5
        s["bias_tok"] = s["bias_val"] = s["mask"] = None
        if case["bias"]:
            s["bias_tok"] = _ints(g, -1, V - 1, (B, case["bias"]))
            s["bias_val"] = torch.randn(B, case["bias"], generator=g, device="cuda") * 4
        if case["mask"]:   # a third of the rows is free, a third in running text, a third inside a narrow rule
            words = _ints(g, -2 ** 31, 2 ** 31 - 1, (rows, (V + 31) // 32))
            kind = _ints(g, 0, 2, (rows, 1))
            thin = words & (words << 7) & (words >> 5) & (words << 3) & (words << 11)
            s["mask"] = torch.where(kind == 0, torch.full_like(words, -1), torch.where(kind == 1, words, thin))
    else:
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        if op == "rotate":
            rows = case["rows"]
            s["positions"] = _ints(g, 0, case["far"], (rows,))
        else:
            n, off = _ragged(case, g)
            rows = int(off[-1])
            kv_len = (torch.rand(case["B"], generator=g, device="cuda") * 0.875 + 0.125) * case["kv"]
            kv_len = kv_len.to(torch.int32)
            kv_len[-1] = case["kv"]
            if op == "append":
                kv_len = torch.maximum(kv_len, n)
            elif case["B"] > 2:
                kv_len[0] = 0            # a request whose cache is still empty
            s["table"], pages = _pages(case, kv_len, g)
            s.update(row_off=off, kv_len=kv_len, n=n)
        s["rows"] = rows
        # queries, keys and values as one projection leaves them
        qkv = _normal(g, (rows, hq + 2 * hkv, d), dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq: hq + hkv], qkv[:, hq + hkv:]
        if op == "attend":
            s["q"] = s["q"].contiguous()
            s["k"] = s["v"] = None
            data = torch.empty(pages, hkv, case["page"] // 16, 18 * d, dtype=torch.uint8, device="cuda")
            step = max(1, (1 << 27) // (hkv * case["page"] * d))
            for at in range(0, pages, step):
                m = min(step, pages - at)
                x = torch.randn(2, m, hkv, case["page"], d, generator=g, device="cuda")
                (kc, ks), (vc, vs) = _quantize(x[0] / K_SCALE), _quantize(x[1] / V_SCALE)
                data[at: at + m] = _pack(kc, ks, vc, vs)
            s["cache"] = data
        else:
            s["inv_freq"], s["gain"] = _frequencies(case)
            s["q_weight"] = s["k_weight"] = None
            if case["norm"]:
                s["q_weight"] = 1 + _normal(g, (d,), torch.float32, 0.1)
                s["k_weight"] = 1 + _normal(g, (d,), torch.float32, 0.1)
                s["q_weight"], s["k_weight"] = s["q_weight"].to(dt), s["k_weight"].to(dt)
        if op == "append":
            s["cache"] = torch.zeros(pages, hkv, case["page"] // 16, 18 * d, dtype=torch.uint8, device="cuda")
    if own:
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if op in ("rotate", "append"):
            s["rope"] = _rope(case)
        if op in ("append", "attend"):
            s["paged"] = _cache(s["cache"], case)
    return s


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------
def _quantize(x):
    """Codes (uint8, of 4 bits) and scales (e4m3) of x [..., D], 16 dimensions to a scale: scale = e4m3(max|x| / 6),
    code = e2m1(x / scale); both to nearest, ties to even, saturating."""
    y = x.float().unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    z = y / scale.float()[..., None]
    z = torch.where(scale.float()[..., None] == 0, torch.zeros_like(z), z)
    a = z.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i, edge in enumerate(E2M1_EDGES):
        code += (a > edge) if i % 2 == 0 else (a >= edge)
    return (code | (z < 0).to(torch.uint8) << 3).flatten(-2), scale


def _pack(kc, ks, vc, vs):
    """Codes [..., P, D] and scales [..., P, D/16] as tiles [..., P/16, 18 D]."""
    p, d = kc.shape[-2:]
    w, lead = d // 16, kc.shape[:-2]
    pair = lambda c: (c[..., 0::2] | (c[..., 1::2] << 4))  # noqa: E731
    k = pair(kc).reshape(*lead, p // 16, 8 * d)
    v = pair(vc).reshape(*lead, p // 16, 2, 8, 8, w).transpose(-3, -2).reshape(*lead, p // 16, 8 * d)
    ks = ks.view(torch.uint8).reshape(*lead, p // 16, d)
    vs = vs.view(torch.uint8).reshape(*lead, p // 16, 2, 8, w).transpose(-2, -1).reshape(*lead, p // 16, d)
    return torch.cat((k, v, ks, vs), -1)


def _unpack(tiles, d):
    """Keys and values [..., tokens, D] in 32 bits (without the cache's scales) from tiles [..., T, 18 D]."""
    lead, w = tiles.shape[:-1], d // 16
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=tiles.device)

    def values(b, scale):
        x = torch.stack((b & 15, b >> 4), -1).flatten(-2).int()
        return (table[x].unflatten(-1, (-1, 16)) * scale.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)

    k = values(tiles[..., : 8 * d].reshape(*lead, 16, d // 2), tiles[..., 16 * d: 17 * d].reshape(*lead, 16, w))
    v = values(tiles[..., 8 * d: 16 * d].reshape(*lead, 2, 8, 8, w).transpose(-3, -2).reshape(*lead, 16, d // 2),
               tiles[..., 17 * d:].reshape(*lead, 2, w, 8).transpose(-2, -1).reshape(*lead, 16, w))
    return k.flatten(-3, -2), v.flatten(-3, -2)


def _norm_rope(x, weight, positions, inv_freq, gain, case):
    """x [rows, heads, D] in 32 bits: root-mean-square norm of each head where there is a weight, then the rotation of
    its first `rot` dimensions; angles in 64 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = positions.double()[:, None] * inv_freq
    c, s = ((f(angle) * gain).float()[:, None] for f in (torch.cos, torch.sin))
    rot = case["rot"]
    y = x.clone()
    if case["layout"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    return y


def _row_places(s):
    """Each row's request and its position in that request."""
    rows = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    req = torch.searchsorted(s["row_off"][1:], rows, right=True)
    return req, (s["kv_len"] - s["n"])[req] + rows - s["row_off"][req]


def _run_append(s):
    case = s["case"]
    d, hkv, page = case["d"], case["hkv"], case["page"]
    w = d // 16
    req, pos = _row_places(s)
    rope = (pos, s["inv_freq"], s["gain"], case)
    q = _norm_rope(s["q"], s["q_weight"], *rope).to(s["q"].dtype)
    kc, ks = _quantize(_norm_rope(s["k"], s["k_weight"], *rope) / K_SCALE)
    vc, vs = _quantize(s["v"].float() / V_SCALE)
    at = s["table"][req, (pos // page).long()].long()[:, None, None]
    tile, t = (pos % page // 16).long()[:, None, None], (pos % 16).long()[:, None, None]
    head = torch.arange(hkv, device="cuda")[None, :, None]
    i, c = torch.arange(d // 2, device="cuda"), torch.arange(w, device="cuda")
    pair = lambda x: x[..., 0::2] | (x[..., 1::2] << 4)  # noqa: E731
    data = s["cache"]
    data[at, head, tile, t * (d // 2) + i] = pair(kc)
    data[at, head, tile, 8 * d + w * (64 * (t // 8) + 8 * (i // w) + t % 8) + i % w] = pair(vc)
    data[at, head, tile, 16 * d + t * w + c] = ks.view(torch.uint8)
    data[at, head, tile, 17 * d + t // 8 * (d // 2) + 8 * c + t % 8] = vs.view(torch.uint8)
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda")
    return dict(q=q, k=table[kc.int()].to(torch.float8_e4m3fn), k_scale=ks,
                v=table[vc.int()].to(torch.float8_e4m3fn), v_scale=vs)


def _run_attend(s):
    case = s["case"]
    d, hq, hkv, B, most = case["d"], case["hq"], case["hkv"], case["B"], case["most"]
    group, L = hq // hkv, s["table"].shape[1] * case["page"]
    req, pos = _row_places(s)
    j = torch.arange(s["rows"], device="cuda") - s["row_off"][req]
    q = torch.zeros(B, most, hq, d, device="cuda")
    q[req, j] = s["q"].float()
    q = q.view(B, most, hkv, group, d).transpose(1, 2).reshape(B, hkv, most * group, d)
    tiles = s["cache"][s["table"].clamp(min=0)].transpose(1, 2).flatten(2, 3)      # [B, hkv, tiles, 18 D]
    k, v = _unpack(tiles, d)
    p = (q @ k.transpose(-1, -2)) * (K_SCALE / math.sqrt(d))
    end = s["kv_len"][:, None].expand(B, most)
    if case["causal"]:
        end = (s["kv_len"] - s["n"])[:, None] + torch.arange(most, device="cuda") + 1
    token = torch.arange(L, device="cuda")
    seen = (token < end[..., None]) & (token < s["kv_len"][:, None, None])
    if case["window"]:
        seen &= token >= end[..., None] - case["window"]
    seen = seen[:, None, :, None].expand(B, 1, most, group, L).reshape(B, 1, most * group, L)
    p.masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(p.sub_(base))
    total = p.sum(-1, keepdim=True)
    v = torch.where((token < s["kv_len"][:, None])[:, None, :, None], v, 0)
    out = (p @ v) * V_SCALE / torch.where(total == 0, torch.ones_like(total), total)
    lse = (base + torch.log(total)).squeeze(-1)
    shape = lambda x: x.view(B, hkv, most, group, -1).transpose(1, 2).reshape(B, most, hq, -1)[req, j]  # noqa: E731
    return dict(out=shape(out).to(s["q"].dtype), lse=shape(lse).squeeze(-1))


def _run_penalize(s):
    case = s["case"]
    B, V, most = case["B"], case["V"], case["most"]
    rows = torch.arange(s["rows"], device="cuda")
    req = torch.searchsorted(s["row_off"][1:], rows.int(), right=True)
    j = rows - s["row_off"][req]
    place = torch.arange(case["hist"], device="cuda")
    there, prompt = place < s["hist_len"][:, None], place < s["prompt_len"][:, None]
    counts = torch.zeros(B, V, dtype=torch.int32, device="cuda")
    counts.scatter_add_(1, s["hist"].long(), (there & ~prompt).int())
    seen = torch.zeros(B, V, dtype=torch.int32, device="cuda")
    seen.scatter_add_(1, s["hist"].long(), (there & prompt).int())
    n = counts[req]
    n.scatter_add_(1, s["draft_tok"][req].long(), (torch.arange(most, device="cuda") < j[:, None]).int())
    z = s["logits"].float()
    one = lambda x: x[req][:, None]  # noqa: E731
    z = torch.where((n > 0) | (seen > 0)[req], torch.where(z > 0, z / one(s["repetition"]), z * one(s["repetition"])), z)
    z -= (n > 0) * one(s["presence"])
    z -= n * one(s["frequency"])
    if s["bias_tok"] is not None:
        bias = torch.zeros(B, V + 1, device="cuda")
        bias.scatter_add_(1, torch.where(s["bias_tok"] < 0, V, s["bias_tok"]).long(), s["bias_val"])
        z += bias[:, :V][req]
    if s["mask"] is not None:
        token = torch.arange(V, device="cuda")
        z.masked_fill_((s["mask"][:, token // 32] >> (token % 32).int()) & 1 == 0, -math.inf)
    return z.to(s["logits"].dtype)


def run(s):
    op, case = s["case"]["op"], s["case"]
    if own:
        import speculative_decoding_draft_gb300 as ds
        if op == "rotate":
            r = ds.norm_rope(s["q"], s["k"], s["positions"], s["rope"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                             eps=1e-6, status=s["status"])
            return dict(q=r["q"], k=r["k"])
        if op == "append":
            r = ds.cache_append(s["paged"], s["k"], s["v"], s["row_off"], s["kv_len"], s["table"], rope=s["rope"],
                                k_weight=s["k_weight"], q=s["q"], q_weight=s["q_weight"], eps=1e-6, status=s["status"])
            c = ds.cache_read(s["paged"], s["row_off"], s["kv_len"], s["table"], s["rows"], status=s["status"])
            return dict(q=r["q"], k=c["k"], k_scale=c["k_scale"], v=c["v"], v_scale=c["v_scale"])
        if op == "attend":
            r = ds.attend_paged(s["q"], s["paged"], s["row_off"], s["kv_len"], s["table"], causal=case["causal"],
                                window=case["window"], max_rows=case["most"], want_lse=True, status=s["status"])
            return dict(out=r["out"], lse=r["lse"])
        return ds.penalize_logits(s["logits"], s["row_off"], s["hist"], s["hist_len"], s["prompt_len"],
                                  s["repetition"], s["presence"], s["frequency"], draft_tok=s["draft_tok"],
                                  bias_tok=s["bias_tok"], bias_val=s["bias_val"], mask=s["mask"],
                                  status=s["status"])["logits"]
    if op == "rotate":
        return {h: _norm_rope(s[h], s[h + "_weight"], s["positions"], s["inv_freq"], s["gain"], case).to(s[h].dtype)
                for h in ("q", "k")}
    return {"append": _run_append, "attend": _run_attend, "penalize": _run_penalize}[op](s)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "rotate":
        heads = case["rows"] * (case["hq"] + case["hkv"]) * case["d"]
        return dict(bytes=2 * heads * size + 4 * case["rows"], flops=(4 if case["norm"] else 0) * heads + 3 * heads)
    B, most = case["B"], case["most"]
    rows = sum(most - i % (most - _least(case) + 1) for i in range(B))
    if op == "penalize":
        table = rows * ((case["V"] + 31) // 32) * 4 if case["mask"] else 0
        lists = B * (case["hist"] * 2 + most * 4 + case["bias"] * 8)
        return dict(bytes=2 * rows * case["V"] * size + table + lists, flops=3 * rows * case["V"])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    tokens = case["kv"] + (B - 1) * case["kv"] * 0.5625                       # kept lengths are 1/8 to 1 of kv
    held = 2 * (d // 2 + d // 16)                                             # a token's bytes in one head
    if op == "append":
        # queries in and out, keys and values in, the cache written, read back and returned
        return dict(bytes=rows * (2 * hq * d * size + 2 * hkv * d * size + hkv * (2 * held + 2 * (d + d // 16))),
                    flops=rows * (7 * (hq + hkv) * d + 6 * hkv * d))
    if case["window"]:
        span = case["window"] + most - 1
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
    turn = torch.polar(torch.full_like(angle, s["gain"]), angle)[:, None]
    part, rest = x[..., : case["rot"]], x[..., case["rot"]:]
    if case["layout"] == "half":
        z = torch.complex(*part.contiguous().chunk(2, -1)) * turn
        return torch.cat((z.real, z.imag, rest), -1)
    z = torch.view_as_complex(part.contiguous().unflatten(-1, (-1, 2))) * turn
    return torch.cat((torch.view_as_real(z).flatten(-2), rest), -1)


def _exact_values(x):
    """What 4 bits keep of x [..., D]: the nearest elements and scales, as numbers."""
    y = x.double().unflatten(-1, (-1, 16))
    scale = (y.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn).double()
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    z = torch.where(scale[..., None] > 0, y / scale[..., None], 0.0)
    near = (z.abs()[..., None] - grid).abs()
    # of two that are as near, the even code
    best = (near + torch.tensor([0, 1e-13] * 4, dtype=torch.float64, device="cuda")).argmin(-1)
    return (grid[best] * z.sign()).flatten(-2), scale


def _exact_held(tiles, d):
    """Keys and values [heads, tokens, D] of one request's tiles [heads, T, 18 D], byte by byte from the layout."""
    t, i = torch.arange(16, device="cuda")[:, None], torch.arange(d, device="cuda")
    w = d // 16
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    places = ((t * (d // 2) + i // 2, 16 * d + t * w + i // 16, K_SCALE),
              (8 * d + w * (64 * (t // 8) + 8 * (i // (2 * w)) + t % 8) + i % (2 * w) // 2,
               17 * d + t // 8 * (d // 2) + 8 * (i // 16) + t % 8, V_SCALE))
    for element, scale, f in places:
        code = (tiles[..., element].int() >> (4 * (i % 2)).int()) & 15
        x = grid[(code & 7).long()] * (1 - 2 * (code >> 3)) * f
        yield (x * tiles[..., scale].view(torch.float8_e4m3fn).double()).flatten(1, 2)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "rotate":
        return {h: _exact_heads(s[h], s[h + "_weight"], s["positions"], s) for h in ("q", "k")}
    off = s["row_off"].tolist()
    if op == "append":
        pos = torch.cat([torch.arange(b - a, device="cuda") + e - (b - a)
                         for a, b, e in zip(off, off[1:], s["kv_len"].tolist())])
        v, vs = _exact_values(s["v"].double() / V_SCALE)
        # a key near the border of two codes has no code of its own in 64 bits: only the queries and values are held
        return dict(q=_exact_heads(s["q"], s["q_weight"], pos, s), k=None, k_scale=None, v=v, v_scale=vs)
    if op == "penalize":
        if s["rows"] * case["V"] > 1 << 28:
            return None
        out = torch.empty(s["rows"], case["V"], dtype=torch.float64, device="cuda")
        for r in range(case["B"]):
            hist, prompt = s["hist"][r, : s["hist_len"][r]].long(), int(s["prompt_len"][r])
            said = torch.bincount(hist[prompt:], minlength=case["V"]).double()
            told = torch.bincount(hist[:prompt], minlength=case["V"])
            rep, pre, fre = (s[k][r].double() for k in ("repetition", "presence", "frequency"))
            for i in range(off[r], off[r + 1]):
                z = s["logits"][i].double()
                z = torch.where((said + told) > 0, torch.where(z > 0, z / rep, z * rep), z)
                z = z - pre * said.clamp(max=1) - fre * said
                if s["bias_tok"] is not None:
                    real = s["bias_tok"][r] >= 0
                    z.index_add_(0, s["bias_tok"][r][real].long(), s["bias_val"][r][real].double())
                if s["mask"] is not None:
                    bits = (s["mask"][i][:, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
                    z[bits.flatten()[: case["V"]] == 0] = -math.inf
                out[i] = z
                said[int(s["draft_tok"][r, i - off[r]])] += 1
        return out
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    out = torch.zeros(s["rows"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((s["rows"], hq), -math.inf, dtype=torch.float64, device="cuda")
    for r in range(case["B"]):
        a, b, end = off[r], off[r + 1], int(s["kv_len"][r])
        if not end:
            continue
        pages = s["table"][r, : -(-end // case["page"])].long()
        held = s["cache"][pages].transpose(0, 1).flatten(1, 2)                 # [hkv, tiles, 18 D]
        k, v = (x[:, :end] for x in _exact_held(held, d))
        for i in range(a, b):
            hi = end - (b - a) + (i - a) + 1 if case["causal"] else end
            lo = max(0, hi - case["window"]) if case["window"] else 0
            if hi <= lo:
                continue
            q = s["q"][i].double().view(hkv, hq // hkv, d)
            score = torch.einsum("hgd,htd->hgt", q, k[:, lo:hi]) / math.sqrt(d)
            lse[i] = torch.logsumexp(score, -1).flatten()
            out[i] = torch.einsum("hgt,htd->hgd", torch.softmax(score, -1), v[:, lo:hi]).reshape(hq, d)
    return dict(out=out, lse=lse)
