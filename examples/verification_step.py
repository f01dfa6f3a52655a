"""Speculative decoding of a small random target model, with every operator of the verification step.

    python examples/verification_step.py [--steps 8] [--temperature 0.0] [--bits 4]

Each step drafts up to K tokens a request, schedules how many of them to verify, runs the target model over
the ragged rows (per layer: project, norm, rotate and append in one call, attend over the cache, of 4 or 8 bits),
penalises and masks the rows' logits, and accepts or rejects.  Rejected tokens need no clean-up: the next
step's rows take their places in the cache.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_draft_gb300 as ds  # noqa: E402


class Target:
    """A decoder of random weights: attention layers with normed, rotated heads and a gated residual."""

    def __init__(self, B, V=512, layers=2, hq=4, hkv=2, d=64, page=16, most=512, seed=0, bits=4):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        w = hq * d

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

        self.B, self.V, self.hq, self.hkv, self.d = B, V, hq, hkv, d
        self.embed = normal(V, w, std=1.0)
        self.head = normal(w, V, std=2.0 * w ** -0.5)
        self.layers = [dict(qkv=normal(w, (hq + 2 * hkv) * d, std=w ** -0.5), out=normal(w, w, std=w ** -0.5),
                            qn=(1 + normal(d, std=0.1)), kn=(1 + normal(d, std=0.1))) for _ in range(layers)]
        per = -(-most // page)
        self.table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
        self.caches = [ds.PagedCache8.empty(B * per, hkv, d, page) if bits == 8 else
                       ds.PagedCache.empty(B * per, hkv, d, page, k_scale=0.25, v_scale=0.25) for _ in range(layers)]
        self.rope = ds.Rope(d, base=1e4, scaling="yarn", factor=4.0, original_len=128)
        self.status = ds.new_status("cuda")

    def rows(self, tokens, row_off, kv_len, max_rows):
        """Logits (float32) of the rows' tokens, the last of each request's kv_len."""
        n, hq, hkv, d = len(tokens), self.hq, self.hkv, self.d
        x = self.embed[tokens.long()]
        for layer, cache in zip(self.layers, self.caches):
            y = torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).bfloat16()
            heads = (y @ layer["qkv"]).view(n, hq + 2 * hkv, d)
            q = ds.cache_append(cache, heads[:, hq:hq + hkv], heads[:, hq + hkv:], row_off, kv_len, self.table,
                                rope=self.rope, k_weight=layer["kn"], q=heads[:, :hq], q_weight=layer["qn"],
                                status=self.status)["q"]
            y = ds.attend_paged(q, cache, row_off, kv_len, self.table, max_rows=max_rows, status=self.status)["out"]
            x = x + y.view(n, hq * d) @ layer["out"]
        return (torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).bfloat16() @ self.head).float()


class Decoder:
    """Texts that grow by verified steps.  State: every request's tokens (`text`, the last of them not yet in the
    cache) and how many there are."""

    def __init__(self, target, prompts, room=256, penalties=(1.2, 0.4, 0.2), seed=1):
        B = target.B
        self.t, self.seed = target, seed
        self.text = torch.zeros(B, room, dtype=torch.int32, device="cuda")
        self.length = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        for r, p in enumerate(prompts):
            self.text[r, :len(p)] = torch.tensor(p, dtype=torch.int32)
        self.prompt = self.length.clone()
        self.rep, self.pre, self.fre = (torch.full((B,), x, device="cuda") for x in penalties)
        off = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        off[1:] = (self.length - 1).cumsum(0)
        if off[-1]:                                    # the prompts but for their last tokens
            most = max(len(p) for p in prompts)
            flat = self.text[:, :most][torch.arange(most, device="cuda") < (self.length - 1)[:, None]]
            target.rows(flat, off, self.length - 1, most)

    def allowed(self, rows_req, rows_j, drafts):
        """The grammar: a row's token differs from the one before it in its last bit."""
        last = self.text.gather(1, (self.length - 1)[:, None].long())[:, 0]
        before = torch.cat((last[:, None], drafts), 1)[rows_req, rows_j]
        odd, even = torch.tensor(0xAAAAAAAA - 2 ** 32, device="cuda"), torch.tensor(0x55555555, device="cuda")
        word = torch.where(before % 2 == 0, odd, even).to(torch.int32)
        return word[:, None].expand(-1, (self.t.V + 31) // 32).contiguous()

    def logits(self, drafts, ell, row_off, K):
        """Penalised and masked logits of the ragged rows: the last token of each text and its first ell drafts."""
        t = self.t
        rows = int(row_off[-1])
        req = torch.searchsorted(row_off[1:], torch.arange(rows, device="cuda", dtype=torch.int32), right=True)
        j = torch.arange(rows, device="cuda") - row_off[req]
        last = self.text.gather(1, (self.length - 1)[:, None].long())
        tokens = torch.cat((last, drafts), 1)[req, j]
        z = t.rows(tokens, row_off, self.length + ell, K + 1)
        return ds.penalize_logits(z, row_off, self.text, self.length, self.prompt, self.rep, self.pre, self.fre,
                                  draft_tok=drafts, mask=self.allowed(req, j, drafts), status=t.status,
                                  out=dict(logits=z))["logits"]

    def take(self, tokens, counts):
        place = torch.arange(tokens.shape[1], device="cuda")
        new = place < counts[:, None]
        r = torch.arange(self.t.B, device="cuda")[:, None].expand_as(new)
        self.text[r[new], (self.length[:, None] + place)[new].long()] = tokens[new]
        self.length += counts

    def step(self, draft, K, temperature):
        """One speculative step; draft: base logits, factors and confidences of the draft model."""
        t = self.t
        temp = torch.full((t.B,), temperature, device="cuda")
        K_r = torch.full((t.B,), K, dtype=torch.int32, device="cuda")
        anchor = self.text.gather(1, (self.length - 1)[:, None].long())[:, 0].contiguous()
        self.seed += 1
        d = ds.draft_markov_sample(draft["U"], draft["E"], draft["W"], anchor, K_r, temp, self.seed, status=t.status)
        s = ds.schedule_survival(draft["conf"], K_r, draft["sps"], status=t.status)
        z = self.logits(d["draft_tok"], s["ell"], s["tgt_off"], K)
        v = ds.verify_ragged(d["draft_logits"], z, s["tgt_off"], s["ell"], d["draft_tok"], temp, self.seed + 1000,
                             draft_lse=d["draft_lse"], status=t.status)
        counts = v["n_acc"] + 1
        self.take(v["out_tok"], counts)
        return v["n_acc"], s["ell"]

    def plain_step(self):
        """One greedy token of each request, without speculation."""
        t = self.t
        none = torch.zeros(t.B, 1, dtype=torch.int32, device="cuda")
        off = torch.arange(t.B + 1, dtype=torch.int32, device="cuda")
        z = self.logits(none, torch.zeros_like(self.length), off, 0)
        self.take(z.argmax(-1, keepdim=True).to(torch.int32), torch.ones_like(self.length))


def draft_model(B, K, V, rank=16, seed=5):
    """Random drafts of fair confidence (float32: the small vocabulary runs on the CUDA cores)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    steps = torch.arange(B * (K + 1) + 1, dtype=torch.float64, device="cuda")
    return dict(U=r(B, K, V) * 2, E=r(V, rank) * 0.3, W=r(rank, V) * 0.3, conf=torch.sigmoid(r(B, K) + 1.5),
                sps=1.0 / (1.0 + steps / 64))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--bits", type=int, default=4, choices=(4, 8))
    a = ap.parse_args()
    B, K = 6, 4
    t = Target(B, bits=a.bits)
    dec = Decoder(t, [[7 + r, 11, 3 * r] + list(range(r)) for r in range(B)])
    for i in range(a.steps):
        n, ell = dec.step(draft_model(B, K, t.V, seed=5 + i), K, a.temperature)
        print(f"step {i}: verified {ell.tolist()}, accepted {n.tolist()}")
    for r in range(B):
        print(f"request {r}: {dec.text[r, :dec.length[r]].tolist()}")
    print(ds.check(t.status))


if __name__ == "__main__":
    main()
