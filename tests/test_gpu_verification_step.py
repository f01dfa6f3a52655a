"""The operators together, in the example's decoder: greedy speculation has to emit what plain greedy decoding
emits, token by token, whatever the drafts."""
import os
import sys

import pytest
import torch

import speculative_decoding_draft_gb300 as ds

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from speculative_decoding_draft_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import verification_step
    finally:
        sys.path.pop(0)
    return verification_step


def prompts(B):
    return [[7 + r, 11, 3 * r] + list(range(r)) for r in range(B)]


def test_greedy_speculation_is_greedy_decoding(example):
    B, K, steps = 6, 4, 10
    plain = example.Decoder(example.Target(B), prompts(B))
    for _ in range(steps * (K + 1)):
        plain.plain_step()
    assert ds.check(plain.t.status) == "DSPARK_OK"
    spec = example.Decoder(example.Target(B), prompts(B))
    accepted = 0
    for i in range(steps):
        draft = example.draft_model(B, K, spec.t.V, seed=50 + i)
        # half of the drafts are what the model would say next, so that steps accept and reject
        for r in range(0, B, 2):
            at = int(spec.length[r])
            for k in range(K if (i + r) % 3 else 2):
                draft["U"][r, k, plain.text[r, at + k]] += 100.0
        n, ell = spec.step(draft, K, 0.0)
        assert (n <= ell).all()
        accepted += int(n.sum())
    assert ds.check(spec.t.status) == "DSPARK_OK"
    assert accepted > steps                               # otherwise nothing was speculated
    for r in range(B):
        m = int(spec.length[r])
        assert spec.text[r, :m].tolist() == plain.text[r, :m].tolist()
        out = spec.text[r, int(spec.prompt[r]) - 1:m]     # the grammar holds along every emitted token
        assert ((out[1:] + out[:-1]) % 2 == 1).all()


def test_sampled_steps_keep_the_grammar(example):
    B, K = 5, 3
    dec = example.Decoder(example.Target(B), prompts(B))
    for i in range(6):
        dec.step(example.draft_model(B, K, dec.t.V, seed=9 + i), K, 1.0)
    assert ds.check(dec.t.status) == "DSPARK_OK"
    for r in range(B):
        out = dec.text[r, int(dec.prompt[r]) - 1:int(dec.length[r])]
        assert len(out) > 6 and ((out[1:] + out[:-1]) % 2 == 1).all()
        assert (out >= 0).all() and (out < dec.t.V).all()
