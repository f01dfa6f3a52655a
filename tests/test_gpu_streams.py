"""Calls of the draft, the schedulers and the verification on a stream of their own (``stream=``) while the current one
is busy: what a call allocates and the fill of its status word must follow the given stream's order."""
import pytest
import torch

import speculative_decoding_draft_gb300 as ds
from speculative_decoding_draft_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def calls():
    """name -> (call(**kw), the outputs that are compared), on one small step in fp32.  Of the drafts the first position
    is compared, which every request has."""
    cfg = wl.small_config(name="tiny", B=5, K_max=4, V=1003, rank=7)
    g = {k: v.to(DEV) for k, v in wl.draft_inputs(cfg, "cpu").items()}
    h = {k: v.to(DEV) for k, v in wl.rnn_head(cfg, "cpu").items()}
    B, K = cfg.B, cfg.K_max
    head, req = (g["U"], g["E"], g["W"]), (g["anchor"], g["K_r"], g["temperature"], 3)
    conf, sps = wl.confidences(cfg, "cpu").to(DEV), torch.ones(B * (K + 1) + 2, dtype=torch.float64, device=DEV)
    cap = torch.full((1,), 7, dtype=torch.int32, device=DEV)
    d, s = ds.draft_markov_sample(*head, *req), ds.schedule_survival(conf, g["K_r"], sps)
    flat, _ = wl.flatten_targets(wl.target_dense(cfg, g["U"], g["K_r"]), s["ell"])
    ragged = (s["tgt_off"], s["ell"], d["draft_tok"], g["temperature"], 5)
    W = torch.randn(64, 1032, device=DEV).bfloat16()

    def first(r):
        return dict(tok=r["draft_tok"][:, 0], lse=r["draft_lse"][:, 0], status=r["status"])

    def recomputing():                                      # bf16 only
        cfg = wl.small_config(name="qwen", B=33, K_max=3, V=1032)
        g = {k: v.to(DEV) for k, v in wl.draft_inputs(cfg, "cpu").items()}
        W, req = ds.pack_projection(g["W"]), (g["anchor"], g["K_r"], g["temperature"], 3)
        d = ds.draft_markov_sample(g["U"], g["E"], W, *req, want_logits=False)
        s = ds.schedule_survival(wl.confidences(cfg, "cpu").to(DEV), g["K_r"],
                                 torch.ones(cfg.B * (cfg.K_max + 1) + 2, dtype=torch.float64, device=DEV))
        flat, _ = wl.flatten_targets(wl.target_dense(cfg, g["U"], g["K_r"]), s["ell"])
        return lambda **kw: ds.verify_markov(g["U"], g["E"], W, g["anchor"], d["draft_lse"], d["draft_tok_logit"], flat,
                                             s["tgt_off"], s["ell"], d["draft_tok"], g["temperature"], 5, **kw)

    return {
        "draft_markov_sample": (lambda **kw: first(ds.draft_markov_sample(*head, *req, **kw)), ("tok", "lse")),
        "draft_rnn_sample": (lambda **kw: first(ds.draft_rnn_sample(*head, h["rnn_W"], h["rnn_x"], *req, **kw)),
                             ("tok", "lse")),
        "schedule_survival": (lambda **kw: ds.schedule_survival(conf, g["K_r"], sps, **kw),
                              ("ell", "tgt_off", "theta_best", "b_star")),
        "schedule_capacity": (lambda **kw: ds.schedule_capacity(conf, g["K_r"], sps, **kw),
                              ("capacity", "theta_best", "ell", "tgt_off")),
        "schedule_topk": (lambda **kw: ds.schedule_topk(conf, g["K_r"], cap, **kw), ("ell", "tgt_off")),
        "schedule_threshold": (lambda **kw: ds.schedule_threshold(conf, g["K_r"], 0.5, **kw), ("ell", "tgt_off")),
        "verify_ragged": (lambda **kw: ds.verify_ragged(d["draft_logits"], flat, *ragged, draft_lse=d["draft_lse"], **kw),
                          ("n_acc",)),
        "verify_markov": (recomputing(), ("n_acc",)),
        "pack_projection": (lambda **kw: vars(ds.pack_projection(W, **kw)), ("data",)),
    }


@pytest.mark.parametrize("name", ["draft_markov_sample", "draft_rnn_sample", "schedule_survival", "schedule_capacity",
                                  "schedule_topk", "schedule_threshold", "verify_ragged", "verify_markov"])
def test_the_status_word_is_cleared_on_the_stream_of_the_call(calls, name):
    call, outputs = calls[name]
    want = call()
    assert ds.check(want["status"]) == "DSPARK_OK"
    words = [torch.full((1,), 8, dtype=torch.int32, device=DEV) for _ in range(256)]   # freed words that hold an error
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    del words[::2]
    torch.cuda._sleep(200_000_000)                          # a tenth of a second that the current stream has to do
    got = call(stream=side)
    with torch.cuda.stream(side):
        kept = {h: got[h].clone() for h in outputs}
    assert ds.check(got["status"], stream=side) == "DSPARK_OK"
    side.synchronize()
    assert all(torch.equal(kept[h], want[h]) for h in outputs)


@pytest.mark.parametrize("name", ["verify_ragged", "schedule_survival", "pack_projection"])
def test_a_stream_may_be_a_handle(calls, name):
    call, outputs = calls[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side.cuda_stream, 0, torch.cuda.default_stream()):
        got = call(stream=handle)
        torch.cuda.synchronize()
        assert all(torch.equal(got[h], want[h]) for h in outputs)
