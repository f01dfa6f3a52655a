"""The operators around a ragged verification step where they once went wrong: norm weights off their boundary."""
import math

import pytest
import torch

import speculative_decoding_draft_gb300 as ds
from test_gpu_serving import DTYPES, E2M1, attend_check, built, filled, gen, i32, offsets, ok, paged, randn  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------------------------------
# what 4 bits keep
# ---------------------------------------------------------------------------------------------------------------
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
