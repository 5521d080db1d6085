"""The 8-bit pool, block mass and eviction on the GPU where ordinary calls do not go: walks that end early, values at
the ends of their ranges, many requests."""
import numpy as np
import pytest
import torch

from position_agnostic_paged_b200 import lazy_attn as la
from tests._q8_cases import U_F16, PoolCase, check

pytestmark = pytest.mark.gpu

PREFILL_U = dict(u_qk=4 * U_F16, u_p=U_F16)


# ------------------------------------------------------------------------------------------ prefill
@pytest.mark.parametrize("tokens", [6, 70])
@pytest.mark.parametrize("segs", [[(0, 0)], [(1, 0)], [(2, 0), (2, 200)], [(2, 0), (3, 200)], [(2, 0)]])
def test_prefill_of_short_walks(segs, tokens):
    """One and two tiles of up to 8 words per CTA (9 and 16 words at one offset, two offsets): the walk's end comes
    while the first tiles' keys are still unread.  One and two row tiles, many CTAs at once, the same bits every time."""
    reqs = [(segs, 300 + r % 3, tokens) for r in range(40)]
    c = PoolCase(la.Cfg(8, 2), [129, 256, 100, 16], reqs, seed=len(segs) + tokens).to()
    out = c.prefill()
    assert c.dev["status"].item() == 0
    few = PoolCase(la.Cfg(8, 2), [129, 256, 100, 16], reqs[:2], seed=len(segs) + tokens)
    few.q = c.q[:2 * tokens]
    check(out[:2 * tokens], *few.reference(**PREFILL_U)[:2], f"prefill of {tokens} tokens over {len(segs)} short walks")
    for _ in range(20):
        assert torch.equal(c.prefill(), out)
    assert c.dev["status"].item() == 0
