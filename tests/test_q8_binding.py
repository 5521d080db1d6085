"""What the binding of the 8-bit pool, block mass and eviction calls refuses before anything is launched."""
import pytest
import torch

from position_agnostic_paged_b200 import lazy_attn as la

MEMBERS = ("k_codes", "v_codes", "k_scale", "v_scale", "blk_meta")


@pytest.mark.parametrize("name", MEMBERS)
def test_pool_members_are_on_one_device(name):
    pool = la.Q8Pool.empty(4, 2, device="cpu")
    parts = {n: getattr(pool, n) for n in MEMBERS}
    la.Q8Pool(**parts)
    parts[name] = parts[name].to("meta")
    with pytest.raises(ValueError):
        la.Q8Pool(**parts)
