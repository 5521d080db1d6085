"""What the binding of the 8-bit pool, block mass and eviction calls refuses before anything is launched."""
import os
import subprocess
import sys

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


def _calls(ws, status):
    """Every call with arguments that pass all other checks but the last, that the tensors are on a GPU."""
    cfg, pool = la.Cfg(8, 2), la.Q8Pool.empty(4, 2, device="cpu")
    i = lambda *a: torch.tensor(a, dtype=torch.int32)                                    # noqa: E731
    q, x, f = torch.zeros(1, 8, 128).bfloat16(), torch.zeros(1, 2, 128).bfloat16(), torch.zeros(2)
    kv = torch.zeros(4, 2, 16, 128).bfloat16()
    return dict(
        write=lambda: la.kv_write_q8(cfg, x, x, i(0), i(0), pool, ws, status),
        decode=lambda: la.decode_attn_q8(cfg, q, i(0), i(0, 1), i(0, 2), 2, pool, q, ws, None, status),
        mass=lambda: la.decode_attn_mass(cfg, q, i(0), i(0, 1), i(0, 2), 2, pool.blk_meta, kv, kv, q, f, ws, status),
        prefill=lambda: la.prefill_attn_q8(cfg, q, i(0, 1), i(0), 1, i(0, 1), i(0, 2), 2, pool, q, ws, status),
        evict=lambda: la.evict_blocks(i(0, 1), i(0, 2), 2, f, i(1), 0, 0, i(0, 0), i(0, 0), f.clone(), None, status))


@pytest.mark.parametrize("call", ["write", "decode", "mass", "prefill", "evict"])
def test_workspace_and_status_are_what_they_seem(call):
    good, status = torch.empty(1 << 20, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        _calls(good, status)[call]()
    if call != "evict":
        for ws in (torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty(1 << 12, dtype=torch.uint8)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                _calls(ws, status)[call]()
    for st in (torch.zeros(1, dtype=torch.int64), torch.zeros(1, dtype=torch.uint8), torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError, match="d_status"):
            _calls(good, st)[call]()


def test_a_short_frequency_table_is_refused():
    """The library reads 64 of them."""
    for n in (0, 1, 63):
        cfg = la.Cfg(8, 2, rope_theta=(0.1,) * n)
        for call in (cfg.c, lambda: la.decode_q8_workspace_bytes(cfg, 1, 1), lambda: la.decode_workspace_bytes(cfg, 1, 1)):
            with pytest.raises(ValueError):
                call()
    assert la.decode_q8_workspace_bytes(la.Cfg(8, 2, rope_theta=(0.1,) * 64), 1, 1) > 0


def test_codec_tables_and_cache_need_no_torch():
    """A host program without torch: table words, position tables, workspace sizes, the block cache and its simulation."""
    code = """
import sys
sys.modules["torch"] = None          # import torch raises ImportError
import numpy as np
from position_agnostic_paged_b200 import cache_sim, lazy_attn as la, rope
assert la.pack_words(np.array([3]), np.array([16])).tolist() == [16 << 17 | 3]
assert len(rope.llama31_theta()) == 64 and rope.alibi_slopes(8)[0] == 0.5
assert la.decode_q8_workspace_bytes(la.Cfg(8, 2), 2, 4) > 0 and la.decode_noalloc_capacity() > 0
cache = la.BlockCache(8)
assert cache.access(1, 3)[0] is False and cache.access(1, 3)[0] is True
assert cache_sim.simulate("agnostic", [16, 16], [[0, 1], [1, 0]], 4)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
