"""The 8-bit pool, block mass and eviction on the GPU where ordinary calls do not go: walks that end early, values at
the ends of their ranges, many requests."""
import numpy as np
import pytest
import torch

from position_agnostic_paged_b200 import lazy_attn as la
from tests._q8_cases import BLK, D, U_BF16, U_F16, PoolCase, bf16, check, write_reference
from tests.test_gpu_q8 import _check_evict, _device_pool, _same_pool, _state, _write

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


# ------------------------------------------------------------------------------- scales far from 1
def _attend_all(c, what, u=None):
    """Decode with and without block mass, and prefill (the decode's kernel for up to 16 rows, the prefill's above)."""
    ref, bound, mref, mbound = c.reference(**(u or {}))
    c.to()
    check(c.decode(), ref, bound, f"decode {what}", rel=np.inf)
    m = torch.zeros(c.words.size, device="cuda")
    check(c.decode(m), ref, bound, f"decode with mass {what}", rel=np.inf)
    check(m, mref, mbound, f"mass {what}", rel=np.inf)
    check(c.prefill(), *c.reference(**(u or PREFILL_U))[:2], f"prefill {what}", rel=np.inf)
    assert c.dev["status"].item() == 0


@pytest.mark.parametrize("hq", [2, 8, 10, 40])
@pytest.mark.parametrize("v_exp", [(119, 126), (-126 + 6, 126), (110, 126)])
def test_largest_value_scales(v_exp, hq):
    """V scales up to 2^119, the largest that a write makes of bf16 values, beside each other and beside the smallest."""
    reqs = [([(0, 0), (1, 100)], 150, 1), ([(2, 0)], 40, 1), ([(1, 0), (0, 60)], 159, 1)]
    _attend_all(PoolCase(la.Cfg(hq, 2), [100, 60, 33], reqs, seed=hq, v_exp=v_exp), f"V scales 2^{v_exp}, {hq} heads")


@pytest.mark.parametrize("hq", [4, 20])
def test_value_scales_at_the_end_of_a_float(hq):
    """Scales of 2^127 and 1.5 x 2^127 times codes of at most 1: values that bf16 holds."""
    c = PoolCase(la.Cfg(hq, 1), [40, 40], [([(0, 0), (1, 40)], 79, 1), ([(1, 0)], 20, 1)], seed=1)
    rng = np.random.default_rng(0)
    one = np.array([0x38, 0x30, 0xB8, 0x00], np.uint8)                        # 1, 0.5, -1, 0
    live = (np.arange(16) < (c.meta & 255)[:, None])[:, None, :, None]
    c.v_codes = np.where(live, one[rng.integers(0, 4, c.v_codes.shape)], c.v_codes)
    c.v_scale[:] = 2.0 ** 127
    c.v_scale[c.doc_blocks[1]] = 1.5 * 2.0 ** 127
    _attend_all(c, f"V scales 2^127, {hq} heads")


@pytest.mark.parametrize("order", [0, 1])
@pytest.mark.parametrize("hq,n", [(4, 1), (4, 4), (8, 2), (16, 1), (16, 20)])
def test_small_weight_times_large_values(hq, n, order):
    """A block whose weights are about 2^-130, below the smallest float, with values about 2^127: it
    contributes like the near blocks of ordinary values.  Scores come from ALiBi alone (a query of zeros)."""
    slope, far = 0.05, 1800                                                   # 0.05 x 1800 x log2 e = 130
    segs = [[(0, 0), (1, far)], [(1, far), (0, 0)]][order]
    c = PoolCase(la.Cfg(hq, 1, alibi_slopes=(slope,) * hq), [16, 32], [(segs, far + 40, n), ([(1, 0)], 31, 1)], seed=2, k_exp=(0, 1))
    c.v_scale[c.doc_blocks[0]] = 2.0 ** 119
    c.v_scale[c.doc_blocks[1]] = 2.0 ** -5
    c.q.zero_()
    ref, _, mref, mbound = c.reference()
    codes, c.v_codes = c.v_codes, c.v_codes & 0x7F
    total = c.reference()[0]                                                  # sum of weight times |value|
    c.v_codes = codes
    # The scores have no error but the bias's rounding to float (2^-16 of the largest is taken for it), the weights
    # 2^-11 as f16 (parts of e4m3: less) and 2^-14 for their exponents, sums of numbers up to 256 in fp32, and
    # for what underflows f16 (48 keys x 2^-24 of the largest product); the output is rounded to bf16.
    bound = 1.02 * ((np.expm1(2 * slope * (far + 60) * 2.0 ** -16) + U_F16 + 2.0 ** -14) * total + U_BF16 * np.abs(ref))
    assert np.abs(ref[:n]).mean() > 20 * bound[:n].mean()
    c.to()
    what = f"far values of 2^127, {hq} heads"
    if n == 1:
        check(c.decode(), ref, bound, f"decode {what}", rel=np.inf)
        m = torch.zeros(c.words.size, device="cuda")
        check(c.decode(m), ref, bound, f"decode with mass {what}", rel=np.inf)
        check(m, mref, mbound, f"mass {what}", rel=np.inf)
    check(c.prefill(), ref, bound, f"prefill of {n} tokens, {what}", rel=np.inf)
    assert c.dev["status"].item() == 0


# -------------------------------------------------------------------------------------------- write
@pytest.mark.parametrize("n", [12, 1300])
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), float("-inf")])
def test_write_beside_nan_and_infinity(odd, n):
    """A NaN or infinite value where the block's old scale is no power of two: its partner 64 dims away, like every
    other element, is stored as it is alone."""
    rng = np.random.default_rng(n)
    nb = n // BLK + 2
    st = _state(nb, 2, 4, [6] + [3] * (nb - 1))
    for b in range(1, nb):
        st["meta"][b] = b << 8 | 3
    st["k_scale"], st["v_scale"] = st["k_scale"] * np.float32(1.37), st["v_scale"] * np.float32(0.77)
    j = 6 + np.arange(n)
    k, v = bf16(rng.standard_normal((n, 2, D)) * 0.05), bf16(rng.standard_normal((n, 2, D)) * 0.05)
    v[np.arange(n), :, np.arange(n) * 7 % D] = odd
    cfg = la.Cfg(2, 2)
    pool = _device_pool(st)
    assert _write(cfg, pool, k, v, j, j) == 0
    _same_pool(pool, write_reference(cfg, st, k, v, j, j))


# ------------------------------------------------------------------------------ queries that are not finite
@pytest.mark.parametrize("odd", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("q8,n", [(True, 1), (True, 4), (True, 5), (True, 40), (False, 1)])
def test_query_with_an_infinite_element(q8, n, odd):
    """A head whose query has an infinite or NaN element has NaN as output if it sees a key, and no other does."""
    reqs = [([(0, 0), (1, 60)], 100, n), ([(1, 0)], 20, n), ([(2, 7)], 7, n), ([(2, 500)], 400, n)]
    c = PoolCase(la.Cfg(8, 2), [60, 50, 1], reqs, seed=3, q8=q8)
    u = dict(u_qk=2.0 ** -22, u_p=U_BF16) if not q8 else PREFILL_U if n > 1 else {}
    ref, bound, mref, mbound = c.reference(**u)
    # the last sees nothing, the third one key (with which half of all infinite scores are -infinity)
    seen = [(0, 3), (2 * n - 1, 0)] + [(3 * n - 1, h) for h in range(8)]
    for row, h in seen + [(3 * n, 1)]:
        c.q[row, h, 5 + h] = odd
    c.to()
    outs = [c.prefill()] if n > 1 else [c.decode(torch.zeros(c.words.size, device="cuda"))] + ([c.decode()] if q8 else [])
    for out in outs:
        assert out[[r for r, _ in seen], [h for _, h in seen]].isnan().all()
        out, want, b = out.clone(), ref.copy(), bound.copy()
        for row, h in seen:
            out[row, h], want[row, h] = 0.0, 0.0
        check(out, want, b, f"rows beside one with {odd}")
        assert (out[3 * n:] == 0).all()


# Pairs (dim i, position, a, b) whose rotated key a cos - b sin lies within half an fp32 ulp of a border between two codes
# (at base 500000 and scale 1), but not on it
NEAR_BORDERS = [
    (16, 43762, 1.5234375, 0.45703125), (11, 7729, 1.421875, -0.169921875), (6, 14393, 1.4140625, -0.259765625),
    (18, 3240, 1.3046875, 0.2421875), (23, 36115, 1.0703125, 0.1181640625), (17, 47531, 1.7890625, 1.2578125),
    (16, 25219, 1.5859375, 0.578125), (13, 28760, 1.7421875, -0.23828125), (2, 52631, 1.40625, -1.203125),
    (5, 18802, 1.4140625, 1.078125), (2, 12948, 1.21875, -1.8046875), (10, 33080, 1.15625, -0.330078125),
    (22, 28053, 1.0, -0.365234375), (4, 46713, 1.546875, 0.70703125), (13, 35991, 1.5703125, -1.234375),
    (8, 44164, 1.6328125, -0.1787109375), (1, 33282, 1.0546875, -0.130859375), (12, 20225, 1.859375, 0.2490234375)]


@pytest.mark.parametrize("n", [len(NEAR_BORDERS), 1200])
def test_write_keys_next_to_a_border(n):
    """The quotient is rounded to fp32 before it is rounded to a code: in these keys that decides."""
    rng = np.random.default_rng(n)
    k = bf16(rng.standard_normal((n, 1, D)))
    j = rng.integers(0, 60000, n)
    for t, (i, pos, a, b) in enumerate(NEAR_BORDERS):
        k[t, 0, i], k[t, 0, i + 64], j[t] = a, b, pos
    k[:, 0, 63], k[:, 0, 127] = 300.0, 0.0                         # the scale is 1
    slot = np.arange(n) * BLK + j % BLK                            # a block each
    cfg, st = la.Cfg(1, 1), _state(n, 1, 1, [0] * n)
    pool = _device_pool(st)
    assert _write(cfg, pool, k, k, slot, j) == 0
    want = write_reference(cfg, st, k, k, slot, j)
    assert (want["k_scale"] == 1).all()
    _same_pool(pool, want)


@pytest.mark.parametrize("n", [200, 1300])
def test_write_subnormal_keys(n):
    """Keys of a few times 2^-133, whose products with cos and sin are rounded below fp32's normal range."""
    rng = np.random.default_rng(n)
    k = bf16(rng.integers(-20, 21, (n, 4, D)) * 2.0 ** -133)
    assert float(k.abs().max()) == 20 * 2.0 ** -133
    cfg, nb = la.Cfg(4, 4), n // BLK + 1
    st = _state(nb, 4, 1, [0] * nb)
    j = np.arange(n)
    pool = _device_pool(st)
    assert _write(cfg, pool, k, k, j, j) == 0
    _same_pool(pool, write_reference(cfg, st, k, k, j, j))


@pytest.mark.parametrize("hkv,n,order", [(3, 1500, "asc"), (5, 1025, "shuffle"), (8, 1500, "asc"), (8, 1500, "shuffle"),
                                         (11, 1100, "asc"), (11, 1100, "shuffle"), (64, 1025, "asc")])
def test_large_write_of_many_heads(hkv, n, order):
    """More than four heads: a warp takes several, its staging buffers again and their phases on; from slot 5 of a
    partly filled block on, the last block partly filled, some tokens skipped."""
    rng = np.random.default_rng([n, hkv])
    nb = (n + 5) // BLK + 3
    st = _state(nb, hkv, n, [16] + [5] + [0] * (nb - 2))
    j = BLK + 5 + np.arange(n)
    slot = j.copy()
    slot[40:44] = -1
    slot[70], j[70] = slot[75], j[75]
    if order == "shuffle":
        p = rng.permutation(n)
        j, slot = j[p], slot[p]
    k, v = bf16(rng.standard_normal((n, hkv, D)) * 2), bf16(rng.standard_normal((n, hkv, D)) * 2.0 ** rng.integers(-9, 3, (n, hkv, 1)))
    cfg = la.Cfg(hkv, hkv)
    pool = _device_pool(st)
    assert _write(cfg, pool, k, v, slot, j) == la.DSTATUS_BAD_SLOT
    _same_pool(pool, write_reference(cfg, st, k, v, slot, j))


# -------------------------------------------------------------------------------------------- evict
@pytest.mark.parametrize("reqs", [2048, 2049, 8193, 20000])
def test_evict_of_thousands_of_requests(reqs):
    """On both sides of the number from which a kernel of its own writes the row pointers, and of its CTAs' shares."""
    rng = np.random.default_rng(reqs)
    n = rng.integers(0, 7, reqs)
    ind = np.concatenate([[3], 3 + np.cumsum(n)])
    total = int(ind[-1]) + 2
    assert _check_evict(rng.integers(0, 1 << 32, total, dtype=np.uint32), ind, 5, rng.random(total).astype(np.float32),
                        rng.integers(-1, 8, reqs), 1, 1) == la.DSTATUS_BAD_TABLE


def test_evict_of_the_most_requests():
    """2^20 requests of no or one word: right, and not in time that grows with their square."""
    reqs = 1 << 20
    rng = np.random.default_rng(7)
    n, keep = rng.integers(0, 2, reqs), rng.integers(0, 2, reqs)
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(np.asarray(a, dt))).cuda()      # noqa: E731
    ind = np.concatenate([[0], np.cumsum(n)])
    total = int(ind[-1])
    table, mass = t(np.arange(total), np.int32), t(rng.random(total), np.float32)
    out, gone, mo = torch.full_like(table, -1), torch.full_like(table, -1), torch.zeros_like(mass)
    io, first = torch.full((reqs + 1,), -1, dtype=torch.int32, device="cuda"), t(ind, np.int32)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    kd = t(keep, np.int32)
    a.record()
    la.evict_blocks(table, first, 1, mass, kd, 0, 0, out, io, mo, gone)
    b.record()
    torch.cuda.synchronize()
    stays = (n * keep)[n > 0] > 0                                  # of each word
    assert np.array_equal(io.cpu().numpy(), np.concatenate([[0], np.cumsum(n * keep)]))
    k = int(stays.sum())
    assert np.array_equal(out[:k].cpu().numpy(), np.nonzero(stays)[0]) and (out[k:] == -1).all()
    assert np.array_equal(gone[:total - k].cpu().numpy(), np.nonzero(~stays)[0]) and (gone[total - k:] == -1).all()
    assert torch.equal(mo[:k], mass[torch.from_numpy(stays).cuda()])
    assert a.elapsed_time(b) < 1000.0


# ---------------------------------------------------------------------------------------- positions
@pytest.mark.parametrize("kind", ["rope", "alibi"])
@pytest.mark.parametrize("hq,q8", [(8, True), (40, True), (8, False)])
def test_positions_at_the_ends_of_int(hq, q8, kind):
    """The largest int sees every key, the smallest and -1 (a padded row) none."""
    top, low = 2 ** 31 - 1, -2 ** 31
    cfg = la.Cfg(hq, 2) if kind == "rope" else la.Cfg(hq, 2, alibi_slopes=(0.0,) * hq)
    reqs = [([(0, 0), (1, 100)], p, 1) for p in (top, low, -1, top - 20)] + [([(1, 32767)], p, 1) for p in (low, top, -1)]
    c = PoolCase(cfg, [100, 37], reqs, seed=hq, q8=q8).to()
    u = {} if q8 else dict(u_qk=2.0 ** -22, u_p=U_BF16)
    ref, bound, mref, mbound = c.reference(**u)
    assert (np.abs(ref).max((1, 2)) > 0).tolist() == [True, False, False, True, False, True, False]
    m = torch.zeros(c.words.size, device="cuda")
    check(c.decode(m), ref, bound, f"decode at the last position, {hq} heads {kind} q8={q8}")
    check(m, mref, mbound, f"mass at the last position, {hq} heads {kind} q8={q8}")
    if q8:
        check(c.decode(), ref, bound, f"decode at the last position, {hq} heads {kind}")
        check(c.prefill(), *c.reference(**PREFILL_U)[:2], f"prefill at the last position, {hq} heads {kind}")
    assert c.dev["status"].item() == 0


# ---------------------------------------------------------------------------------------- precision
@pytest.mark.parametrize("hq,hkv", [(8, 8), (32, 8), (32, 1), (25, 1)])
def test_block_mass_decode_keeps_its_weights(hq, hkv):
    """The bf16 pool's decode with block mass: weights as two bf16 parts (2^-16), so that the output's rounding is what
    is left also where large values cancel."""
    docs = [100, 333, 48, 5]
    reqs = [([(0, 0), (1, 100), (2, 433)], 480, 1), ([(3, 0)], 4, 1), ([(1, 0), (1, 333)], 500, 1), ([(2, 7)], 30, 1)]
    c = PoolCase(la.Cfg(hq, hkv), docs, reqs, seed=hq, q8=False).to()
    ref, bound, mref, mbound = c.reference(u_qk=2.0 ** -22, u_p=2.0 ** -16)
    m = torch.zeros(c.words.size, device="cuda")
    check(c.decode(m), ref, bound, f"decode with mass, weights in two parts, {hq}/{hkv}")
    check(m, mref, mbound, f"mass {hq}/{hkv}")


# ----------------------------------------------------------------------------- what a call leaves alone
@pytest.mark.parametrize("blocks,max_words", [(0, 3), (2, 0)])
@pytest.mark.parametrize("most", [1, 40])
def test_prefill_without_keys_leaves_other_rows(blocks, max_words, most):
    """No blocks, or no words: zeros for the requests' rows, and nothing for the rows before and behind them."""
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")                      # noqa: E731
    q = torch.randn(100, 8, D, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 5.0)
    la.prefill_attn_q8(la.Cfg(8, 2), q, i(3, 4, 4, 4 + most), i(0, 0, 0), most, i(0, 0, 0), i(0, 0, 0, 0), max_words,
                       la.Q8Pool.empty(blocks, 2), out, None)
    assert (out[3:4 + most] == 0).all() and (out[:3] == 5).all() and (out[4 + most:] == 5).all()


@pytest.mark.parametrize("most", [3, 12, 200])
def test_prefill_of_requests_without_tokens(most):
    """Row pointers that give no request a token, for every size of max_q, and inputs overwritten right behind the call."""
    docs = [100]
    c = PoolCase(la.Cfg(8, 2), docs, [([(0, 0)], 90, 2), ([(0, 5)], 90, 2)], seed=1).to()
    d = c.dev
    out = torch.full_like(d["q"], 5.0)
    ws = c.ws(la.prefill_q8_workspace_bytes(c.cfg, 2, 4, most, c.max_words, c.words.size))
    for _ in range(50):
        cu = torch.full((3,), 2, dtype=torch.int32, device="cuda")
        la.prefill_attn_q8(c.cfg, d["q"], cu, d["pos0"], most, d["table"], d["indptr"], c.max_words, c.pool, out, ws, d["status"])
        cu.copy_(torch.tensor([0, 2, 4], dtype=torch.int32), non_blocking=True)
    assert (out == 5).all() and d["status"].item() == 0


def _guarded(n):
    """A workspace of exactly n bytes, and the bytes behind it (1 MiB, so that nothing can land outside)."""
    buf = torch.full((n + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    return buf[:n], buf[n:]


@pytest.mark.parametrize("reqs,doc,tokens", [(1, 2000, 1), (1, 2000, 4), (1, 2000, 300), (3, 700, 5), (40, 90, 12), (300, 20, 1), (5, 3, 2)])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 1), (5, 5)])
def test_workspaces_are_not_left(hq, hkv, reqs, doc, tokens):
    """Calls with exactly the workspace that they ask for write nothing behind it."""
    c = PoolCase(la.Cfg(hq, hkv), [doc, 37], [([(0, 0), (1, doc)], doc + 30, tokens)] * reqs, seed=doc).to()
    n, mw, d = reqs, c.max_words, c.dev
    guards = []
    if tokens == 1:
        for mass in (None, torch.zeros(c.words.size, device="cuda")):
            ws, g = _guarded(la.decode_q8_workspace_bytes(c.cfg, n, mw, mass is not None))
            c.decode(mass, ws=ws)
            guards.append(g)
        k = torch.randn(c.num_blocks, hkv, BLK, D, device="cuda").to(torch.bfloat16)
        ws, g = _guarded(la.decode_mass_workspace_bytes(c.cfg, n, mw))
        la.decode_attn_mass(c.cfg, d["q"], d["pos0"], d["table"], d["indptr"], mw, d["meta"], k, k, torch.empty_like(d["q"]),
                            mass, ws, d["status"])
        guards.append(g)
    ws, g = _guarded(la.prefill_q8_workspace_bytes(c.cfg, n, d["q"].shape[0], tokens, mw, c.words.size))
    c.prefill(ws=ws)
    guards.append(g)
    m = 1025 + doc
    ws, g = _guarded(la.kv_write_q8_workspace_bytes(c.cfg, m, m // BLK + 1))
    kv, at = torch.randn(m, hkv, D, device="cuda").to(torch.bfloat16), torch.arange(m, dtype=torch.int32, device="cuda")
    la.kv_write_q8(c.cfg, kv, kv, at, at, la.Q8Pool.empty(m // BLK + 1, hkv), ws, d["status"])
    guards.append(g)
    assert d["status"].item() == 0
    assert all((g == 0xA5).all() for g in guards)


@pytest.mark.parametrize("tokens", [2, 9, 70])
def test_prefill_of_requests_longer_than_max_words(tokens):
    """Words past max_words are ignored and reported, with few rows, one and two row tiles."""
    segs = [(0, 0), (1, 200)]
    c = PoolCase(la.Cfg(8, 2), [200, 150], [(segs, 349 - r, tokens) for r in range(3)], seed=tokens).to()
    d, mw = c.dev, 15                                              # of 13 + 10 words
    out = torch.full_like(d["q"], 7.0)
    ws = c.ws(la.prefill_q8_workspace_bytes(c.cfg, 3, out.shape[0], tokens, mw, c.words.size))
    la.prefill_attn_q8(c.cfg, d["q"], d["cu"], d["pos0"], tokens, d["table"], d["indptr"], mw, c.pool, out, ws, d["status"])
    assert d["status"].item() == la.DSTATUS_BAD_TABLE
    keep = np.concatenate([np.arange(i, i + mw) for i in c.indptr[:-1]])
    c.words, c.indptr = c.words[keep], [mw * r for r in range(4)]
    check(out, *c.reference(**PREFILL_U)[:2], f"prefill of {tokens} tokens, words past max_words")


@pytest.mark.parametrize("n", [30, 1200])
def test_write_of_a_call_that_contradicts_itself(n):
    """Tokens of one block with local indices from different blocks: each key is turned by its own, the metadata word is
    the largest."""
    rng = np.random.default_rng(n)
    nb = n // BLK + 2
    st = _state(nb, 3, n, [7] * nb)
    slot = rng.permutation(nb * BLK)[:n]
    j = slot % BLK + BLK * rng.integers(0, 2000, n)
    k, v = bf16(rng.standard_normal((n, 3, D))), bf16(rng.standard_normal((n, 3, D)))
    cfg = la.Cfg(3, 3)
    pool = _device_pool(st)
    assert _write(cfg, pool, k, v, slot, j) == 0
    _same_pool(pool, write_reference(cfg, st, k, v, slot, j))
