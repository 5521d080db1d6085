"""The 8-bit pool, block mass and eviction on the GPU against their values in 64 bits."""
import numpy as np
import pytest
import torch

from position_agnostic_paged_b200 import lazy_attn as la
from position_agnostic_paged_b200 import rope
from tests._q8_cases import (BLK, D, U_BF16, U_F16, PoolCase, bf16, check, evict_reference, la_pack, to_e4m3, write_reference)

pytestmark = pytest.mark.gpu

HEADS = [(8, 8), (32, 8), (6, 2), (40, 8), (16, 1), (22, 2), (32, 1), (25, 1)]
# the query rounded to f16; the key's cos and sin, one product and the sum
PREFILL_U = dict(u_qk=4 * U_F16, u_p=U_F16)


def _requests(n=5, seed=0):
    """Documents of one token to some hundred, shared by requests at several offsets, with gaps, a
    document twice in one request, a request without words and one whose query sees nothing."""
    docs = [1, 15, 16, 17, 100, 333, 48, 5]
    reqs = [([(4, 0), (5, 100), (3, 433), (0, 450)], 450, 1),
            ([(5, 0), (5, 333), (6, 700), (7, 748)], 752, 1),
            ([], 10, 1),
            ([(2, 0)], 0, 1),                      # sees one key
            ([(4, 500)], 499, 1),                  # sees none
            ([(1, 31000), (3, 32000)], 32016, 1),
            ([(4, 0), (5, 100)], 251, 1)]          # stops inside a block of a document
    return docs, (reqs * (n // len(reqs) + 1))[:n]


def _cfg(hq, hkv, kind="rope"):
    if kind == "alibi":
        return la.Cfg(hq, hkv, alibi_slopes=tuple(rope.alibi_slopes(hq)))
    if kind == "llama31":
        return la.Cfg(hq, hkv, rope_theta=tuple(rope.llama31_theta()))
    return la.Cfg(hq, hkv, softmax_scale=0.11 if kind == "scale" else 0.0)


# ------------------------------------------------------------------------------------------- decode
@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_decode(hq, hkv, q8, mass):
    if not q8 and not mass:
        pytest.skip("decode over the bf16 pool without block mass is lazy_decode_attn")
    docs, reqs = _requests(9)
    c = PoolCase(_cfg(hq, hkv), docs, reqs, seed=hq * 100 + hkv, q8=q8).to()
    u = dict() if q8 else dict(u_qk=2.0 ** -22, u_p=U_BF16)
    ref, bound, mref, mbound = c.reference(**u)
    start = torch.rand(c.words.size, device="cuda") * 4
    m = start.clone() if mass else None
    out = c.decode(m)
    assert c.dev["status"].item() == 0
    check(out, ref, bound, f"decode {'q8' if q8 else 'bf16'} {hq}/{hkv} mass={mass}")
    if mass:
        want = start.double().cpu().numpy() + mref
        check(m, want, mbound + 2.0 ** -24 * want, f"block mass {'q8' if q8 else 'bf16'} {hq}/{hkv}")
        m2, out2 = start.clone(), c.decode(m3 := start.clone())
        c.decode(m2)
        assert torch.equal(m2, m) and torch.equal(m3, m) and torch.equal(out2, out)   # the same bits every time


@pytest.mark.parametrize("kind", ["alibi", "llama31", "scale"])
@pytest.mark.parametrize("q8", [True, False])
def test_decode_variants(kind, q8):
    docs, reqs = _requests(7)
    c = PoolCase(_cfg(16, 4, kind), docs, reqs, seed=5, q8=q8).to()
    ref, bound, mref, mbound = c.reference(**({} if q8 else dict(u_qk=2.0 ** -22, u_p=U_BF16)))
    m = torch.zeros(c.words.size, device="cuda")
    check(c.decode(m), ref, bound, f"decode {kind} q8={q8}")
    check(m, mref, mbound, f"block mass {kind} q8={q8}")


@pytest.mark.parametrize("words", [1, 2, 3, 31, 32, 33, 64, 65, 259, 1000])
def test_decode_lengths(words):
    """One request over words - 1 full blocks and one of 5 tokens, for splits of every kind."""
    c = PoolCase(la.Cfg(8, 2), [16 * words - 11], [([(0, 3)], 16 * words, 1)], seed=words).to()
    ref, bound, mref, mbound = c.reference()
    m = torch.zeros(words, device="cuda")
    check(c.decode(), ref, bound, f"decode {words} words")
    check(c.decode(m), ref, bound, f"decode {words} words with mass")
    check(m, mref, mbound, f"mass {words} words")


def test_decode_many_short_requests():
    """More requests than the workspace has warps, most of one or no word."""
    docs = [3, 16, 30]
    reqs = [([(r % 3, 0)] if r % 4 else [], 40, 1) for r in range(700)]
    c = PoolCase(la.Cfg(8, 1), docs, reqs, seed=1).to()
    ref, bound, mref, mbound = c.reference()
    m = torch.zeros(c.words.size, device="cuda")
    check(c.decode(m), ref, bound, "decode 700 requests")
    check(m, mref, mbound, "mass 700 requests")


@pytest.mark.parametrize("k_exp,v_exp,q_scale", [((-120, -100), (-125, -90), 1.0), ((-10, 12), (-60, 60), 1.0),
                                                 ((90, 100), (100, 110), 2.0 ** -100), ((-100, -90), (0, 1), 2.0 ** 100)])
def test_decode_extreme_scales(k_exp, v_exp, q_scale):
    """Scales far from 1, within one request: no overflow, and small blocks keep their weight."""
    docs, reqs = _requests(7)
    for mass in (False, True):
        c = PoolCase(la.Cfg(8, 2, softmax_scale=1e-3 if k_exp[1] == 12 else 0.0), docs, reqs, seed=9, k_exp=k_exp,
                     v_exp=v_exp, q_scale=q_scale).to()
        ref, bound, mref, mbound = c.reference()
        m = torch.zeros(c.words.size, device="cuda") if mass else None
        check(c.decode(m), ref, bound, f"decode scales {k_exp} {v_exp}", rel=np.inf)
        if mass:
            check(m, mref, mbound, f"mass scales {k_exp} {v_exp}", rel=np.inf)


def test_decode_block_of_zeros():
    """A block whose values are all zero has the smallest scale; its softmax weight still counts."""
    c = PoolCase(la.Cfg(4, 1), [16, 16, 16], [([(0, 0), (1, 16), (2, 32)], 60, 1)], seed=3)
    b = c.doc_blocks[1][0]
    c.v_codes[b], c.v_scale[b] = 0, 2.0 ** -126
    c.k_codes[c.doc_blocks[2][0]], c.k_scale[c.doc_blocks[2][0]] = 0, 2.0 ** -126
    ref, bound, mref, mbound = c.reference()
    c.to()
    m = torch.zeros(3, device="cuda")
    check(c.decode(m), ref, bound, "decode zero block")
    check(m, mref, mbound, "mass zero block")
    check(c.prefill(), *c.reference(**PREFILL_U)[:2], "prefill zero block")


@pytest.mark.parametrize("q8", [True, False])
def test_decode_faults_are_reported(q8):
    docs, reqs = _requests(4)
    c = PoolCase(la.Cfg(8, 2), docs, reqs, seed=2, q8=q8)
    c.words[3] = la_pack(c.num_blocks + 5, 48)         # no such block: left out
    c.to()
    ref, bound, mref, mbound = c.reference(**({} if q8 else dict(u_qk=2.0 ** -22, u_p=U_BF16)))
    m = torch.zeros(c.words.size, device="cuda")
    check(c.decode(m), ref, bound, "decode with a bad block")
    check(m, mref, mbound, "mass with a bad block")
    assert c.dev["status"].item() == la.DSTATUS_BAD_BLOCK
    c.dev["status"].zero_()
    m.zero_()
    c.decode(m, max_words=c.max_words - 1)             # the longest request has one word too many
    assert c.dev["status"].item() == la.DSTATUS_BAD_BLOCK | la.DSTATUS_BAD_TABLE
    last = [c.indptr[r + 1] - 1 for r in range(4) if c.indptr[r + 1] - c.indptr[r] == c.max_words]
    assert all(m[i].item() == 0.0 for i in last)


@pytest.mark.parametrize("q8", [True, False])
def test_decode_table_slice_and_untouched_rows(q8):
    """Requests 2 .. 4 of a larger table, through row pointers that do not start at 0."""
    docs, reqs = _requests(6)
    c = PoolCase(la.Cfg(8, 2), docs, reqs, seed=4, q8=q8).to()
    ref, bound, mref, mbound = c.reference(**({} if q8 else dict(u_qk=2.0 ** -22, u_p=U_BF16)))
    d = c.dev
    full_out = torch.full((8, 8, D), 3.0, dtype=torch.bfloat16, device="cuda")
    m = torch.full((c.words.size,), 0.5, device="cuda")
    n, lo, hi = 3, c.indptr[2], c.indptr[5]
    ind, out = d["indptr"][2:6], full_out[2:5]
    if q8:
        ws = c.ws(la.decode_q8_workspace_bytes(c.cfg, n, c.max_words, True))
        la.decode_attn_q8(c.cfg, d["q"][2:5], d["pos0"][2:5], d["table"], ind, c.max_words, c.pool, out, ws, m, d["status"])
    else:
        ws = c.ws(la.decode_mass_workspace_bytes(c.cfg, n, c.max_words))
        la.decode_attn_mass(c.cfg, d["q"][2:5], d["pos0"][2:5], d["table"], ind, c.max_words, d["meta"], *c.kv, out, m, ws,
                            d["status"])
    check(out, ref[2:5], bound[2:5], "decode slice")
    assert (full_out[:2] == 3).all() and (full_out[5:] == 3).all()
    want = np.where((np.arange(c.words.size) >= lo) & (np.arange(c.words.size) < hi), mref + 0.5, 0.5)
    check(m, want, mbound + 2.0 ** -23, "mass slice")


def test_decode_no_words_and_no_blocks():
    cfg = la.Cfg(8, 2)
    q = torch.randn(2, 8, D, device="cuda").to(torch.bfloat16)
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")                      # noqa: E731
    out = torch.full_like(q, 5.0)
    la.decode_attn_q8(cfg, q, i(0, 0), i(), i(0, 0, 0), 0, la.Q8Pool.empty(2, 2), out, None)
    assert (out == 0).all()
    out.fill_(5.0)
    la.decode_attn_q8(cfg, q, i(0, 0), i(1), i(0, 1, 1), 1, la.Q8Pool.empty(0, 2), out, None)
    assert (out == 0).all()
    out.fill_(5.0)
    la.prefill_attn_q8(cfg, q, i(0, 1, 2), i(0, 0), 1, i(), i(0, 0, 0), 0, la.Q8Pool.empty(2, 2), out, None)
    assert (out == 0).all()


def test_large_pool_offsets_pass_32_bits():
    """Blocks at the end of a pool of 2^17 blocks: code offsets above 2^31 bytes."""
    cfg = la.Cfg(8, 8)
    c = PoolCase(cfg, [40], [([(0, 0)], 39, 1), ([(0, 7)], 46, 2)], seed=8, spare=0)
    nb, small = 1 << 17, c.num_blocks
    c.to()
    big = la.Q8Pool(torch.full((nb, 8, BLK, D), 0x7F, dtype=torch.uint8, device="cuda"),
                    torch.full((nb, 8, BLK, D), 0x7F, dtype=torch.uint8, device="cuda"),
                    torch.ones(nb, 8, device="cuda"), torch.ones(nb, 8, device="cuda"),
                    torch.zeros(nb, dtype=torch.int32, device="cuda"))
    for a in ("k_codes", "v_codes", "k_scale", "v_scale", "blk_meta"):
        getattr(big, a)[nb - small:] = getattr(c.pool, a)
    c.pool = big
    c.dev["table"] += nb - small
    ref, bound, *_ = c.reference()
    d = c.dev
    out = torch.zeros(2, 8, D, dtype=torch.bfloat16, device="cuda")
    ws = c.ws(la.decode_q8_workspace_bytes(cfg, 2, c.max_words))
    la.decode_attn_q8(cfg, d["q"][:2], d["pos0"], d["table"], d["indptr"], c.max_words, big, out, ws, None, d["status"])
    check(out, ref[:2], bound[:2], "decode large pool")
    check(c.prefill(), *c.reference(**PREFILL_U)[:2], "prefill large pool")
    k = torch.randn(3, 8, D, device="cuda").to(torch.bfloat16)
    slot = torch.tensor([nb * BLK - 16 * small - 16, nb * BLK - 16 * small - 15, 3], dtype=torch.int32, device="cuda")
    j = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    la.kv_write_q8(cfg, k, k, slot, j, big, None, d["status"])
    row = big.v_codes[nb - small - 1, :, 1].view(torch.float8_e4m3fn).float() * big.v_scale[nb - small - 1][:, None]
    assert ((row - k[1].float()).abs() <= 2.0 ** -4 * k[1].float().abs() + 2.0 ** -9 * big.v_scale[nb - small - 1][:, None]).all()
    assert d["status"].item() == 0


# ------------------------------------------------------------------------------------------ prefill
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_prefill(hq, hkv):
    docs, reqs = _requests(7)
    lens = [1, 70, 3, 5, 2, 17, 40]
    reqs = [(s, p - n + 1 if n < p else p, n) for (s, p, _), n in zip(reqs, lens)]
    c = PoolCase(_cfg(hq, hkv), docs, reqs, seed=hq * 10 + hkv).to()
    check(c.prefill(), *c.reference(**PREFILL_U)[:2], f"prefill {hq}/{hkv}")
    assert c.dev["status"].item() == 0


@pytest.mark.parametrize("kind", ["alibi", "llama31", "scale"])
def test_prefill_variants(kind):
    docs, reqs = _requests(7)
    reqs = [(s, max(0, p - 30), 31) for s, p, _ in reqs]
    c = PoolCase(_cfg(8, 2, kind), docs, reqs, seed=6).to()
    check(c.prefill(), *c.reference(**PREFILL_U)[:2], f"prefill {kind}")


@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 64, 127, 128, 129, 300])
def test_prefill_lengths(n):
    """One request's own prompt of n tokens (all causal), and one that has no tokens."""
    c = PoolCase(la.Cfg(8, 2), [max(n, 1)], [([(0, 0)], 0, n), ([(0, 0)], 5, 0)], seed=n).to()
    check(c.prefill(), *c.reference(**PREFILL_U)[:2], f"prefill {n} tokens")


def test_prefill_extreme_scales():
    docs, reqs = _requests(7)
    reqs = [(s, max(0, p - 4), 5) for s, p, _ in reqs]
    for k_exp, v_exp, q_scale in (((-120, -100), (-125, -90), 1.0), ((-10, 12), (-60, 60), 1.0),
                                  ((90, 100), (100, 110), 2.0 ** -100)):
        c = PoolCase(la.Cfg(8, 2, softmax_scale=1e-3 if k_exp[1] == 12 else 0.0), docs, reqs, seed=9, k_exp=k_exp,
                     v_exp=v_exp, q_scale=q_scale).to()
        check(c.prefill(), *c.reference(**PREFILL_U)[:2], f"prefill scales {k_exp} {v_exp}", rel=np.inf)


@pytest.mark.parametrize("kind", ["rope", "alibi", "llama31"])
@pytest.mark.parametrize("hq,hkv,most", [(8, 8, 32), (8, 8, 16), (6, 2, 10), (6, 2, 5), (8, 2, 8), (8, 2, 4), (32, 8, 1),
                                         (16, 1, 1), (16, 1, 8), (22, 2, 1), (22, 2, 2), (32, 1, 1), (5, 5, 17), (8, 2, 32),
                                         (8, 2, 33)])
def test_prefill_few_rows(hq, hkv, most, kind):
    """Query rows of a few tokens, with positions of their own: up to 16, 128 and more rows per KV head."""
    docs, reqs = _requests(14)
    lens = [most, 1, max(1, most // 2), most, 0, (most + 1) // 2, most] * 2
    # the last query keeps its place; the fourth request has tokens in front of its only key
    reqs = [(s, max(0, p - n + 1), n) for (s, p, _), n in zip(reqs, lens)]
    c = PoolCase(_cfg(hq, hkv, kind), docs, reqs, seed=hq + most).to()
    n = c.q.shape[0]
    out = torch.full((n + 3, hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    c.prefill(out[:n])
    check(out[:n], *c.reference(**PREFILL_U)[:2], f"prefill of {most} tokens {hq}/{hkv} {kind}")
    assert (out[n:] == 3).all()
    assert c.dev["status"].item() == 0


@pytest.mark.parametrize("most", [2, 5])
def test_prefill_few_rows_many_requests(most):
    """More units than two per SM, of 8 and of 20 rows."""
    docs, reqs = _requests(7)
    reqs = [(s, max(0, p - most + 1), most) for s, p, _ in reqs] * 12
    c = PoolCase(la.Cfg(16, 4), docs, reqs, seed=most).to()
    check(c.prefill(), *c.reference(**PREFILL_U)[:2], f"prefill of {most} tokens, {len(reqs)} requests")


def test_prefill_few_rows_one_long_request():
    """Many partial results of one request; a document met again at another offset."""
    c = PoolCase(la.Cfg(8, 2), [2000, 333], [([(1, 0), (0, 333), (1, 2400), (1, 2733)], 3060, 4)], seed=3).to()
    check(c.prefill(), *c.reference(**PREFILL_U)[:2], "prefill of 4 tokens over 3000")


@pytest.mark.parametrize("most", [3, 5])
def test_prefill_few_rows_bad_block(most):
    docs, reqs = _requests(4)
    reqs = [(s, max(0, p - most + 1), most) for s, p, _ in reqs]
    c = PoolCase(la.Cfg(8, 2), docs, reqs, seed=2)
    c.words[3] = la_pack(c.num_blocks + 5, 48)
    c.to()
    check(c.prefill(), *c.reference(**PREFILL_U)[:2], f"prefill of {most} tokens with a bad block")
    assert c.dev["status"].item() == la.DSTATUS_BAD_BLOCK


@pytest.mark.parametrize("most", [4, 40])
def test_prefill_extreme_scales_rows(most):
    docs, reqs = _requests(7)
    reqs = [(s, max(0, p - most + 1), most) for s, p, _ in reqs]
    for k_exp, v_exp in (((-120, -100), (-125, -90)), ((90, 100), (100, 110))):
        c = PoolCase(la.Cfg(8, 2), docs, reqs, seed=9, k_exp=k_exp, v_exp=v_exp,
                     q_scale=2.0 ** -100 if k_exp[0] > 0 else 1.0).to()
        check(c.prefill(), *c.reference(**PREFILL_U)[:2], f"prefill of {most} tokens, scales {k_exp} {v_exp}", rel=np.inf)


def test_prefill_faults_and_rows_behind_the_last_sequence():
    docs, reqs = _requests(4)
    reqs = [(s, max(0, p - 8), 9) for s, p, _ in reqs]
    c = PoolCase(la.Cfg(8, 2), docs, reqs, seed=2)
    c.words[3] = la_pack(c.num_blocks + 5, 48)
    c.to()
    n = c.q.shape[0]
    out = torch.full((n + 3, 8, D), 3.0, dtype=torch.bfloat16, device="cuda")
    c.prefill(out[:n])
    check(out[:n], *c.reference(**PREFILL_U)[:2], "prefill with a bad block")
    assert (out[n:] == 3).all()
    assert c.dev["status"].item() == la.DSTATUS_BAD_BLOCK


# -------------------------------------------------------------------------------------------- write
def _state(nb, hkv, seed, filled):
    """A pool whose blocks hold filled[b] tokens; unwritten slots hold arbitrary codes."""
    rng = np.random.default_rng(seed)
    shape = (nb, hkv, BLK, D)
    return dict(k_codes=to_e4m3(rng.standard_normal(shape) * 150), v_codes=to_e4m3(rng.standard_normal(shape) * 150),
                k_scale=(2.0 ** rng.integers(-12, -6, (nb, hkv))).astype(np.float32),
                v_scale=(2.0 ** rng.integers(-12, -6, (nb, hkv))).astype(np.float32),
                meta=np.array([i << 8 | f if f else 0 for i, f in enumerate(filled)], np.int64))


def _device_pool(st):
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a.astype(dt))).cuda()          # noqa: E731
    return la.Q8Pool(t(st["k_codes"], np.uint8), t(st["v_codes"], np.uint8), t(st["k_scale"], np.float32),
                     t(st["v_scale"], np.float32), t(st["meta"], np.int32))


def _write(cfg, pool, k, v, slot, j):
    i = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()               # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = len(slot)
    ws = torch.empty(max(16, la.kv_write_q8_workspace_bytes(cfg, n, pool.num_blocks)), dtype=torch.uint8, device="cuda")
    la.kv_write_q8(cfg, k.cuda(), v.cuda(), i(slot), i(j), pool, ws, status)
    return int(status.item())


def _same_pool(pool, want):
    for n in ("k_scale", "v_scale"):
        assert np.array_equal(getattr(pool, n).cpu().numpy(), want[n]), n
    assert np.array_equal(pool.blk_meta.cpu().numpy(), want["meta"].astype(np.int32))
    for n in ("k_codes", "v_codes"):
        got = getattr(pool, n).cpu().numpy()
        nan = (want[n] & 0x7F) == 0x7F                     # a NaN's sign is not defined
        assert np.array_equal(got[~nan], want[n][~nan]) and ((got[nan] & 0x7F) == 0x7F).all(), n


@pytest.mark.parametrize("hkv", [1, 2, 8, 11])
@pytest.mark.parametrize("n,order", [(1, "asc"), (2, "asc"), (15, "asc"), (16, "asc"), (17, "shuffle"), (130, "asc"),
                                     (130, "shuffle"), (1024, "asc"), (1025, "asc"), (1500, "shuffle")])
def test_write(n, order, hkv):
    """n tokens from slot 5 of a partly filled block on: codes, scales and metadata exactly."""
    if n > 1000 and hkv > 2:
        pytest.skip("the same code as 2 heads, slow on the CPU")
    rng = np.random.default_rng([n, hkv])
    nb = (n + 5) // 16 + 3
    st = _state(nb, hkv, n, [16] + [5] + [0] * (nb - 2))
    j = 16 + 5 + np.arange(n)
    slot = j.copy()
    if order == "shuffle":
        p = rng.permutation(n)
        j, slot = j[p], slot[p]
    k, v = bf16(rng.standard_normal((n, hkv, D)) * 2), bf16(rng.standard_normal((n, hkv, D)) * 2.0 ** rng.integers(-9, 3, (n, hkv, 1)))
    cfg = la.Cfg(hkv, hkv)
    pool = _device_pool(st)
    assert _write(cfg, pool, k, v, slot, j) == 0
    _same_pool(pool, write_reference(cfg, st, k, v, slot, j))


@pytest.mark.parametrize("n", [40, 1300])
def test_write_faults_and_repeated_slots(n):
    rng = np.random.default_rng(n)
    nb = n // 16 + 4
    st = _state(nb, 2, n, [9] + [0] * (nb - 1))
    j = 9 + np.arange(n)
    slot = j.copy()
    slot[3], slot[5] = -1, nb * 16                          # outside the pool
    slot[7] += 1                                            # not aligned, on a slot that token 8 writes
    slot[20], j[20] = slot[11], j[11]                       # the same slot twice: the later one stays
    k, v = bf16(rng.standard_normal((n, 2, D))), bf16(rng.standard_normal((n, 2, D)))
    k[11] *= 64                                             # the overwritten token does not raise the scale
    cfg = la.Cfg(2, 2)
    pool = _device_pool(st)
    assert _write(cfg, pool, k, v, slot, j) == la.DSTATUS_BAD_SLOT | la.DSTATUS_BAD_ALIGN
    _same_pool(pool, write_reference(cfg, st, k, v, slot, j))


def test_write_values_at_the_edges():
    """Zeros, the largest and smallest bf16, borders of scales and codes, infinities and NaN (V only:
    a rotation of infinities is NaN or infinity by its signs)."""
    cfg = la.Cfg(1, 1)
    rows = [np.zeros(D), np.full(D, 3.38e38), np.full(D, 1e-40), np.full(D, 448.0), np.full(D, 450.0), np.full(D, 2.0 ** -130),
            np.where(np.arange(D) % 2, 464.0, 17.0), 1.0 + np.arange(D) / 128, np.exp2(-np.arange(D) / 4.0),
            np.where(np.arange(D) == 3, np.inf, 2.5), np.where(np.arange(D) == 3, np.nan, 2.5), np.full(D, -np.inf)]
    n = len(rows)
    v = bf16(np.array(rows)[:, None])
    k = torch.where(v.isfinite(), v, torch.zeros_like(v))
    st = _state(n, 1, 1, [0] * n)
    j = np.arange(n) * 16 + 7
    pool = _device_pool(st)
    assert _write(cfg, pool, k, v, j, j) == 0
    _same_pool(pool, write_reference(cfg, st, k, v, j, j))
    # a larger token later: codes that fall below the new scale's normal range
    k2 = bf16(np.full((1, 1, D), 1.0))
    st2 = write_reference(cfg, st, k, v, j, j)
    assert _write(cfg, pool, k2 * 2.0 ** 20, k2 * 2.0 ** 20, [16 * 8 + 8], [16 * 8 + 8]) == 0
    _same_pool(pool, write_reference(cfg, st2, k2 * 2.0 ** 20, k2 * 2.0 ** 20, [16 * 8 + 8], [16 * 8 + 8]))


def test_write_scales_that_are_not_powers_of_two():
    rng = np.random.default_rng(4)
    st = _state(3, 2, 4, [16, 6, 0])
    st["k_scale"] = st["k_scale"] * np.float32(1.37)
    st["v_scale"] = st["v_scale"] * np.float32(0.77)
    j = 16 + 6 + np.arange(12)
    k, v = bf16(rng.standard_normal((12, 2, D)) * 0.05), bf16(rng.standard_normal((12, 2, D)) * 0.05)
    cfg = la.Cfg(2, 2)
    pool = _device_pool(st)
    assert _write(cfg, pool, k, v, j, j) == 0
    _same_pool(pool, write_reference(cfg, st, k, v, j, j))


@pytest.mark.parametrize("kind", ["alibi", "llama31"])
def test_write_variants(kind):
    rng = np.random.default_rng(3)
    cfg = _cfg(4, 2, kind)
    st = _state(4, 2, 3, [0] * 4)
    j = np.arange(50)
    k, v = bf16(rng.standard_normal((50, 2, D))), bf16(rng.standard_normal((50, 2, D)))
    pool = _device_pool(st)
    assert _write(cfg, pool, k, v, j, j) == 0
    _same_pool(pool, write_reference(cfg, st, k, v, j, j))


# -------------------------------------------------------------------------------------------- evict
def _evict(words, indptr, max_words, mass, keep, n_first, n_last, room=0, evicted=True):
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(np.asarray(a, dt))).cuda()      # noqa: E731
    n = len(words)
    out = dict(table=torch.full((n + room,), -1, dtype=torch.int32, device="cuda"),
               ind=torch.full((len(indptr) + room,), -1, dtype=torch.int32, device="cuda"),
               mass=torch.full((n + room,), -3.0, device="cuda"),
               gone=torch.full((n + room,), -1, dtype=torch.int32, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    la.evict_blocks(t(np.asarray(words, np.uint32).view(np.int32), np.int32), t(indptr, np.int32), max_words,
                    t(mass, np.float32), t(keep, np.int32), n_first, n_last, out["table"], out["ind"], out["mass"],
                    out["gone"] if evicted else None, status)
    return {k: v.cpu().numpy() for k, v in out.items()}, int(status.item())


def _check_evict(words, indptr, max_words, mass, keep, n_first, n_last):
    got, status = _evict(words, indptr, max_words, mass, keep, n_first, n_last, room=5)
    table, ind, m, gone = evict_reference(words, indptr, max_words, mass, keep, n_first, n_last)
    assert got["ind"][:len(ind)].tolist() == ind
    assert np.array_equal(got["table"][:len(table)].view(np.uint32), np.array(table, np.uint32))
    assert np.array_equal(got["mass"][:len(m)], np.array(m, np.float32), equal_nan=True)
    assert np.array_equal(got["gone"][:len(gone)].view(np.uint32), np.array(gone, np.uint32))
    # nothing behind the last entries is written
    assert (got["table"][len(table):] == -1).all() and (got["mass"][len(m):] == -3).all()
    assert (got["gone"][len(gone):] == -1).all() and (got["ind"][len(ind):] == -1).all()
    return status


@pytest.mark.parametrize("n_first,n_last", [(0, 0), (2, 3), (4, 16), (0, 1000)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict(ties, n_first, n_last):
    rng = np.random.default_rng(n_first + ties)
    n = [0, 1, 2, 7, 31, 32, 33, 100, 0, 1023, 1024, 1025, 3000, 5]
    indptr = np.concatenate([[0], np.cumsum(n)])
    words = rng.integers(0, 1 << 32, indptr[-1], dtype=np.uint32)
    mass = np.exp(2 * rng.standard_normal(indptr[-1])).astype(np.float32)
    if ties:
        mass = np.round(mass).astype(np.float32)
    for keep in ([0] * len(n), n, [max(0, x // 2) for x in n], [x - 1 for x in n], [1] * len(n), [x + 5 for x in n],
                 [-4] * len(n), [5, 1, 1, 3, 30, 9, 33, 60, 2, 1000, 64, 500, 21, 4]):
        assert _check_evict(words, indptr, max(n), mass, keep, n_first, n_last) == 0


def test_evict_special_weights():
    sp = np.array([0.0, -0.0, np.nan, np.inf, -np.inf, 1e-45, -1e-45, 3e38, -1.0, np.nan, np.inf, 1.0, -0.0, 0.0, 2.0, 1.0],
                  np.float32)
    for keep in range(17):
        _check_evict(np.arange(16, dtype=np.uint32), [0, 16], 16, sp, [keep], 0, 0)
        _check_evict(np.arange(16, dtype=np.uint32), [0, 16], 16, sp, [keep], 3, 4)


@pytest.mark.parametrize("n", [32768, 60000])
def test_evict_long(n):
    """More words than one pass of a CTA, and than its shared memory holds."""
    rng = np.random.default_rng(n)
    mass = np.round(np.exp(rng.standard_normal(n)) * 8).astype(np.float32) / 8
    words = rng.integers(0, 1 << 32, n, dtype=np.uint32)
    ind = np.array([0, n // 3, n])
    for keep in ([100, 5000], [n // 4, n // 2], [n, 1]):
        _check_evict(words, ind, n, mass, keep, 4, 64)
    _check_evict(words, ind, n, np.zeros(n, np.float32), [77, 1500], 4, 64)


@pytest.mark.parametrize("n", [4095, 4097, 5000, 400003])
def test_evict_cluster(n):
    """Requests of one CTA and of a cluster, empty ones among them; more keys than a cluster's shared memory holds."""
    rng = np.random.default_rng(n)
    lens = [n, 0, 1, 31, 4097, 300]
    ind = np.concatenate([[0], np.cumsum(lens)])
    mass = np.round(rng.random(ind[-1]) * 5000).astype(np.float32) / 5000
    words = rng.integers(0, 1 << 32, ind[-1], dtype=np.uint32)
    for keep in ([n - 7, 3, 1, 30, 2048, 150], [n // 2, 0, 0, 5, 33, 299]):
        want = la.DSTATUS_BAD_TABLE if max(lens) > n else 0
        assert _check_evict(words, ind, n, mass, keep, 4, 64) == want


def test_evict_request_longer_than_max_words():
    mass = np.arange(20, dtype=np.float32)
    assert _check_evict(np.arange(20, dtype=np.uint32), [0, 12, 20], 9, mass, [5, 6], 1, 2) == la.DSTATUS_BAD_TABLE


def test_evict_slice_without_evicted():
    """Row pointers that do not start at 0; no list of evicted words."""
    rng = np.random.default_rng(1)
    words, mass = rng.integers(0, 1 << 32, 50, dtype=np.uint32), rng.random(50).astype(np.float32)
    ind = [10, 25, 25, 45]
    got, status = _evict(words, ind, 20, mass, [6, 2, 9], 1, 1, evicted=False)
    table, indo, m, _ = evict_reference(words, ind, 20, mass, [6, 2, 9], 1, 1)
    assert got["ind"].tolist() == indo and (got["gone"] == -1).all()
    assert np.array_equal(got["table"][:len(table)].view(np.uint32), np.array(table, np.uint32))
    _check_evict(words, ind, 20, mass, [6, 2, 9], 1, 1)


def test_evict_no_requests_and_many():
    got, _ = _evict([], [0], 0, [], [], 0, 0)
    assert got["ind"].tolist() == [0]
    rng = np.random.default_rng(2)
    n = rng.integers(0, 9, 3000)
    ind = np.concatenate([[0], np.cumsum(n)])
    _check_evict(np.arange(ind[-1], dtype=np.uint32), ind, 8, rng.random(ind[-1]).astype(np.float32),
                 rng.integers(0, 9, 3000), 1, 1)


# ----------------------------------------------------------------------- as a program uses them
@pytest.mark.parametrize("most", [1, 4, 12, 70])
def test_max_words_far_above_the_tables(most):
    """max_words only bounds: the largest int is a valid bound."""
    docs, reqs = _requests(7)
    reqs = [(s, max(0, p - most + 1), most) for s, p, _ in reqs]
    c = PoolCase(la.Cfg(8, 2), docs, reqs, seed=most).to()
    d, n, big = c.dev, c.q_pos0.size, 2 ** 31 - 1
    out = torch.full_like(d["q"], 7.0)
    if most == 1:
        ws = c.ws(la.decode_q8_workspace_bytes(c.cfg, n, big))
        la.decode_attn_q8(c.cfg, d["q"], d["pos0"], d["table"], d["indptr"], big, c.pool, out, ws, None, d["status"])
        check(out, *c.reference()[:2], "decode, largest max_words")
    ws = c.ws(la.prefill_q8_workspace_bytes(c.cfg, n, out.shape[0], most, big, c.words.size))
    la.prefill_attn_q8(c.cfg, d["q"], d["cu"], d["pos0"], most, d["table"], d["indptr"], big, c.pool, out, ws, d["status"])
    check(out, *c.reference(**PREFILL_U)[:2], f"prefill of {most} tokens, largest max_words")
    words = np.arange(50, dtype=np.uint32)
    assert _check_evict(words, [0, 20, 50], big, np.linspace(0, 1, 50, dtype=np.float32), [5, 7], 1, 2) == 0


def test_write_decode_evict_decode_together():
    """Prompts written in 8 bits, prefilled, decoded token by token with their weights accumulated,
    the tables halved, and decoded further over the shorter tables."""
    cfg = la.Cfg(8, 2)
    rng = np.random.default_rng(11)
    B, n0, steps = 3, 100, 20
    per = -(-(n0 + 2 * steps) // BLK)
    nb = B * per + 2
    phys = rng.permutation(nb)[:B * per].reshape(B, per)
    st = dict(k_codes=np.zeros((nb, 2, BLK, D), np.uint8), v_codes=np.zeros((nb, 2, BLK, D), np.uint8),
              k_scale=np.ones((nb, 2), np.float32), v_scale=np.ones((nb, 2), np.float32), meta=np.zeros(nb, np.int64))
    pool = _device_pool(st)
    slot_of = lambda r, t: int(phys[r, t // BLK]) * BLK + t % BLK                            # noqa: E731

    def put(slot, j):
        nonlocal st
        k, v = bf16(rng.standard_normal((len(slot), 2, D))), bf16(rng.standard_normal((len(slot), 2, D)))
        assert _write(cfg, pool, k, v, slot, j) == 0
        st = write_reference(cfg, st, k, v, slot, j)
        _same_pool(pool, st)

    def case(tables, pos, n=1):
        c = PoolCase.__new__(PoolCase)
        c.cfg, c.q8, c.num_blocks, c.meta = cfg, True, nb, st["meta"]
        c.k_codes, c.v_codes, c.k_scale, c.v_scale = st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"]
        c.words = np.array([w for t in tables for w in t], np.uint32)
        c.indptr = np.concatenate([[0], np.cumsum([len(t) for t in tables])]).tolist()
        c.q_pos0, c.cu = np.array(pos, np.int32), np.arange(B + 1, dtype=np.int32) * n
        c.q = bf16(rng.standard_normal((B * n, 8, D)) * 2)
        c.max_words = max(len(t) for t in tables)
        c.to()
        c.pool = pool                                          # the pool as the library wrote it
        return c

    put([slot_of(r, t) for r in range(B) for t in range(n0)], [t for _ in range(B) for t in range(n0)])
    words = lambda r, n: [la_pack(int(b), 0) for b in phys[r, :-(-n // BLK)]]                # noqa: E731
    c = case([words(r, n0) for r in range(B)], [0] * B, n0)
    check(c.prefill(), *c.reference(**PREFILL_U)[:2], "prompt")
    tables, total = [words(r, n0) for r in range(B)], [np.zeros(len(words(r, n0))) for r in range(B)]
    slack, mass, cut = [np.zeros(len(t)) for t in total], None, None
    for step in range(2 * steps):
        t = n0 + step
        put([slot_of(r, t) for r in range(B)], [t] * B)
        if t % BLK == 0:                                       # the token opened a block: one more word
            for r in range(B):
                tables[r] = tables[r] + [la_pack(int(phys[r, t // BLK]), 0)]
                total[r], slack[r] = np.append(total[r], 0.0), np.append(slack[r], 0.0)
        c = case(tables, [t] * B)
        mass = torch.from_numpy(np.concatenate(total).astype(np.float32)).cuda()
        ref, bound, mref, mbound = c.reference()
        check(c.decode(mass), ref, bound, f"token {t}")
        want = np.concatenate(total) + mref
        check(mass, want, mbound + 2.0 ** -22 * (1 + want), f"mass at token {t}")
        cutp = np.cumsum([0] + [len(x) for x in tables])
        got = mass.cpu().numpy()
        total = [got[cutp[r]:cutp[r + 1]].astype(np.float64) for r in range(B)]
        if step == steps:
            keep = [len(x) // 2 for x in tables]
            res, status = _evict(c.words, c.indptr, c.max_words, got, keep, 1, 2)
            table, ind, m, _ = evict_reference(c.words, c.indptr, c.max_words, got, keep, 1, 2)
            assert status == 0 and res["table"][:len(table)].view(np.uint32).tolist() == [int(x) for x in table]
            tables = [[int(x) for x in table[ind[r]:ind[r + 1]]] for r in range(B)]
            total = [np.array(m[ind[r]:ind[r + 1]], np.float64) for r in range(B)]
            cut = [len(x) for x in tables]
    assert cut is not None


def test_graphs_and_streams():
    """Every call captured once and replayed on other inputs, and eager calls on two streams at once."""
    docs, reqs = _requests(7)
    c = PoolCase(la.Cfg(8, 2), docs, reqs, seed=21).to()
    d = c.dev
    words = c.words.size
    mass, out, pout = torch.zeros(words, device="cuda"), torch.zeros_like(d["q"]), torch.zeros_like(d["q"])
    wsd = c.ws(la.decode_q8_workspace_bytes(c.cfg, 7, c.max_words, True))
    wsp = c.ws(la.prefill_q8_workspace_bytes(c.cfg, 7, 7, 1, c.max_words, words))
    keep = torch.tensor([max(1, (c.indptr[r + 1] - c.indptr[r]) // 2) for r in range(7)], dtype=torch.int32, device="cuda")
    to, mo, io = torch.zeros_like(d["table"]), torch.zeros_like(mass), torch.zeros_like(d["indptr"])
    kr = torch.randn(2000, 2, D, device="cuda").to(torch.bfloat16)
    spare = torch.tensor(np.setdiff1d(np.arange(c.num_blocks), np.concatenate(c.doc_blocks))[0], device="cuda")
    slot1 = (spare * BLK + torch.arange(3, device="cuda")).int()
    j1 = torch.arange(3, dtype=torch.int32, device="cuda")
    other = la.Q8Pool.empty(200, 2)
    wsw = c.ws(la.kv_write_q8_workspace_bytes(c.cfg, 2000, 200))
    big = torch.arange(2000, dtype=torch.int32, device="cuda")

    def calls():
        la.kv_write_q8(c.cfg, kr[:3], kr[:3], slot1, j1, c.pool, None, d["status"])
        la.kv_write_q8(c.cfg, kr, kr, big, big, other, wsw, d["status"])
        c.decode(mass, out, wsd)
        c.prefill(pout, wsp)
        la.evict_blocks(d["table"], d["indptr"], c.max_words, mass, keep, 1, 1, to, io, mo, None, d["status"])

    calls()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            calls()
    d["q"].copy_(torch.randn_like(d["q"]))
    c.q = d["q"].cpu()
    kr.mul_(0.5)
    mass.zero_()
    other.blk_meta.zero_()
    g.replay()
    torch.cuda.synchronize()
    ref, bound, mref, mbound = c.reference()
    check(out, ref, bound, "replayed decode")
    check(mass, mref, mbound, "replayed mass")
    check(pout, *c.reference(**PREFILL_U)[:2], "replayed prefill")
    got = (other.v_codes.view(torch.float8_e4m3fn).float() * other.v_scale[..., None, None]).permute(0, 2, 1, 3).reshape(-1, 2, D)[:2000]
    amax = kr.float().abs().amax(2).reshape(125, 16, 2).amax(1).repeat_interleave(16, 0)[..., None]
    assert ((got - kr.float()).abs() <= 2.0 ** -4 * kr.float().abs() + 2.0 ** -10 * amax / 224).all()
    # the same words on two streams, each with its own workspace and outputs
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(out) for _ in range(2)]
    ms = [torch.zeros_like(mass) for _ in range(2)]
    wss = [torch.empty_like(wsd) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                ms[i].zero_()
            c.decode(ms[i], outs[i], wss[i], stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs) and all(torch.equal(m, mass) for m in ms)
    assert d["status"].item() == 0
