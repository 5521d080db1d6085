"""Refusals and workspace sizes of the 8-bit pool, block mass and eviction calls.  Every call here
is refused, or does nothing, on the host: nothing is launched and no pointer is read."""
import copy
import ctypes
import pickle

import pytest
import torch

from position_agnostic_paged_b200 import lazy_attn as la

OK = la.Cfg(8, 2)
P = 1 << 20          # stands for an aligned device pointer


def _pool(**kw):
    f = dict(k_codes=P, v_codes=P, k_scale=P, v_scale=P, blk_meta=P, num_blocks=8)
    f.update(kw)
    return la.LazyQ8Pool(*[f[n] for n in ("k_codes", "v_codes", "k_scale", "v_scale", "blk_meta", "num_blocks")])


def _ref(x):
    return ctypes.byref(x) if x is not None else None


def _write(cfg=OK, pool=None, no_pool=False, **kw):
    a = dict(k=P, v=P, n=3, slot=P, j=P, ws=P, wsb=1 << 20)
    a.update(kw)
    c = cfg.c() if cfg else None
    pl = None if no_pool else (pool or _pool())
    return la._lib.lazy_kv_write_q8(_ref(c), a["k"], a["v"], a["n"], a["slot"], a["j"], _ref(pl), a["ws"], a["wsb"], None, None)


def _decode(cfg=OK, pool=None, no_pool=False, **kw):
    a = dict(q=P, qp=P, n=2, table=P, indptr=P, mw=4, out=P, mass=None, ws=P, wsb=1 << 30)
    a.update(kw)
    c = cfg.c() if cfg else None
    pl = None if no_pool else (pool or _pool())
    return la._lib.lazy_decode_attn_q8(_ref(c), a["q"], a["qp"], a["n"], a["table"], a["indptr"], a["mw"], _ref(pl),
                                       a["out"], a["mass"], a["ws"], a["wsb"], None, None)


def _mass(cfg=OK, **kw):
    a = dict(q=P, qp=P, n=2, table=P, indptr=P, mw=4, meta=P, k=P, v=P, nb=8, out=P, mass=P, ws=P, wsb=1 << 30)
    a.update(kw)
    c = cfg.c()
    return la._lib.lazy_decode_attn_mass(_ref(c), a["q"], a["qp"], a["n"], a["table"], a["indptr"], a["mw"], a["meta"],
                                         a["k"], a["v"], a["nb"], a["out"], a["mass"], a["ws"], a["wsb"], None, None)


def _prefill(cfg=OK, pool=None, no_pool=False, **kw):
    a = dict(q=P, cu=P, p0=P, n=2, tq=6, mq=3, table=P, indptr=P, mw=4, out=P, ws=P, wsb=1 << 30)
    a.update(kw)
    c = cfg.c() if cfg else None
    pl = None if no_pool else (pool or _pool())
    return la._lib.lazy_prefill_attn_q8(_ref(c), a["q"], a["cu"], a["p0"], a["n"], a["tq"], a["mq"], a["table"],
                                        a["indptr"], a["mw"], _ref(pl), a["out"], a["ws"], a["wsb"], None, None)


def _evict(**kw):
    a = dict(table=P, indptr=2 * P, n=2, mw=4, mass=3 * P, keep=4 * P, nf=1, nl=1, to=5 * P, io=6 * P, mo=7 * P, ev=8 * P)
    a.update(kw)
    return la._lib.lazy_evict_blocks(a["table"], a["indptr"], a["n"], a["mw"], a["mass"], a["keep"], a["nf"], a["nl"],
                                     a["to"], a["io"], a["mo"], a["ev"], None, None)


@pytest.mark.parametrize("call", [_write, _decode, _prefill])
def test_pool_is_checked(call):
    assert call(no_pool=True) == la.LAZY_EINVAL
    for f in ("k_codes", "v_codes", "k_scale", "v_scale", "blk_meta"):
        assert call(pool=_pool(**{f: None})) == la.LAZY_EINVAL
    assert call(pool=_pool(k_codes=P + 8)) == la.LAZY_EINVAL
    assert call(pool=_pool(v_codes=P + 1)) == la.LAZY_EINVAL
    assert call(pool=_pool(num_blocks=-1)) == la.LAZY_EINVAL
    assert call(pool=_pool(num_blocks=(1 << 17) + 1)) == la.LAZY_ERANGE


@pytest.mark.parametrize("call", [_write, _decode, _prefill, _mass])
def test_shapes_are_checked(call):
    assert call(cfg=la.Cfg(8, 2, head_dim=64)) == la.LAZY_ESHAPE
    assert call(cfg=la.Cfg(8, 2, block_size=32)) == la.LAZY_ESHAPE
    assert call(cfg=la.Cfg(8, 3)) == la.LAZY_ESHAPE
    assert call(cfg=la.Cfg(64, 1)) == la.LAZY_ESHAPE
    assert call(n=-1) == la.LAZY_EINVAL
    assert call(n=0) == la.LAZY_OK


def test_write_refusals():
    assert _write(cfg=None) == la.LAZY_EINVAL
    for f in ("k", "v", "slot", "j"):
        assert _write(**{f: None}) == la.LAZY_EINVAL
    assert _write(k=P + 8) == la.LAZY_EINVAL and _write(v=P + 2) == la.LAZY_EINVAL
    assert _write(n=5000, ws=None) == la.LAZY_EWORKSPACE
    assert _write(n=5000, wsb=la.kv_write_q8_workspace_bytes(OK, 5000, 8) - 1) == la.LAZY_EWORKSPACE
    assert _write(n=5000, ws=P + 4) == la.LAZY_EINVAL
    assert la.kv_write_q8_workspace_bytes(OK, 1024, 1 << 17) == 0


def test_decode_refusals():
    for f in ("q", "qp", "table", "indptr", "out"):
        assert _decode(**{f: None}) == la.LAZY_EINVAL
        assert _mass(**{f: None}) == la.LAZY_EINVAL
    for f in ("meta", "k", "v", "mass"):
        assert _mass(**{f: None}) == la.LAZY_EINVAL
    assert _mass(k=P + 8) == la.LAZY_EINVAL
    assert _mass(nb=(1 << 17) + 1) == la.LAZY_ERANGE
    for call in (_decode, _mass):
        assert call(q=P + 4) == la.LAZY_EINVAL and call(out=P + 4) == la.LAZY_EINVAL
    assert _decode(mw=-1) == la.LAZY_EINVAL
    assert _decode(ws=None) == la.LAZY_EWORKSPACE
    assert _decode(ws=P + 8) == la.LAZY_EINVAL
    assert _decode(wsb=la.decode_q8_workspace_bytes(OK, 2, 4) - 1) == la.LAZY_EWORKSPACE
    # block mass needs more room, and a workspace without it is not enough
    assert la.decode_q8_workspace_bytes(OK, 2, 4, True) > la.decode_q8_workspace_bytes(OK, 2, 4)
    assert _decode(mass=P, wsb=la.decode_q8_workspace_bytes(OK, 2, 4)) == la.LAZY_EWORKSPACE
    assert _mass(wsb=la.decode_mass_workspace_bytes(OK, 2, 4) - 1) == la.LAZY_EWORKSPACE
    assert _decode(n=1 << 28) == la.LAZY_ERANGE
    assert _mass(mw=(1 << 20) + 1) == la.LAZY_ERANGE and _decode(mass=P, mw=(1 << 20) + 1) == la.LAZY_ERANGE


def test_prefill_refusals():
    for f in ("q", "cu", "p0", "table", "indptr", "out"):
        assert _prefill(**{f: None}) == la.LAZY_EINVAL
    for f in ("tq", "mq", "mw"):
        assert _prefill(**{f: -1}) == la.LAZY_EINVAL
    assert _prefill(ws=None) == la.LAZY_EWORKSPACE
    assert _prefill(ws=P + 8) == la.LAZY_EINVAL
    assert _prefill(q=P + 4) == la.LAZY_EINVAL and _prefill(out=P + 8) == la.LAZY_EINVAL
    assert _prefill(n=65536) == la.LAZY_ERANGE and _prefill(mq=1 << 30) == la.LAZY_ERANGE
    assert _prefill(wsb=la.prefill_q8_workspace_bytes(OK, 2, 6, 3, 4, 8) - 1) == la.LAZY_EWORKSPACE
    assert _prefill(tq=0) == la.LAZY_OK and _prefill(mq=0) == la.LAZY_OK


def test_evict_refusals():
    for f in ("table", "indptr", "mass", "keep", "to", "io", "mo"):
        assert _evict(**{f: None}) == la.LAZY_EINVAL
    for f in ("n", "mw", "nf", "nl"):
        assert _evict(**{f: -1}) == la.LAZY_EINVAL
    assert _evict(n=(1 << 20) + 1) == la.LAZY_ERANGE
    # outputs must not be inputs or each other
    assert _evict(to=P) == la.LAZY_EINVAL
    assert _evict(mo=3 * P) == la.LAZY_EINVAL
    assert _evict(io=2 * P) == la.LAZY_EINVAL
    assert _evict(ev=P) == la.LAZY_EINVAL
    assert _evict(ev=5 * P) == la.LAZY_EINVAL


def test_binding_checks_types_shapes_and_devices():
    pool = la.Q8Pool.empty(4, 2, device="cpu")
    assert pool.num_blocks == 4 and pool.c().num_blocks == 4
    with pytest.raises(ValueError):
        la.Q8Pool(pool.k_codes.half(), pool.v_codes, pool.k_scale, pool.v_scale, pool.blk_meta)
    with pytest.raises(ValueError):
        la.Q8Pool(pool.k_codes, pool.v_codes, pool.k_scale.double(), pool.v_scale, pool.blk_meta)
    with pytest.raises(ValueError):
        la.Q8Pool(pool.k_codes, pool.v_codes[:, :1], pool.k_scale, pool.v_scale, pool.blk_meta)
    with pytest.raises(ValueError):
        la.Q8Pool(pool.k_codes.transpose(2, 3).contiguous().transpose(2, 3), pool.v_codes, pool.k_scale, pool.v_scale,
                  pool.blk_meta)
    i = lambda *a: torch.tensor(a, dtype=torch.int32)                                    # noqa: E731
    x = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                                                      # CPU tensors
        la.kv_write_q8(OK, x, x, i(0), i(0), pool)
    with pytest.raises(ValueError):                                                      # another head count
        la.kv_write_q8(la.Cfg(8, 4), x, x, i(0), i(0), pool)
    with pytest.raises(ValueError):
        la.kv_write_q8(OK, x.half(), x, i(0), i(0), pool)
    with pytest.raises(ValueError):
        la.kv_write_q8(OK, x, x, i(0).long(), i(0), pool)
    q = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                                                      # mass: one per word
        la.decode_attn_q8(OK, q, i(0), i(0, 0), i(0, 2), 2, pool, q, None, torch.zeros(1))
    with pytest.raises(ValueError):
        la.decode_attn_q8(OK, q, i(0), i(0, 0), i(0), 2, pool, q, None)
    f = torch.zeros(2)
    with pytest.raises(ValueError):                                                      # too little room
        la.evict_blocks(i(0, 0), i(0, 2), 2, f, i(1), 0, 0, i(0), i(0, 0), f.clone())


def test_cfg_stays_a_plain_value():
    """The calls keep a C structure of the configuration; copies, pickles and mutable fields are as without it."""
    for cfg in (la.Cfg(8, 2), la.Cfg(8, 2, alibi_slopes=(0.5,) * 8), la.Cfg(8, 2, rope_theta=(0.1,) * 64)):
        assert la.decode_q8_workspace_bytes(cfg, 1, 1) == la.decode_q8_workspace_bytes(cfg, 1, 1)
        for other in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg))):
            assert other == cfg and other._shared_c() is not cfg._shared_c()
        assert cfg.c() is not cfg.c() and cfg._shared_c() is cfg._shared_c()
    theta = [0.1] * 64
    cfg = la.Cfg(8, 2, rope_theta=theta)
    assert cfg._shared_c().rope_theta[3] == 0.1
    theta[3] = 0.25
    assert cfg._shared_c().rope_theta[3] == 0.25
