"""Paged-pool cases for the 8-bit pool, block mass and eviction, with their values in 64 bits.

A case holds documents (token counts) in a pool of 16-token blocks, placed by a seeded permutation,
and requests: segments (document, offset) and query positions.  Pool contents are random e4m3 codes
and scales, or bf16; unwritten slots hold NaN.  The reference values come from the definition:
softmax over the keys t <= p of scale q^T R(-(p - t)) k, in float64, with error bounds that follow
from the roundings the kernels document (unit roundoff eps / 2: bf16 2^-8, f16 2^-11, fp32 2^-24).
"""
from __future__ import annotations

import numpy as np
import torch

from position_agnostic_paged_b200 import lazy_attn as la

D, BLK = 128, 16
U_BF16, U_F16 = 2.0 ** -8, 2.0 ** -11


def e4m3(codes: np.ndarray) -> np.ndarray:
    return torch.from_numpy(codes).view(torch.float8_e4m3fn).to(torch.float64).numpy()


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Codes of x (rounded to float32, then to nearest even; +-448 beyond the range)."""
    f = np.clip(np.asarray(x, np.float64), -448.0, 448.0).astype(np.float32)
    return torch.from_numpy(f).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def bf16(x) -> torch.Tensor:
    return torch.as_tensor(np.ascontiguousarray(x)).to(torch.float32).to(torch.bfloat16)


def theta_of(cfg: la.Cfg) -> np.ndarray:
    if cfg.alibi_slopes is not None:
        return np.zeros(D // 2)
    if cfg.rope_theta is not None:
        return np.array(cfg.rope_theta, np.float64)
    return np.float64(np.float32(cfg.rope_base)) ** (-2.0 * np.arange(D // 2) / D)


def rotate(x: np.ndarray, pos, theta: np.ndarray) -> np.ndarray:
    a = np.asarray(pos, np.float64)[..., None] * theta
    c, s = np.cos(a), np.sin(a)
    lo, hi = x[..., :D // 2], x[..., D // 2:]
    return np.concatenate([lo * c - hi * s, hi * c + lo * s], -1)


class PoolCase:
    """docs: token counts; requests: list of (segments [(document, offset)], first query position, queries)."""

    def __init__(self, cfg: la.Cfg, docs, requests, seed=0, q8=True, spare=3, k_exp=(-2, 3), v_exp=(-3, 4), q_scale=1.0):
        self.cfg, self.q8 = cfg, q8
        rng = np.random.default_rng([seed, 77])
        hkv = cfg.num_kv_heads
        nb_doc = [-(-n // BLK) for n in docs]
        nb = sum(nb_doc) + spare
        phys = rng.permutation(nb)
        first = np.concatenate([[0], np.cumsum(nb_doc)]).astype(int)
        self.num_blocks = nb
        self.meta = np.zeros(nb, np.int64)
        self.doc_blocks = []
        for d, n in enumerate(docs):
            ids = phys[first[d]:first[d + 1]]
            self.doc_blocks.append(ids)
            for i, b in enumerate(ids):
                self.meta[b] = i << 8 | min(BLK, n - i * BLK)
        valid = np.arange(BLK) < (self.meta & 255)[:, None]                  # [nb, 16]
        shape = (nb, hkv, BLK, D)
        if q8:
            self.k_codes = to_e4m3(rng.standard_normal(shape) * 100)
            self.v_codes = to_e4m3(rng.standard_normal(shape) * 100)
            self.k_scale = (2.0 ** rng.integers(k_exp[0], k_exp[1], (nb, hkv)) / 64).astype(np.float32)
            self.v_scale = (2.0 ** rng.integers(v_exp[0], v_exp[1], (nb, hkv)) / 64).astype(np.float32)
            hole = np.broadcast_to(~valid[:, None, :, None], shape)
            self.k_codes[hole] = 0x7F                                         # NaN
            self.v_codes[hole] = 0xFF
        else:
            k = rng.standard_normal(shape) * 2.0 ** rng.integers(*k_exp, (nb, hkv, 1, 1))
            v = rng.standard_normal(shape) * 2.0 ** rng.integers(*v_exp, (nb, hkv, 1, 1))
            self.k_pool, self.v_pool = bf16(k), bf16(v)
            hole = torch.from_numpy(np.broadcast_to(~valid[:, None, :, None], shape).copy())
            self.k_pool[hole] = float("nan")
            self.v_pool[hole] = float("inf")
        words, self.indptr, pos0, cu = [], [0], [], [0]
        for segs, p0, n in requests:
            for d, off in segs:
                words += [la_pack(b, off) for b in self.doc_blocks[d]]
            self.indptr.append(len(words))
            pos0.append(p0)
            cu.append(cu[-1] + n)
        self.words = np.array(words, np.uint32)
        self.q_pos0, self.cu = np.array(pos0, np.int32), np.array(cu, np.int32)
        self.q = bf16(rng.standard_normal((cu[-1], cfg.num_q_heads, D)) * q_scale)
        self.max_words = max(1, int(np.diff(self.indptr).max(initial=0)))

    # ------------------------------------------------------------------ device side
    def to(self, dev="cuda"):
        t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(dt))).to(dev)          # noqa: E731
        self.dev = dict(meta=t(self.meta, np.int32), table=t(self.words.view(np.int32), np.int32),
                        indptr=t(self.indptr, np.int32), pos0=t(self.q_pos0, np.int32), cu=t(self.cu, np.int32),
                        q=self.q.to(dev), status=torch.zeros(1, dtype=torch.int32, device=dev))
        if self.q8:
            self.pool = la.Q8Pool(t(self.k_codes, np.uint8), t(self.v_codes, np.uint8), t(self.k_scale, np.float32),
                                  t(self.v_scale, np.float32), self.dev["meta"])
        else:
            self.kv = (self.k_pool.to(dev), self.v_pool.to(dev))
        return self

    def ws(self, n):
        return torch.empty(max(int(n), 16), dtype=torch.uint8, device=self.dev["q"].device)

    def decode(self, mass=None, out=None, ws=None, max_words=None, stream=None):
        """One step with each request's first query; returns the output tensor."""
        d, mw = self.dev, self.max_words if max_words is None else max_words
        out = torch.full_like(d["q"], 7.0) if out is None else out
        n = self.q_pos0.size
        if self.q8:
            ws = self.ws(la.decode_q8_workspace_bytes(self.cfg, n, mw, mass is not None)) if ws is None else ws
            la.decode_attn_q8(self.cfg, d["q"], d["pos0"], d["table"], d["indptr"], mw, self.pool, out, ws, mass,
                              d["status"], stream)
        else:
            ws = self.ws(la.decode_mass_workspace_bytes(self.cfg, n, mw)) if ws is None else ws
            la.decode_attn_mass(self.cfg, d["q"], d["pos0"], d["table"], d["indptr"], mw, d["meta"], *self.kv, out, mass,
                                ws, d["status"], stream)
        return out

    def prefill(self, out=None, ws=None, stream=None):
        d = self.dev
        out = torch.full_like(d["q"], 7.0) if out is None else out
        n, mq = self.q_pos0.size, max(1, int(np.diff(self.cu).max(initial=0)))
        if ws is None:
            ws = self.ws(la.prefill_q8_workspace_bytes(self.cfg, n, out.shape[0], mq, self.max_words, self.words.size))
        la.prefill_attn_q8(self.cfg, d["q"], d["cu"], d["pos0"], mq, d["table"], d["indptr"], self.max_words, self.pool,
                           out, ws, d["status"], stream)
        return out

    # ------------------------------------------------------------------ 64-bit values
    def reference(self, u_qk=U_F16, u_p=U_F16):
        """(out, bound on |kernel's out - out|, mass, bound on |kernel's mass - mass|) of one call.

        The score error: roundings of the rotated query (and key) to u_qk, and 2^-16 for the fp32
        steps (angles to 2^-20, 128 products summed in fp32), relative to
        S = max over keys of scale sum over pairs (|q_a| + |q_b|) (|k_a| + |k_b|), which bounds
        scale sum |q_d k_d| under any rotation.  A score error of e changes a weight by a factor within
        exp(+-2 e); the weights are rounded to u_p (below the smallest normal f16: 2^-24 of the largest),
        the output to bf16.  Block mass uses unrounded fp32 weights of a query in two f16 or three
        bf16 parts: 2^-16 again, and 2^-17 for the logarithms (2^-22 of numbers up to 32)."""
        cfg = self.cfg
        hq, hkv = cfg.num_q_heads, cfg.num_kv_heads
        G = hq // hkv
        scale = cfg.softmax_scale if cfg.softmax_scale > 0 else 1.0 / np.sqrt(D)
        th = theta_of(cfg)
        out = np.zeros((self.q.shape[0], hq, D))
        bound = np.zeros_like(out)
        mass = np.zeros(self.words.size)
        mbound = np.zeros(self.words.size)
        qf = self.q.double().numpy()
        for r in range(self.q_pos0.size):
            w = self.words[self.indptr[r]:self.indptr[r + 1]].astype(np.int64)
            blk, off = w % (1 << 17), w >> 17
            ok = blk < self.num_blocks
            blk = np.where(ok, blk, 0)
            meta = np.where(ok, self.meta[blk], 0)
            pos = (off + (meta >> 8) * BLK)[:, None] + np.arange(BLK)
            live = np.arange(BLK) < (meta & 255)[:, None]
            if self.q8:
                k = e4m3(self.k_codes[blk]) * self.k_scale[blk].astype(np.float64)[..., None, None]
                v = e4m3(self.v_codes[blk]) * self.v_scale[blk].astype(np.float64)[..., None, None]
            else:
                k, v = self.k_pool[blk].double().numpy(), self.v_pool[blk].double().numpy()
            n = self.cu[r + 1] - self.cu[r]
            for i in range(n):
                p = int(self.q_pos0[r]) + i
                sees = live & (pos <= p)
                if not sees.any():
                    continue
                wi, sl = np.nonzero(sees)
                for h in range(hkv):
                    kk, vv = k[wi, h, sl], v[wi, h, sl]                          # [t, D]
                    t_off = off[wi]
                    q = qf[self.cu[r] + i, h * G:(h + 1) * G]                    # [G, D]
                    # rotating the key by its offset and the query by its position, both relative to p
                    kr = rotate(kk, t_off - p, th)
                    s = scale * q @ kr.T                                          # [G, t]
                    if cfg.alibi_slopes is not None:
                        sl_h = np.array(cfg.alibi_slopes[h * G:(h + 1) * G])
                        s = s - sl_h[:, None] * (p - pos[wi, sl])
                    qm, km = np.abs(q[:, :64]) + np.abs(q[:, 64:]), np.abs(kk[:, :64]) + np.abs(kk[:, 64:])
                    S = scale * (qm @ km.T).max(1)                                # [G]
                    if cfg.alibi_slopes is not None:
                        S = S + np.abs(sl_h) * np.abs(p - pos[wi, sl]).max()      # its fp32 rounding
                    e = np.exp(s - s.max(1, keepdims=True))
                    w_ = e / e.sum(1, keepdims=True)
                    o, A = w_ @ vv, w_ @ np.abs(vv)
                    row = self.cu[r] + i
                    out[row, h * G:(h + 1) * G] = o
                    de = np.expm1(2 * S * (u_qk + 2.0 ** -16))[:, None]
                    tiny = len(wi) * 2.0 ** -24 * np.abs(vv).max(0)
                    bound[row, h * G:(h + 1) * G] = 1.02 * ((de + u_p) * A + tiny + U_BF16 * np.abs(o)) + 1e-30
                    m = np.zeros((G, w.size))
                    for g in range(G):
                        np.add.at(m[g], wi, w_[g])
                    mass[self.indptr[r]:self.indptr[r + 1]] += m.sum(0)
                    dm = np.expm1(2 * S * 2.0 ** -16 + 2.0 ** -16)
                    mbound[self.indptr[r]:self.indptr[r + 1]] += (m * dm[:, None]).sum(0) + 1e-30
        return out, bound, mass, mbound


def la_pack(block: int, offset: int) -> int:
    return int(offset) << 17 | int(block)


def check(got: torch.Tensor, ref: np.ndarray, bound: np.ndarray, what: str, rel: float = 5e-3) -> None:
    """Every element within its bound, and the whole within `rel` in the 2-norm.  The bounds add all
    roundings up at their worst; in the 2-norm they average: a uniform rounding error is its largest value
    over sqrt(3), 2.3e-3 for the bf16 output, and 2^-11 / sqrt(3) per product of a score, so that scores
    with standard deviation up to about 8 are off by up to 2e-3 and the weights with them."""
    from tests._report import record
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    err = np.abs(g - ref)
    if err.size:
        rl = float(np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-30))
        record(what, float(err.max()), rl, float(bound.max()), rel)
    worst = float((err - bound).max(initial=-1.0))
    assert worst <= 0, f"{what}: {int((err > bound).sum())} of {err.size} beyond their bounds, by {worst:.3e} at most"
    assert not err.size or rl <= rel, f"{what}: rel_l2 {rl:.3e}"


def write_reference(cfg, state: dict, k_raw, v_raw, slot, j) -> dict:
    """The pool after lazy_kv_write_q8: codes and scales of state (k_codes, v_codes, k_scale, v_scale, meta)."""
    nb = state["meta"].size
    th = theta_of(cfg)
    x = {"k": rotate(k_raw.double().numpy(), np.asarray(j)[:, None], th), "v": v_raw.double().numpy()}
    out = {n: a.copy() for n, a in state.items()}
    touched, tok = {}, {}
    for t, (s, jj) in enumerate(zip(slot, j)):
        if not (0 <= s < nb * BLK) or jj < 0 or s % BLK != jj % BLK:
            continue
        touched[s // BLK] = max(touched.get(s // BLK, 0), jj // BLK << 8 | s % BLK + 1)
        tok.setdefault(s // BLK, {})[s % BLK] = t
    for b, m in touched.items():
        nv = int(state["meta"][b]) & 255
        ts = np.array([tok[b].get(s, -1) for s in range(BLK)])
        for n in "kv":
            for h in range(cfg.num_kv_heads):
                new = x[n][ts[ts >= 0], h]
                amax = np.abs(new[np.isfinite(new)]).max(initial=0.0)
                need = 2.0 ** -126
                if amax > 448 * need:
                    need = 2.0 ** np.ceil(np.log2(amax / 448))
                    if need / 2 * 448 >= amax:
                        need /= 2
                old = float(state[n + "_scale"][b, h])
                sc = max(old, need) if nv > 0 else need
                codes = out[n + "_codes"][b, h]
                if nv > 0 and sc != old:
                    stay = (np.arange(BLK) < nv) & (ts < 0)
                    codes[stay] = to_e4m3(e4m3(codes[stay]) * (old / sc))
                with np.errstate(invalid="ignore"):
                    codes[ts >= 0] = to_e4m3(new / sc)
                out[n + "_scale"][b, h] = sc
        out["meta"][b] = max(int(state["meta"][b]), m)
    return out


def evict_reference(words, indptr, max_words, mass, keep, n_first, n_last):
    """(table, indptr, mass, evicted) after lazy_evict_blocks, as lists."""
    table, ind, m_out, gone = [], [0], [], []
    for r in range(len(keep)):
        w, m = words[indptr[r]:indptr[r + 1]], mass[indptr[r]:indptr[r + 1]]
        n = min(len(w), max_words)
        key = [(0 if i < n_first or i >= n - n_last else 1, -(np.inf if np.isnan(m[i]) else float(m[i])), i) for i in range(n)]
        best = {i for *_, i in sorted(key)[:max(0, int(keep[r]))]}
        table += [w[i] for i in range(n) if i in best]
        m_out += [m[i] for i in range(n) if i in best]
        gone += [w[i] for i in range(len(w)) if i not in best]
        ind.append(len(table))
    return table, ind, m_out, gone
