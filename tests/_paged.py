"""Plain 64-bit forms of the paged cache's writer and attentions, and their cases, for the tests."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests import _quant as Q

SENTINEL = -123.0
JUNK = (-1, 1 << 30, -(1 << 31), 777777)  # page numbers where no call looks


def visible(pos, n, window):
    """[R, n] truth values: which keys the rows at `pos` see. window None, or (left, right, sinks)."""
    j = np.arange(n)[None, :]
    if window is None:
        return np.ones((len(pos), n), bool)
    left, right, sinks = window
    p = np.asarray(pos, np.int64)[:, None]
    see = np.ones((len(pos), n), bool)
    if left >= 0:
        see &= j >= p - left
    if right >= 0:
        see &= j <= p + right
    return see | (j < sinks)


def attention(q, k, v, scale, see):
    """float64 softmax(scale q k^T) v over the keys that see [R, n] names, q [R, Hq, D], k, v [n, Hkv, D], zeros
    for a row without one, and the bound of the kernel's error, which is that of _quant.attention: weights and
    result rounded to bf16 (2^-8 each of A = sum_j p_j |v_j|), 2^-10 A for the second order, the approximate
    exponential and the sums, and 2 delta A for the scores' fp32 products, delta = D 2^-23 max_j scale sum_d |q_d k_jd|."""
    R, Hq, D = q.shape
    g = Hq // k.shape[1]
    out, tol = np.zeros((R, Hq, D)), np.zeros((R, Hq, D))
    some = see.any(1)
    if k.shape[0] == 0 or not some.any():
        return out, tol
    hide = ~see[some]
    for h in range(Hq):
        used = see.any(0)[:, None]  # what no row sees may hold anything
        kk, vv = np.where(used, k[:, h // g], 0.0), np.where(used, v[:, h // g], 0.0)
        z = scale * (q[some, h] @ kk.T)
        z[hide] = -np.inf
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        mag = scale * (np.abs(q[some, h]) @ np.abs(kk).T)
        mag[hide] = 0.0
        delta = D * 2.0**-23 * mag.max(1, keepdims=True)
        out[some, h] = p @ vv
        tol[some, h] = (2.0**-7 + 2.0**-10 + 2 * delta) * (p @ np.abs(vv)) + 1e-30
    return out, tol


def rotate(x, cs, sn):
    """float64 rows x [n, H, D] turned by angles with cosines and sines [n, D / 2] (fp32 values), and the error bound:
    two fp32 products and their sum (2^-22 of the terms), one rounding to bf16 (2^-8)."""
    h = x.shape[-1] // 2
    a, b, c, s = x[..., :h], x[..., h:], cs[:, None, :].astype(np.float64), sn[:, None, :].astype(np.float64)
    y = np.concatenate([a * c - b * s, b * c + a * s], -1)
    terms = np.concatenate([np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)], -1)
    return y, 2.0**-8 * np.abs(y) + 2.0**-21 * terms + 1e-37


class Pool:
    """Pages and tables on the CPU for sequences of up to `lens` positions: dense float64 rows k, v [B, L, Hkv, D] lie
    in pages handed out in no order, every other row of the pool is `fill`. kind "split": two arrays; "one": a pool
    [n_pages, 2, page, Hkv, D] of both; "wide": pages with a gap between them and tables that are rows of a
    larger array."""

    def __init__(self, rng, B, L, Hkv, D, page, lens, kind="split", fill=float("nan"), spare=2, only=None):
        self.page, self.kind, self.B, self.L, self.Hkv, self.D = page, kind, B, L, Hkv, D
        self.lens = lens
        per = -(-L // page)
        need = [[i for i in range(-(-n // page)) if only is None or only(b, i)] for b, n in enumerate(lens)]
        self.n_pages = max(1, sum(map(len, need))) + spare
        order = rng.permutation(self.n_pages)
        self.table = rng.choice(np.array(JUNK, np.int64), size=(B, per)).astype(np.int32)
        at = 0
        for b, pages in enumerate(need):
            for i in pages:
                self.table[b, i] = order[at]
                at += 1
        self.k = np.full((self.n_pages, page, Hkv, D), fill)
        self.v = self.k.copy()
        self.need = need

    def put(self, k, v):
        """Rows [B, L, Hkv, D] of every position below its sequence's length that has a page."""
        for b, n in enumerate(self.lens):
            for i in self.need[b]:
                m = min(self.page, n - i * self.page)
                self.k[self.table[b, i], :m] = k[b, i * self.page : i * self.page + m]
                self.v[self.table[b, i], :m] = v[b, i * self.page : i * self.page + m]

    def device(self, E, device="cuda"):
        k, v = Q.bf16(self.k), Q.bf16(self.v)
        t = torch.from_numpy(self.table)
        if self.kind == "one":
            pool = torch.stack([k, v], 1).to(device)
            k, v = pool[:, 0], pool[:, 1]
        elif self.kind == "wide":
            wide = [torch.full((self.n_pages, x[0].numel() + 24), float("nan"), dtype=torch.bfloat16) for x in (k, v)]
            for w, x in zip(wide, (k, v)):
                w[:, : x[0].numel()] = x.reshape(self.n_pages, -1)
            k, v = (w.to(device)[:, : x[0].numel()].unflatten(1, x.shape[1:]) for w, x in zip(wide, (k, v)))
            big = torch.full((self.B, t.shape[1] + 5), 12345, dtype=torch.int32)
            big[:, : t.shape[1]] = t
            return E.PagedCache(k, v, big.to(device)[:, : t.shape[1]])
        else:
            k, v = k.to(device), v.to(device)
        return E.PagedCache(k, v, t.to(device))


def places(rng, R, n, L, kind):
    """Row positions of one sequence: idx ascending, scattered over [0, n) or up to L; or None with a start."""
    hi = max(1, min(L, n))
    if R <= hi:
        return np.sort(rng.choice(hi, size=R, replace=False)).astype(np.int64)
    return np.arange(R, dtype=np.int64)


class Case:
    """Inputs on the CPU, and the library's call and the 64-bit result on them. at: "idx", "start" or None."""

    def __init__(self, B, L, Hq, Hkv, D, page, Rs, lens=None, window=None, at="idx", rows=None, kind="split", seed=0, q_scale=1.0,
                 scale=None, pos=None, fill=float("nan"), scope=0):
        rng = np.random.default_rng(seed)
        self.B, self.L, self.Hq, self.Hkv, self.D, self.Rs, self.window, self.at = B, L, Hq, Hkv, D, Rs, window, at
        self.lens, self.scope = lens, scope
        self.rows = max(1, max(Rs)) if rows is None else rows
        self.scale = Q.default_scale(D) if scale is None else scale
        ns = [min(n, scope) if scope else n for n in (lens if lens is not None else [L] * B)]
        self.ns = ns
        self.q = Q.bf16(rng.standard_normal((B, self.rows, Hq, D)) * q_scale)
        self.k = Q.f64(Q.bf16(rng.standard_normal((B, L, Hkv, D))))
        self.v = Q.f64(Q.bf16(rng.standard_normal((B, L, Hkv, D)) * 2.0 ** (0.5 * rng.standard_normal((B, L, Hkv, 1)))))
        if at == "idx":
            self.pos = [places(rng, r, n, L, at) for r, n in zip(Rs, ns)] if pos is None else pos
        elif at == "start":
            self.start = [max(0, min(L, n) - r) for r, n in zip(Rs, ns)] if pos is None else pos
            self.pos = [s + np.arange(r) for s, r in zip(self.start, Rs)]
        else:
            self.pos = [np.arange(r) for r in Rs]
        # only pages that some row may look at exist: the rest of the table is junk, the rest of the pool `fill`
        self.pool = Pool(rng, B, L, Hkv, D, page, ns, kind, fill, only=self._looks(page))
        self.pool.put(self.k, self.v)
        if window is not None:  # rows of a page that no row sees hold junk too
            for b, n in enumerate(ns):
                lo, hi, s = self._hull(b)
                for j in range(n):
                    if not (j < s or lo <= j < hi) and j // page in self.pool.need[b]:
                        for x in (self.pool.k, self.pool.v):
                            x[self.pool.table[b, j // page], j % page] = fill

    def _hull(self, b):
        n, (left, right, sinks) = self.ns[b], self.window
        if len(self.pos[b]) == 0:
            return 0, 0, 0
        lo = 0 if left < 0 else max(0, int(self.pos[b][0]) - left)
        hi = n if right < 0 else min(n, int(self.pos[b][-1]) + right + 1)
        return lo, hi, min(n, sinks)

    def _looks(self, page):
        if self.window is None:
            return None

        def only(b, i):
            lo, hi, s = self._hull(b)
            return i * page < s or (i * page < hi and (i + 1) * page > lo)

        return only

    def params(self, E):
        return E.Params(B=self.B, L=self.L, Hq=self.Hq, Hkv=self.Hkv, D=self.D, V=8, C_max=1, k=1, scope_lo=0, scope_hi=self.scope)

    def inputs(self, E):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        d = dict(p=self.params(E), q=self.q.cuda(), cache=self.pool.device(E), R=i32(self.Rs),
                 out=torch.full((self.B, self.rows, self.Hq, self.D), SENTINEL, dtype=torch.bfloat16, device="cuda"),
                 kv_len=None if self.lens is None else i32(self.lens), dev_err=torch.zeros(1, dtype=torch.int32, device="cuda"))
        if self.window is not None and self.at == "idx":
            idx = np.full((self.B, self.rows + 3), 1 << 29, np.int32)  # rows of a wider array
            for b, x in enumerate(self.pos):
                idx[b, : len(x)] = x
            d["idx"] = i32(idx)[:, : self.rows]
        if self.window is not None and self.at == "start":
            d["start"] = i32(self.start)
        return d

    def call(self, E, d, **kw):
        kw = dict(dict(kv_len=d["kv_len"], scale=self.scale, dev_err=d["dev_err"]), **kw)
        if self.window is None:
            return E.paged_attention(d["p"], d["q"], d["cache"], d["R"], d["out"], **kw)
        left, right, sinks = self.window
        return E.paged_window_attention(d["p"], d["q"], d["cache"], d["R"], d["out"], left=left, right=right, sinks=sinks, idx=d.get("idx"),
                                        start=d.get("start"), **kw)

    def check(self, got, skip=(), lost=()):
        """skip: sequences that are not written; lost: (sequence, row) pairs that are not."""
        got = Q.f64(got)
        for b, r in enumerate(self.Rs):
            if b in skip:
                assert (got[b] == SENTINEL).all()
                continue
            n = self.ns[b]
            want, tol = attention(Q.f64(self.q[b, :r]), self.k[b, :n], self.v[b, :n], self.scale, visible(self.pos[b], n, self.window))
            off = np.abs(got[b, :r] - want) - tol
            for x, i in lost:
                if x == b:
                    assert (got[b, i] == SENTINEL).all()
                    off[i] = 0
            assert not (off > 0).any() and not np.isnan(off).any(), (b, np.nanmax(off), np.argwhere(~(off <= 0))[:3])
            assert (got[b, r:] == SENTINEL).all(), "rows at and past R were written"

    def run(self, E, **kw):
        d = self.inputs(E)
        self.call(E, d, **kw)
        torch.cuda.synchronize()
        assert int(d["dev_err"].item()) == 0, hex(int(d["dev_err"].item()))
        self.check(d["out"])
        return d


def table_of(L, D, theta=10000.0):
    a = np.arange(L)[:, None] * theta ** (-np.arange(0, D, 2) / D)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def default_scale(D):
    return 1.0 / math.sqrt(D)
