"""GPU tests of rows written into a paged cache with the rotation on the way, and of a run of the operators together as a
denoising loop uses them."""
import numpy as np
import pytest
import torch

import oracle as O
from tests import _paged as P
from tests import _quant as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import entropy_gated_kv_gb300 as E

    E.lib()
    return E


class Append:
    def __init__(self, B, L, Hq, Hkv, D, page, Rs, at, rows=None, kind="split", seed=0, fused=False):
        rng = np.random.default_rng(seed)
        self.B, self.L, self.Hq, self.Hkv, self.D, self.Rs, self.at = B, L, Hq, Hkv, D, Rs, at
        self.rows = max(1, max(Rs)) if rows is None else rows
        self.pool = P.Pool(rng, B, L, Hkv, D, page, [L] * B, kind, fill=P.SENTINEL)
        self.cs, self.sn = P.table_of(L, D)
        H = Hq + 2 * Hkv
        self.x = Q.bf16(rng.standard_normal((B, self.rows, H, D)))
        if not fused:
            self.parts = [t.contiguous().cuda() for t in self.x.split([Hq, Hkv, Hkv], 2)]
        else:
            self.parts = list(self.x.cuda().split([Hq, Hkv, Hkv], 2))
        if at == "start":
            self.start = [int(rng.integers(0, L - r + 1)) for r in Rs]
            self.pos = [s + np.arange(r) for s, r in zip(self.start, Rs)]
        elif at == "idx":
            self.pos = [np.sort(rng.choice(L, size=r, replace=False)) for r in Rs]
        else:
            self.pos = [np.arange(r) for r in Rs]

    def inputs(self, E):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        d = dict(cache=self.pool.device(E), R=i32(self.Rs), dev_err=torch.zeros(1, dtype=torch.int32, device="cuda"),
                 p=E.Params(B=self.B, L=self.L, Hq=self.Hq, Hkv=self.Hkv, D=self.D, V=8, C_max=1, k=1),
                 q_out=torch.full((self.B, self.rows, self.Hq, self.D), P.SENTINEL, dtype=torch.bfloat16, device="cuda"),
                 rope=(torch.from_numpy(self.cs).cuda(), torch.from_numpy(self.sn).cuda()), idx=None, start=None)
        if self.at == "idx":
            idx = np.full((self.B, self.rows + 2), -7, np.int32)
            for b, x in enumerate(self.pos):
                idx[b, : len(x)] = x
            d["idx"] = i32(idx)[:, : self.rows]
        if self.at == "start":
            d["start"] = i32(self.start)
        return d

    def call(self, E, d, queries=True, **kw):
        q, k, v = self.parts
        more = dict(q_new=q, q_out=d["q_out"]) if queries else {}
        return E.kv_append_paged(d["p"], d["cache"], k, v, d["R"], idx=d["idx"], start=d["start"], rope=d["rope"], dev_err=d["dev_err"],
                                 **more, **kw)

    def check(self, d, rotated=True, queries=True, skip=(), lost=()):
        """skip: sequences, lost: (sequence, row) pairs that are not written at all."""
        k0, v0 = self.pool.k.copy(), self.pool.v.copy()
        tol_k = np.zeros_like(k0)
        got_q = Q.f64(d["q_out"])
        Hq, Hkv, page = self.Hq, self.Hkv, self.pool.page
        for b, r in enumerate(self.Rs):
            x = Q.f64(self.x[b])
            seen = np.zeros(self.rows, bool)
            for i in range(r):
                if b in skip or (b, i) in lost:
                    continue
                seen[i] = True
                pos = int(self.pos[b][i])
                at = (self.pool.table[b, pos // page], pos % page)
                y, t = P.rotate(x[i : i + 1], self.cs[pos : pos + 1], self.sn[pos : pos + 1])
                if not rotated:
                    y, t = x[i : i + 1], np.zeros_like(t)
                k0[at], tol_k[at] = y[0, Hq : Hq + Hkv], t[0, Hq : Hq + Hkv]
                v0[at] = x[i, Hq + Hkv :]
                if queries:
                    assert (np.abs(got_q[b, i] - y[0, :Hq]) <= t[0, :Hq]).all(), (b, i)
            untouched = ~seen if queries else np.ones(self.rows, bool)
            assert (got_q[b, untouched] == P.SENTINEL).all()
        assert (np.abs(Q.f64(d["cache"].k) - k0) <= tol_k).all()
        assert (Q.f64(d["cache"].v) == v0).all()


CASES = [
    # B, L, Hq, Hkv, D, page, rows
    (1, 1, 1, 1, 64, 16, [1]),
    (1, 300, 8, 8, 64, 16, [47]),
    (1, 300, 28, 4, 128, 32, [1]),
    (32, 40, 28, 4, 128, 16, [1] * 32),
    (3, 500, 14, 2, 128, 64, [95, 0, 500]),
    (2, 1000, 32, 32, 128, 1024, [1000, 17]),
    (40, 70, 3, 1, 64, 16, [(7 * b) % 71 for b in range(40)]),
    (2, 30, 5, 5, 128, 16, [30, 1]),
    (1, 20, 256, 128, 64, 16, [20]),            # more pieces in a row than threads in a CTA
]


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("at", ["idx", "start", None])
@pytest.mark.parametrize("B,L,Hq,Hkv,D,page,Rs", CASES)
def test_append(E, B, L, Hq, Hkv, D, page, Rs, at, fused):
    c = Append(B, L, Hq, Hkv, D, page, Rs, at, seed=L, fused=fused)
    d = c.inputs(E)
    c.call(E, d)
    torch.cuda.synchronize()
    assert int(d["dev_err"].item()) == 0
    c.check(d)


@pytest.mark.parametrize("kind", ["one", "wide"])
def test_pools(E, kind):
    c = Append(3, 200, 6, 2, 128, 16, [95, 1, 200], "idx", kind=kind, seed=1)
    d = c.inputs(E)
    c.call(E, d)
    c.check(d)


def test_without_rotation_or_queries(E):
    c = Append(2, 200, 6, 2, 128, 32, [95, 40], "idx", seed=2)
    d = c.inputs(E)
    d["rope"] = None
    c.call(E, d)
    c.check(d, rotated=False)
    d = c.inputs(E)
    assert c.call(E, d, queries=False) is None
    c.check(d, queries=False)


def test_new_query_array_and_stream(E):
    c = Append(2, 200, 6, 2, 64, 32, [95, 40], "start", seed=3)
    d = c.inputs(E)
    q, k, v = c.parts
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = E.kv_append_paged(d["p"], d["cache"], k, v, d["R"], start=d["start"], rope=d["rope"], q_new=q, stream=s)
    s.synchronize()
    assert (out[1, 40:] == 0).all()
    d["q_out"][0], d["q_out"][1, :40] = out[0], out[1, :40]
    c.check(d)


def test_values_keep_their_bits(E):
    """NaN payloads, infinities and subnormal values of V, and of K without a rotation."""
    c = Append(1, 64, 2, 2, 64, 16, [64], None, seed=4)
    bits = torch.randint(-(1 << 15), 1 << 15, (1, 64, 2, 64), dtype=torch.int16, generator=torch.Generator().manual_seed(1))
    c.parts[1] = bits.view(torch.bfloat16).cuda()
    c.parts[2] = bits.flip(1).view(torch.bfloat16).cuda()
    d = c.inputs(E)
    d["rope"] = None
    c.call(E, d)
    t = d["cache"].table[0].long()
    for got, want in ((d["cache"].k, c.parts[1]), (d["cache"].v, c.parts[2])):
        assert torch.equal(got[t].reshape(64, 2, 64).view(torch.int16), want[0].view(torch.int16))


def test_bad_rows_are_skipped(E):
    C = E._capi
    c = Append(3, 200, 6, 2, 128, 16, [20, 20, 20], "idx", rows=24, seed=5)
    d = c.inputs(E)
    d["R"][1] = 25
    c.call(E, d)
    torch.cuda.synchronize()
    assert int(d["dev_err"].item()) == C.EC_DEVERR_BAD_R
    c.check(d, skip=(1,))
    d = c.inputs(E)
    d["idx"][0, 19] = 200
    d["idx"][1, 0] = -1
    d["idx"][2, 7] = d["idx"][2, 8]  # a position given twice: the first of the two is skipped
    c.call(E, d)
    torch.cuda.synchronize()
    assert int(d["dev_err"].item()) == C.EC_DEVERR_BAD_IDX
    c.check(d, lost=((0, 19), (1, 0), (2, 7)))


def test_bad_starts(E):
    C = E._capi
    c = Append(3, 64, 2, 2, 64, 16, [4, 4, 4], "start", seed=6)
    for bad in (-4, -(1 << 31), (1 << 31) - 1, 64):
        d = c.inputs(E)
        d["start"][1] = bad
        c.call(E, d)
        torch.cuda.synchronize()
        assert int(d["dev_err"].item()) == C.EC_DEVERR_BAD_IDX
        c.check(d, skip=(1,))


def test_bad_pages_keep_the_pool(E):
    C = E._capi
    c = Append(2, 64, 2, 2, 64, 16, [64, 64], None, seed=7)
    d = c.inputs(E)
    for b, i, bad in ((0, 1, -1), (1, 3, c.pool.n_pages)):
        d["cache"].table[b, i] = bad
    c.call(E, d)
    torch.cuda.synchronize()
    assert int(d["dev_err"].item()) == C.EC_DEVERR_BAD_PAGE
    # the rows of the two pages are lost, their queries are not
    got = d["q_out"].clone()
    for b, i in ((0, 1), (1, 3)):
        d["q_out"][b, i * 16 : (i + 1) * 16] = P.SENTINEL
    c.check(d, lost=[(0, r) for r in range(16, 32)] + [(1, r) for r in range(48, 64)])
    assert not (got == P.SENTINEL).all(-1).any()


def test_graph_replay(E):
    c = Append(3, 200, 6, 2, 128, 16, [20, 5, 11], "idx", rows=24, seed=8)
    d = c.inputs(E)
    c.call(E, d)  # the first launch outside a capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(E, d)
    other = Append(3, 200, 6, 2, 128, 16, [24, 0, 3], "idx", rows=24, seed=9)
    od = other.inputs(E)
    for x, y in zip(c.parts, other.parts):
        x.copy_(y)
    for n in ("R", "idx", "q_out"):
        d[n].copy_(od[n])
    for n in ("k", "v", "table"):
        getattr(d["cache"], n).copy_(getattr(od["cache"], n))
    g.replay()
    torch.cuda.synchronize()
    other.check(d)


def test_denoising_loop(E):
    """A batch of sequences in pages, as a decoding loop runs them: the prompts' rows in one call, then steps whose recompute
    set ec_select_recompute leaves (st.idx, st.R), each refreshed and attended to; every step against a dense 64-bit cache."""
    B, L, Hq, Hkv, D, V, C_max, k, page = 3, 192, 8, 2, 64, 512, 16, 24, 16
    rng = np.random.default_rng(12)
    p = E.Params(B=B, L=L, Hq=Hq, Hkv=Hkv, D=D, V=V, C_max=C_max, k=k, tau=100.0, logits_dtype="f32")
    st = E.DecodeState(p)
    prompt = [176, 170, 160]
    mask = np.zeros((B, L), np.uint8)
    for b, n in enumerate(prompt):
        mask[b, n:] = 1
    st.mask.copy_(torch.from_numpy(mask))
    per = L // page
    table = torch.from_numpy(rng.permutation(B * per).astype(np.int32).reshape(B, per)).cuda()
    cache = E.PagedCache.empty(B * per, page, Hkv, D, table)
    rope = E.rope_table(L, D, 10000.0)
    cs, sn = (t.cpu().numpy() for t in rope)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dense = {"k": np.zeros((B, L, Hkv, D)), "v": np.zeros((B, L, Hkv, D))}

    def fresh(rows):
        return Q.bf16(rng.standard_normal((B, rows, Hq + 2 * Hkv, D)))

    def follow(x, pos):  # the dense cache: positions keep the rows that the pages hold, as their bits
        for b, ps in enumerate(pos):
            y, _ = P.rotate(Q.f64(x[b, : len(ps)]), cs[ps], sn[ps])
            dense["k"][b, ps] = y[:, Hq : Hq + Hkv]
            dense["v"][b, ps] = Q.f64(x[b, : len(ps), Hq + Hkv :])

    def pages(t):
        return Q.f64(t[table.long()].reshape(B, L, Hkv, D))

    x = fresh(max(prompt))
    dx = x.cuda()
    R = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    E.kv_append_paged(p, cache, dx[:, :, Hq : Hq + Hkv], dx[:, :, Hq + Hkv :], R, rope=rope, dev_err=err)
    follow(x, [np.arange(n) for n in prompt])
    kv_len = torch.full((B,), L, dtype=torch.int32, device="cuda")
    ws = E.workspace(E.paged_attention_workspace_size(p, L))
    for step in range(4):
        pos, count = E.candidates(p, st, "sliding", 0, C_max)
        logits = torch.from_numpy(rng.standard_normal((B * C_max, V)).astype(np.float32) * 3).cuda()
        ids, ent, conf = E.entropy_decode(logits)
        E.select_recompute(p, st, pos, count, ids, ent, conf)
        Rs = st.R.cpu().numpy()
        assert (Rs > 0).all() and (Rs < 64).all()
        rows = 64
        idx = [st.idx[b, :n].cpu().numpy() for b, n in enumerate(Rs)]
        x = fresh(rows)
        dx = x.cuda()
        q = E.kv_append_paged(p, cache, dx[:, :, Hq : Hq + Hkv], dx[:, :, Hq + Hkv :], st.R, idx=st.idx, rope=rope, q_new=dx[:, :, :Hq],
                              dev_err=err)
        follow(x, idx)
        for name in ("k", "v"):
            assert (np.abs(pages(getattr(cache, name)) - dense[name]) <= 2.0**-7 * np.abs(dense[name]) + 2.0**-18).all()
        kk, vv = pages(cache.k), pages(cache.v)
        for window in (None, (40, 12, 4)):
            out = torch.full((B, rows, Hq, D), P.SENTINEL, dtype=torch.bfloat16, device="cuda")
            if window is None:
                E.paged_attention(p, q, cache, st.R, out, kv_len=kv_len, ws=ws, dev_err=err)
            else:
                E.paged_window_attention(p, q, cache, st.R, out, *window, idx=st.idx, kv_len=kv_len, ws=ws, dev_err=err)
            got = Q.f64(out)
            for b, n in enumerate(Rs):
                want, tol = P.attention(Q.f64(q[b, :n]), kk[b], vv[b], 1 / np.sqrt(D), P.visible(idx[b], L, window))
                assert (np.abs(got[b, :n] - want) <= tol).all(), (step, window, b)
                assert (got[b, n:] == P.SENTINEL).all()
                if window is None:
                    ref = O.attention(Q.f64(q[b, :n]), kk[b], vv[b], 1 / np.sqrt(D))
                    assert np.allclose(ref, want, rtol=1e-9, atol=1e-12)
        assert int(err.item()) == 0


@pytest.mark.parametrize("R", [1, 40])
def test_append_and_attention_in_one_graph(E, R):
    """The refresh and the attention behind it, captured together and replayed: the second reads what the first has written."""
    B, L, Hq, Hkv, D, page = 2, 300, 8, 2, 128, 16
    a = Append(B, L, Hq, Hkv, D, page, [R, R], "idx", seed=R)
    d = a.inputs(E)
    for x in ("k", "v"):
        getattr(d["cache"], x).normal_()
    out = torch.full((B, R, Hq, D), P.SENTINEL, dtype=torch.bfloat16, device="cuda")
    ws = E.workspace(E.paged_attention_workspace_size(d["p"], R))

    def both():
        a.call(E, d)
        E.paged_window_attention(d["p"], d["q_out"], d["cache"], d["R"], out, 60, 60, 4, idx=d["idx"], ws=ws, dev_err=d["dev_err"])

    both()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for seed in (1, 2):
        for x in a.parts:
            x.normal_(generator=torch.Generator(device="cuda").manual_seed(seed))
        for x in ("k", "v"):
            getattr(d["cache"], x).zero_()
        g.replay()
        torch.cuda.synchronize()
        assert int(d["dev_err"].item()) == 0
        t = d["cache"].table.long()
        k, v = (Q.f64(getattr(d["cache"], x)[t].flatten(1, 2)[:, :L]) for x in ("k", "v"))
        for b in range(B):
            assert (np.abs(v[b, a.pos[b]] - Q.f64(a.parts[2][b])) == 0).all()
            want, tol = P.attention(Q.f64(d["q_out"][b]), k[b], v[b], D**-0.5, P.visible(a.pos[b], L, (60, 60, 4)))
            assert (np.abs(Q.f64(out[b]) - want) <= tol).all()


def test_append_binding_checks(E):
    c = Append(2, 64, 4, 2, 64, 16, [5, 5], "idx", rows=6, seed=1)
    d = c.inputs(E)
    q, k, v = c.parts
    p, cache, R, idx, rope = d["p"], d["cache"], d["R"], d["idx"], d["rope"]
    bad = [
        lambda: E.kv_append_paged(p, cache, k.float(), v, R),
        lambda: E.kv_append_paged(p, cache, k, v[:, :5], R),
        lambda: E.kv_append_paged(p, cache, k.cpu(), v, R),
        lambda: E.kv_append_paged(p, cache, k.transpose(2, 3).contiguous().transpose(2, 3), v, R),
        lambda: E.kv_append_paged(p, cache, k, v, R, q_out=d["q_out"]),
        lambda: E.kv_append_paged(p, cache, k, v, R, q_new=q, q_out=d["q_out"][:, :5]),
        lambda: E.kv_append_paged(p, cache, k, v, R, idx=idx, start=R),
        lambda: E.kv_append_paged(p, cache, k, v, R, rope=(rope[0][:5], rope[1])),
        lambda: E.kv_append_paged(p, cache, k, v, R, rope=(rope[0], rope[1].double())),
        lambda: E.kv_append_paged(p, cache, k, v, R.long()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    pool = cache.k.flatten()
    for f in (lambda: E.kv_append_paged(p, cache, k, v, R, q_new=q, q_out=q),
              lambda: E.kv_append_paged(p, cache, pool[: k.numel()].view_as(k), v, R)):
        with pytest.raises(E.EcError):
            f()


def test_append_of_no_rows_array(E):
    c = Append(2, 64, 4, 2, 64, 16, [5, 5], "idx", rows=6, seed=1)
    d = c.inputs(E)
    q, k, v = c.parts
    for x in (k.flatten(), k[0], k[:, 0, 0, 0], k[None]):
        with pytest.raises(ValueError):
            E.kv_append_paged(d["p"], d["cache"], x, v, d["R"])


def test_far_pages_are_written(E):
    """Rows of pages past 2^31 elements of the pool."""
    page, H, D = 1024, 2, 128
    n = (1 << 31) // (page * H * D) + 9
    k, v = (torch.empty(n, page, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[n - 1]], dtype=torch.int32, device="cuda")
    p = E.Params(B=1, L=page, Hq=H, Hkv=H, D=D, V=8, C_max=1, k=1)
    x = torch.randn(1, 7, 2 * H, D, device="cuda").to(torch.bfloat16)
    start = torch.tensor([100], dtype=torch.int32, device="cuda")
    E.kv_append_paged(p, E.PagedCache(k, v, table), x[:, :, :H], x[:, :, H:], torch.tensor([7], dtype=torch.int32, device="cuda"), start=start)
    assert torch.equal(k[n - 1, 100:107], x[0, :, :H]) and torch.equal(v[n - 1, 100:107], x[0, :, H:])
