"""GPU tests of the attentions over an 8-bit cache and over a shared prefix, element by element
against 64 bits with the bound that tests/_quant.py derives from the kernel's roundings."""
import numpy as np
import pytest
import torch

from tests import _quant as Q

pytestmark = pytest.mark.gpu

SENTINEL = -123.0


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import entropy_gated_kv_gb300 as E

    E.lib()
    return E


class Case:
    """Inputs on the CPU, and the library's call and the 64-bit result on them."""

    def __init__(self, B, L, Hq, Hkv, D, Rs, lens=None, Lp=None, quant=True, seed=0, q_scale=1.0, spread=0.5, scale=None):
        rng = np.random.default_rng(seed)
        self.B, self.L, self.Hq, self.Hkv, self.D, self.Rs, self.lens, self.Lp = B, L, Hq, Hkv, D, Rs, lens, Lp
        self.quant, self.scale, self.scope = quant, Q.default_scale(D) if scale is None else scale, 0
        self.q = Q.bf16(rng.standard_normal((B, L, Hq, D)) * q_scale)
        self.own, self.pre = self._cache(rng, B, L, spread), None
        if Lp is not None:
            self.pre = self._cache(rng, 1, Lp, spread)

    def _cache(self, rng, B, L, spread):
        if self.quant:
            return Q.random_cache(rng, B, L, self.Hkv, self.D, spread)
        return tuple(Q.bf16(rng.standard_normal((B, L, self.Hkv, self.D)) * 2.0 ** (spread * rng.standard_normal((B, L, self.Hkv, 1))))
                     for _ in range(2))

    def device_cache(self, E, t):
        t = tuple(x.cuda() for x in t)
        return E.QuantCache(t[0], t[1], t[2], t[3]) if self.quant else t

    def params(self, E):
        return E.Params(B=self.B, L=self.L, Hq=self.Hq, Hkv=self.Hkv, D=self.D, V=8, C_max=1, k=1, scope_lo=0, scope_hi=self.scope)

    def inputs(self, E):
        d = dict(p=self.params(E), q=self.q.cuda(), cache=self.device_cache(E, self.own),
                 R=torch.tensor(self.Rs, dtype=torch.int32, device="cuda"),
                 out=torch.full((self.B, self.L, self.Hq, self.D), SENTINEL, dtype=torch.bfloat16, device="cuda"),
                 kv_len=None if self.lens is None else torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                 scale=self.scale, dev_err=torch.zeros(1, dtype=torch.int32, device="cuda"))
        if self.pre is not None:
            t = self.pre if self.quant else tuple(x[0] for x in self.pre)
            d["prefix"] = self.device_cache(E, t)
        return d

    def call(self, E, d, **kw):
        f = E.prefix_attention if "prefix" in d else E.partial_attention_quant
        a = [d["p"], d["q"]] + ([d["prefix"]] if "prefix" in d else []) + [d["cache"], d["R"], d["out"]]
        return f(*a, kv_len=d["kv_len"], scale=d["scale"], dev_err=d["dev_err"], **kw)

    def _values(self, t):
        return (Q.widen(t[0], t[2]), Q.widen(t[1], t[3])) if self.quant else (Q.f64(t[0]), Q.f64(t[1]))

    def check(self, got, skip=()):
        k, v = self._values(self.own)
        pk = pv = np.zeros((0, self.Hkv, self.D))
        if self.pre is not None:
            pk, pv = (x[0] for x in self._values(self.pre))
        got = Q.f64(got)
        for b, r in enumerate(self.Rs):
            if b in skip:
                assert (got[b] == SENTINEL).all()
                continue
            n = self.L if self.lens is None else self.lens[b]
            n = min(n, self.scope) if self.scope else n
            want, tol = Q.attention(Q.f64(self.q[b, :r]), np.concatenate([pk, k[b, :n]]), np.concatenate([pv, v[b, :n]]), self.scale)
            off = np.abs(got[b, :r] - want) - tol
            assert not (off > 0).any() and np.isfinite(got[b, :r]).all(), (b, off.max(), np.argwhere(off > 0)[:3])
            assert (got[b, r:] == SENTINEL).all(), "rows at and past R were written"

    def run(self, E, **kw):
        d = self.inputs(E)
        self.call(E, d, **kw)
        torch.cuda.synchronize()
        assert int(d["dev_err"].item()) == 0
        self.check(d["out"])
        return d


QUANT = [
    # B, L, Hq, Hkv, D, rows, lengths
    (1, 256, 8, 8, 64, [47], None),
    (1, 1, 1, 1, 64, [1], None),                            # one key
    (1, 1, 1, 1, 128, [1], [0]),                            # no key: zeros
    (1, 1000, 4, 4, 128, [1], None),                        # a single token, split over the SMs
    (1, 2047, 28, 4, 128, [1], None),                       # grouped heads, odd length
    (1, 1024, 32, 32, 128, [95], None),
    (3, 300, 6, 2, 128, [5, 0, 300], [300, 17, 129]),       # an empty sequence, blocks that end inside
    (2, 512, 8, 8, 64, [129, 257], [512, 0]),               # rows past one tile, a sequence without keys
    (1, 384, 128, 1, 64, [3], None),                        # 128 heads on one KV head
    (1, 300, 96, 2, 128, [11], [200]),                      # g = 48: tiles cut between heads of a row
    (2, 140, 14, 2, 128, [140, 33], [131, 128]),            # g = 7
    (40, 70, 2, 1, 64, [(7 * b) % 5 for b in range(40)], [(11 * b) % 71 for b in range(40)]),  # more than a warp of sequences
    (1, 4000, 2, 1, 128, [3], [3999]),                      # one tile over many CTAs
    (4, 640, 16, 16, 128, [640] * 4, [640, 5, 333, 640]),   # more tiles than CTAs
]


@pytest.mark.parametrize("B,L,Hq,Hkv,D,Rs,lens", QUANT)
def test_quant_attention(E, B, L, Hq, Hkv, D, Rs, lens):
    Case(B, L, Hq, Hkv, D, Rs, lens, seed=L + B).run(E)


PREFIX = [
    # B, Lp, L, Hq, Hkv, D, rows, lengths
    (1, 1, 1, 1, 1, 128, [1], None),
    (1, 129, 5, 2, 2, 64, [5], None),
    (4, 300, 64, 8, 2, 128, [1, 1, 1, 1], None),                   # single tokens: one shared tile per head
    (5, 640, 40, 6, 3, 128, [3, 0, 40, 17, 1], [40, 3, 0, 17, 39]),  # ragged rows across tile borders
    (4, 256, 200, 4, 4, 64, [31, 7, 2, 9], [0, 0, 0, 0]),          # nothing but the prefix
    (2, 512, 384, 4, 4, 128, [384, 256], None),                    # full tiles: each sequence by itself
    (3, 0, 100, 4, 2, 128, [9, 100, 2], [100, 0, 3]),              # no prefix
    (37, 700, 9, 14, 2, 128, [b % 4 for b in range(37)], [(5 * b) % 10 for b in range(37)]),
    (8, 5000, 33, 2, 1, 128, [11] * 8, None),                      # one head: tiles split over the SMs
]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("B,Lp,L,Hq,Hkv,D,Rs,lens", PREFIX)
def test_prefix_attention(E, B, Lp, L, Hq, Hkv, D, Rs, lens, quant):
    Case(B, L, Hq, Hkv, D, Rs, lens, Lp=Lp, quant=quant, seed=L + B).run(E)


@pytest.mark.parametrize("Lp", [None, 300])
@pytest.mark.parametrize("quant", [False, True])
def test_sharp_softmax(E, quant, Lp):
    # scores of deviation 11 D^0.5 scale: maxima that jump by far more than the rescale threshold
    if Lp is None and not quant:
        Lp = 0
    Case(2, 700, 8, 2, 128, [60, 3], [700, 650], Lp=Lp, quant=quant, seed=3, scale=1.0, spread=0.2).run(E)


def test_one_key_takes_all_and_values_of_every_magnitude(E):
    # V rows from 2^-60 to 2^60: each row's weight and value meet in full range
    c = Case(1, 500, 4, 2, 128, [20], seed=8, spread=0.5)
    rng = np.random.default_rng(9)
    x = Q.bf16(rng.standard_normal((1, 500, 2, 128)) * 2.0 ** rng.integers(-60, 60, (1, 500, 2, 1)))
    code, e = Q.quantise(Q.f64(x))
    c.own[1].copy_(torch.from_numpy(code).float().to(torch.float8_e4m3fn))
    c.own[3][:, :, :500] = torch.from_numpy(e.transpose(0, 2, 1))
    c.run(E)


def test_scope_cuts_the_keys(E):
    for quant, Lp in ((True, None), (False, 200)):
        c = Case(2, 600, 4, 2, 128, [40, 9], [600, 100], Lp=Lp, quant=quant, seed=12)
        c.scope = 333
        c.run(E)
        c.lens = None
        c.run(E)


@pytest.mark.parametrize("quant", [False, True])
def test_what_lies_past_a_length_is_not_used(E, quant):
    lens = [1, 127, 0, 200, 256]
    c = Case(5, 256, 4, 2, 128, [9, 3, 2, 130, 1], lens, Lp=100, quant=quant, seed=5)
    d = c.inputs(E)
    for b, n in enumerate(lens):
        for x in d["cache"] if not quant else (d["cache"].k, d["cache"].v):
            raw = x.view(torch.int16 if not quant else torch.uint8)
            raw[b, n:] = 0x7FC1 if not quant else 0x7F  # NaN
        if quant:
            d["cache"].k_exp[b, :, n:] = 255
            d["cache"].v_exp[b, :, n:] = 255
    c.call(E, d)
    c.check(d["out"])
    if quant:
        del d["prefix"]
        c.pre = None
        d["out"].fill_(SENTINEL)
        c.call(E, d)
        c.check(d["out"])


def test_nan_and_infinity_among_the_keys(E):
    # a NaN value row reaches every row of its KV head and no other; a key whose scores are all -infinity
    # has no weight; with nothing but such keys a row is zeros
    c = Case(1, 300, 2, 2, 64, [6], Lp=0, quant=False, seed=2)
    d = c.inputs(E)
    d["q"].abs_()
    k, v = d["cache"]
    v[0, 7, 0, 3] = float("nan")
    k[0, 9, 1] = float("-inf")
    c.call(E, d)
    got = Q.f64(d["out"])[0, :6]
    assert np.isnan(got[:, 0, 3]).all() and np.isfinite(got[:, 1]).all()
    c.q = c.q.abs()
    k64, v64 = Q.f64(c.own[0])[0], Q.f64(c.own[1])[0]
    keep = np.arange(300) != 9
    want, tol = Q.attention(Q.f64(c.q[0, :6])[:, 1:], k64[keep][:, 1:], v64[keep][:, 1:], c.scale)
    assert (np.abs(got[:, 1:] - want) <= tol).all()
    k[0, :, 1] = float("-inf")
    c.call(E, d)
    assert (Q.f64(d["out"])[0, :6, 1] == 0).all()


def test_bad_sizes_are_reported_and_their_sequences_skipped(E):
    from entropy_gated_kv_gb300 import _capi as C

    for Lp in (None, 200):
        c = Case(4, 50, 4, 2, 64, [5, 51, 7, -1], [50, 50, 51, 3], Lp=Lp, seed=1)
        d = c.inputs(E)
        c.call(E, d)
        assert E.read_device_error(d["dev_err"])[1] == C.EC_DEVERR_BAD_R | C.EC_DEVERR_BAD_LEN
        c.check(d["out"], skip=(1, 2, 3))


def test_prefix_and_own_make_the_whole_cache(E):
    # the same keys, cut into a prefix and the rest, against the library's attention over one cache
    B, Lp, L, H, D = 3, 384, 128, 4, 128
    rng = np.random.default_rng(21)
    q = Q.bf16(rng.standard_normal((B, Lp + L, H, D))).cuda()
    pk, pv = (Q.bf16(rng.standard_normal((Lp, H, D))).cuda() for _ in range(2))
    k, v = (Q.bf16(rng.standard_normal((B, L, H, D))).cuda() for _ in range(2))
    R = torch.tensor([30, 128, 1], dtype=torch.int32, device="cuda")
    whole = [torch.cat([a[None].expand(B, -1, -1, -1), b], 1).contiguous() for a, b in ((pk, k), (pv, v))]
    out = torch.zeros_like(q)
    E.partial_attention(E.Params(B=B, L=Lp + L, Hq=H, Hkv=H, D=D, V=8, C_max=1, k=1), q, *whole, R, out)
    mine = torch.zeros(B, L, H, D, dtype=torch.bfloat16, device="cuda")
    E.prefix_attention(E.Params(B=B, L=L, Hq=H, Hkv=H, D=D, V=8, C_max=1, k=1), q[:, :L].contiguous(), (pk, pv), (k, v), R, mine)
    for b in range(B):
        r = int(R[b])
        want, tol = Q.attention(Q.f64(q[b, :r]), Q.f64(whole[0][b]), Q.f64(whole[1][b]), Q.default_scale(D))
        # both calls are within `tol` of the exact result
        assert (np.abs(Q.f64(out[b, :r]) - Q.f64(mine[b, :r])) <= 2 * tol).all()


def test_a_denoising_loop_on_an_8_bit_cache(E):
    """Three steps of a block behind a shared prompt: quantise the prompt once, then per step refresh the
    recompute rows, attend, and read the rows back; every step against 64 bits."""
    B, Lp, L, Hq, Hkv, D = 3, 333, 96, 14, 2, 128
    rng = np.random.default_rng(31)
    pre = E.QuantCache.empty(1, Lp, Hkv, D)
    pk, pv = (Q.bf16(rng.standard_normal((1, Lp, Hkv, D))) for _ in range(2))
    E.kv_scatter_quant(E.Params(B=1, L=Lp, Hq=Hq, Hkv=Hkv, D=D, V=8, C_max=1, k=1), pre, pk.cuda(), pv.cuda(),
                       torch.arange(Lp, dtype=torch.int32, device="cuda")[None].contiguous(),
                       torch.tensor([Lp], dtype=torch.int32, device="cuda"))
    p = E.Params(B=B, L=L, Hq=Hq, Hkv=Hkv, D=D, V=8, C_max=1, k=1)
    cache = E.QuantCache.empty(B, L, Hkv, D)
    ws = E.workspace(E.prefix_attention_workspace_size(p))
    state = [np.zeros((B, L, Hkv, D)) for _ in range(2)]
    pre64 = [c * 2.0 ** (e.astype(float) - 127)[..., None] for c, e in (Q.quantise(Q.f64(x)) for x in (pk, pv))]
    for step, Rs in enumerate(([L] * B, [40, 7, 1], [1, 0, 96])):
        fresh = [Q.bf16(rng.standard_normal((B, L, Hkv, D))) for _ in range(2)]
        q = Q.bf16(rng.standard_normal((B, L, Hq, D)))
        idx = torch.zeros(B, L, dtype=torch.int32)
        for b, r in enumerate(Rs):
            pos = np.sort(rng.permutation(L)[:r])
            idx[b, :r] = torch.from_numpy(pos)
            for s, x in zip(state, fresh):
                c, e = Q.quantise(Q.f64(x[b, :r]))
                s[b, pos] = c * 2.0 ** (e.astype(float) - 127)[..., None]
        R, di = torch.tensor(Rs, dtype=torch.int32, device="cuda"), idx.cuda()
        E.kv_scatter_quant(p, cache, fresh[0].cuda(), fresh[1].cuda(), di, R)
        out = torch.zeros(B, L, Hq, D, dtype=torch.bfloat16, device="cuda")
        E.prefix_attention(p, q.cuda(), pre, cache, R, out, ws=ws)
        back = E.kv_gather_quant(p, cache, None, torch.full((B,), L, dtype=torch.int32, device="cuda"))
        np.testing.assert_array_equal(Q.f64(back[0]), state[0])
        np.testing.assert_array_equal(Q.f64(back[1]), state[1])
        for b, r in enumerate(Rs):
            want, tol = Q.attention(Q.f64(q[b, :r]), np.concatenate([pre64[0][0], state[0][b]]),
                                    np.concatenate([pre64[1][0], state[1][b]]), Q.default_scale(D))
            assert (np.abs(Q.f64(out[b, :r]) - want) <= tol).all(), step


@pytest.mark.parametrize("Lp", [None, 600])
def test_same_bits_again_in_a_graph_and_on_two_streams(E, Lp):
    c = Case(3, 400, 8, 2, 128, [40, 1, 133], [400, 77, 300], Lp=Lp, seed=17)
    d = c.run(E)
    first = d["out"].clone()
    ws = [E.workspace(E.prefix_attention_workspace_size(d["p"])).fill_(255) for _ in range(2)]  # NaN patterns
    outs = [torch.full_like(first, SENTINEL) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for s, w, o in zip(streams, ws, outs):
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.call(E, {**d, "out": o}, ws=w)
        graphs.append(g)
    for rep in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), first.view(torch.int16))
    # replayed with other sizes: the plan is made from them on the device
    d["R"].copy_(torch.tensor([1, 400, 0], dtype=torch.int32))
    c.Rs = [1, 400, 0]
    outs[0].fill_(SENTINEL)
    graphs[0].replay()
    torch.cuda.synchronize()
    c.check(outs[0])


def test_keys_past_32_bit_offsets(E):
    # 131104 positions x 128 heads x 128 bytes: the last keys lie past 2^31 bytes; with a peaked row that
    # attends to one of them, the output is that value
    L, H, D = 131104, 128, 128
    cache = E.QuantCache.empty(1, L, H, D)
    cache.k_exp.fill_(127)
    cache.v_exp.fill_(127)
    rng = np.random.default_rng(2)
    for h, pos in ((0, L - 1), (77, 131072), (127, L - 17)):
        cache.k[0, pos, h] = torch.full((D,), 8.0, device="cuda").to(torch.float8_e4m3fn)
        cache.v[0, pos, h] = torch.from_numpy(rng.integers(1, 8, D).astype(np.float32)).cuda().to(torch.float8_e4m3fn)
    q = torch.ones(1, L, H, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    E.partial_attention_quant(E.Params(B=1, L=L, Hq=H, Hkv=H, D=D, V=8, C_max=1, k=1), q, cache,
                              torch.tensor([2], dtype=torch.int32, device="cuda"), out, scale=1.0)
    for h, pos in ((0, L - 1), (77, 131072), (127, L - 17)):
        # the other weights are exp(-1024) = 0
        np.testing.assert_array_equal(Q.f64(out[0, 1, h]), Q.code_values(cache.v[0, pos, h]))
    assert not out[0, 1, 5].any()


def test_binding_refusals(E):
    c = Case(2, 48, 4, 2, 64, [3, 4], Lp=32, quant=False)
    d = c.inputs(E)
    p, q, (pk, pv), (k, v), R, out = (d[n] for n in ("p", "q", "prefix", "cache", "R", "out"))
    ok = dict(p=p, q=q, prefix=(pk, pv), cache=(k, v), R=R, out=out)
    E.prefix_attention(**ok)
    for name, bad in [("q", q.float()), ("q", q[:, :, :2]), ("out", out.transpose(1, 2)), ("R", R.long()), ("R", R[:1]),
                      ("cache", (k, v[:, :40])), ("cache", (k.half(), v.half())), ("cache", (k[:, ::2], v[:, ::2])),
                      ("prefix", (pk[:, :1], pv[:, :1])), ("prefix", (pk.cpu(), pv.cpu()))]:
        with pytest.raises(ValueError):
            E.prefix_attention(**{**ok, name: bad})
    with pytest.raises(E.EcError):  # a workspace that is too small
        E.prefix_attention(**ok, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(E.EcError):  # the output over the queries
        E.prefix_attention(**{**ok, "out": q})
    with pytest.raises(E.EcError):
        E.prefix_attention(**ok, scale=0.0)
    with pytest.raises(ValueError):
        E.prefix_attention(**ok, kv_len=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(E.EcError):  # types of the two caches differ
        E.prefix_attention(**{**ok, "cache": E.QuantCache.empty(2, 48, 2, 64)})
    with pytest.raises(ValueError):
        E.partial_attention_quant(p, q, E.QuantCache.empty(2, 40, 2, 64), R, out)


WHOLE = [
    # B, L, Hq, Hkv, D, rows, lengths, Lp: about as many tiles as SMs, of about one length (a tile to a CTA)
    (8, 200, 16, 16, 128, [100, 128, 5, 90, 128, 1, 77, 128], [200, 130, 128, 199, 1, 200, 0, 200], None),
    (6, 1100, 40, 20, 64, [64, 3, 60, 11, 64, 40], [1100, 800, 700, 901, 640, 1099], None),
    (5, 60, 28, 28, 128, [60, 60, 33, 1, 60], [60, 0, 59, 2, 60], 700),
]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("B,L,Hq,Hkv,D,Rs,lens,Lp", WHOLE)
def test_a_tile_to_a_cta(E, B, L, Hq, Hkv, D, Rs, lens, Lp, quant):
    if not quant and Lp is None:
        Lp = 0
    Case(B, L, Hq, Hkv, D, Rs, lens, Lp=Lp, quant=quant, seed=L + B).run(E)


@pytest.mark.parametrize("quant", [False, True])
def test_queries_and_outputs_at_odd_multiples_of_16_bytes(E, quant):
    c = Case(2, 150, 6, 2, 64, [150, 31], [150, 70], Lp=100, quant=quant, seed=23)
    d = c.inputs(E)
    for n in ("q", "out"):
        t = torch.empty(d[n].numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(d[n].shape)
        d[n] = t.copy_(d[n])
        assert t.data_ptr() % 32 == 16
    c.call(E, d)
    c.check(d["out"])


REPEATS = [
    # shapes with several items to a CTA, both streams, ragged ends, the merge; run often, with the same bits
    (7, 500, 24, 8, 128, [90, 128, 1, 0, 300, 500, 17], [500, 1, 500, 400, 0, 333, 499], 1000),
    (4, 900, 16, 16, 64, [900, 1, 450, 130], [900, 899, 64, 65], 130),
    (16, 64, 32, 4, 128, [1] * 16, list(range(0, 64, 4)), 3000),
]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("B,L,Hq,Hkv,D,Rs,lens,Lp", REPEATS)
def test_the_same_bits_every_time(E, B, L, Hq, Hkv, D, Rs, lens, Lp, quant):
    c = Case(B, L, Hq, Hkv, D, Rs, lens, Lp=Lp, quant=quant, seed=B)
    d = c.inputs(E)
    ws = E.workspace(E.prefix_attention_workspace_size(d["p"]))
    c.call(E, d, ws=ws)
    c.check(d["out"])
    first = d["out"].clone()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for n in range(60):
        if n % 3 == 0:
            flush.fill_(n)  # the caches from memory, not from L2
        ws.fill_(255)
        d["out"].fill_(SENTINEL)
        c.call(E, d, ws=ws)
        assert torch.equal(d["out"].view(torch.int16), first.view(torch.int16)), n
    assert int(d["dev_err"].item()) == 0


@pytest.mark.parametrize("up", [0, 20])  # exponent bytes around 120, and above 134 (two factors)
@pytest.mark.parametrize("B,L,Hq,Hkv,D,Rs,lens,Lp", [
    (2, 256, 6, 3, 128, [9, 140], [256, 200], None),           # one block a tile or two
    (1, 4000, 4, 2, 64, [3], [3999], None),                    # a tile over many CTAs, merged
    (4, 200, 8, 4, 128, [1, 5, 0, 2], [200, 64, 10, 0], 900),  # a shared prefix, every row merged
])
def test_nan_in_an_8_bit_cache(E, B, L, Hq, Hkv, D, Rs, lens, Lp, up):
    """NaN codes in rows of ordinary exponents and rows of byte 255, among the keys that take part: a NaN key
    makes its head's rows NaN, a NaN value its column of them; every other value is as it was."""
    c = Case(B, L, Hq, Hkv, D, Rs, lens, Lp=Lp, seed=41 + up, q_scale=2.0**-up)
    for t in (c.own, c.pre):
        if t is not None and up:
            t[2].copy_((t[2].int() + up).to(torch.uint8))
            t[3].copy_((t[3].int() + up).to(torch.uint8))
    g = Hq // Hkv
    where = [("own", 0, 0), ("own", 0, lens[0] - 1), ("own", 0, 63), ("own", 0, lens[0] // 2)]
    if Lp is not None:
        where += [("pre", 0, Lp - 1), ("pre", 0, 128)]
    for kv in (0, 1):
        for name, b, pos in where:
            for byte in (None, 255):
                d = c.inputs(E)
                cache = d["cache"] if name == "own" else d["prefix"]
                code = (cache.k, cache.v)[kv].view(torch.uint8)
                h, col = 1, D - 3
                if byte is None:
                    code[b, pos, h, col] = 0x7F if pos % 2 else 0xFF
                else:
                    code[b, pos, h] = 0x7F
                    (cache.k_exp, cache.v_exp)[kv][b, h, pos] = byte
                clean = c.inputs(E)
                c.call(E, clean)
                c.call(E, d)
                assert int(d["dev_err"].item()) == 0
                c.check(clean["out"])
                nan = np.zeros((B, L, Hq, D), bool)
                for i, r in enumerate(Rs):
                    if name == "pre" or i == b:
                        nan[i, :r, h * g : (h + 1) * g, slice(None) if kv == 0 or byte else col] = True
                got, was = Q.f64(d["out"]), Q.f64(clean["out"])
                np.testing.assert_array_equal(np.isnan(got), nan)
                np.testing.assert_array_equal(got[~nan], was[~nan])


# the modes of the plan that these sizes have (on 152 SMs) are checked in test_device_code_on_cpu.py
BORDERS = [
    (34, 8, 32, 32, 64, [1 + b % 2 for b in range(34)], [b % 9 for b in range(34)], 700),   # shared, as many tiles as there are places
    (36, 8, 32, 32, 64, [1 + b % 2 for b in range(36)], [b % 9 for b in range(36)], 700),   # more: each tile by itself
    (5, 130, 28, 28, 128, [128, 120, 128, 101, 128], [130, 0, 59, 2, 128], 700),            # a tile to a CTA, prefix and own blocks
    (3, 260, 80, 40, 64, [64, 50, 33], [260, 129, 7], 1000),                                # the same, grouped heads
]


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("B,L,Hq,Hkv,D,Rs,lens,Lp", BORDERS)
def test_each_mode_of_the_plan_behind_a_prefix(E, B, L, Hq, Hkv, D, Rs, lens, Lp, quant):
    Case(B, L, Hq, Hkv, D, Rs, lens, Lp=Lp, quant=quant, seed=L + B).run(E)


@pytest.mark.parametrize("by_pos", [False, True])
def test_a_step_on_8_bit_caches_from_the_selection(E, by_pos):
    """Selection, quantised refresh and attention in one row on the device: idx and R are those that
    select_recompute leaves, with partial and full steps in one batch; everything against 64 bits."""
    B, L, Hq, Hkv, D, Lp, k, C_max, n_dec = 4, 120, 8, 2, 128, 300, 12, 16, 2
    rng = np.random.default_rng(51 + by_pos)
    p = E.Params(B=B, L=L, Hq=Hq, Hkv=Hkv, D=D, V=1000, C_max=C_max, k=k, n_dec=n_dec, tau=1.0)
    masked = np.stack([np.sort(rng.permutation(L)[:40]) for _ in range(B)])
    mask = np.zeros((B, L), np.uint8)
    np.put_along_axis(mask, masked, 1, 1)
    st = E.DecodeState.from_arrays(p, tokens=rng.integers(0, 1000, (B, L)), mask=mask)
    own = Q.random_cache(rng, B, L, Hkv, D)
    cache = E.QuantCache(*(t.cuda() for t in own))
    pre = Q.random_cache(rng, 1, Lp, Hkv, D)
    prompt = E.QuantCache(*(t.cuda() for t in pre))
    k64, v64 = Q.widen(own[0], own[2]), Q.widen(own[1], own[3])
    pk64, pv64 = Q.widen(pre[0], pre[2])[0], Q.widen(pre[1], pre[3])[0]
    ws = [E.workspace(f(p)) for f in (E.partial_attention_quant_workspace_size, E.prefix_attention_workspace_size)]
    seen = set()
    for step in range(3):
        left = st.mask.cpu().numpy()
        cand = np.stack([np.resize(rng.permutation(np.flatnonzero(left[b])), C_max) for b in range(B)]).astype(np.int32)
        entropy = rng.random((B, C_max)).astype(np.float32)
        entropy[step % B] += 2.0  # above tau: this sequence's step is full
        conf = -rng.random((B, C_max)).astype(np.float32)
        fresh = [Q.bf16(rng.standard_normal((B, L, Hkv, D))) for _ in range(2)]  # by position
        q = Q.bf16(rng.standard_normal((B, L, Hq, D)))
        E.select_recompute(p, st, torch.from_numpy(cand).cuda(), torch.full((B,), C_max, dtype=torch.int32, device="cuda"),
                           torch.zeros(B * C_max, dtype=torch.int32, device="cuda"), torch.from_numpy(entropy.ravel()).cuda(),
                           torch.from_numpy(conf.ravel()).cuda())
        at = st.idx.long().clamp(0, L - 1)[..., None, None]
        rows = [x.cuda() if by_pos else x.cuda().take_along_dim(at, 1) for x in fresh]
        E.kv_scatter_quant(p, cache, *rows, st.idx, st.R, src_by_position=by_pos, dev_err=st.dev_err)
        qr = q.cuda().take_along_dim(at, 1)
        outs = [torch.full_like(qr, SENTINEL) for _ in range(2)]
        E.partial_attention_quant(p, qr, cache, st.R, outs[0], ws=ws[0], dev_err=st.dev_err)
        E.prefix_attention(p, qr, prompt, cache, st.R, outs[1], ws=ws[1], dev_err=st.dev_err)
        assert E.read_device_error(st.dev_err) == (0, 0)
        R, idx = st.R.cpu().numpy(), st.idx.cpu().numpy()
        for b in range(B):
            r, pos = R[b], idx[b, : R[b]]
            seen.add(r == L)
            assert 0 < r <= L and (np.diff(pos) > 0).all()
            for x64, x in ((k64, fresh[0]), (v64, fresh[1])):
                c, e = Q.quantise(Q.f64(x[b, pos]))
                x64[b, pos] = c * 2.0 ** (e.astype(float) - 127)[..., None]
        for out, kk, vv in ((outs[0], k64, v64), (outs[1], [np.concatenate([pk64, x]) for x in k64],
                                                  [np.concatenate([pv64, x]) for x in v64])):
            for b in range(B):
                want, tol = Q.attention(Q.f64(q[b, idx[b, : R[b]]]), kk[b], vv[b], Q.default_scale(D))
                got = Q.f64(out[b])
                assert (np.abs(got[: R[b]] - want) <= tol).all(), (step, b)
                assert (got[R[b] :] == SENTINEL).all()
    assert seen == {True, False}  # partial and full steps
