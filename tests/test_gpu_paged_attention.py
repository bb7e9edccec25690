"""GPU tests of the attentions over a paged cache, element by element against 64 bits with the bound that
tests/_paged.py derives from the kernels' roundings. Whatever no row may look at is NaN in the pool and a junk page
number in the table."""
import numpy as np
import pytest
import torch

from tests import _paged as P
from tests import _quant as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import entropy_gated_kv_gb300 as E

    E.lib()
    return E


FULL = [
    # B, L, Hq, Hkv, D, page, rows, lengths
    (1, 1, 1, 1, 64, 16, [1], None),                                # one key
    (1, 1, 1, 1, 128, 16, [1], [0]),                                # no key: zeros
    (1, 17, 2, 1, 128, 16, [1], [17]),                              # a page that ends inside a tile
    (1, 2047, 28, 4, 128, 64, [1], None),                           # a single token, odd length, split over the SMs
    (1, 1000, 4, 4, 64, 16, [1], None),
    (5, 700, 14, 2, 128, 32, [1, 0, 1, 1, 1], [700, 5, 0, 129, 64]),   # single tokens, ragged, an empty sequence
    (40, 70, 2, 1, 64, 16, [(7 * b) % 3 for b in range(40)], [(11 * b) % 71 for b in range(40)]),  # more than a warp of sequences
    (200, 300, 8, 8, 128, 16, [1] * 200, [(37 * b) % 301 for b in range(200)]),  # more sequences than SMs
    (3, 300, 6, 2, 128, 16, [5, 0, 4], [300, 17, 129]),
    (2, 300, 32, 2, 128, 32, [1, 1], [300, 299]),                   # sixteen packed rows
    (2, 500, 34, 2, 64, 32, [1, 1], [500, 65]),                     # seventeen
    (1, 4000, 2, 1, 128, 256, [16], [3999]),                        # thirty-two, one tile over many CTAs
    (1, 1024, 3, 1, 128, 1024, [11], None),                         # thirty-three
    (1, 384, 128, 1, 64, 128, [3], None),                           # 128 heads on one KV head
    (1, 300, 96, 2, 128, 16, [11], [200]),                          # g = 48: rows of a tile left over
    (2, 140, 14, 2, 128, 16, [140, 33], [131, 128]),                # g = 7
    (1, 256, 8, 8, 64, 16, [47], None),
    (1, 1024, 32, 32, 128, 64, [95], None),
    (2, 512, 8, 8, 64, 64, [129, 257], [512, 0]),                   # two tiles, three; a sequence without keys
    (4, 640, 16, 16, 128, 128, [640] * 4, [640, 5, 333, 640]),      # more tiles than CTAs
    (1, 130, 2, 2, 128, 512, [130], None),                          # pages larger than the sequence
    (6, 900, 7, 1, 128, 32, [95, 1, 40, 0, 128, 19], [900, 899, 33, 7, 640, 127]),
    (1, 9000, 2, 2, 128, 16, [200], [8999]),                        # few tiles, many blocks: cut items of two tiles
    (2, 30000, 4, 2, 64, 16, [1, 2], [30000, 17]),                  # few rows, many chunks: cut items
    (1, 20000, 1, 1, 64, 64, [100], [19999]),                       # one tile a sequence: cut items
    (30, 300, 8, 8, 64, 32, [40 + b for b in range(30)], [(31 * b) % 301 for b in range(30)]),  # more items than SMs
    (1, 700, 14, 2, 128, 16, [95], [613]),                          # pairs of tiles in clusters
    (2, 100, 28, 4, 64, 16, [40, 3], [90, 100]),                    # a second tile without rows, CTAs without blocks
]


@pytest.mark.parametrize("kind", ["split", "one", "wide"])
@pytest.mark.parametrize("B,L,Hq,Hkv,D,page,Rs,lens", FULL)
def test_paged_attention(E, B, L, Hq, Hkv, D, page, Rs, lens, kind):
    P.Case(B, L, Hq, Hkv, D, page, Rs, lens, at=None, kind=kind, seed=L + B).run(E)


WINDOW = [
    # B, L, Hq, Hkv, D, page, rows, lengths, (left, right, sinks)
    (1, 1, 1, 1, 64, 16, [1], None, (0, 0, 0)),                      # itself
    (3, 400, 14, 2, 128, 16, [1, 1, 1], [400, 31, 1], (63, 0, 4)),   # single tokens with sinks
    (3, 400, 14, 2, 64, 32, [1, 1, 1], [400, 130, 200], (63, 5, 0)),
    (1, 5000, 28, 4, 128, 64, [1], [4999], (-1, 0, 0)),              # the causal form
    (1, 5000, 4, 1, 128, 16, [1], None, (3000, -1, 100)),
    (2, 300, 2, 2, 128, 16, [16, 9], [300, 120], (20, 7, 3)),        # few rows, each with its own window
    (2, 300, 2, 1, 64, 16, [16, 3], [300, 120], (-1, 0, 0)),
    (1, 600, 4, 4, 128, 32, [40], None, (0, 0, 0)),                  # every row sees one key
    (2, 512, 7, 1, 128, 64, [95, 40], [512, 300], (64, 64, 16)),
    (2, 700, 8, 8, 128, 64, [95, 60], [700, 431], (130, 40, 200)),   # sinks past a block
    (1, 700, 3, 3, 64, 128, [700], None, (-1, 0, 0)),                # causal, several tiles
    (1, 900, 2, 1, 128, 16, [900], [900], (100, 100, 0)),
    (2, 1500, 7, 1, 128, 32, [1500, 700], [1500, 900], (257, 63, 5)),
    (1, 300, 2, 2, 128, 16, [300], [150], (10, 10, 0)),              # rows past the last key that see nothing
    (1, 300, 2, 2, 128, 16, [300], [150], (10, 10, 1)),
    (4, 260, 4, 4, 64, 16, [3, 130, 0, 260], [0, 260, 100, 7], (5, 5, 2)),
    (1, 8000, 2, 2, 128, 64, [64], None, (2000, 2000, 64)),          # a window split over the SMs
]


@pytest.mark.parametrize("at", ["idx", "start", None])
@pytest.mark.parametrize("B,L,Hq,Hkv,D,page,Rs,lens,window", WINDOW)
def test_window_attention(E, B, L, Hq, Hkv, D, page, Rs, lens, window, at):
    P.Case(B, L, Hq, Hkv, D, page, Rs, lens, window, at, seed=L + B).run(E)


# Clusters of one CTA, clusters with many blocks each, the same sizes with lengths that only the device knows.
@pytest.mark.parametrize("lens", [None, "ragged"])
@pytest.mark.parametrize("B,L,Hq,Hkv,D,R", [
    (4, 300, 32, 32, 64, 20), (4, 1024, 32, 32, 64, 20), (4, 2300, 28, 28, 64, 20), (3, 500, 32, 32, 64, 1), (3, 1100, 32, 32, 128, 1),
    (1, 9000, 32, 32, 64, 95), (1, 9000, 8, 8, 64, 300), (16, 1100, 28, 4, 64, 18)])
def test_clusters(E, B, L, Hq, Hkv, D, R, lens):
    lens = None if lens is None else [(L - 7 * b * b * b) % (L + 1) for b in range(B)]
    P.Case(B, L, Hq, Hkv, D, 16 if R == 1 else 64, [R] * B, lens, at=None, kind="split", seed=L).run(E)


# A line whose shares end anywhere: in the middle of an item, before its first block, at its end.
@pytest.mark.parametrize("R", [1, 30, 130])
@pytest.mark.parametrize("seed", range(8))
def test_shares_of_the_line(E, R, seed):
    rng = np.random.default_rng(seed)
    B, L = int(rng.integers(20, 42)), int(rng.choice([100, 130, 400, 900, 1300]))
    R = min(R, L)  # more rows than positions are refused
    lens = [int(x) for x in rng.integers(0, L + 1, B) * (rng.random(B) < 0.9)]
    rows = [int(x) for x in rng.integers(0, R + 1, B)]
    rows[0] = R
    P.Case(B, L, 8, 8, 64, 32, rows, lens, at=None, kind="split", seed=seed).run(E)


@pytest.mark.parametrize("R", [1, 60, 300])
@pytest.mark.parametrize("seed", range(6))
def test_shares_of_the_line_in_windows(E, R, seed):
    rng = np.random.default_rng(100 + seed)
    B, L = int(rng.integers(20, 42)), int(rng.choice([130, 700, 1500]))
    R = min(R, L)
    lens = [int(x) for x in rng.integers(1, L + 1, B)]
    rows = [min(n, int(x)) for n, x in zip(lens, rng.integers(0, R + 1, B))]
    window = (int(rng.choice([0, 50, 400])), int(rng.choice([0, 50, -1])), int(rng.choice([0, 3, 200])))
    P.Case(B, L, 8, 8, 64, 32, rows, lens, window, at="idx" if seed % 2 else "start", rows=R, seed=seed).run(E)


@pytest.mark.parametrize("R", [1, 20, 150])
@pytest.mark.parametrize("window", [None, (-1, 0, 0)])
def test_sequences_that_share_pages(E, R, window):
    c = P.Case(3, 700, 8, 4, 64, 32, [R, R, 1], [700, 500, 130], window, at="start", kind="one", seed=R)
    c.k[1:, :128], c.v[1:, :128] = c.k[0, :128], c.v[0, :128]  # a prefix of four pages
    c.pool.table[1:, :4] = c.pool.table[0, :4]
    c.run(E)


@pytest.mark.parametrize("pos,window", [
    ([[0, 1, 298, 299]], (3, 3, 0)),           # rows far from each other: keys between them that no row sees
    ([[5, 5, 5, 200]], (40, 0, 9)),            # the same position more than once
    ([[299, 299, 299, 299]], (0, 0, 300)),     # the sinks are everything
    ([[10, 20, 30, 40]], (300, 300, 0)),       # a window over everything
])
@pytest.mark.parametrize("g", [1, 12])
def test_positions(E, pos, window, g):
    P.Case(1, 300, 2 * g, 2, 128, 16, [4], None, window, "idx", pos=[np.array(x) for x in pos], seed=3, fill=0.25).run(E)


@pytest.mark.parametrize("R", [1, 20, 150])
@pytest.mark.parametrize("window", [None, (200, 20, 4)])
def test_sharp_softmax(E, R, window):
    # scores of deviation 11 D^0.5 scale: maxima that jump by far more than the rescale threshold
    P.Case(2, 600, 4, 2, 128, 32, [R, R], [600, 517], window, seed=R, q_scale=11.0).run(E)


@pytest.mark.parametrize("R", [1, 20, 150])
def test_negative_scores(E, R):
    # every score far below zero: the running maximum starts at -infinity, not at zero
    c = P.Case(1, 400, 2, 1, 64, 16, [R], [333], (100, 3, 2), seed=R)
    c.q = torch.full_like(c.q, 3.0)
    c.k = np.abs(c.k) * -8.0
    c.k = Q.f64(Q.bf16(c.k))
    c.pool.put(c.k, c.v)
    c.run(E)


@pytest.mark.parametrize("R", [1, 20, 150])
def test_infinite_scores(E, R):
    """Keys of -infinity have no weight; a row whose every key is one is zeros."""
    c = P.Case(2, 300, 2, 2, 64, 16, [R, R], [300, 200], None, None, seed=R)
    c.q = c.q.abs() + 0.01
    k = c.k.copy()
    k[0, ::3] = -np.inf
    k[1] = -np.inf
    c.pool.put(k, c.v)
    d = c.inputs(E)
    c.call(E, d)
    torch.cuda.synchronize()
    got = Q.f64(d["out"])
    assert (got[1] == 0).all()
    see = np.ones((R, 300), bool)
    see[:, ::3] = False
    want, tol = P.attention(Q.f64(c.q[0]), c.k[0], c.v[0], c.scale, see)
    assert (np.abs(got[0] - want) <= tol).all()


@pytest.mark.parametrize("R", [1, 20, 150])
def test_nan_in_the_keys_reaches_its_rows(E, R):
    c = P.Case(1, 300, 2, 2, 64, 16, [R], None, None, None, seed=R)
    k = c.k.copy()
    k[0, 100, 1, 5] = np.nan
    c.pool.put(k, c.v)
    d = c.inputs(E)
    c.call(E, d)
    got = Q.f64(d["out"])
    assert np.isnan(got[0, :, 1]).all() and np.isfinite(got[0, :, 0]).all()


@pytest.mark.parametrize("R", [1, 20])
@pytest.mark.parametrize("scope", [100, 129])
def test_scope(E, R, scope):
    P.Case(2, 300, 4, 2, 128, 16, [R, R], [300, 64], None, None, seed=R, scope=scope).run(E)
    c = P.Case(2, 300, 4, 2, 128, 16, [R, R], [300, 300], (500, 500, 0), None, seed=R, scope=scope)
    d = c.inputs(E)
    d["kv_len"] = None
    c.call(E, d)
    c.check(d["out"])


@pytest.mark.parametrize("R", [1, 20, 150])
@pytest.mark.parametrize("window", [None, (40, 10, 4)])
def test_bad_sizes_skip_their_sequence(E, R, window):
    c = P.Case(5, 300, 4, 2, 128, 16, [R] * 5, [300, 200, 100, 64, 300], window, seed=R)
    for field, bad, bit in (("R", [R, -1, R + 1, R, R], E._capi.EC_DEVERR_BAD_R), ("kv_len", [300, -1, 301, 64, 300], E._capi.EC_DEVERR_BAD_LEN)):
        d = c.inputs(E)
        d[field] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        c.call(E, d)
        torch.cuda.synchronize()
        assert int(d["dev_err"].item()) == bit
        c.check(d["out"], skip=(1, 2))


@pytest.mark.parametrize("R", [1, 20, 150])
def test_bad_positions_skip_their_row(E, R):
    c = P.Case(2, 300, 4, 2, 128, 16, [R, R], [300, 200], (40, 10, 4), seed=R)
    d = c.inputs(E)
    d["idx"][0, R - 1] = 300
    d["idx"][1, 0] = -1
    c.call(E, d)
    torch.cuda.synchronize()
    assert int(d["dev_err"].item()) == E._capi.EC_DEVERR_BAD_IDX
    c.check(d["out"], lost=((0, R - 1), (1, 0)))


@pytest.mark.parametrize("R", [1, 20, 150])
@pytest.mark.parametrize("page", [16, 64])
def test_bad_pages_read_as_zeros(E, R, page):
    c = P.Case(2, 300, 4, 2, 128, page, [R, R], [300, 200], None, None, seed=R)
    d = c.inputs(E)
    d["cache"].table[0, 2] = -1
    d["cache"].table[1, 0] = c.pool.n_pages
    c.call(E, d)
    torch.cuda.synchronize()
    assert int(d["dev_err"].item()) == E._capi.EC_DEVERR_BAD_PAGE
    for b, i in ((0, 2), (1, 0)):
        c.k[b, i * page : (i + 1) * page] = 0
        c.v[b, i * page : (i + 1) * page] = 0
    c.check(d["out"])


@pytest.mark.parametrize("R", [1, 20, 150])
def test_the_same_bits_again(E, R):
    c = P.Case(3, 1500, 14, 2, 128, 32, [R] * 3, [1500, 700, 1], (700, 30, 5), seed=R)
    d = c.run(E)
    first = d["out"].clone()
    for _ in range(3):
        d["out"].fill_(P.SENTINEL)
        c.call(E, d)
        assert torch.equal(d["out"], first)


@pytest.mark.parametrize("R", [1, 20, 150])
@pytest.mark.parametrize("window", [None, (300, 30, 5)])
def test_streams_and_graphs(E, R, window):
    """On a stream of its own, and captured and replayed with other inputs and sizes in the same buffers."""
    c = P.Case(3, 900, 14, 2, 128, 32, [R] * 3, [900, 700, 1], window, seed=R)
    other = P.Case(3, 900, 14, 2, 128, 32, [1, R, R], [900, 64, 333], window, rows=c.rows, seed=R + 100)
    d, od = c.inputs(E), other.inputs(E)
    pools = []
    for x in ("k", "v"):  # one pool that holds either's pages
        t = torch.full((max(c.pool.n_pages, other.pool.n_pages), 32, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        t[: c.pool.n_pages] = getattr(d["cache"], x)
        pools.append(t)
    d["cache"] = E.PagedCache(*pools, d["cache"].table)
    ws = E.workspace(E.paged_attention_workspace_size(d["p"], c.rows))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.call(E, d, ws=ws, stream=s)
    s.synchronize()
    c.check(d["out"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.call(E, d, ws=ws)
    ws.fill_(255)  # no initial contents
    d["q"].copy_(od["q"])
    d["R"].copy_(od["R"])
    d["kv_len"].copy_(od["kv_len"])
    for x in ("k", "v"):
        getattr(d["cache"], x)[: other.pool.n_pages].copy_(getattr(od["cache"], x))
    d["cache"].table.copy_(od["cache"].table)
    if "idx" in d:
        d["idx"].copy_(od["idx"])
    d["out"].fill_(P.SENTINEL)
    g.replay()
    torch.cuda.synchronize()
    assert int(d["dev_err"].item()) == 0
    other.check(d["out"])


def test_two_calls_at_once(E):
    """Two streams with a workspace each."""
    cases = [P.Case(2, 3000, 8, 2, 128, 64, [r, r], [3000, 2500], None, None, seed=r) for r in (2, 90)]
    ds = [c.inputs(E) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, d, s in zip(cases, ds, streams):
            c.call(E, d, stream=s)
    torch.cuda.synchronize()
    for c, d in zip(cases, ds):
        c.check(d["out"])


@pytest.mark.parametrize("R", [1, 95])
def test_far_pages(E, R):
    """Pages past 2^31 elements of the pool."""
    page, H, D = 1024, 2, 128
    n_pages = (1 << 31) // (page * H * D) + 40
    k = torch.empty(n_pages, page, H, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = P.Case(1, 2 * page, H, H, D, page, [R], None, None, None, seed=R)
    d = c.inputs(E)
    src = d["cache"]
    far = torch.tensor([[n_pages - 1, n_pages - 9]], dtype=torch.int32, device="cuda")
    for i in range(2):
        k[far[0, i].long()] = src.k[src.table[0, i].long()]
        v[far[0, i].long()] = src.v[src.table[0, i].long()]
    d["cache"] = E.PagedCache(k, v, far)
    c.call(E, d)
    c.check(d["out"])


@pytest.mark.parametrize("g", [1, 12, 40])
@pytest.mark.parametrize("R,seed", [(4, 0), (4, 1), (60, 2), (300, 3)])
def test_positions_out_of_order(E, R, g, seed):
    """A row is right, or not written and reported; none is wrong."""
    rng = np.random.default_rng(seed)
    pos = [rng.permutation(500)[:R], np.sort(rng.permutation(500)[:R])]
    c = P.Case(2, 500, 2 * g, 2, 64, 16, [R, R], None, (30, 9, 5), "idx", pos=pos, seed=seed, fill=0.25)
    d = c.inputs(E)
    every = P.Pool(np.random.default_rng(1), 2, 500, 2, 64, 16, [500, 500])  # every position has a page
    every.put(c.k, c.v)
    d["cache"] = every.device(E)
    c.call(E, d)
    torch.cuda.synchronize()
    lost = [(0, r) for r in range(R) if bool((d["out"][0, r] == P.SENTINEL).all())]
    assert int(d["dev_err"].item()) == (E._capi.EC_DEVERR_BAD_IDX if lost else 0)
    c.check(d["out"], lost=lost)


def test_binding_checks_its_tensors(E):
    c = P.Case(2, 300, 4, 2, 64, 16, [3, 3], None, (9, 9, 0), seed=1)
    d = c.inputs(E)
    p, q, cache, R, out = (d[n] for n in ("p", "q", "cache", "R", "out"))
    w = dict(left=1, right=1, idx=d["idx"])
    bad = [
        lambda: E.paged_attention(p, q.float(), cache, R, out),
        lambda: E.paged_attention(p, q[0], cache, R, out),
        lambda: E.paged_attention(p, q.cpu(), cache, R, out),
        lambda: E.paged_attention(p, q, cache, R, out[:, :2]),
        lambda: E.paged_attention(p, q.transpose(0, 1), cache, R, out),
        lambda: E.paged_attention(p, q, (cache.k, cache.v), R, out),
        lambda: E.paged_attention(p, q, cache, R.long(), out),
        lambda: E.paged_attention(p, q, cache, R[:1], out),
        lambda: E.paged_attention(p, q, cache, R, out, kv_len=R.float()),
        lambda: E.paged_attention(p, q, cache, R, out, ws=torch.empty(1 << 20, dtype=torch.uint8)),
        lambda: E.paged_attention(p, q, cache, R, out, dev_err=R),
        lambda: E.paged_window_attention(p, q, cache, R, out, 1, 1, idx=d["idx"], start=R),
        lambda: E.paged_window_attention(p, q, cache, R, out, 1, 1, idx=d["idx"][:, :2]),
        lambda: E.paged_window_attention(p, q, cache, R, out, 1, 1, idx=d["idx"].long()),
        lambda: E.paged_window_attention(p, q, cache, R, out, 1, 1, idx=d["idx"].t().contiguous().t()),
        lambda: E.paged_window_attention(p, q, cache, R, out, 1, 1, start=R.cpu()),
        lambda: E.PagedCache(cache.k, cache.v[:1], cache.table),
        lambda: E.PagedCache(cache.k, cache.v.float(), cache.table),
        lambda: E.PagedCache(cache.k, cache.v, cache.table.long()),
        lambda: E.PagedCache(cache.k, cache.v, cache.table[0]),
        lambda: E.PagedCache(cache.k, cache.v, cache.table.t().contiguous().t()),
        lambda: E.PagedCache(cache.k, cache.v, cache.table[:1].expand(2, -1)),
        lambda: E.PagedCache(cache.k.transpose(1, 2), cache.v.transpose(1, 2), cache.table),
        lambda: E.PagedCache(cache.k, torch.stack([cache.v, cache.v], 1)[:, 0], cache.table),
        lambda: E.paged_attention(E.Params(B=2, L=400, Hq=4, Hkv=2, D=64, V=8, C_max=1, k=1), q, cache, R, out),  # the table is too short
        lambda: E.paged_attention(E.Params(B=2, L=300, Hq=4, Hkv=4, D=64, V=8, C_max=1, k=1), q, cache, R, out),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    for f in (lambda: E.paged_attention(p, q, cache, R, q), lambda: E.paged_attention(p, q, cache, R, out, scale=0.0),
              lambda: E.paged_window_attention(p, q, cache, R, out, -2, 1, idx=d["idx"]),
              lambda: E.paged_window_attention(p, q, cache, R, out, sinks=-1, **w)):
        with pytest.raises(E.EcError):
            f()


def test_cache_follows_its_tensors(E):
    """A tensor exchanged or changed in place after the cache was made."""
    c = P.Case(2, 300, 4, 2, 64, 16, [3, 40], [300, 123], None, None, seed=2)
    d = c.run(E)
    cache = d["cache"]
    table = cache.table.clone()
    swap = torch.where((table >= 0) & (table < c.pool.n_pages), c.pool.n_pages - 1 - table, table)
    cache.k, cache.v, cache.table = cache.k.flip(0), cache.v.flip(0), swap
    d["out"].fill_(P.SENTINEL)
    c.call(E, d)
    c.check(d["out"])
    swap.resize_(1, swap.shape[1])  # the cache keeps the shape that it was given
    cache.k.transpose_(0, 1)
    d["out"].fill_(P.SENTINEL)
    c.call(E, d)
    c.check(d["out"])
    for bad in (table.t().contiguous().t(), table[:1].contiguous()):
        cache.table = bad
        for _ in range(2):
            with pytest.raises(ValueError):
                c.call(E, d)
    cache.table = swap.resize_(*table.shape)
    k = cache.k
    cache.k = moved = k.clone()
    c.call(E, d)
    for n in (moved.untyped_storage().nbytes() // 2, 0):
        moved.untyped_storage().resize_(n)
        with pytest.raises(ValueError):
            c.call(E, d)
    cache.k, cache.v = k, cache.v.float()
    with pytest.raises(ValueError):
        c.call(E, d)
