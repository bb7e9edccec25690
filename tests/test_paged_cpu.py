"""Paged cache, without a GPU: refusals of the C entries and of the binding, and workspace sizes. No pointer is read:
every call fails before it reaches CUDA."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def capi():
    from entropy_gated_kv_gb300 import build as B

    B.build()
    from entropy_gated_kv_gb300 import _capi as C

    C.load()
    return C


def at(i, off=0):
    """Addresses 64 GB apart."""
    return ((i + 1) << 36) + off


def params(C, **kw):
    base = dict(B=2, L=1024, Hq=8, Hkv=4, D=128, V=8, C_max=1, k=1, n_dec=1, tau=1.0, logits_dtype=C.EC_BF16)
    base.update(kw)
    return C.EcParams(**base)


def pool(C, **kw):
    a = dict(page_size=64, n_pages=40, page_stride=64 * 4 * 128, k=at(0), v=at(1), table=at(2), table_stride=16)
    a.update(kw)
    return C.EcPagedKv(**a)


def rows(C, x, heads, rows_max, **kw):
    a = dict(x=x, batch_stride=rows_max * heads * 128, row_stride=heads * 128)
    a.update(kw)
    return C.EcRows(**a)


PAGE = 64 * 4 * 128 * 2  # bytes of a page of K


def bad_pools(C):
    INV, UNS = C.EC_ERR_INVALID_ARG, C.EC_ERR_UNSUPPORTED
    return [(dict(page_size=8), UNS), (dict(page_size=48), UNS), (dict(page_size=2048, page_stride=2048 * 512), UNS), (dict(page_size=0), UNS),
            (dict(page_size=-16), UNS), (dict(n_pages=0), INV), (dict(n_pages=-1), INV), (dict(k=None), INV), (dict(v=None), INV),
            (dict(table=None), INV), (dict(k=at(0, 8)), INV), (dict(v=at(1, 2)), INV), (dict(table=at(2, 2)), INV),
            (dict(page_stride=64 * 4 * 128 - 8), INV), (dict(page_stride=64 * 4 * 128 + 4), INV), (dict(page_stride=-64 * 4 * 128), INV),
            (dict(page_stride=1 << 36), UNS), (dict(n_pages=1 << 30), UNS), (dict(table_stride=15), INV), (dict(table_stride=0), INV),
            (dict(table_stride=(1 << 31) + 1), INV), (dict(v=at(0)), INV), (dict(v=at(0, PAGE // 2)), INV),
            (dict(page_stride=2 * 64 * 4 * 128, v=at(0, PAGE - 16)), INV), (dict(page_stride=2 * 64 * 4 * 128, v=at(0, PAGE + 16)), INV)]


def test_append_refusals(capi):
    lib, C = capi.load(), capi
    INV, UNS = C.EC_ERR_INVALID_ARG, C.EC_ERR_UNSUPPORTED
    good = params(C)

    def call(p=good, c=None, n=32, k=None, v=None, q=None, q_out=at(13), cs=at(14), sn=at(15), idx=at(16), stride=1024, start=None, R=at(17),
             err=None, no_q=False):
        ref = lambda x, d: ctypes.byref(d if x is None else x)  # noqa: E731
        return lib.ec_kv_append_paged(ctypes.byref(p), ref(c, pool(C)), n, ref(k, rows(C, at(10), 4, 32)), ref(v, rows(C, at(11), 4, 32)),
                                      None if no_q else ref(q, rows(C, at(12), 8, 32)), q_out, cs, sn, idx, stride, start, R, err, None)

    for kw, want in bad_pools(C):
        assert call(c=pool(C, **kw)) == want, kw
    for kw, want in [(dict(B=0), INV), (dict(B=4097), INV), (dict(L=0), INV), (dict(Hkv=0), INV), (dict(Hkv=3), INV), (dict(D=96), UNS)]:
        assert call(p=params(C, **kw)) == want, kw
    assert call(n=0) == INV and call(n=1025) == INV and call(n=-1) == INV
    for arg, heads, base in (("k", 4, 10), ("v", 4, 11), ("q", 8, 12)):
        for kw in (dict(x=None), dict(x=at(base, 8)), dict(batch_stride=-8), dict(row_stride=-8), dict(batch_stride=12), dict(row_stride=heads * 128 + 4),
                   dict(row_stride=heads * 128 - 8), dict(row_stride=1 << 37), dict(batch_stride=1 << 41)):
            assert call(**{arg: rows(C, **dict(dict(x=at(base), heads=heads, rows_max=32), **kw))}) == INV, (arg, kw)
        assert call(**{arg: rows(C, at(0, 32), heads, 32)}) == INV  # inside the pool
        assert call(**{arg: rows(C, at(13), heads, 32)}) == INV  # under q_out
    assert call(q_out=None) == INV and call(no_q=True) == INV  # one without the other
    assert call(cs=None) == INV and call(sn=None) == INV
    assert call(cs=at(14, 8)) == INV and call(sn=at(15, 4)) == INV and call(q_out=at(13, 2)) == INV
    assert call(R=None) == INV and call(R=at(17, 2)) == INV and call(err=at(18, 1)) == INV and call(idx=at(16, 2)) == INV
    assert call(stride=31) == INV and call(stride=(1 << 31) + 1) == INV
    assert call(start=at(19)) == INV  # with idx
    assert call(idx=None, start=at(19, 2)) == INV
    assert call(q_out=at(0, PAGE)) == INV and call(q_out=at(1)) == INV and call(q_out=at(16)) == INV and call(q_out=at(2)) == INV
    assert call(c=pool(C, table=at(0, 64))) == INV and call(R=at(1, 64)) == INV and call(cs=at(1)) == INV
    assert call(idx=None, start=at(0, 32)) == INV
    ref = ctypes.byref
    k = rows(C, at(10), 4, 32)
    assert lib.ec_kv_append_paged(None, ref(pool(C)), 32, ref(k), ref(k), None, None, None, None, None, 0, None, at(17), None, None) == INV
    assert lib.ec_kv_append_paged(ref(good), None, 32, ref(k), ref(k), None, None, None, None, None, 0, None, at(17), None, None) == INV
    assert lib.ec_kv_append_paged(ref(good), ref(pool(C)), 32, None, ref(k), None, None, None, None, None, 0, None, at(17), None, None) == INV


def test_attention_refusals(capi):
    lib, C = capi.load(), capi
    INV, UNS = C.EC_ERR_INVALID_ARG, C.EC_ERR_UNSUPPORTED
    good, big = params(C), 1 << 31

    def plain(p=good, n=32, q=at(20), c=None, R=at(21), kv_len=at(22), scale=0.1, out=at(23), ws=at(24), nws=big, err=None):
        c = pool(C) if c is None else c
        return lib.ec_paged_attention(ctypes.byref(p), n, q, ctypes.byref(c), R, kv_len, scale, out, ws, nws, err, None)

    def window(p=good, n=32, q=at(20), c=None, R=at(21), kv_len=at(22), scale=0.1, out=at(23), ws=at(24), nws=big, err=None, idx=at(25), stride=1024,
               start=None, left=5, right=5, sinks=1):
        c = pool(C) if c is None else c
        return lib.ec_paged_window_attention(ctypes.byref(p), n, q, ctypes.byref(c), idx, stride, start, R, kv_len, left, right, sinks, scale, out,
                                             ws, nws, err, None)

    for f in (plain, window):
        for kw, want in bad_pools(C):
            assert f(c=pool(C, **kw)) == want, kw
        for kw, want in [(dict(B=0), INV), (dict(L=0), INV), (dict(Hkv=3), INV), (dict(D=96), UNS), (dict(Hq=516), UNS),
                         (dict(scope_lo=5, scope_hi=2000), INV)]:
            assert f(p=params(C, **kw)) == want, kw
        assert f(n=0) == INV and f(n=1025) == INV
        assert f(p=params(C, B=4096, L=65536), n=65536, c=pool(C, table_stride=1024)) == UNS
        for scale in (0.0, -0.1, float("nan"), float("inf")):
            assert f(scale=scale) == INV
        for name, i in (("q", 20), ("R", 21), ("out", 23), ("ws", 24)):
            assert f(**{name: None}) == INV and f(**{name: at(i, 2)}) == INV
        assert f(kv_len=at(22, 1)) == INV and f(err=at(26, 2)) == INV and f(nws=16) == INV
        for over in (at(20, 64), at(0), at(1, PAGE), at(2), at(21), at(22)):
            assert f(out=over) == INV, over
            assert f(ws=over & ~15) == INV, over
        assert f(ws=at(23, 16)) == INV
    assert window(idx=at(25, 2)) == INV and window(stride=31) == INV and window(start=at(27)) == INV
    assert window(idx=None, start=at(27, 2)) == INV
    assert window(left=-2) == INV and window(right=-2) == INV and window(sinks=-1) == INV
    assert window(out=at(25)) == INV and window(idx=None, start=at(23)) == INV


def test_workspace_sizes(capi):
    lib, C = capi.load(), capi
    f = lib.ec_paged_attention_workspace_size
    assert f(None, 4) == 0 and f(ctypes.byref(params(C, D=96)), 4) == 0
    assert f(ctypes.byref(params(C)), 0) == 0 and f(ctypes.byref(params(C)), 1025) == 0
    sizes = [f(ctypes.byref(params(C)), n) for n in (1, 32, 1024)]
    assert all(0 < s < 1 << 30 for s in sizes)
    # it does not grow with the batch
    assert f(ctypes.byref(params(C, B=4096)), 1) <= 4 * f(ctypes.byref(params(C)), 1) + (1 << 22)


def test_binding_refuses_what_is_not_on_the_gpu(capi):
    import entropy_gated_kv_gb300 as E

    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        E.PagedCache(k, k.clone(), torch.zeros(1, 4, dtype=torch.int32))
