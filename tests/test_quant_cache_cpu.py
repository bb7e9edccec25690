"""The 8-bit cache and the shared-prefix attention without a GPU: what the C ABI and the binding
refuse, the workspace sizes, and the plain row format that the GPU tests compare with.

The pointers are never dereferenced: every call fails validation before it reaches CUDA.
"""
import ctypes

import numpy as np
import pytest
import torch

from tests import _quant as Q


@pytest.fixture(scope="module")
def capi():
    from entropy_gated_kv_gb300 import build as B

    B.build()
    from entropy_gated_kv_gb300 import _capi as C

    C.load()
    return C


def params(C, **kw):
    base = dict(B=1, L=1024, Hq=32, Hkv=32, D=128, V=8, C_max=1, k=1, n_dec=1, tau=1.0, logits_dtype=C.EC_BF16)
    base.update(kw)
    return C.EcParams(**base)


STEP = 1 << 32  # far apart: no two buffers overlap


def at(i, off=0):
    return STEP * (i + 1) + off


def kv(C, dtype=None, len=1024, first=0, **kw):
    a = dict(k=at(first), v=at(first + 1), k_exp=at(first + 2), v_exp=at(first + 3))
    a.update(kw)
    return C.EcKv(C.EC_E4M3 if dtype is None else dtype, len, a["k"], a["v"], a["k_exp"], a["v_exp"])


def test_scatter_and_gather_refusals(capi):
    lib, C = capi.load(), capi
    INV, UNS = C.EC_ERR_INVALID_ARG, C.EC_ERR_UNSUPPORTED
    good = params(C)

    def scatter(p=good, c=None, kn=at(8), vn=at(9), by_pos=0, idx=at(10), R=at(11)):
        c = kv(C) if c is None else c
        return lib.ec_kv_scatter_quant(ctypes.byref(p), ctypes.byref(c), kn, vn, by_pos, idx, R, None, None)

    def gather(p=good, c=None, kn=at(8), vn=at(9), idx=at(10), R=at(11)):
        c = kv(C) if c is None else c
        return lib.ec_kv_gather_quant(ctypes.byref(p), ctypes.byref(c), idx, R, kn, vn, None, None)

    for f in (scatter, gather):
        for kw, want in [(dict(B=0), INV), (dict(B=4097), INV), (dict(L=0), INV), (dict(Hkv=0), INV), (dict(Hkv=65537), INV),
                         (dict(D=96), UNS)]:
            assert f(p=params(C, **kw)) == want, kw
        assert f(c=kv(C, len=1023)) == INV  # not the sequence length
        assert f(c=kv(C, dtype=C.EC_BF16)) == UNS
        assert f(c=kv(C, dtype=7)) == INV
        for name in ("k", "v", "k_exp", "v_exp"):
            assert f(c=kv(C, **{name: None})) == INV
            assert f(c=kv(C, **{name: at(0, 8)})) == INV  # alignment
        assert f(kn=None) == INV and f(vn=None) == INV and f(R=None) == INV
        assert f(kn=at(8, 2)) == INV and f(vn=at(9, 4)) == INV
        assert f(kn=at(0, 1024)) == INV and f(vn=at(2, 16)) == INV  # inside the cache
    assert scatter(c=kv(C, v=at(0, 4096))) == INV  # the cache's arrays overlap
    assert scatter(idx=None) == INV and scatter(by_pos=2) == INV
    assert gather(kn=at(8), vn=at(8, 256)) == INV
    assert lib.ec_kv_scatter_quant(None, None, at(8), at(9), 0, at(10), at(11), None, None) == INV
    assert lib.ec_kv_scatter_quant(ctypes.byref(good), None, at(8), at(9), 0, at(10), at(11), None, None) == INV


def test_attention_refusals(capi):
    lib, C = capi.load(), capi
    INV, UNS = C.EC_ERR_INVALID_ARG, C.EC_ERR_UNSUPPORTED
    good = params(C)
    big = 1 << 31

    def quant(p=good, q=at(20), c=None, R=at(21), n=at(22), scale=0.1, out=at(23), ws=at(24), nws=big):
        c = kv(C) if c is None else c
        return lib.ec_partial_attention_quant(ctypes.byref(p), q, ctypes.byref(c), R, n, scale, out, ws, nws, None, None)

    def prefix(p=good, q=at(20), c=None, R=at(21), n=at(22), scale=0.1, out=at(23), ws=at(24), nws=big, pre=None):
        c = kv(C) if c is None else c
        pre = kv(C, len=500, first=30) if pre is None else pre
        return lib.ec_prefix_attention(ctypes.byref(p), q, ctypes.byref(pre), ctypes.byref(c), R, n, scale, out, ws, nws,
                                       None, None)

    for f in (quant, prefix):
        for kw, want in [(dict(B=0), INV), (dict(L=0), INV), (dict(Hkv=5), INV), (dict(D=96), UNS), (dict(Hq=256, Hkv=1), UNS),
                         (dict(scope_lo=5, scope_hi=2000), INV)]:
            assert f(p=params(C, **kw)) == want, kw
        for scale in (0.0, -0.1, float("nan"), float("inf")):
            assert f(scale=scale) == INV
        assert f(q=None) == INV and f(R=None) == INV and f(out=None) == INV and f(ws=None) == INV
        assert f(q=at(20, 2)) == INV and f(out=at(23, 8)) == INV and f(ws=at(24, 4)) == INV
        assert f(nws=1024) == INV
        assert f(c=kv(C, len=1000)) == INV and f(c=kv(C, k_exp=None)) == INV
        assert f(out=at(20, 1024)) == INV  # over q
        assert f(out=at(1)) == INV and f(out=at(2)) == INV  # over the cache's values, its exponents
        assert f(ws=at(0)) == INV and f(ws=at(23, 16)) == INV
    assert quant(c=kv(C, dtype=C.EC_BF16)) == UNS
    assert prefix(pre=kv(C, len=-1, first=30)) == INV
    assert prefix(pre=kv(C, len=(1 << 20) + 1, first=30)) == INV
    assert prefix(pre=kv(C, len=500, first=30, v=None)) == INV
    assert prefix(pre=kv(C, len=500, first=30, v=at(31, 2))) == INV
    assert prefix(pre=kv(C, dtype=C.EC_BF16, len=500, first=30)) == UNS  # 8-bit cache, bf16 prefix
    assert prefix(c=kv(C, dtype=C.EC_BF16)) == UNS
    assert prefix(pre=kv(C, len=500, first=30, k=at(23))) == INV  # out over the prefix


def test_workspace_sizes(capi):
    lib, C = capi.load(), capi
    for f in (lib.ec_partial_attention_quant_workspace_size, lib.ec_prefix_attention_workspace_size):
        assert f(ctypes.byref(params(C, D=96))) == 0 and f(None) == 0
        assert f(ctypes.byref(params(C))) > f(ctypes.byref(params(C, D=64))) > 0
        # bounded by the SM count, whatever the batch and the length
        assert f(ctypes.byref(params(C, B=64, L=1 << 17, Hq=4, Hkv=4))) <= 8 * 160 * (128 * (128 * 4 + 8) + 32) + 32


def test_binding_refuses_cpu_tensors_types_and_shapes(capi):
    import entropy_gated_kv_gb300 as E

    p = E.Params(B=1, L=32, Hq=4, Hkv=2, D=64, V=8, C_max=1, k=1)
    t = torch.zeros(1, 32, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        E.QuantCache(t, t, None, None)
    c8 = t.to(torch.float8_e4m3fn)
    e = torch.zeros(1, 2, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        E.QuantCache(c8, c8, e, e)
    with pytest.raises(ValueError):
        E.prefix_attention(p, t, (t[0], t[0]), (t, t), None, t)


def test_plain_row_format():
    # against torch's own conversion, and the exponent's definition at its borders
    rng = np.random.default_rng(0)
    x = Q.f64(Q.bf16(rng.standard_normal((400, 64)) * 2.0 ** rng.integers(-100, 100, (400, 1))))
    c, e = Q.quantise(x)
    want = torch.from_numpy(x * 2.0 ** (127.0 - e[:, None])).float().to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(c, Q.code_values(want))
    m = np.abs(x).max(1)
    assert (m <= 448 * 2.0 ** (e - 127.0)).all() and (m > 224 * 2.0 ** (e - 127.0)).all()
    for a, byte in [(0.0, 17), (448.0, 127), (450.0, 128), (224.0, 126), (1e-38, 17), (3.3e38, 247)]:
        row = np.zeros((1, 64))
        row[0, 3] = -float(Q.bf16(np.array([a])).float())
        assert Q.quantise(row)[1][0] == byte, a
    for bad in (np.nan, np.inf, -np.inf):
        row = np.ones((1, 64))
        row[0, 5] = bad
        c, e = Q.quantise(row)
        assert e[0] == 255 and np.isnan(c).all()


def test_sizes_that_leave_32_bits_are_refused(capi):
    lib, C = capi.load(), capi
    # 2 L Hkv and B L Hq at 2^31 and just below, where the next check (a null pointer) answers
    for L, Hkv, want in [(1 << 16, 1 << 14, C.EC_ERR_UNSUPPORTED), ((1 << 16) - 1, 1 << 14, C.EC_ERR_INVALID_ARG)]:
        p, c = params(C, L=L, Hq=Hkv, Hkv=Hkv), kv(C, len=L)
        assert lib.ec_kv_scatter_quant(ctypes.byref(p), ctypes.byref(c), None, at(9), 0, at(10), at(11), None, None) == want
        assert lib.ec_kv_gather_quant(ctypes.byref(p), ctypes.byref(c), at(10), at(11), None, at(9), None, None) == want
    for B, L, want in [(128, 1 << 17, C.EC_ERR_UNSUPPORTED), (128, (1 << 17) - 1, C.EC_ERR_INVALID_ARG)]:
        p, c = params(C, B=B, L=L, Hq=128, Hkv=128, D=64), kv(C, len=L)
        assert lib.ec_partial_attention_quant(ctypes.byref(p), None, ctypes.byref(c), at(21), None, 0.1, at(23), at(24), 1 << 31,
                                              None, None) == want


def test_outputs_over_sizes_and_indices_are_refused(capi):
    lib, C = capi.load(), capi
    p, c = params(C), kv(C)
    P, INV = ctypes.byref, C.EC_ERR_INVALID_ARG
    assert lib.ec_partial_attention_quant(P(p), at(20), P(c), at(23, 64), None, 0.1, at(23), at(24), 1 << 31, None, None) == INV
    assert lib.ec_partial_attention_quant(P(p), at(20), P(c), at(21), at(24, 64), 0.1, at(23), at(24), 1 << 31, None, None) == INV
    assert lib.ec_partial_attention_quant(P(p), at(20), P(c), at(21), None, 3e38, at(23), at(24), 1 << 31, None, None) == INV
    assert lib.ec_kv_scatter_quant(P(p), P(c), at(8), at(9), 0, at(0, 64), at(11), None, None) == INV
    assert lib.ec_kv_scatter_quant(P(p), P(c), at(8), at(9), 0, at(10), at(3, 64), None, None) == INV
    assert lib.ec_kv_gather_quant(P(p), P(c), at(8, 64), at(11), at(8), at(9), None, None) == INV
    assert lib.ec_kv_gather_quant(P(p), P(c), at(10), at(9, 64), at(8), at(9), None, None) == INV


def test_params_are_copied_and_pickled_after_use(capi):
    import copy
    import pickle

    import entropy_gated_kv_gb300 as E

    p = E.Params(B=2, L=32, Hq=4, Hkv=2, D=64, V=8, C_max=1, k=1)
    one = E.partial_attention_quant_workspace_size(p)
    assert one > E.partial_attention_quant_workspace_size(E.Params(B=2, L=32, Hq=4, Hkv=2, D=128, V=8, C_max=1, k=1)) // 4
    for q in (copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p))):
        assert q == p
        q.D = 128  # a copy's change reaches the C view, and the copy's only
        assert E.partial_attention_quant_workspace_size(q) > one
        assert E.partial_attention_quant_workspace_size(p) == one
    p.D = 96
    assert E.partial_attention_quant_workspace_size(p) == 0


def test_unaligned_words_are_refused(capi):
    lib, C = capi.load(), capi
    p, c = params(C), kv(C)
    P, INV = ctypes.byref, C.EC_ERR_INVALID_ARG
    for R, n, err in [(at(21, 2), None, None), (at(21), at(22, 1), None), (at(21), None, at(25, 2))]:
        assert lib.ec_partial_attention_quant(P(p), at(20), P(c), R, n, 0.1, at(23), at(24), 1 << 31, err, None) == INV
    for idx, R, err in [(at(10, 2), at(11), None), (at(10), at(11, 1), None), (at(10), at(11), at(12, 3))]:
        assert lib.ec_kv_scatter_quant(P(p), P(c), at(8), at(9), 0, idx, R, err, None) == INV
        assert lib.ec_kv_gather_quant(P(p), P(c), idx, R, at(8), at(9), err, None) == INV


class _Tensor:
    """What the binding asks of a CUDA tensor."""

    def __init__(self, shape, dtype, ptr):
        self.shape, self.dtype, self.ptr, self.contiguous, self.device, self.index = shape, dtype, ptr, True, "cuda:0", 0

    def data_ptr(self):
        return self.ptr

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous


def test_a_cache_tensor_changed_in_place_is_checked_again(capi):
    import entropy_gated_kv_gb300 as E

    def fresh():
        k, v = (_Tensor((2, 40, 3, 64), torch.float8_e4m3fn, at(i)) for i in (0, 1))
        ke, ve = (_Tensor((2, 3, 48), torch.uint8, at(i)) for i in (2, 3))
        return E.QuantCache(k, v, ke, ve)

    c = fresh()
    view = c.view()
    assert c.view() is view  # nothing has changed
    for name in ("k", "v", "k_exp", "v_exp"):
        for attribute, value in (("shape", (2, 20, 3, 64)), ("dtype", torch.int8), ("contiguous", False)):
            c = fresh()
            c.view()
            setattr(getattr(c, name), attribute, value)  # the address stays
            for _ in range(2):
                with pytest.raises(ValueError):
                    c.view()
    # all of them to another length: a new view, and calls for the old length are refused
    c = fresh()
    for t in (c.k, c.v):
        t.shape = (2, 20, 3, 64)
    for t in (c.k_exp, c.v_exp):
        t.shape = (2, 3, 32)
    assert c.view().shape == (2, 20, 3, 64) and c.view().c.len == 20
    with pytest.raises(ValueError, match="cache must be"):
        E.kv_scatter_quant(E.Params(B=2, L=40, Hq=3, Hkv=3, D=64, V=8, C_max=1, k=1), c, None, None, None, None)


def test_params_hold_their_fields_and_nothing_else(capi):
    import dataclasses

    import entropy_gated_kv_gb300 as E

    p = E.Params(B=2, L=32, Hq=4, Hkv=2, D=64, V=8, C_max=1, k=1)
    names = [f.name for f in dataclasses.fields(E.Params)]
    for _ in range(2):
        assert list(p.__dict__) == names == list(vars(p))
        assert E.Params(**p.__dict__) == p and E.Params(**{**vars(p), "D": 128}).D == 128
        assert dataclasses.asdict(p) == p.__dict__
        one = E.prefix_attention_workspace_size(p)  # the C view is made, and used again
    # a change reaches the C view however it is made
    other = E.prefix_attention_workspace_size(E.Params(B=2, L=32, Hq=4, Hkv=2, D=128, V=8, C_max=1, k=1))
    assert other != one
    p.__dict__["D"] = 128
    assert E.prefix_attention_workspace_size(p) == other
    vars(p).update(D=64)
    assert E.prefix_attention_workspace_size(p) == one
    p.D = 128
    assert E.prefix_attention_workspace_size(p) == other
    assert E.prefix_attention_workspace_size(dataclasses.replace(p, D=64)) == one
