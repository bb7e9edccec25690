"""GPU tests of the 8-bit K/V cache: the quantising scatter and the gather that reads rows back,
bit for bit against the plain format in 64 bits (tests/_quant.py)."""
import numpy as np
import pytest
import torch

from tests import _quant as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import entropy_gated_kv_gb300 as E

    E.lib()
    return E


def params(E, B, L, Hkv, D):
    return E.Params(B=B, L=L, Hq=Hkv, Hkv=Hkv, D=D, V=8, C_max=1, k=1)


def rows_of(rng, B, L, Hkv, D):
    """bf16 rows of very different magnitudes, among them zero rows, subnormals, the largest value
    and rows on the exponent's border (448 2^e and its successor)."""
    x = rng.standard_normal((B, L, Hkv, D)) * 2.0 ** rng.integers(-120, 110, (B, L, Hkv, 1))
    kind = rng.integers(0, 12, (B, L, Hkv))
    x[kind == 0] = 0.0
    x[kind == 1] *= 2.0**-20  # below the smallest exponent, subnormals
    near = rng.integers(-30, 30, (B, L, Hkv))[..., None]
    edge = np.where(rng.random((B, L, Hkv, 1)) < 0.5, 448.0, 450.0) * 2.0**near
    x = np.where((kind == 2)[..., None], np.clip(x, -edge, edge), x)
    x[..., 1] = np.where(kind == 2, -edge[..., 0], x[..., 1])
    x[..., 2] = np.where(kind == 3, 3.3895e38, x[..., 2])
    return Q.bf16(np.clip(x, -3.3895e38, 3.3895e38))


def positions(rng, L, r):
    return np.sort(rng.permutation(L)[:r]).astype(np.int32)


def cache_of(E, B, L, Hkv, D, fill=0x5A):
    S = -(-L // 16) * 16
    u8 = lambda *s: torch.full(s, fill, dtype=torch.uint8, device="cuda")  # noqa: E731
    return E.QuantCache(u8(B, L, Hkv, D).view(torch.float8_e4m3fn), u8(B, L, Hkv, D).view(torch.float8_e4m3fn),
                        u8(B, Hkv, S), u8(B, Hkv, S))


@pytest.mark.parametrize("B,L,Hkv,D,Rs", [
    (1, 256, 8, 64, [47]),
    (1, 1024, 32, 128, [95]),
    (1, 1, 1, 64, [1]),
    (1, 1, 1, 128, [1]),
    (3, 77, 3, 128, [77, 0, 5]),      # odd length (padded exponent rows), an empty sequence, row_vecs 48
    (2, 300, 1, 64, [300, 299]),
    (2, 40, 65, 64, [39, 2]),         # more vectors per position than one pass of a CTA
    (40, 17, 2, 128, [17] * 40),
])
@pytest.mark.parametrize("by_pos", [False, True])
def test_scatter_and_gather_bits(E, B, L, Hkv, D, Rs, by_pos):
    rng = np.random.default_rng(B * 1000 + L)
    k, v = rows_of(rng, B, L, Hkv, D), rows_of(rng, B, L, Hkv, D)
    idx = np.zeros((B, L), np.int32)
    for b, r in enumerate(Rs):
        idx[b, :r] = positions(rng, L, r)
    p, cache = params(E, B, L, Hkv, D), cache_of(E, B, L, Hkv, D)
    di, dR = torch.from_numpy(idx).cuda(), torch.tensor(Rs, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.kv_scatter_quant(p, cache, k.cuda(), v.cuda(), di, dR, src_by_position=by_pos, dev_err=err)
    out = tuple(torch.full((B, L, Hkv, D), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    E.kv_gather_quant(p, cache, di, dR, out=out, dev_err=err)
    assert E.read_device_error(err) == (0, 0)
    for x, code, eb, back in ((k, cache.k, cache.k_exp, out[0]), (v, cache.v, cache.v_exp, out[1])):
        want_c, want_e = Q.quantise(Q.f64(x))
        got_c, got_e = Q.code_values(code), eb.cpu().numpy()
        raw, got = code.view(torch.uint8).cpu().numpy(), Q.f64(back)
        for b, r in enumerate(Rs):
            pos = idx[b, :r]
            src = pos if by_pos else np.arange(r)
            np.testing.assert_array_equal(got_c[b, pos], want_c[b, src])
            np.testing.assert_array_equal(got_e[b][:, pos].T, want_e[b, src])
            rest = np.setdiff1d(np.arange(L), pos)
            assert (raw[b, rest] == 0x5A).all() and (got_e[b][:, rest] == 0x5A).all(), "other rows were written"
            assert (got_e[b][:, L:] == 0x5A).all(), "the padding was written"
            # exact: a code times its power of two is a bf16 number
            np.testing.assert_array_equal(got[b, :r], want_c[b, src] * 2.0 ** (want_e[b, src].astype(float) - 127)[..., None])
            assert (got[b, r:] == -7.0).all(), "rows at and past R were written"


def test_every_code_and_exponent_reads_back_exactly(E):
    L = 247 - 17 + 1
    cache = cache_of(E, 1, L, 4, 64)
    codes = torch.arange(256, dtype=torch.uint8).view(4, 64)
    codes[1, 63] = codes[3, 63] = 0  # 0x7F and 0xFF, NaN: written only in rows of exponent byte 255
    for t, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
        t.view(torch.uint8).copy_(codes.cuda()[None, None].expand(1, L, 4, 64))
        e[:, :, :L] = torch.arange(17, 248, dtype=torch.uint8, device="cuda")
    k, v = E.kv_gather_quant(params(E, 1, L, 4, 64), cache, None, torch.tensor([L], dtype=torch.int32, device="cuda"))
    want = Q.widen(cache.k, cache.k_exp)
    fits = np.abs(want) < 3.39e38  # byte 247 with codes above 255/256 448 has no bf16 value
    for got in (Q.f64(k), Q.f64(v)):
        np.testing.assert_array_equal(got[fits], want[fits])
        assert np.isinf(got[~fits]).all()


def test_non_finite_rows(E):
    p, cache = params(E, 1, 40, 2, 128), cache_of(E, 1, 40, 2, 128)
    rng = np.random.default_rng(3)
    x = rng.standard_normal((1, 40, 2, 128))
    x[0, 3, 1, 77], x[0, 5, 0, 0], x[0, 6, 0, 127] = np.nan, np.inf, -np.inf
    k = Q.bf16(x)
    idx, R = torch.arange(40, dtype=torch.int32, device="cuda")[None], torch.tensor([40], dtype=torch.int32, device="cuda")
    E.kv_scatter_quant(p, cache, k.cuda(), k.cuda(), idx.contiguous(), R)
    back, _ = E.kv_gather_quant(p, cache, idx.contiguous(), R)
    want_c, want_e = Q.quantise(Q.f64(k))
    np.testing.assert_array_equal(Q.code_values(cache.k), want_c)
    np.testing.assert_array_equal(cache.k_exp[0, :, :40].T.cpu().numpy(), want_e[0])
    nan_rows = np.zeros((40, 2), bool)
    nan_rows[3, 1] = nan_rows[5, 0] = nan_rows[6, 0] = True
    np.testing.assert_array_equal(np.isnan(Q.f64(back)[0]).all(-1), nan_rows)
    np.testing.assert_array_equal(np.isnan(Q.f64(back)[0]).any(-1), nan_rows)


def test_bad_indices_are_reported_and_skipped(E):
    from entropy_gated_kv_gb300 import _capi as C

    p = params(E, 3, 32, 2, 64)
    k = Q.bf16(np.random.default_rng(1).standard_normal((3, 32, 2, 64))).cuda()
    idx = torch.zeros(3, 32, dtype=torch.int32)
    idx[0, :5] = torch.tensor([1, 4, 4, 9, 32])   # a repeated position, one past the end
    idx[1, :3] = torch.tensor([7, -1, 3])         # descending and negative
    idx[2, :2] = torch.tensor([0, 1])
    R = torch.tensor([5, 3, 33], dtype=torch.int32, device="cuda")
    cache, err = cache_of(E, 3, 32, 2, 64), torch.zeros(1, dtype=torch.int32, device="cuda")
    E.kv_scatter_quant(p, cache, k, k, idx.cuda(), R, dev_err=err)
    assert E.read_device_error(err)[1] == C.EC_DEVERR_BAD_IDX | C.EC_DEVERR_BAD_R
    written = (cache.k_exp[:, 0, :32].cpu() != 0x5A)
    want = torch.zeros(3, 32, dtype=torch.bool)
    want[0, [1, 4, 9]] = True  # the second 4 is written, the first is skipped
    want[1, 3] = True
    assert torch.equal(written, want)
    c, _ = Q.quantise(Q.f64(k))
    np.testing.assert_array_equal(Q.code_values(cache.k)[0, 4], c[0, 2])
    err.zero_()
    out = tuple(torch.zeros(3, 32, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    E.kv_gather_quant(p, cache, idx.cuda(), R, out=out, dev_err=err)
    assert E.read_device_error(err)[1] == C.EC_DEVERR_BAD_IDX | C.EC_DEVERR_BAD_R
    assert not out[0][0, 4].any() and out[0][0, 2].any()  # the bad row is left as it was
    assert torch.equal(out[0][0, 1], out[0][0, 2])        # a repeated position reads twice


def test_full_refresh_past_32_bit_offsets(E):
    # 2^31 code bytes lie below position 131080 (128 x 128 bytes each): the rows behind are read and written
    # where they belong
    L, Hkv, D = 131080 + 24, 128, 128
    p = params(E, 1, L, Hkv, D)
    cache = E.QuantCache.empty(1, L, Hkv, D)
    rng = np.random.default_rng(4)
    pos = np.array([0, 5, 131071, 131072, 131079, L - 1], np.int32)
    idx = torch.zeros(1, L, dtype=torch.int32, device="cuda")
    idx[0, :6] = torch.from_numpy(pos).cuda()
    new = torch.zeros(1, L, Hkv, D, dtype=torch.bfloat16, device="cuda")
    x = Q.bf16(rng.standard_normal((6, Hkv, D)))
    new[0, torch.from_numpy(pos).cuda().long()] = x.cuda()
    R = torch.tensor([6], dtype=torch.int32, device="cuda")
    E.kv_scatter_quant(p, cache, new, new.clone(), idx, R, src_by_position=True)
    c, e = Q.quantise(Q.f64(x))
    np.testing.assert_array_equal(Q.code_values(cache.v[0, torch.from_numpy(pos).cuda().long()]), c)
    np.testing.assert_array_equal(cache.v_exp[0][:, torch.from_numpy(pos).cuda().long()].T.cpu().numpy(), e)
    assert int((cache.k.view(torch.uint8) != 0).any(-1).any(-1).sum()) == 6
    del new
    k, _ = E.kv_gather_quant(p, cache, idx, R)
    np.testing.assert_array_equal(Q.f64(k[0, :6]), c * 2.0 ** (e.astype(float) - 127)[..., None])


def test_graph_and_another_stream(E):
    p, cache = params(E, 2, 200, 4, 128), cache_of(E, 2, 200, 4, 128)
    rng = np.random.default_rng(6)
    k, v = (Q.bf16(rng.standard_normal((2, 200, 4, 128))).cuda() for _ in range(2))
    idx = torch.stack([torch.from_numpy(positions(rng, 200, 200)) for _ in range(2)]).cuda()
    R = torch.tensor([50, 200], dtype=torch.int32, device="cuda")
    out = tuple(torch.zeros(2, 200, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        E.kv_scatter_quant(p, cache, k, v, idx, R)
        E.kv_gather_quant(p, cache, idx, R, out=out)
    k.copy_(Q.bf16(rng.standard_normal((2, 200, 4, 128))).cuda())
    R.copy_(torch.tensor([200, 3], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    c, e = Q.quantise(Q.f64(k))
    want = c * 2.0 ** (e.astype(float) - 127)[..., None]
    np.testing.assert_array_equal(Q.f64(out[0])[0], want[0])
    np.testing.assert_array_equal(Q.f64(out[0])[1, :3], want[1, :3])
    # the caller's stream, with the outputs made by the call
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    k2, _ = E.kv_gather_quant(p, cache, idx, R, stream=s2)
    s2.synchronize()
    np.testing.assert_array_equal(Q.f64(k2)[0], want[0])


@pytest.mark.parametrize("D", [64, 128])
def test_buffers_at_odd_multiples_of_16_bytes(E, D):
    # the alignment that the interface asks for, and no more
    B, L, Hkv = 2, 77, 3
    rng = np.random.default_rng(D)
    p = params(E, B, L, Hkv, D)

    def shifted(shape, dtype):  # a tensor that starts 16 bytes into its buffer
        n = int(np.prod(shape)) * (2 if dtype == torch.bfloat16 else 1)
        return torch.full((n + 16,), 0x5A, dtype=torch.uint8, device="cuda")[16:].view(dtype).view(shape)

    cache = E.QuantCache(*(shifted((B, L, Hkv, D), torch.uint8).view(torch.float8_e4m3fn) for _ in range(2)),
                         *(shifted((B, Hkv, 80), torch.uint8) for _ in range(2)))
    x = [rows_of(rng, B, L, Hkv, D) for _ in range(2)]
    new, out = [shifted((B, L, Hkv, D), torch.bfloat16) for _ in range(2)], [shifted((B, L, Hkv, D), torch.bfloat16) for _ in range(2)]
    for a, b in zip(new, x):
        a.copy_(b)
    assert all(t.data_ptr() % 32 == 16 for t in (*new, *out, cache.k, cache.v_exp))
    Rs = [77, 40]
    idx = torch.from_numpy(np.stack([np.pad(positions(rng, L, r), (0, L - r)) for r in Rs])).cuda()
    R = torch.tensor(Rs, dtype=torch.int32, device="cuda")
    E.kv_scatter_quant(p, cache, *new, idx, R)
    E.kv_gather_quant(p, cache, idx, R, out=tuple(out))
    for a, b in zip(out, x):
        c, e = Q.quantise(Q.f64(b))
        want = c * 2.0 ** (e.astype(float) - 127)[..., None]
        for i, r in enumerate(Rs):
            np.testing.assert_array_equal(Q.f64(a)[i, :r], want[i, :r])


def test_a_cache_whose_tensors_are_exchanged(E):
    p, cache = params(E, 1, 32, 2, 64), E.QuantCache.empty(1, 32, 2, 64)
    x = Q.bf16(np.random.default_rng(0).standard_normal((1, 32, 2, 64))).cuda()
    idx, R = torch.arange(32, dtype=torch.int32, device="cuda")[None].contiguous(), torch.tensor([32], dtype=torch.int32, device="cuda")
    E.kv_scatter_quant(p, cache, x, x, idx, R)
    old, other = cache.k, E.QuantCache.empty(1, 32, 2, 64)
    cache.k, cache.k_exp = other.k, other.k_exp
    k, v = E.kv_gather_quant(p, cache, idx, R)
    assert not k.any() and v.any()
    cache.k = old[:, :, :1]  # the same address, another shape
    with pytest.raises(ValueError):
        E.kv_gather_quant(p, cache, idx, R)
    with pytest.raises(ValueError):  # and stays refused
        E.kv_gather_quant(p, cache, idx, R)
    cache.k = other.k
    E.kv_gather_quant(p, cache, idx, R)


def test_a_cache_whose_tensors_change_in_place(E):
    p, cache = params(E, 1, 32, 2, 64), E.QuantCache.empty(1, 32, 2, 64)
    idx, R = torch.arange(32, dtype=torch.int32, device="cuda")[None].contiguous(), torch.tensor([32], dtype=torch.int32, device="cuda")
    E.kv_gather_quant(p, cache, idx, R)
    at = cache.k.data_ptr()
    cache.k.resize_(1, 16, 2, 64)
    assert cache.k.data_ptr() == at
    with pytest.raises(ValueError):
        E.kv_gather_quant(p, cache, idx, R)
    cache.k.resize_(1, 32, 2, 64)
    E.kv_gather_quant(p, cache, idx, R)
    cache.v.as_strided_((1, 32, 2, 64), (4096, 64, 2048, 1))
    with pytest.raises(ValueError):
        E.kv_gather_quant(p, cache, idx, R)


@pytest.mark.parametrize("D", [64, 128])
def test_nan_codes_read_as_nan_in_any_row(E, D):
    # all 256 codes under every exponent, e4m3's NaN codes among them: at each place of a 16-byte piece and
    # beside 0x7E, 0x00 and each other (a carry from one byte to the next)
    L, H = 247 - 17 + 1, 512 // D + 2
    rng = np.random.default_rng(D)
    codes = np.zeros((H, D), np.uint8)
    codes[: 256 // D] = np.arange(256, dtype=np.uint8).reshape(-1, D)
    codes[256 // D : 512 // D] = rng.permutation(256).astype(np.uint8).reshape(-1, D)
    codes[-2] = np.resize(np.array([0xFF, 0x7E, 0x7F, 0x00, 0xFF, 0xFF, 0xFE, 0x7F], np.uint8), D)
    codes[-1] = 0xFE
    codes[-1, D // 2 + 3] = 0x7F
    cache = cache_of(E, 1, L, H, D)
    for t, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
        t.view(torch.uint8).copy_(torch.from_numpy(codes).cuda()[None, None].expand(1, L, H, D))
        e[:, :, :L] = torch.arange(17, 248, dtype=torch.uint8, device="cuda")
    k, v = E.kv_gather_quant(params(E, 1, L, H, D), cache, None, torch.tensor([L], dtype=torch.int32, device="cuda"))
    want = Q.widen(cache.k, cache.k_exp)
    nan = (codes & 0x7F) == 0x7F
    assert (np.isnan(want[0]) == nan).all()
    fits = np.abs(want) < 3.39e38  # not NaN, and not past bf16's largest value
    for got in (Q.f64(k), Q.f64(v)):
        np.testing.assert_array_equal(np.isnan(got[0]), np.broadcast_to(nan, (L, H, D)))
        np.testing.assert_array_equal(got[fits], want[fits])
