"""GPU tests of the paged cache's operators at the ends of what they accept."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import entropy_gated_kv_gb300 as E

    E.lib()
    return E


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_few_rows_in_a_large_array(E):
    """Two rows in an array whose rows' pieces, all in all, are more than 2^31: nothing past R is read or written."""
    rows, Hkv, D, page = 65600, 2048, 128, 16  # 2^15 pieces a row
    p = E.Params(B=1, L=rows, Hq=Hkv, Hkv=Hkv, D=D, V=8, C_max=1, k=1)
    x = torch.empty(1, rows, Hkv, D, dtype=torch.bfloat16, device="cuda")  # 34 GB; keys and values are the same rows
    x[0, :2].normal_()
    table = torch.full((1, -(-rows // page)), -1, dtype=torch.int32, device="cuda")
    table[0, 7] = 1
    cache = E.PagedCache.empty(3, page, Hkv, D, table)
    err = i32([0])
    E.kv_append_paged(p, cache, x, x, i32([2]), start=i32([7 * page + 14]), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0  # any other position has no page
    for t in (cache.k, cache.v):
        assert torch.equal(t[1, 14:], x[0, :2])
        assert not t[0].any() and not t[2].any() and not t[1, :14].any()


def test_storage_that_shrank_where_it_lay(E):
    """A cache whose memory was given back and taken anew, smaller, may find it at the same address."""
    torch.cuda.empty_cache()
    k = torch.zeros(256, 64, 8, 128, dtype=torch.bfloat16, device="cuda")  # 32 MiB
    v, table = torch.zeros_like(k), torch.zeros(1, 8, dtype=torch.int32, device="cuda")
    cache = E.PagedCache(k, v, table)
    for t in (k, v):
        full = t.untyped_storage().nbytes()
        t.untyped_storage().resize_(0)
        t.untyped_storage().resize_(full - full // 4)
        with pytest.raises(ValueError, match="has become smaller"):
            cache.view()
        t.untyped_storage().resize_(full)
    cache.view()


@pytest.mark.parametrize("R", [4, 300])
def test_a_position_that_comes_back(E, R):
    """idx that fall and come back to a position are reported; the row above its successor is left out, the others are in their
    places. (The two rows of the one position hold the same bits here: which of two different ones stays is not specified.)"""
    L, H, D, page = 400, 2, 128, 16
    p = E.Params(B=1, L=L, Hq=H, Hkv=H, D=D, V=8, C_max=1, k=1)
    pos = list(range(R))
    pos[1:3] = [9, 0]
    pos[3:] = range(20, 20 + R - 3)
    x = torch.randn(1, R, 2 * H, D, device="cuda").to(torch.bfloat16)
    x[0, 2] = x[0, 0]
    table = torch.randperm(L // page, device="cuda").to(torch.int32)[None]
    cache, err = E.PagedCache.empty(L // page, page, H, D, table), i32([0])
    E.kv_append_paged(p, cache, x[:, :, :H], x[:, :, H:], i32([R]), idx=i32([pos]), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == E._capi.EC_DEVERR_BAD_IDX
    want = torch.zeros(L, 2 * H, D, dtype=torch.bfloat16, device="cuda")
    for r in [0, *range(3, R)]:
        want[pos[r]] = x[0, r]
    got = torch.cat([cache.k[table[0].long()].flatten(0, 1), cache.v[table[0].long()].flatten(0, 1)], 1)
    assert torch.equal(got, want)


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1.0])
@pytest.mark.parametrize("L,lengths", [(300, False), (300, True), (20000, False), (20000, True)])  # joined on the chip, by a second launch
@pytest.mark.parametrize("R", [1, 20, 150])
def test_rows_without_weight_are_zeros(E, R, L, lengths, value):
    """Every score of the second sequence is -infinity: its rows are zeros, whatever the values are."""
    B, H, D, page = 2, 2, 64, 64
    p = E.Params(B=B, L=L, Hq=H, Hkv=H, D=D, V=8, C_max=1, k=1)
    per = -(-L // page)
    table = torch.arange(B * per, device="cuda").to(torch.int32).view(B, per)
    cache = E.PagedCache.empty(B * per, page, H, D, table)
    cache.v.fill_(1.0)
    cache.k[per:], cache.v[per:] = -float("inf"), value
    q, err = torch.ones(B, R, H, D, dtype=torch.bfloat16, device="cuda"), i32([0])
    out = torch.full_like(q, -123.0)
    E.paged_attention(p, q, cache, i32([R, R]), out, kv_len=i32([L, L]) if lengths else None, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert (out[0] == 1).all()
    assert (out[1] == 0).all()
