"""GPU tests of windows that end before, or reach far past, what a sequence has. Whatever no row may look at is NaN in the pool
and a junk page number in the table, so that a page looked up for nothing is reported."""
import pytest
import torch

from tests import _paged as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import entropy_gated_kv_gb300 as E

    E.lib()
    return E


@pytest.mark.parametrize("R", [1, 20, 150])
@pytest.mark.parametrize("sinks", [0, 4, 130])
@pytest.mark.parametrize("n", [1, 100, 150, 160, 250])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_rows_past_the_last_key(E, R, sinks, n, page):
    """Positions from 290 on with ten keys to either side, of sequences that end before: the first keys are all they see, or none."""
    P.Case(2, 450, 4, 2, 64, page, [R, R], [n, 280], (10, 10, sinks), at="start", pos=[290, 300], seed=n).run(E)


@pytest.mark.parametrize("side", [0, 1, 2])
@pytest.mark.parametrize("much", [2**31 - 1, 2**31, 2**32, 2**32 + 3, 2**63 - 1, 2**64])
def test_windows_wider_than_32_bits(E, side, much):
    """A side, or the first keys, of any size: all there is."""
    window = [5, 5, 0]
    window[side] = much
    every = [5, 5, 0]
    every[side] = 400
    c = P.Case(1, 300, 2, 1, 64, 16, [20], None, tuple(every), at="start", pos=[140], seed=1)
    d = c.inputs(E)
    c.window = tuple(window)
    c.call(E, d)
    torch.cuda.synchronize()
    assert int(d["dev_err"].item()) == 0
    c.window = tuple(every)
    c.check(d["out"])


@pytest.mark.parametrize("side", [0, 1, 2])
def test_windows_below_32_bits(E, side):
    c = P.Case(1, 300, 2, 1, 64, 16, [20], None, (5, 5, 0), at="start", pos=[140], seed=1)
    d = c.inputs(E)
    for bad in (-2 if side < 2 else -1, -(2**31) - 1, -(2**32), -(2**32) + 7, -(2**63)):
        c.window = tuple(bad if i == side else 5 for i in range(3))
        with pytest.raises(E.EcError):
            c.call(E, d)
