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
