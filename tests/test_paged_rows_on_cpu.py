"""The paged kernels' arithmetic on the CPU: their own header compiled for the host (tests/host), at the sizes that the
interface accepts and no GPU test can hold."""
import pytest

from tests.test_device_code_on_cpu import program, run  # noqa: F401

AT_ONCE = 384  # pieces that a CTA of the append takes at once
MOST = 1 << 20  # rows
# pieces of a row: one head of 64; queries, K and V of 8 and of 128 heads of 128; the widest rows that are accepted
NARROW, ORDINARY, WIDE, WIDEST = 8, 36 * 8, 3 * 128 * 9, 3 * (1 << 22)


@pytest.mark.parametrize("R", [0, 1, 2, 385])
@pytest.mark.parametrize("rows_max,pieces", [(385, NARROW), (385, WIDE), (385, WIDEST), (4096, ORDINARY), (MOST, NARROW), (MOST, ORDINARY),
                                             (MOST, WIDE), (65600, 1 << 15)])
def test_rows_fall_to_the_ctas_once(program, rows_max, pieces, R):  # noqa: F811
    assert run(program("append"), rows_max, pieces, AT_ONCE, R) == (0, "ok\n")


@pytest.mark.parametrize("rows_max,pieces", [(4096, ORDINARY), (MOST, NARROW), (MOST, WIDE)])
def test_every_row(program, rows_max, pieces):  # noqa: F811
    assert run(program("append"), rows_max, pieces, AT_ONCE, rows_max) == (0, "ok\n")


def test_a_product_that_wraps_is_noticed(program):  # noqa: F811
    # what the tests above must notice: min(rows of a CTA, R - r0) pieces, formed in CTAs past row R too
    assert run(program("append"), 385, ORDINARY, AT_ONCE, 1, "wrapped") == (0, "ok\n")
    for rows_max, pieces in ((385, WIDEST), (MOST, WIDE), (65600, 1 << 15)):
        code, out = run(program("append"), rows_max, pieces, AT_ONCE, 1, "wrapped")
        assert code == 1, (rows_max, pieces, out)
