"""Which form a paged attention takes, asked of the kernels' own header on the CPU: clusters, an item each, only where a call
that one long item holds up costs little more than the line's join does."""
import pytest

from tests.test_device_code_on_cpu import program, run  # noqa: F401

ALL = -2, 0, 0  # no window
CAUSAL = -1, 0, 0


def choice(program, B, L, Hq, Hkv, rows, window=ALL, places="none", lengths=True):  # noqa: F811
    code, out = run(program("choice"), B, L, Hq, Hkv, rows, *window, places, int(lengths))
    assert code == 0, out
    kind, cluster = out.split()
    return kind, int(cluster)


@pytest.mark.parametrize("window", [CAUSAL, (-1, -1, 0), (4, -1, 0), (-1, 1000, 4), (32768, 0, 0), (1 << 20, 1 << 20, 0), (16384, 0, 4)])
@pytest.mark.parametrize("places", ["idx", "start"])
@pytest.mark.parametrize("B,L,rows", [(16, 32768, 1), (32, 8192, 1), (16, 16384, 4), (16, 8192, 18), (16, 8192, 32), (4, 32768, 32)])
def test_windows_without_a_bound_are_ragged(program, B, L, rows, window, places):  # noqa: F811
    """One long sequence of many must not hold up the call: 97 us for 27 with 16 tokens of 28/4 heads, one behind 32768 keys."""
    assert choice(program, B, L, 28, 4, rows, ALL)[1] == 0
    assert choice(program, B, L, 28, 4, rows, window, places)[1] == 0


@pytest.mark.parametrize("B,L,rows", [(16, 32768, 2), (16, 16384, 4), (4, 32768, 32), (16, 4096, 32), (4, 8192, 95), (4, 32768, 95), (1, 32768, 32)])
@pytest.mark.parametrize("lengths", [False, True])
def test_rows_that_may_lie_apart(program, B, L, rows, lengths):  # noqa: F811
    """Positions only the device knows, a narrow window: the rows of one sequence may reach over all of it."""
    for window in ((128, 128, 4), (512, 512, 4), (0, 0, 0)):
        assert choice(program, B, L, 28, 4, rows, window, "idx", lengths)[1] == 0
        assert choice(program, B, L, 28, 4, rows, window, "start", lengths)[1] > 0  # beside each other


@pytest.mark.parametrize("B,L,Hq,Hkv,rows,window,places,lengths,want", [
    (1, 2047, 28, 4, 1, ALL, "none", False, ("rows", 8)),                  # a single token
    (64, 8192, 28, 4, 1, ALL, "none", True, ("rows", 0)),                  # a batch of them
    (1, 1024, 32, 32, 95, ALL, "none", True, ("tiles", 4)),                # a partial step
    (1, 32768, 32, 32, 95, ALL, "none", True, ("tiles", 4)),
    (8, 2048, 28, 4, 95, ALL, "none", True, ("tiles", 0)),
    (4, 2048, 28, 4, 2048, ALL, "none", True, ("tiles", 0)),               # full steps
    (16, 32767, 28, 4, 1, (1023, 0, 4), "idx", True, ("rows", 2)),         # the last 1024 keys of a long sequence
    (16, 32768, 28, 4, 1, (8191, 0, 4), "idx", True, ("rows", 2)),         # or a quarter of it
    (8, 4096, 32, 32, 95, (256, 256, 64), "idx", True, ("tiles", 0)),
    (4, 32768, 28, 4, 2, (512, 512, 4), "idx", True, ("rows", 6)),          # apart or not, clusters are the faster
    (16, 16384, 28, 4, 2, (512, 512, 4), "idx", True, ("rows", 2)),
    (4, 8192, 28, 4, 4, (512, 512, 4), "idx", True, ("tiles", 6)),
    (4, 32768, 28, 4, 4, (512, 512, 4), "idx", True, ("tiles", 6)),
    (1, 32768, 28, 4, 95, (512, 512, 4), "idx", True, ("tiles", 8)),
    (2, 8192, 28, 4, 95, (512, 512, 4), "idx", True, ("tiles", 5)),
    (4, 8192, 28, 4, 1, CAUSAL, "idx", True, ("rows", 6)),                 # short enough that one long sequence costs no more than a join
    (2, 2048, 28, 4, 95, CAUSAL, "start", True, ("tiles", 5)),
    (1, 4096, 28, 4, 1, CAUSAL, "idx", True, ("rows", 8)),                 # one sequence
])
def test_choices(program, B, L, Hq, Hkv, rows, window, places, lengths, want):  # noqa: F811
    assert choice(program, B, L, Hq, Hkv, rows, window, places, lengths) == want
