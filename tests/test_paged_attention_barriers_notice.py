"""What the model of the paged tile kernel's barriers (test_paged_attention_barriers.py) must notice: the model with one wait or
arrival left out goes wrong under some schedule."""
import pytest

from tests.test_cached_attention_barriers import Bar, Broken, held
from tests.test_paged_attention_barriers import LINES, ROLES, Cta


class Statistics(Bar):
    """The split form's join: whoever arrives has just overwritten statistics of the item before, which both streams must
    have read (o_free) by then."""

    def __init__(self, o_free):
        super().__init__(2)
        self.o_free = o_free

    def arrive(self):
        if self.o_free.done < self.done:
            raise Broken(f"statistics of item {self.done - 1} are overwritten before they are read")
        super().arrive()


class Watched(Cta):
    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        if not self.pair:
            self.join = Statistics(self.o_free)
            for st in range(2):
                self.roles[f"softmax {st}"] = self.softmax(st)


class NoWaitForReaders(Watched):
    """The softmax warps do not wait for o_free before they join."""

    def softmax(self, st):
        for w in super().softmax(st):
            if w is None or w[0] is not self.o_free:
                yield w


class Turn(Bar):
    lost = False

    def arrive(self):
        if self.lost:
            self.lost = False
        else:
            super().arrive()


class NoExtraTurns(Cta):
    """Stream 1 takes no more turns than it has products: not as many as stream 0 where that has a block more."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.turn = [Turn(1), Turn(1)]
        for st in range(2):
            self.roles[f"issuer {st}"] = self.issuer(st)

    def issuer(self, st):
        items = turns = 0
        for w in super().issuer(st):
            if w is not None and any(w[0] is b for b in self.item_full):
                items, turns = items + 1, 0
            if w is not None and st == 1 and not self.pair and w[0] is self.turn[1]:
                blocks = self.items[items - 1][0]
                turns += 1
                if turns > (blocks // 2 + 1 if blocks > 1 else 0):
                    self.turn[0].lost = True
                    continue
            yield w


def schedules(make, line, pair, ring, cut=0.5):
    for seed in range(8):
        for role in [None, *ROLES]:
            make([(n, True, cut) for n in line], pair, ring, seed).run(held(role, seed))


@pytest.mark.parametrize("line", LINES, ids=str)
def test_statistics_are_read_before_they_are_overwritten(line):
    schedules(Watched, line, False, 3)


# (a stream with a block of the item has waited already: its first product needs O, and so the readers)
@pytest.mark.parametrize("line", [[1, 1], [4, 1], [1] * 7, [2, 1, 3]], ids=str)
def test_a_join_that_does_not_wait_for_the_readers(line):
    with pytest.raises(Broken, match="overwritten before"):
        schedules(NoWaitForReaders, line, False, 3)


@pytest.mark.parametrize("line", [[1, 1], [3, 1], [5, 2], [1, 7, 1, 2]], ids=str)
def test_streams_with_unequal_turns(line):
    with pytest.raises(Broken):
        schedules(NoExtraTurns, line, False, 3)


def test_streams_of_equal_turns_need_no_more():
    schedules(NoExtraTurns, [4, 2, 4], False, 3)


@pytest.mark.parametrize("line", [[6, 4], [4, 4, 4]], ids=str)
def test_a_pair_whose_places_are_freed_without_the_fixer(line):
    with pytest.raises(Broken):
        schedules(lambda *a: Cta(*a, fixer_releases=False), line, True, 5)
