"""The barriers of the cached attention (csrc/attention_cached.cu), role by role, under schedules that
hold one role up for as long as the others can go on without it.

A waiter on an mbarrier sees the parity of its phase only. So a wait for phase n must end while n is
the barrier's last complete phase: earlier, it would pass too soon on the phase before; later (two
phases on), it would be told to wait again, and run out. The model is the kernel's item loop: the
producers, issuers, softmax warps (one for four) and dequantising warps of a CTA, copies and
products completing at any later time."""
import random

import pytest

ITEMS = 4  # items handed out and not yet finished


class Broken(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def passes(self, n, who):
        """Whether a wait for phase n returns now; raises where parity tells the waiter something untrue."""
        if n < 0 or self.done == n + 1:
            return True
        if self.done > n + 1 or (self.done & 1) != (n & 1):
            raise Broken(f"{who} waits for phase {n}, the barrier has completed {self.done}")
        return False


class Cta:
    """blocks: key blocks of each item; ragged: whether its last block is cut by a length (bf16)."""

    def __init__(self, blocks, ragged, q8, always_waits=False):
        self.blocks, self.ragged, self.q8, self.always_waits = list(blocks) + [0], list(ragged) + [False], q8, always_waits
        two = lambda n: [[Bar(n) for _ in range(2)] for _ in range(2)]  # noqa: E731
        self.item_full, self.item_empty = [Bar(1) for _ in range(ITEMS)], [Bar(8 if q8 else 4) for _ in range(ITEMS)]
        self.q_full, self.q_empty, self.join, self.o_free = Bar(2), Bar(2), Bar(2), Bar(2)
        self.s_full, self.p_full, self.pv_done = two(1), two(1), two(1)
        self.v_here = [Bar(1) for _ in range(2)]
        self.unit = [[Bar(1) for _ in range(4)] for _ in range(2)]  # K's two halves, V's two
        self.raw_full, self.raw_empty = [[Bar(1) for _ in range(4)] for _ in range(2)], [[Bar(1) for _ in range(4)] for _ in range(2)]
        self.copies, self.products = [], [[], []]  # arrivals to come: in any order; in order
        self.roles = {}
        for st in range(2):
            self.roles[f"producer {st}"] = self.producer(st)
            self.roles[f"issuer {st}"] = self.issuer(st)
            self.roles[f"softmax {st}"] = self.softmax(st)
            if q8:
                for kv in range(2):
                    self.roles[f"dequantiser {'KV'[kv]}{st}"] = self.dequantiser(st, kv)

    # Roles yield (barrier, phase) to wait and None to let others run.
    def next_item(self, n):
        yield self.item_full[n % ITEMS], n // ITEMS

    def producer(self, st):
        c = 0
        for n, nblk in enumerate(self.blocks):
            if st == 0:
                yield self.item_empty[n % ITEMS], n // ITEMS - 1
                self.item_full[n % ITEMS].arrive()
                yield None
            for _ in range(st, nblk, 2):
                for u in range(4):
                    if self.q8:
                        yield self.raw_empty[st][u], c - 1
                        self.copies.append(self.raw_full[st][u])
                    else:
                        if c:
                            yield (self.pv_done if u >> 1 else self.s_full)[st][u & 1], c - 1
                        self.copies.append(self.unit[st][u])
                    yield None
                c += 1

    def dequantiser(self, st, kv):
        c = 0
        for n, nblk in enumerate(self.blocks):
            yield from self.next_item(n)
            if nblk == 0:
                return
            for _ in range(st, nblk, 2):
                for h in range(2):
                    yield self.raw_full[st][2 * kv + h], c
                    if c:
                        yield (self.pv_done if kv else self.s_full)[st][h], c - 1
                    self.raw_empty[st][2 * kv + h].arrive()
                    self.unit[st][2 * kv + h].arrive()
                    yield None
                c += 1
            self.item_empty[n % ITEMS].arrive()

    def issuer(self, st):
        used = 0

        def scores(i, c, h, last):
            yield self.unit[st][h], c
            if c:
                yield self.pv_done[st][h], c - 1
            self.products[st].append(self.s_full[st][h])
            if h == 1 and i >= last:
                self.products[st].append(self.q_empty)
            yield None

        for n, nblk in enumerate(self.blocks):
            yield from self.next_item(n)
            if nblk == 0:
                return
            last = nblk - 2
            yield self.q_full, n
            if st < nblk:
                yield from scores(st, used, 0, last)
                yield from scores(st, used, 1, last)
            else:
                self.q_empty.arrive()
                yield None
            if n > 0 and (st < nblk or self.always_waits):
                yield self.o_free, n - 1
            for i in range(st, nblk, 2):
                for h in range(2):
                    yield self.unit[st][2 + h], used
                    if self.ragged[n] and i == nblk - 1:
                        self.v_here[st].arrive()
                        yield None
                    yield self.p_full[st][h], used
                    self.products[st].append(self.pv_done[st][h])
                    yield None
                    if i < last:
                        yield from scores(i + 2, used + 1, h, last)
                used += 1
            self.item_empty[n % ITEMS].arrive()

    def softmax(self, st):
        used = n_ragged = 0
        yield from self.next_item(0)
        if self.blocks[0]:
            self.q_full.arrive()
        for n, nblk in enumerate(self.blocks[:-1]):
            for i in range(st, nblk, 2):
                for h in range(2):
                    yield self.s_full[st][h], used
                    if self.ragged[n] and i == nblk - 1:
                        yield self.v_here[st], n_ragged
                        n_ragged += 1
                    if not (i < 2 and h == 0):  # a rescale, if there is one
                        yield self.pv_done[st][h ^ 1], used if h else used - 1
                    self.p_full[st][h].arrive()
                    yield None
                used += 1
            yield from self.next_item(n + 1)
            if self.blocks[n + 1]:
                yield self.q_empty, n
            if st < nblk:
                yield self.pv_done[st][1], used - 1
            if n > 0:
                yield self.o_free, n - 1
            self.join.arrive()
            yield None
            yield self.join, n
            if self.blocks[n + 1]:
                self.q_full.arrive()
            yield None
            self.o_free.arrive()
            self.item_empty[n % ITEMS].arrive()

    def run(self, order):
        """order(names) puts what can run next first. Every waiter's barrier is looked at after each step,
        as it would be by a warp that polls without ever being early or late."""
        at = dict.fromkeys(self.roles)
        while at:
            ready = [r for r, w in at.items() if w is None or w[0].passes(w[1], r)]
            ready += ["copies"] * bool(self.copies) + [f"products {st}" for st in range(2) if self.products[st]]
            if not ready:
                raise Broken(f"nothing goes on: {sorted(at)}")
            r = order(ready)
            if r == "copies":
                self.copies.pop(random.randrange(len(self.copies))).arrive()
            elif r.startswith("products"):
                self.products[int(r[-1])].pop(0).arrive()
            else:
                try:
                    at[r] = next(self.roles[r])
                except StopIteration:
                    del at[r]


ROLES = [f"{r} {st}" for r in ("producer", "issuer", "softmax", "products") for st in range(2)] + \
        [f"dequantiser {k}{st}" for k in "KV" for st in range(2)] + ["copies"]
LINES = [[1], [1, 1], [1, 1, 1, 1, 1, 1], [3, 1], [2, 1, 1, 4, 1], [5, 1, 1, 1, 1, 1, 2, 3, 1], [2, 2, 2, 2, 2, 2], [1, 7, 1, 2]]


def held(role, seed):
    """Others first, `role` when nothing else can go on; or, with no role, any order."""
    rng = random.Random(seed)
    random.seed(seed)

    def order(ready):
        rest = [r for r in ready if r != role]
        return rng.choice(rest or ready)

    return order


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("line", LINES, ids=str)
def test_every_wait_ends_on_its_own_phase(line, q8):
    for seed in range(6):
        ragged = [random.Random(seed * 100 + i).random() < 0.5 and not q8 for i in range(len(line))]
        for role in [None, *ROLES]:
            Cta(line, ragged, q8).run(held(role, seed))


@pytest.mark.parametrize("q8", [False, True])
def test_a_wait_that_nothing_holds_back_is_noticed(q8):
    # an issuer without work in an item, that waits all the same until the item before has left O: the
    # item ends without it, and its wait is two phases late
    with pytest.raises(Broken, match="issuer 1 waits for phase 0, the barrier has completed 2"):
        Cta([1, 1], [False, False], q8, always_waits=True).run(held("issuer 1", 0))
