"""The linear scan's hand-over of states, modelled on the CPU: what must not be tried on a GPU.

Inside a CTA (forward and backward) the warps with tokens, the one that publishes, the one that looks back and the one
that scouts meet at named barriers, two of each kind by turns.  The model runs them as threads in random orders, with
barriers that count arrivals as the hardware does, and checks that nobody waits for ever, that no barrier mixes two turns,
and that every buffer holds the tile its reader expects.  Between CTAs a chunk's state comes from the records of the chunks
before it: whatever is published when it looks, the state is the one that a walk through all chunks in order gives, bit for
bit."""
import random

import numpy as np
import pytest

WARPS = 3  # with tokens
INFOS, WINDOW = 8, 4


class Barrier:
    def __init__(self, count):
        self.count, self.arrived, self.phase = count, [], 0

    def arrive(self, who, turn):
        assert (who, turn) not in self.arrived and all(t == turn for _, t in self.arrived), "two turns in one phase"
        self.arrived.append((who, turn))
        if len(self.arrived) == self.count:
            self.arrived, self.phase = [], self.phase + 1


class Cta:
    """One CTA's roles as generators: each yields None after a step, or a function that says whether it may go on."""

    def __init__(self, tiles, backward):
        self.tiles, self.backward = tiles, backward
        n = WARPS
        self.bars = {k: [Barrier(c), Barrier(c)] for k, c in (("ready", n + 1), ("total", 3), ("state", n + 2), ("sums", n + 1))}
        self.info = [None] * INFOS
        for k in range(3):
            self.info[k] = self.tile(k)
        self.action = [[None] * n for _ in range(2)]
        self.total, self.carry = [None] * 2, [None] * 2
        self.sums = [[None] * n for _ in range(2)]
        self.stage = [[None] * (3 if backward else 2) for _ in range(n)]
        self.seen = {k: 0 for k in range(tiles)}

    def tile(self, k):
        return k if k < self.tiles else -1

    def look(self, k):  # a tile's layout: there, and of this tile
        assert self.info[k % INFOS] in (k, -1), (k, self.info)
        return self.info[k % INFOS]

    def sync(self, kind, k, who):
        bar = self.bars[kind][k & 1]
        phase = bar.phase
        bar.arrive(who, k)
        return lambda: bar.phase > phase

    def arrive(self, kind, k, who):
        self.bars[kind][k & 1].arrive(who, k)

    def warp(self, w):
        stages = len(self.stage[w])

        def load(k):
            if self.look(k) >= 0:
                self.stage[w][k % stages] = k

        def front(k):
            if self.look(k) < 0:
                return
            assert self.stage[w][k % stages] == k
            self.action[k & 1][w] = ("of the warp", k)
            yield
            self.arrive("ready", k, w)
            yield

        def rear(k):
            yield self.sync("state", k, w)
            assert self.look(k) == k and self.carry[k & 1] == k and self.action[k & 1][w] == ("of those before", k)
            yield
            if self.backward:
                assert self.stage[w][k % stages] == k
                self.sums[k & 1][w] = k
                yield
                self.arrive("sums", k, w)
            self.seen[k] += 1
            yield

        load(0)
        load(1)
        yield from front(0)
        k = 0
        while self.look(k) >= 0:
            load(k + 2)
            yield
            yield from front(k + 1)
            yield from rear(k)
            k += 1

    def publisher(self):
        k = 0

        def add(k):
            yield self.sync("sums", k, "publisher")
            assert self.look(k) == k and self.sums[k & 1] == [k] * WARPS

        while self.look(k) >= 0:
            yield self.sync("ready", k, "publisher")
            assert self.action[k & 1] == [("of the warp", k)] * WARPS
            yield
            self.total[k & 1] = k
            self.action[k & 1] = [("of those before", k)] * WARPS
            yield
            self.arrive("total", k, "publisher")
            yield
            if self.backward and k > 0:
                yield from add(k - 1)
            k += 1
        if self.backward and k > 0:
            yield from add(k - 1)

    def receiver(self):
        k = 0
        while self.look(k) >= 0:
            yield  # looks back
            yield self.sync("total", k, "receiver")
            self.carry[k & 1] = k
            yield
            assert self.look(k) == k and self.total[k & 1] == k
            yield
            self.arrive("state", k, "receiver")
            k += 1

    def scout(self):
        k = 0
        while self.look(k) >= 0:
            self.info[(k + 3) % INFOS] = self.tile(k + 3)
            yield
            yield self.sync("total", k, "scout")
            self.arrive("state", k, "scout")
            yield
            assert self.look(k) == k
            k += 1


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 11])
def test_warps_meet_in_every_order(tiles, backward):
    for seed in range(300):
        rng = random.Random(seed)
        cta = Cta(tiles, backward)
        roles = {**{w: cta.warp(w) for w in range(WARPS)}, "publisher": cta.publisher(), "receiver": cta.receiver(), "scout": cta.scout()}
        waits = dict.fromkeys(roles)
        slow = rng.choice(list(roles))  # one that lags
        while roles:
            ready = [r for r in roles if waits[r] is None or waits[r]()]
            assert ready, "nobody can go on"
            pick = rng.choice([r for r in ready if r != slow] or ready) if rng.random() < 0.9 else rng.choice(ready)
            try:
                waits[pick] = next(roles[pick])
            except StopIteration:
                del roles[pick]
        assert all(n == WARPS for n in cta.seen.values())


def step(a, b, h, packed=True):
    return b if a < 0 else np.float32(np.float64(a) * np.float64(h) + np.float64(b))


def test_a_chunks_state_does_not_depend_on_what_is_published():
    rng = np.random.default_rng(0)
    for _ in range(200):
        n = int(rng.integers(2, 40))
        a, b = rng.random(n, dtype=np.float32), rng.standard_normal(n).astype(np.float32)
        a[rng.random(n) < 0.1] = -1  # a sequence starts in the chunk
        after, h = [], np.float32(0)
        for i in range(n):
            h = step(a[i], b[i], h)
            after.append(h)
        flags = [2] + [0] * (n - 1)
        got = [after[0]] + [None] * (n - 1)
        pending = list(range(1, n))
        while pending:
            i = int(rng.choice(pending))
            if flags[i] == 0:
                flags[i] = 1
                continue
            start = None
            for j in range(1, min(WINDOW, i) + 1):  # the nearest chunk whose state is known, all nearer ones with their action
                if flags[i - j] == 2:
                    start = j
                    break
                if flags[i - j] == 0:
                    break
            if start is None:
                continue
            h = got[i - start]
            for j in range(start - 1, 0, -1):
                h = step(a[i - j], b[i - j], h)
            got[i] = step(a[i], b[i], h)
            flags[i] = 2
            pending.remove(i)
        assert all(x.tobytes() == y.tobytes() for x, y in zip(got, after))
