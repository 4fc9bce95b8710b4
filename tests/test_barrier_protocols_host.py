"""Models of the barriers between the roles of the persistent kernels (window_prompt.cu, the long calls of
attn_mass.cu), run on the host. A wait names a phase by its parity, so a role that falls two phases behind takes one
phase for another. Every role is run in random orders and as the one that is scheduled last; what a shared buffer holds
is followed beside its barriers."""
import os
import random

import pytest


class Bar:
    """An mbarrier: arrivals of `count` end a phase."""

    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self, n=1):
        self.left -= n
        assert self.left >= 0
        if self.left == 0:
            self.phase += 1
            self.left = self.count

    def done(self, parity):
        return (self.phase & 1) != (parity & 1)


class Deadlock(Exception):
    pass


class Machine:
    """Roles are generators that yield what they wait for. Copies and products end some time after their issue,
    products of one tile in order."""

    def __init__(self, seed, last=None):
        self.rnd, self.last, self.live, self.wait, self.rank = random.Random(seed), last, {}, {}, {}
        self.issued, self.ended, self.new = {}, {}, []

    def add(self, name, role):
        self.live[name], self.rank[name] = role, self.rnd.random()
        self.step(name)

    def step(self, name):
        try:
            self.wait[name] = next(self.live[name])
        except StopIteration:
            del self.live[name]
        while self.new:
            self.add(*self.new.pop())

    def later(self, act, queue=None):
        n = self.issued[queue] = self.issued.get(queue, 0) + 1

        def role():
            yield lambda: queue is None or self.ended.get(queue, 0) == n - 1
            act()
            self.ended[queue] = n

        self.new.append((("later", queue, n), role()))

    def run(self):
        while self.live:
            ready = [n for n in self.live if self.wait[n]()]
            if not ready:
                raise Deadlock(sorted(map(str, self.live)))
            if self.last in ready and len(ready) > 1:
                ready.remove(self.last)
            self.step(self.rnd.choice(ready) if self.rnd.random() < .5 else min(ready, key=self.rank.get))


def at(bar, parity):
    return lambda: bar.done(parity)


def go():
    return True


def prompt(items, stages, seed, last=None, own_tails=True):
    """window_prompt_kernel: items are (tiles of query rows, steps). own_tails: each tile has a barrier for V's last tile."""
    m = Machine(seed, last)
    full, empty = [Bar(1) for _ in range(stages)], [Bar(2) for _ in range(stages)]
    item_full, item_read = [Bar(1), Bar(1)], [Bar(11), Bar(11)]
    q_full, s_full, o_done, turn = ([Bar(1), Bar(1)] for _ in range(4))
    p_ready = [[Bar(4), Bar(4)], [Bar(4), Bar(4)]]
    q_free, loads_done, near_end, tail_ready = Bar(8), Bar(1), Bar(1), Bar(1)
    tail_done = [Bar(1), Bar(1)]
    slot, entry, q, scores, bad = [None, None], [None] * stages, [None, None], [None, None], [None, None]
    zeroed, stored = [-1], [0, 0]

    def read(i):
        assert slot[i & 1][0] == i
        return slot[i & 1][1]

    def item_warp():
        loaded = 0
        for i in range(len(items) + 1):
            if i:
                steps = items[i - 1][1]
                if steps:
                    yield at(near_end, loaded)
            if i >= 2:
                yield at(item_read[i & 1], (i >> 1) - 1)
            slot[i & 1] = (i, items[i] if i < len(items) else None)
            item_full[i & 1].arrive()
            if i and steps:
                yield at(tail_ready, loaded)
                loaded += 1
                zeroed[0] = i - 1
                tail_done[0].arrive()
                if own_tails and items[i - 1][0] == 2:
                    tail_done[1].arrive()

    def copy_warp():
        use = loaded = 0
        for i in range(len(items) + 1):
            yield at(item_full[i & 1], i >> 1)
            it = read(i)
            item_read[i & 1].arrive()
            if it is None:
                return
            tiles, steps = it
            if not steps:
                continue
            if loaded:
                yield at(q_free, loaded - 1)
            bad[loaded & 1] = i
            for t in range(tiles):
                def landed(t=t, i=i):
                    q[t] = i
                    q_full[t].arrive()
                q[t] = None
                m.later(landed)
            for j in range(steps):
                if j == max(0, steps - 2):
                    near_end.arrive()
                for _ in range(2):
                    s = use % stages
                    if use >= stages:
                        yield at(empty[s], use // stages - 1)

                    def landed(s=s, use=use):
                        entry[s] = use
                        full[s].arrive()
                    entry[s] = None
                    m.later(landed)
                    use += 1
                yield go
            loads_done.arrive()
            loaded += 1

    def matrix(t):
        base = loaded = mine = step = phase = 0

        def arrived(use):
            return at(full[use % stages], use // stages)

        def holds(use):
            assert entry[use % stages] == use

        for i in range(len(items) + 1):
            yield at(item_full[i & 1], i >> 1)
            it = read(i)
            item_read[i & 1].arrive()
            if it is None:
                return
            tiles, steps = it
            if not steps:
                continue
            first, item = base, loaded
            base += 2 * steps
            loaded += 1
            if t >= tiles:
                continue

            def my_turn():
                nonlocal phase
                if tiles == 2:
                    k = phase
                    phase += 1
                    if t or k:
                        yield at(turn[t], k - (t == 0))

            def hand_over():
                if tiles == 2:
                    turn[t ^ 1].arrive()

            yield at(q_full[t], mine)
            own, mine = mine, mine + 1
            yield arrived(first)
            yield from my_turn()
            assert q[t] == i
            holds(first)

            def formed(i=i):
                assert q[t] == i and scores[t] is None
                scores[t] = ("S", i, 0)
                s_full[t].arrive()
            m.later(formed, t)
            hand_over()
            yield arrived(first + 1)
            for j in range(steps):
                more, use = j + 1 < steps, first + 2 * j + 1
                if more:
                    yield arrived(use + 1)
                else:
                    if t == 0:
                        tail_ready.arrive()
                    yield at(tail_done[t], own) if own_tails else at(tail_done[0], item)
                    assert zeroed[0] >= i
                yield at(p_ready[t][0], step)
                yield from my_turn()
                yield at(p_ready[t][1], step)
                holds(use)
                assert scores[t] == ("P", i, j)
                if more:
                    holds(use + 1)

                    def formed(i=i, j=j, use=use):
                        holds(use)
                        holds(use + 1)
                        scores[t] = ("S", i, j + 1)
                        s_full[t].arrive()
                    m.later(formed, t)
                    hand_over()
                    yield arrived(use + 2)
                else:
                    def formed(use=use):
                        holds(use)
                        scores[t] = None
                        o_done[t].arrive()
                    m.later(formed, t)
                    hand_over()
                step += 1

    def softmax(w):
        t, lead = w >> 2, w % 4 == 0
        base = loaded = step = outs = 0
        for i in range(len(items) + 1):
            yield at(item_full[i & 1], i >> 1)
            it = read(i)
            item_read[i & 1].arrive()
            if it is None:
                return
            tiles, steps = it
            first, item = base, loaded
            base += 2 * steps
            loaded += steps > 0
            if t >= tiles:
                continue

            def release(use):
                if lead:
                    empty[use % stages].arrive(3 - tiles)

            for j in range(steps):
                yield at(s_full[t], step)
                assert scores[t][1:] == (i, j)
                release(first + 2 * j)
                if j:
                    release(first + 2 * j - 1)
                if j + 1 == steps:
                    yield at(loads_done, item)
                    assert bad[item & 1] == i
                    q_free.arrive(3 - tiles)
                for c in range(2):
                    yield go
                    if c:
                        stored[t] += 1
                        if stored[t] == 4:
                            stored[t], scores[t] = 0, ("P", i, j)
                    p_ready[t][c].arrive()
                step += 1
            if steps:
                yield at(o_done[t], outs)
                outs += 1
                release(first + 2 * steps - 1)

    m.add("items", item_warp())
    m.add("copies", copy_warp())
    for t in range(2):
        m.add(f"matrix{t}", matrix(t))
    for w in range(8):
        m.add(f"softmax{w}", softmax(w))
    m.run()


PROMPT_ROLES = ["items", "copies", "matrix0", "matrix1"] + [f"softmax{w}" for w in (0, 3, 4, 7)]


def weights(blocks, stages, seed, last=None, buffers=3):
    """mass_long_kernel: blocks are the steps of each item; two tiles of positions."""
    m = Machine(seed, last)
    full, empty = [Bar(1) for _ in range(stages)], [Bar(16) for _ in range(stages)]
    s_full, s_empty = ([[Bar(n) for _ in range(4)] for _ in range(2)] for n in (1, 8))
    item_full, item_read = [Bar(1), Bar(1)], [Bar(18), Bar(18)]
    k_full, part_full = [Bar(8), Bar(8)], [Bar(4), Bar(4)]
    slot, entry, held = [None, None], [None] * stages, [None] * buffers

    def copy_warp():
        use = 0
        for i in range(len(blocks) + 1):
            if i >= 2:
                yield at(item_read[i & 1], (i >> 1) - 1)
            slot[i & 1] = (i, blocks[i] if i < len(blocks) else None)
            item_full[i & 1].arrive()
            if i == len(blocks) or not blocks[i]:
                continue
            for e in range(2 + blocks[i]):
                s = use % stages
                if use >= stages:
                    yield at(empty[s], use // stages - 1)

                def landed(s=s, use=use, e=e):
                    entry[s] = ("K" if e < 2 else "Q", use)
                    full[s].arrive()
                entry[s] = None
                m.later(landed)
                use += 1
                yield go

    def read(i):
        assert slot[i & 1][0] == i
        return slot[i & 1][1]

    def matrix(t):
        use, product, mine = 0, t, 0
        for i in range(len(blocks) + 1):
            yield at(item_full[i & 1], i >> 1)
            steps = read(i)
            item_read[i & 1].arrive()
            if steps is None:
                return
            if not steps:
                continue
            use += 2
            yield at(k_full[t], mine)
            mine += 1
            for _ in range(steps):
                s, buf, own, before = use % stages, product % buffers, product >> 1, product - buffers
                yield at(full[s], use // stages)
                if before >= 0:
                    yield at(s_empty[t ^ 1][before >> 1 & 3], before >> 3)
                assert entry[s] == ("Q", use) and held[buf] is None
                held[buf] = [product, 0]

                def formed(own=own):
                    s_full[t][own & 3].arrive()
                m.later(formed, t)
                use += 1
                product += 2

    def sums(w):
        t, half = (w >> 2) & 1, w >> 3
        use, product, mine = 0, t, 0
        for i in range(len(blocks) + 1):
            yield at(item_full[i & 1], i >> 1)
            steps = read(i)
            if steps is None:
                return
            if steps:
                for e in range(2):
                    s = use % stages
                    yield at(full[s], use // stages)
                    assert entry[s] == ("K", use)
                    if e == t:
                        k_full[t].arrive()
                    empty[s].arrive()
                    use += 1
                for _ in range(steps):
                    s, buf, own = use % stages, product % buffers, product >> 1
                    yield at(full[s], use // stages)
                    assert entry[s] == ("Q", use)
                    yield at(s_full[t][own & 3], own >> 2)
                    yield go
                    assert held[buf][0] == product
                    held[buf][1] += 1
                    if held[buf][1] == 8:
                        held[buf] = None
                    s_empty[t][own & 3].arrive()
                    yield go
                    empty[s].arrive()
                    use += 1
                    product += 2
                if half:
                    part_full[t].arrive()
                else:
                    yield at(part_full[t], mine)
                mine += 1
            assert read(i) == steps
            item_read[i & 1].arrive()

    m.add("copies", copy_warp())
    for t in range(2):
        m.add(f"matrix{t}", matrix(t))
    for w in range(16):
        m.add(f"sums{w}", sums(w))
    m.run()


WEIGHT_ROLES = ["copies", "matrix0", "matrix1"] + [f"sums{w}" for w in (0, 5, 8, 13)]


@pytest.mark.parametrize("last", [None] + PROMPT_ROLES)
def test_prompts(last):
    for seed in range(40):
        r = random.Random(seed)
        items = [(r.choice([1, 2, 2]), r.choice([0, 1, 1, 2, 3, 5, 9])) for _ in range(r.randint(1, 9))]
        prompt(items, r.choice([5, 8]), seed, last)


@pytest.mark.parametrize("stages", [5, 8])
def test_short_items_of_one_tile_behind_two(stages):
    """The second tile's thread may come to its tail when a whole item of one tile has gone by without it."""
    items = [(2, 1), (1, 1), (2, 2), (1, 2), (1, 1), (2, 1)]
    for last in PROMPT_ROLES:
        for seed in range(5):
            prompt(items, stages, seed, last)


def test_a_tail_that_both_tiles_share_is_found():
    """With one barrier for both tiles that thread waits for a phase that is over: the models see it."""
    with pytest.raises(Deadlock):
        for seed in range(20):
            prompt([(2, 1), (1, 1)], 5, seed, "matrix1", own_tails=False)


def test_the_kernel_has_a_tail_barrier_for_each_tile():
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(here, "sparse_kv_long_sfi_gb300", "csrc", "window_prompt.cu")) as f:
        source = f.read()
    assert "wait_one(&tail_done[t], own & 1)" in source and "if (lane < w.tiles) mbar_arrive(&tail_done[lane])" in source


@pytest.mark.parametrize("last", [None] + WEIGHT_ROLES)
def test_weights(last):
    for seed in range(20):
        r = random.Random(seed)
        weights([r.choice([0, 1, 2, 5, 9]) for _ in range(r.randint(1, 8))], 6, seed, last)
