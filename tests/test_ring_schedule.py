"""The waits of the prompt and chunk attention kernel, replayed on the CPU.

Its roles (scheduler, K/V loader, S and P V issuers, two softmax groups) run here as
generators over barriers with the kernel's counts and phase parities, with latencies
drawn at random.  An mbarrier shows a waiter only the parity of its phase; the replay
knows the phase, so a wait that passes on any other than the one it is for is seen, as
is one that comes too late and one that never ends.

The orders are those of csrc/grouped_prompt.cu: K_0, K_1, V_0, K_2, V_1, ... then the
output's stage in one ring of slots (5, or 8 at head dim 64), what landed told by
barriers per kind.  With one barrier per slot, and K awaited ahead of the S region, a
wait can pass on the phase of two rounds before; that variant is replayed too, to show
that the replay tells them apart.
"""
import heapq
import random

import pytest


class Barrier:
    def __init__(self, count, name):
        self.count = self.left = count
        self.phase, self.name = 0, name  # phases completed

    def arrive(self):
        self.left -= 1
        assert self.left >= 0, f"{self.name}: more arrivals than its count"
        if self.left == 0:
            self.phase += 1
            self.left = self.count

    def passes(self, index):
        """What try_wait.parity answers a waiter for phase `index`."""
        return (self.phase & 1) != (index & 1)

    def check(self, who, index):
        assert self.phase == index + 1, \
            f"{who}: wait for phase {index} of {self.name} passed at {self.phase}"


class Replay:
    def __init__(self, seed, items, ring, by_kind, k_first, n_posted=3):
        self.rng = random.Random(seed)
        self.items, self.ring, self.by_kind, self.k_first = items, ring, by_kind, k_first
        self.n_posted = n_posted
        self.now, self.events, self.order, self.tensor_free = 0, [], 0, 0

        def bars(n, count, name):
            return [Barrier(count, f"{name}[{i}]") for i in range(n)]
        self.full = bars(ring, 1, "full")  # one per slot
        self.kind = {k: bars(ring, 1, k + "_full") for k in ("k", "v", "st")}
        self.empty = bars(ring, 1, "kv_empty")
        self.q_full, self.q_free = bars(2, 1, "q_full"), bars(2, 1, "q_free")
        self.s_full, self.s_free = bars(2, 1, "s_full"), bars(2, 1, "s_free")
        self.p_full, self.pv_done = bars(2, 1, "p_full"), bars(2, 1, "pv_done")
        self.it_full = bars(n_posted, 1, "it_full")
        self.it_empty = bars(n_posted, 5, "it_empty")
        self.stage_left = [0] * ring

    # ---- time
    def after(self, dt, fn):
        self.order += 1
        heapq.heappush(self.events, (self.now + dt, self.order, fn))

    def products(self, dt, *then):
        """Queued on the tensor core; then: arrivals when they are done (commit)."""
        self.tensor_free = max(self.now, self.tensor_free) + dt
        for fn in then:
            self.after(self.tensor_free - self.now + 20, fn)

    def memory(self):
        return self.rng.choice([5, 20, 100, 400, 2000])

    # ---- what landed in slot u, the i-th of its kind: (barrier, phase)
    def landed(self, kind, u, i):
        if self.by_kind:
            return self.kind[kind][i % self.ring], i // self.ring
        return self.full[u % self.ring], u // self.ring

    def take(self, k):
        return self.it_full[k % self.n_posted], k // self.n_posted

    def taken(self, k):
        self.it_empty[k % self.n_posted].arrive()

    # ---- roles: yield a delay, or (barrier, phase) to wait for
    def scheduler(self):
        for k in range(len(self.items) + 1):  # the last one says that there are no more
            yield self.rng.choice([5, 500, 3000])
            yield self.it_empty[k % self.n_posted], k // self.n_posted - 1
            self.it_full[k % self.n_posted].arrive()
            due = 0 if k == 0 else k - 1
            if k != 1 and due < len(self.items):
                for x in range(2):
                    yield self.q_free[x], due - 1
                    self.after(self.memory(), self.q_full[x].arrive)

    def loader(self):
        u, count = 0, {"k": 0, "v": 0, "st": 0}
        for k, it in enumerate(self.items):
            yield self.take(k)
            self.taken(k)
            yield self.rng.choice([5, 800])
            n = it["n"]
            for i in range(2 * n):
                kind = "v" if i > 0 and (i % 2 == 0 or (i + 1) // 2 == n) else "k"
                yield self.empty[u % self.ring], u // self.ring - 1
                self.after(self.memory(), self.landed(kind, u, count[kind])[0].arrive)
                u += 1
                count[kind] += 1
            if it["whole"]:
                yield self.empty[u % self.ring], u // self.ring - 1
                self.landed("st", u, count["st"])[0].arrive()
                u += 1
                count["st"] += 1

    def s_issuer(self):
        u0 = k0 = 0
        done, last = [0, 0], None
        for k, it in enumerate(self.items):
            yield self.take(k)
            self.taken(k)
            q_there = [False, False]
            for t in range(it["n"]):
                u = u0 + (0 if t == 0 else 2 * t - 1)
                if self.k_first:
                    yield self.landed("k", u, k0 + t)
                for x in range(2):
                    if t >= it["tiles"][x]:
                        continue
                    if not q_there[x]:
                        yield self.q_full[x], k
                        q_there[x] = True
                    if last is not None:
                        yield last
                    if not self.k_first:
                        yield self.landed("k", u, k0 + t)
                    yield 100
                    free = [self.q_free[x].arrive] if t + 1 == it["tiles"][x] else []
                    self.products(256, self.s_full[x].arrive, *free)
                    last = self.s_free[x], done[x]
                    done[x] += 1
                self.products(0, self.empty[u % self.ring].arrive)
            for x in range(2):
                if it["tiles"][x] == 0:
                    yield self.q_full[x], k
                    self.q_free[x].arrive()
            u0 += 2 * it["n"] + it["whole"]
            k0 += it["n"]

    def pv_issuer(self):
        u0 = v0 = 0
        done = [0, 0]
        for k, it in enumerate(self.items):
            yield self.take(k)
            self.taken(k)
            n = it["n"]
            for t in range(n):
                u = u0 + (2 * t + 2 if t + 1 < n else 2 * t + 1)
                yield self.landed("v", u, v0 + t)
                for x in range(2):
                    if t >= it["tiles"][x]:
                        continue
                    yield self.p_full[x], done[x]
                    yield 100
                    self.products(256, self.pv_done[x].arrive)
                    done[x] += 1
                self.products(0, self.empty[u % self.ring].arrive)
            u0 += 2 * n + it["whole"]
            v0 += n

    def softmax(self, x):
        done = u0 = stages = 0
        for k, it in enumerate(self.items):
            yield self.take(k)
            self.taken(k)
            tiles = it["tiles"][x]
            for j in range(tiles):
                yield self.s_full[x], done
                yield self.rng.choice([100, 250, 400])
                self.s_free[x].arrive()
                yield self.rng.choice([300, 1000, 2000])
                if j > 0:
                    yield self.pv_done[x], done - 1
                self.p_full[x].arrive()
                done += 1
            if tiles > 0:
                yield self.pv_done[x], done - 1
            u, i = u0 + 2 * it["n"], stages
            u0, stages = u + it["whole"], stages + it["whole"]
            if not it["rows"][x]:
                continue
            if it["whole"]:
                yield self.landed("st", u, i)
            yield self.rng.choice([100, 1300, 4000])
            if it["whole"]:  # the last of those that use the stage lets it go
                slot = u % self.ring
                self.stage_left[slot] += 1
                if self.stage_left[slot] == 1 + it["rows"][1]:
                    self.stage_left[slot] = 0
                    self.empty[slot].arrive()

    def run(self):
        roles = {"scheduler": self.scheduler(), "loader": self.loader(), "S": self.s_issuer(),
                 "P V": self.pv_issuer(), "A": self.softmax(0), "B": self.softmax(1)}
        waiting, left = {}, set(roles)

        def step(who):
            for want in roles[who]:
                if isinstance(want, int):
                    self.after(want, lambda: step(who))
                    return
                bar, index = want
                if not bar.passes(index):
                    waiting[who] = want
                    return
                bar.check(who, index)
            left.discard(who)

        for who in roles:
            step(who)
        while left or self.events:
            for who in list(waiting):
                bar, index = waiting[who]
                if bar.passes(index):
                    bar.check(who, index)
                    del waiting[who]
                    step(who)
            if self.events:
                self.now, _, fn = heapq.heappop(self.events)
                fn()
            elif not any(bar.passes(index) for bar, index in waiting.values()):
                stuck = {who: bar.name for who, (bar, _) in waiting.items()}
                assert not left, f"waits that never end: {stuck}"


def items(seed):
    """Work items of a CTA: units of one or two tiles, parts, bad sequences (no keys)."""
    rng = random.Random(seed)
    bad, split = rng.choice([0, 0.2, 0.6]), rng.random() < 0.5
    out = []
    for _ in range(rng.choice([3, 8, 20])):
        two = rng.random() < 0.6
        if rng.random() < bad:
            out.append(dict(n=0, tiles=[0, 0], whole=1, rows=[True, two]))
            continue
        n = rng.choice([1, 1, 2, 2, 3, 4, 7])
        first = max(0, n - rng.choice([0, 0, 1])) if two else n
        out.append(dict(n=n, tiles=[first, n if two else 0],
                        whole=0 if split and rng.random() < 0.5 else 1, rows=[True, two]))
    return out


@pytest.mark.parametrize("ring", [5, 8])
@pytest.mark.parametrize("k_first", [True, False])  # paged keys, contiguous rows
def test_every_wait_is_for_its_own_phase(ring, k_first):
    for seed in range(600):
        Replay(seed, items(seed), ring, by_kind=True, k_first=k_first).run()


def test_one_barrier_for_a_slot_would_let_a_wait_pass_early():
    caught = 0
    for seed in range(600):
        try:
            Replay(seed, items(seed), 5, by_kind=False, k_first=True).run()
        except AssertionError as e:
            assert "wait for phase" in str(e)
            caught += 1
    assert caught > 0
