"""The waits of cross attention at head dim 64, replayed on the CPU as those of prompts and
chunks are (test_ring_schedule): every tile has an S region of its own there, so that an S
product waits for the softmax of its own tile's last one, and not of the product before."""
import pytest

from test_ring_schedule import Replay, items


class OwnRegions(Replay):
    late = 0  # products that a wait is skipped for

    def s_issuer(self):
        u0 = k0 = 0
        done = [0, 0]
        for k, it in enumerate(self.items):
            yield self.take(k)
            self.taken(k)
            q_there = [False, False]
            for t in range(it["n"]):
                u = u0 + (0 if t == 0 else 2 * t - 1)
                for x in range(2):
                    if t >= it["tiles"][x]:
                        continue
                    if not q_there[x]:
                        yield self.q_full[x], k
                        q_there[x] = True
                    if done[x] > 0 and done[x] != self.late:
                        yield self.s_free[x], done[x] - 1
                    yield self.landed("k", u, k0 + t)
                    yield 100
                    # the region is free: its last product was loaded
                    assert self.s_free[x].phase == done[x], "S overwritten"
                    free = [self.q_free[x].arrive] if t + 1 == it["tiles"][x] else []
                    self.products(256, self.s_full[x].arrive, *free)
                    done[x] += 1
                self.products(0, self.empty[u % self.ring].arrive)
            for x in range(2):
                if it["tiles"][x] == 0:
                    yield self.q_full[x], k
                    self.q_free[x].arrive()
            u0 += 2 * it["n"] + it["whole"]
            k0 += it["n"]


def unmasked(seed):
    """Items whose two tiles read all of their keys."""
    out = items(seed)
    for it in out:
        it["tiles"] = [it["n"], it["n"] if it["rows"][1] else 0]
    return out


def test_every_wait_is_for_its_own_phase():
    for seed in range(600):
        OwnRegions(seed, unmasked(seed), 8, by_kind=True, k_first=False).run()


def test_a_missing_wait_is_seen():
    class Missing(OwnRegions):
        late = 2
    with pytest.raises(AssertionError):
        for seed in range(600):
            Missing(seed, unmasked(seed), 8, by_kind=True, k_first=False).run()
