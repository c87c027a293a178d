"""A model of the rings of slots that the tensor-memory page attention hands its
K and V tiles through, with random delays: two producers (K and V), one issuing
thread, one softmax thread a stream that releases slots.

A barrier's wait only tells a phase from its neighbours, so a wait is early if
it returns for a phase that is not the one meant: then a slot is overwritten
while it is read, or armed twice. K of tile t is use 2t of a ring, V use 2t + 1
(t counted a stream where each stream has a ring). When a stream's scores of a
tile are complete, the V slot of its tile before is released and then the K
slot. The other order lets the V producer pass early where K and V alternate in
a slot (an odd number of slots)."""
import random

import pytest


def early_waits(seed, slots, shared, by_parity, v_first, tiles):
    rng = random.Random(seed)
    rings = 1 if shared else 2
    full = [[0] * slots for _ in range(rings)]  # completed phases
    empty = [[0] * slots for _ in range(rings)]
    arrived = [[0] * slots for _ in range(rings)]
    landing, scores, weights, bad = [], [0, 0], [0, 0], []
    place = lambda kv, t: (0 if shared else t & 1, 2 * (t if shared else t // 2) + kv)
    tile_of = lambda s, u: 2 * u + s if by_parity else u
    over = lambda done, phase: (done & 1) != (phase & 1)  # what a parity wait sees

    def until(cond):
        while not cond():
            yield

    def pause():
        for _ in range(int(rng.expovariate(1 / rng.choice((1, 3, 30))))):
            yield

    def producer(kv):
        for t in range(tiles):
            r, use = place(kv, t)
            slot, phase = use % slots, use // slots
            if phase:
                yield from until(lambda: over(empty[r][slot], phase - 1))
                if empty[r][slot] != phase:
                    bad.append(("producer", kv, t))
            yield from pause()
            landing.append((r, slot, phase))
            yield

    def landed():
        if landing and rng.random() < 0.3:
            r, slot, phase = landing.pop(rng.randrange(len(landing)))
            if full[r][slot] != phase:
                bad.append(("armed twice", r, slot))
            full[r][slot] += 1

    def take(kv, t):
        r, use = place(kv, t)
        yield from until(lambda: over(full[r][use % slots], use // slots))
        if full[r][use % slots] != use // slots + 1:
            bad.append(("issuer", kv, t))

    def issuer():
        u = -1
        while tile_of(0, u) < tiles:
            for s in range(2):
                t, ahead, own = tile_of(s, u), tile_of(s, u + 1), by_parity or s == 0
                if u >= 0 and t < tiles:
                    if own:
                        yield from take(1, t)
                    yield from until(lambda: weights[s] > u)
                if ahead < tiles:
                    if own:
                        yield from take(0, ahead)
                    yield from pause()
                    scores[s] += 1
            u += 1

    def arrive(kv, t):
        r, use = place(kv, t)
        arrived[r][use % slots] += 1
        if arrived[r][use % slots] == (2 if shared else 1):
            arrived[r][use % slots] = 0
            empty[r][use % slots] += 1

    def softmax(s):
        u = 0
        while tile_of(s, u) < tiles:
            yield from until(lambda: scores[s] > u)
            t = tile_of(s, u)
            release = [(1, t - (2 if by_parity else 1)), (0, t)]
            for _ in range(2 if shared and by_parity else 1):
                for kv, x in release if v_first else release[::-1]:
                    if x >= 0:
                        arrive(kv, x)
                        yield from pause()
            yield from pause()
            weights[s] = u = u + 1

    threads = [producer(0), producer(1), issuer(), softmax(0), softmax(1)]
    for _ in range(400000):
        if bad or not threads:
            break
        i = rng.randrange(len(threads))
        try:
            for _ in range(rng.choice((1, 1, 1, 50))):
                next(threads[i])
        except StopIteration:
            threads.pop(i)
        landed()
    assert bad or not threads  # every wait ends
    return bad


@pytest.mark.parametrize("slots,shared,by_parity", [(3, False, True), (4, False, True), (2, False, True), (5, True, False),
                                                    (8, True, False), (4, True, False)])
def test_no_wait_is_early(slots, shared, by_parity):
    for seed in range(40):
        assert not early_waits(seed, slots, shared, by_parity, True, 12 + seed % 7)


def test_the_other_order_is_caught():
    assert any(early_waits(seed, 3, False, True, False, 12 + seed % 7) for seed in range(40))
