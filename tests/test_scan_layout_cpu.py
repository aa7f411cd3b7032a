"""Numbering of a packed batch's tiles and how a wave finds a tile's sequence, as the
kernels of the recurrence and the convolution do it, in Python: every tile of every
sequence has a number of its own below the count that the host launches, and the number
leads back to it; any bounds at all stay inside the tensor."""

import random

import pytest


def span(cu, b, total):
    a = min(max(cu[b], 0), total)
    return a, min(max(cu[b + 1], a), total) - a


def tile_of(cu, j, tile, total):
    """64 lanes look at one sequence each; (sequence, its tile)."""
    batch, start, n = len(cu) - 1, 0, len(cu) - 1

    def begun(s):
        return min(max(cu[s], 0), total) // tile + s <= j

    while n > 64:
        step, end = (n + 63) // 64, start + n
        hits = sum(1 for lane in range(64) if lane * step < n and begun(start + lane * step))
        start += max(hits - 1, 0) * step
        n = min(step, end - start)
    hits = sum(1 for lane in range(64) if lane < n and begun(start + lane))
    b = start + max(hits, 1) - 1
    assert 0 <= b < batch
    i = j - (min(max(cu[b], 0), total) // tile + b)
    return b, (i if 0 <= i <= total // tile else total // tile + 1)


@pytest.mark.parametrize("batch,longest", [(1, 5000), (3, 700), (9, 260), (64, 300), (65, 40), (500, 200), (5000, 3)])
@pytest.mark.parametrize("tile", [64, 128, 256, 512])
@pytest.mark.parametrize("lead", [0, 300])
def test_numbers_lead_back_to_their_tiles(batch, longest, tile, lead):
    rng = random.Random(batch * tile + lead)
    cu = [lead]
    for _ in range(batch):
        cu.append(cu[-1] + rng.choice([0, 1, tile, rng.randint(0, longest)]))
    total = cu[-1] + lead
    count = total // tile + batch
    seen = {}
    for b in range(batch):
        t0, n = span(cu, b, total)
        for i in range(max(1, -(-n // tile))):
            j = t0 // tile + b + i
            assert j < count and j not in seen
            seen[j] = (b, i)
    for j in range(count):
        b, i = tile_of(cu, j, tile, total)
        if j in seen:
            assert (b, i) == seen[j]
        else:  # nobody's: behind the end of the sequence that it is found for
            assert i * tile >= max(span(cu, b, total)[1], 1)


@pytest.mark.parametrize("batch", [1, 7, 130])
def test_any_bounds_stay_inside(batch):
    rng = random.Random(batch)
    for _ in range(50):
        total = rng.choice([0, 1, 90, 3000])
        cu = [rng.choice([-5, 0, total, total + 1, 2 ** 31 - 1, -2 ** 31, rng.randint(0, total)]) for _ in range(batch + 1)]
        for j in range(total // 128 + batch):
            b, i = tile_of(cu, j, 128, total)
            t0, n = span(cu, b, total)
            assert 0 <= t0 <= total and 0 <= n <= total - t0 and i >= 0
            if i * 128 < n:
                assert t0 + i * 128 < total


def queues_of(width):
    groups = -(-width // 64)
    each = -(-groups // 16)
    return groups, each, -(-groups // each)


@pytest.mark.parametrize("width", [1, 64, 65, 2048, 2049, 2560, 4096, 12288, 65536])
@pytest.mark.parametrize("batch,per", [(1, 1), (1, 5), (3, 4)])
@pytest.mark.parametrize("back", [False, True])
def test_whoever_is_waited_for_holds_a_lower_ticket(width, batch, per, back):
    """Tickets of a queue cover every tile of its run of channel groups once, a tile's predecessor
    (its successor in the backward) before the tile; the queues cover all groups."""
    groups, each, queues = queues_of(width)
    tiles = batch * per
    grid = tiles * queues * each
    covered = set()
    for queue in range(queues):
        issued = len(range(queue, grid, queues))  # workgroups that take a ticket of this queue
        assert issued == tiles * each
        done = set()
        for ticket in range(issued):
            run = queue if queues % 8 else queue % 8 * (queues // 8) + queue // 8  # neighbouring ones on an XCD
            group, j = run * each + ticket % each, ticket // each
            j = tiles - 1 - j if back else j
            b, i = j % batch, j // batch
            if group >= groups:
                continue
            before = (group, b, i + 1 if back else i - 1)
            assert before in done or before[2] in (-1, per)
            assert (group, b, i) not in covered
            done.add((group, b, i))
            covered.add((group, b, i))
    assert len(covered) == groups * tiles
