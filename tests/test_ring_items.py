"""A model of the barriers by which two streams share the attention's ring of K
and V tiles, over several items: stream m of an item uses its tiles m, m + 2, ...
(K, then V of each), so an odd number of tiles changes which stream has a slot.
An item's products of both streams are over before either begins the next one's
(its Q is only then in place); copies run ahead over items as slots come free."""
import numpy as np
import pytest


def _ring(seed, slots, items, release_first, steps=200000):
    """'done'; 'early': a wait passed before its tile had landed; 'lost': a tile
    was sent for into a slot still in use; 'stuck'.  A wait passes where a phase
    of its parity is the last one over, as the hardware decides it."""
    r = np.random.default_rng(seed)
    base = np.concatenate([[0], 2 * np.cumsum(items)])
    total = int(base[-1])
    full, empty, sent, flying = [0] * slots, [0] * slots, 0, []
    used = [False] * total
    item, at = 0, [0, 2]  # place of each stream in the item, K and V counted
    passes = lambda over, n: (over - 1) % 2 == n % 2
    for _ in range(steps):
        if item == len(items):
            return "done"
        if min(at) >= 2 * items[item]:  # both streams have ended the item
            item, at = item + 1, [0, 2]
            continue
        who = r.integers(4)
        if who == 0 and sent < total:
            if sent < slots or passes(empty[sent % slots], sent // slots - 1):
                if sent >= slots and not used[sent - slots]:
                    return "lost"
                flying.append(sent)
                sent += 1
        elif who == 1 and flying:
            full[flying.pop(r.integers(len(flying))) % slots] += 1
        elif who >= 2 and at[who - 2] < 2 * items[item]:
            x = int(base[item]) + at[who - 2]
            s, n = x % slots, x // slots
            if release_first and x >= slots and not passes(empty[s], n - 1):
                continue
            if passes(full[s], n):
                if full[s] != n + 1:
                    return "early"
                used[x] = True
                empty[s] += 1
                at[who - 2] += 3 if at[who - 2] % 2 else 1
    return "stuck"


ITEMS = [[1] * 30, [1, 2, 3, 1, 4, 5, 1, 1, 7, 2, 9], [3] * 12, [5, 5, 1, 5, 2, 5], [13, 1, 8], [2, 1] * 9]


@pytest.mark.parametrize("slots", [5, 6, 12])
@pytest.mark.parametrize("items", ITEMS, ids=str)
def test_streams_share_the_ring_over_items(slots, items):
    for seed in range(40):
        assert _ring(seed, slots, items, True) == "done", seed


@pytest.mark.parametrize("slots", [5, 6])
def test_the_model_shows_a_missing_wait(slots):
    seen = {_ring(seed, slots, items, False) for seed in range(30) for items in ([13, 9, 8], [40])}
    assert seen & {"early", "lost", "stuck"}
