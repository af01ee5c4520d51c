"""Pins of the float64 forms of the tree operators and of the adjustments of
logits: hand-worked values and identities, and a mistake that each has to show."""
import numpy as np
import pytest

from oracle import tree_oracle as TO

#        0
#      / | \
#     1  2  5
#    / \     \
#   3   4     6      7: a root of its own
PARENT = [-1, 0, 0, 1, 1, 0, 5, -1]


def test_mask_by_hand():
    sees, depth = TO.tree_mask(PARENT)
    want = [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 4], [0, 5], [0, 5, 6], [7]]
    assert [list(np.flatnonzero(r)) for r in sees] == want
    assert list(depth) == [0, 1, 1, 2, 2, 1, 2, 0]
    assert list(TO.pack_bits(sees)[:, 0]) == [1, 3, 5, 11, 19, 33, 97, 128]
    sees, depth = TO.tree_mask(PARENT, 4)
    assert list(depth) == [0, 1, 1, 2, -1, -1, -1, -1] and not sees[4:].any()
    # a parent that is the node itself takes its subtree out
    sees, depth = TO.tree_mask([-1, 1, 1, 0, 2])
    assert list(depth) == [0, -1, -1, 1, -1] and not sees[[1, 2, 4]].any()


def test_bits_past_a_word():
    sees = np.zeros((1, 70), bool)
    sees[0, [0, 31, 32, 69]] = True
    assert list(TO.pack_bits(sees)[0].view(np.uint32)) == [0x80000001, 1, 32]


def test_attention_identities():
    rng = np.random.default_rng(5)
    n, nq, nkv, d, C = 5, 4, 2, 8, 9
    q, k, v = rng.normal(size=(n, nq, d)), rng.normal(size=(C, nkv, d)), rng.normal(size=(C, nkv, d))
    kt, vt = rng.normal(size=(n, nkv, d)), rng.normal(size=(n, nkv, d))
    sees, _ = TO.tree_mask([-1, 0, 1, 0, 3])
    o, lse, _ = TO.tree_attention(q, k, v, kt, vt, sees, 0.3)
    # each path alone, as a chain, gives its last node's output
    for i in range(n):
        at = np.flatnonzero(sees[i])
        oc, lc, _ = TO.tree_attention(q[at], k, v, kt[at], vt[at], np.tril(np.ones((len(at),) * 2, bool)), 0.3)
        assert np.allclose(o[i], oc[-1], atol=1e-14) and np.allclose(lse[i], lc[-1], atol=1e-13)
    # keys in the cache or in the tree are one set
    oa, la, _ = TO.tree_attention(q[:1], k[:0], v[:0], np.concatenate([k, kt[:1]]), np.concatenate([v, vt[:1]]),
                                  np.ones((1, C + 1), bool), 0.3)
    assert np.allclose(oa[0], o[0], atol=1e-14) and np.allclose(la[0], lse[0], atol=1e-13)
    # no key; one key; equal keys
    oz, lz, _ = TO.tree_attention(q[:1], k[:0], v[:0], kt[:1], vt[:1], np.zeros((1, 1), bool), 0.3)
    assert (oz == 0).all() and (lz == -np.inf).all()
    o1, l1, _ = TO.tree_attention(q[:1], k[:0], v[:0], kt[:1], vt[:1], np.ones((1, 1), bool), 0.3)
    assert np.allclose(o1[0], np.repeat(vt[0], 2, axis=0)) and np.allclose(l1[0, 0], 0.3 * q[0, 0] @ kt[0, 0])
    oe, _, _ = TO.tree_attention(q[:1], np.ones_like(k), v, kt[:1], vt[:1], np.zeros((1, 1), bool), 0.3)
    assert np.allclose(oe[0, 3], v[:, 1].mean(0))
    # a mask of one node more is another answer
    wrong = sees.copy()
    wrong[4, 1] = True
    assert not np.allclose(TO.tree_attention(q, k, v, kt, vt, wrong, 0.3)[0][4], o[4], atol=1e-3)


@pytest.mark.parametrize("tok,R,want", [
    # the target says 11 at the root (node 1), 14 there (node 4), then 99
    ([11, 14, 0, 0, 99, 0, 0, 0], 5, (2, 99, [0, 1, 4, -1, -1], [11, 14, 99, -1, -1], 99)),
    # no child of the root says 50
    ([50, 14, 0, 0, 99, 0, 0, 0], 3, (0, 50, [0, -1, -1], [50, -1, -1], 50)),
    # a path of two nodes is full
    ([11, 14, 0, 0, 99, 0, 0, 0], 2, (1, 14, [0, 1], [11, 14], 14)),
    # a draw that failed ends the path without a correction
    ([15, 0, 0, 0, 0, -1, 0, 0], 4, (1, -1, [0, 5, -1, -1], [15, -1, -1, -1], 15)),
    ([-1] * 8, 2, (0, -1, [0, -1], [-1, -1], 10)),
])
def test_accept_by_hand(tok, R, want):
    tree = [10, 11, 12, 13, 14, 15, 16, 17]
    assert TO.tree_accept(tok, tree, PARENT, R) == want


def test_accept_takes_the_first_of_equal_children():
    assert TO.tree_accept([7, 1, 8, 3], [0, 7, 7, 8], [-1, 0, 0, 2], 4)[2] == [0, 1, -1, -1]
    assert TO.tree_accept([7, 1, 8, 3], [0, 7, 7, 8], [-1, 0, 0, 2], 4, n=1)[:2] == (0, 7)
    assert TO.tree_accept([7], [0], [-1], 1, n=0) == (-1, -1, [-1], [-1], -1)


def test_accept_of_a_chain_is_the_greedy_rule():
    from oracle import dflash_oracle as O
    rng = np.random.default_rng(3)
    for _ in range(200):
        R = int(rng.integers(2, 6))
        logits = rng.normal(size=(R, 3))
        draft = rng.integers(0, 3, R - 1)
        n, corr, emitted, nxt = O.verify_accept(logits, draft)
        tok = logits.argmax(1)
        got = TO.tree_accept(tok, np.concatenate([[9], draft]), list(range(-1, R - 1)), R)
        assert got[0] == n and got[1] == corr and list(got[3]) == list(emitted) and got[4] == nxt


def test_adjust_by_hand():
    z = [2.0, -2.0, 1.0, 0.0, -1.0, 3.0]
    x, _ = TO.adjust_row(z, prompt=[0, 1], made=[1, 2, 2, 9, -1], repetition=2.0, frequency=0.25, presence=0.5,
                         bias=[(3, 1.0), (3, 0.5), (4, -np.inf), (-1, 7.0), (6, 7.0)],
                         allowed=np.array([1, 1, 1, 1, 1, 0], bool))
    # 0: 2/2; 1: -2*2 - .25 - .5; 2: 1/2 - 2*.25 - .5; 3: two biases; 4: banned; 5: not allowed
    assert list(x) == [1.0, -4.75, -0.5, 1.5, -np.inf, -np.inf]
    assert list(TO.adjust_row(z)[0]) == z
    # the prompt alone asks for no frequency or presence penalty
    assert TO.adjust_row(z, prompt=[5], presence=1.0)[0][5] == 3.0


# ---- the ring of K and V tiles that two streams share (a model of its barriers) ----
def _ring(seed, slots, release_first, tiles=40):
    """Copies land in any order; stream m uses tiles m, m + 2, ... (K then V of
    each).  A wait passes where a phase of its parity is the last one over, as
    the hardware decides it.  'early': it passed before the tile had landed."""
    r = np.random.default_rng(seed)
    full, empty, sent, flying = [0] * slots, [0] * slots, 0, []
    at = [0, 2]  # each stream's next tile, K and V counted
    passes = lambda over, n: (over - 1) % 2 == n % 2
    while min(at) < 2 * tiles:
        who = r.integers(4)
        if who == 0 and sent < 2 * tiles:
            if sent < slots or passes(empty[sent % slots], sent // slots - 1):
                flying.append(sent)
                sent += 1
        elif who == 1 and flying:
            full[flying.pop(r.integers(len(flying))) % slots] += 1
        elif who >= 2 and at[who - 2] < 2 * tiles:
            x = at[who - 2]
            s, n = x % slots, x // slots
            if release_first and x >= slots and not passes(empty[s], n - 1):
                continue
            if passes(full[s], n):
                if full[s] != n + 1:
                    return "early"
                empty[s] += 1
                at[who - 2] += 3 if x % 2 else 1
    return "done"


@pytest.mark.parametrize("slots", [5, 6, 12])
def test_two_streams_share_a_ring(slots):
    assert all(_ring(seed, slots, True) == "done" for seed in range(150))


@pytest.mark.parametrize("slots", [5, 6])
def test_a_ring_whose_slots_change_hands_needs_the_release(slots):
    assert "early" in {_ring(seed, slots, False) for seed in range(30)}
