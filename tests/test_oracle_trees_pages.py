"""Pins of the oracles of windows, drafted trees (oracle/attention.py) and of the cache's rows and
pages (oracle/pages.py) on the CPU: cases worked by hand, and what must hold whatever the input."""
import numpy as np
import pytest

import synth
from oracle import attention as oa
from oracle import pages as op


def bits(x):
    return synth.bf16_bits(np.asarray(x, np.float32))


def uniform_rows(n, nh=1, hd=4):
    """Queries of zeros (every score 0: the mean of what is seen), values 2^s in dim 0."""
    v = np.zeros((n, 1, hd))
    v[:, 0, 0] = 2.0 ** np.arange(n)
    return bits(np.zeros((n, nh, hd))), bits(np.zeros((n, 1, hd))), bits(v)


def test_window_by_hand():
    q, k, v = uniform_rows(6)
    r = oa.prompt(q, k, v, [0, 6], True, 1.0, window=2, sinks=1)
    assert np.allclose(r["out"][:, 0, 0], [1, 3 / 2, 7 / 3, 13 / 3, 25 / 3, 49 / 3])
    assert r["keys"].tolist() == [1, 2, 3, 3, 3, 3]
    r = oa.prompt(q, k, v, [0, 6], True, 1.0, window=1)
    assert np.allclose(r["out"][:, 0, 0], 2.0 ** np.arange(6))
    r = oa.paged(q[:2], k, v, np.array([[0, 1, 2]]), [6], [0, 2], 2, False, 1.0, window=2, sinks=1)
    assert np.allclose(r["out"][:, 0, 0], [(1 + 8 + 16 + 32) / 4, (1 + 16 + 32) / 3])   # what is behind a row is seen


@pytest.mark.parametrize("window", [1, 3, 7, 11, 40])
@pytest.mark.parametrize("sinks", [0, 2, 11, 40])
def test_paged_window_equals_packed(window, sinks):
    g = np.random.default_rng(window + sinks)
    n, nh, nkv, hd = 11, 4, 2, 8
    q, k, v = (bits(g.normal(size=(n, h, hd))) for h in (nh, nkv, nkv))
    order = g.permutation(6)[:3]
    kc, vc = bits(g.normal(size=(24, nkv, hd))), bits(g.normal(size=(24, nkv, hd)))
    slot = order[np.arange(n) // 4] * 4 + np.arange(n) % 4
    kc[slot], vc[slot] = k, v
    a = oa.prompt(q, k, v, [0, n], True, 0.4, window=window, sinks=sinks)
    b = oa.paged(q[-5:], kc, vc, order[None], [n], [0, 5], 4, True, 0.4, window=window, sinks=sinks)
    assert np.allclose(a["out"][-5:], b["out"], atol=1e-14) and np.allclose(a["lse"][-5:], b["lse"])
    if window >= n or sinks >= n:
        assert np.array_equal(a["out"], oa.prompt(q, k, v, [0, n], True, 0.4)["out"])


def test_tree_mask_by_hand():
    #        0        3 (a second root)
    #      1   2      |
    #      |          5
    #      4
    mask, pos = oa.tree_mask([-1, 0, 0, -1, 1, 3], [10], [0, 6])
    assert mask[:, 0].tolist() == [1, 3, 5, 8, 19, 40] and not mask[:, 1:].any()
    assert pos.tolist() == [4, 5, 5, 4, 6, 5]
    mask, pos = oa.tree_mask(np.arange(-1, 127), [128], [0, 128])             # a chain
    assert mask[127].tolist() == [2 ** 32 - 1] * 4 and pos.tolist() == list(range(128))
    mask, pos = oa.tree_mask([0, 5, -7, 1], [4], [0, 4])                      # no parents, and one
    assert mask[:, 0].tolist() == [1, 2, 4, 10] and pos.tolist() == [0, 0, 0, 1]


def test_a_chain_is_causal_and_branches_do_not_meet():
    g = np.random.default_rng(3)
    nh, nkv, hd, n, kv = 4, 2, 8, 5, 13
    q, kc, vc = bits(g.normal(size=(n, nh, hd))), bits(g.normal(size=(16, nkv, hd))), bits(g.normal(size=(16, nkv, hd)))
    table = np.array([[2, 0, 3, 1]])
    chain, _ = oa.tree_mask(np.arange(-1, n - 1), [kv], [0, n])
    a = oa.tree(q, kc, vc, table, [kv], [0, n], chain, 4, 0.5)
    b = oa.paged(q, kc, vc, table, [kv], [0, n], 4, True, 0.5)
    assert np.array_equal(a["out"], b["out"]) and np.array_equal(a["lse"], b["lse"])
    # nodes 1 and 2 below 0, 3 below 1, 4 below 2: each path is a chain of its own
    tree, pos = oa.tree_mask([-1, 0, 0, 1, 2], [kv], [0, n])
    assert pos.tolist() == [8, 9, 9, 10, 10]
    r = oa.tree(q, kc, vc, table, [kv], [0, n], tree, 4, 0.5)
    flat = table[0][np.arange(16) // 4] * 4 + np.arange(16) % 4
    for path in ([0, 1, 3], [0, 2, 4]):
        keys = np.concatenate([flat[:8], flat[8 + np.array(path)]])
        s = oa.prompt(np.concatenate([q[:1]] * 8 + [q[path]]), kc[keys], vc[keys], [0, 11], True, 0.5)
        assert np.allclose(r["out"][path], s["out"][8:], atol=1e-14)


def test_compact_by_hand():
    cache = np.arange(2 * 16).reshape(2, 16, 1)
    table = np.array([[3, 1, -1], [0, 2, -1]])
    # request 0: context 2, tree of 5 over places 2..6, path 0, 2, 4; request 1: nothing accepted
    after, lens = op.compact(cache, table, [7, 6], [0, 5, 9], np.array([[0, 2, 4], [1, 2, 3]]), [3, 0], 4)
    assert lens.tolist() == [5, 2]
    want = cache.copy()
    want[:, 15], want[:, 4] = cache[:, 4], cache[:, 6]
    assert np.array_equal(after, want)
    # a path that turns back ends; one that leaves the block too
    _, lens = op.compact(cache, table, [7, 6], [0, 5, 9], np.array([[1, 3, 2], [0, 4, 3]]), [3, 3], 4)
    assert lens.tolist() == [4, 3]


def test_resize_by_hand():
    table = np.array([[5, 0, -1], [5, 1, -1], [2, -1, -1]])
    refs = np.array([1, 1, 1, 0, 0, 2, 0, 0])
    # grows within its page, gives one back, takes two
    t, kv, r, copies, served = op.resize(table, [6, 8, 3], [8, 4, 12], refs, 4)
    assert t.tolist() == [[5, 0, -1], [5, -1, -1], [2, 1, 3]] and kv.tolist() == [8, 4, 12]
    assert r.tolist() == [1, 1, 1, 1, 0, 2, 0, 0] and (copies == -1).all() and served.all()
    # three share page 7, two of them grow: both take copies; then the last alone keeps it
    table, refs = np.array([[7, -1], [7, -1], [7, -1]]), np.array([0, 0, 0, 0, 0, 0, 0, 3])
    t, kv, r, copies, served = op.resize(table, [2, 2, 2], [3, 2, 5], refs, 4)
    assert t.tolist() == [[0, -1], [7, -1], [1, 2]] and copies.tolist() == [[7, 0], [-1, -1], [7, 1]]
    assert r.tolist() == [1, 1, 1, 0, 0, 0, 0, 1]
    t, kv, r, copies, served = op.resize(table, [2, 2, 2], [3, 3, 3], refs, 4)
    assert t.tolist() == [[0, -1], [1, -1], [7, -1]] and copies.tolist() == [[7, 0], [7, 1], [-1, -1]]
    # the pool runs out in the middle: what needs nothing is served all the same
    table, refs = np.array([[0, -1, -1], [1, -1, -1], [2, -1, -1], [3, -1, -1]]), np.array([1, 1, 1, 1, 0])
    t, kv, r, copies, served = op.resize(table, [4, 4, 4, 1], [8, 12, 8, 4], refs, 4)
    assert served.tolist() == [1, 0, 0, 1] and kv.tolist() == [8, 4, 4, 4]
    assert t.tolist() == [[0, 4, -1], [1, -1, -1], [2, -1, -1], [3, -1, -1]] and r.tolist() == [1] * 5


def test_select_by_hand():
    table, refs = np.array([[0, 1], [2, 9], [3, -1]]), np.array([1, 1, 1, 1, 0])
    t, kv, r = op.select(table, [7, 4, 0], [0, 0, -1, 2, 5], refs, 4)
    assert t.tolist() == [[0, 1], [0, 1], [-1, -1], [-1, -1], [-1, -1]] and kv.tolist() == [7, 7, 0, 0, 0]
    assert r.tolist() == [2, 2, 0, 1, 0]


def count(table, kv, page, P):
    refs = np.zeros(P, np.int64)
    for row, n in zip(table, kv):
        np.add.at(refs, row[:-(-n // page)], 1)
    return refs


def test_counts_always_count_the_table():
    g = np.random.default_rng(5)
    P, W, page, B = 60, 6, 4, 9
    table, kv, refs = np.full((B, W), -1), np.zeros(B, np.int64), np.zeros(P, np.int64)
    for _ in range(200):
        new = np.clip(kv + g.integers(-9, 12, B), 0, W * page)
        before = table.copy(), kv.copy()
        table, kv, refs, copies, served = op.resize(table, kv, new, refs, page)
        assert np.array_equal(refs, count(table, kv, page, P)) and np.array_equal(kv[served == 1], new[served == 1])
        for b in np.flatnonzero(kv > before[1]):          # what a request will write into is its own
            assert all(refs[p] == 1 for p in table[b, before[1][b] // page:-(-kv[b] // page)])
            keep = before[1][b] // page
            assert np.array_equal(table[b, :keep], before[0][b, :keep])
        table, kv, refs = op.select(table, kv, g.integers(-1, B, B), refs, page)
        assert np.array_equal(refs, count(table, kv, page, P))
