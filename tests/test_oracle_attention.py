"""Pins of the attention oracle (oracle/attention.py) on the CPU: hand-worked rows, the
rotation's invariants, and the paged form against the packed one."""
import numpy as np
import pytest

import synth
from oracle import attention as oa
from oracle import context_kv as ck


def bits(x):
    return synth.bf16_bits(np.asarray(x, np.float32))


def test_one_key_returns_its_value():
    q, k, v = bits(np.ones((1, 2, 4))), bits(np.full((1, 1, 4), 3.0)), bits([[[1.0, -2.0, 0.5, 8.0]]])
    r = oa.prompt(q, k, v, [0, 1], True, 0.5)
    assert np.array_equal(r["out"][0, 0], [1.0, -2.0, 0.5, 8.0]) and np.array_equal(r["out"][0, 1], r["out"][0, 0])
    assert r["lse"][0, 0] == 0.5 * 12.0


def test_weights_by_hand():
    # scores 0 and ln 3 (as scale * q.k): weights 1/4 and 3/4
    q, k = bits([[[1.0, 0.0]], [[1.0, 0.0]]]), bits([[[0.0, 5.0]], [[1.0, 7.0]]])
    v = bits([[[4.0, 0.0]], [[0.0, 8.0]]])
    r = oa.prompt(q, k, v, [0, 2], False, np.log(3.0))
    assert np.allclose(r["out"][:, 0], [[1.0, 6.0], [1.0, 6.0]], atol=1e-15)
    assert np.allclose(r["lse"], np.log(4.0))
    r = oa.prompt(q, k, v, [0, 2], True, np.log(3.0))
    assert np.array_equal(r["out"][0, 0], [4.0, 0.0]) and np.allclose(r["out"][1, 0], [1.0, 6.0])


def test_rows_without_keys_are_zero_and_rows_behind_are_not_written():
    q, c = bits(np.ones((4, 1, 4))), bits(np.ones((8, 1, 4)))
    # two query tokens at the end of one cached token: the first sees nothing
    r = oa.paged(q, c, c, np.array([[0], [1]]), [1, 0], [0, 2, 3], 4, True, 1.0)
    assert np.array_equal(r["out"][0, 0], np.zeros(4)) and r["lse"][0, 0] == -np.inf
    assert np.array_equal(r["out"][1, 0], np.ones(4))
    assert np.array_equal(r["out"][2, 0], np.zeros(4)) and r["written"].tolist() == [True, True, True, False]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("page", [1, 4])
def test_paged_equals_packed(causal, page):
    g = np.random.default_rng(3)
    n, nh, nkv, hd = 11, 4, 2, 8
    q, k, v = (bits(g.normal(size=(n, h, hd))) for h in (nh, nkv, nkv))
    pages = -(-n // page)
    order = g.permutation(pages + 3)[:pages]
    kc, vc = bits(g.normal(size=((pages + 3) * page, nkv, hd))), bits(g.normal(size=((pages + 3) * page, nkv, hd)))
    slot = order[np.arange(n) // page] * page + np.arange(n) % page
    kc[slot], vc[slot] = k, v
    a = oa.prompt(q, k, v, [0, n], causal, 0.4)
    b = oa.paged(q[-3:], kc, vc, order[None], [n], [0, 3], page, causal, 0.4)
    assert np.allclose(a["out"][-3:], b["out"], atol=1e-14) and np.allclose(a["lse"][-3:], b["lse"])


def test_a_page_outside_the_cache_hides_its_keys():
    g = np.random.default_rng(4)
    c, q = bits(g.normal(size=(16, 1, 4))), bits(g.normal(size=(1, 1, 4)))
    for bad in (-1, 4, 1 << 30):
        r = oa.paged(q, c, c, np.array([[0, bad, 2]]), [12], [0, 1], 4, True, 1.0)
        s = oa.paged(q, c, c, np.array([[0, 2]]), [8], [0, 1], 4, True, 1.0)
        assert np.allclose(r["out"], s["out"]) and r["keys"][0] == 8


def test_append_is_the_context_kv_rotation():
    g = np.random.default_rng(5)
    x, w = bits(g.normal(size=(5, 3, 8))), bits(1 + 0.1 * g.normal(size=8))
    pos = np.array([0, 1, 77, 40000, 131071])
    got = oa.append(x, w, pos, 1e-6, 1e4)
    for m in range(5):
        want = ck.rope_rotate_half(ck.rms_norm(ck.bf16_decode(x[m]), ck.bf16_decode(w), 1e-6), pos[m], 1e4)
        assert np.allclose(got[m], want, atol=1e-12)
    plain = oa.append(x, None, pos, 1e-6, 1e4)
    assert np.array_equal(plain[0], ck.bf16_decode(x[0]))                    # position 0
    assert np.allclose((plain ** 2).sum(-1), (ck.bf16_decode(x) ** 2).sum(-1))
