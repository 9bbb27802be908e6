"""Drafted trees: masks, attention over the cache, and the accepted path moved together, against
the oracles.  The attention's bound is test_gpu_attention's, masks and moved rows are exact."""
import numpy as np
import pytest
import torch

import draft_sampling_lossless_amd as dsl
from oracle import attention as oa
from oracle import pages as op

from gpu_util import dev, host, say
from test_gpu_attention import INF, NAN, SENT, bits, check_rows, paged_case, value

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(dspark_lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def tree_of(g, n, depth=None):
    """Random parents: any earlier node, or near ones (deep trees); a few roots."""
    p = [-1] + [int(g.integers(max(0, j - 3) if depth else 0, j)) for j in range(1, n)]
    for j in range(1, n):
        if g.random() < 0.05:
            p[j] = -1
    return p


# ---------------------------------------------------------------- masks

@pytest.mark.parametrize("lens", [[1], [25], [128], [0, 1, 2, 0, 64], [65, 127, 33], [5] * 300])
def test_tree_mask(lens):
    g = np.random.default_rng(len(lens) + sum(lens))
    parent = np.array([p for i, n in enumerate(lens) for p in (tree_of(g, n, i % 2) if n else [])], np.int32)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    kv = np.array([n + g.integers(0, 5000) for n in lens], np.int32)
    T = int(cu[-1])
    extra = np.concatenate([parent, np.zeros(3, np.int32)])                # rows behind the last tree
    mask = torch.full((T + 3, 4), SENT, dtype=torch.int32, device="cuda")
    pos = torch.full((T + 3,), SENT, dtype=torch.int32, device="cuda")
    dsl.tree_mask(dev(extra), dev(kv), dev(cu), max(max(lens), 1), mask=mask, positions=pos)
    want, places = oa.tree_mask(parent, kv, cu)
    assert np.array_equal(host(mask)[:T].view(np.uint32), want) and np.array_equal(host(pos)[:T], places)
    assert (host(mask)[T:] == SENT).all() and (host(pos)[T:] == SENT).all()


def test_tree_mask_chains_odd_parents_and_max_q():
    n = 128
    chain = np.arange(-1, n - 1, dtype=np.int32)
    mask, pos = dsl.tree_mask(dev(chain), dev(np.array([500], np.int32)), dev(np.array([0, n], np.int32)), n)
    want, places = oa.tree_mask(chain, [500], [0, n])
    assert np.array_equal(host(mask).view(np.uint32), want) and np.array_equal(host(pos), places)
    odd = np.array([0, 1, 5, -2, 1, -2 ** 31, 2 ** 31 - 1, 4], np.int32)    # itself, a later one, none
    mask, pos = dsl.tree_mask(dev(odd), dev(np.array([3], np.int32)), dev(np.array([0, 8], np.int32)), 8)
    want, places = oa.tree_mask(odd, [3], [0, 8])
    assert np.array_equal(host(mask).view(np.uint32), want) and np.array_equal(host(pos), places)
    mask = torch.full((8, 4), SENT, dtype=torch.int32, device="cuda")
    pos = torch.full((8,), SENT, dtype=torch.int32, device="cuda")
    dsl.tree_mask(dev(odd), dev(np.array([3], np.int32)), dev(np.array([0, 8], np.int32)), 5, mask=mask, positions=pos)
    assert np.array_equal(host(mask)[:5].view(np.uint32), want[:5]) and (host(mask)[5:] == SENT).all()
    assert (host(pos)[5:] == SENT).all()


# ---------------------------------------------------------------- attention

def run(c, mask, lse=True, max_q=None):
    T, nh, hd = c["q"].shape
    out = torch.full((T, nh, hd), SENT, dtype=torch.int16, device="cuda")
    ls = torch.full((T, nh), 7.0, dtype=torch.float32, device="cuda") if lse else None
    dsl.tree_attention(dev(c["q"]), dev(c["kc"]), dev(c["vc"]), dev(c["table"]), dev(c["kv"]), dev(c["cu"]), dev(mask),
                       max_q or c["max_q"], c["page"], out=out, lse=ls)
    return out, ls


def widen(c):
    """The same call under a table for long contexts, which lets large trees take workgroups of
    256 rows (from 2^19 keys times kv heads that the tables have room for)."""
    B, have = c["table"].shape
    width = -(-2 ** 19 // (c["kc"].shape[1] * B * c["page"]))
    return dict(c, table=np.concatenate([c["table"], np.full((B, max(0, width - have)), -1, np.int32)], 1))


def ref(c, mask):
    return oa.tree(c["q"], c["kc"], c["vc"], c["table"], c["kv"], c["cu"], mask, c["page"], c["hd"] ** -0.5)


def masks(g, c):
    parent = [p for n in np.diff(c["cu"]) for p in (tree_of(g, int(n), n % 2) if n else [])]
    return oa.tree_mask(parent, c["kv"], c["cu"])[0]


@pytest.mark.parametrize("nh,nkv,hd,page,qlen,kvlen", [
    (4, 1, 128, 16, [1], [1]),
    (8, 8, 128, 16, [4], [133]),                              # few rows
    (8, 2, 128, 1, [4, 3], [133, 40]),
    (8, 2, 128, 64, [4], [5003]),                             # split and joined
    (8, 2, 64, 16, [2, 1, 4], [33, 1, 64]),
    (8, 2, 256, 32, [3, 4], [95, 700]),
    (32, 8, 128, 16, [25], [613]),                            # many rows
    (8, 2, 128, 64, [60, 17], [1500, 17]),
    (8, 2, 128, 1, [33, 64], [900, 70]),
    (4, 1, 64, 16, [128], [400]),                             # every word of a mask
    (4, 1, 64, 1, [128, 100], [128, 2000]),
    (4, 2, 256, 16, [40, 9], [300, 20]),
    (4, 2, 256, 8, [97], [140]),
    (10, 2, 128, 4, [11, 2, 30], [31, 32, 33]),               # groups of 5
    (8, 2, 64, 32, [20, 0, 2], [50, 60, 1100]),
    (8, 2, 128, 16, [20, 3, 1], [7, 0, 2]),                   # fewer keys than nodes, none
    (16, 1, 128, 16, [40], [200]),                            # 640 rows
    (8, 2, 128, 16, [16] * 70, [200] * 70),
    (16, 2, 128, 16, [30, 17, 32], [3000, 520, 700]),         # blocks of 256 rows: one, two, part of one
    (16, 2, 64, 64, [40, 33], [2600, 700]),
    (16, 2, 128, 1, [20, 17], [2300, 90]),                    # more slots than are looked up at once
    (16, 2, 64, 2, [24, 128], [1100, 1500]),
    (6, 2, 128, 32, [64, 5], [18000, 300]),                  # more groups of 16 than are looked up at once
])
def test_tree_attention(nh, nkv, hd, page, qlen, kvlen):
    say(f"tree nh={nh} nkv={nkv} hd={hd} page={page} q={qlen[:4]} kv={kvlen[:4]}")
    g = np.random.default_rng(nh + hd + page)
    c = paged_case(g, nh, nkv, hd, page, qlen, kvlen)
    mask = masks(g, c)
    out, lse = run(c, mask)
    r = check_rows(out, lse, ref(c, mask), hd, "tree")
    say(f"  worst error at {r:.2f} of its bound")
    assert torch.equal(out, run(c, mask)[0]) and torch.equal(out, run(c, mask, lse=False)[0])
    c = widen(c)
    out, lse = run(c, mask)
    r = check_rows(out, lse, ref(c, mask), hd, "wide")
    say(f"  worst error at {r:.2f} of its bound")
    assert torch.equal(out, run(c, mask)[0]) and torch.equal(out, run(c, mask, lse=False)[0])


@pytest.mark.parametrize("nh,n", [(4, 3), (4, 40), (1, 128), (2, 100)])
def test_any_mask(nh, n):
    """Masks that are no trees: random bits, none (rows that see the context alone, or nothing at
    all), bits of nodes that do not exist."""
    g = np.random.default_rng(n)
    for kv in (n, n + 1, n + 45):
        c = paged_case(g, nh, 1, 128, 16, [n], [kv])
        mask = g.integers(0, 2 ** 32, (n, 4), dtype=np.uint32)
        mask[::3] = 0
        out, lse = run(widen(c), mask)
        check_rows(out, lse, ref(c, mask), 128, f"wide, kv {kv}")
        out, lse = run(c, mask)
        check_rows(out, lse, ref(c, mask), 128, f"kv {kv}")
        if kv == n:
            assert (host(out)[::3] == 0).all() and np.isneginf(host(lse)[::3]).all()
    mask[:] = 2 ** 32 - 1                          # everything: paged attention without a causal mask
    out, lse = run(c, mask)
    full = oa.paged(c["q"], c["kc"], c["vc"], c["table"], c["kv"], c["cu"], 16, False, 128 ** -0.5)
    check_rows(out, lse, full, 128, "full")


def test_every_place_of_a_block_in_a_tile():
    g = np.random.default_rng(4)
    for ctx in range(0, 36, 5):
        for page in (16, 1):
            c = paged_case(g, 2, 1, 64, page, [37], [ctx + 37])
            mask = masks(g, c)
            out, lse = run(c, mask)
            check_rows(out, lse, ref(c, mask), 64, f"context {ctx}")
            c = widen(paged_case(g, 4, 1, 128, page, [37], [2 * ctx + 37]))
            out, lse = run(c, mask)
            check_rows(out, lse, ref(c, mask), 128, f"wide, context {2 * ctx}")


def test_a_chain_is_causal_attention():
    g = np.random.default_rng(6)
    for nh, qlen, kvlen, page in ((4, [3, 2], [400, 90], 16), (8, [20, 33], [1300, 40], 1), (8, [17], [3000], 64)):
        c = paged_case(g, nh, 2, 128, page, qlen, kvlen)
        parent = np.concatenate([np.arange(-1, n - 1) for n in qlen])
        out, lse = run(c, oa.tree_mask(parent, c["kv"], c["cu"])[0])
        chain = oa.paged(c["q"], c["kc"], c["vc"], c["table"], c["kv"], c["cu"], page, True, 128 ** -0.5)
        check_rows(out, lse, chain, 128, "chain")


def test_branches_do_not_see_each_others_infinities():
    g = np.random.default_rng(8)
    parent = [-1, 0, 0, 1, 2, 1, 4]
    for nh, page in ((2, 16), (8, 16), (8, 1), (32, 16), (32, 1)):   # every kernel
        c = widen(paged_case(g, nh, 1, 128, page, [7], [60]))
        mask = oa.tree_mask(parent, c["kv"], c["cu"])[0]
        at = 53 + 2                                # node 2, seen by 2, 4 and 6
        slot = int(c["table"][0, at // page]) * page + at % page
        for kb, vb in ((NAN, INF), (INF, NAN), (0xFF80, NAN)):
            c["kc"][slot], c["vc"][slot] = kb, vb
            out, lse = run(c, mask)
            if kb != 0xFF80:
                assert np.isnan(value(out)[[2, 4, 6]]).any(axis=(1, 2)).all()
            # (such a tile's values are added key by key: another order of the same float32 sums,
            # which the bound counts, so that bits may differ from a clean tile's)
            w = ref(c, mask)
            w["written"][[2, 4, 6]] = False
            check_rows(out, lse, w, 128, f"{nh} {page} {kb:x}")


def test_tree_rows_left_alone_hidden_pages_and_two_streams():
    g = np.random.default_rng(9)
    c = paged_case(g, 8, 2, 128, 16, [25, 9], [613, 90])
    mask = masks(g, c)
    out, _ = run(c, mask, max_q=9)
    assert (host(out)[9:25] == SENT).all()
    w = ref(c, mask)
    w["written"][9:25] = False
    check_rows(out, None, w, 128, "max_q")
    c["table"][0, 37], c["table"][1, 1] = -1, 10 ** 9      # a page of the block, one of the context
    out, lse = run(c, mask)
    check_rows(out, lse, ref(c, mask), 128, "hidden")
    d = widen(paged_case(g, 16, 2, 128, 16, [25, 18], [613, 90]))
    d["table"][0, [0, 37]], d["table"][1, 1] = -1, 10 ** 9
    m = masks(g, d)
    check_rows(*run(d, m), ref(d, m), 128, "hidden, wide")
    args = [dev(c[k]) for k in ("q", "kc", "vc", "table", "kv", "cu")] + [dev(mask)]
    outs = [torch.empty_like(out) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in outs]
    torch.cuda.synchronize()
    for _ in range(10):
        for o, s in zip(outs, streams):
            with torch.cuda.stream(s):
                dsl.tree_attention(*args, c["max_q"], 16, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)


def test_trees_in_a_graph_follow_the_lengths():
    """Masks, and attention by workgroups of 256 rows, captured once; lengths and trees change."""
    g = np.random.default_rng(31)
    B, n, page = 2, 40, 16
    c = widen(paged_case(g, 8, 2, 128, page, [n] * B, [900] * B))
    q = dev(np.concatenate([c["q"].reshape(B * n, -1), c["q"].reshape(B * n, -1)], 1)).unflatten(1, (-1, 128))[:, :8]   # strided
    args = [q] + [dev(c[k]) for k in ("kc", "vc", "table", "kv", "cu")]
    parent = dev(np.array(tree_of(g, n) * B, np.int32))
    mask, pos = torch.empty((B * n, 4), dtype=torch.int32, device="cuda"), torch.empty(B * n, dtype=torch.int32, device="cuda")
    out = torch.empty((B * n, 8, 128), dtype=torch.int16, device="cuda")
    ws = torch.empty(dsl.paged_attention_workspace_size(B * n, B, n, 8, 2, 128), dtype=torch.uint8, device="cuda")

    def body():
        dsl.tree_mask(parent, args[4], args[5], n, mask=mask, positions=pos)
        dsl.tree_attention(*args, mask, n, page, out=out, workspace=ws)

    body()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for kv in ([900, 41], [300, 899], [40, 640]):
        trees = tree_of(g, n) + tree_of(g, n, 1)
        parent.copy_(torch.tensor(trees, dtype=torch.int32))
        args[4].copy_(torch.tensor(kv, dtype=torch.int32))
        graph.replay()
        got = out.clone()
        out.fill_(SENT)
        body()
        assert torch.equal(got, out)
        c["kv"] = np.array(kv, np.int32)
        want, places = oa.tree_mask(trees, kv, c["cu"])
        assert np.array_equal(host(mask).view(np.uint32), want) and np.array_equal(host(pos), places)
        check_rows(got, None, ref(c, want), 128, str(kv))


# ---------------------------------------------------------------- accepted paths

def compact_case(g, L, nkv, hd, page, blocks, ctxs):
    kv = [n + c for n, c in zip(blocks, ctxs)]
    need = [-(-n // page) for n in kv]
    order = g.permutation(sum(need) + 2)
    table, at = np.full((len(kv), max(max(need), 1)), -1, np.int32), 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    slots = (sum(need) + 2) * page
    cache = lambda: g.integers(0, 2 ** 16, (L, slots, nkv, hd), dtype=np.uint16)  # noqa: E731
    return dict(kc=cache(), vc=cache(), table=table, kv=np.array(kv, np.int32),
                cu=np.concatenate([[0], np.cumsum(blocks)]).astype(np.int32), page=page)


def check_compact(c, path, accepted):
    k, v = dev(c["kc"]), dev(c["vc"])
    lens = dsl.kv_compact(k, v, dev(c["table"]), dev(c["kv"]), dev(c["cu"]), dev(path), dev(accepted), c["page"])
    for got, was in ((k, c["kc"]), (v, c["vc"])):
        want, new = op.compact(was, c["table"], c["kv"], c["cu"], path, accepted, c["page"])
        assert np.array_equal(host(got).view(np.uint16), want) and np.array_equal(host(lens), new)


@pytest.mark.parametrize("L,nkv,hd,page,blocks,ctxs", [
    (1, 1, 8, 16, [4], [0]),
    (5, 8, 128, 16, [25], [517]),
    (2, 8, 128, 1, [64, 1, 0, 128], [3, 90, 5, 0]),
    (3, 3, 40, 4, [30] * 9, list(range(9))),
    (2, 40, 128, 64, [128, 128], [63, 64]),       # rows longer than a workgroup's pieces
    (1, 2, 64, 32, [17] * 200, list(range(200))),
])
def test_compact(L, nkv, hd, page, blocks, ctxs):
    g = np.random.default_rng(L + hd + page)
    c = compact_case(g, L, nkv, hd, page, blocks, ctxs)
    most = max(max(blocks), 1)
    path = np.full((len(blocks), most), -1, np.int32)
    accepted = np.zeros(len(blocks), np.int32)
    for b, n in enumerate(blocks):
        accepted[b] = g.integers(0, n + 1)
        path[b, :accepted[b]] = np.sort(g.permutation(n)[:accepted[b]])
    check_compact(c, path, accepted)
    for b, n in enumerate(blocks):                # all of it: nothing moves
        path[b, :n] = np.arange(n)
    check_compact(c, path, np.array(blocks, np.int32))


def test_compact_odd_paths():
    g = np.random.default_rng(2)
    c = compact_case(g, 2, 2, 64, 16, [9] * 8, [20, 3, 0, 15, 16, 17, 40, 2])
    path = np.array([[0, 2, 2, 5], [3, 1, 4, 5], [8, 9, 10, 11], [-1, 0, 1, 2], [0, 4, 8, 2 ** 31 - 1], [-5, -4, 3, 4],
                     [2, 3, 4, 8], [1, 2, 3, 4]], np.int32)
    for accepted in ([4] * 8, [-3, 0, 1, 2, 3, 9, 2 ** 31 - 1, -2 ** 31]):
        check_compact(c, path, np.array(accepted, np.int32))
    c["table"][1, 0], c["table"][6, 2], c["table"][7, 0] = -1, 1 << 30, -9   # rows without a page
    check_compact(c, path, np.full(8, 4, np.int32))
    c["kv"][:4] = [4, 0, 9, 8]                    # fewer cached than nodes
    check_compact(c, path, np.full(8, 4, np.int32))


def test_compact_one_layer_and_repeats():
    g = np.random.default_rng(3)
    c = compact_case(g, 1, 8, 128, 16, [40, 33], [100, 7])
    path, accepted = np.array([[0, 3, 9, 30], [1, 2, 7, -1]], np.int32), np.array([4, 3], np.int32)
    k, v = dev(c["kc"][0]), dev(c["vc"][0])
    dsl.kv_compact(k, v, dev(c["table"]), dev(c["kv"]), dev(c["cu"]), dev(path), dev(accepted), 16)
    want, _ = op.compact(c["kc"], c["table"], c["kv"], c["cu"], path, accepted, 16)
    assert np.array_equal(host(k).view(np.uint16), want[0])


# ---------------------------------------------------------------- a round

def test_a_round_with_a_tree():
    """Room for the tree, its tokens appended, attention, the accepted path kept and the rest's
    pages given back; the next round's attention over what is left equals one that had appended
    the accepted tokens as a chain."""
    g = np.random.default_rng(11)
    L, nh, nkv, hd, page, B = 2, 8, 2, 128, 16, 3
    ctx, n = [37, 5, 160], [9, 16, 12]
    P, W = 64, 16
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    kv_len = torch.zeros(B, dtype=torch.int32, device="cuda")
    as_dev = lambda x: dev(np.array(x, np.int32))  # noqa: E731
    kc = torch.zeros((L, P * page, nkv, hd), dtype=torch.int16, device="cuda")
    vc = torch.zeros_like(kc)

    def slots(lo, hi):
        t = host(table)
        keys = [(b, s) for b in range(B) for s in range(lo[b], hi[b])]
        return dev(np.array([t[b, s // page] * page + s % page for b, s in keys], np.int64))

    def append(k, v, positions, lo, hi):
        for layer in range(L):
            dsl.kv_append(dev(k[layer]), dev(v[layer]), as_dev(positions), slots(lo, hi), kc[layer], vc[layer])

    def draw(m):
        return [bits(g, m, nkv, hd) for _ in range(L)], [bits(g, m, nkv, hd) for _ in range(L)]

    _, served = dsl.pages_resize(table, kv_len, as_dev(ctx), refs, page)
    assert host(served).all()
    append(*draw(sum(ctx)), [p for c in ctx for p in range(c)], [0] * B, ctx)
    parent = [p for m in n for p in [-1] + [int(g.integers(0, j)) for j in range(1, m)]]
    cu = as_dev(np.concatenate([[0], np.cumsum(n)]))
    full = [c + m for c, m in zip(ctx, n)]
    dsl.pages_resize(table, kv_len, as_dev(full), refs, page)
    mask, positions = dsl.tree_mask(as_dev(parent), kv_len, cu, max(n))
    k, v = draw(sum(n))
    append(k, v, host(positions), ctx, full)
    q = bits(g, sum(n), nh, hd, std=2.0)
    for layer in range(L):
        out = dsl.tree_attention(dev(q), kc[layer], vc[layer], table, kv_len, cu, mask, max(n), page)
        want = oa.tree(q, host(kc[layer]).view(np.uint16), host(vc[layer]).view(np.uint16), host(table), host(kv_len),
                       host(cu), host(mask).view(np.uint32), page, hd ** -0.5)
        check_rows(out, None, want, hd, f"layer {layer}")
    # the path to each tree's last node
    path, begin = np.full((B, max(n)), -1, np.int32), np.concatenate([[0], np.cumsum(n)])
    chains = []
    for b in range(B):
        node, up = n[b] - 1, []
        while node >= 0:
            up.append(node)
            node = parent[begin[b] + node]
        chains.append(up[::-1])
        path[b, :len(up)] = up[::-1]
    accepted = [len(c) for c in chains]
    new_len = dsl.kv_compact(kc, vc, table, kv_len, cu, dev(path), as_dev(accepted), page)
    dsl.pages_resize(table, kv_len, new_len, refs, page)
    kept = [c + a for c, a in zip(ctx, accepted)]
    assert host(kv_len).tolist() == kept
    assert int(refs.sum()) == sum(-(-m // page) for m in kept) == int((table >= 0).sum())
    got = [x.clone() for x in (kc, vc)]
    take = np.concatenate([begin[b] + np.array(chains[b]) for b in range(B)])
    append([x[take] for x in k], [x[take] for x in v], [ctx[b] + i for b in range(B) for i in range(accepted[b])], ctx, kept)
    at = slots([0] * B, kept)
    assert torch.equal(got[0][:, at], kc[:, at]) and torch.equal(got[1][:, at], vc[:, at])
