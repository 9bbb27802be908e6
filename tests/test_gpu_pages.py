"""The pool of pages: resize, select and page copies, bit for bit against oracle/pages.py."""
import numpy as np
import pytest
import torch

import draft_sampling_lossless_amd as dsl
from oracle import pages as op

from gpu_util import dev, host, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu(dspark_lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def i32(x):
    return np.ascontiguousarray(x, np.int32)


def check_resize(table, kv, new, refs, page):
    t, k, r = dev(i32(table)), dev(i32(kv)), dev(i32(refs))
    copies, served = dsl.pages_resize(t, k, dev(i32(new)), r, page)
    want = op.resize(table, kv, new, refs, page)
    for got, w, name in zip((t, k, r, copies, served), want, ("page_table", "kv_len", "refs", "copies", "served")):
        assert np.array_equal(host(got), w), name
    return want


def pool(g, B, W, P, page, lens, share=0.0):
    """A table of random pages; some rows share a beginning with the row before."""
    table, refs, at = np.full((B, W), -1), np.zeros(P, np.int64), 0
    order = g.permutation(P)
    for b, n in enumerate(lens):
        hold, own = -(-n // page), 0
        if b and g.random() < share:
            own = min(hold, -(-lens[b - 1] // page))
            table[b, :own] = table[b - 1, :own]
        table[b, own:hold] = order[at:at + hold - own]
        at += hold - own
        np.add.at(refs, table[b, :hold], 1)
    return table, refs


@pytest.mark.parametrize("B,W,P,page", [
    (1, 1, 1, 1), (1, 40, 64, 16), (3, 5, 9, 4), (64, 8, 512, 16), (65, 3, 4097, 2), (300, 10, 3001, 8),
    (1024, 4, 4099, 16), (1025, 4, 4097, 16), (4096, 3, 20001, 4), (7, 700, 5001, 16),
])
@pytest.mark.parametrize("share", [0.0, 0.8])
def test_resize(B, W, P, page, share):
    say(f"resize B={B} W={W} P={P} page={page} share={share}")
    g = np.random.default_rng(B + W + P)
    lens = g.integers(0, W * page + 1, B)
    while sum(-(-n // page) for n in lens) > P:            # they fit, whatever is shared
        lens //= 2
    table, refs = pool(g, B, W, P, page, lens, share)
    for _ in range(3):
        new = np.clip(lens + g.integers(-2 * page, 2 * page + 2, B), -3, W * page + 3)
        table, lens, refs, copies, served = check_resize(table, lens, new, refs, page)
        say(f"  copies {int((copies[:, 0] >= 0).sum())}, not served {int((served == 0).sum())}, free {int((refs == 0).sum())}")
    check_resize(table, lens, np.zeros(B), refs, page)     # everything given back
    check_resize(table, lens, np.full(B, W * page), refs, page)   # more than there is


@pytest.mark.parametrize("free", range(0, 14))
def test_a_pool_that_runs_out(free):
    """Every place at which the free pages can end, in and between the requests' needs; copies
    among them, and the request that would have kept the shared page."""
    page, W = 4, 6
    table, P = np.full((6, W), -1), 40
    refs = np.ones(P, np.int64)
    table[0, :2], table[1, :2], table[2, :2], table[3, :1], table[5, :2] = [0, 1], [0, 1], [0, 1], [2], [3, 4]
    refs[[0, 1]] = 3
    kv, new = np.array([6, 6, 6, 4, 0, 7]), np.array([13, 7, 10, 12, 5, 8])
    refs[20:20 + free] = 0
    check_resize(table, kv, new, refs, page)
    check_resize(table, kv, np.array([13, 7, 6, 12, 5, 8]), refs, page)       # two of three grow
    check_resize(table, kv, np.array([2, 7, 10, 12, 5, 8]), refs, page)       # one of three gives its pages back


def test_everyone_shares_one_page():
    for B in (2, 257, 4096):
        page, P = 16, 5000
        table, refs = np.full((B, 2), -1), np.zeros(P, np.int64)
        table[:, 0], refs[77] = 77, B
        kv = np.full(B, 5)
        t, k, r, copies, served = check_resize(table, kv, kv + 1, refs, page)
        assert (copies[:-1, 0] == 77).all() and t[-1, 0] == 77 and r[77] == 1 and served.all()


@pytest.mark.parametrize("B", [2, 64, 130])
@pytest.mark.parametrize("gives_back", [False, True])
def test_shared_pages_that_all_leave_are_not_free(B, gives_back):
    """Pairs share a page and both grow, so that its count is 0 for a while; waves without a request
    look through these counts, and the free pages lie behind them."""
    page, P = 16, 20000
    pairs = B // 2
    for first in (256, 4000, 8192 + 256):
        table, refs = np.full((B + 1, 3), -1), np.ones(P, np.int64)
        at = first + 61 * np.arange(pairs) % 3000
        table[:B, 0] = np.repeat(at, 2)
        refs[at], refs[P - 2 * B:] = 2, 0
        kv, new = np.full(B + 1, 7), np.full(B + 1, 20)
        table[B, :2], kv[B], new[B] = [1, 2], 30, 30
        if gives_back:
            new[B] = 10
        t, k, r, copies, served = check_resize(table, kv, new, refs, page)
        assert (copies[0:B:2, 0] == at).all() and (copies[1:B:2, 0] == -1).all() and served.all()
        assert (r[at] == 1).all() and t[0, 0] == (2 if gives_back else P - 2 * B)


@pytest.mark.parametrize("free", [0, 5, 900, 1400, 3000])
def test_groups_that_share_and_a_pool_that_may_not_last(free):
    """1500 requests in groups of 1 to 7 on a page each, most of which grow; 40000 pages, the free ones
    far behind each other."""
    g = np.random.default_rng(free)
    B, P, page = 1500, 40000, 16
    group = np.repeat(np.arange(B), g.integers(1, 8, B))[:B]
    table, refs = np.full((B, 4), -1), np.ones(P, np.int64)
    table[:, 0] = 3 * group
    refs[:] = 1
    for p in set(table[:, 0].tolist()):
        refs[p] = (table[:, 0] == p).sum()
    refs[g.permutation(np.arange(3 * B, P))[:free]] = 0
    order = g.permutation(B)                               # groups lie among each other
    table = table[order]
    kv = np.full(B, 9)
    for grows in (1.0, 0.9, 0.3):
        new = np.where(g.random(B) < grows, g.integers(10, 40, B), g.integers(0, 10, B))
        check_resize(table, kv, new, refs, page)


def test_pages_that_are_not_there_are_passed_over():
    table = np.array([[-1, 3, 99, -7], [5, -1, -1, -1], [2, 1 << 30, -1, -1]])
    refs = np.array([0, 0, 1, 1, 0, 1])
    for new in ([2, 3, 2], [16, 9, 5], [14, 4, 7], [0, 0, 0]):
        check_resize(table, np.array([13, 3, 6]), np.array(new), refs, 4)


@pytest.mark.parametrize("B,rows,W,page", [(1, 1, 1, 1), (4, 9, 5, 4), (256, 256, 66, 16), (4096, 100, 3, 2), (3, 4096, 300, 16)])
def test_select(B, rows, W, page):
    g = np.random.default_rng(B + rows)
    P = 3000
    lens = g.integers(0, W * page + 1, B)
    while sum(-(-n // page) for n in lens) > P:
        lens //= 2
    table, refs = pool(g, B, W, P, page, lens, 0.3)
    table[0, 0] = -1 if B > 3 else table[0, 0]
    src = g.integers(-2, B + 2, rows)
    r = dev(i32(refs))
    t, k = dsl.pages_select(dev(i32(table)), dev(i32(lens)), dev(i32(src)), r, page)
    for got, want in zip((t, k, r), op.select(table, lens, src, refs, page)):
        assert np.array_equal(host(got), want)


@pytest.mark.parametrize("L,nkv,hd,page", [(1, 1, 8, 1), (5, 8, 128, 16), (2, 3, 40, 4), (3, 8, 128, 256), (1, 2, 64, 64)])
def test_copy_pages(L, nkv, hd, page):
    g = np.random.default_rng(L + page)
    P = 24
    k, v = (g.integers(0, 2 ** 16, (L, P * page, nkv, hd), dtype=np.uint16) for _ in range(2))
    copies = i32([[3, 10], [-1, -1], [3, 11], [P, 12], [4, P], [5, -1], [23, 0], [7, 7], [2 ** 31 - 1, 13], [6, 23 - 1]])
    a, b = dev(k), dev(v)
    dsl.kv_copy_pages(a, b, dev(copies), page)
    assert np.array_equal(host(a).view(np.uint16), op.copy_pages(k, copies, page))
    assert np.array_equal(host(b).view(np.uint16), op.copy_pages(v, copies, page))
    dsl.kv_copy_pages(a, b, dev(copies[:0]), page)


def test_far_layers_and_slots():
    """Offsets that pass 32 bits: a cache of 5 GB, pages at both ends."""
    L, page, P, nkv, hd = 5, 64, 8192, 8, 128
    k = torch.zeros((L, P * page, nkv, hd), dtype=torch.int16, device="cuda")
    v = torch.zeros_like(k)
    k[-1, :page], v[-1, -page:] = 5, 6
    dsl.kv_copy_pages(k, v, dev(i32([[0, P - 2], [P - 1, 1]])), page)
    assert (k[-1, -2 * page:-page] == 5).all() and int(k.sum(dtype=torch.int64)) == 2 * 5 * page * nkv * hd
    assert (v[-1, page:2 * page] == 6).all() and int(v.sum(dtype=torch.int64)) == 2 * 6 * page * nkv * hd
    table = i32([[P - 1, P - 2]])
    dsl.kv_compact(k, v, dev(table), dev(i32([70])), dev(i32([0, 9])), dev(i32([[5]])), dev(i32([1])), page)
    assert (k[-1, -page + 61] == 5).all()                   # token 61 took the rows of token 66
    assert (k[-1, -page:-page + 61] == 0).all() and (k[-1, -page + 62:] == 0).all()


def test_rounds_in_a_graph():
    """Forked requests grow, copy, shrink: a round captured once, replayed against the oracle."""
    g = np.random.default_rng(5)
    B, W, P, page, L, nkv, hd = 12, 20, 300, 16, 2, 2, 64
    lens = g.integers(1, 200, B)
    table, refs = pool(g, B, W, P, page, lens, 0.5)
    k, v = (g.integers(0, 2 ** 16, (L, P * page, nkv, hd), dtype=np.uint16) for _ in range(2))
    dk, dv, dt, dl, dr = dev(k), dev(v), dev(i32(table)), dev(i32(lens)), dev(i32(refs))
    dsrc, dgrow, dkeep = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    nt, nl = torch.empty_like(dt), torch.empty_like(dl)
    copies, served = torch.empty((B, 2), dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")

    def body():
        dsl.pages_select(dt, dl, dsrc, dr, page, new_table=nt, new_len=nl)
        dsl.pages_resize(nt, nl, dgrow, dr, page, copies=copies, served=served)
        dsl.kv_copy_pages(dk, dv, copies, page)
        dsl.pages_resize(nt, nl, dkeep, dr, page)
        dt.copy_(nt)
        dl.copy_(nl)

    start = [x.clone() for x in (dk, dv, dt, dl, dr)]
    dgrow.copy_(dl)
    dkeep.copy_(dl)
    dsrc.copy_(torch.arange(B))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        body()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for x, s in zip((dk, dv, dt, dl, dr), start):
        x.copy_(s)
    copied = 0
    for _ in range(8):
        src = g.integers(-1, B, B)
        t, n, r = op.select(table, lens, src, refs, page)
        grow = np.clip(n + g.integers(0, 40, B), 0, W * page)
        t, n, r, c, s = op.resize(t, n, grow, r, page)
        k, v = op.copy_pages(k, c, page), op.copy_pages(v, c, page)
        keep = np.maximum(n - g.integers(0, 40, B), 0)
        table, lens, refs, _, _ = op.resize(t, n, keep, r, page)
        for d, x in ((dsrc, src), (dgrow, grow), (dkeep, keep)):
            d.copy_(torch.from_numpy(i32(x)))
        graph.replay()
        for got, want in ((dt, table), (dl, lens), (dr, refs), (copies, c), (served, s)):
            assert np.array_equal(host(got), want)
        assert np.array_equal(host(dk).view(np.uint16), k) and np.array_equal(host(dv).view(np.uint16), v)
        copied += int((c[:, 0] >= 0).sum())
    assert copied > 10
