"""Paged and prompt attention under a window with sinks, against the oracle (oracle/attention.py,
float64).  The bound is test_gpu_attention's: it counts the keys that a row sees, whichever
those are."""
import numpy as np
import pytest
import torch

import draft_sampling_lossless_amd as dsl
from oracle import attention as oa

from gpu_util import dev, host, say
from test_gpu_attention import INF, NAN, SENT, bits, check_rows, paged_case, value

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _gpu(dspark_lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def drop(c, window, sinks, junk=NAN):
    """The pages that no row sees leave the table; theirs and every unseen key's rows become junk."""
    page = c["page"]
    for b, kv in enumerate(c["kv"].tolist()):
        low = kv - int(c["cu"][b + 1] - c["cu"][b]) - window + 1
        for s in range(kv):
            if sinks <= s < low:
                at = int(c["table"][b, s // page]) * page + s % page
                c["kc"][at] = c["vc"][at] = junk
        for p in range(-(-kv // page)):
            if p * page >= sinks and (p + 1) * page <= low:
                c["table"][b, p] = -1
    return c


def run(c, causal, window, sinks, lse=True, max_q=None):
    T, nh, hd = c["q"].shape
    out = torch.full((T, nh, hd), SENT, dtype=torch.int16, device="cuda")
    ls = torch.full((T, nh), 7.0, dtype=torch.float32, device="cuda") if lse else None
    dsl.paged_attention(dev(c["q"]), dev(c["kc"]), dev(c["vc"]), dev(c["table"]), dev(c["kv"]), dev(c["cu"]),
                        max_q or c["max_q"], c["page"], causal=causal, out=out, lse=ls, window=window, sinks=sinks)
    return out, ls


def ref(c, causal, window, sinks):
    return oa.paged(c["q"], c["kc"], c["vc"], c["table"], c["kv"], c["cu"], c["page"], causal, c["hd"] ** -0.5,
                    window, sinks)


@pytest.mark.parametrize("nh,nkv,hd,page,qlen,kvlen,causal,window,sinks", [
    (4, 1, 128, 16, [1], [1], True, 1, 0),
    (8, 2, 128, 16, [1], [517], True, 1, 0),                  # one key alone
    (8, 2, 128, 16, [1], [517], True, 64, 4),
    (8, 2, 128, 1, [1], [517], True, 33, 3),
    (8, 2, 128, 64, [1], [5003], True, 4000, 70),             # split over ranges and joined
    (8, 2, 128, 1, [3], [5001], True, 2900, 33),              # slots one by one, split
    (4, 2, 64, 16, [1, 1, 1], [33, 1, 64], True, 16, 1),
    (4, 2, 256, 32, [2, 1], [95, 700], True, 31, 2),
    (8, 1, 256, 8, [5, 3], [40, 9], False, 6, 0),
    (10, 2, 128, 4, [1, 2, 3], [31, 32, 33], True, 5, 1),
    (16, 1, 128, 16, [17, 1, 9], [300, 5, 9], True, 100, 4),  # 272 rows: several row blocks
    (8, 8, 128, 256, [4, 16], [255, 257], False, 40, 10),
    (32, 8, 128, 64, [17, 3, 1, 9], [1000, 700, 17, 64], True, 129, 4),
    (6, 2, 64, 2, [7, 8], [7, 100], True, 3, 1),              # narrower than the block
    (8, 2, 64, 16, [128, 1], [200, 3], True, 50, 16),
    (24, 8, 64, 32, [5, 0, 2], [50, 60, 1100], True, 512, 32),
    (8, 2, 128, 16, [2, 1, 3], [0, 0, 2], True, 8, 4),        # nothing cached; fewer keys than query tokens
    (8, 2, 128, 16, [2, 1], [0, 40], False, 8, 4),
    (8, 1, 256, 1, [8, 2], [700, 65], True, 90, 5),
    (8, 1, 256, 32, [16, 16], [90, 300], True, 64, 64),
    (8, 1, 64, 1, [6, 2], [700, 65], False, 200, 1),
    (512, 1, 64, 16, [2], [70], True, 20, 2),
    (8, 2, 128, 16, [4, 2], [900, 300], True, MOST, MOST),    # all of it
    (8, 2, 128, 16, [4, 2], [900, 300], True, 10, MOST),
    (8, 2, 128, 16, [4, 2], [900, 300], True, 10, 600),       # sinks that reach the window of one
])
def test_paged_window(nh, nkv, hd, page, qlen, kvlen, causal, window, sinks):
    say(f"window nh={nh} nkv={nkv} hd={hd} page={page} q={qlen} kv={kvlen} causal={causal} window={window} sinks={sinks}")
    c = drop(paged_case(np.random.default_rng(nh + hd + page), nh, nkv, hd, page, qlen, kvlen), window, sinks)
    out, lse = run(c, causal, window, sinks)
    r = check_rows(out, lse, ref(c, causal, window, sinks), hd, "window")
    say(f"  worst error at {r:.2f} of its bound")
    assert torch.equal(out, run(c, causal, window, sinks)[0])
    assert torch.equal(out, run(c, causal, window, sinks, lse=False)[0])


@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("qlen", [[1], [17]])
def test_every_place_of_a_window_in_a_tile(page, qlen):
    """Windows that begin at each place of a tile of 32 keys, sinks that end at each."""
    g = np.random.default_rng(page)
    for d in range(0, 34, 3):
        c = drop(paged_case(g, 4, 1, 128, page, qlen, [200 + d]), 60 + d % 5, d)
        out, lse = run(c, True, 60 + d % 5, d)
        check_rows(out, lse, ref(c, True, 60 + d % 5, d), 128, f"offset {d}")


@pytest.mark.parametrize("B", [65, 600])
def test_paged_window_many_requests(B):
    g = np.random.default_rng(B)
    qlen, kvlen = g.integers(0, 4, B).tolist(), g.integers(0, 200, B).tolist()
    kvlen[B // 2], kvlen[B - 1] = 3900, 2500
    qlen[B // 2] = qlen[B - 1] = 2
    for window, sinks in ((50, 4), (2100, 40)):
        say(f"window B={B} window={window}")
        c = drop(paged_case(g, 4, 2, 64, 16, qlen, kvlen), window, sinks)
        out, lse = run(c, True, window, sinks)
        check_rows(out, lse, ref(c, True, window, sinks), 64, "window")


def test_a_window_past_the_beginning_is_paged_attention():
    g = np.random.default_rng(2)
    for page, qlen, kvlen in ((16, [1, 2], [3000, 60]), (1, [9, 4], [700, 70]), (64, [17], [2000])):
        c = paged_case(g, 8, 2, 128, page, qlen, kvlen)
        plain = dsl.paged_attention(dev(c["q"]), dev(c["kc"]), dev(c["vc"]), dev(c["table"]), dev(c["kv"]), dev(c["cu"]),
                                    c["max_q"], page)
        for window, sinks in ((3000, 0), (MOST, 5)):
            assert torch.equal(run(c, True, window, sinks, lse=False)[0], plain)


def test_unseen_keys_under_a_window_do_not_matter():
    """NaN and infinities in keys that some rows of a tile see and others do not: the rows that see
    them become NaN, the others stay within their bound (such a tile's values are added key by
    key: another order of the same float32 sums, which the bound counts)."""
    g = np.random.default_rng(8)
    window, sinks, kv = 40, 2, 150
    for page in (16, 1):
        for nh, qlen in ((4, 3), (8, 9)):                # both kernels
            c = paged_case(g, nh, 1, 128, page, [qlen], [kv])
            first = kv - qlen - window + 1               # seen by the first token alone
            slot = lambda s: int(c["table"][0, s // page]) * page + s % page  # noqa: E731
            c["kc"][slot(first)], c["vc"][slot(first)] = INF, NAN
            for s in (sinks, first - 1):                 # seen by none
                c["kc"][slot(s)], c["vc"][slot(s)] = NAN, INF
            c["vc"][slot(kv - 1)] = NAN                  # seen by the last token alone
            out, lse = run(c, True, window, sinks)
            a = value(out)
            assert np.isnan(a[0]).all() and np.isnan(a[-1]).all()
            w = ref(c, True, window, sinks)
            w["written"][[0, -1]] = False
            check_rows(out, lse, w, 128, f"{page} {nh}")


def test_rows_left_alone_and_hidden_pages():
    g = np.random.default_rng(9)
    c = paged_case(g, 8, 2, 128, 16, [5, 3], [300, 90])
    out, _ = run(c, True, 33, 4, max_q=2)
    got = host(out)
    assert (got[[2, 3, 4, 7]] == SENT).all()
    w = ref(c, True, 33, 4)
    w["written"][[2, 3, 4, 7]] = False
    check_rows(out, None, w, 128, "max_q")
    c["table"][0, 17], c["table"][1, 0] = -1, 1 << 30      # a page of the window, the sinks' page
    out, lse = run(c, True, 33, 4)
    check_rows(out, lse, ref(c, True, 33, 4), 128, "hidden")
    c["table"][:] = -1
    out, lse = run(c, True, 33, 4)
    assert (host(out) == 0).all() and np.isneginf(host(lse)).all()


def test_a_block_longer_than_max_q_and_the_window():
    """cu_q gives a request more tokens than max_q: the first max_q see their own windows."""
    g = np.random.default_rng(10)
    for qlen, kvlen in (([120], [1500]), ([120, 4], [1500, 30])):
        c = paged_case(g, 2, 1, 64, 16, qlen, kvlen)
        out, _ = run(c, True, 900, 4, max_q=8)
        w = ref(c, True, 900, 4)
        w["written"][8:120] = False
        check_rows(out, None, w, 64, "long block")
        assert (host(out)[8:120] == SENT).all()


@pytest.mark.parametrize("nh,nkv,hd,page,qlen,kvlen,causal,window,sinks,max_q", [
    # several requests planned, rows straight into registers
    (8, 2, 128, 16, [1, 1, 1], [5000, 4100, 5003], True, 2000, 4, None),
    (8, 2, 128, 1, [1, 3, 1], [5000, 30, 4007], True, 2003, 0, None),
    (16, 2, 64, 64, [2, 2], [6001, 3500], False, 2500, 33, None),
    (4, 2, 256, 32, [4, 1], [5001, 2700], True, 2100, 65, None),
    # several requests planned, tiles shared by eight waves, by four, by several row blocks
    (32, 8, 128, 16, [17, 17], [4000, 3001], True, 1500, 40, None),
    (32, 8, 128, 16, [17, 9], [4000, 3001], True, 1501, 0, None),
    (32, 8, 128, 1, [17, 17], [4000, 3001], True, 1500, 40, None),
    (32, 8, 128, 1, [17, 5], [4000, 3001], True, 1503, 0, None),
    (8, 2, 128, 16, [9, 3], [3000, 2903], True, 1300, 7, None),
    (8, 2, 256, 16, [17, 17], [3000, 2500], True, 1400, 20, None),
    (16, 1, 64, 8, [17, 17], [3000, 2500], False, 1400, 20, None),    # 272 rows
    # one request, cut without a plan
    (32, 8, 128, 16, [17], [9000], True, 1500, 40, None),
    (32, 8, 128, 1, [17], [5000], True, 1500, 0, None),
    (8, 2, 128, 64, [1], [9001], True, 3500, 0, None),
    (8, 2, 64, 16, [33], [5000], False, 1111, 64, None),
    # blocks longer than max_q: their spans pass what the host counts with
    (2, 1, 64, 16, [120], [4000], True, 1500, 4, 8),
    (2, 1, 64, 16, [120, 4], [4000, 2300], True, 1500, 4, 8),
    (8, 2, 128, 16, [700], [4000], True, 1500, 40, 9),
    (8, 2, 128, 1, [700, 12], [4000, 2500], True, 1500, 0, 9),
    # whole, as enough workgroups come without a cut: more slots than are looked up at once
    (64, 64, 64, 1, [17] * 8, [2600, 40, 40, 1900, 17, 40, 40, 40], True, 1500, 40, None),
    (64, 64, 64, 1, [17] * 8, [2600, 40, 40, 1900, 17, 40, 40, 40], True, 1500, 0, None),
])
def test_windows_cut_into_ranges(nh, nkv, hd, page, qlen, kvlen, causal, window, sinks, max_q):
    """Ranges that begin behind the keys left out, and their join."""
    say(f"cut nh={nh} nkv={nkv} hd={hd} page={page} q={qlen} kv={kvlen} causal={causal} window={window} sinks={sinks}")
    c = drop(paged_case(np.random.default_rng(nh + hd + page), nh, nkv, hd, page, qlen, kvlen), window, sinks)
    out, lse = run(c, causal, window, sinks, max_q=max_q)
    w = ref(c, causal, window, sinks)
    for b, n in enumerate(qlen):
        w["written"][int(c["cu"][b]) + min(n, max_q or n):int(c["cu"][b + 1])] = False
    r = check_rows(out, lse, w, hd, "cut")
    say(f"  worst error at {r:.2f} of its bound")
    assert (host(out)[~w["written"]] == SENT).all()
    assert torch.equal(out, run(c, causal, window, sinks, max_q=max_q)[0])
    assert torch.equal(out, run(c, causal, window, sinks, lse=False, max_q=max_q)[0])


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("width", [0, 2000])
@pytest.mark.parametrize("nh,qlen,kvlen", [
    (4, [2], [0]),
    (4, [4], [1]),
    (8, [20], [7]),
    (8, [20, 3, 1, 4], [7, 1, 400, 0]),
])
def test_fewer_keys_than_tokens_under_the_longest_window(nh, qlen, kvlen, width, page):
    """Places before the first key, a window and sinks that pass every length: the begin of the first
    window lies further below 0 than 32 bits less the sinks hold.  width: keys that the table has
    room for, so that requests are cut."""
    say(f"longest window nh={nh} q={qlen} kv={kvlen} width={width} page={page}")
    c = paged_case(np.random.default_rng(sum(qlen)), nh, 2, 128, page, qlen, kvlen)
    B, have = c["table"].shape
    c["table"] = np.concatenate([c["table"], np.full((B, max(0, width // page - have)), -1, np.int32)], 1)
    for window, sinks in ((MOST, MOST), (MOST, 2 ** 30 - 31), (2 ** 30, 2 ** 30), (3, MOST), (MOST, 1)):
        for causal in (True, False):
            out, lse = run(c, causal, window, sinks)
            check_rows(out, lse, ref(c, causal, window, sinks), 128, f"{window} {sinks} {causal}")


# ---------------------------------------------------------------- prompts

def run_prompt(q, k, v, cu, window, sinks, lse=True):
    T, nh, hd = q.shape
    out = torch.full((T, nh, hd), SENT, dtype=torch.int16, device="cuda")
    ls = torch.full((T, nh), 7.0, dtype=torch.float32, device="cuda") if lse else None
    dsl.prompt_attention(dev(q), dev(k), dev(v), dev(cu), out=out, lse=ls, window=window, sinks=sinks)
    return out, ls


@pytest.mark.parametrize("nh,nkv,hd,lens,window,sinks", [
    (4, 1, 128, [1], 1, 0),
    (4, 2, 128, [65, 1, 0, 31], 1, 0),
    (4, 2, 128, [65, 1, 0, 31], 7, 2),
    (4, 1, 64, [300], 64, 4),
    (4, 1, 64, [300, 129, 64], 33, 70),
    (8, 1, 64, [1200], 200, 1),                   # long: eight waves
    (2, 2, 64, [1100], 130, 65),                  # heads that share nothing: 256 tokens a workgroup
    (4, 1, 128, [700], 100, 16),
    (4, 4, 128, [600], 300, 0),
    (2, 1, 128, [600, 40], 1000, 4),              # reaches past the beginning
    (8, 1, 256, [260, 33], 48, 3),
    (2, 2, 256, [300], 64, 64),
    (5, 1, 128, [200, 77], 50, 33),               # groups of 5
    (4, 2, 64, [90], MOST, MOST),
    (4, 2, 64, [90], 5, MOST),
    (16, 1, 128, [150], 32, 32),
    (512, 1, 64, [20, 3], 7, 2),                  # more heads on one than a workgroup has rows
    (2, 1, 64, [3, 0, 17, 40] * 18, 9, 3),        # more sequences than lanes
    (2, 1, 128, [5, 33, 0] * 70, 20, 1),
])
def test_prompt_window(nh, nkv, hd, lens, window, sinks):
    say(f"prompt window nh={nh} nkv={nkv} hd={hd} lens={lens} window={window} sinks={sinks}")
    g = np.random.default_rng(nh + hd + sum(lens))
    T = sum(lens) + 2                             # two rows behind the last sequence
    q, k, v = bits(g, T, nh, hd, std=2.0), bits(g, T, nkv, hd), bits(g, T, nkv, hd)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    out, lse = run_prompt(q, k, v, cu, window, sinks)
    r = check_rows(out, lse, oa.prompt(q, k, v, cu, True, hd ** -0.5, window, sinks), hd, "prompt window")
    say(f"  worst error at {r:.2f} of its bound")
    assert (host(out)[-2:] == SENT).all() and (host(lse)[-2:] == 7.0).all()
    assert torch.equal(out, run_prompt(q, k, v, cu, window, sinks, lse=False)[0])


@pytest.mark.parametrize("nh,nkv,hd,lens,window", [
    (2, 2, 64, [1300], 1100),                     # 256 tokens a workgroup: its last waves see later first tiles
    (4, 1, 64, [1700, 1203], 1090),
    (5, 1, 64, [1250], 1101),                     # a group that no row block divides
    (4, 4, 128, [900, 700], 600),
    (2, 1, 128, [1100, 0, 803], 531),
    (5, 1, 128, [900], 577),
])
@pytest.mark.parametrize("sinks", [0, 37])
def test_prompt_window_of_eight_waves(nh, nkv, hd, lens, window, sinks):
    """Windows and sequences above 1024 with heads of 64, above 512 with 128; every row."""
    say(f"eight waves nh={nh} nkv={nkv} hd={hd} lens={lens} window={window} sinks={sinks}")
    assert min(window, sum(lens) // len(lens)) > (1024 if hd == 64 else 512)
    g = np.random.default_rng(nh + hd + sum(lens))
    T = sum(lens)
    q, k, v = bits(g, T, nh, hd, std=2.0), bits(g, T, nkv, hd), bits(g, T, nkv, hd)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    out, lse = run_prompt(q, k, v, cu, window, sinks)
    r = check_rows(out, lse, oa.prompt(q, k, v, cu, True, hd ** -0.5, window, sinks), hd, "eight waves")
    say(f"  worst error at {r:.2f} of its bound")
    assert torch.equal(out, run_prompt(q, k, v, cu, window, sinks, lse=False)[0])


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_prompt_every_place_of_a_window(hd):
    g = np.random.default_rng(hd)
    for d in range(0, 70, 7):
        n, window, sinks = 190 + d, 60 + d, (3 * d) % 71
        q, k, v = bits(g, n, 2, hd, std=2.0), bits(g, n, 1, hd), bits(g, n, 1, hd)
        cu = np.array([0, n], np.int32)
        out, lse = run_prompt(q, k, v, cu, window, sinks)
        check_rows(out, lse, oa.prompt(q, k, v, cu, True, hd ** -0.5, window, sinks), hd, f"offset {d}")


def test_prompt_window_long_rows():
    """A sequence of many tiles of every kind; some of its rows are checked."""
    g = np.random.default_rng(7)
    n, nh, nkv, hd, window, sinks = 5000, 4, 1, 128, 1500, 100
    q, k, v = bits(g, n, nh, hd, std=2.0), bits(g, n, nkv, hd), bits(g, n, nkv, hd)
    for lead in ([], [40] * 20):                  # eight waves; four
        cu = np.concatenate([[0], np.cumsum(lead + [n])]).astype(np.int32)
        m = int(cu[-1]) - n
        pad = [bits(g, m, h, hd) for h in (nh, nkv, nkv)]
        out, lse = run_prompt(*(np.concatenate([p, x]) for p, x in zip(pad, (q, k, v))), cu, window, sinks)
        rows = np.array([0, 99, 100, 1499, 1500, 1600, 1601, 3333, 4096, 4999])
        for t in rows:
            seen = np.flatnonzero((np.arange(t + 1) > t - window) | (np.arange(t + 1) < sinks))
            r = oa.paged(q[t:t + 1], k[seen], v[seen], np.arange(len(seen))[None], [len(seen)], [0, 1], 1, True, hd ** -0.5)
            check_rows(out[m + t:m + t + 1], lse[m + t:m + t + 1], r, hd, f"row {t}")


def test_prompt_window_unseen_tokens_do_not_matter():
    g = np.random.default_rng(12)
    n, window, sinks = 200, 50, 3
    for hd in (64, 128, 256):
        q, k, v = bits(g, n, 4, hd, std=2.0), bits(g, n, 2, hd), bits(g, n, 2, hd)
        cu = np.array([0, n], np.int32)
        bad = 77                                  # seen by the rows 77 .. 126
        k[bad], v[bad] = INF, NAN
        out, lse = run_prompt(q, k, v, cu, window, sinks)
        sees = (np.arange(n) >= bad) & (np.arange(n) < bad + window)
        assert np.isnan(value(out)[sees]).all(), hd
        w = oa.prompt(q, k, v, cu, True, hd ** -0.5, window, sinks)
        w["written"] &= ~sees
        check_rows(out, lse, w, hd, str(hd))
        v[:] = bits(g, n, 2, hd)
        v[bad] = INF                              # a value alone, its key finite
        k[bad] = bits(g, 2, hd)
        out, _ = run_prompt(q, k, v, cu, window, sinks)
        a = value(out)
        assert not np.isfinite(a[sees]).any() and np.isfinite(a[~sees]).all(), hd


@pytest.mark.parametrize("hd,n,window", [(64, 2300, 1300), (128, 1700, 700), (256, 400, 150)])
def test_prompt_window_unseen_tokens_of_long_windows(hd, n, window):
    """The same where eight waves share a workgroup, at the edges of a row's window and its sinks."""
    g = np.random.default_rng(hd)
    sinks, at = 20, (5, 19, 20, 900 if n > 900 else 200)
    q, k, v = bits(g, n, 4, hd, std=2.0), bits(g, n, 1, hd), bits(g, n, 1, hd)
    for bad in at:
        k1, v1 = k.copy(), v.copy()
        k1[bad], v1[bad] = NAN, INF
        out, lse = run_prompt(q, k1, v1, np.array([0, n], np.int32), window, sinks)
        rows = sorted({bad - 1, bad, bad + 1, bad + window - 1, bad + window, bad + window + 1, n - 1})
        for t in (t for t in rows if 0 <= t < n):
            seen = np.flatnonzero((np.arange(t + 1) > t - window) | (np.arange(t + 1) < sinks))
            if bad in seen:
                assert np.isnan(value(out)[t]).all(), (bad, t)
            else:
                r = oa.paged(q[t:t + 1], k[seen], v[seen], np.arange(len(seen))[None], [len(seen)], [0, 1], 1, True, hd ** -0.5)
                check_rows(out[t:t + 1], lse[t:t + 1], r, hd, f"{bad} {t}")


def test_windows_read_column_ranges():
    """q, k and v as column ranges of one product, under a window; both forms."""
    g = np.random.default_rng(21)
    n, nh, nkv, hd = 150, 8, 2, 128
    q, k, v = bits(g, n, nh, hd, std=2.0), bits(g, n, nkv, hd), bits(g, n, nkv, hd)
    wide = dev(np.concatenate([x.reshape(n, -1) for x in (q, k, v)], 1))
    a, b = nh * hd, nkv * hd
    dq, dk, dv = (wide[:, lo:hi].unflatten(1, (-1, hd)) for lo, hi in ((0, a), (a, a + b), (a + b, a + 2 * b)))
    cu = dev(np.array([0, 100, n], np.int32))
    want = dsl.prompt_attention(dev(q), dev(k), dev(v), cu, window=30, sinks=2)
    assert torch.equal(dsl.prompt_attention(dq, dk, dv, cu, window=30, sinks=2), want)
    table, kv, cq = dev(np.arange(n, dtype=np.int32)[None]), dev(np.array([n], np.int32)), dev(np.array([0, 9], np.int32))
    want = dsl.paged_attention(dev(q[-9:]), dev(k), dev(v), table, kv, cq, 9, 1, window=30, sinks=2)
    assert torch.equal(dsl.paged_attention(dq[-9:], dev(k), dev(v), table, kv, cq, 9, 1, window=30, sinks=2), want)


def test_windows_in_a_graph_follow_the_lengths():
    """A captured paged call under a window, replayed as the cache grows past it."""
    g = np.random.default_rng(13)
    B, page, window, sinks = 3, 16, 100, 4
    c = paged_case(g, 8, 2, 128, page, [2] * B, [400] * B)
    args = [dev(c[n]) for n in ("q", "kc", "vc", "table", "kv", "cu")]
    out = torch.empty_like(args[0])
    ws = torch.empty(dsl.paged_attention_workspace_size(2 * B, B, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    call = lambda o: dsl.paged_attention(*args, 2, page, out=o, window=window, sinks=sinks, workspace=ws)  # noqa: E731
    call(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for kv in ([2, 50, 104], [105, 399, 400], [120, 0, 333]):
        args[4].copy_(torch.tensor(kv, dtype=torch.int32))
        graph.replay()
        got = out.clone()
        eager = torch.empty_like(out)
        call(eager)
        assert torch.equal(got, eager)
        c["kv"] = np.array(kv, np.int32)
        check_rows(got, None, ref(c, True, window, sinks), 128, str(kv))


def test_refusals():
    x, i = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    t = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for kw in (dict(sinks=4), dict(window=0), dict(window=-2 ** 40), dict(window=4, sinks=-1)):
        with pytest.raises((ValueError, dsl.DSparkError)):
            dsl.paged_attention(x, x, x, t, i[:1], i, 2, 1, **kw)
        with pytest.raises((ValueError, dsl.DSparkError)):
            dsl.prompt_attention(x, x, x, i, **kw)
    with pytest.raises(ValueError, match="causal"):
        dsl.prompt_attention(x, x, x, i, causal=False, window=4)
