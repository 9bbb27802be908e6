"""dspark_kv_append, dspark_paged_attention and dspark_prompt_attention against the oracle
(oracle/attention.py, float64).

Bounds.  A rounding to bf16 is off by at most 2^-8 of the value.
  * append: one such rounding of the output, and float32 work of a few tens of operations
    on the pair (x, y): |err| <= 2^-8 |ref| + 2^-18 sqrt(x^2 + y^2).
  * attention: the output's rounding, 2^-8 |ref|; the weights' rounding: with weights
    p (1 + d), |d| <= 2^-8, in the numerator and in the sum that divides it, the row is off
    by |sum p d v - ref sum p d| / sum p (1 + d) <= 2^-8 (A + |ref|) / (1 - 2^-8), A = sum p|v|;
    and float32 errors, each relative to A: a score of magnitude at most
    D = max scale sum|q||k| is off by e_s <= (hd + 4) 2^-24 D (accumulation and scaling)
    and moves a weight by e_s, its exponential by 2^-22 (argument and hardware rounding,
    up to 2^-23 of the argument's magnitude 2 D log2 e), numerator and denominator both; the sums
    over n keys are off by n 2^-24 each.  Together
        |err| <= 2^-8 |ref| + (2^-8 |ref| + A (2^-8 + 2 e_s + 2^-20 (1 + D) + 2 n 2^-24)) (1 + 2^-6),
    the last factor over (1 + 2^-8) / (1 - 2^-8): the output's rounding of the other errors.
  * lse: e_s + 2^-21 (1 + D) + n 2^-24 + 2^-22 |ref|.
"""
import numpy as np
import pytest
import torch

import draft_sampling_lossless_amd as dsl
import synth
from oracle import attention as oa
from oracle import context_kv as ck

from gpu_util import dev, host, say

pytestmark = pytest.mark.gpu

NAN = 0x7FC0
INF = 0x7F80
SENT = 0x7E7E


@pytest.fixture(scope="module", autouse=True)
def _gpu(dspark_lib):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def bits(g, *shape, std=1.0):
    return synth.bf16_bits(g.normal(0, std, shape).astype(np.float32))


def value(t):
    return ck.bf16_decode(host(t).view(np.uint16))


def check_rows(out, lse, ref, hd, label=""):
    """GPU out [T, nh, hd] (bits) and lse against the oracle's rows, row for row."""
    w = ref["written"]
    got = value(out)[w]
    want, mag, dot = ref["out"][w], ref["mag"][w], ref["dot"][w]
    n = ref["keys"][w][:, None]
    es = (hd + 4) * 2.0 ** -24 * dot
    rel = 2.0 ** -8 + 2 * es + 2.0 ** -20 * (1 + dot) + 2 * n * 2.0 ** -24
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 * np.abs(want) + mag * rel[..., None]) * (1 + 2.0 ** -6)
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.size} outside the bound, first at "
                           f"{tuple(np.argwhere(bad)[0])}: {got[bad][0]} vs {want[bad][0]} (bound {tol[bad][0]:.3g})")
    if lse is not None:
        a, b = host(lse).astype(np.float64)[w], ref["lse"][w]
        none = np.isneginf(b)
        assert np.array_equal(none, np.isneginf(a)), f"{label}: rows without keys"
        ltol = es + 2.0 ** -21 * (1 + dot) + n * 2.0 ** -24 + 2.0 ** -22 * np.where(none, 0, np.abs(b))
        assert np.all(np.abs(a[~none] - b[~none]) <= ltol[~none]), f"{label}: lse"
    return float((err / np.maximum(tol, 1e-300)).max()) if err.size else 0.0


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("M,nh,nkv,hd,norm,fused,kout", [
    (1, 1, 1, 128, True, False, False),
    (9, 32, 8, 128, True, True, True),
    (37, 20, 4, 128, False, True, False),
    (5, 16, 2, 64, True, False, True),
    (3, 8, 2, 256, True, True, True),
    (4, 3, 3, 32, False, False, False),
    (301, 0, 8, 128, True, True, False),      # keys and values only
    (2, 40, 40, 256, True, True, True),       # more heads than one pass of a workgroup
])
def test_append(M, nh, nkv, hd, norm, fused, kout):
    say(f"append M={M} nh={nh} nkv={nkv} hd={hd} norm={norm} fused={fused} k_out={kout}")
    g = np.random.default_rng(M + hd)
    S, eps, theta = M + 5, 1e-6, 1e6
    q, k, v = bits(g, M, max(nh, 1), hd), bits(g, M, nkv, hd), bits(g, M, nkv, hd)
    qw = synth.bf16_bits((1 + 0.1 * g.normal(size=hd)).astype(np.float32)) if norm else None
    kw = synth.bf16_bits((1 + 0.1 * g.normal(size=hd)).astype(np.float32)) if norm else None
    pos = g.integers(0, 1 << 20, M).astype(np.int32)
    pos[0] = 0 if M > 1 else 2 ** 31 - 1
    slots = g.permutation(S)[:M].astype(np.int64)
    kc = torch.full((S, nkv, hd), SENT, dtype=torch.int16, device="cuda")
    vc = torch.full((S, nkv, hd), SENT, dtype=torch.int16, device="cuda")
    if fused:
        wide = dev(np.concatenate([x.reshape(M, -1) for x in (q, k, v)], 1))
        a, b = q.shape[1] * hd, nkv * hd
        dq, dk, dv = (wide[:, lo:hi].unflatten(1, (-1, hd)) for lo, hi in ((0, a), (a, a + b), (a + b, a + 2 * b)))
    else:
        dq, dk, dv = dev(q), dev(k), dev(v)
    ko = torch.full((M, nkv, hd), SENT, dtype=torch.int16, device="cuda") if kout else None
    qo = dsl.kv_append(dk, dv, dev(pos), dev(slots), kc, vc, q=dq if nh else None,
                       qnorm_w=dev(qw) if norm and nh else None, knorm_w=dev(kw) if norm else None, k_out=ko,
                       eps=eps, rope_theta=theta)

    def check(t, x, w, label):
        ref = oa.append(x, w, pos, eps, theta)
        pair = np.hypot(ref[..., :hd // 2], ref[..., hd // 2:])
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * np.concatenate([pair, pair], -1)
        assert np.all(np.abs(value(t) - ref) <= tol), label

    if nh:
        check(qo, q, qw, "q")
    else:
        assert qo is None
    check(kc[dev(slots)], k, kw, "k")
    assert np.array_equal(host(vc).view(np.uint16)[slots], v)
    rest = np.setdiff1d(np.arange(S), slots)
    assert np.all(host(kc)[rest] == SENT) and np.all(host(vc)[rest] == SENT)
    if kout:
        assert torch.equal(ko, kc[dev(slots)])


def test_append_in_place_and_skipped_slots():
    g = np.random.default_rng(1)
    M, nh, nkv, hd, S = 12, 8, 2, 128, 40
    q, k, v = bits(g, M, nh, hd), bits(g, M, nkv, hd), bits(g, M, nkv, hd)
    pos = dev(np.arange(100, 100 + M, dtype=np.int32))
    slots = np.arange(M, dtype=np.int64) * 3
    slots[[0, 4, 11]] = [-1, S, 1 << 40]
    out = []
    for place in (False, True):
        kc = torch.full((S, nkv, hd), SENT, dtype=torch.int16, device="cuda")
        vc = torch.full((S, nkv, hd), SENT, dtype=torch.int16, device="cuda")
        wide = dev(np.concatenate([x.reshape(M, -1) for x in (q, k, v)], 1))
        dq, dk, dv = (wide[:, lo:hi].unflatten(1, (-1, hd))
                      for lo, hi in ((0, nh * hd), (nh * hd, (nh + nkv) * hd), ((nh + nkv) * hd, (nh + 2 * nkv) * hd)))
        qo = dq if place else torch.empty((M, nh, hd), dtype=torch.int16, device="cuda")
        ko = dk if place else torch.empty((M, nkv, hd), dtype=torch.int16, device="cuda")
        dsl.kv_append(dk, dv, pos, dev(slots), kc, vc, q=dq, q_out=qo, k_out=ko)
        assert np.array_equal(host(dv).view(np.uint16), v)
        out.append([host(x).copy() for x in (qo, ko, kc, vc)])
    for a, b in zip(*out):
        assert np.array_equal(a, b)
    good = np.array([m for m in range(M) if 0 <= slots[m] < S])
    assert np.all(out[0][2][np.setdiff1d(np.arange(S), slots[good])] == SENT)
    assert np.array_equal(out[0][2][slots[good]], out[0][1][good])
    assert not np.any(np.all(out[0][0] == q.view(np.int16), axis=(1, 2)))     # skipped tokens' q is rotated too


# ---------------------------------------------------------------- paged attention

def paged_case(g, nh, nkv, hd, page, qlen, kvlen, extra_pages=3, std=2.0, poison=True):
    """Caches whose unused slots hold NaN, tables whose unused entries are -1."""
    need = [-(-n // page) for n in kvlen]
    total = sum(need) + extra_pages
    order = g.permutation(total)
    table = np.full((len(kvlen), max(max(need), 1)), -1, np.int32)
    kc = np.full((total * page, nkv, hd), NAN if poison else 0, np.uint16)
    vc = np.full((total * page, nkv, hd), NAN if poison else 0, np.uint16)
    at = 0
    for b, n in enumerate(kvlen):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        slot = table[b, np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
        kc[slot], vc[slot] = bits(g, n, nkv, hd), bits(g, n, nkv, hd)
    cu = np.concatenate([[0], np.cumsum(qlen)]).astype(np.int32)
    return dict(q=bits(g, int(cu[-1]), nh, hd, std=std), kc=kc, vc=vc, table=table, kv=np.array(kvlen, np.int32), cu=cu,
                page=page, hd=hd, max_q=max(max(qlen), 1))


def run_paged(c, causal, scale=None, lse=True, max_q=None, **kw):
    T, nh, hd = c["q"].shape
    out = torch.full((T, nh, hd), SENT, dtype=torch.int16, device="cuda")
    ls = torch.full((T, nh), 7.0, dtype=torch.float32, device="cuda") if lse else None
    dsl.paged_attention(dev(c["q"]), dev(c["kc"]), dev(c["vc"]), dev(c["table"]), dev(c["kv"]), dev(c["cu"]),
                        max_q or c["max_q"], c["page"], causal=causal, scale=scale, out=out, lse=ls, **kw)
    return out, ls


def ref_paged(c, causal, scale=None):
    return oa.paged(c["q"], c["kc"], c["vc"], c["table"], c["kv"], c["cu"], c["page"], causal,
                    c["hd"] ** -0.5 if scale is None else scale)


@pytest.mark.parametrize("nh,nkv,hd,page,qlen,kvlen,causal", [
    (4, 1, 128, 16, [1], [1], True),
    (32, 8, 128, 16, [1], [517], True),
    (8, 2, 128, 64, [1], [5003], True),                       # split over ranges and joined
    (8, 2, 128, 1, [3], [3001], True),                        # slots one by one, split
    (4, 2, 64, 16, [1, 1, 1], [33, 1, 64], True),
    (4, 2, 256, 32, [2, 1], [95, 700], True),
    (8, 1, 256, 8, [5, 3], [40, 9], False),
    (10, 2, 128, 4, [1, 2, 3], [31, 32, 33], True),           # groups of 5
    (16, 1, 128, 16, [17, 1, 9], [300, 5, 9], True),          # 272 rows: several row blocks
    (8, 8, 128, 256, [4, 16], [255, 257], False),             # no shared heads
    (32, 8, 128, 64, [17, 3, 1, 9], [1000, 700, 17, 64], True),
    (6, 2, 64, 2, [7, 8], [7, 100], True),                    # query tokens are the whole sequence
    (8, 2, 64, 16, [128, 1], [200, 3], True),                 # the largest block
    (24, 8, 64, 32, [5, 0, 2], [50, 60, 1100], True),         # a request without query tokens
    (8, 2, 128, 16, [2, 1, 3], [0, 0, 2], True),              # nothing cached; fewer keys than query tokens
    (8, 2, 128, 16, [2, 1], [0, 40], False),
    (8, 1, 256, 16, [3], [150], True),                        # 24, 64 and 128 rows of 256
    (8, 1, 256, 1, [8, 2], [700, 65], True),
    (8, 1, 256, 32, [16, 16], [90, 300], True),
    (8, 1, 64, 16, [3], [150], True),                         # the same of 64
    (8, 1, 64, 1, [6, 2], [700, 65], False),
    (8, 1, 64, 32, [8, 8], [90, 300], True),
    (512, 1, 64, 16, [2], [70], True),                        # more heads on one than a row block
])
def test_paged(nh, nkv, hd, page, qlen, kvlen, causal):
    say(f"paged nh={nh} nkv={nkv} hd={hd} page={page} q={qlen} kv={kvlen} causal={causal}")
    c = paged_case(np.random.default_rng(nh + hd + page), nh, nkv, hd, page, qlen, kvlen)
    out, lse = run_paged(c, causal)
    r = check_rows(out, lse, ref_paged(c, causal), hd, "paged")
    say(f"  worst error at {r:.2f} of its bound")
    again, _ = run_paged(c, causal)
    assert torch.equal(out, again)


@pytest.mark.parametrize("B", [64, 65, 130, 1000])
def test_paged_many_requests(B):
    g = np.random.default_rng(B)
    qlen, kvlen = g.integers(0, 4, B).tolist(), g.integers(0, 60, B).tolist()
    kvlen[B // 2], kvlen[B - 1] = 2100, 1500              # two that are split among many that are not
    qlen[B // 2] = qlen[B - 1] = 2
    say(f"paged B={B}, {sum(qlen)} tokens")
    c = paged_case(g, 4, 2, 64, 16, qlen, kvlen)
    out, lse = run_paged(c, True)
    check_rows(out, lse, ref_paged(c, True), 64, "paged")


def test_paged_most_requests():
    """DSPARK_MAX_SEQS requests, most of one token over few keys, some of none, some long."""
    g = np.random.default_rng(41)
    B = 4096
    qlen, kvlen = (g.random(B) < 0.9).astype(int).tolist(), g.integers(0, 9, B).tolist()
    for b in (0, 1023, 1024, 4095):
        qlen[b], kvlen[b] = 2, 1500
    say(f"paged B={B}, {sum(qlen)} tokens")
    c = paged_case(g, 2, 1, 64, 4, qlen, kvlen)
    out, lse = run_paged(c, True)
    check_rows(out, lse, ref_paged(c, True), 64, "paged")


def test_paged_more_keys_than_a_window_of_slots():
    """70 requests of 20 rows over 2100 keys each, found slot by slot: a workgroup takes a
    request whole and looks its slots up in parts.  A value that is not finite in the last
    part is kept from the rows that do not see it, and the other tokens are checked."""
    g = np.random.default_rng(42)
    B, nh, nkv, hd, n, kv = 70, 32, 8, 64, 5, 2100
    S = B * kv
    say(f"paged B={B} kv={kv} slots")
    kc, vc = bits(g, S, nkv, hd), bits(g, S, nkv, hd)
    table = g.permutation(S).astype(np.int32).reshape(B, kv)
    c = dict(q=bits(g, B * n, nh, hd, std=2.0), kc=kc, vc=vc, table=table, kv=np.full(B, kv, np.int32),
             cu=(np.arange(B + 1) * n).astype(np.int32), page=1, hd=hd, max_q=n)
    table[7, 1500] = -1                                   # a key without a slot, in the second part
    kc[table[7, kv - 2]], vc[table[7, kv - 2]] = NAN, INF   # seen by the last two tokens of request 7
    out, lse = run_paged(c, True)
    for b in (0, 7, 69):
        d = dict(c, q=c["q"][b * n:(b + 1) * n], table=table[b:b + 1], kv=c["kv"][:1], cu=np.array([0, n], np.int32))
        ref, o, ls = ref_paged(d, True), out[b * n:(b + 1) * n], lse[b * n:(b + 1) * n]
        if b == 7:
            assert np.isnan(value(o)[n - 2:]).all()
            ref = {k: v[:n - 2] for k, v in ref.items()}
            o, ls = o[:n - 2], ls[:n - 2]
        check_rows(o, ls, ref, hd, f"request {b}")


@pytest.mark.parametrize("nh,nkv,hd,page,qlen,kvlen,causal", [
    (8, 2, 64, 16, [4, 1], [300, 70], True),
    (8, 2, 256, 1, [2, 1], [300, 900], False),
    (16, 2, 64, 1, [4, 1], [300, 70], True),
    (16, 2, 128, 32, [16, 2], [2000, 70], False),
    (16, 2, 256, 16, [7], [100], True),
])
def test_attention_without_lse_is_the_same(nh, nkv, hd, page, qlen, kvlen, causal):
    g = np.random.default_rng(43)
    c = paged_case(g, nh, nkv, hd, page, qlen, kvlen)
    assert torch.equal(run_paged(c, causal)[0], run_paged(c, causal, lse=False)[0])
    T = sum(kvlen)
    q, k, v = bits(g, T, nh, hd, std=2.0), bits(g, T, nkv, hd), bits(g, T, nkv, hd)
    cu = np.concatenate([[0], np.cumsum(kvlen)]).astype(np.int32)
    want, _ = run_prompt(q, k, v, cu, causal)
    assert torch.equal(dsl.prompt_attention(dev(q), dev(k), dev(v), dev(cu), causal=causal), want)


def test_paged_a_page_listed_twice():
    g = np.random.default_rng(44)
    for qlen in ([2], [6]):                               # both kernels
        c = paged_case(g, 8, 2, 128, 16, qlen, [100])
        c["table"][0, 3] = c["table"][0, 5] = c["table"][0, 0]
        out, lse = run_paged(c, True)
        check_rows(out, lse, ref_paged(c, True), 128, str(qlen))


def test_paged_two_calls_at_once():
    """Calls on two streams, each with its workspace, split and joined at the same time."""
    g = np.random.default_rng(45)
    cases = [paged_case(g, 8, 2, 128, 16, [1, 2], [3000, 900]), paged_case(g, 8, 2, 128, 1, [7, 6], [2500, 1700])]
    want = [run_paged(c, True)[0] for c in cases]
    args = [[dev(c[k]) for k in ("q", "kc", "vc", "table", "kv", "cu")] for c in cases]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, a, o, s in zip(cases, args, outs, streams):
            with torch.cuda.stream(s):
                dsl.paged_attention(*a, c["max_q"], c["page"], out=o)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_paged_unseen_keys_do_not_matter():
    """NaN and infinities in keys and values that a row does not see: later tokens of the
    block (causal), hidden pages, the rest of a page."""
    g = np.random.default_rng(8)
    for page, kv in ((16, 45), (1, 45), (64, 700)):
        c = paged_case(g, 8, 2, 128, page, [6], [kv])
        clean, _ = run_paged(c, True)
        slot = lambda s: int(c["table"][0, s // page]) * page + s % page  # noqa: E731
        for s, kb, vb in ((kv - 1, NAN, NAN), (kv - 2, 0xFF80, INF), (kv - 3, INF, NAN)):
            c["kc"][slot(s)], c["vc"][slot(s)] = kb, vb
        out, _ = run_paged(c, True)
        assert torch.equal(out[:3], clean[:3]), f"page {page}"
        assert np.isnan(value(out)[5]).all()              # and the rows that see them are not spared


def test_paged_values_that_are_not_finite_reach_the_rows_that_see_them():
    g = np.random.default_rng(9)
    c = paged_case(g, 4, 1, 128, 16, [4], [40])
    slot = int(c["table"][0, 37 // 16]) * 16 + 37 % 16
    c["vc"][slot, 0, 5] = INF                             # seen by tokens 1, 2, 3 (keys <= 37, 38, 39), not by 0
    got = value(run_paged(c, True)[0])
    assert np.isposinf(got[1:, :, 5]).all() and np.isfinite(got[0]).all()
    assert np.isfinite(np.delete(got, 5, axis=2)).all()


@pytest.mark.parametrize("kv", [1500, 3001, 20001])     # a few ranges, and more than one group joins
@pytest.mark.parametrize("m", [1, 3, 12, 24])           # paged_rows; four and eight waves of shared tiles
def test_paged_nan_in_a_split_request(m, kv):
    """What is not finite reaches the rows that see it whichever range it lies in: in a
    query, in every key of a range, in one key or value of a range whose other scores lie so
    far below that its weight is zero in the join.  The other kv head's rows do not change."""
    say(f"paged NaN m={m} kv={kv}")
    g = np.random.default_rng(kv + m)
    nh, nkv, hd, page = 8, 2, 64, 16
    c = paged_case(g, nh, nkv, hd, page, [m], [kv])
    c["q"][:, :4] = synth.bf16_bits(np.full((m, 4, hd), 2.0, np.float32))
    slot = c["table"][0, np.arange(kv) // page].astype(np.int64) * page + np.arange(kv) % page
    clean, clean_lse = run_paged(c, True)
    check_rows(clean, clean_lse, ref_paged(c, True), hd, "clean")

    def check(d, label, rows, dims=slice(None)):
        out, lse = run_paged(d, True)
        bad = np.zeros((m, nh), bool)
        bad[rows] = True
        assert torch.equal(out[dev(~bad)], clean[dev(~bad)]) and torch.equal(lse[dev(~bad)], clean_lse[dev(~bad)]), label
        assert not np.isfinite(value(out)[bad][:, dims]).any(), label
        return value(out)[bad], host(lse)[bad]

    q = c["q"].copy()
    q[m - 1, 3, 5] = NAN
    out, lse = check(dict(c, q=q), "query", (m - 1, 3))
    assert np.isnan(out).all() and np.isnan(lse).all()
    mid = slot[kv // 4:3 * kv // 4]                       # holds whole ranges
    first = np.s_[:, :4]
    kc = c["kc"].copy()
    kc[mid, 0] = NAN
    out, lse = check(dict(c, kc=kc), "keys of a range", first)
    assert np.isnan(out).all() and np.isnan(lse).all()
    kc[mid, 0] = synth.bf16_bits(np.full((len(mid), hd), -8.0, np.float32))   # exponents 185 below 0
    low = dict(c, kc=kc)
    clean, clean_lse = run_paged(low, True)
    check_rows(clean, clean_lse, ref_paged(low, True), hd, "low")
    kc = kc.copy()
    kc[slot[kv // 2], 0, 7] = NAN
    out, lse = check(dict(c, kc=kc), "key of a low range", first)
    assert np.isnan(out).all() and np.isnan(lse).all()
    vc = c["vc"].copy()
    vc[slot[kv // 2], 0, 5] = INF
    out, lse = check(dict(low, vc=vc), "value of a low range", first, 5)
    want = value(clean)[:, :4].reshape(-1, hd)
    assert np.array_equal(np.delete(out, 5, 1), np.delete(want, 5, 1))
    assert np.array_equal(lse, host(clean_lse)[:, :4].reshape(-1))


def test_paged_pages_outside_the_cache_hide_their_keys():
    g = np.random.default_rng(10)
    for page in (1, 16, 64):
        c = paged_case(g, 8, 2, 128, page, [2, 1], [200, 90])
        pages = c["kc"].shape[0] // page
        c["table"][0, 0], c["table"][1, 1], c["table"][0, 2] = -1, pages, 2 ** 31 - 1
        out, lse = run_paged(c, True)
        check_rows(out, lse, ref_paged(c, True), 128, f"page {page}")
    c["table"][:] = -7                                    # every page
    out, lse = run_paged(c, True)
    assert not value(out).any() and np.isneginf(host(lse)).all()


@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_paged_pages_outside_the_cache_hide_their_keys_from_many_rows(page, hd):
    g = np.random.default_rng(46)
    c = paged_case(g, 8, 2, hd, page, [6, 5], [700, 90])
    pages = c["kc"].shape[0] // page
    for b, p, to in ((0, 0, -1), (0, 3, 2 ** 31 - 1), (1, 1, pages), (1, 0, -2 ** 31), (0, c["table"].shape[1] - 1, -1)):
        c["table"][b, p] = to
    out, lse = run_paged(c, True)
    check_rows(out, lse, ref_paged(c, True), hd)
    c["table"][0] = pages                                 # every page of one request
    out, lse = run_paged(c, True)
    check_rows(out, lse, ref_paged(c, True), hd)
    assert not value(out)[:6].any() and np.isneginf(host(lse)[:6]).all()


def test_paged_lengths_beyond_the_table_and_rows_behind():
    g = np.random.default_rng(11)
    c = paged_case(g, 8, 2, 128, 16, [2, 3], [64, 40])
    c["q"] = np.concatenate([c["q"], bits(g, 4, 8, 128)])        # four rows behind the last request
    c["kv"][0] = 1000                                            # the table holds 64 keys a request
    ref = ref_paged(c, False)
    out, lse = run_paged(c, False)
    check_rows(out, lse, ref, 128)
    assert np.all(host(out)[5:] == SENT) and np.all(host(lse)[5:] == 7.0)
    c["kv"][:] = -3
    out, _ = run_paged(c, False)
    assert not host(out)[:5].any()
    # tokens beyond max_q are left as they were
    c = paged_case(g, 8, 2, 128, 16, [5], [64])
    ref = ref_paged(c, True)
    out, _ = run_paged(c, True, max_q=2)
    assert np.all(host(out)[2:] == SENT)
    ref["written"][2:] = False
    check_rows(out, None, ref, 128)
    c = paged_case(g, 8, 2, 128, 16, [9, 7], [64, 900])          # more than 16 rows
    ref = ref_paged(c, True)
    out, _ = run_paged(c, True, max_q=6)
    for lo, hi in ((6, 9), (15, 16)):
        assert np.all(host(out)[lo:hi] == SENT)
        ref["written"][lo:hi] = False
    check_rows(out, None, ref, 128)


def test_paged_large_scores_and_scale():
    g = np.random.default_rng(12)
    c = paged_case(g, 8, 2, 128, 16, [3], [600], std=60.0)       # scores of hundreds: one weight is all
    out, lse = run_paged(c, True)
    check_rows(out, lse, ref_paged(c, True), 128)
    out, lse = run_paged(c, True, scale=0.003)
    check_rows(out, lse, ref_paged(c, True, 0.003), 128)


@pytest.mark.parametrize("std", [3e4, 1e6, 1e12])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_scores_beyond_any_exponent(hd, std):
    """Scores of 1e9 to 1e25: each row takes the value of its largest score.  Keys are
    multiples of one direction, so that the largest differs from the next by far more than
    float32 sums are off by."""
    g = np.random.default_rng(48)
    n, nh, nkv = 2100, 4, 2
    base = g.choice([-1.0, 1.0], (nkv, hd)) * g.uniform(0.5, 1.0, (nkv, hd))
    size = g.permutation(n) / n * 2 - 1                               # distinct multiples, -1 .. 1
    k = synth.bf16_bits((std * size[:, None, None] * base).astype(np.float32))
    q = synth.bf16_bits((std * g.choice([-1.0, 1.0], (n, nh, 1)) * np.repeat(base, nh // nkv, 0)).astype(np.float32))
    v = bits(g, n, nkv, hd)
    qd, kd, vd = ck.bf16_decode(q), ck.bf16_decode(k), ck.bf16_decode(v)

    def check(out, lse, rows, seen, label):
        got, ls = value(out), host(lse).astype(np.float64)
        checked = 0
        for i, t in enumerate(rows):
            for h in range(nh):
                x = (kd[:seen(t), h * nkv // nh] @ qd[t, h]) * hd ** -0.5
                order = np.argsort(x)
                if len(x) > 1 and x[order[-1]] - x[order[-2]] < 1e-4 * np.abs(x).max():
                    continue                          # (two keys rounded alike)
                checked += 1
                assert np.array_equal(got[i, h], vd[order[-1], h * nkv // nh]), f"{label} token {t} head {h}"
                # sums of hd products of one sign, the scaling, the change of base and back
                assert abs(ls[i, h] - x[order[-1]]) <= ((hd + 4) * 2.0 ** -24 + 2.0 ** -21) * np.abs(x[order[-1]])
        assert checked > len(rows)

    out, lse = run_prompt(q, k, v, [0, n], True)
    check(out[::37], lse[::37], range(0, n, 37), lambda t: t + 1, "prompt")
    table = g.permutation(n).astype(np.int32)
    kc, vc = np.zeros_like(k), np.zeros_like(v)
    kc[table], vc[table] = k, v
    for m in (2, 12):                                 # both kernels, split and joined
        c = dict(q=q[n - m:], kc=kc, vc=vc, table=table[None], kv=np.array([n], np.int32), cu=np.array([0, m], np.int32),
                 page=1, hd=hd, max_q=m)
        out, lse = run_paged(c, True)
        check(out, lse, range(n - m, n), lambda t: t + 1, f"paged {m}")


# Exact scores.  q = (2^16 u, 2^8 u, u, 0, ..) and k = the three 8-bit digits of an integer N,
# |N| < 2^24, with its sign: every product and every partial sum of q . k = N u is exact in
# float32, in any order, so the largest score of a row is known to the last bit.

def exact_scores(g, N, u, hd):
    """N [n, nkv] and u [nkv], powers of two -> q [nkv, hd] (the query of every token), k, v."""
    N = np.asarray(N, np.int64)
    k = np.zeros((*N.shape, hd), np.float32)
    q = np.zeros((N.shape[1], hd), np.float32)
    for i, shift in enumerate((16, 8, 0)):
        k[..., i] = np.sign(N) * ((np.abs(N) >> shift) & 255)
        q[:, i] = np.asarray(u, np.float64) * 2.0 ** shift
    assert np.array_equal((k.astype(np.float64) * q).sum(-1), N * np.asarray(u, np.float64)) and np.abs(N).max() < 1 << 24
    return synth.bf16_bits(q), synth.bf16_bits(k), bits(g, *N.shape, hd)


def check_winner(out, lse, N, u, v, rows, hd, label):
    """Each row is the value of its largest score: the other key lies 64 and more below it as
    an exponent of two and weighs at most 2^-32 of it (a weight may be up to 2^32 before the
    division), the filling nothing; dividing the value times its weight by that weight is off
    by 2^-22, and the value is a bf16.  rows: (row, keys it sees).
    lse: seven roundings of 2^-24 (the scale, its product with log2 e, the score's with that,
    the weight's logarithm added, the changes of base): 2^-21 of it."""
    got, ls = value(out), host(lse).astype(np.float64)
    vd, checked = ck.bf16_decode(v), 0
    for i, seen in rows:
        for h in range(N.shape[1]):
            x = N[:seen, h]
            best = int(np.argmax(x))
            if (x == x[best]).sum() > 1:
                continue                              # only keys of the filling
            checked += 1
            assert np.array_equal(got[i, h], vd[best, h]), f"{label} row {i} head {h}: {got[i, h, :3]} for key {best}"
            want = hd ** -0.5 * float(x[best]) * u[h]
            assert abs(ls[i, h] - want) <= 2.0 ** -21 * abs(want), f"{label} row {i} head {h}: lse"
    assert checked >= N.shape[1]


def run_exact(g, N, u, hd, label):
    """Both attentions on exact scores: prompts in both forms, few and many rows over pages and slots."""
    n, nkv = N.shape
    q1, k, v = exact_scores(g, N, u, hd)
    q = np.ascontiguousarray(np.broadcast_to(q1, (n, nkv, hd)))
    for causal in (True, False):
        out, lse = run_prompt(q, k, v, [0, n], causal)
        rows = [(t, t + 1 if causal else n) for t in range(0, n, 11)] + [(n - 1, n)]
        check_winner(out, lse, N, u, v, rows, hd, f"{label} prompt causal={causal}")
    for m in (1, 40, 80):                             # paged_rows; four and eight waves of shared tiles
        for page in (16, 1):
            pages = -(-n // page) + 2
            order = g.permutation(pages)[:-(-n // page)].astype(np.int32)
            slot = order[np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
            kc, vc = np.full((pages * page, nkv, hd), NAN, np.uint16), np.full((pages * page, nkv, hd), NAN, np.uint16)
            kc[slot], vc[slot] = k, v
            c = dict(q=q[:m], kc=kc, vc=vc, table=order[None], kv=np.array([n], np.int32),
                     cu=np.array([0, m], np.int32), page=page, hd=hd, max_q=m)
            out, lse = run_paged(c, False)
            check_winner(out, lse, N, u, v, [(t, n) for t in range(m)], hd, f"{label} paged {m} page {page}")


# where the two keys lie: one range and one wave's tiles, one tile apart, a range the other's
# neighbour, ends of a split request; and the larger one first
PLACES = [(400, 5, 263), (600, 5, 263), (600, 5, 40), (600, 263, 5), (2100, 5, 2000), (2100, 5, 261), (2100, 2000, 5)]


@pytest.mark.parametrize("n,first,second", PLACES)
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_maxima_on_both_sides_of_a_large_exponent(hd, n, first, second):
    """Two keys outweigh the others, one with an exponent a 2^30, the other, larger, with
    b 2^30: a row's maximum goes from below 2^30 in magnitude to above it or back, within a
    wave's tiles, between waves and between ranges."""
    say(f"maxima hd={hd} n={n} at {first}, {second}")
    pairs = [(0.8, 1.05), (0.95, 1.05), (0.999, 1.005), (0.72, 1.3), (-1.05, -0.99), (-1.005, -0.999), (-1.4, -0.75),
             (-1.2, 0.999)]
    per = 2.0 ** 30 / (hd ** -0.5 * np.log2(np.e))    # the score of an exponent of 2^30
    u = np.full(len(pairs), 2.0 ** np.ceil(np.log2(2.5 * per / (2 ** 24 - 1))))
    N = np.zeros((n, len(pairs)), np.int64)
    for h, (a, b) in enumerate(pairs):
        N[:, h] = 0 if a > 0 else round(-2.4 * per / u[h])
        N[first, h], N[second, h] = round(a * per / u[h]), round(b * per / u[h])
    run_exact(np.random.default_rng(hd + n), N, u, hd, f"hd {hd} n {n}")


@pytest.mark.parametrize("n,first,second", PLACES)
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_neighbouring_maxima_beyond_a_large_exponent(hd, n, first, second):
    """Two keys whose scores are neighbours in float32, with exponents beyond 2^30 in
    magnitude: 64 and more apart, so the larger one's value is the row's."""
    say(f"neighbours hd={hd} n={n} at {first}, {second}")
    per = 2.0 ** 30 / (hd ** -0.5 * np.log2(np.e))
    start = int(0.9 * 2 ** 24)
    u = np.full(16, 2.0 ** np.ceil(np.log2(per / start)))
    N = np.zeros((n, 16), np.int64)
    for h in range(16):
        at = start + 7 * (h // 2)
        if h % 2:
            N[:, h], N[first, h], N[second, h] = 1 - 2 ** 24, -at - 1, -at
        else:
            N[first, h], N[second, h] = at, at + 1
    run_exact(np.random.default_rng(hd + n), N, u, hd, f"hd {hd} n {n}")


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_values_up_to_the_stated_size_stay_finite(hd):
    """Maxima of 2^27 to 2^30 in magnitude, as exponents, leave weights of up to 2^32 before the
    division; values up to 2^95 over the number of keys, here 2^86, stay finite."""
    n, nkv = 400, 16
    per = 2.0 ** 30 / (hd ** -0.5 * np.log2(np.e))
    g = np.random.default_rng(hd)
    u = np.full(nkv, 2.0 ** np.ceil(np.log2(per / (2 ** 24 - 1))))
    N = np.zeros((n, nkv), np.int64)
    for h in range(nkv):
        top = int(per * g.uniform(0.125, 0.999) / u[h])
        N[:, h] = top if h % 2 else -top
    q1, k, _ = exact_scores(g, N, u, hd)
    q = np.ascontiguousarray(np.broadcast_to(q1, (n, nkv, hd)))
    v = synth.bf16_bits((2.0 ** 86 * g.choice([-1.0, 1.0], (n, nkv, hd))).astype(np.float32))
    order = np.arange(n // 16, dtype=np.int32)
    for m in (1, 40, n):
        if m == n:
            out, _ = run_prompt(q, k, v, [0, n], False)
        else:
            out, _ = run_paged(dict(q=q[:m], kc=k, vc=v, table=order[None], kv=np.array([n], np.int32),
                                    cu=np.array([0, m], np.int32), page=16, hd=hd, max_q=m), False)
        # equal scores: the mean of the values, whose weights are equal and so their roundings too;
        # the sums of n terms are off by n 2^-24 of n 2^86 each, the output's rounding by 2^-8
        want = ck.bf16_decode(v).mean(0)
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** 86 * (2 * n + 8) * 2.0 ** -24
        assert np.all(np.abs(value(out) - want) <= tol), f"{m} rows"


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_rows_whose_every_score_is_minus_infinity(hd):
    """They get zeros and a log-sum-exp of -inf, as rows without keys do, cut into ranges or
    not; a score among them that is not a number reaches the row."""
    g = np.random.default_rng(hd)
    for n in (90, 2100):
        q, k, v = bits(g, n, 4, hd), bits(g, n, 2, hd), bits(g, n, 2, hd)
        k[:, :, 0] = synth.bf16_bits(np.abs(g.normal(1, 0.2, (n, 2))).astype(np.float32) + np.float32(0.1))
        q[:, 1, 0] = 0xFF80
        k[40, 0, 0] = 0xFF80                              # (-inf)^2: the head's largest score
        order = np.arange(n, dtype=np.int32)

        def check(out, lse, rows):
            out, lse = value(out), host(lse)
            for i, seen in rows:
                if seen <= 40:
                    assert not out[i, 1].any() and np.isneginf(lse[i, 1]), f"n {n} row {i}"
                else:
                    assert np.isnan(out[i, 1]).all()      # an infinite maximum
                assert np.isfinite(out[i, 2:]).all() and np.isfinite(lse[i, 2:]).all()

        out, lse = run_prompt(q, k, v, [0, n], True)
        check(out, lse, [(t, t + 1) for t in range(0, n, 7)])
        k[40, 0, 0] = synth.bf16_bits(np.ones(1, np.float32))[0]
        for m in (2, 20, 40):
            c = dict(q=q[:m], kc=k, vc=v, table=order[None], kv=np.array([n], np.int32), cu=np.array([0, m], np.int32),
                     page=1, hd=hd, max_q=m)
            out, lse = run_paged(c, False)
            assert not value(out)[:, 1].any() and np.isneginf(host(lse)[:, 1]).all()
            assert value(out)[:, 0].any() and np.isfinite(value(out)).all()
            one = dict(c, kc=k.copy())
            one["kc"][n // 2, 0, 0] = 0                   # -inf * 0: NaN reaches the row
            out, lse = run_paged(one, False)
            assert np.isnan(value(out)[:, 1]).all() and np.isnan(host(lse)[:, 1]).all()
            assert np.isfinite(value(out)[:, [0, 2, 3]]).all()


def test_paged_offsets_beyond_32_bits():
    """A cache of 5 GiB a side, its last pages in use: slot offsets pass 2^32 bytes."""
    g = np.random.default_rng(13)
    nh, nkv, hd, page = 8, 8, 128, 16
    pages = 5 * 2 ** 30 // (page * nkv * hd * 2)
    small = paged_case(g, nh, nkv, hd, page, [2, 1], [100, 650], extra_pages=0)
    kc = torch.empty((pages * page, nkv, hd), dtype=torch.int16, device="cuda")
    vc = torch.empty((pages * page, nkv, hd), dtype=torch.int16, device="cuda")
    n = small["kc"].shape[0]
    kc[-n:], vc[-n:] = dev(small["kc"]), dev(small["vc"])
    for p in (16, 1):
        table = np.where(small["table"] >= 0, small["table"] + pages - n // page, -1).astype(np.int32)
        if p == 1:
            table = np.where(np.repeat(table, 16, 1) >= 0, np.repeat(table, 16, 1) * 16 + np.tile(np.arange(16), table.shape[1]),
                             -1).astype(np.int32)
        out = dsl.paged_attention(dev(small["q"]), kc, vc, dev(table), dev(small["kv"]), dev(small["cu"]), 2, p)
        check_rows(out, None, ref_paged(small, True), hd, f"page {p}")
    # the append reaches the last slot too
    k, v = bits(g, 1, nkv, hd), bits(g, 1, nkv, hd)
    dsl.kv_append(dev(k), dev(v), dev(np.zeros(1, np.int32)), dev(np.array([pages * page - 1])), kc, vc)
    assert np.array_equal(host(kc[-1]).view(np.uint16), k[0]) and np.array_equal(host(vc[-1]).view(np.uint16), v[0])


def test_paged_parts_join_by_their_lse():
    g = np.random.default_rng(14)
    c = paged_case(g, 8, 2, 128, 16, [4], [320])
    whole, _ = run_paged(c, False)
    parts = []
    for lo, hi in ((0, 8), (8, 20)):
        d = dict(c, table=np.ascontiguousarray(c["table"][:, lo:hi]), kv=np.array([(hi - lo) * 16], np.int32))
        out, lse = run_paged(d, False)
        parts.append((value(out), host(lse).astype(np.float64)))
    both = np.logaddexp(parts[0][1], parts[1][1])
    joined = sum(o * np.exp(l - both)[..., None] for o, l in parts)
    ref = ref_paged(c, False)
    # each part is within the bound of its own rows; the weighted sum is within theirs together
    tol = 2.0 ** -7 * 2 * ref["mag"] + 1e-4
    assert np.all(np.abs(joined - value(whole)) <= tol)


def test_paged_strided_queries_streams_and_graph():
    g = np.random.default_rng(15)
    c = paged_case(g, 8, 2, 128, 16, [2, 1, 3], [700, 64, 1300])
    want, _ = run_paged(c, True)
    T = c["q"].shape[0]
    wide = torch.zeros((T, 8 * 128 + 512), dtype=torch.int16, device="cuda")
    wide[:, :1024] = dev(c["q"]).view(T, -1)
    q = wide[:, :1024].unflatten(1, (8, 128))
    kc, vc, tb, kv, cu = dev(c["kc"]), dev(c["vc"]), dev(c["table"]), dev(c["kv"]), dev(c["cu"])
    ws = torch.empty(dsl.paged_attention_workspace_size(T, 3, 3, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty((T, 8, 128), dtype=torch.int16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        dsl.paged_attention(q, kc, vc, tb, kv, cu, 3, 16, out=out, workspace=ws)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsl.paged_attention(q, kc, vc, tb, kv, cu, 3, 16, out=out, workspace=ws)
    for kvs in ([700, 64, 1300], [10, 70, 1200], [640, 1, 3]):           # lengths change between replays
        kv.copy_(dev(np.array(kvs, np.int32)))
        out.fill_(SENT)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        d = dict(c, kv=np.array(kvs, np.int32))
        assert torch.equal(out, run_paged(d, True)[0])


def test_paged_block_captured_and_replayed():
    """More than 16 rows, planned and joined on the device: lengths, pages and counts of
    query tokens change between replays, and the program's own calls run in between."""
    g = np.random.default_rng(47)
    c = paged_case(g, 8, 2, 64, 1, [9, 9, 9], [1400, 600, 1100])
    a = [dev(c[k]) for k in ("q", "kc", "vc", "table", "kv", "cu")]
    out = torch.empty((27, 8, 64), dtype=torch.int16, device="cuda")
    ws = torch.empty(dsl.paged_attention_workspace_size(27, 3, 9, 8, 2, 64), dtype=torch.uint8, device="cuda")
    dsl.paged_attention(*a, 9, 1, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsl.paged_attention(*a, 9, 1, out=out, workspace=ws)
    for kv, cu in (([1400, 600, 1100], [0, 9, 18, 27]), ([9, 600, 3], [0, 5, 5, 14]), ([0, 33, 1100], [0, 1, 9, 18]),
                   ([1400, 600, 1100], [0, 9, 18, 27])):
        d = dict(c, kv=np.array(kv, np.int32), cu=np.array(cu, np.int32))
        d["table"] = np.ascontiguousarray(c["table"][:, ::-1]) if kv[0] == 9 else c["table"]
        for t, x in zip(a[3:], (d["table"], d["kv"], d["cu"])):
            t.copy_(dev(x))
        out.fill_(SENT)
        want, _ = run_paged(d, True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# ---------------------------------------------------------------- prompt attention

def run_prompt(q, k, v, cu, causal, scale=None):
    T, nh, hd = q.shape
    out = torch.full((T, nh, hd), SENT, dtype=torch.int16, device="cuda")
    lse = torch.full((T, nh), 7.0, dtype=torch.float32, device="cuda")
    dsl.prompt_attention(dev(q), dev(k), dev(v), dev(np.array(cu, np.int32)), causal=causal, scale=scale, out=out, lse=lse)
    return out, lse


@pytest.mark.parametrize("nh,nkv,hd,lens", [
    (4, 1, 128, [1]),
    (8, 2, 128, [63, 64, 65]),
    (8, 8, 128, [130, 1, 200]),
    (32, 8, 128, [17, 90]),
    (10, 2, 128, [5, 0, 77, 2]),            # groups of 5, an empty sequence
    (16, 1, 128, [33, 40]),
    (4, 2, 64, [300]),
    (6, 2, 64, [1, 2, 3, 129]),
    (4, 2, 256, [150, 31]),
    (2, 2, 256, [65]),
    (4, 2, 128, [700]),                     # several key tiles and row tiles
    (512, 1, 64, [2, 3]),                   # a token's heads are more than a row tile
    (4, 2, 64, [1300, 901]),                # long sequences of small heads
])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt(nh, nkv, hd, lens, causal):
    say(f"prompt nh={nh} nkv={nkv} hd={hd} lens={lens} causal={causal}")
    g = np.random.default_rng(nh + hd + len(lens))
    T = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = bits(g, T + 3, nh, hd, std=2.0), bits(g, T + 3, nkv, hd), bits(g, T + 3, nkv, hd)
    k[T:], v[T:] = NAN, NAN                 # tokens behind the last sequence
    out, lse = run_prompt(q, k, v, cu, causal)
    ref = oa.prompt(q, k, v, cu, causal, hd ** -0.5)
    r = check_rows(out, lse, ref, hd, "prompt")
    say(f"  worst error at {r:.2f} of its bound")
    assert np.all(host(out)[T:] == SENT) and np.all(host(lse)[T:] == 7.0)
    assert torch.equal(out, run_prompt(q, k, v, cu, causal)[0])


@pytest.mark.parametrize("B", [64, 65, 200])
def test_prompt_many_sequences(B):
    g = np.random.default_rng(B)
    lens = g.integers(0, 12, B)
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    q, k, v = bits(g, T, 8, 64, std=2.0), bits(g, T, 2, 64), bits(g, T, 2, 64)
    out, lse = run_prompt(q, k, v, cu, True)
    check_rows(out, lse, oa.prompt(q, k, v, cu, True, 64 ** -0.5), 64, "prompt")


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_most_sequences(causal):
    """DSPARK_MAX_SEQS sequences, most of a token or none, the last ones longer."""
    g = np.random.default_rng(26)
    lens = g.integers(0, 3, 4096)
    lens[4094:] = 70, 33
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    q, k, v = bits(g, T, 2, 64, std=2.0), bits(g, T, 1, 64), bits(g, T, 1, 64)
    out, lse = run_prompt(q, k, v, cu, causal)
    check_rows(out, lse, oa.prompt(q, k, v, cu, causal, 64 ** -0.5), 64, "prompt")


def test_prompt_unseen_keys_do_not_matter():
    g = np.random.default_rng(21)
    for hd, lens in ((128, [100, 150]), (64, [70, 80]), (256, [90])):
        T = sum(lens)
        cu = np.concatenate([[0], np.cumsum(lens)])
        q, k, v = bits(g, T, 8, hd, std=2.0), bits(g, T, 2, hd), bits(g, T, 2, hd)
        clean, _ = run_prompt(q, k, v, cu, True)
        at = lens[0] - 40                    # in the first sequence: tokens before it, and all others, are untouched
        k[at], v[at] = NAN, NAN
        k[at + 2], v[at + 2] = INF, 0xFF80
        out, _ = run_prompt(q, k, v, cu, True)
        assert torch.equal(out[:at], clean[:at]) and torch.equal(out[lens[0]:], clean[lens[0]:]), f"hd {hd}"
        assert np.isnan(value(out)[at:lens[0]]).all()
        full, _ = run_prompt(q, k, v, cu, False)
        assert np.isnan(value(full)[:lens[0]]).all() and np.isfinite(value(full)[lens[0]:]).all()


def test_prompt_unseen_keys_with_large_scores():
    """A key that outweighs all others by far, in tiles that some rows see only in part or
    not at all: rows before it are what they are without it."""
    g = np.random.default_rng(24)
    for hd in (64, 128, 256):
        T = 200
        q, k, v = bits(g, T, 4, hd, std=2.0), bits(g, T, 2, hd), bits(g, T, 2, hd)
        clean, _ = run_prompt(q, k, v, [0, T], True)
        for at in (40, 63, 64, 100, 130, 199):
            big = k.copy()
            big[at] = synth.bf16_bits((100 * ck.bf16_decode(q[at - 1, :2])).astype(np.float32))
            out, lse = run_prompt(q, big, v, [0, T], True)
            assert torch.equal(out[:at], clean[:at]), f"hd {hd} key {at}"
            ref = oa.prompt(q, big, v, [0, T], True, hd ** -0.5)
            check_rows(out, lse, ref, hd, f"hd {hd} key {at}")


@pytest.mark.parametrize("hd,lens", [(64, [1150, 1100]), (128, [700, 601])])
def test_prompt_unseen_keys_of_long_sequences(hd, lens):
    """The two tests before, at lengths where eight waves work on a tile."""
    g = np.random.default_rng(25)
    T = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = bits(g, T, 4, hd, std=2.0), bits(g, T, 2, hd), bits(g, T, 2, hd)
    clean, _ = run_prompt(q, k, v, cu, True)
    for at in (300, 511, 512, lens[0] - 40, lens[0] - 1):
        big = k.copy()
        big[at] = synth.bf16_bits((100 * ck.bf16_decode(q[at - 1, :2])).astype(np.float32))
        out, _ = run_prompt(q, big, v, cu, True)
        assert torch.equal(out[:at], clean[:at]) and torch.equal(out[lens[0]:], clean[lens[0]:]), f"key {at}"
        bad = v.copy()
        big[at], bad[at] = NAN, INF
        out, _ = run_prompt(q, big, bad, cu, True)
        assert torch.equal(out[:at], clean[:at]) and torch.equal(out[lens[0]:], clean[lens[0]:]), f"key {at}"
        assert np.isnan(value(out)[at:lens[0]]).all()
        bad = v.copy()
        bad[at, 0, 3] = INF
        out, _ = run_prompt(q, k, bad, cu, True)
        assert torch.equal(out[:at], clean[:at]) and torch.equal(out[lens[0]:], clean[lens[0]:]), f"value {at}"
        assert np.isposinf(value(out)[at:lens[0], :2, 3]).all() and np.isfinite(value(out)[at:lens[0], 2:]).all()


def test_prompt_strided_columns_and_graph():
    g = np.random.default_rng(22)
    T, nh, nkv, hd = 260, 8, 2, 128
    q, k, v = bits(g, T, nh, hd, std=2.0), bits(g, T, nkv, hd), bits(g, T, nkv, hd)
    cu = dev(np.array([0, 100, 260], np.int32))
    want, _ = run_prompt(q, k, v, [0, 100, 260], True)
    wide = dev(np.concatenate([x.reshape(T, -1) for x in (q, k, v)], 1))
    a, b = nh * hd, nkv * hd
    dq, dk, dv = (wide[:, lo:hi].unflatten(1, (-1, hd)) for lo, hi in ((0, a), (a, a + b), (a + b, a + 2 * b)))
    out = torch.empty((T, nh, hd), dtype=torch.int16, device="cuda")
    dsl.prompt_attention(dq, dk, dv, cu, out=out)
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsl.prompt_attention(dq, dk, dv, cu, out=out)
    for mid in (100, 1, 260, 0):
        cu[1] = mid
        out.fill_(SENT)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run_prompt(q, k, v, [0, mid, 260], True)[0])


def test_prompt_long_rows_sampled():
    """4100 tokens: many key tiles; a sample of rows against the oracle."""
    g = np.random.default_rng(23)
    T, nh, nkv, hd = 4100, 4, 1, 128
    q, k, v = bits(g, T, nh, hd, std=2.0), bits(g, T, nkv, hd), bits(g, T, nkv, hd)
    out, lse = run_prompt(q, k, v, [0, T], True)
    rows = np.unique(np.concatenate([g.integers(0, T, 40), [0, 63, 64, 4095, 4096, T - 1]]))
    for t in rows:
        ref = oa.paged(q[t:t + 1], k[:t + 1], v[:t + 1], np.arange(t + 1)[None], [t + 1], [0, 1], 1, True, hd ** -0.5)
        check_rows(out[t:t + 1], lse[t:t + 1], ref, hd, f"token {t}")


# ---------------------------------------------------------------- as they are used together

def test_prompt_then_rounds_over_one_cache():
    """A prompt through append and prompt attention, then two verify blocks through append
    and paged attention on the cache so filled: every block's rows equal the rows prompt
    attention gives for the whole text, up to the bound."""
    g = np.random.default_rng(31)
    nh, nkv, hd, page = 8, 2, 128, 16
    first, total = [50, 7, 81], [61, 24, 98]
    pages = 24
    order = g.permutation(pages)
    table, at = np.full((3, 8), -1, np.int32), 0
    for b, n in enumerate(total):
        table[b, :-(-n // page)] = order[at:at + -(-n // page)]
        at += -(-n // page)
    text = [tuple(bits(g, n, h, hd) for h in (nh, nkv, nkv)) for n in total]
    qw, kw = (synth.bf16_bits((1 + 0.1 * g.normal(size=hd)).astype(np.float32)) for _ in range(2))
    kc = torch.full((pages * page, nkv, hd), SENT, dtype=torch.int16, device="cuda")
    vc = torch.full((pages * page, nkv, hd), SENT, dtype=torch.int16, device="cuda")

    def append(lo, hi):
        parts = [np.concatenate([t[x][a:z] for t, a, z in zip(text, lo, hi)]) for x in range(3)]
        pos = np.concatenate([np.arange(a, z) for a, z in zip(lo, hi)]).astype(np.int32)
        slots = np.concatenate([table[b, np.arange(a, z) // page].astype(np.int64) * page + np.arange(a, z) % page
                                for b, (a, z) in enumerate(zip(lo, hi))])
        ko = torch.empty(parts[1].shape, dtype=torch.int16, device="cuda")
        q = dsl.kv_append(dev(parts[1]), dev(parts[2]), dev(pos), dev(slots), kc, vc, q=dev(parts[0]), qnorm_w=dev(qw),
                          knorm_w=dev(kw), k_out=ko)
        return q, ko, dev(parts[2]), dev(np.concatenate([[0], np.cumsum([z - a for a, z in zip(lo, hi)])]).astype(np.int32))

    q, k, v, cu = append([0, 0, 0], first)
    prompt = dsl.prompt_attention(q, k, v, cu)
    got = [[prompt[cu[b]:cu[b + 1]]] for b in range(3)]
    for lo, hi in ((first, [55, 16, 82]), ([55, 16, 82], total)):
        q, _, _, cu = append(lo, hi)
        out = dsl.paged_attention(q, kc, vc, dev(table), dev(np.array(hi, np.int32)), cu, 16, page)
        for b in range(3):
            got[b].append(out[cu[b]:cu[b + 1]])
    kc2, vc2 = kc, vc
    kc, vc = torch.empty_like(kc), torch.empty_like(vc)
    q, k, v, cu = append([0, 0, 0], total)
    assert torch.equal(dsl.prompt_attention(q, k, v, cu)[:first[0]], torch.cat(got[0])[:first[0]])
    ref = oa.prompt(host(q).view(np.uint16), host(k).view(np.uint16), host(v).view(np.uint16), host(cu), True, hd ** -0.5)
    check_rows(torch.cat([torch.cat(x) for x in got]), None, ref, hd, "rounds")
    used = np.concatenate([table[b, np.arange(n) // page] * page + np.arange(n) % page for b, n in enumerate(total)])
    assert torch.equal(kc2[dev(used.astype(np.int64))], kc[dev(used.astype(np.int64))])
    assert torch.equal(vc2[dev(used.astype(np.int64))], vc[dev(used.astype(np.int64))])


def test_decode_steps_captured_once():
    """Append and attention of one new token per request in one graph, replayed step by
    step: positions, slots and lengths are advanced by the program between the replays, and
    a second graph of the same workspace runs in turn with it."""
    g = np.random.default_rng(33)
    B, nh, nkv, hd, page, steps = 5, 8, 2, 128, 16, 6
    start = np.array([0, 15, 40, 600, 1300])
    width = 90
    table = g.permutation(B * width).reshape(B, width).astype(np.int32)
    slot = lambda b, t: int(table[b, t // page]) * page + t % page  # noqa: E731
    shape = (B * width * page, nkv, hd)
    old_k, old_v = bits(g, *shape), bits(g, *shape)
    kc, vc, ke, ve = dev(old_k), dev(old_v), dev(old_k), dev(old_v)
    q, k, v = (torch.empty((B, h, hd), dtype=torch.int16, device="cuda") for h in (nh, nkv, nkv))
    qo, out, other = (torch.empty((B, nh, hd), dtype=torch.int16, device="cuda") for _ in range(3))
    pos, kv = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    slots, cu, tb = torch.empty(B, dtype=torch.int64, device="cuda"), dev(np.arange(B + 1, dtype=np.int32)), dev(table)
    ws = torch.empty(dsl.paged_attention_workspace_size(B, B, 1, nh, nkv, hd), dtype=torch.uint8, device="cuda")
    for t in (q, k, v, pos, kv, slots):
        t.zero_()

    def step(o, causal):
        dsl.kv_append(k, v, pos, slots, kc, vc, q=q, q_out=qo)
        dsl.paged_attention(qo, kc, vc, tb, kv, cu, 1, page, causal=causal, out=o, workspace=ws)

    step(out, True)
    torch.cuda.synchronize()
    kc.copy_(ke), vc.copy_(ve)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr, o in zip(graphs, (out, other)):
        with torch.cuda.graph(gr):
            step(o, o is out)
    for n in range(steps):
        at = start + n
        new = [bits(g, B, h, hd) for h in (nh, nkv, nkv)]
        for t, x in zip((q, k, v, pos, kv, slots), new + [at.astype(np.int32), (at + 1).astype(np.int32),
                                                          np.array([slot(b, at[b]) for b in range(B)], np.int64)]):
            t.copy_(dev(x))
        for gr in graphs:
            gr.replay()
        qe = dsl.kv_append(k, v, pos, slots, ke, ve, q=q)
        want = dsl.paged_attention(qe, ke, ve, tb, kv, cu, 1, page)
        assert torch.equal(qo, qe) and torch.equal(kc, ke) and torch.equal(vc, ve), f"step {n}"
        assert torch.equal(out, want) and torch.equal(other, want), f"step {n}"   # one token sees all: causal or not
    ref = oa.paged(host(qo).view(np.uint16), host(kc).view(np.uint16), host(vc).view(np.uint16), table, start + steps,
                   np.arange(B + 1), page, True, hd ** -0.5)
    check_rows(out, None, ref, hd, "last step")


def test_draft_block_over_a_context_kv_cache():
    """context_kv fills two layers' caches; a draft block is appended behind the context
    of each layer and attends to all of it (not causal)."""
    g = np.random.default_rng(32)
    M, L, nkv, hd, nh, N = 90, 2, 2, 128, 8, 7
    H, S = 256, 128
    kc = torch.zeros((L, S, nkv, hd), dtype=torch.int16, device="cuda")
    vc = torch.zeros((L, S, nkv, hd), dtype=torch.int16, device="cuda")
    slot = g.permutation(S).astype(np.int64)
    w = lambda *s: dev(bits(g, *s, std=0.06))  # noqa: E731
    ones = dev(synth.bf16_bits(np.ones(H, np.float32)))
    knorm = dev(synth.bf16_bits(np.ones((L, hd), np.float32)))
    dsl.context_kv(w(M, H), w(H, H), None, ones, w(L * 2 * nkv * hd, H), w(L * 2 * nkv * hd), knorm,
                   dev(np.arange(M, dtype=np.int32)), dev(slot[:M]), kc, vc)
    table = dev(slot[None, :M + N].astype(np.int32))
    for layer in range(L):
        q, k, v = bits(g, N, nh, hd), bits(g, N, nkv, hd), bits(g, N, nkv, hd)
        qr = dsl.kv_append(dev(k), dev(v), dev(np.arange(M, M + N, dtype=np.int32)), dev(slot[M:M + N]), kc[layer],
                           vc[layer], q=dev(q), knorm_w=knorm[layer])
        out = dsl.paged_attention(qr, kc[layer], vc[layer], table, dev(np.array([M + N], np.int32)),
                                  dev(np.array([0, N], np.int32)), N, 1, causal=False)
        ref = oa.paged(host(qr).view(np.uint16), host(kc[layer]).view(np.uint16), host(vc[layer]).view(np.uint16),
                       host(table), [M + N], [0, N], 1, False, hd ** -0.5)
        check_rows(out, None, ref, hd, f"layer {layer}")
