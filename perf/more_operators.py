"""Workloads of the operators around a drafted tree and a long context, on one paged cache.

  mask     ``tree_mask``: a drafted tree's parents, as a list, to what every node sees and
           where it stands, once a round
  tree     ``tree_attention``: every node of a request's tree over the request's pages and
           over its own ancestors, once a layer
  window   ``paged_attention`` with a window and sinks: the round's few query tokens see the
           last keys and a few first ones
  prompt   ``prompt_attention`` with a window and sinks
  compact  ``kv_compact``: the accepted path of each tree moved together, in every layer
  pages    a round's bookkeeping on the device: ``pages_resize`` takes pages for the block to
           come and gives back those of the rejected tokens; with forks, ``pages_select``
           first makes requests children of others and ``kv_copy_pages`` carries out the
           copies that growing into a shared page asks for

``run`` makes one pass: with ``own`` false in elementary torch operations, with ``own``
true through the library.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16
WORDS = 4                                          # 32-bit words of a node's mask


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one user's tree of the anchor and 24 drafts: all latency
        dict(name="mask one tree", op="mask", batch=1, lo=25, hi=25, lens=1),
        # the largest trees of the largest batch
        dict(name="mask 512 trees", op="mask", batch=512, lo=33, hi=128, lens=2),
        # one user's tree over a short context: the smallest verify of a tree
        dict(name="tree one block", op="tree", batch=1, lo=25, hi=25, kv_lo=613, kv_hi=613, page=16, nh=32, nkv=8, hd=128, lens=3),
        # a serving batch of trees of every size over contexts of every length: matrix work and cache alike
        dict(name="tree 64 ragged", op="tree", batch=64, lo=9, hi=64, kv_lo=65, kv_hi=8192, page=64, nh=32, nkv=8, hd=128, lens=4),
        # one user far into a long document, one new token, a layer that looks back 1024 tokens
        dict(name="window one long", op="window", batch=1, lo=1, hi=1, kv_lo=131071, kv_hi=131071, page=16, nh=32, nkv=8, hd=128, causal=True, window=1024, sinks=4, lens=5),
        # the verify step of the largest round under a wide window; most contexts have outgrown it
        dict(name="window 256 blocks", op="window", batch=256, lo=1, hi=17, kv_lo=17, kv_hi=32768, page=64, nh=32, nkv=8, hd=128, causal=True, window=2048, sinks=4, lens=6),
        # a few chat turns, a narrow window, heads of 64 in groups of 8: short calls, mostly edges of windows
        dict(name="window prompt 5 short", op="prompt", batch=5, lo=1, hi=700, nh=16, nkv=2, hd=64, window=128, sinks=4, lens=7),
        # a long document under a wide window: the largest matrix work
        dict(name="window prompt one long", op="prompt", batch=1, lo=16384, hi=16384, nh=32, nkv=8, hd=128, window=4096, sinks=16, lens=8),
        # one user's round: four of the accepted drafts move up, in five layers
        dict(name="compact one", op="compact", batch=1, layers=5, nodes=25, a_lo=5, a_hi=5, ctx=517, page=16, nkv=8, hd=128, lens=9),
        # the largest round's trees
        dict(name="compact 256", op="compact", batch=256, layers=5, nodes=64, a_lo=1, a_hi=17, ctx=100, page=64, nkv=8, hd=128, lens=10),
        # an ordinary batch's round: pages for 17 tokens each, and back to what was accepted
        dict(name="pages 64 requests", op="pages", batch=64, beams=0, kv_lo=1, kv_hi=2048, grow=17, total=16384, page=16, layers=0, nkv=8, hd=128, lens=11),
        # 64 requests of four beams each choose among their own, and each goes on in pages of its own
        dict(name="pages 256 forked", op="pages", batch=256, beams=4, kv_lo=17, kv_hi=1024, grow=17, total=8192, page=16, layers=5, nkv=8, hd=128, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(32, 8, 128), (16, 2, 64), (8, 8, 128), (20, 4, 128), (16, 1, 128), (24, 8, 64), (8, 2, 256)]


def draw(rng):
    op = rng.choice(["mask", "tree", "tree", "window", "window", "prompt", "prompt", "compact", "pages"])
    nh, nkv, hd = rng.choice(HEADS)
    lens = rng.randrange(100, 1 << 20)
    if op == "mask":
        hi = _log(rng, 2, 128)
        return dict(op=op, batch=_log(rng, 1, 512), lo=rng.randint(1, hi), hi=hi, lens=lens)
    if op == "tree":
        batch, hi = _log(rng, 1, 128), _log(rng, 2, 128)
        kv_hi = max(hi + 1, min(_log(rng, 130, 32768), (1 << 35) // (batch * nh * hd * hi), (1 << 28) // (batch * nkv * hd)))
        return dict(op=op, batch=batch, lo=rng.randint(1, hi), hi=hi, kv_lo=rng.randint(hi, kv_hi), kv_hi=kv_hi,
                    page=rng.choice([1, 16, 32, 64, 256]), nh=nh, nkv=nkv, hd=hd, lens=lens)
    if op == "window":
        batch, hi, window = _log(rng, 1, 256), _log(rng, 1, 17), _log(rng, 16, 8192)
        window = max(16, min(window, (1 << 28) // (batch * nkv * hd)))
        kv_hi = _log(rng, 32, 131071)
        return dict(op=op, batch=batch, lo=rng.randint(1, hi), hi=hi, kv_lo=rng.randint(17, kv_hi), kv_hi=kv_hi,
                    page=rng.choice([1, 16, 32, 64, 256]), nh=nh, nkv=nkv, hd=hd, causal=rng.random() < 0.8, window=window,
                    sinks=rng.choice([0, 1, 4, 16, 64, 100]), lens=lens)
    if op == "prompt":
        batch, window = _log(rng, 1, 24), _log(rng, 16, 4096)
        hi = max(2, min(_log(rng, 2, 8192), (1 << 36) // (batch * nh * hd * window) + window))
        return dict(op=op, batch=batch, lo=rng.randint(1, hi), hi=hi, nh=nh, nkv=nkv, hd=hd, window=window,
                    sinks=rng.choice([0, 1, 4, 16, 64, 100]), lens=lens)
    if op == "compact":
        batch, nodes = _log(rng, 1, 256), rng.randint(4, 128)
        a_hi = rng.randint(1, nodes - 1)
        return dict(op=op, batch=batch, layers=rng.choice([1, 2, 5]), nodes=nodes, a_lo=rng.randint(1, a_hi), a_hi=min(a_hi, 17 + a_hi // 4),
                    ctx=rng.randint(0, 300), page=rng.choice([1, 16, 32, 64, 256]), nkv=nkv, hd=hd, lens=lens)
    beams = rng.choice([0, 0, 2, 4, 8])
    batch = _log(rng, 1, 512) if not beams else beams * _log(rng, 1, 64)
    page, grow = rng.choice([16, 32, 64]), rng.randint(1, 64)
    kv_hi = _log(rng, 32, 1024 if beams else 4096)
    need = batch * (-(-(kv_hi + grow) // page) + 1)
    return dict(op=op, batch=batch, beams=beams, kv_lo=rng.randint(17, kv_hi), kv_hi=kv_hi, grow=grow, total=need + rng.randint(0, 5000),
                page=page, layers=1 if beams else 0, nkv=2, hd=128, lens=lens)


def _lengths(case):
    """The lengths of a ragged batch belong to the case; the values come from the seed."""
    r = random.Random(case["lens"])
    if case["op"] in ("mask", "prompt"):
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    if case["op"] == "compact":
        a = [r.randint(min(case["a_lo"], case["a_hi"]), case["a_hi"]) for _ in range(case["batch"])]
        return a, [r.randint(0, 2 * case["ctx"]) for _ in a]
    if case["op"] == "pages":
        group = max(1, case["beams"])                         # beams of one request are as long as each other
        kv = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["batch"] // group)]
        return [n for n in kv for _ in range(group)]
    q = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    return q, [max(a, r.randint(case["kv_lo"], case["kv_hi"])) for a in q]


def _window_keys(p, kv, window, sinks, causal):
    """Keys that the token at position p sees."""
    end = p + 1 if causal else kv
    low = max(0, p - window + 1)
    return max(0, end - low) + min(sinks, low, end)


def work(case):
    op = case["op"]
    if op == "mask":
        n = sum(_lengths(case))
        return {"bytes": n * (4 + 4 * WORDS + 4) + 8 * case["batch"], "flops": n}
    if op == "compact":
        a, _ = _lengths(case)
        rows = sum(v - 1 for v in a)                          # (the anchor stays where it is)
        return {"bytes": rows * 2 * case["layers"] * case["nkv"] * case["hd"] * 2 * 2 + 4 * sum(a) + 16 * len(a), "flops": 0}
    if op == "pages":
        kv, page = _lengths(case), case["page"]
        taken = sum(-(-(n + case["grow"]) // page) - -(-n // page) for n in kv)
        small = 4 * (4 * taken + 6 * len(kv))
        if not case["beams"]:
            return {"bytes": small, "flops": 0}
        held = sum(-(-n // page) for n in kv)
        copies = sum(1 for n in kv if n % page) // 2          # about: the last child of a page keeps it
        return {"bytes": small + 4 * 4 * held + copies * 2 * case["layers"] * page * case["nkv"] * case["hd"] * 2 * 2, "flops": 0}
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    if op == "prompt":
        n = _lengths(case)
        pairs = sum(_window_keys(p, v, case["window"], case["sinks"], True) for v in n for p in range(v))
        return {"bytes": 4 * hd * (nh + nkv) * sum(n) + 4 * (len(n) + 1), "flops": 4 * hd * nh * pairs}
    q, kv = _lengths(case)
    if op == "tree":
        pages = sum(-(-n // case["page"]) for n in kv)
        # the drafts of a tree see about log2 of its size of each other
        pairs = sum(a * (b - a) + int(a * (1 + math.log2(a))) for a, b in zip(q, kv))
        return {"bytes": 4 * hd * (sum(q) * nh + sum(kv) * nkv) + 4 * (pages + 2 * len(q) + 1) + 4 * WORDS * sum(q), "flops": 4 * hd * nh * pairs}
    seen = sum(_window_keys(b - a, b, case["window"] + a - 1, case["sinks"], False) for a, b in zip(q, kv))
    pairs = sum(_window_keys(b - a + j, b, case["window"], case["sinks"], case["causal"]) for a, b in zip(q, kv) for j in range(a))
    return {"bytes": 4 * hd * (sum(q) * nh + seen * nkv) + 4 * (seen // case["page"] + 2 * len(q) + 1), "flops": 4 * hd * nh * pairs}


# ---------------------------------------------------------------- inputs

def _sums(n):
    out = [0]
    for v in n:
        out.append(out[-1] + v)
    return out


def _parents(r, n):
    """A drafted tree: node 0 is the anchor, the others hang below earlier ones."""
    return [-1] + [max(0, j - 1 - int(r.expovariate(0.4))) for j in range(1, n)]


def _bits_of(parent, n):
    """Masks of one tree, as WORDS unsigned words a node."""
    seen = []
    for j in range(n):
        seen.append((seen[parent[j]] if parent[j] >= 0 else 0) | 1 << j)
    return [[v >> 32 * w & 0xFFFFFFFF for w in range(WORDS)] for v in seen]


def _signed(rows):
    return [[v - (1 << 32) if v >= 1 << 31 else v for v in row] for row in rows]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    r = random.Random(int(seed) * 7919 + case["lens"])
    op = case["op"]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(BF16)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    s = dict(case=case)
    if op == "mask":
        n = _lengths(case)
        s["parent"], s["cu_q"], s["max_q"] = ints([p for v in n for p in _parents(r, v)]), ints(_sums(n)), max(n)
        s["kv_len"] = ints([v + r.randint(0, 8192) for v in n])
        s["mask"] = torch.empty(sum(n), WORDS, dtype=torch.int32, device=dev)
        s["positions"] = torch.empty(sum(n), dtype=torch.int32, device=dev)
        return s
    nkv, hd, page = case["nkv"], case["hd"], case.get("page")
    if op == "prompt":
        n, nh = _lengths(case), case["nh"]
        t = sum(n)
        s["q"], s["k"] = normal(t, nh, hd, std=2.0), normal(t, nkv, hd)
        s["v"] = normal(t, (nh + 2 * nkv) * hd)[:, (nh + nkv) * hd:].view(t, nkv, hd)
        s["cu"], s["lens"], s["out"], s["scale"] = ints(_sums(n)), n, torch.empty_like(s["q"]), hd ** -0.5
        return s

    def paged(kv, kept):
        """A table of pages in no order; of request b the pages kept(b, p) are there, others dropped."""
        need = [-(-n // page) for n in kv]
        rows = [[p for p in range(m) if kept(b, p)] for b, m in enumerate(need)]
        total = sum(map(len, rows)) + 3
        order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        table = torch.full((len(kv), max(1, max(need))), -1, dtype=torch.int32, device=dev)
        at = [(b, p) for b, row in enumerate(rows) for p in row]
        if at:
            b, p = torch.tensor(at, device=dev).T.contiguous()
            table[b, p] = order[:len(at)]
        return table, total

    if op in ("tree", "window"):
        q, kv = _lengths(case)
        nh, w = case["nh"], case.get("window")
        kept = (lambda b, p: True) if op == "tree" else \
            (lambda b, p: p * page < case["sinks"] or (p + 1) * page > kv[b] - q[b] - w + 1)   # pages behind the window are given back
        s["page_table"], total = paged(kv, kept)
        s["kv_len"], s["cu_q"], s["max_q"], s["max_kv"] = ints(kv), ints(_sums(q)), max(q), max(kv)
        s["q"], s["scale"] = normal(sum(q), nh, hd, std=2.0), hd ** -0.5
        s["out"] = torch.empty_like(s["q"])
        s["k_cache"], s["v_cache"] = normal(total * page, nkv, hd), normal(total * page, nkv, hd)
        if op == "tree":
            s["mask"] = ints(_signed([row for n in q for row in _bits_of(_parents(r, n), n)]))
        if own:
            import draft_sampling_lossless_amd as dsl
            need = dsl.paged_attention_workspace_size(s["q"].shape[0], case["batch"], s["max_q"], nh, nkv, hd)
            s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device=dev)
        return s
    if op == "compact":
        a, ctx = _lengths(case)
        n, b = case["nodes"], case["batch"]
        kv = [c + n for c in ctx]
        s["page_table"], total = paged(kv, lambda b, p: True)
        s["kv_len"], s["cu_q"] = ints(kv), ints(_sums([n] * b))
        paths = [[0] + sorted(r.sample(range(2, n), v - 1)) for v in a]       # the anchor, then nodes that all move
        s["path"] = ints([p + [-1] * (max(a) - len(p)) for p in paths])
        s["accepted"], s["new_len"] = ints(a), torch.empty(b, dtype=torch.int32, device=dev)
        s["k_cache"], s["v_cache"] = normal(case["layers"], total * page, nkv, hd), normal(case["layers"], total * page, nkv, hd)
        return s
    # pages: beams of a request share all but their last page before the call
    kv, beams, total = _lengths(case), case["beams"], case["total"]
    width = -(-(max(kv) + case["grow"]) // page)
    group = max(1, beams)
    order = r.sample(range(total), total)
    table, refs, at = [], [0] * total, 0
    for b, n in enumerate(kv):
        m = -(-n // page)
        own_from = 0 if b % group == 0 else m - 1
        row = (table[b - b % group][:own_from] if own_from else []) + order[at:at + m - own_from]
        at += m - own_from
        for p in row:
            refs[p] += 1
        table.append(row + [-1] * (width - m))
    s["page_table"], s["refs"], s["kv_len"] = ints(table), ints(refs), ints(kv)
    s["grown"], s["kept"] = ints([n + case["grow"] for n in kv]), ints(kv)
    s["copies"] = torch.empty(case["batch"], 2, dtype=torch.int32, device=dev)
    s["served"] = torch.empty(case["batch"], dtype=torch.int32, device=dev)
    if beams:
        s["src"] = ints([b - b % beams + r.randrange(beams) for b in range(case["batch"])])
        s["other_table"], s["other_len"] = torch.empty_like(s["page_table"]), torch.empty_like(s["kv_len"])
        s["k_cache"], s["v_cache"] = normal(case["layers"], total * page, nkv, hd), normal(case["layers"], total * page, nkv, hd)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"mask": _mask_plain, "tree": _paged_plain, "window": _paged_plain, "prompt": _prompt_plain,
                "compact": _compact_plain, "pages": _pages}[op](s)
    import draft_sampling_lossless_amd as dsl
    if op == "mask":
        mask, positions = dsl.tree_mask(s["parent"], s["kv_len"], s["cu_q"], s["max_q"], mask=s["mask"], positions=s["positions"])
        return dict(mask=mask, positions=positions)
    if op == "tree":
        return dsl.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["cu_q"], s["mask"],
                                  s["max_q"], c["page"], scale=s["scale"], out=s["out"], workspace=s["workspace"])
    if op == "window":
        return dsl.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["cu_q"], s["max_q"],
                                   c["page"], causal=c["causal"], scale=s["scale"], out=s["out"], workspace=s["workspace"],
                                   window=c["window"], sinks=c["sinks"])
    if op == "prompt":
        return dsl.prompt_attention(s["q"], s["k"], s["v"], s["cu"], causal=True, scale=s["scale"], out=s["out"],
                                    window=c["window"], sinks=c["sinks"])
    if op == "compact":
        dsl.kv_compact(s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["cu_q"], s["path"], s["accepted"],
                       c["page"], new_len=s["new_len"])
        return _compact_outputs(s)
    return _pages(s)


def _mask_plain(s):
    cu, n, m = s["cu_q"].long(), s["max_q"], s["parent"].shape[0]
    dev = cu.device
    t = torch.arange(m, device=dev)
    of = (t[:, None] >= cu[None, 1:]).sum(1)
    j = t - cu[of]
    seen = torch.zeros(m + 1, 32 * WORDS, dtype=torch.bool, device=dev)        # row m: nothing above a root
    seen[t, j] = True
    up = torch.where(s["parent"] >= 0, cu[of] + s["parent"], torch.full_like(t, m))
    up = torch.cat((up, up.new_tensor([m])))
    for _ in range(max(1, (n - 1).bit_length())):                              # ancestors 1, 2, 4, .. up
        seen = seen | seen[up]
        up = up[up]
    seen = seen[:m]
    words = (seen.view(m, WORDS, 32).long() << torch.arange(32, device=dev)).sum(-1)
    s["mask"].copy_(torch.where(words >= 1 << 31, words - (1 << 32), words))
    s["positions"].copy_(s["kv_len"].long()[of] - (cu[1:] - cu[:-1])[of] + seen.sum(1) - 1)
    return dict(mask=s["mask"], positions=s["positions"])


def _attend(q, k, v, seen, scale):
    """q [.., R, hd], k and v [.., L, hd], seen broadcastable to [.., R, L]; float32 throughout."""
    w = torch.matmul(q, k.transpose(-1, -2).contiguous()) * scale
    w = torch.where(seen, w, torch.full((), -math.inf, device=w.device))
    w = torch.exp(w - w.amax(-1, keepdim=True).clamp(min=-3e38))
    return torch.matmul(w, v) / w.sum(-1, keepdim=True).clamp(min=1e-37)


def _paged_plain(s):
    """Trees and windows: the keys that some row of a request may see are gathered, and masked."""
    c = s["case"]
    nh, nkv, hd, page, b = c["nh"], c["nkv"], c["hd"], c["page"], c["batch"]
    dev, cu, kv_len, m = s["q"].device, s["cu_q"].long(), s["kv_len"].long(), s["max_q"]
    ctx = kv_len - (cu[1:] - cu[:-1])
    if c["op"] == "tree":
        key = torch.arange(s["max_kv"], device=dev)[None].expand(b, -1)
    else:
        sinks, low = c["sinks"], (ctx - c["window"] + 1).clamp(min=c["sinks"])
        far = min(s["max_kv"], c["window"] + m)
        key = torch.cat((torch.arange(sinks, device=dev)[None].expand(b, -1), low[:, None] + torch.arange(far, device=dev)), 1)
    held = key < kv_len[:, None]                                               # [B, L]
    col = (key // page).clamp(max=s["page_table"].shape[1] - 1)
    slot = s["page_table"].long().gather(1, col).clamp(min=0) * page + key % page
    k = s["k_cache"][slot].float().transpose(1, 2).contiguous()                # [B, nkv, L, hd]
    v = s["v_cache"][slot].float().transpose(1, 2).contiguous()
    j = torch.arange(m, device=dev)
    at = (cu[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float()                                                     # [B, m, nh, hd]
    q = q.view(b, m, nkv, nh // nkv, hd).transpose(1, 2).reshape(b, nkv, -1, hd)
    pos = ctx[:, None] + j                                                     # [B, m]
    if c["op"] == "tree":
        node = key - ctx[:, None]                                              # [B, L]; below 0: context
        word = (node.clamp(0, 127) // 32)[:, None].expand(b, m, -1)
        bit = s["mask"].long()[at].gather(2, word) >> (node.clamp(0, 127) % 32)[:, None] & 1
        seen = (node < 0)[:, None] | (bit == 1)
    else:
        seen = (key[:, None] < sinks) | (key[:, None] > pos[:, :, None] - c["window"])
        if c["causal"]:
            seen = seen & (key[:, None] <= pos[:, :, None])
    seen = seen & held[:, None]
    out = _attend(q, k, v, seen.repeat_interleave(nh // nkv, 1)[:, None], s["scale"])
    out = out.view(b, nkv, m, nh // nkv, hd).transpose(1, 2).reshape(b, m, nh, hd)
    t = torch.arange(s["q"].shape[0], device=dev)
    of = (t[:, None] >= cu[None, 1:]).sum(1)
    s["out"].copy_(out[of, t - cu[of]])
    return s["out"]


def _prompt_plain(s):
    c = s["case"]
    nh, nkv, hd, window, sinks = c["nh"], c["nkv"], c["hd"], c["window"], c["sinks"]
    dev, begin = s["q"].device, 0
    for n in s["lens"]:
        for lo in range(0, n, 1024):                                           # blocks of rows, over what they may see
            hi = min(n, lo + 1024)
            low = max(0, lo - window + 1)
            key = torch.cat((torch.arange(min(sinks, low), device=dev), torch.arange(low, hi, device=dev)))
            k = s["k"][begin + key].float().transpose(0, 1)
            v = s["v"][begin + key].float().transpose(0, 1)
            q = s["q"][begin + lo:begin + hi].float().view(hi - lo, nkv, nh // nkv, hd).permute(1, 2, 0, 3).reshape(nkv, -1, hd)
            p = torch.arange(lo, hi, device=dev)[:, None]
            seen = (key <= p) & ((key > p - window) | (key < sinks))
            out = _attend(q, k, v, seen.repeat(nh // nkv, 1)[None], s["scale"])
            s["out"][begin + lo:begin + hi] = out.view(nh, hi - lo, hd).transpose(0, 1).to(BF16)
        begin += n
    return s["out"]


def _compact_outputs(s):
    return dict(new_len=s["new_len"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _compact_plain(s):
    page, path = s["case"]["page"], s["path"].long()
    i = torch.arange(path.shape[1], device=path.device)[None].expand_as(path)
    ctx = s["kv_len"].long() - (s["cu_q"][1:] - s["cu_q"][:-1])
    there = i < s["accepted"][:, None]
    of = torch.arange(path.shape[0], device=path.device)[:, None].expand_as(path)[there]

    def slot(key):
        return s["page_table"].long()[of, key // page] * page + key % page

    src, dst = slot((ctx[:, None] + path)[there]), slot((ctx[:, None] + i)[there])
    s["k_cache"][:, dst] = s["k_cache"][:, src]
    s["v_cache"][:, dst] = s["v_cache"][:, src]
    s["new_len"].copy_(ctx + s["accepted"])
    return _compact_outputs(s)


def _pages(s):
    """A round: (fork,) room for the block, (copies,) back to what was accepted."""
    c = s["case"]
    page, beams = c["page"], c["beams"]
    if own:
        import draft_sampling_lossless_amd as dsl
        resize, select, copy = dsl.pages_resize, dsl.pages_select, dsl.kv_copy_pages
    else:
        resize, select, copy = _resize_plain, _select_plain, _copy_plain
    if beams:
        select(s["page_table"], s["kv_len"], s["src"], s["refs"], page, new_table=s["other_table"], new_len=s["other_len"])
        s["page_table"], s["other_table"] = s["other_table"], s["page_table"]
        s["kv_len"], s["other_len"] = s["other_len"], s["kv_len"]
    resize(s["page_table"], s["kv_len"], s["grown"], s["refs"], page, copies=s["copies"], served=s["served"])
    out = dict(copies=s["copies"], served=s["served"])
    if beams:
        copy(s["k_cache"], s["v_cache"], s["copies"], page)
        out.update(k_cache=s["k_cache"], v_cache=s["v_cache"])
    grown = s["page_table"].clone()                        # (what the block's tokens go into)
    resize(s["page_table"], s["kv_len"], s["kept"], s["refs"], page)
    out.update(grown=grown, page_table=s["page_table"], kv_len=s["kv_len"], refs=s["refs"])
    return out


def _select_plain(table, kv_len, src, refs, page, new_table, new_len):
    col, p = torch.arange(table.shape[1], device=table.device), refs.shape[0]
    held = torch.where(col < ((kv_len + page - 1) // page)[:, None], table, torch.full_like(table, -1))
    none = src < 0
    new_table.copy_(torch.where(none[:, None], torch.full_like(held[:1], -1), held[src.clamp(min=0).long()]))
    new_len.copy_(torch.where(none, torch.zeros_like(src), kv_len[src.clamp(min=0).long()]))
    for t, sign in ((new_table, 1), (held, -1)):
        there = (t >= 0) & (t < p)
        refs.index_add_(0, t.clamp(0, p - 1).flatten().long(), sign * there.flatten().int())


def _copy_plain(k_cache, v_cache, copies, page):
    there = (copies >= 0).all(1)
    src, dst = copies.long()[there].T
    for cache in (k_cache, v_cache):
        pages = cache.view(cache.shape[0], -1, page, *cache.shape[2:])
        pages[:, dst] = pages[:, src]


def _resize_plain(table, kv_len, new_len, refs, page, copies=None, served=None):
    b, w = table.shape
    dev, p = table.device, refs.shape[0]
    col = torch.arange(w, device=dev)
    old, new = kv_len.clamp(0, w * page), new_len.clamp(0, w * page)
    hold, want = (old + page - 1) // page, (new + page - 1) // page
    drop = (col >= want[:, None]) & (col < hold[:, None])                      # pages given back, first of all
    gone = drop & (table >= 0) & (table < p)
    refs.index_add_(0, table.clamp(0, p - 1).flatten().long(), -gone.flatten().int())
    table.copy_(torch.where(drop, torch.full_like(table, -1), table))
    # growing into a page that others hold too takes a copy of it, request after request
    grows = new > old
    end = (old // page).clamp(max=w - 1).long()
    last = table.gather(1, end[:, None])[:, 0]
    count = refs[last.clamp(0, p - 1).long()]
    shared = grows & (old % page != 0) & (last >= 0) & (last < p) & (count > 1)
    before = ((last[:, None] == last[None]) & shared[None] & shared[:, None]).tril(-1).sum(1)
    copied = shared & (count - before > 1)
    need = torch.where(grows, want - hold, torch.zeros_like(want)) + copied
    total = need.cumsum(0)
    free = refs == 0
    rank = free.cumsum(0)
    ok = ~grows | (total <= rank[-1]) | ((need == 0) & ~shared)
    # the r-th free page by number goes to the r-th need
    by_rank = torch.zeros(p + 1, dtype=torch.int32, device=dev)
    by_rank[torch.where(free, rank - 1, torch.full_like(rank, p))] = torch.arange(p, dtype=torch.int32, device=dev)
    first = total - need
    copied = copied & ok
    cell = (col >= hold[:, None]) & (col < want[:, None]) & (ok & grows)[:, None]
    at = (first + copied)[:, None] + col - hold[:, None]
    fresh = by_rank[at.clamp(0, p)]
    mine = by_rank[first.clamp(0, p)]
    refs.index_add_(0, last.clamp(0, p - 1).long(), -copied.int())
    refs.index_add_(0, mine.long().clamp(0, p - 1), copied.int())
    refs.index_add_(0, fresh.flatten().long(), cell.flatten().int())
    table.copy_(torch.where(cell, fresh, table))
    table.scatter_(1, end[:, None], torch.where(copied, mine, table.gather(1, end[:, None])[:, 0])[:, None])
    kv_len.copy_(torch.where(ok, new, old))
    if copies is not None:
        none = torch.full_like(last, -1)
        copies.copy_(torch.stack((torch.where(copied, last, none), torch.where(copied, mine, none)), 1))
    if served is not None:
        served.copy_(ok)


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    return {"mask": _mask_exact, "tree": _attention_exact, "window": _attention_exact, "prompt": _attention_exact,
            "compact": _compact_exact, "pages": _pages_exact}[case["op"]](case, s)


def _mask_exact(case, s):
    parent, kv, rows, positions, at = s["parent"].tolist(), s["kv_len"].tolist(), [], [], 0
    for b, n in enumerate(_lengths(case)):
        tree = parent[at:at + n]
        rows += _signed(_bits_of(tree, n))
        depth = []
        for j in range(n):
            depth.append(depth[tree[j]] + 1 if tree[j] >= 0 else 0)
        positions += [kv[b] - n + d for d in depth]
        at += n
    return dict(mask=torch.tensor(rows, dtype=torch.int32, device="cuda"),
                positions=torch.tensor(positions, dtype=torch.int32, device="cuda"))


def _attention_exact(case, s):
    nh, nkv, hd, op = case["nh"], case["nkv"], case["hd"], case["op"]
    group = nh // nkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lengths = _lengths(case)
    q_lens, kv_lens = (lengths, lengths) if op == "prompt" else lengths
    begin = 0
    for b, (nq, nk) in enumerate(zip(q_lens, kv_lens)):
        ctx, window, sinks = nk - nq, case.get("window"), case.get("sinks", 0)
        for lo in range(0, nq, 512):
            hi = min(nq, lo + 512)
            pos = ctx + torch.arange(lo, hi, device="cuda")
            low = 0 if op == "tree" else max(0, ctx + lo - window + 1)
            key = torch.arange(low, nk, device="cuda")
            if op != "tree":
                key = torch.cat((torch.arange(min(sinks, low), device="cuda"), key))
            if op == "prompt":
                key = key[key < hi]
                k, v = s["k"][begin + key], s["v"][begin + key]
            else:
                slot = s["page_table"][b, key // case["page"]].long() * case["page"] + key % case["page"]
                k, v = s["k_cache"][slot], s["v_cache"][slot]
            if op == "tree":
                word = s["mask"][begin + lo:begin + hi].long()[:, ((key - ctx).clamp(min=0) // 32)]
                seen = (key < ctx) | ((word >> ((key - ctx).clamp(min=0) % 32)) % 2 == 1)
            else:
                back = pos[:, None] - key
                seen = (back < window) | (key < sinks)
                if op == "prompt" or case["causal"]:
                    seen = seen & (back >= 0)
            for g in range(nkv):
                kd, vd = k[:, g].double(), v[:, g].double()
                for h in range(g * group, (g + 1) * group):
                    w = (s["q"][begin + lo:begin + hi, h].double() @ kd.T.contiguous()) * s["scale"]
                    out[begin + lo:begin + hi, h] = torch.softmax(w.masked_fill(~seen, -math.inf), -1) @ vd
        begin += nq
    return out


def _compact_exact(case, s):
    page, n = case["page"], case["nodes"]
    table, path = s["page_table"].tolist(), s["path"].tolist()
    a, ctx = _lengths(case)
    src, dst = [], []
    for b in range(case["batch"]):
        for i in range(a[b]):
            for to, node in ((src, path[b][i]), (dst, i)):
                key = ctx[b] + node
                to.append(table[b][key // page] * page + key % page)
    src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
    out = dict(new_len=torch.tensor([x + y for x, y in zip(ctx, a)], dtype=torch.int32, device="cuda"))
    for name in ("k_cache", "v_cache"):
        moved = s[name].clone()
        moved[:, dst] = s[name][:, src]
        out[name] = moved
    return out


def _pages_exact(case, s):
    """The bookkeeping one request and one page after the other."""
    page = case["page"]
    table, kv, refs = s["page_table"].tolist(), s["kv_len"].tolist(), s["refs"].tolist()
    if case["beams"]:
        old, old_kv, src = table, kv, s["src"].tolist()
        table, kv = [list(old[b]) for b in src], [old_kv[b] for b in src]
        for rows, lens, sign in ((table, kv, 1), (old, old_kv, -1)):
            for row, n in zip(rows, lens):
                for p in row[:-(-n // page)]:
                    refs[p] += sign

    def resize(new):
        copies, served = [[-1, -1] for _ in new], [1] * len(new)
        for b, n in enumerate(new):                                            # what is given back
            for p in range(-(-n // page), -(-kv[b] // page)):
                refs[table[b][p]] -= 1
                table[b][p] = -1
        free = sorted(p for p, r in enumerate(refs) if r == 0)
        for b, n in enumerate(new):
            if n > kv[b]:
                last = table[b][kv[b] // page] if kv[b] % page else -1
                if last >= 0 and refs[last] > 1:
                    copies[b] = [last, free.pop(0)]
                    refs[last] -= 1
                    refs[copies[b][1]] = 1
                    table[b][kv[b] // page] = copies[b][1]
                for p in range(-(-kv[b] // page), -(-n // page)):
                    table[b][p] = free.pop(0)
                    refs[table[b][p]] = 1
            kv[b] = n
        return copies, served

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    copies, served = resize(s["grown"].tolist())
    out = dict(copies=ints(copies), served=ints(served))
    if case["beams"]:
        src, dst = ints([c for c in copies if c[0] >= 0]).view(-1, 2).long().T
        for name in ("k_cache", "v_cache"):
            cache = s[name].clone()
            pages = cache.view(cache.shape[0], -1, page, *cache.shape[2:])
            pages[:, dst] = pages[:, src]
            out[name] = cache
    out["grown"] = ints(table)
    resize(s["kept"].tolist())
    out.update(page_table=ints(table), kv_len=ints(kv), refs=ints(refs))
    return out
