"""Workloads of the attention operators that stand around a speculative round.

Three operators share one key-value cache, the one ``context_kv`` fills (a layer's
[num_slots, nkv, hd] in bfloat16):

  append  ``kv_append``: norm and rotate the new tokens' queries and keys, and put
          keys and values into the cache at their slots;
  paged   ``paged_attention``: the round's few query tokens of every request (one of a
          plain decode, the anchor and the drafts of a verify, the draft's own block)
          over the request's pages of that cache;
  prompt  ``prompt_attention``: causal or full attention over whole packed prompts.

``run`` makes one pass: with ``own`` false in elementary torch operations, with ``own``
true through the library.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16
EPS, THETA = 1e-6, 1e6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one request's verify block (the anchor and 8 drafts): a decode loop of a single user, all latency
        dict(name="append one block", op="append", tokens=9, nh=32, nkv=8, hd=128, slots=4096, norm=True, keys_out=False),
        # the verify blocks of 256 requests with 16 drafts each: the largest round
        dict(name="append 256 blocks", op="append", tokens=4352, nh=32, nkv=8, hd=128, slots=32768, norm=True, keys_out=False),
        # a prefill chunk; the rotated keys also stay packed, for the attention over the prompt
        dict(name="append prompt chunk", op="append", tokens=8192, nh=32, nkv=8, hd=128, slots=16384, norm=True, keys_out=True),
        # one user, a short context, one new token: the smallest attention call
        dict(name="decode one short", op="paged", batch=1, q_lo=1, q_hi=1, kv_lo=517, kv_hi=517, page=16, nh=32, nkv=8, hd=128, causal=True, lens=1),
        # one user far into a long document: the cache's length is all there is to split
        dict(name="decode one long", op="paged", batch=1, q_lo=1, q_hi=1, kv_lo=131071, kv_hi=131071, page=64, nh=32, nkv=8, hd=128, causal=True, lens=2),
        # an ordinary serving batch, contexts of every length
        dict(name="decode 64 ragged", op="paged", batch=64, q_lo=1, q_hi=1, kv_lo=1, kv_hi=8192, page=16, nh=32, nkv=8, hd=128, causal=True, lens=3),
        # the verify step of the largest round: blocks cut to the admitted length
        dict(name="verify 256 blocks", op="paged", batch=256, q_lo=1, q_hi=17, kv_lo=17, kv_hi=4096, page=64, nh=32, nkv=8, hd=128, causal=True, lens=4),
        # the parallel draft: every position of the block sees the context and the whole block; slots given one by one
        dict(name="draft 64 blocks", op="paged", batch=64, q_lo=16, q_hi=16, kv_lo=100, kv_hi=4000, page=1, nh=32, nkv=8, hd=128, causal=False, lens=5),
        # a handful of chat turns just arrived: short prompts in one packed call
        dict(name="prompt 8 short", op="prompt", batch=8, lo=1, hi=127, nh=32, nkv=8, hd=128, causal=True, lens=6),
        # a packed prefill batch of prompts of different lengths
        dict(name="prompt 12 packed", op="prompt", batch=12, lo=1, hi=2048, nh=32, nkv=8, hd=128, causal=True, lens=7),
        # one long prompt: the largest matrix work
        dict(name="prompt one long", op="prompt", batch=1, lo=8192, hi=8192, nh=32, nkv=8, hd=128, causal=True, lens=8),
        # a small encoder-like draft backbone that sees its whole chunk: heads of 64, groups of 8, odd lengths
        dict(name="prompt full heads 64", op="prompt", batch=4, lo=901, hi=1000, nh=16, nkv=2, hd=64, causal=False, lens=9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(32, 8, 128), (16, 2, 64), (8, 8, 128), (20, 4, 128), (16, 1, 128), (24, 8, 64), (8, 2, 256)]


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "prompt"])
    nh, nkv, hd = rng.choice(HEADS)
    lens = rng.randrange(10, 1 << 20)
    if op == "append":
        tokens = _log(rng, 1, 8191)
        return dict(op=op, tokens=tokens, nh=nh, nkv=nkv, hd=hd, slots=tokens + rng.randrange(1, 8192),
                    norm=rng.random() < 0.7, keys_out=rng.random() < 0.5)
    if op == "paged":
        batch, q_hi = _log(rng, 1, 256), _log(rng, 1, 17)
        kv_hi = max(32, min(_log(rng, 32, 131071), (1 << 28) // (batch * nkv * hd)))
        return dict(op=op, batch=batch, q_lo=rng.randint(1, q_hi), q_hi=q_hi, kv_lo=rng.randint(17, kv_hi), kv_hi=kv_hi,
                    page=rng.choice([1, 16, 32, 64, 256]), nh=nh, nkv=nkv, hd=hd, causal=rng.random() < 0.7, lens=lens)
    batch = _log(rng, 1, 32)
    hi = max(2, min(_log(rng, 2, 6000), int(math.sqrt((1 << 37) // (batch * nh * hd)))))
    return dict(op=op, batch=batch, lo=rng.randint(1, hi), hi=hi, nh=nh, nkv=nkv, hd=hd, causal=rng.random() < 0.7,
                lens=lens)


def _lengths(case):
    """The lengths of a ragged batch belong to the case; the values come from the seed."""
    r = random.Random(case["lens"])
    if case["op"] == "prompt":
        return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    return q, [max(a, r.randint(case["kv_lo"], case["kv_hi"])) for a in q]


def _pairs(nq, nk, causal):
    """Visible (query, key) pairs of nq queries at the end of nk keys."""
    return nq * nk - (nq * (nq - 1) // 2 if causal else 0)


def work(case):
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    if case["op"] == "append":
        row = 2 * hd * (2 * nh + 4 * nkv + (nkv if case["keys_out"] else 0)) + 12
        return {"bytes": case["tokens"] * row + (4 * hd if case["norm"] else 0), "flops": case["tokens"] * (nh + nkv) * hd * 8}
    if case["op"] == "paged":
        q, kv = _lengths(case)
        pages = sum(-(-n // case["page"]) for n in kv)
        return {"bytes": 4 * hd * (sum(q) * nh + sum(kv) * nkv) + 4 * (pages + 2 * len(q) + 1),
                "flops": 4 * hd * nh * sum(_pairs(a, b, case["causal"]) for a, b in zip(q, kv))}
    n = _lengths(case)
    return {"bytes": 4 * hd * (nh + nkv) * sum(n) + 4 * (len(n) + 1),
            "flops": 4 * hd * nh * sum(_pairs(a, a, case["causal"]) for a in n)}


# ---------------------------------------------------------------- inputs

def _sums(n):
    out = [0]
    for v in n:
        out.append(out[-1] + v)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(BF16)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    s = dict(case=case, scale=hd ** -0.5)
    if case["op"] == "append":
        m, slots = case["tokens"], case["slots"]
        qkv = normal(m, (nh + 2 * nkv) * hd)       # the projections' one product, read in place
        s["q"] = qkv[:, :nh * hd].view(m, nh, hd)
        s["k"] = qkv[:, nh * hd:(nh + nkv) * hd].view(m, nkv, hd)
        s["v"] = qkv[:, (nh + nkv) * hd:].view(m, nkv, hd)
        s["qw"] = (1 + 0.1 * torch.randn(hd, generator=g, device=dev)).to(BF16) if case["norm"] else None
        s["kw"] = (1 + 0.1 * torch.randn(hd, generator=g, device=dev)).to(BF16) if case["norm"] else None
        start = int(torch.randint(0, 32768, (1,), generator=g, device=dev))
        s["positions"] = torch.arange(start, start + m, dtype=torch.int32, device=dev)
        s["slots"] = torch.randperm(slots, generator=g, device=dev)[:m]
        s["k_cache"], s["v_cache"] = normal(slots, nkv, hd), normal(slots, nkv, hd)
        s["q_out"] = torch.empty(m, nh, hd, dtype=BF16, device=dev)
        s["k_out"] = torch.empty(m, nkv, hd, dtype=BF16, device=dev) if case["keys_out"] else None
    elif case["op"] == "paged":
        q, kv = _lengths(case)
        page = case["page"]
        need = [-(-n // page) for n in kv]
        total, width = sum(need) + 3, max(need)
        order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        first = ints(_sums(need)[:-1])[:, None]
        cols = torch.arange(width, dtype=torch.int32, device=dev)[None]
        table = order[(first + cols).clamp(max=total - 1).long()]
        s["page_table"] = torch.where(cols < ints(need)[:, None], table, torch.full_like(table, -1)).contiguous()
        s["kv_len"], s["cu_q"], s["max_q"], s["max_kv"] = ints(kv), ints(_sums(q)), max(q), max(kv)
        s["q"] = normal(sum(q), nh, hd, std=2.0)
        s["k_cache"], s["v_cache"] = normal(total * page, nkv, hd), normal(total * page, nkv, hd)
        s["out"] = torch.empty_like(s["q"])
    else:
        n = _lengths(case)
        t = sum(n)
        s["q"], s["k"] = normal(t, nh, hd, std=2.0), normal(t, nkv, hd)   # as kv_append leaves them
        s["v"] = normal(t, (nh + 2 * nkv) * hd)[:, (nh + nkv) * hd:].view(t, nkv, hd)
        s["cu"], s["max_len"] = ints(_sums(n)), max(n)
        s["out"] = torch.empty_like(s["q"])
    if own:
        import draft_sampling_lossless_amd as dsl
        if case["op"] == "paged":
            need = dsl.paged_attention_workspace_size(s["q"].shape[0], case["batch"], s["max_q"], nh, nkv, hd)
            s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import draft_sampling_lossless_amd as dsl
        if op == "append":
            dsl.kv_append(s["k"], s["v"], s["positions"], s["slots"], s["k_cache"], s["v_cache"], q=s["q"],
                          qnorm_w=s["qw"], knorm_w=s["kw"], q_out=s["q_out"], k_out=s["k_out"], eps=EPS,
                          rope_theta=THETA)
            return _append_outputs(s)
        if op == "paged":
            return dsl.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_len"], s["cu_q"],
                                       s["max_q"], s["case"]["page"], causal=s["case"]["causal"], scale=s["scale"],
                                       out=s["out"], workspace=s["workspace"])
        return dsl.prompt_attention(s["q"], s["k"], s["v"], s["cu"], causal=s["case"]["causal"],
                                    scale=s["scale"], out=s["out"])
    return {"append": _append_plain, "paged": _paged_plain, "prompt": _prompt_plain}[op](s)


def _append_outputs(s):
    out = dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    if s["k_out"] is not None:
        out["k"] = s["k_out"]
    return out


def _append_plain(s):
    hd = s["case"]["hd"]
    i = torch.arange(hd // 2, dtype=torch.float64, device=s["q"].device)
    angle = s["positions"].double()[:, None] * THETA ** (-2 * i / hd)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotated(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        a, b = x[..., :hd // 2], x[..., hd // 2:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1).to(BF16)

    s["q_out"].copy_(rotated(s["q"], s["qw"]))
    k = rotated(s["k"], s["kw"])
    s["k_cache"][s["slots"]] = k
    s["v_cache"][s["slots"]] = s["v"]
    if s["k_out"] is not None:
        s["k_out"].copy_(k)
    return _append_outputs(s)


def _attend(q, k, v, seen, scale):
    """q [B, nkv, R, hd], k and v [B, nkv, L, hd], seen [B, 1, R, L]; float32 throughout."""
    w = torch.matmul(q, k.transpose(-1, -2).contiguous()) * scale
    w = torch.where(seen, w, torch.full((), -math.inf, device=w.device))
    w = torch.exp(w - w.amax(-1, keepdim=True).clamp(min=-3e38))
    return torch.matmul(w, v) / w.sum(-1, keepdim=True).clamp(min=1e-37)


def _paged_plain(s):
    c = s["case"]
    nh, nkv, hd, page, b = c["nh"], c["nkv"], c["hd"], c["page"], c["batch"]
    dev, cu, kv_len, n, m = s["q"].device, s["cu_q"].long(), s["kv_len"].long(), s["max_kv"], s["max_q"]
    key = torch.arange(n, device=dev)
    held = key < kv_len[:, None]                                              # [B, L]
    slot = s["page_table"][:, key // page].long().clamp(min=0) * page + key % page
    k = s["k_cache"][slot].float().transpose(1, 2).contiguous()               # [B, nkv, L, hd]
    v = s["v_cache"][slot].float().transpose(1, 2).contiguous()
    j = torch.arange(m, device=dev)
    q = s["q"][(cu[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)].float()    # [B, m, nh, hd]
    q = q.view(b, m, nkv, nh // nkv, hd).transpose(1, 2).reshape(b, nkv, -1, hd)
    last = (kv_len - (cu[1:] - cu[:-1]))[:, None] + j if c["causal"] else (kv_len - 1)[:, None].expand(b, m)
    seen = held[:, None] & (key <= last[:, :, None])                          # [B, m, L]
    out = _attend(q, k, v, seen.repeat_interleave(nh // nkv, 1)[:, None], s["scale"])
    out = out.view(b, nkv, m, nh // nkv, hd).transpose(1, 2).reshape(b, m, nh, hd)
    t = torch.arange(s["q"].shape[0], device=dev)
    of = (t[:, None] >= cu[None, 1:]).sum(1)
    s["out"].copy_(out[of, t - cu[of]])
    return s["out"]


def _prompt_plain(s):
    c = s["case"]
    nh, nkv, hd, b = c["nh"], c["nkv"], c["hd"], c["batch"]
    dev, cu, n = s["q"].device, s["cu"].long(), s["max_len"]
    j = torch.arange(n, device=dev)
    at = (cu[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)                   # [B, L]
    k = s["k"][at].float().transpose(1, 2).contiguous()
    v = s["v"][at].float().transpose(1, 2).contiguous()
    q = s["q"][at].float().view(b, n, nkv, nh // nkv, hd).permute(0, 2, 3, 1, 4).reshape(b, nkv, -1, hd)
    seen = (j < (cu[1:] - cu[:-1])[:, None])[:, None].expand(b, n, n)
    if c["causal"]:
        seen = seen & (j[None] <= j[:, None])
    out = _attend(q, k, v, seen.repeat(1, nh // nkv, 1)[:, None], s["scale"])
    out = out.view(b, nh, n, hd)                                              # heads in their own order
    t = torch.arange(s["q"].shape[0], device=dev)
    of = (t[:, None] >= cu[None, 1:]).sum(1)
    s["out"].copy_(out[of, :, t - cu[of]])
    return s["out"]


# ---------------------------------------------------------------- the definition, in 64 bits

def _softmax_rows(q, k, v, first, scale):
    """Rows of q over k, v; row r sees the keys 0 .. first + r (all of them where first is None)."""
    w = (q @ k.T.contiguous()) * scale
    if first is not None:
        rows = torch.arange(q.shape[0], device=q.device)[:, None] + first
        w = w.masked_fill(torch.arange(k.shape[0], device=q.device)[None] > rows, -math.inf)
    return torch.softmax(w, -1) @ v


def exact(case, seed):
    s = prepare(case, seed)
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    if case["op"] == "append":
        i = torch.arange(hd // 2, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["positions"].double()[:, None, None] * torch.exp(i * (-2 * math.log(THETA) / hd)))

        def rotated(x, w):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()
            z = torch.complex(x[..., :hd // 2].contiguous(), x[..., hd // 2:].contiguous()) * turn
            return torch.cat((z.real, z.imag), -1)

        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        k = rotated(s["k"], s["kw"])
        kc[s["slots"]], vc[s["slots"]] = k, s["v"].double()
        out = dict(q=rotated(s["q"], s["qw"]), k_cache=kc, v_cache=vc)
        if case["keys_out"]:
            out["k"] = k
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "paged":
        lens, kv = _lengths(case)
        page = case["page"]
        kp, vp = s["k_cache"].view(-1, page, nkv, hd), s["v_cache"].view(-1, page, nkv, hd)
        begin = 0
        for b, (nq, nk) in enumerate(zip(lens, kv)):
            pages = s["page_table"][b, :-(-nk // page)].long()
            k, v = kp[pages].reshape(-1, nkv, hd)[:nk].double(), vp[pages].reshape(-1, nkv, hd)[:nk].double()
            for h in range(nh):
                g = h // (nh // nkv)
                out[begin:begin + nq, h] = _softmax_rows(s["q"][begin:begin + nq, h].double(), k[:, g].contiguous(),
                                                         v[:, g].contiguous(), nk - nq if case["causal"] else None,
                                                         s["scale"])
            begin += nq
        return out
    begin = 0
    for n in _lengths(case):
        end = begin + n
        for h in range(nh):
            g = h // (nh // nkv)
            out[begin:end, h] = _softmax_rows(s["q"][begin:end, h].double(), s["k"][begin:end, g].double(),
                                              s["v"][begin:end, g].double(), 0 if case["causal"] else None, s["scale"])
        begin = end
    return out
