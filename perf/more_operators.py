"""Cases of serving long contexts from the 4-bit cache, and what they are measured against.

Three operators, each through the package's public calls:

  prefix_attend  attention of a few new queries per sequence over a prefix that the whole
                 batch shares and over each sequence's own pages
  cache_weigh    the attention weight that every cached token gets from the new queries,
                 added to what it has had so far
  cache_evict    every head of a sequence that has outgrown its budget keeps its first
                 tokens, its newest ones and those with the most weight, moved to the
                 front of the sequence's pages

``run`` computes either the plain form (elementary torch operations) or the calls a user
makes, according to ``own``.  The 4-bit cache is the same bytes in both: pages of 32 tokens,
[pages][Hkv][bytes], and in a page of one head K codes [32][d_h/2], V codes [32][d_v/2],
K words [32][d_h/64], V words [32][d_v/64].  Byte i of a row of codes holds element 2i in its
low and 2i+1 in its high half; the 32-bit word of 64 elements holds the bf16 scale s in its
upper half and the zero point z in its lowest byte; an element is s (code - z).
"""
import math

import torch

own = False

PAGE = 32      # tokens in a page
GROUP = 64     # elements that share a scale and a zero point


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # Two sequences behind one short instruction: the latency of a call.
        {"name": "prefix_attend_short", "op": "prefix_attend", "B": 2, "Hq": 8, "Hk": 2, "nq": 1, "dh": 64, "dv": 64,
         "prefix": 500, "lo": 1, "hi": 40},
        # A decode step of 32 conversations that share a system prompt, the heads of the GQA workload.
        {"name": "prefix_attend_gqa", "op": "prefix_attend", "B": 32, "Hq": 32, "Hk": 8, "nq": 1, "dh": 128, "dv": 128,
         "prefix": 8192, "lo": 64, "hi": 1024},
        # Questions on one long document: 64 answers in progress behind 32768 shared tokens.
        {"name": "prefix_attend_document", "op": "prefix_attend", "B": 64, "Hq": 32, "Hk": 8, "nq": 1, "dh": 128,
         "dv": 128, "prefix": 32768, "lo": 16, "hi": 2048},
        # Four proposed tokens per sequence, an odd prefix, very different lengths, values narrower than keys.
        {"name": "prefix_attend_ragged", "op": "prefix_attend", "B": 24, "Hq": 16, "Hk": 4, "nq": 4, "dh": 128,
         "dv": 64, "prefix": 5001, "lo": 4, "hi": 3000},
        # All query heads on one key head, the heads of the MQA workload: samples drawn from one prompt.
        {"name": "prefix_attend_mqa", "op": "prefix_attend", "B": 16, "Hq": 64, "Hk": 1, "nq": 1, "dh": 128, "dv": 128,
         "prefix": 16384, "lo": 1, "hi": 300},
        # A single short sequence: the latency of a call.
        {"name": "cache_weigh_short", "op": "cache_weigh", "B": 1, "Hq": 8, "Hk": 1, "nq": 1, "dh": 64, "dv": 64,
         "lo": 700, "hi": 700},
        # Eight long sequences, the sizes of the GQA decode workload.
        {"name": "cache_weigh_gqa", "op": "cache_weigh", "B": 8, "Hq": 32, "Hk": 8, "nq": 1, "dh": 128, "dv": 128,
         "lo": 16384, "hi": 32768},
        # Four proposed tokens of each of 48 sequences of very different lengths, values narrower than keys.
        {"name": "cache_weigh_ragged", "op": "cache_weigh", "B": 48, "Hq": 16, "Hk": 4, "nq": 4, "dh": 128, "dv": 64,
         "lo": 4, "hi": 12000},
        # A few sequences a token past a small budget: the latency of a call.
        {"name": "cache_evict_one", "op": "cache_evict", "B": 4, "Hk": 2, "dh": 64, "dv": 64, "lo": 513, "hi": 513,
         "keep": 512, "first": 4, "recent": 64},
        # A full batch in steady state: up to a page of new tokens past the budget.
        {"name": "cache_evict_steady", "op": "cache_evict", "B": 64, "Hk": 8, "dh": 128, "dv": 128, "lo": 4097,
         "hi": 4128, "keep": 4096, "first": 4, "recent": 256},
        # Long prompts cut to their budget after the prefill.
        {"name": "cache_evict_prompt", "op": "cache_evict", "B": 8, "Hk": 8, "dh": 128, "dv": 128, "lo": 16384,
         "hi": 32768, "keep": 4096, "first": 16, "recent": 512},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix_attend", "prefix_attend", "cache_weigh", "cache_evict"])
    dh, dv = rng.choice([(64, 64), (128, 128), (128, 64)])
    Hk = rng.choice([1, 2, 3, 4, 8])
    if op == "cache_evict":
        B = _log(rng, 1, 64)
        hi = _log(rng, 40, min(32768, 2000000 // (B * Hk)))
        keep = _log(rng, max(8, hi // 16), hi)
        return {"op": op, "B": B, "Hk": Hk, "dh": dh, "dv": dv, "lo": rng.choice([1, (hi + 1) // 2, hi]), "hi": hi,
                "keep": keep, "first": rng.choice([0, 1, 4, keep // 8]),
                "recent": rng.choice([0, 1, 3, keep // 16, keep // 3])}
    group = rng.choice([1, 2, 4, 5, 8])
    nq = rng.choice([1, 1, 1, 2, 3, 5])
    B = _log(rng, 1, 64)
    case = {"op": op, "B": B, "Hq": Hk * group, "Hk": Hk, "nq": nq, "dh": dh, "dv": dv}
    if op == "prefix_attend":
        case["prefix"] = _log(rng, 1, min(32768, 60000000 // (B * Hk * group * nq)))
        hi = _log(rng, nq, max(nq, min(4096, 800000 // (B * Hk))))
    else:
        hi = _log(rng, 33, min(60000, 1000000 // (B * Hk)))
    case["lo"], case["hi"] = rng.choice([nq, max(nq, hi // 2), hi]), hi
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _channels(g, d):
    """Channel scales of a projection's output: around 1, and a few that stand out."""
    s = torch.exp(0.3 * _randn(g, d))
    s[torch.randint(0, d, (max(1, d // 32),), generator=g, device="cuda")] *= 6.0
    return s


def _pack(x):
    """Code bytes [..., d/2] and word bytes [..., d/16] of rows x [..., d] rounded to 4 bits."""
    x = x.float().unflatten(-1, (-1, GROUP))
    lo = x.amin(-1, keepdim=True).clamp(max=0.0)
    hi = x.amax(-1, keepdim=True).clamp(min=0.0)
    s = ((hi - lo) / 15.0).to(torch.bfloat16).float()
    one = torch.where(s > 0, s, torch.ones_like(s))
    z = torch.round(-lo / one).clamp(max=15.0)
    c = (torch.round(x / one) + z).clamp(0.0, 15.0).to(torch.uint8).flatten(-2)
    sb = s.to(torch.bfloat16).view(torch.uint8)
    zb = torch.cat([z.to(torch.uint8), torch.zeros_like(z, dtype=torch.uint8)], -1)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([zb, sb], -1).flatten(-2)


def _page_bytes(dh, dv):
    return PAGE * (dh // 2 + dv // 2 + dh // 16 + dv // 16)


def _fields(pool, dh, dv):
    """Views of a pool [pages, Hk, bytes]: K codes, V codes, K words, V words, each [pages, Hk, 32, ...]."""
    at, out = 0, []
    for w in (dh // 2, dv // 2, dh // 16, dv // 16):
        out.append(pool[..., at:at + PAGE * w].unflatten(-1, (PAGE, w)))
        at += PAGE * w
    return out


def _fill(g, pool, dh, dv):
    """Every page of the pool filled with tokens, some pages at a time."""
    pages, Hk = pool.shape[:2]
    kc, vc, kw, vw = _fields(pool, dh, dv)
    ck = _channels(g, dh)
    at_once = max(1, (1 << 27) // (Hk * PAGE * (dh + dv)))
    for p in range(0, pages, at_once):
        n = min(at_once, pages - p)
        for codes, words, d, scales in ((kc, kw, dh, ck), (vc, vw, dv, None)):
            x = _randn(g, n, Hk, PAGE, d)
            codes[p:p + n], words[p:p + n] = _pack((x if scales is None else x * scales).to(torch.bfloat16))


def prepare(case, seed):
    g = _gen(seed)
    op, B, Hk, dh, dv, lo, hi = (case[k] for k in ("op", "B", "Hk", "dh", "dv", "lo", "hi"))
    s = {"case": case}
    lengths = torch.randint(lo, hi + 1, (B,), generator=g, device="cuda")
    wide = -(-hi // PAGE)
    shared = -(-case.get("prefix", 0) // PAGE)
    pages = shared + B * wide + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    s["pool"] = torch.zeros((pages, Hk, _page_bytes(dh, dv)), dtype=torch.uint8, device="cuda")
    _fill(g, s["pool"], dh, dv)
    s["table"] = order[shared:shared + B * wide].view(B, wide).contiguous()
    s["lengths"] = lengths.to(torch.int32)
    if op == "prefix_attend":
        s["prefix_table"] = order[:shared].contiguous()
        s["prefix_length"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
    if op != "cache_evict":
        s["Q"] = _randn(g, B, case["Hq"], case["nq"], dh).to(torch.bfloat16)
    if op == "cache_weigh":
        # Every row's log-sum-exp, as the attention over the same tokens left it; weights of some steps before.
        seen = torch.arange(wide * PAGE, device="cuda") < lengths[:, None, None] - case["nq"]
        s["LSE"] = _scores(s, case)[1].contiguous()
        s["weights"] = torch.where(seen, torch.exp(2.0 * _randn(g, B, Hk, wide * PAGE) - 6.0), 0.0).contiguous()
    if op == "cache_evict":
        # Accumulated weights: a few tokens have most of it, some have had none yet (ties).
        w = torch.exp(2.0 * _randn(g, B, Hk, wide * PAGE) - 4.0)
        w = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.02, 0.0, w)
        s["weights"] = torch.where(torch.arange(wide * PAGE, device="cuda") < lengths[:, None, None], w, 0.0).contiguous()
    return s


# ---------------------------------------------------------------------------
# Plain forms (fp32, one rounding at the end)
# ---------------------------------------------------------------------------
def _values(codes, words):
    """fp32 elements of rows of code bytes [..., d/2] and word bytes [..., d/16]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    w = words.unflatten(-1, (-1, 4))
    s = w[..., 2:4].contiguous().view(torch.bfloat16).float()
    return (s * (c - w[..., 0:1].float())).flatten(-2)


def _rows(pool, case, table, values):
    """fp32 keys (or values) [..., Hk, tokens, d] of the pages of table [..., pages]."""
    f = _fields(pool, case["dh"], case["dv"])
    at = table.long()
    x = _values(f[1][at], f[3][at]) if values else _values(f[0][at], f[2][at])
    return x.transpose(-4, -3).flatten(-3, -2)


def _scores(s, case):
    """Scores of the rows over their sequences' own keys [B, Hk, rows of a head, keys] (-inf where hidden), and their LSE."""
    B, Hq, nq, dh = s["Q"].shape
    K = _rows(s["pool"], case, s["table"], False)
    Hk, n = K.shape[1], K.shape[2]
    S = torch.matmul(s["Q"].float().reshape(B, Hk, -1, dh), K.transpose(-1, -2)).view(B, Hk, -1, nq, n) / math.sqrt(dh)
    last = s["lengths"].long()[:, None] - nq + torch.arange(nq, device=S.device)     # the last key that a row sees
    seen = torch.arange(n, device=S.device) <= last[..., None]
    S = S.masked_fill(~seen[:, None, None], -math.inf)
    return S.flatten(2, 3), torch.logsumexp(S, -1).view(B, Hq, nq)


def _prefix_attend_plain(s, case):
    B, Hq, nq, dh = s["Q"].shape
    dv, n = case["dv"], case["prefix"]
    S = _scores(s, case)[0]
    Hk = S.shape[1]
    Kp, Vp = (_rows(s["pool"], case, s["prefix_table"], v)[:, :n] for v in (False, True))       # [Hk, prefix, d]
    q = s["Q"].float().reshape(B, Hk, -1, dh).transpose(0, 1).flatten(1, 2)                       # [Hk, B rows, dh]
    P = torch.matmul(q, Kp.transpose(-1, -2)) / math.sqrt(dh)
    P = P.view(Hk, B, -1, n).transpose(0, 1)                                                     # [B, Hk, rows, prefix]
    m = torch.maximum(S.amax(-1, keepdim=True), P.amax(-1, keepdim=True))
    S, P = torch.exp(S - m), torch.exp(P - m)
    l = S.sum(-1, keepdim=True) + P.sum(-1, keepdim=True)
    O = torch.matmul(P.transpose(0, 1).reshape(Hk, -1, n), Vp).view(Hk, B, -1, dv).transpose(0, 1)
    O = (O + torch.matmul(S, _rows(s["pool"], case, s["table"], True))) / l
    return [O.reshape(B, Hq, nq, dv).to(torch.bfloat16), (m + torch.log(l)).reshape(B, Hq, nq)]


def _cache_weigh_plain(s, case):
    S = _scores(s, case)[0]
    P = torch.exp(S - s["LSE"].view(S.shape[:3])[..., None])
    s["weights"] += torch.where(S == -math.inf, torch.zeros_like(P), P).sum(2)
    return [s["weights"]]


def _first_true(mask):
    """The places of a mask's true entries [..., n], ascending, then those of the others."""
    return torch.sort((~mask).to(torch.uint8), dim=-1, stable=True).indices


def _cache_evict_plain(s, case):
    pool, w, keep, first, recent = s["pool"], s["weights"], case["keep"], case["first"], case["recent"]
    B, Hk, cap = w.shape
    j = torch.arange(cap, device=w.device)
    n = s["lengths"].long()[:, None, None]
    m = n.clamp(max=keep)
    over = n > keep
    # The middle tokens in the order of their weights, equal ones by place; the first of them stay.
    middle = (j >= first) & (j < n - recent)
    by_weight = torch.sort(w, dim=-1, descending=True, stable=True).indices
    order = by_weight.gather(-1, _first_true(middle.expand_as(w).gather(-1, by_weight)))
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order).contiguous())
    stay = torch.where(over, torch.where(middle, rank < keep - first - recent, j < n), j < n)
    # Places below m - recent that became free take the tokens from behind; the newest follow in order.
    hole = over & ~stay & (j < m - recent)
    mover = over & stay & (j >= m - recent) & (j < n - recent)
    places = torch.where(j < m, torch.where(over & (j >= m - recent), j + n - m, j), -1).expand_as(w).contiguous()
    to, frm = _first_true(hole), _first_true(mover)
    moved = j < hole.sum(-1, keepdim=True)
    spare = torch.full_like(places[..., :1], -1)
    places = torch.cat([places, spare], -1).scatter_(-1, torch.where(moved, to, cap), frm)[..., :cap]
    new_weights = torch.where(places >= 0, w.gather(-1, places.clamp(min=0)), 0.0)
    # The tokens whose place changes, as bytes, all read before any is written.
    b, h, to = torch.nonzero((places >= 0) & (places != j), as_tuple=True)
    at = places[b, h, to]
    page_of = lambda x: s["table"].long()[b, x // PAGE]  # noqa: E731
    for f in _fields(pool, case["dh"], case["dv"]):
        f[page_of(to), h, to % PAGE] = f[page_of(at), h, at % PAGE]
    kept = torch.nn.functional.pad(places, (0, max(0, keep - cap)), value=-1)[..., :keep]
    return [m.view(B).to(torch.int32), new_weights, kept.to(torch.int32), pool]


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "prefix_attend":
        return _prefix_attend_plain(s, case)
    if case["op"] == "cache_weigh":
        return _cache_weigh_plain(s, case)
    return _cache_evict_plain(s, case)


# ---------------------------------------------------------------------------
# The calls a user makes
# ---------------------------------------------------------------------------
def _run_own(s, case):
    import exact_scaled_dot_gb300 as esd
    cache = esd.QuantCache(s["pool"], case["dh"], case["dv"])
    if case["op"] == "prefix_attend":
        return list(esd.attn_fwd_prefix_cache(s["Q"], cache, s["prefix_table"], s["prefix_length"], s["table"],
                                              s["lengths"]))
    if case["op"] == "cache_weigh":
        return [esd.attn_cache_weigh(s["Q"], cache, s["table"], s["lengths"], s["LSE"], s["weights"])]
    # The pool is the state's own; a move neither rounds nor computes, so that it comes back as its bytes.
    return list(esd.attn_cache_evict(cache, s["table"], s["lengths"], s["weights"], case["keep"], first=case["first"],
                                     recent=case["recent"])) + [s["pool"]]


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, B, Hk, dh, dv = (case[k] for k in ("op", "B", "Hk", "dh", "dv"))
    token = (dh + dv) // 2 + (dh + dv) // 16          # bytes of one head
    mean = (case["lo"] + case["hi"]) / 2
    cap = -(-case["hi"] // PAGE) * PAGE
    table = 4 * B * (mean / PAGE + 1)
    if op == "cache_evict":
        keep, first, recent = case["keep"], case["first"], case["recent"]
        # A middle token behind the budget stays as often as any: it moves, and the newest move.
        over = max(0.0, mean - keep)
        middle = max(1.0, mean - first - recent)
        moves = over * min(1.0, (keep - first - recent) / middle) + (recent if over > 0 else 0)
        return {"bytes": B * Hk * (4 * mean + 4 * cap + 4 * keep + 2 * moves * token) + table,
                "flops": 4 * B * Hk * mean}
    rows = B * case["Hq"] * case["nq"]
    if op == "cache_weigh":
        return {"bytes": B * mean * Hk * (dh // 2 + dh // 16 + 8) + rows * (2 * dh + 4) + table,
                "flops": 2 * rows * mean * dh}
    keys = case["prefix"] + B * mean
    return {"bytes": keys * Hk * token + rows * (2 * dh + 2 * dv + 4) + table + case["prefix"] / 8,
            "flops": 2 * rows * (case["prefix"] + mean) * (dh + dv)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(s, case, pages):
    """Keys and values [Hk, tokens, d] in fp64 of the pages numbered `pages`."""
    dh, dv, Hk = case["dh"], case["dv"], case["Hk"]
    page = s["pool"][pages.long()].to(torch.int64)             # [pages, Hk, bytes]
    got, at = [], 0
    word_at = PAGE * (dh + dv) // 2
    for d in (dh, dv):
        code = page[..., at:at + PAGE * d // 2].reshape(-1, Hk, PAGE, d // 2)
        word = page[..., word_at:word_at + PAGE * d // 16].reshape(-1, Hk, PAGE, d // GROUP, 4)
        at, word_at = at + PAGE * d // 2, word_at + PAGE * d // 16
        nib = torch.stack([code % 16, code // 16], -1).reshape(-1, Hk, PAGE, d // GROUP, GROUP).double()
        bits = ((word[..., 3] * 256 + word[..., 2]) * 65536).to(torch.int32)      # an fp32 with bf16's bits on top
        v = (nib - word[..., :1].double()) * bits.view(torch.float32).double()[..., None]
        got.append(v.reshape(-1, Hk, PAGE, d).permute(1, 0, 2, 3).reshape(Hk, -1, d))
    return got


def _exact_own_scores(s, case, b, K):
    """Scores of sequence b's rows [Hk, group, nq, n] over its own keys."""
    n, nq, dh = K.shape[1], case["nq"], case["dh"]
    q = s["Q"][b].double().reshape(case["Hk"], -1, nq, dh)
    sc = torch.einsum("hgid,hjd->hgij", q, K) * dh ** -0.5
    hidden = torch.arange(n, device=sc.device)[None] > torch.arange(n - nq, n, device=sc.device)[:, None]
    return torch.where(hidden, torch.full_like(sc, -math.inf), sc)


def _exact_prefix_attend(s, case):
    """Sequence by sequence: softmax over the prefix and the sequence's own keys, put one behind the other."""
    nq, dh, dv, Hk = case["nq"], case["dh"], case["dv"], case["Hk"]
    Kp, Vp = (x[:, :case["prefix"]] for x in _exact_rows(s, case, s["prefix_table"]))
    O, L = [], []
    for b in range(case["B"]):
        n = int(s["lengths"][b])
        K, V = (x[:, :n] for x in _exact_rows(s, case, s["table"][b, :-(-n // PAGE)]))
        q = s["Q"][b].double().reshape(Hk, -1, nq, dh)
        sc = torch.cat([torch.einsum("hgid,hjd->hgij", q, Kp) * dh ** -0.5, _exact_own_scores(s, case, b, K)], -1)
        L.append(torch.logsumexp(sc, -1).reshape(-1, nq))
        O.append(torch.einsum("hgij,hjd->hgid", torch.softmax(sc, -1), torch.cat([Vp, V], 1)).reshape(-1, nq, dv))
    return [torch.stack(O), torch.stack(L)]


def _exact_cache_weigh(s, case):
    w = s["weights"].double()
    for b in range(case["B"]):
        n = int(s["lengths"][b])
        K = _exact_rows(s, case, s["table"][b, :-(-n // PAGE)])[0][:, :n]
        sc = _exact_own_scores(s, case, b, K)
        lse = s["LSE"][b].double().reshape(case["Hk"], -1, case["nq"], 1)
        w[b, :, :n] += torch.exp(sc - lse).sum((1, 2))
    return [w]


def _exact_cache_evict(s, case):
    """The weights that stay, head by head, from lists: sorted by weight, then the free places filled."""
    keep, first, recent = case["keep"], case["first"], case["recent"]
    w = s["weights"].double().cpu().numpy()
    out = w * 0.0
    for b, n in enumerate(s["lengths"].tolist()):
        m = min(n, keep)
        for h in range(case["Hk"]):
            if n <= keep:
                out[b, h, :n] = w[b, h, :n]
                continue
            mid = range(first, n - recent)
            best = (-w[b, h, first:n - recent]).argsort(kind="stable")[:keep - first - recent] + first
            chosen = set(best.tolist())
            free = [p for p in mid if p not in chosen and p < m - recent]
            late = [p for p in mid if p in chosen and p >= m - recent]
            out[b, h, :m - recent] = w[b, h, :m - recent]
            out[b, h, free] = w[b, h, late]
            out[b, h, m - recent:m] = w[b, h, n - recent:n]
    return [None, torch.from_numpy(out), None, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefix_attend":
        return _exact_prefix_attend(s, case)
    if case["op"] == "cache_weigh":
        return _exact_cache_weigh(s, case)
    return _exact_cache_evict(s, case)
