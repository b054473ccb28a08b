"""Cases of the operators around the attention kernels, and what they are measured against.

Five operators, each through the package's public calls:

  norm_rope      RMS norm of every query and key row over its head width, then the
                 rotation by the row's position, on one axis or several
  norm_rope_bwd  the gradients of its rows and of its two weight vectors
  rope_axes      the rotation alone, with several position axes (time, height, width)
  cache_write    keys and values of new tokens rounded to 4 bits into their cache slots,
                 and read back as the values that the cache now stands for
  cache_attend   attention of a few new queries per sequence over the 4-bit cache

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
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One decode step of eight sequences: queries and keys as slices of one fused projection.
        {"name": "norm_rope_step", "op": "norm_rope", "T": 8, "Hq": 32, "Hk": 8, "d": 128, "sections": "64",
         "restart": False, "fused": True, "base": 10000.0, "maxpos": 65536},
        # Two prompts of 4096 tokens, the heads and width of the causal GQA workload.
        {"name": "norm_rope_prompt", "op": "norm_rope", "T": 8192, "Hq": 32, "Hk": 8, "d": 128, "sections": "64",
         "restart": False, "fused": True, "base": 10000.0, "maxpos": 4096},
        # Image tokens with rows and columns of their own, an odd number of them, narrow heads.
        {"name": "norm_rope_image", "op": "norm_rope", "T": 4097, "Hq": 16, "Hk": 16, "d": 64, "sections": "16,16",
         "restart": True, "fused": False, "base": 10000.0, "maxpos": 256},
        # A short ragged training batch.
        {"name": "norm_rope_bwd_ragged", "op": "norm_rope_bwd", "T": 333, "Hq": 5, "Hk": 1, "d": 64, "sections": "32",
         "restart": False, "fused": False, "base": 500000.0, "maxpos": 131072},
        # A training step over 32768 tokens, the heads and width of the causal GQA workload.
        {"name": "norm_rope_bwd_train", "op": "norm_rope_bwd", "T": 32768, "Hq": 32, "Hk": 8, "d": 128,
         "sections": "64", "restart": False, "fused": True, "base": 10000.0, "maxpos": 4096},
        # A short clip with text: time, height and width share the frequencies of one row.
        {"name": "rope_axes_clip", "op": "rope_axes", "T": 1025, "Hq": 16, "Hk": 2, "d": 128, "sections": "16,24,24",
         "inverse": False, "restart": False, "fused": True, "base": 1000000.0, "maxpos": 2048},
        # Gradients of a long video turned back, all heads with keys of their own, part of the width turned.
        {"name": "rope_axes_video_grad", "op": "rope_axes", "T": 65537, "Hq": 16, "Hk": 16, "d": 128,
         "sections": "16,20,20", "inverse": True, "restart": True, "fused": False, "base": 10000.0, "maxpos": 512},
        # One new token of each of 64 sequences written to the cache.
        {"name": "cache_write_step", "op": "cache_write", "T": 64, "Hk": 8, "dh": 128, "dv": 128, "pages": 4096},
        # A prompt of 16384 tokens written to scattered pages.
        {"name": "cache_write_prompt", "op": "cache_write", "T": 16384, "Hk": 8, "dh": 128, "dv": 128, "pages": 4096},
        # A single short sequence: the latency of a call.
        {"name": "cache_attend_short", "op": "cache_attend", "B": 1, "Hq": 8, "Hk": 1, "nq": 1, "dh": 64, "dv": 64,
         "lo": 700, "hi": 700},
        # Decode of eight long sequences, the sizes of the GQA decode workload.
        {"name": "cache_attend_gqa", "op": "cache_attend", "B": 8, "Hq": 32, "Hk": 8, "nq": 1, "dh": 128, "dv": 128,
         "lo": 16384, "hi": 32768},
        # Four proposed tokens of each of 48 sequences of very different lengths, values narrower than keys.
        {"name": "cache_attend_ragged", "op": "cache_attend", "B": 48, "Hq": 16, "Hk": 4, "nq": 4, "dh": 128, "dv": 64,
         "lo": 4, "hi": 12000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "rope_axes", "cache_write", "cache_attend", "cache_attend"])
    if op == "cache_write":
        dh, dv = rng.choice([(64, 64), (128, 128), (128, 64)])
        return {"op": op, "T": _log(rng, 1, 16384), "Hk": rng.choice([1, 2, 3, 4, 8]), "dh": dh, "dv": dv,
                "pages": _log(rng, 520, 4096)}
    if op == "cache_attend":
        dh, dv = rng.choice([(64, 64), (128, 128), (128, 64)])
        Hk = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 5, 8])
        nq = rng.choice([1, 1, 1, 2, 3, 5])
        B = _log(rng, 1, 64)
        hi = _log(rng, 33, min(60000, 1000000 // (B * Hk)))
        return {"op": op, "B": B, "Hq": Hk * group, "Hk": Hk, "nq": nq, "dh": dh, "dv": dv,
                "lo": rng.choice([nq, max(nq, hi // 2), hi]), "hi": hi}
    d = rng.choice([32, 64, 64, 96, 128, 128, 128])
    half = d // 2
    axes = 1 if op != "rope_axes" and rng.random() < 0.5 else rng.choice([2, 3])
    cut = sorted(rng.sample(range(1, half), axes - 1))
    sections = [b - a for a, b in zip([0] + cut, cut + [half])]
    if rng.random() < 0.25 and sections[-1] > 1:
        sections[-1] -= rng.randint(1, sections[-1] - 1)     # the rest of the width is not turned
    Hk = rng.choice([1, 2, 3, 8])
    Hq = Hk * rng.choice([1, 2, 4])
    case = {"op": op, "T": _log(rng, 1, 1000000 // (Hq + Hk)), "Hq": Hq, "Hk": Hk, "d": d,
            "sections": ",".join(str(s) for s in sections), "restart": rng.random() < 0.5,
            "fused": rng.random() < 0.5, "base": rng.choice([10000.0, 500000.0, 1000000.0]),
            "maxpos": _log(rng, 100, 1000000)}
    if op == "rope_axes":
        case["inverse"] = rng.random() < 0.5
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


def _sections(case):
    return [int(s) for s in case["sections"].split(",")]


def _channels(g, d):
    """Channel scales of a projection's output: around 1, and a few that stand out."""
    s = torch.exp(0.3 * _randn(g, d))
    s[torch.randint(0, d, (max(1, d // 32),), generator=g, device="cuda")] *= 6.0
    return s


def _rows(case, g, T, Hq, Hk, d):
    """Queries and keys [T, H, d]: slices of one fused [T, (Hq + 2 Hk) d], or tensors of their own."""
    if case["fused"]:
        x = _randn(g, T, Hq + 2 * Hk, d)
        x *= _channels(g, d)
        x = x.to(torch.bfloat16)
        return x[:, :Hq], x[:, Hq:Hq + Hk]
    return ((_randn(g, T, Hq, d) * _channels(g, d)).to(torch.bfloat16),
            (_randn(g, T, Hk, d) * _channels(g, d)).to(torch.bfloat16))


def _quantize_plain(x):
    """Codes, scales and zero points of groups of 64 elements of x [..., d] (fp32 arithmetic)."""
    x = x.float().unflatten(-1, (-1, GROUP))
    lo = x.amin(-1, keepdim=True).clamp(max=0.0)
    hi = x.amax(-1, keepdim=True).clamp(min=0.0)
    s = ((hi - lo) / 15.0).to(torch.bfloat16).float()
    one = torch.where(s > 0, s, torch.ones_like(s))
    z = torch.round(-lo / one).clamp(max=15.0)
    c = (torch.round(x / one) + z).clamp(0.0, 15.0)
    c = torch.where(s > 0, c, torch.zeros_like(c))
    z = torch.where(s > 0, z, torch.zeros_like(z))
    return c.flatten(-2), s.squeeze(-1), z.squeeze(-1)


def _pack(c, s, z):
    """Code bytes [..., d/2] and word bytes [..., d/64, 4] of one row."""
    c = c.to(torch.uint8)
    codes = c[..., 0::2] | (c[..., 1::2] << 4)
    sb = s.to(torch.bfloat16).view(torch.uint8).unflatten(-1, (-1, 2))
    zb = torch.stack([z.to(torch.uint8), torch.zeros_like(z, dtype=torch.uint8)], -1)
    return codes, torch.cat([zb, sb], -1)


def _page_bytes(dh, dv):
    return PAGE * (dh // 2 + dv // 2 + dh // 16 + dv // 16)


def _fields(pool, dh, dv):
    """Views of a pool [pages, Hk, bytes]: K codes, V codes, K words, V words, each [pages, Hk, 32, ...]."""
    at, out = 0, []
    for w in (dh // 2, dv // 2, dh // 16, dv // 16):
        out.append(pool[..., at:at + PAGE * w].unflatten(-1, (PAGE, w)))
        at += PAGE * w
    return out


def _store(pool, page, off, K, V):
    """Rows K, V [n, Hk, d] rounded to 4 bits into slots (page, off) of the pool."""
    kc, vc, kw, vw = _fields(pool, K.shape[-1], V.shape[-1])
    for x, codes, words in ((K, kc, kw), (V, vc, vw)):
        c, w = _pack(*_quantize_plain(x))
        codes[page, :, off] = c
        words[page, :, off] = w.flatten(-2)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "cache_write":
        T, Hk, dh, dv, pages = (case[k] for k in ("T", "Hk", "dh", "dv", "pages"))
        s["pool"] = torch.zeros((pages, Hk, _page_bytes(dh, dv)), dtype=torch.uint8, device="cuda")
        s["K"] = (_randn(g, T, Hk, dh) * _channels(g, dh)).to(torch.bfloat16)
        s["V"] = _randn(g, T, Hk, dv).to(torch.bfloat16)
        # A prompt fills pages taken from anywhere in the pool; its last page ends in the middle.
        n = -(-T // PAGE)
        order = torch.randperm(pages, generator=g, device="cuda")[:n]
        t = torch.arange(T, device="cuda")
        s["slots"] = order[t // PAGE] * PAGE + t % PAGE
        return s
    if op == "cache_attend":
        B, Hq, Hk, nq, dh, dv, lo, hi = (case[k] for k in ("B", "Hq", "Hk", "nq", "dh", "dv", "lo", "hi"))
        lengths = torch.randint(lo, hi + 1, (B,), generator=g, device="cuda")
        wide = -(-hi // PAGE)
        pages = B * wide + 3
        table = torch.randperm(pages, generator=g, device="cuda")[:B * wide].view(B, wide)
        s["pool"] = torch.zeros((pages, Hk, _page_bytes(dh, dv)), dtype=torch.uint8, device="cuda")
        off = torch.arange(PAGE, device="cuda").repeat(wide)
        ck = _channels(g, dh)
        for b in range(B):
            _store(s["pool"], table[b].repeat_interleave(PAGE), off, (_randn(g, wide * PAGE, Hk, dh) * ck).to(torch.bfloat16),
                   _randn(g, wide * PAGE, Hk, dv).to(torch.bfloat16))
        s["Q"] = _randn(g, B, Hq, nq, dh).to(torch.bfloat16)
        s["table"] = table.to(torch.int32).contiguous()
        s["lengths"] = lengths.to(torch.int32)
        return s
    T, Hq, Hk, d = (case[k] for k in ("T", "Hq", "Hk", "d"))
    s["Q"], s["K"] = _rows(case, g, T, Hq, Hk, d)
    s["pos"] = torch.randint(0, case["maxpos"], (len(_sections(case)), T), generator=g, device="cuda", dtype=torch.int32)
    if op != "rope_axes":
        s["gq"] = (1.0 + 0.2 * _randn(g, d)).to(torch.bfloat16)
        s["gk"] = (1.0 + 0.2 * _randn(g, d)).to(torch.bfloat16)
    if op == "norm_rope_bwd":
        s["dYq"] = (0.1 * _randn(g, T, Hq, d)).to(torch.bfloat16)
        s["dYk"] = (0.1 * _randn(g, T, Hk, d)).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# Plain forms (fp32, angles in fp64, one rounding at the end)
# ---------------------------------------------------------------------------
def _angles(case, pos, d):
    """cos and sin [T, 1, d/2] in fp32: block k of section a turns by pos[a] w_k."""
    sec = torch.tensor(_sections(case), device=pos.device)
    axis = torch.repeat_interleave(torch.arange(len(sec), device=pos.device), sec)
    n = axis.numel()
    k = torch.arange(n, device=pos.device)
    first = (torch.cumsum(sec, 0) - sec)[axis]
    if case["restart"]:
        power = (k - first).double() / sec[axis].double()
    else:
        power = 2.0 * k.double() / d
    a = pos.double()[axis].T * torch.pow(torch.tensor(case["base"], dtype=torch.float64, device=pos.device), -power)
    a = torch.nn.functional.pad(a, (0, d // 2 - n))
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _turn(x, c, s):
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * c - x1 * s, x0 * s + x1 * c], -1).flatten(-2)


def _norm_rope_plain(x, g, c, s):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return _turn(x * r * g.float(), c, s).to(torch.bfloat16)


def _norm_rope_bwd_plain(x, g, dy, c, s):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * r
    u = _turn(dy.float(), c, -s)
    dg = (u * n).sum((0, 1))
    u = u * g.float()
    dx = r * (u - n * (u * n).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), dg


def _values(codes, words):
    """fp32 elements of rows of code bytes [..., d/2] and word bytes [..., d/16]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    w = words.unflatten(-1, (-1, 4))
    s = w[..., 2:4].contiguous().view(torch.bfloat16).float()
    return (s * (c - w[..., 0:1].float())).flatten(-2)


def _attend_plain(s, pool, table, lengths, dh, dv):
    Q = s["Q"].float()
    B, Hq, nq, _ = Q.shape
    kc, vc, kw, vw = _fields(pool, dh, dv)
    at = table.long()

    def rows(codes, words):
        x = _values(codes[at], words[at])                     # [B, pages, Hk, 32, d]
        return x.transpose(1, 2).flatten(2, 3)                # [B, Hk, keys, d]

    K, V = rows(kc, kw), rows(vc, vw)
    Hk, n = K.shape[1], K.shape[2]
    S = torch.matmul(Q.reshape(B, Hk, -1, dh), K.transpose(-1, -2)).view(B, Hk, -1, nq, n) / math.sqrt(dh)
    last = lengths.long()[:, None] - nq + torch.arange(nq, device=Q.device)          # the last key that a row sees
    seen = torch.arange(n, device=Q.device) <= last[..., None]
    S = S.masked_fill(~seen[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    p = torch.exp(S - torch.where(m == -math.inf, torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    O = torch.matmul(p.view(B, Hk, -1, n), V).view(B, Hk, -1, nq, dv) / torch.where(l > 0, l, torch.ones_like(l))
    return O.view(B, Hq, nq, dv).to(torch.bfloat16), (m + torch.log(l)).view(B, Hq, nq)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _run_own(s, case, op)
    if op == "cache_write":
        page, off = s["slots"] // PAGE, s["slots"] % PAGE
        _store(s["pool"], page, off, s["K"], s["V"])
        kc, vc, kw, vw = _fields(s["pool"], case["dh"], case["dv"])
        return [_values(kc[page, :, off], kw[page, :, off]).to(torch.bfloat16),
                _values(vc[page, :, off], vw[page, :, off]).to(torch.bfloat16)]
    if op == "cache_attend":
        return list(_attend_plain(s, s["pool"], s["table"], s["lengths"], case["dh"], case["dv"]))
    c, sn = _angles(case, s["pos"], case["d"])
    if op == "norm_rope":
        return [_norm_rope_plain(s["Q"], s["gq"], c, sn), _norm_rope_plain(s["K"], s["gk"], c, sn)]
    if op == "norm_rope_bwd":
        dq, dgq = _norm_rope_bwd_plain(s["Q"], s["gq"], s["dYq"], c, sn)
        dk, dgk = _norm_rope_bwd_plain(s["K"], s["gk"], s["dYk"], c, sn)
        return [dq, dk, dgq, dgk]
    if case["inverse"]:
        sn = -sn
    return [_turn(s["Q"].float(), c, sn).to(torch.bfloat16), _turn(s["K"].float(), c, sn).to(torch.bfloat16)]


# ---------------------------------------------------------------------------
# The calls a user makes
# ---------------------------------------------------------------------------
def _run_own(s, case, op):
    import exact_scaled_dot_gb300 as esd
    if op == "cache_write":
        cache = esd.QuantCache(s["pool"], case["dh"], case["dv"])
        esd.attn_cache_append(cache, s["K"], s["V"], s["slots"])
        return list(esd.attn_cache_read(cache, s["slots"]))
    if op == "cache_attend":
        cache = esd.QuantCache(s["pool"], case["dh"], case["dv"])
        return list(esd.attn_fwd_decode_cache(s["Q"], cache, s["table"], s["lengths"]))
    rot = esd.RotaryAxes(s["pos"], _sections(case), base=case["base"], restart=case["restart"])
    if op == "norm_rope":
        return list(esd.attn_qk_norm_rope(s["Q"], s["K"], s["gq"], s["gk"], rot, eps=EPS))
    if op == "norm_rope_bwd":
        return list(esd.attn_qk_norm_rope_bwd(s["Q"], s["K"], s["gq"], s["gk"], s["dYq"], s["dYk"], rot, eps=EPS))
    return list(esd.attn_rope_axes(s["Q"], s["K"], rot, inverse=case["inverse"]))


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "cache_write":
        T, Hk, d = case["T"], case["Hk"], case["dh"] + case["dv"]
        packed = d // 2 + d // 16
        return {"bytes": T * Hk * (2 * d + packed + packed + 2 * d) + 16 * T, "flops": 6 * T * Hk * d}
    if op == "cache_attend":
        B, Hq, Hk, nq, dh, dv = (case[k] for k in ("B", "Hq", "Hk", "nq", "dh", "dv"))
        keys = B * (case["lo"] + case["hi"]) // 2
        return {"bytes": keys * Hk * ((dh + dv) // 2 + (dh + dv) // 16) + B * Hq * nq * (2 * dh + 2 * dv + 4)
                + 4 * (keys // PAGE + B), "flops": 2 * keys * Hq * nq * (dh + dv)}
    T, rows, d = case["T"], case["T"] * (case["Hq"] + case["Hk"]), case["d"]
    pos = 4 * T * len(_sections(case))
    if op == "norm_rope_bwd":
        return {"bytes": 6 * rows * d + pos + 12 * d, "flops": 14 * rows * d}
    if op == "norm_rope":
        return {"bytes": 4 * rows * d + pos + 4 * d, "flops": 7 * rows * d}
    return {"bytes": 4 * rows * d + pos, "flops": 3 * rows * d}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _rotation64(case, pos):
    """Complex numbers e^{i a} [T, 1, d/2], one for each block of two elements."""
    d, parts, first = case["d"], [], 0
    for axis, width in enumerate(_sections(case)):
        k = torch.arange(width, dtype=torch.float64, device=pos.device)
        w = case["base"] ** (-(k / width)) if case["restart"] else case["base"] ** (-2.0 * (k + first) / d)
        parts.append(torch.polar(torch.ones((pos.shape[1], width), dtype=torch.float64, device=pos.device),
                                 pos[axis].double()[:, None] * w))
        first += width
    parts.append(torch.ones((pos.shape[1], d // 2 - first), dtype=torch.complex128, device=pos.device))
    return torch.cat(parts, 1)[:, None]


def _blocks(x):
    return torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous())


def _flat(z):
    return torch.view_as_real(z).flatten(-2)


def _exact_norm_rope(x, g, R):
    x = x.double()
    return _flat(_blocks(x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * g.double()) * R)


def _exact_norm_rope_bwd(x, g, dy, R):
    """From d(x_i / rms) = dx_i / rms - x_i (x . dx) / (d rms^3)."""
    x, g = x.double(), g.double()
    rms = torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    u = _flat(_blocks(dy) * R.conj())
    dg = torch.einsum("thd,thd->d", u, x / rms)
    u = u * g
    return u / rms - x * (x * u).sum(-1, keepdim=True) / (x.shape[-1] * rms ** 3), dg


def _exact_4bit(x):
    """What a row stands for once its groups of 64 are rounded to 4 bits."""
    x = x.double()
    out = torch.empty_like(x)
    for a in range(0, x.shape[-1], GROUP):
        v = x[..., a:a + GROUP]
        low = torch.minimum(v.min(-1, keepdim=True).values, torch.zeros((), dtype=v.dtype, device=v.device))
        high = torch.maximum(v.max(-1, keepdim=True).values, torch.zeros((), dtype=v.dtype, device=v.device))
        step = ((high - low) / 15).to(torch.bfloat16).double()
        div = torch.where(step == 0, torch.ones_like(step), step)
        zero = torch.clamp(torch.round(-low / div), max=15)
        out[..., a:a + GROUP] = step * (torch.clamp(torch.round(v / div) + zero, 0, 15) - zero)
    return out


def _exact_attend(s, case):
    """Sequence by sequence: the pages put together, softmax over the keys that each row sees."""
    dh, dv, Hk, nq = case["dh"], case["dv"], case["Hk"], case["nq"]
    raw = s["pool"].to(torch.int64)
    O, L = [], []
    for b in range(case["B"]):
        n = int(s["lengths"][b])
        page = raw[s["table"][b, :-(-n // PAGE)].long()]       # [pages, Hk, bytes]
        KV, at = [], 0
        word_at = PAGE * (dh + dv) // 2
        for d in (dh, dv):
            code = page[..., at:at + PAGE * d // 2].reshape(-1, Hk, PAGE, d // 2)
            word = page[..., word_at:word_at + PAGE * d // 16].reshape(-1, Hk, PAGE, d // GROUP, 4)
            at, word_at = at + PAGE * d // 2, word_at + PAGE * d // 16
            nib = torch.stack([code % 16, code // 16], -1).reshape(-1, Hk, PAGE, d // GROUP, GROUP).double()
            bits = ((word[..., 3] * 256 + word[..., 2]) * 65536).to(torch.int32)      # an fp32 with bf16's bits on top
            v = (nib - word[..., :1].double()) * bits.view(torch.float32).double()[..., None]
            KV.append(v.reshape(-1, Hk, PAGE, d).permute(1, 0, 2, 3).reshape(Hk, -1, d)[:, :n])
        q = s["Q"][b].double().reshape(Hk, -1, nq, dh)
        sc = torch.einsum("hgid,hjd->hgij", q, KV[0]) * dh ** -0.5
        hidden = torch.arange(n, device=sc.device)[None] > torch.arange(n - nq, n, device=sc.device)[:, None]
        sc = torch.where(hidden, torch.full_like(sc, -math.inf), sc)
        L.append(torch.logsumexp(sc, -1).reshape(-1, nq))
        O.append(torch.einsum("hgij,hjd->hgid", torch.softmax(sc, -1), KV[1]).reshape(-1, nq, dv))
    return [torch.stack(O), torch.stack(L)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "cache_write":
        return [_exact_4bit(s["K"]), _exact_4bit(s["V"])]
    if op == "cache_attend":
        return _exact_attend(s, case)
    R = _rotation64(case, s["pos"])
    if op == "norm_rope":
        return [_exact_norm_rope(s["Q"], s["gq"], R), _exact_norm_rope(s["K"], s["gk"], R)]
    if op == "norm_rope_bwd":
        dq, dgq = _exact_norm_rope_bwd(s["Q"], s["gq"], s["dYq"], R)
        dk, dgk = _exact_norm_rope_bwd(s["K"], s["gk"], s["dYk"], R)
        return [dq, dk, dgq, dgk]
    R = R.conj() if case["inverse"] else R
    return [_flat(_blocks(s["Q"]) * R), _flat(_blocks(s["K"]) * R)]
