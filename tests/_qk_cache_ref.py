"""Plain 64-bit forms of the query/key norm with rotation, of the rotation over
several axes, and of the 4-bit cache: numpy on the CPU, used by the tests."""
import numpy as np
import torch

PAGE = 32
GROUP = 64

# A rounding to bf16 is off by at most half a step, 2^-8 of the value.
BF16 = 2.0 ** -8
F16 = 2.0 ** -11
# Cosine and sine of an angle in fp32: the reduction's and the hardware
# function's absolute errors (each a few 1e-7), and the products' roundings.
TURN = 2e-6


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def angles(pos, sections, d, base, restart):
    """[tokens, d/2] angles; pos [axes, tokens]."""
    out = np.zeros((pos.shape[1], d // 2))
    first = 0
    for a, n in enumerate(sections):
        for i in range(n):
            k = first + i
            w = base ** (-i / n) if restart else base ** (-2.0 * k / d)
            out[:, k] = pos[a].astype(np.float64) * w
        first += n
    return out


def turn(x, a):
    """Rows x [T, H, d] turned by a [T, d/2]."""
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    y = np.empty_like(x)
    y[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
    y[..., 1::2] = x[..., 0::2] * s + x[..., 1::2] * c
    return y


def pair_size(x):
    """|x_2k| + |x_2k+1| at both places of a block: what a turn's error scales with."""
    s = np.abs(x[..., 0::2]) + np.abs(x[..., 1::2])
    return np.repeat(s, 2, axis=-1)


def norm_rope(x, g, a, eps):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x * r * g
    return turn(u, a), BF16, TURN * pair_size(u)


def norm_rope_bwd(x, g, dy, a, eps):
    """dx, dg and bounds on the fp32 part of their errors."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    e = turn(dy, -a)
    t = e * g
    dx = r * (t - n * (t * n).mean(-1, keepdims=True))
    size = pair_size(dy)     # turned back, a component errs in proportion to its block
    dx_err = TURN * r * (size * np.abs(g) + np.abs(n) * (size * np.abs(g) * np.abs(n)).mean(-1, keepdims=True))
    return dx, (e * n).sum((0, 1)), dx_err, TURN * (size * np.abs(n)).sum((0, 1))


def assert_within(got, ref, bound, what):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside the bound, worst "
                           f"{np.nanmax(np.abs(got - ref) / np.maximum(bound, 1e-300)):.2f} times it")


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64)).to(torch.bfloat16).double().numpy()


def quantize(x):
    """Codes, scales and zero points of rows x [..., d]."""
    v = x.reshape(*x.shape[:-1], -1, GROUP)
    lo = np.minimum(v.min(-1), 0.0)
    hi = np.maximum(v.max(-1), 0.0)
    s = bf16((hi - lo) / 15.0)
    one = np.where(s > 0, s, 1.0)
    z = np.where(s > 0, np.minimum(np.rint(-lo / one), 15.0), 0.0)
    c = np.clip(np.rint(v / one[..., None]) + z[..., None], 0.0, 15.0) * (s > 0)[..., None]
    return c.reshape(x.shape), s, z


def values(c, s, z):
    v = c.reshape(*c.shape[:-1], -1, GROUP)
    return (s[..., None] * (v - z[..., None])).reshape(c.shape)


def pack_rows(c, s, z):
    """Bytes of code rows [..., d/2] and of word rows [..., d/16]."""
    c = c.astype(np.uint8)
    codes = c[..., 0::2] | (c[..., 1::2] << 4)
    sbits = torch.from_numpy(np.ascontiguousarray(s)).to(torch.bfloat16).view(torch.int16).numpy().astype(np.uint16)
    word = (sbits.astype(np.uint32) << 16) | z.astype(np.uint32)
    return codes, np.ascontiguousarray(word).view(np.uint8).reshape(*word.shape[:-1], -1)


def fields(block, dh, dv):
    """Views of pool bytes [..., block]: K codes, V codes, K words, V words, each [..., 32, width]."""
    out, at = [], 0
    for w in (dh // 2, dv // 2, dh // 16, dv // 16):
        out.append(block[..., at:at + PAGE * w].reshape(*block.shape[:-1], PAGE, w))
        at += PAGE * w
    assert at == block.shape[-1]
    return out


def store(pool, slots, K, V):
    """Rows K, V [n, Hkv, d] into slots of pool bytes [pages, Hkv, block] (in place)."""
    dh, dv = K.shape[-1], V.shape[-1]
    at = 0
    kc, kw = pack_rows(*quantize(K))
    vc, vw = pack_rows(*quantize(V))
    for rows in (kc, vc, kw, vw):
        w = rows.shape[-1]
        for i, slot in enumerate(slots):
            if 0 <= slot < pool.shape[0] * PAGE:
                a = at + (slot % PAGE) * w
                pool[slot // PAGE, :, a:a + w] = rows[i]
        at += PAGE * w
    assert at == PAGE * (dh + dv) * 9 // 16


def load(pool, slots, dh, dv):
    """The values K, V [n, Hkv, d] of slots of pool bytes."""
    kc, vc, kw, vw = fields(pool, dh, dv)
    out = []
    for codes, words in ((kc, kw), (vc, vw)):
        c, w = codes[slots // PAGE, :, slots % PAGE], words[slots // PAGE, :, slots % PAGE]
        c = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], -1).astype(np.float64)
        w = np.ascontiguousarray(w).view(np.uint32)
        s = (w & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)
        out.append(values(c, s, (w & 0xFF).astype(np.float64)))
    return out


def attend(q, K, V, length, scale):
    """q [Hq, n_q, dh] over K, V [length, Hkv, d]: O, LSE and bounds on the
    error that the kernel's arithmetic may have (before O's rounding)."""
    Hq, nq, dh = q.shape
    Hkv, dv = K.shape[1], V.shape[2]
    O, L = np.zeros((Hq, nq, dv)), np.full((Hq, nq), -np.inf)
    Oerr, Lerr = np.zeros_like(O), np.zeros((Hq, nq))
    for r in range(Hq):
        h = r // (Hq // Hkv)
        for i in range(nq):
            n = min(length, length - nq + 1 + i)
            if n <= 0:
                continue
            k, v = K[:n, h], V[:n, h]
            s = scale * (k @ q[r, i])
            # fp32 sums of at most 128 exact products and four more roundings, then an
            # exponent whose argument and result round in fp32.
            ds = 132 * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(q[r, i]))
            m = s.max()
            p = np.exp(s - m)
            L[r, i] = m + np.log(p.sum())
            A = p / p.sum()
            O[r, i] = A @ v
            rel = ds + 2.0 ** -20 * (1.0 + np.abs(s - m) + abs(m) * 2.0 ** -2)
            # A weight is rounded to fp16 relative to itself, or on the grid 2^-24 of a weight
            # whose largest possible value is 2^14 times the largest scale's power of two.
            step = np.abs(v).max() / 7.0 if n else 0.0
            Oerr[r, i] = ((F16 + 2 * rel) * A) @ np.abs(v) + n * 2.0 ** -25 * 15 * 2 * step / 64 / max(p.sum(), 1.0)
            # The codes and the zero points are summed apart, in fp32: sums of up to
            # 15 s per weight over n / 16 + 8 steps, each of which rounds or cuts off at
            # most 2^-23 of the sum.  15 s is the group's range, at most 2 max |v| + s.
            span = np.repeat(np.abs(v.reshape(n, -1, GROUP)).max(-1), GROUP, axis=-1) * 2.2
            Oerr[r, i] += 2 * (n / 16 + 8) * 2.0 ** -23 * (A @ span)
            Lerr[r, i] = rel.max() + 2.0 ** -20 * (1 + abs(L[r, i]) * 0.25)
    return O, L, Oerr, Lerr
