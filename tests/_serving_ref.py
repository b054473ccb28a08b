"""64-bit forms of the calls that serve from the 4-bit cache (shared prefix,
attention weights, eviction), and caches to run them on."""
import numpy as np

import _qk_cache_ref as ref

PAGE = 32


class Paged:
    """A pool of pages [pages, Hkv, block] that held something else before, and
    the tokens written to it: one page table row per length, pages in any order."""

    def __init__(self, rng, Hkv, dh, dv, lengths, max_pages=None, spread=0.0):
        self.Hkv, self.dh, self.dv = Hkv, dh, dv
        self.lengths = [int(n) for n in lengths]
        need = [-(-n // PAGE) for n in self.lengths]
        self.max_pages = max(1, max(need)) if max_pages is None else max_pages
        pages = len(need) * self.max_pages + 3
        block = PAGE * (dh + dv) * 9 // 16
        self.pool = rng.integers(0, 256, (pages, Hkv, block)).astype(np.uint8)
        # Unused words hold NaN and infinite scales too.
        self.pool[:, :, PAGE * (dh + dv) // 2:] |= rng.integers(0, 2, (pages, Hkv, 1)).astype(np.uint8) * 0x7F
        order = rng.permutation(pages)[:len(need) * self.max_pages]
        self.table = order.reshape(len(need), self.max_pages).astype(np.int32)
        self.K, self.V = [], []
        for b, n in enumerate(self.lengths):
            size = np.exp2(spread * rng.normal(size=(n, Hkv, 1)))
            K, V = ref.bf16(rng.normal(size=(n, Hkv, dh))), ref.bf16(rng.normal(size=(n, Hkv, dv)) * size)
            if n:
                ref.store(self.pool, self.slots(b, n), K, V)
                K, V = ref.load(self.pool, self.slots(b, n), dh, dv)
            self.K.append(K.reshape(n, Hkv, dh))
            self.V.append(V.reshape(n, Hkv, dv))

    def slots(self, b, n, at=0):
        j = np.arange(at, at + n)
        return self.table[b][j // PAGE].astype(np.int64) * PAGE + j % PAGE


def behind(rng, prefix, lengths, **kw):
    """A cache whose first sequence is `prefix` (a Paged of one), and which has others of `lengths`."""
    c = Paged(rng, prefix.Hkv, prefix.dh, prefix.dv, lengths, **kw)
    c.pool = np.concatenate([c.pool, prefix.pool])
    c.prefix_table = (prefix.table[0] + (len(c.pool) - len(prefix.pool))).astype(np.int32)
    c.K, c.V, c.lengths = prefix.K + c.K, prefix.V + c.V, prefix.lengths + c.lengths
    return c


def attend_prefix(q, Kp, Vp, K, V, length, scale):
    """q [Hq, n_q, dh] over the prefix and `length` own keys: O, LSE and bounds on
    the kernel's error, as _qk_cache_ref.attend has them.  The parts are put
    together in fp32: a product and a sum for each of at most 256, relative to
    what they sum."""
    Hq, nq, _ = q.shape
    rows = []
    for i in range(nq):
        own = max(0, length - nq + 1 + i)
        k, v = np.concatenate([Kp, K[:own]]), np.concatenate([Vp, V[:own]])
        O, L, Oerr, Lerr = ref.attend(q[:, i:i + 1], k, v, len(k), scale)
        if len(k):
            A = 258 * 2.0 ** -23 * np.abs(v).max(0)                   # [Hkv, dv]
            Oerr = Oerr + np.repeat(A, Hq // K.shape[1], 0)[:, None]
            Lerr = Lerr + 258 * 2.0 ** -23
        rows.append((O, L, Oerr, Lerr))
    return [np.concatenate(x, 1) for x in zip(*rows)]


def weigh(q, K, lse, length, w, scale):
    """weights [Hkv, cap] with those of q [Hq, n_q, dh] over K [length, Hkv, dh] added, and bounds."""
    Hq, nq, dh = q.shape
    Hkv = K.shape[1]
    group = Hq // Hkv
    out, err = w.astype(np.float64), np.zeros(w.shape)
    for r in range(Hq):
        h = r // group
        for i in range(nq):
            n = length - nq + 1 + i
            if n <= 0 or lse[r, i] == -np.inf:
                continue
            k = K[:n, h]
            s = scale * (k @ q[r, i])
            a = np.exp(s - lse[r, i])
            # The score as in attend; then the exponent's terms, in units of log2(e), each
            # rounded (the scale's factor, LSE's, their sum), and the power, off by 2^-22.
            ds = 132 * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(q[r, i]))
            rel = ds + 2.0 ** -23 * (2.0 + 2.0 * np.abs(s) + 2.0 * abs(lse[r, i]))
            out[h, :n] += a
            err[h, :n] += a * rel + 2.0 ** -126
    # fp32 sums of all rows and of what was there.
    return out, err + (group * nq + 4) * 2.0 ** -24 * np.abs(out)


def evict(w, n, keep, first, recent):
    """Of one head's weights [cap] and n tokens: the place that the token at each
    of `keep` places had (-1: none), and the weights at the new places."""
    m = min(n, keep)
    src = np.full(keep, -1, dtype=np.int64)
    src[:m] = np.arange(m)
    if n > keep:
        front = keep - recent
        mid = list(range(first, n - recent))
        key = lambda j: (np.inf, 1) if np.isnan(w[j]) else (w[j], 0)  # noqa: E731
        best = sorted(mid, key=lambda j: (-key(j)[0], -key(j)[1], j))[:keep - first - recent]
        stay = set(best)
        holes = [j for j in mid if j not in stay and j < front]
        late = sorted(j for j in best if j >= front)
        assert len(holes) == len(late)
        src[holes] = late
        src[front:] = np.arange(n - recent, n)
    new = np.zeros_like(w)
    new[:m] = w[src[:m]]
    return src, new
