"""GPU tests of attention over the 4-bit cache with values of very different
sizes along a sequence, each element against the 64-bit form under a bound that
is relative to its own group's weighted values."""
import numpy as np
import pytest
import torch

import _qk_cache_ref as ref
from _qk_cache_ref import assert_within, f64
from test_cache_gpu import _bf16, _filled

pytestmark = pytest.mark.gpu
PAGE, GROUP = 32, 64


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from exact_scaled_dot_gb300 import build as b
    b.build()
    import exact_scaled_dot_gb300 as esd
    esd.load()
    assert torch.cuda.is_available(), "a CUDA device is required"
    esd.attn_clear_status()
    yield
    assert esd.attn_get_status() == 0


def _attend(q, K, V, length, scale):
    """q [Hq, n_q, dh] over K, V [length, Hkv, d]: O, LSE and bounds on their errors.

    With A the row's softmax weights and, per group of 64 elements, big_j the group's
    largest |v| of key j:
      rel_j      a score's error (132 roundings of fp32) and its exponential's, relative to A_j;
      2^-11 A_j  the rounding of the weight A_j s_j to fp16;
      2^-30 n 2.2 max_j (A_j big_j)
                 weights below fp16's normal range are rounded to multiples of 2^-24 (off by
                 2^-25), where the row's largest in the group counts at least 2^5, times codes
                 less zero points of up to 15, and 15 s_j <= 2.2 big_j;
      (2^-14 + (n / 16 + 8) 2^-22) A_j 2.2 big_j
                 the sums of codes and of zero points, apart: products of subnormal operands are
                 cut as if the operand were 2^-14, 2^10 times a code's unit, so at 2^-14 of a
                 unit, for up to 16 of them a step; and a step's sum at 2^-23 of itself."""
    Hq, nq, _ = q.shape
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
            m = s.max()
            p = np.exp(s - m)
            L[r, i] = m + np.log(p.sum())
            A = p / p.sum()
            O[r, i] = A @ v
            ds = 132 * 2.0 ** -24 * scale * (np.abs(k) @ np.abs(q[r, i]))
            rel = ds + 2.0 ** -20 * (1.0 + np.abs(s - m) + abs(m) / 4)
            big = np.repeat(np.abs(v.reshape(n, -1, GROUP)).max(-1), GROUP, axis=-1)
            Oerr[r, i] = ((ref.F16 + rel) * A) @ np.abs(v) + (A @ rel) * np.abs(O[r, i])
            Oerr[r, i] += n * 2.0 ** -30 * 2.2 * (A[:, None] * big).max(0)
            Oerr[r, i] += (2.0 ** -14 + (n / 16 + 8) * 2.0 ** -22) * 2.2 * (A @ big)
            Lerr[r, i] = A @ rel + 2.0 ** -20 * (1 + abs(L[r, i]) / 4)
    return O, L, Oerr, Lerr


def _check(Q, cache, table, lens, vals, scale=None):
    import exact_scaled_dot_gb300 as esd
    scale = Q.shape[-1] ** -0.5 if scale is None else scale
    O, LSE = esd.attn_fwd_decode_cache(Q.cuda(), cache, table, lens, scale=scale)
    torch.cuda.synchronize()
    assert esd.attn_get_status() == 0
    for b in range(Q.shape[0]):
        o, l, oerr, lerr = _attend(f64(Q[b]), *vals[b], int(lens[b]), scale)
        assert_within(f64(LSE[b]), l, lerr, f"LSE[{b}]")
        assert_within(f64(O[b]), o, ref.BF16 * np.abs(o) + oerr, f"O[{b}]")
    return O, LSE


# n keys, Hkv, d and the table's extra columns: one CTA a sequence (of eight and of four
# warps), and ranges of pages with one and with several pages for each warp.
LAYOUTS = {"eight_warps": (1024, 2, 128, 0), "four_warps": (512, 160, 64, 0), "ranges": (900, 2, 128, 70),
           "longer_ranges": (2048, 64, 64, 70)}


# ---------------------------------------------------------------------------
# The sum of the weights does not know the values' scale
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("early,late", [(None, 30), (None, 40), (None, 80), (-90, 40), (-90, 80), (80, -90), (40, None)])
def test_values_that_appear_along_the_sequence(layout, early, late):
    """Pages whose values are zero or tiny ahead of pages with large ones, and the other
    way round, for every warp: 2^early (None: 0), then 2^late."""
    n, Hkv, d, spare = LAYOUTS[layout]
    rng = np.random.default_rng(40)

    def V(b, n):
        # Warps take every fourth or eighth page, ranges start at multiples of 8 here.
        page = np.arange(n) // PAGE
        first = page < page[-1] // 2 if layout != "longer_ranges" else page % 8 < 4
        size = np.where(first, 0.0 if early is None else 2.0 ** early, 0.0 if late is None else 2.0 ** late)
        return torch.from_numpy(rng.normal(size=(n, Hkv, d)) * size[:, None, None]).to(torch.bfloat16)

    cache, table, lens, vals = _filled(rng, [n], Hkv, d, d, V=V, wide=-(-n // PAGE) + spare)
    _check(_bf16(rng, 1, Hkv, 1, d), cache, table, lens, vals)


def test_many_keys_above_the_first():
    """Values of zero (the smallest scale there is), and hundreds of thousands of keys whose scores
    exceed the first pages' a little: the sum of their weights stays in fp32's range."""
    import exact_scaled_dot_gb300 as esd
    Hkv, d, wide = 400, 64, 10000
    cache = esd.QuantCache(torch.zeros((2, Hkv, esd.attn_cache_page_bytes(1, d, d)), dtype=torch.uint8, device="cuda"), d, d)
    K = torch.zeros((2 * PAGE, Hkv, d), dtype=torch.bfloat16, device="cuda")
    K[PAGE:] = 15 / 64                     # s = 2^-6, codes of 15
    esd.attn_cache_append(cache, K, torch.zeros_like(K), torch.arange(2 * PAGE, device="cuda"))
    table = torch.ones((1, wide), dtype=torch.int32, device="cuda")
    table[0, :4] = 0
    Q = torch.ones((1, Hkv, 1, d), dtype=torch.bfloat16, device="cuda")
    scale = 7.8 * np.log(2) / 15           # the later keys' scores are 7.8 ln 2
    O, LSE = esd.attn_fwd_decode_cache(Q, cache, table, torch.tensor([wide * PAGE], dtype=torch.int32, device="cuda"),
                                       scale=scale)
    torch.cuda.synchronize()
    assert esd.attn_get_status() == 0
    want = np.log(4 * PAGE + (wide - 4) * PAGE * np.exp(15 * np.float32(scale).astype(np.float64)))
    # each lane adds 4 (wide / 4) weights of about the same size one after the other: at most
    # that many roundings of 2^-24 in the sum, and some more in the scores and exponentials
    assert (O == 0).all()
    assert_within(f64(LSE), np.full((1, Hkv, 1), want), wide * 2.0 ** -24 + 2.0 ** -18, "LSE")
