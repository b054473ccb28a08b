"""GPU tests of attention over the 4-bit cache with values of very different
sizes: along a sequence, between keys of different weight, and between the two
64-element groups of a row, each element against the 64-bit form under a bound
that is relative to its own group's weighted values."""
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


# ---------------------------------------------------------------------------
# A row's weights are as precise as its own largest one allows
# ---------------------------------------------------------------------------
def _along(rng, scores, Hkv, d):
    """Queries [1, 2 Hkv, 1, d] and a K for _filled whose scores with a KV head's first query
    are about `scores` [n] (natural log, at the scale d^-1/2), with its second about -`scores`."""
    u = rng.normal(size=(Hkv, d))
    Q = torch.from_numpy(np.stack([u, -u], 1).reshape(1, 2 * Hkv, 1, d)).to(torch.bfloat16)
    unit = u * np.sqrt(d) / (u * u).sum(-1, keepdims=True)

    def K(b, n):
        return torch.from_numpy(scores[:, None, None] * unit + 0.02 * rng.normal(size=(n, Hkv, d))).to(torch.bfloat16)

    return Q, K


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("at", [0, 0.5, 1])
@pytest.mark.parametrize("e", [24, 32, 40])
def test_a_large_value_on_a_key_that_carries_no_weight(layout, at, e):
    """One key 2^-80 below the others for the first query of each KV head, with values 2^e times
    theirs; the second query of the head sees little else."""
    n, Hkv, d, spare = LAYOUTS[layout]
    rng = np.random.default_rng(41)
    key = int(round(at * (n - 1)))
    scores = 0.3 * rng.normal(size=n)
    scores[key] = -80 * np.log(2)

    def V(b, n):
        v = 0.7 + 0.1 * rng.normal(size=(n, Hkv, d))
        v[key] *= 2.0 ** e
        return torch.from_numpy(v).to(torch.bfloat16)

    Q, K = _along(rng, scores, Hkv, d)
    cache, table, lens, vals = _filled(rng, [n], Hkv, d, d, K=K, V=V, wide=-(-n // PAGE) + spare)
    O, _ = _check(Q, cache, table, lens, vals)
    O = f64(O)[0].reshape(Hkv, 2, d)
    assert (np.abs(O[:, 0] - 0.7) < 0.2).all() and (np.abs(O[:, 1]) > 0.1 * 2.0 ** e).all()


@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_a_large_value_whose_weight_fades(layout):
    """The first pages have values of 2^40; scores that rise by 80 octaves along the sequence
    leave nothing of them in the first query, and nothing of the last ones in the second."""
    n, Hkv, d, spare = LAYOUTS[layout]
    rng = np.random.default_rng(42)

    def V(b, n):
        size = np.where(np.arange(n) < n // 4, 2.0 ** 40, 1.0)[:, None, None]
        return torch.from_numpy((0.7 + 0.1 * rng.normal(size=(n, Hkv, d))) * size).to(torch.bfloat16)

    Q, K = _along(rng, np.linspace(-40, 40, n) * np.log(2), Hkv, d)
    cache, table, lens, vals = _filled(rng, [n], Hkv, d, d, K=K, V=V, wide=-(-n // PAGE) + spare)
    _check(Q, cache, table, lens, vals)


@pytest.mark.parametrize("spare", [0, 70])
@pytest.mark.parametrize("e", [-80, -40, -28, 28, 40, 80])
@pytest.mark.parametrize("group,nq", [(2, 1), (3, 4)])
def test_groups_of_different_scale(spare, e, group, nq):
    """Dims 64-127 of every value 2^e times dims 0-63; up to 8 and more query rows."""
    rng = np.random.default_rng(43)

    def V(b, n):
        v = rng.normal(size=(n, 2, 128))
        v[..., 64:] *= 2.0 ** e
        return torch.from_numpy(v).to(torch.bfloat16)

    cache, table, lens, vals = _filled(rng, [700, 33], 2, 128, 128, V=V, wide=22 + spare)
    _check(_bf16(rng, 2, 2 * group, nq, 128), cache, table, lens, vals)


@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("dv,group,nq", [(128, 2, 1), (64, 2, 1), (64, 3, 5)])
def test_scores_and_scales_of_every_size(layout, dv, group, nq):
    """Scores over some 100 octaves, the values' scales over 80, independent of each other."""
    n, Hkv, d, spare = LAYOUTS[layout]
    Hkv, d = min(Hkv, 8), max(d, dv)
    rng = np.random.default_rng(44)

    def V(b, n):
        size = 2.0 ** rng.uniform(-40, 40, size=(n, Hkv, dv // GROUP, 1))
        return torch.from_numpy((rng.normal(size=(n, Hkv, dv // GROUP, GROUP)) * size).reshape(n, Hkv, dv)).to(torch.bfloat16)

    cache, table, lens, vals = _filled(rng, [n, n // 3], Hkv, d, dv, V=V, wide=-(-n // PAGE) + spare,
                                       K=lambda b, n: _bf16(rng, n, Hkv, d, scale=12.0))
    _check(_bf16(rng, 2, Hkv * group, nq, d), cache, table, lens, vals)


@pytest.mark.parametrize("spare", [0, 70])
def test_scores_of_some_millions(spare):
    """One key far above the rest, at the size where neighbouring fp32 scores are 1/2 apart."""
    rng = np.random.default_rng(45)
    K = lambda b, n: torch.zeros((n, 1, 64), dtype=torch.bfloat16).index_fill_(0, torch.tensor([n // 2]), 15.0)  # noqa: E731
    cache, table, lens, vals = _filled(rng, [300], 1, 64, 64, K=K, wide=10 + spare)
    Q = torch.full((1, 4, 1, 64), 3.0, dtype=torch.bfloat16)
    import exact_scaled_dot_gb300 as esd
    O, LSE = esd.attn_fwd_decode_cache(Q.cuda(), cache, table, lens, scale=2100.0)
    torch.cuda.synchronize()
    score, v = 15 * 3 * 64 * 2100.0, vals[0][1][150, 0]
    assert 2.0 ** 22 < score < 2.0 ** 23
    # its weight is all there is: fp16's rounding of it, the sums' of codes and zero points, bf16's
    assert_within(f64(O), np.broadcast_to(v, (1, 4, 1, 64)), ref.BF16 * np.abs(v) + ref.F16 * np.abs(v) + 2.0 ** -13 * np.abs(v).max(), "O")
    assert_within(f64(LSE), np.full((1, 4, 1), score), 2.0 ** -20 * score, "LSE")


# ---------------------------------------------------------------------------
# Long sums
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("Hq,Hkv,d", [(320, 320, 64), (4800, 1, 128)])
def test_the_mean_of_many_values(Hq, Hkv, d):
    """Equal weights over 320000 keys of one CTA: O is the mean of the values, far below each of them.

    A step of 16 keys may cut the sum of codes that it adds to by 2^-23 of itself: up to 64 steps
    of 16 codes of 15 until the zero points are taken out, and what is left of the sum beside
    (3 sqrt(80000) of a warp's keys, below 2^12 here), so 2^-23 (960 + 2^8) of a code for each key;
    a key's zero point is added to up to 127 others in fp32: 2^-24 128 15."""
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(47)
    pages, wide = 60, 10000
    V = torch.from_numpy(rng.normal(size=(pages * PAGE, Hkv, d))).to(torch.bfloat16)
    cache = esd.QuantCache.empty(pages, Hkv, d, d)
    esd.attn_cache_append(cache, torch.zeros_like(V).cuda(), V.cuda(), torch.arange(pages * PAGE, device="cuda"))
    c, s, z = ref.quantize(f64(V))
    table = rng.integers(0, pages, (1, wide)).astype(np.int32)
    O, LSE = esd.attn_fwd_decode_cache(torch.zeros((1, Hq, 1, d), dtype=torch.bfloat16, device="cuda"), cache,
                                       torch.from_numpy(table).cuda(),
                                       torch.tensor([wide * PAGE], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert esd.attn_get_status() == 0
    v = ref.values(c, s, z).reshape(pages, PAGE, Hkv, d).sum(1)
    mean = np.einsum("p,phd->hd", np.bincount(table[0], minlength=pages).astype(np.float64), v) / (wide * PAGE)
    mean = np.repeat(mean, Hq // Hkv, 0)[None, :, None]
    cut = (2.0 ** -23 * (960 + 256) + 2.0 ** -24 * 128 * 15) * s.max()
    assert_within(f64(O), mean, ref.BF16 * np.abs(mean) + cut, "O")
    want = np.full((1, Hq, 1), np.log(wide * PAGE))
    assert_within(f64(LSE), want, 2.0 ** -22 * want, "LSE")


# ---------------------------------------------------------------------------
# Rows without a key
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("spare", [0, 70])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_query_row_that_is_not_finite_and_sees_no_key(spare, value):
    """O = 0 and LSE = -inf, as for any row without a key, in sequences of no and of few tokens."""
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(46)
    lengths, nq = [0, 1, 3, 40], 4
    cache, table, lens, _ = _filled(rng, lengths, 1, 128, 64, wide=2 + spare)
    Q = _bf16(rng, 4, 5, nq, 128).cuda()
    O, LSE = esd.attn_fwd_decode_cache(Q, cache, table, lens)
    unseen = torch.tensor([[i < nq - n for i in range(nq)] for n in lengths], device="cuda")[:, None].expand(4, 5, nq)
    Q[unseen] = value
    O2, LSE2 = esd.attn_fwd_decode_cache(Q, cache, table, lens)
    torch.cuda.synchronize()
    assert esd.attn_get_status() == 0
    assert (O2[unseen] == 0).all() and LSE2[unseen].isneginf().all()
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
