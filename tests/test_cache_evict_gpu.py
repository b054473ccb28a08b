"""GPU tests of eviction: the tokens kept, their places, weights and bytes, exactly; and of
a serving loop with all the calls over the cache."""
import numpy as np
import pytest
import torch

import _qk_cache_ref as ref
import _serving_ref as srv
from _qk_cache_ref import assert_within, bf16, f64

pytestmark = pytest.mark.gpu
PAGE = 32


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


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _pool(rng, B, Hkv, dh, dv, max_pages):
    pages = B * max_pages + 2
    pool = rng.integers(0, 256, (pages, Hkv, PAGE * (dh + dv) * 9 // 16)).astype(np.uint8)
    return pool, rng.permutation(pages)[:B * max_pages].reshape(B, max_pages).astype(np.int32)


def _expected(pool, table, lengths, w, keep, first, recent, dh, dv):
    """The pool, the weights, the new lengths and the kept places of the definition."""
    B, Hkv, _ = w.shape
    out, new = pool.copy(), np.zeros_like(w)
    kept = np.zeros((B, Hkv, keep), np.int32)
    src_fields, dst_fields = ref.fields(pool, dh, dv), None
    for b, n in enumerate(lengths):
        for h in range(Hkv):
            kept[b, h], new[b, h] = srv.evict(w[b, h], n, keep, first, recent)
            to = np.arange(min(n, keep))
            at = kept[b, h][to]
            move = at != to
            to, at = to[move], at[move]
            start = 0
            for width, f in zip((dh // 2, dv // 2, dh // 16, dv // 16), src_fields):
                rows = f[table[b, at // PAGE], h, at % PAGE]
                for t, row in zip(to, rows):
                    a = start + (t % PAGE) * width
                    out[table[b, t // PAGE], h, a:a + width] = row
                start += PAGE * width
    return out, new, np.minimum(lengths, keep).astype(np.int32), kept


def _weights(rng, shape, kind):
    w = np.exp(2 * rng.normal(size=shape)).astype(np.float32)
    if kind == "ties":
        w = np.round(w * 2).astype(np.float32) / 2
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "odd":                 # whatever a user's own scores hold
        w = rng.normal(size=shape).astype(np.float32)
        for v in (np.nan, np.inf, -np.inf, 0.0, -0.0, -np.nan, 1e-45, -1e-45):
            w[rng.random(shape) < 0.08] = v
    return w


@pytest.mark.parametrize("dh,dv", [(64, 64), (128, 128), (128, 64)])
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
@pytest.mark.parametrize("keep,first,recent,lengths", [
    (1, 0, 0, [5, 1, 0]),
    (1, 0, 1, [40, 2, 1]),
    (4, 4, 0, [33, 4, 5]),                        # nothing between to choose
    (64, 4, 16, [65, 64, 100]),
    (50, 0, 0, [200, 51, 0]),
    (50, 3, 40, [95, 60, 49]),                    # the newest overlap their new places
    (100, 10, 33, [700, 130, 101]),
    (40, 7, 33, [41, 74, 150]),                   # first and newest alone
])
def test_exact(keep, first, recent, lengths, kind, dh, dv):
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(keep + first + len(kind))
    B, Hkv = len(lengths), 2
    max_pages = -(-max(lengths) // PAGE) + 1
    pool, table = _pool(rng, B, Hkv, dh, dv, max_pages)
    w = _weights(rng, (B, Hkv, max_pages * PAGE), kind)
    want = _expected(pool, table, np.array(lengths), w, keep, first, recent, dh, dv)
    for in_place in (False, True):
        cache = esd.QuantCache(_dev(pool), dh, dv)
        W = _dev(w)
        n, nw, kept = esd.attn_cache_evict(cache, _dev(table), _dev(np.array(lengths, np.int32)), W, keep, first=first,
                                           recent=recent, new_weights=W if in_place else None)
        torch.cuda.synchronize()
        assert np.array_equal(n.cpu().numpy(), want[2])
        assert np.array_equal(kept.cpu().numpy(), want[3])
        assert np.array_equal(nw.cpu().numpy(), want[1], equal_nan=True)
        assert np.array_equal(cache.pool.cpu().numpy(), want[0])
        assert in_place or np.array_equal(W.cpu().numpy(), w, equal_nan=True)


@pytest.mark.parametrize("n,keep,recent", [(9000, 4096, 256), (9000, 8990, 3000), (5000, 4999, 0), (40000, 100, 1)])
def test_long(n, keep, recent):
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(n + keep)
    dh, dv, B, Hkv = 64, 64, 2, 2
    max_pages = -(-n // PAGE)
    pool, table = _pool(rng, B, Hkv, dh, dv, max_pages)
    w = _weights(rng, (B, Hkv, max_pages * PAGE), "ties")
    lengths = np.array([n, n // 2])
    want = _expected(pool, table, lengths, w, keep, 5, recent, dh, dv)
    cache = esd.QuantCache(_dev(pool), dh, dv)
    got, nw, kept = esd.attn_cache_evict(cache, _dev(table), _dev(lengths.astype(np.int32)), _dev(w), keep, first=5,
                                         recent=recent)
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want[3]) and np.array_equal(got.cpu().numpy(), want[2])
    assert np.array_equal(nw.cpu().numpy(), want[1]) and np.array_equal(cache.pool.cpu().numpy(), want[0])


@pytest.mark.parametrize("B,pages,lengths,keep,recent", [
    (160, 205, [6500, 6401, 6560], 1500, 40),        # many heads of sequences past shared memory
    (100, 20, [600, 640, 513], 512, 64),             # many heads
    (100, 205, [6500, 1501, 6560], 1500, 40),        # fewer of them, long
    (2, 210, [4100, 4097], 4096, 600),               # room for many moves, but few and the newest by a few places
    (2, 210, [6000, 4700], 4096, 600),               # the newest by more and by little more than they are
])
@pytest.mark.parametrize("in_place", [False, True])
def test_divisions_of_the_work(B, pages, lengths, keep, recent, in_place):
    """The sequences behind those of `lengths` stay as they are."""
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(B + keep)
    pool, first_rows = _pool(rng, len(lengths), 2, 64, 64, pages)
    table = np.full((B, pages), -1, np.int32)
    table[:len(lengths)] = first_rows
    lengths = np.concatenate([lengths, rng.integers(0, keep + 1, B - len(lengths))])
    w = _weights(rng, (B, 2, pages * PAGE), "ties")
    want = _expected(pool, table, lengths, w, keep, 5, recent, 64, 64)
    cache, W = esd.QuantCache(_dev(pool), 64, 64), _dev(w)
    got, nw, kept = esd.attn_cache_evict(cache, _dev(table), _dev(lengths.astype(np.int32)), W, keep, first=5,
                                         recent=recent, new_weights=W if in_place else None)
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want[3]) and np.array_equal(got.cpu().numpy(), want[2])
    assert np.array_equal(nw.cpu().numpy(), want[1]) and np.array_equal(cache.pool.cpu().numpy(), want[0])


def test_budget_past_the_table_and_no_workspace():
    """A budget that no sequence reaches changes nothing and needs no workspace."""
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(2)
    pool, table = _pool(rng, 2, 1, 64, 64, 2)
    w = _weights(rng, (2, 1, 64), "plain")
    cache = esd.QuantCache(_dev(pool), 64, 64)
    assert esd.attn_cache_evict_workspace_bytes(cache, 2, 2, 1000, first=4, recent=8) == 0
    n, nw, kept = esd.attn_cache_evict(cache, _dev(table), _dev(np.array([64, 10], np.int32)), _dev(w), 1000, first=4,
                                       recent=8)
    torch.cuda.synchronize()
    assert n.tolist() == [64, 10] and np.array_equal(cache.pool.cpu().numpy(), pool)
    assert np.array_equal(nw.cpu().numpy()[1, 0], np.where(np.arange(64) < 10, w[1, 0], 0))
    assert np.array_equal(kept.cpu().numpy()[1, 0], np.where(np.arange(1000) < 10, np.arange(1000), -1))


def test_bad_pages_and_lengths():
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(12)
    dh = dv = 64
    pool, table = _pool(rng, 2, 1, dh, dv, 4)
    w = _weights(rng, (2, 1, 128), "plain")
    bad = table.copy()
    bad[0, 1], bad[1, 3] = -1, len(pool)
    cache = esd.QuantCache(_dev(pool), dh, dv)
    n, nw, kept = esd.attn_cache_evict(cache, _dev(bad), _dev(np.array([128, 1 << 30], np.int32)), _dev(w), 64, first=2,
                                       recent=8)
    torch.cuda.synchronize()
    assert esd.attn_get_status() == esd.ATTN_ERR_PAGE
    esd.attn_clear_status()
    want = _expected(pool, table, np.array([128, 128]), w, 64, 2, 8, dh, dv)
    assert n.tolist() == [64, 64] and np.array_equal(kept.cpu().numpy(), want[3])
    got = cache.pool.cpu().numpy()
    # moves between good pages happened, the others' places are as they were
    for b in range(2):
        vals = [f for f in ref.fields(got, dh, dv)]
        old = [f for f in ref.fields(pool, dh, dv)]
        for to in range(64):
            at = want[3][b, 0, to]
            if not 0 <= bad[b, to // PAGE] < len(pool):
                continue
            from_ok = 0 <= bad[b, at // PAGE] < len(pool)
            src = (table[b, at // PAGE], 0, at % PAGE) if from_ok else (table[b, to // PAGE], 0, to % PAGE)
            for x, y in zip(vals, old):
                assert np.array_equal(x[table[b, to // PAGE], 0, to % PAGE], y[src])
    neg = esd.attn_cache_evict(cache, _dev(table), _dev(np.array([-7, 0], np.int32)), _dev(w), 64)
    torch.cuda.synchronize()
    assert neg[0].tolist() == [0, 0] and (neg[1] == 0).all() and (neg[2] == -1).all()


def test_refuses_lengths_in_place():
    import exact_scaled_dot_gb300 as esd
    cache = esd.QuantCache(torch.zeros((4, 1, 32 * 128 * 9 // 16), dtype=torch.uint8, device="cuda"), 64, 64)
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((1, 1, 64), device="cuda")
    with pytest.raises(esd.AttnError):
        esd.attn_cache_evict(cache, table, n, w, 4, new_lengths=n)


@pytest.mark.parametrize("B", [3, 40])
def test_serving_loop(B):
    """Steps of a captured loop (write the new tokens, attend over the shared prefix and the
    sequences' own tokens, add the weights up, cut to the budget), against 64-bit forms over
    what the cache holds at each step."""
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(B)
    Hq, Hkv, nq, dh, dv, prefix, keep, first, recent, steps = 8, 2, 2, 128, 64, 75, 40, 2, 8, 6
    lengths = [int(x) for x in rng.integers(30, keep + 1, B)]
    c = srv.Paged(rng, Hkv, dh, dv, [prefix] + lengths, max_pages=4)
    cache = esd.QuantCache(_dev(c.pool), dh, dv)
    # (as wide as a prefix that is worked on in tiles of 128 rows, where there are many rows)
    ptab = _dev(np.concatenate([c.table[0], np.zeros(220 if B > 30 else 0, np.int32)]))
    plen, table = _dev(np.array([prefix], np.int32)), _dev(c.table[1:])
    n = _dev(np.array(lengths, np.int32))
    n2, wts = torch.empty_like(n), torch.zeros((B, Hkv, 4 * PAGE), device="cuda")
    Q = torch.empty((B, Hq, nq, dh), dtype=torch.bfloat16, device="cuda")
    Kn = torch.empty((B * nq, Hkv, dh), dtype=torch.bfloat16, device="cuda")
    Vn = torch.empty((B * nq, Hkv, dv), dtype=torch.bfloat16, device="cuda")
    O, LSE = torch.empty((B, Hq, nq, dv), dtype=torch.bfloat16, device="cuda"), torch.empty((B, Hq, nq), device="cuda")
    kept = torch.empty((B, Hkv, keep), dtype=torch.int32, device="cuda")
    i = torch.arange(nq, device="cuda")
    seen = [torch.empty_like(wts), torch.empty_like(n)]            # the weights and lengths before the cut

    def step():
        at = n.long()[:, None] + i
        slots = (table.long().gather(1, at // PAGE) * PAGE + at % PAGE).flatten()
        esd.attn_cache_append(cache, Kn, Vn, slots)
        n.add_(nq)
        esd.attn_fwd_prefix_cache(Q, cache, ptab, plen, table, n, O=O, LSE=LSE)
        esd.attn_cache_weigh(Q, cache, table, n, LSE, wts)
        seen[0].copy_(wts), seen[1].copy_(n)
        esd.attn_cache_evict(cache, table, n, wts, keep, first=first, recent=recent, new_lengths=n2, new_weights=wts,
                             kept=kept)
        n.copy_(n2)

    state = (cache.pool.clone(), n.clone(), wts.clone())
    for t in (Q, Kn, Vn):
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((cache.pool, n, wts), state):
        t.copy_(s)
    heads = [[(c.K[b + 1][:, h], c.V[b + 1][:, h]) for h in range(Hkv)] for b in range(B)]     # the tokens of each head
    for _ in range(steps):
        q, k, v = (bf16(rng.normal(size=t.shape)) for t in (Q, Kn, Vn))
        for t, x in ((Q, q), (Kn, k), (Vn, v)):
            t.copy_(_dev(x))
        before = f64(wts).astype(np.float32)
        graph.replay()
        torch.cuda.synchronize()
        kq, vq = ref.values(*ref.quantize(k)).reshape(B, nq, Hkv, dh), ref.values(*ref.quantize(v)).reshape(B, nq, Hkv, dv)
        got_w, got_kept, got_n, lse = f64(seen[0]), kept.cpu().numpy(), n.cpu().numpy(), f64(LSE)
        for b in range(B):
            for h in range(Hkv):
                heads[b][h] = tuple(np.concatenate([x, y[b, :, h]]) for x, y in zip(heads[b][h], (kq, vq)))
            K, V = (np.stack([heads[b][h][x] for h in range(Hkv)], 1) for x in (0, 1))
            length = len(K)
            assert length == int(seen[1][b])
            rO, rL, eO, eL = srv.attend_prefix(q[b], c.K[0], c.V[0], K, V, length, dh ** -0.5)
            assert_within(f64(O)[b], rO, eO + 2.0 ** -8 * (np.abs(rO) + eO), "O")
            assert_within(lse[b], rL, eL, "LSE")
            want, err = srv.weigh(q[b], K, lse[b], length, before[b], dh ** -0.5)
            assert_within(got_w[b], want, err, "weights")
            for h in range(Hkv):
                src, _ = srv.evict(got_w[b, h].astype(np.float32), length, keep, first, recent)
                assert np.array_equal(src, got_kept[b, h])
                m = min(length, keep)
                assert got_n[b] == m
                heads[b][h] = tuple(x[src[:m]] for x in heads[b][h])
    # the prefix's pages are as they were
    pages = c.table[0, :-(-prefix // PAGE)]
    assert np.array_equal(cache.pool.cpu().numpy()[pages], c.pool[pages])


@pytest.mark.parametrize("n", [50000, 200003])
@pytest.mark.parametrize("keep", [300, 9000])
@pytest.mark.parametrize("in_place", [False, True])
def test_weights_past_shared_memory(n, keep, in_place):
    """One head of more tokens than its CTA keeps weights of, and of more than it keeps decisions of; of equal
    weights only some stay.  Moves below and above what takes a second kernel."""
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(n + keep)
    pages = -(-n // PAGE)
    pool, table = _pool(rng, 1, 1, 64, 64, pages)
    w = np.minimum(_weights(rng, (1, 1, pages * PAGE), "ties"), 8.0)
    want = _expected(pool, table, np.array([n]), w, keep, 3, 40, 64, 64)
    least = want[1][0, 0, 3:keep - 40].min()
    assert 0 < (want[1][0, 0, 3:keep - 40] == least).sum() < (w[0, 0, 3:n - 40] == least).sum()
    cache, W = esd.QuantCache(_dev(pool), 64, 64), _dev(w)
    got, nw, kept = esd.attn_cache_evict(cache, _dev(table), _dev(np.array([n], np.int32)), W, keep, first=3, recent=40,
                                         new_weights=W if in_place else None)
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want[3]) and np.array_equal(got.cpu().numpy(), want[2])
    assert np.array_equal(nw.cpu().numpy(), want[1]) and np.array_equal(cache.pool.cpu().numpy(), want[0])


def test_outputs_next_to_inputs():
    """Arrays that are parts of one buffer, one right behind the other, are not refused; one element nearer
    they are."""
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(8)
    pool, table = _pool(rng, 2, 1, 64, 64, 3)
    w, lengths, keep = _weights(rng, (2, 1, 96), "plain"), np.array([90, 50], np.int32), 40
    want = _expected(pool, table, lengths, w, keep, 4, 8, 64, 64)
    cache, both = esd.QuantCache(_dev(pool), 64, 64), torch.zeros(2 * 192, device="cuda")
    n = _dev(np.concatenate([lengths, lengths]))
    both[:192] = _dev(w).flatten()
    W = both[:192].view(2, 1, 96)
    for out in (dict(new_lengths=n[1:3]), dict(new_weights=both[1:193].view(2, 1, 96)),
                dict(new_weights=both[191:383].view(2, 1, 96))):
        with pytest.raises(esd.AttnError):
            esd.attn_cache_evict(cache, _dev(table), n[:2], W, keep, first=4, recent=8, **out)
    got, nw, kept = esd.attn_cache_evict(cache, _dev(table), n[:2], W, keep, first=4, recent=8, new_lengths=n[2:],
                                         new_weights=both[192:].view(2, 1, 96))
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want[3]) and np.array_equal(n.cpu().numpy()[2:], want[2])
    assert np.array_equal(nw.cpu().numpy(), want[1]) and np.array_equal(cache.pool.cpu().numpy(), want[0])


@pytest.mark.parametrize("keep,lengths", [(40, [90, 50]), (2500, [5000, 2501]), (1 << 30, [60, 0])])
def test_without_the_places_kept(keep, lengths):
    """kept=False: the same tokens, weights and lengths; also with the largest budget, whose places would take
    4 GiB a head."""
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(keep)
    pages = -(-max(lengths) // PAGE)
    pool, table = _pool(rng, 2, 2, 64, 64, pages)
    w, lengths = _weights(rng, (2, 2, pages * PAGE), "ties"), np.array(lengths, np.int32)
    want = _expected(pool, table, lengths, w, min(keep, pages * PAGE), 4, 8, 64, 64)
    cache = esd.QuantCache(_dev(pool), 64, 64)
    before = torch.cuda.memory_allocated()
    got, nw, kept = esd.attn_cache_evict(cache, _dev(table), _dev(lengths), _dev(w), keep, first=4, recent=8, kept=False)
    torch.cuda.synchronize()
    assert kept is None and torch.cuda.memory_allocated() - before < 1 << 24
    assert np.array_equal(got.cpu().numpy(), want[2]) and np.array_equal(nw.cpu().numpy(), want[1])
    assert np.array_equal(cache.pool.cpu().numpy(), want[0])
