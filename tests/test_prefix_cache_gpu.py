"""GPU tests of attention over a shared prefix and each sequence's own pages of the
4-bit cache, against a 64-bit softmax over both (bounds: _serving_ref.attend_prefix,
plus half a bf16 step of O)."""
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


def _queries(rng, B, Hq, nq, dh, scale=1.0):
    return bf16(rng.normal(size=(B, Hq, nq, dh)) * scale)


def _tile_pages(B, Hq, Hkv, nq):
    """Pages of a prefix table from which on a prefix is worked on in tiles of 128 rows."""
    return -(-8192 // (Hkv * -(-B * (Hq // Hkv) * nq // 16)))


def _prefix_table(table, B, Hq, Hkv, nq, tiles):
    """The prefix's table, its width what the rule on sizes goes by (what is behind the prefix is not read)."""
    rows, width = B * (Hq // Hkv) * nq, len(table)
    if tiles:
        assert rows > 64
        width = max(width, _tile_pages(B, Hq, Hkv, nq))
    else:
        assert rows <= 64 or width < _tile_pages(B, Hq, Hkv, nq)
    return np.concatenate([table, np.full(width - len(table), -7, np.int32)])


def _case(seed, B, Hq, Hkv, nq, dh, dv, prefix, lengths, spread=0.0, more_pages=0, tiles=None):
    """The cache with the prefix as its first row, Q, and what the library gets.  tiles: whether
    the prefix goes to the tensor core's tiles (None: where there are rows for it)."""
    tiles = B * (Hq // Hkv) * nq > 64 if tiles is None else tiles
    rng = np.random.default_rng(seed)
    lengths = [lengths] * B if isinstance(lengths, int) else lengths
    wide = max(1, max(-(-n // PAGE) for n in [prefix] + lengths)) + more_pages
    c = srv.Paged(rng, Hkv, dh, dv, [prefix] + lengths, max_pages=wide, spread=spread)
    q = _queries(rng, B, Hq, nq, dh)
    own = max(1, max(-(-n // PAGE) for n in lengths)) + more_pages
    args = dict(prefix_table=_dev(_prefix_table(c.table[0], B, Hq, Hkv, nq, tiles)),
                prefix_length=_dev(np.array([prefix], np.int32)),
                page_table=_dev(c.table[1:, :own]), lengths=_dev(np.array(lengths, np.int32)))
    return c, q, args


def _check(c, q, O, LSE, nq, dh):
    O, LSE = f64(O), f64(LSE)
    for b, n in enumerate(c.lengths[1:]):
        rO, rL, eO, eL = srv.attend_prefix(q[b], c.K[0], c.V[0], c.K[b + 1], c.V[b + 1], n, dh ** -0.5)
        assert_within(O[b], rO, eO + 2.0 ** -8 * (np.abs(rO) + eO), "O")
        empty = rL == -np.inf
        assert np.array_equal(LSE[b] == -np.inf, empty) and (O[b][empty] == 0).all()
        assert_within(np.where(empty, 0.0, LSE[b]), np.where(empty, 0.0, rL), eL, "LSE")


def _run(c, q, args, dh, dv, **kw):
    import exact_scaled_dot_gb300 as esd
    cache = esd.QuantCache(_dev(c.pool), dh, dv)
    return esd.attn_fwd_prefix_cache(_dev(q).to(torch.bfloat16), cache, **args, **kw)


@pytest.mark.parametrize("dh,dv", [(64, 64), (128, 128), (128, 64)])
@pytest.mark.parametrize("B,Hq,Hkv,nq,prefix,lengths", [
    (1, 1, 1, 1, 1, 1),                                   # one key on each side
    (1, 4, 2, 1, 0, 70),                                  # no prefix
    (2, 4, 2, 1, 40, 0),                                  # no own keys
    (2, 2, 1, 3, 33, [0, 2]),                             # rows that see the prefix alone
    (3, 8, 2, 1, 500, [1, 40, 33]),
    (2, 5, 1, 2, 31, [32, 64]),
    (2, 6, 3, 5, 64, [5, 129]),
    (4, 8, 8, 16, 65, [16, 20, 100, 31]),                 # the most rows per head
    (40, 4, 1, 1, 127, 3),                                # more rows than a tile of 128
    (30, 16, 2, 3, 300, [3 + 7 * i for i in range(30)]),  # 720 rows of a head
    (2, 32, 1, 16, 129, [16, 50]),                        # 1024 rows of one head
])
def test_against_64_bits(B, Hq, Hkv, nq, prefix, lengths, dh, dv):
    for tiles in (False, True) if B * (Hq // Hkv) * nq > 64 else (False,):
        c, q, args = _case(B * 100 + prefix, B, Hq, Hkv, nq, dh, dv, prefix, lengths, tiles=tiles)
        O, LSE = _run(c, q, args, dh, dv)
        torch.cuda.synchronize()
        _check(c, q, O, LSE, nq, dh)


@pytest.mark.parametrize("prefix", [2047, 2048, 4100])
@pytest.mark.parametrize("B,dv", [(3, 128), (19, 128), (19, 64)])
def test_long_prefix(prefix, B, dv):
    """Many splits of the prefix, long own sequences that several CTAs share, wide tables."""
    c, q, args = _case(prefix, B, 8, 2, 2, 128, dv, prefix, [2, 1500, 2993] + [40] * (B - 3), more_pages=90)
    O, LSE = _run(c, q, args, 128, dv)
    torch.cuda.synchronize()
    _check(c, q, O, LSE, 2, 128)


@pytest.mark.parametrize("B", [2, 64])
def test_both_empty(B):
    """Nothing to see at all: 0 and -inf, whatever the pages and the row hold."""
    c, q, args = _case(5, B, 4, 2, 2, 128, 64, 0, 0)
    q[0, 0] = np.nan
    O, LSE = _run(c, q, args, 128, 64)
    torch.cuda.synchronize()
    assert (f64(O) == 0).all() and (f64(LSE) == -np.inf).all()


@pytest.mark.parametrize("B", [2, 40])
@pytest.mark.parametrize("spread", [4.0, 12.0])
def test_values_of_very_different_sizes(B, spread):
    """Scales of the values many octaves apart from key to key: every row keeps what it weighs."""
    dh = dv = 128
    c, q, args = _case(B, B, 8, 2, 1, dh, dv, 300, 33, spread=spread)
    q *= 4.0
    O, LSE = _run(c, q, args, dh, dv)
    torch.cuda.synchronize()
    O = f64(O)
    for b in range(B):
        K, V = np.concatenate([c.K[0], c.K[b + 1]]), np.concatenate([c.V[0], c.V[b + 1]])
        for r in range(8):
            s = K[:, r // 4] @ q[b, r, 0] * dh ** -0.5
            p = np.exp(s - s.max())
            A = p / p.sum()
            want = A @ V[:, r // 4]
            bound = _weighted_bound(A, s, K[:, r // 4], V[:, r // 4], q[b, r, 0], dh)
            assert_within(O[b, r, 0], want, bound + 2.0 ** -8 * (np.abs(want) + bound), "O")


def _many_heads(seed, B, group, dh, dv, prefix, lengths):
    """19 KV heads: eight ranges of the prefix, each of many of its tiles."""
    rng = np.random.default_rng(seed)
    p = srv.Paged(rng, 19, dh, dv, [prefix])
    return rng, p, lambda: srv.behind(rng, p, lengths), _queries(rng, B, 19 * group, 1, dh)


def _many_args(c, B, group):
    return dict(prefix_table=_dev(_prefix_table(c.prefix_table, B, 19 * group, 19, 1, True)),
                prefix_length=_dev(np.array(c.lengths[:1], np.int32)), page_table=_dev(c.table),
                lengths=_dev(np.array(c.lengths[1:], np.int32)))


@pytest.mark.parametrize("dh,dv", [(64, 64), (128, 128), (128, 64)])
@pytest.mark.parametrize("B,group", [(40, 2), (40, 4), (20, 5)])
@pytest.mark.parametrize("prefix", [1100, 4100])
def test_many_tiles_in_a_range(B, group, prefix, dh, dv):
    """Rows of 80 (one row tile), 160 and 100 a head; ranges of two to nine tiles of 64 keys."""
    _, _, cache, q = _many_heads(prefix + B, B, group, dh, dv, prefix, [1 + i for i in range(B)])
    c = cache()
    O, LSE = _run(c, q, _many_args(c, B, group), dh, dv)
    torch.cuda.synchronize()
    O, LSE = f64(O), f64(LSE)
    for b in (0, B // 2, B - 1):
        for h in (0, 7, 18):
            at = slice(h * group, (h + 1) * group)
            rO, rL, eO, eL = srv.attend_prefix(q[b, at], c.K[0][:, h:h + 1], c.V[0][:, h:h + 1], c.K[b + 1][:, h:h + 1],
                                               c.V[b + 1][:, h:h + 1], c.lengths[b + 1], dh ** -0.5)
            assert_within(O[b, at], rO, eO + 2.0 ** -8 * (np.abs(rO) + eO), "O")
            assert_within(LSE[b, at], rL, eL, "LSE")


@pytest.mark.parametrize("B,group", [(40, 4), (20, 4)])
@pytest.mark.parametrize("dh,dv", [(64, 64), (128, 128), (128, 64)])
def test_scores_that_climb_for_some_rows(B, group, dh, dv):
    """Two sequences' scores rise by 11 octaves every 64 keys, so that those rows' sums of
    weights pass what a tile may hold again and again while the others' never do."""
    rng, p, cache, q = _many_heads(B + dv, B, group, dh, dv, 4100, [3] * B)
    u = np.sign(rng.normal(size=(19, dh)))
    climb = 8.0 * (np.arange(4100) // 64 % 9) / dh ** 0.5
    K = bf16(rng.normal(size=(4100, 19, dh)) * 0.25 + climb[:, None, None] * u)
    ref.store(p.pool, p.slots(0, 4100), K, bf16(rng.normal(size=(4100, 19, dv))))
    p.K[0], p.V[0] = ref.load(p.pool, p.slots(0, 4100), dh, dv)
    c = cache()
    q = bf16(q * 0.01)
    few = (9, B - 3)
    for b in few:
        q[b, :, 0] = bf16(np.repeat(u, group, 0) * (1 + np.arange(19 * group)[:, None] % 3 * 0.25))
    args = _many_args(c, B, group)
    O, LSE = _run(c, q, args, dh, dv)
    for _ in range(5):
        again = _run(c, q, args, dh, dv)
        assert torch.equal(O, again[0]) and torch.equal(LSE, again[1])
    O, LSE = f64(O), f64(LSE)
    for b in (*few, 0):
        for h in (0, 7, 18):
            at = slice(h * group, (h + 1) * group)
            rO, rL, eO, eL = srv.attend_prefix(q[b, at], c.K[0][:, h:h + 1], c.V[0][:, h:h + 1], c.K[b + 1][:, h:h + 1],
                                               c.V[b + 1][:, h:h + 1], c.lengths[b + 1], dh ** -0.5)
            assert_within(O[b, at], rO, eO + 2.0 ** -8 * (np.abs(rO) + eO), "O")
            assert_within(LSE[b, at], rL, eL, "LSE")


@pytest.mark.parametrize("group", [4, 16])
@pytest.mark.parametrize("at", [40, 700])
@pytest.mark.parametrize("of", ["k", "v", "both"])
def test_scales_that_change_along_the_prefix(group, at, of):
    """Keys or values whose scales leave what went before, from one token on: some tiles are
    taken with their scales in the operands, the others with the scales beside them."""
    dh = dv = 128
    B, prefix = 24, 2300
    rng, p, cache, q = _many_heads(at, B, group, dh, dv, prefix, [2] * B)
    size = np.where(np.arange(prefix) < at, 1.0, np.exp2(rng.integers(-15, 12, prefix)))[:, None, None]
    K, V = rng.normal(size=(prefix, 19, dh)), rng.normal(size=(prefix, 19, dv))
    # (large keys would leave one score each row: they get small ones)
    K, V = bf16(K * (np.minimum(size, 2.0) if of != "v" else 1.0)), bf16(V * (size if of != "k" else 1.0))
    if of != "v":
        K[at + 5] *= 2.0 ** -14                     # further apart than a tile's scales may be
    K[:, :, 64:] = np.abs(K[:, :, 64:])             # a zero point of 0
    ref.store(p.pool, p.slots(0, prefix), K, V)
    p.K[0], p.V[0] = ref.load(p.pool, p.slots(0, prefix), dh, dv)
    c = cache()
    O, LSE = _run(c, q, _many_args(c, B, group), dh, dv)
    torch.cuda.synchronize()
    O, LSE = f64(O), f64(LSE)
    for b in (0, 13, 23):
        for h in (0, 18):
            K, V = (np.concatenate([x[0], x[b + 1]])[:, h] for x in (c.K, c.V))
            for r in range(h * group, (h + 1) * group, 3):
                _, rL, _, eL = ref.attend(q[b, r:r + 1], K[:, None], V[:, None], len(K), dh ** -0.5)
                assert_within(LSE[b, r], rL[0], eL[0] + 258 * 2.0 ** -23, "LSE")
                s = K @ q[b, r, 0] * dh ** -0.5
                A = np.exp(s - s.max())
                A /= A.sum()
                want, bound = A @ V, _weighted_bound(A, s, K, V, q[b, r, 0], dh)
                assert_within(O[b, r, 0], want, bound + 2.0 ** -8 * (np.abs(want) + bound), "O")


def _weighted_bound(A, s, K, V, q, dh):
    """Per group of 64 dims: what the weights times the group's largest values are off by
    together, 2^-11 of each product, 2^-29 of the largest, as the header says; the scores'
    errors; the sums'."""
    size = np.repeat(np.abs(V.reshape(len(V), -1, 64)).max(-1), 64, -1)
    ds = 132 * 2.0 ** -24 * dh ** -0.5 * (np.abs(K) @ np.abs(q))
    rel = 2.0 ** -11 + 2 * (ds + 2.0 ** -20 * (1 + np.abs(s - s.max()) + abs(s.max()) / 4))
    prod = A[:, None] * size
    bound = (rel[:, None] * prod).sum(0) + len(V) * 2.0 ** -27 * prod.max(0)
    return bound + 2 * (len(V) / 16 + 8) * 2.0 ** -23 * 2.2 * prod.sum(0)


@pytest.mark.parametrize("B", [1, 33])
def test_rows_that_are_not_finite(B):
    c, q, args = _case(9, B, 4, 1, 2, 64, 64, 50, 9)
    q[0, 1, 0, 5] = np.inf
    q[B - 1, 3, 1, 60] = np.nan
    O, LSE = _run(c, q, args, 64, 64)
    torch.cuda.synchronize()
    bad = np.zeros((B, 4, 2), bool)
    bad[0, 1, 0] = bad[B - 1, 3, 1] = True
    assert np.array_equal(np.isnan(f64(LSE)), bad)
    assert np.array_equal(np.isnan(f64(O)).all(-1), bad) and not np.isnan(f64(O)[~bad]).any()


@pytest.mark.parametrize("B", [2, 36])
@pytest.mark.parametrize("size", [2.0 ** -40, 2.0 ** 30])
def test_queries_of_any_size(B, size):
    """Scores that are all alike or far apart; the scale brings large rows back."""
    c, q, args = _case(11, B, 4, 1, 1, 128, 128, 200, 40)
    q = bf16(q * size)
    O, LSE = _run(c, q, args, 128, 128, scale=dh_scale(size))
    torch.cuda.synchronize()
    O, LSE = f64(O), f64(LSE)
    for b, n in enumerate(c.lengths[1:]):
        rO, rL, eO, eL = srv.attend_prefix(q[b], c.K[0], c.V[0], c.K[b + 1], c.V[b + 1], n, dh_scale(size))
        assert_within(O[b], rO, eO + 2.0 ** -8 * (np.abs(rO) + eO), "O")
        assert_within(LSE[b], rL, eL, "LSE")


def dh_scale(size):
    return float(np.float32(128 ** -0.5 * (1.0 / size if size > 1 else 1.0)))


def test_same_as_the_decode_over_one_table():
    """With the prefix's pages in front of each sequence's (a prefix of whole pages), the decode
    over the cache is the same function."""
    import exact_scaled_dot_gb300 as esd
    c, q, args = _case(3, 6, 16, 4, 2, 128, 64, 5 * PAGE, [2, 50, 64, 33, 7, 100])
    cache = esd.QuantCache(_dev(c.pool), 128, 64)
    Q = _dev(q).to(torch.bfloat16)
    O, LSE = esd.attn_fwd_prefix_cache(Q, cache, **args)
    table = torch.cat([args["prefix_table"][:5].expand(6, -1), args["page_table"]], 1).contiguous()
    O2, LSE2 = esd.attn_fwd_decode_cache(Q, cache, table, args["lengths"] + 5 * PAGE)
    torch.cuda.synchronize()
    assert (LSE - LSE2).abs().max() < 1e-4
    assert ((O - O2).abs().float() <= 2.0 ** -7 * O2.abs().float() + 2e-3).all()


@pytest.mark.parametrize("B", [2, 40])
def test_indices_out_of_range_are_left_out_and_reported(B):
    import exact_scaled_dot_gb300 as esd
    c, q, args = _case(21, B, 4, 2, 1, 128, 128, 4 * PAGE, [70] * B)
    cache = esd.QuantCache(_dev(c.pool), 128, 128)
    Q = _dev(q).to(torch.bfloat16)
    good = dict(args)

    def reported(**kw):
        out = esd.attn_fwd_prefix_cache(Q, cache, **{**args, **kw})
        torch.cuda.synchronize()
        assert esd.attn_get_status() == esd.ATTN_ERR_PAGE
        esd.attn_clear_status()
        return out

    # the prefix's second page: its keys are left out
    t = args["prefix_table"].clone()
    t[1] = 2 ** 31 - 1
    O, LSE = reported(prefix_table=t)
    keep = np.r_[0:PAGE, 2 * PAGE:4 * PAGE]
    c.K[0], c.V[0], whole = c.K[0][keep], c.V[0][keep], (c.K[0], c.V[0])
    _check(c, q, O, LSE, 1, 128)
    c.K[0], c.V[0] = whole
    # lengths past the tables are cut to them
    O, LSE = reported(prefix_table=args["prefix_table"][:4].contiguous(),
                      prefix_length=torch.tensor([1 << 30], dtype=torch.int32, device="cuda"))
    _check(c, q, O, LSE, 1, 128)
    O, LSE = reported(page_table=torch.full_like(args["page_table"], -5))
    c.lengths = [4 * PAGE] + [0] * B
    _check(c, q, O, LSE, 1, 128)
    # negative lengths are no keys
    O, LSE = esd.attn_fwd_prefix_cache(Q, cache, **{**good, "lengths": torch.full_like(args["lengths"], -3)})
    _check(c, q, O, LSE, 1, 128)


@pytest.mark.parametrize("B", [3, 50])
def test_captured_call_follows_lengths_and_tables(B):
    import exact_scaled_dot_gb300 as esd
    c, q, args = _case(31, B, 8, 2, 1, 128, 128, 200, [5 + i for i in range(B)])
    cache = esd.QuantCache(_dev(c.pool), 128, 128)
    Q = _dev(q).to(torch.bfloat16)
    O, LSE = (torch.empty((B, 8, 1, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((B, 8, 1), device="cuda"))
    ws = torch.empty(esd.attn_fwd_prefix_cache_workspace_bytes(cache, B, 8, 1, len(args["prefix_table"]),
                                                               args["page_table"].shape[1]),
                     dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        esd.attn_fwd_prefix_cache(Q, cache, **args, O=O, LSE=LSE, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        esd.attn_fwd_prefix_cache(Q, cache, **args, O=O, LSE=LSE, workspace=ws)
    O2, LSE2 = torch.empty_like(O), torch.empty_like(LSE)
    with torch.cuda.graph(other):                    # the same workspace in another graph
        esd.attn_fwd_prefix_cache(Q, cache, **args, O=O2, LSE=LSE2, workspace=ws)
    for prefix, less in ((200, 0), (7, 3), (0, 1), (129, 2)):
        args["prefix_length"].fill_(prefix)
        lengths = [max(0, 5 + i - less) for i in range(B)]
        args["lengths"].copy_(torch.tensor(lengths, dtype=torch.int32))
        ws.fill_(0xFF)                               # what a workspace holds on entry does not matter
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
        kp, vp = c.K[0], c.V[0]
        c.K[0], c.V[0], c.lengths = kp[:prefix], vp[:prefix], [prefix] + lengths
        _check(c, q, O, LSE, 1, 128)
        c.K[0], c.V[0] = kp, vp


@pytest.mark.parametrize("B", [4, 48])
def test_repeatable_and_on_another_stream(B):
    import exact_scaled_dot_gb300 as esd
    c, q, args = _case(41, B, 8, 1, 2, 64, 64, 1000, [2 + 9 * i for i in range(B)])
    cache = esd.QuantCache(_dev(c.pool), 64, 64)
    Q = _dev(q).to(torch.bfloat16)
    O, LSE = esd.attn_fwd_prefix_cache(Q, cache, **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    O2, LSE2 = esd.attn_fwd_prefix_cache(Q, cache, **args, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    _check(c, q, O, LSE, 2, 64)


def test_two_streams_at_once():
    """Calls of both divisions, weights and evictions that overlap on the GPU, each with buffers of
    its own: the bits of the same calls one after the other."""
    import exact_scaled_dot_gb300 as esd
    jobs = []
    for seed, B, nq in ((51, 40, 2), (52, 48, 1), (53, 3, 2)):
        c, q, args = _case(seed, B, 8, 2, nq, 128, 128, 3000, [nq + 21 * i for i in range(B)])
        w = torch.rand((B, 2, args["page_table"].shape[1] * PAGE), device="cuda")
        jobs.append((_dev(c.pool), _dev(q).to(torch.bfloat16), args, w))

    def run(pool, Q, args, w):
        cache, w = esd.QuantCache(pool, 128, 128), w.clone()
        O, LSE = esd.attn_fwd_prefix_cache(Q, cache, **args)
        own = dict(page_table=args["page_table"], lengths=args["lengths"])
        esd.attn_cache_weigh(Q, cache, **own, LSE=LSE, weights=w)
        return O, LSE, w, *esd.attn_cache_evict(cache, **own, weights=w, keep=40, first=4, recent=8), pool

    want = []
    for pool, *rest in jobs:
        want.append(run(pool.clone(), *rest))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(4):
        pools = [pool.clone() for pool, *_ in jobs]
        torch.cuda.synchronize()
        got = []
        for s, pool, (_, *rest) in zip(streams, pools, jobs):
            with torch.cuda.stream(s):
                got.append(run(pool, *rest))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("B", [3, 40])
def test_pages_past_32_bits(B):
    """The last pages of a pool of 4.7 GB give the bits that those of a small one do."""
    import exact_scaled_dot_gb300 as esd
    c, q, args = _case(61, B, 8, 2, 1, 64, 64, 900, [1 + 13 * i for i in range(B)])
    pool, Q = _dev(c.pool), _dev(q).to(torch.bfloat16)
    far = (4_700_000_000 // pool[0].numel()) - len(pool)
    large = torch.empty((far + len(pool), *pool.shape[1:]), dtype=torch.uint8, device="cuda")
    large[far:] = pool
    w = torch.rand((B, 2, args["page_table"].shape[1] * PAGE), device="cuda")
    got = []
    for p, by in ((pool, 0), (large, far)):
        cache, weights = esd.QuantCache(p, 64, 64), w.clone()
        table, prefix = args["page_table"] + by, args["prefix_table"] + by
        O, LSE = esd.attn_fwd_prefix_cache(Q, cache, prefix, args["prefix_length"], table, args["lengths"])
        esd.attn_cache_weigh(Q, cache, table, args["lengths"], LSE, weights)
        got.append((O, LSE, weights, *esd.attn_cache_evict(cache, table, args["lengths"], weights, 20, first=2, recent=4)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert torch.equal(large[far:], pool)


def _phases(seed, group, K, V, phase):
    """A prefix of eight ranges of 7 tiles of 64 keys for 19 KV heads, without own keys: K(n, u, phase) and
    V(n, phase) give the keys and values [n, 19, 128] of each phase of a range (tile i of it is in phase(i)),
    the first key of the last phase is far smaller than the others of its tile, so that scales are beside
    the operands from there on.  Rows are alike up to a factor, along u."""
    B, dh, tiles = 24, 128, 7
    rng, p, cache, q = _many_heads(seed, B, group, dh, dh, 8 * tiles * 64, [0] * B)
    u = np.sign(rng.normal(size=(19, dh)))
    of = np.repeat([phase(i % tiles) for i in range(8 * tiles)], 64)
    keys, values = np.zeros((len(of), 19, dh)), np.zeros((len(of), 19, dh))
    for x in np.unique(of):
        n = int((of == x).sum())
        keys[of == x], values[of == x] = K(rng, n, u, x), V(rng, n, x)
    first = np.flatnonzero((of == of.max()) & (np.roll(of, 1) != of.max()))
    keys[first] *= 2.0 ** -16
    ref.store(p.pool, p.slots(0, len(of)), bf16(keys), bf16(values))
    p.K[0], p.V[0] = ref.load(p.pool, p.slots(0, len(of)), dh, dh)
    c = cache()
    q = bf16(u[None].repeat(group, 1)[:, :, None] * (1 + np.arange(B)[:, None, None, None] % 3 * 0.25)
             + 0.01 * q)
    O, LSE = _run(c, q, _many_args(c, B, group), dh, dh)
    torch.cuda.synchronize()
    O, LSE = f64(O), f64(LSE)
    for b in (0, 13, 23):
        for h in (0, 18):
            K, V = c.K[0][:, h], c.V[0][:, h]
            for r in range(h * group, (h + 1) * group, 3):
                _, rL, _, eL = ref.attend(q[b, r:r + 1], K[:, None], V[:, None], len(K), dh ** -0.5)
                assert_within(LSE[b, r], rL[0], eL[0] + 258 * 2.0 ** -23, "LSE")
                s = K @ q[b, r, 0] * dh ** -0.5
                A = np.exp(s - s.max())
                A /= A.sum()
                want, bound = A @ V, _weighted_bound(A, s, K, V, q[b, r, 0], dh)
                assert_within(O[b, r, 0], want, bound + 2.0 ** -8 * (np.abs(want) + bound), "O")


@pytest.mark.parametrize("group", [4, 16])
@pytest.mark.parametrize("octaves", [20, 30, 60, 90])
@pytest.mark.parametrize("groups", [(1,), (0, 1)])
def test_no_values_before_the_scales_part(group, octaves, groups):
    """A group of 64 dims has no value but 0 while scales are in the operands, and small ones behind."""
    def values(rng, n, phase):
        V = rng.normal(size=(n, 19, 128))
        for g in groups:
            V[:, :, 64 * g:64 * g + 64] *= 2.0 ** -octaves if phase else 0.0
        return V
    _phases(group + octaves, group, lambda rng, n, u, phase: 0.3 * rng.normal(size=(n, 19, 128)), values,
            lambda tile: int(tile > 2))


@pytest.mark.parametrize("group", [4, 16])
@pytest.mark.parametrize("octaves", [25, 35, 80, 120])
def test_values_that_no_longer_weigh_before_the_scales_part(group, octaves):
    """Scores rise by more octaves than the values fall while scales are in the operands, at keys whose
    values are 0; behind, what there was before weighs less than the small values."""
    climb = (octaves + 8) * np.log(2.0) * 128 ** -0.5

    def keys(rng, n, u, phase):
        return 0.02 * rng.normal(size=(n, 19, 128)) + (climb if phase else 0.0) * u

    def values(rng, n, phase):
        return rng.normal(size=(n, 19, 128)) * (2.0 ** 40, 0.0, 2.0 ** (40 - octaves))[phase]
    _phases(group + octaves, group, keys, values, lambda tile: 0 if tile < 2 else 1 if tile < 4 else 2)
