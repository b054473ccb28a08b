"""GPU tests of the 4-bit cache: what is written (bit for bit), what is read
back, and attention over it, against 64-bit forms over the stored values.

Bounds of the attention: _qk_cache_ref.attend, plus half a bf16 step of O."""
import numpy as np
import pytest
import torch

import _qk_cache_ref as ref
from _qk_cache_ref import assert_within, f64

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


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy(rng.normal(size=shape) * scale).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# Writing and reading
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,Hkv,dh,dv", [(1, 1, 64, 64), (33, 2, 128, 128), (100, 3, 128, 64), (1000, 8, 128, 128)])
@pytest.mark.parametrize("strided", [False, True])
def test_append_and_read(T, Hkv, dh, dv, strided):
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(T + dh)
    pages = T // PAGE + 5
    K = _bf16(rng, T, Hkv, dh) * torch.from_numpy(np.exp(2 * rng.normal(size=(T, Hkv, 1)))).to(torch.bfloat16)
    V = _bf16(rng, T, Hkv, dv)
    K[0, 0, :64] = 0.0                                  # an all-zero group
    K[T // 2, 0] = K[T // 2, 0].abs()                   # no negative element
    V[T // 3, -1] = -V[T // 3, -1].abs()                # no positive one
    V[-1, 0, :64] = torch.arange(64).to(torch.bfloat16) * 0.5    # ties of the rounding
    slots = rng.permutation(pages * PAGE)[:T]
    slots[rng.random(T) < 0.1] = -1                     # padding
    before = rng.integers(0, 256, (pages, Hkv, esd.attn_cache_page_bytes(Hkv, dh, dv) // Hkv)).astype(np.uint8)
    cache = esd.QuantCache(torch.from_numpy(before.copy()).cuda(), dh, dv)
    if strided:
        x = torch.zeros((T, 2 * Hkv + 1, 128), dtype=torch.bfloat16, device="cuda")
        Kd, Vd = x[:, :Hkv, :dh], x[:, Hkv:2 * Hkv, 128 - dv:]
        Kd.copy_(K), Vd.copy_(V)
    else:
        Kd, Vd = K.cuda(), V.cuda()
    S = torch.from_numpy(slots).cuda()
    esd.attn_cache_append(cache, Kd, Vd, S)
    Kr, Vr = esd.attn_cache_read(cache, S)
    torch.cuda.synchronize()
    want = before.copy()
    ref.store(want, slots, f64(K), f64(V))
    assert np.array_equal(cache.pool.cpu().numpy(), want)     # the tokens' bytes, and no others
    on = slots >= 0
    kv, vv = ref.load(want, slots[on], dh, dv)
    for got, val in ((Kr, kv), (Vr, vv)):
        got = f64(got)
        assert np.array_equal(got[on], ref.bf16(val))
        assert (got[~on] == 0).all()
    if strided:                                               # results into views, nothing beside them
        x.fill_(7.0)
        esd.attn_cache_read(cache, S, K=Kd, V=Vd)
        torch.cuda.synchronize()
        assert torch.equal(Kd, Kr) and torch.equal(Vd, Vr)
        assert (x[:, 2 * Hkv:] == 7).all() and (x[:, :Hkv, dh:] == 7).all() and (x[:, Hkv:2 * Hkv, :128 - dv] == 7).all()


def test_scales_of_every_size_round_trip():
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(8)
    T = 240
    mag = torch.from_numpy(2.0 ** np.arange(-120, 120)[:, None, None])
    K = (torch.from_numpy(rng.normal(size=(T, 1, 64))) * mag).to(torch.bfloat16)
    cache = esd.QuantCache.empty(8, 1, 64, 64)
    S = torch.arange(T, device="cuda")
    esd.attn_cache_append(cache, K.cuda(), (-K).cuda(), S)
    Kr, Vr = esd.attn_cache_read(cache, S)
    torch.cuda.synchronize()
    for got, x in ((Kr, f64(K)), (Vr, -f64(K))):
        c, s, z = ref.quantize(x)
        # (fp32 scales below its normal range lose bits: those rows are left out)
        keep = (s > 2.0 ** -120)[..., 0]
        assert keep.sum() > 220
        assert np.array_equal(f64(got)[keep], ref.bf16(ref.values(c, s, z))[keep])


@pytest.mark.parametrize("columns", [3, 80])
def test_indices_past_the_pool_are_left_out_and_reported(columns):
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(4)
    cache = esd.QuantCache(torch.zeros((3, 2, 32 * 128 * 9 // 16), dtype=torch.uint8, device="cuda"), 64, 64)
    K = _bf16(rng, 4, 2, 64).cuda()
    slots = torch.tensor([5, 96, 1 << 40, -(1 << 40)], device="cuda")
    esd.attn_cache_append(cache, K, K, slots)
    torch.cuda.synchronize()
    assert esd.attn_get_status() == esd.ATTN_ERR_PAGE
    esd.attn_clear_status()
    Kr, _ = esd.attn_cache_read(cache, slots)
    torch.cuda.synchronize()
    assert esd.attn_get_status() == esd.ATTN_ERR_PAGE
    esd.attn_clear_status()
    assert (Kr[1:] == 0).all() and (Kr[0] != 0).any()
    want = np.zeros((3, 2, 32 * 128 * 9 // 16), dtype=np.uint8)
    ref.store(want, slots.cpu().numpy(), f64(K), f64(K))
    assert np.array_equal(cache.pool.cpu().numpy(), want)
    # a page number outside the pool: its keys are left out; a length above the table: cut
    esd.attn_cache_append(cache, _bf16(rng, 96, 2, 64).cuda(), _bf16(rng, 96, 2, 64).cuda(), torch.arange(96, device="cuda"))
    Q = _bf16(rng, 2, 4, 1, 64).cuda()
    two = torch.full((2, columns), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    two[:, :3] = torch.tensor([[0, 3, 2], [0, -1, 2]])
    O, LSE = esd.attn_fwd_decode_cache(Q, cache, two, torch.tensor([90, 10000], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert esd.attn_get_status() == esd.ATTN_ERR_PAGE
    esd.attn_clear_status()
    left = torch.tensor([[0, 2], [0, 2]], dtype=torch.int32, device="cuda")
    O2, LSE2 = esd.attn_fwd_decode_cache(Q, cache, left, torch.tensor([58, 64], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    np.testing.assert_allclose(f64(O), f64(O2), atol=1e-2, rtol=2 * ref.BF16)
    np.testing.assert_allclose(f64(LSE), f64(LSE2), atol=1e-5, rtol=0)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def _filled(rng, lengths, Hkv, dh, dv, K=None, V=None, spare=3, wide=None):
    """A pool with the sequences in scattered pages; everything that no
    sequence owns is 0xFF (scales of NaN), page numbers past a sequence's
    end are out of range.  Returns cache, table, lengths (device) and the values."""
    import exact_scaled_dot_gb300 as esd
    B = len(lengths)
    need = [-(-n // PAGE) for n in lengths]
    wide = max(1, max(need)) if wide is None else wide
    pages = sum(need) + spare
    order = rng.permutation(pages)
    pool = np.full((pages, Hkv, esd.attn_cache_page_bytes(Hkv, dh, dv) // Hkv), 0xFF, dtype=np.uint8)
    table = np.full((B, wide), 2 ** 31 - 1, dtype=np.int32)
    vals, used = [], 0
    for b, n in enumerate(lengths):
        table[b, :need[b]] = order[used:used + need[b]]
        used += need[b]
        if n == 0:
            vals.append([np.zeros((0, Hkv, w)) for w in (dh, dv)])
            continue
        k = _bf16(rng, n, Hkv, dh) if K is None else K(b, n)
        v = _bf16(rng, n, Hkv, dv) if V is None else V(b, n)
        t = np.arange(n)
        slots = table[b, t // PAGE].astype(np.int64) * PAGE + t % PAGE
        ref.store(pool, slots, f64(k), f64(v))
        vals.append(ref.load(pool, slots, dh, dv))
    return (esd.QuantCache(torch.from_numpy(pool).cuda(), dh, dv), torch.from_numpy(table).cuda(),
            torch.tensor(lengths, dtype=torch.int32, device="cuda"), vals)


def _attend_and_check(Q, cache, table, lens, vals, scale=None, **kw):
    import exact_scaled_dot_gb300 as esd
    B, Hq, nq, dh = Q.shape
    O = torch.full((B, Hq, nq, cache.d_v), float("nan"), dtype=torch.bfloat16, device="cuda")
    LSE = torch.full((B, Hq, nq), float("nan"), dtype=torch.float32, device="cuda")
    esd.attn_fwd_decode_cache(Q.cuda(), cache, table, lens, O=O, LSE=LSE, scale=scale, **kw)
    torch.cuda.synchronize()
    assert esd.attn_get_status() == 0
    for b in range(B):
        o, l, oerr, lerr = ref.attend(f64(Q[b]), *vals[b], int(lens[b]), dh ** -0.5 if scale is None else scale)
        assert_within(f64(O[b]), o, ref.BF16 * np.abs(o) + oerr, f"O[{b}]")
        got = f64(LSE[b])
        assert np.array_equal(np.isneginf(got), np.isneginf(l)), f"LSE[{b}]"
        on = ~np.isneginf(l)
        assert_within(got[on], l[on], lerr[on], f"LSE[{b}]")
    return O, LSE


# B lengths, Hq, Hkv, n_q, dh, dv
CASES = {
    "one_key": ([1], 1, 1, 1, 64, 64),
    "page_ends": ([31, 32, 33, 63, 64, 65], 8, 2, 1, 128, 128),
    "no_key": ([0, 5, 0, 40], 4, 2, 1, 128, 64),
    "no_key_at_all": ([0, 0, 0], 4, 2, 1, 64, 64),
    "one_page_of_many_sequences": ([5, 31, 32, 1, 0, 17, 30, 2, 9, 12, 3, 0, 0, 28, 6, 7, 8] * 4, 4, 2, 1, 64, 64),
    "rows_before_the_first_token": ([1, 2, 3, 300], 6, 2, 4, 64, 64),
    "group_5_of_3_queries": ([17, 450, 129], 10, 2, 3, 128, 128),
    "nine_rows": ([500, 31], 9, 1, 1, 128, 128),
    "seventeen_rows": ([257, 700], 17, 1, 1, 128, 64),
    "sixteen_queries": ([16, 900], 4, 2, 16, 64, 64),
    "mqa_64_rows": ([2100], 64, 1, 1, 128, 128),
    "mha": ([333, 64], 8, 8, 2, 128, 128),
    "ragged_split": ([4000, 1, 700, 255, 256, 257], 8, 2, 1, 128, 128),
    "long": ([9001], 4, 1, 2, 128, 64),
    "more_tiles_than_ctas": ([4200], 300, 1, 16, 64, 64),
    "many_short": ([int(n) for n in np.random.default_rng(36).integers(0, 700, 41)], 16, 4, 1, 128, 128),
    "many_short_16_rows": ([int(n) for n in np.random.default_rng(37).integers(0, 500, 44)], 8, 4, 5, 64, 64),
}


@pytest.mark.parametrize("spare_columns", [0, 70])
@pytest.mark.parametrize("name", list(CASES))
def test_attention_over_the_cache(name, spare_columns):
    """With the narrowest table, and with a wide one (which is cut into ranges of pages instead)."""
    lengths, Hq, Hkv, nq, dh, dv = CASES[name]
    rng = np.random.default_rng(len(name))
    wide = max(1, max(-(-n // PAGE) for n in lengths)) + spare_columns
    cache, table, lens, vals = _filled(rng, lengths, Hkv, dh, dv, wide=wide)
    _attend_and_check(_bf16(rng, len(lengths), Hq, nq, dh), cache, table, lens, vals)


def test_peaked_scores_and_given_scale():
    rng = np.random.default_rng(21)
    cache, table, lens, vals = _filled(rng, [1000, 70], 2, 128, 128, K=lambda b, n: _bf16(rng, n, 2, 128, scale=3.0))
    _attend_and_check(_bf16(rng, 2, 8, 1, 128, scale=3.0), cache, table, lens, vals, scale=0.1)


def test_scores_that_grow_along_the_sequence():
    """Every page raises the running maximum, so O and the sums are rescaled throughout."""
    rng = np.random.default_rng(22)
    u = rng.normal(size=64)

    def K(b, n):
        return torch.from_numpy(np.linspace(0, 12, n)[:, None, None] * u + 0.1 * rng.normal(size=(n, 1, 64))).to(torch.bfloat16)

    cache, table, lens, vals = _filled(rng, [1500], 1, 64, 64, K=K)
    _attend_and_check(torch.from_numpy(u[None, None, None]).to(torch.bfloat16).expand(1, 4, 1, 64).contiguous(), cache,
                      table, lens, vals)


@pytest.mark.parametrize("lo,hi", [(-30, 30), (30, -30), (-90, -80), (60, 80)])
def test_value_scales_that_change_along_the_sequence(lo, hi):
    rng = np.random.default_rng(23)

    def V(b, n):
        e = np.linspace(lo, hi, n)[:, None, None]
        return torch.from_numpy(rng.normal(size=(n, 2, 128)) * 2.0 ** e).to(torch.bfloat16)

    cache, table, lens, vals = _filled(rng, [900, 40], 2, 128, 128, V=V)
    _attend_and_check(_bf16(rng, 2, 4, 1, 128), cache, table, lens, vals)


def test_zero_keys_values_and_queries():
    rng = np.random.default_rng(24)
    zero = lambda d: (lambda b, n: torch.zeros((n, 1, d), dtype=torch.bfloat16))  # noqa: E731
    cache, table, lens, vals = _filled(rng, [100], 1, 128, 64, K=zero(128), V=zero(64))
    O, _ = _attend_and_check(_bf16(rng, 1, 4, 1, 128), cache, table, lens, vals)
    assert (O == 0).all()
    cache, table, lens, vals = _filled(rng, [100], 1, 128, 64)
    _attend_and_check(torch.zeros((1, 4, 1, 128), dtype=torch.bfloat16), cache, table, lens, vals)


@pytest.mark.parametrize("e", [-100, -20, 20, 60])
def test_query_scales(e):
    """Queries far from 1 with the scale that brings the scores back."""
    rng = np.random.default_rng(25)
    cache, table, lens, vals = _filled(rng, [200], 2, 64, 64)
    Q = (_bf16(rng, 1, 4, 2, 64).double() * 2.0 ** e).to(torch.bfloat16)
    _attend_and_check(Q, cache, table, lens, vals, scale=2.0 ** -e / 8)


def test_tiny_scale_beside_masked_keys():
    """Scores that all vanish (the scale times the queries' own is below fp32's range): equal weights."""
    rng = np.random.default_rng(34)
    cache, table, lens, vals = _filled(rng, [200, 35], 2, 128, 64)
    Q = (_bf16(rng, 2, 4, 3, 128).double() * 2.0 ** -115).to(torch.bfloat16)
    _attend_and_check(Q, cache, table, lens, vals, scale=2.0 ** -40)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_a_query_row_that_is_not_finite_gives_nan_alone(value):
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(35)
    cache, table, lens, _ = _filled(rng, [3000, 35], 2, 128, 128)
    Q = _bf16(rng, 2, 4, 2, 128).cuda()
    O, LSE = esd.attn_fwd_decode_cache(Q, cache, table, lens)
    Q[0, 1, 0, 77] = Q[1, 2, 1, 0] = value
    O2, LSE2 = esd.attn_fwd_decode_cache(Q, cache, table, lens)
    torch.cuda.synchronize()
    assert esd.attn_get_status() == 0
    row = torch.zeros((2, 4, 2), dtype=torch.bool, device="cuda")
    row[0, 1, 0] = row[1, 2, 1] = True
    assert O2[row].isnan().all() and LSE2[row].isnan().all()
    assert torch.equal(O2[~row], O[~row]) and torch.equal(LSE2[~row], LSE[~row])


def test_a_timeout_replaces_a_page_report():
    """Only a timeout stops later calls, so it must not be lost behind an earlier report."""
    import exact_scaled_dot_gb300 as esd
    cache = esd.QuantCache.empty(1, 1, 64, 64)
    cache.pool.zero_()
    try:
        esd.attn_cache_read(cache, torch.tensor([32], device="cuda"))
        torch.cuda.synchronize()
        assert esd.attn_get_status() == esd.ATTN_ERR_PAGE
        esd.attn_selftest_wait_timeout(50_000_000)
        torch.cuda.synchronize()
        assert esd.attn_get_status() == esd.ATTN_ERR_TIMEOUT
    finally:
        esd.attn_clear_status()


def test_shared_pages_and_a_wider_table():
    """Sequences that share their first pages (a forked prompt), in a table wider than any of them."""
    rng = np.random.default_rng(26)
    cache, table, lens, vals = _filled(rng, [320, 64, 50], 2, 128, 128, wide=200)
    table[1, :2] = table[0, :2]
    vals[1] = [x[:64] for x in vals[0]]
    _attend_and_check(_bf16(rng, 3, 4, 1, 128), cache, table, lens, vals)


def test_workspace_contents_do_not_matter():
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(27)
    cache, table, lens, vals = _filled(rng, [3000, 20], 1, 64, 64)
    Q = _bf16(rng, 2, 4, 1, 64)
    need = esd.attn_fwd_decode_cache_workspace_bytes(cache, 2, 4, 1, table.shape[1])
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    a = _attend_and_check(Q, cache, table, lens, vals, workspace=ws)
    b = _attend_and_check(Q, cache, table, lens, vals, workspace=ws.fill_(0))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_offsets_past_32_bits():
    """A pool above 2^32 bytes, the sequence in its last pages."""
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(28)
    Hkv, d = 8, 128
    block = esd.attn_cache_page_bytes(Hkv, d, d)
    pages = (1 << 32) // block + 40
    cache = esd.QuantCache.empty(pages, Hkv, d, d)
    n = 100
    t = np.arange(n)
    table = np.array([[pages - 1, pages - 3, pages - 2, 0]], dtype=np.int32)
    slots = table[0, t // PAGE].astype(np.int64) * PAGE + t % PAGE
    K, V = _bf16(rng, n, Hkv, d), _bf16(rng, n, Hkv, d)
    esd.attn_cache_append(cache, K.cuda(), V.cuda(), torch.from_numpy(slots).cuda())
    vals = [ref.values(*ref.quantize(f64(x))) for x in (K, V)]
    Kr, _ = esd.attn_cache_read(cache, torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    assert np.array_equal(f64(Kr), ref.bf16(vals[0]))
    _attend_and_check(_bf16(rng, 1, 16, 1, d), cache, torch.from_numpy(table).cuda(),
                      torch.tensor([n], dtype=torch.int32, device="cuda"), [vals])


def test_agrees_with_the_decode_forward_over_what_was_read_back():
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(29)
    Hq, Hkv, d, n = 8, 2, 128, 640
    cache, table, lens, _ = _filled(rng, [n], Hkv, d, d)
    Q = _bf16(rng, 1, Hq, 4, d).cuda()
    O, LSE = esd.attn_fwd_decode_cache(Q, cache, table, lens)
    t = torch.arange(n, device="cuda")
    K, V = esd.attn_cache_read(cache, table[0, t // PAGE].long() * PAGE + t % PAGE)
    to = lambda x: x.transpose(0, 1)[None].contiguous()  # noqa: E731
    O2, LSE2, _ = esd.attn_fwd_decode(Q, to(K), to(V), causal=True)
    torch.cuda.synchronize()
    # K and V rounded to bf16 on one side: 2^-8 of the values, and of the scores (below 8 here)
    np.testing.assert_allclose(f64(LSE), f64(LSE2), atol=8 * ref.BF16, rtol=0)
    np.testing.assert_allclose(f64(O), f64(O2), atol=2e-2, rtol=4 * ref.BF16)


def test_serving_steps_captured_and_replayed():
    """norm + rotation -> append -> attention, one token of each sequence per
    step, captured once and replayed while the sequences grow, against the
    same steps run eagerly (bit for bit) and the 64-bit form (last step)."""
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(30)
    B, Hq, Hkv, d, steps = 3, 8, 2, 128, 40
    start = [30, 0, 63]
    wide = 4
    cache, _, _, _ = _filled(rng, [PAGE * wide] * B, Hkv, d, d)
    table = torch.from_numpy(rng.permutation(B * wide).astype(np.int32).reshape(B, wide)).cuda()
    x = _bf16(rng, steps, B, Hq + 2 * Hkv, d).cuda()
    gq, gk = (_bf16(rng, d).cuda() for _ in range(2))
    now = torch.zeros((B, Hq + 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor(start, dtype=torch.int32, device="cuda")

    def step():
        pos = lens.clone()                       # the new token's position
        lens.add_(1)
        slots = table.gather(1, (pos // PAGE).long()[:, None])[:, 0].long() * PAGE + pos % PAGE
        Yq, Yk = esd.attn_qk_norm_rope(now[:, :Hq], now[:, Hq:Hq + Hkv], gq, gk, esd.RotaryAxes(pos))
        esd.attn_cache_append(cache, Yk, now[:, Hq + Hkv:], slots)
        return esd.attn_fwd_decode_cache(Yq[:, :, None], cache, table, lens)

    pool0 = cache.pool.clone()
    eager = []
    for i in range(steps):
        now.copy_(x[i])
        eager.append([t.clone() for t in step()])
    pool1 = cache.pool.clone()
    cache.pool.copy_(pool0)
    lens.copy_(torch.tensor(start, dtype=torch.int32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(steps):
        now.copy_(x[i])
        graph.replay()
        assert torch.equal(out[0], eager[i][0]) and torch.equal(out[1], eager[i][1]), i
    assert torch.equal(cache.pool, pool1)
    # the last step in 64 bits, over what the cache holds
    pool = cache.pool.cpu().numpy()
    Yq, _ = esd.attn_qk_norm_rope(now[:, :Hq], now[:, Hq:Hq + Hkv], gq, gk, esd.RotaryAxes(lens - 1))
    vals = []
    for b in range(B):
        t = np.arange(int(lens[b]))
        vals.append(ref.load(pool, table[b].cpu().numpy()[t // PAGE].astype(np.int64) * PAGE + t % PAGE, d, d))
    _attend_and_check(Yq[:, :, None].cpu(), cache, table, lens, vals)


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, give what they give alone."""
    import exact_scaled_dot_gb300 as esd
    rng = np.random.default_rng(31)
    made = [_filled(rng, [5000, 100], 2, 128, 128) for _ in range(2)]
    Q = [_bf16(rng, 2, 8, 1, 128).cuda() for _ in range(2)]
    want = [esd.attn_fwd_decode_cache(q, m[0], m[1], m[2]) for q, m in zip(Q, made)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[esd.attn_fwd_decode_cache(q, m[0], m[1], m[2], stream=s) for q, m, s in zip(Q, made, streams)]
           for _ in range(20)]
    torch.cuda.synchronize()
    for g in got:
        for (o, l), (o2, l2) in zip(g, want):
            assert torch.equal(o, o2) and torch.equal(l, l2)
