"""GPU tests of the attention weights added up per cached token, against a 64-bit form
(bounds: _serving_ref.weigh)."""
import numpy as np
import pytest
import torch

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


def _case(seed, B, Hq, Hkv, nq, dh, dv, lengths, max_pages=None):
    rng = np.random.default_rng(seed)
    c = srv.Paged(rng, Hkv, dh, dv, lengths, max_pages=max_pages)
    q = bf16(rng.normal(size=(B, Hq, nq, dh)))
    w = np.abs(rng.normal(size=(B, Hkv, c.max_pages * PAGE))).astype(np.float32)
    lse = np.full((B, Hq, nq), -np.inf, np.float32)
    for b, n in enumerate(c.lengths):
        for r in range(Hq):
            for i in range(nq):
                m = n - nq + 1 + i
                if m > 0:
                    s = c.K[b][:m, r // (Hq // Hkv)] @ q[b, r, i] * dh ** -0.5
                    lse[b, r, i] = s.max() + np.log(np.exp(s - s.max()).sum())
    return c, q, w, lse


def _check(c, q, w, lse, got, dh):
    for b, n in enumerate(c.lengths):
        want, err = srv.weigh(q[b], c.K[b], lse[b].astype(np.float64), n, w[b], dh ** -0.5)
        assert_within(got[b], want, err, "weights")
        assert np.array_equal(got[b][:, n:], w[b][:, n:])      # places without a token are left alone


@pytest.mark.parametrize("dh,dv", [(64, 64), (128, 128), (128, 64)])
@pytest.mark.parametrize("B,Hq,Hkv,nq,lengths", [
    (1, 1, 1, 1, [1]),
    (2, 4, 2, 1, [0, 32]),
    (3, 5, 1, 2, [33, 1, 31]),                  # (a row before the first token)
    (2, 6, 3, 5, [64, 200]),
    (4, 8, 8, 16, [16, 3, 65, 100]),
    (2, 32, 1, 16, [17, 40]),                   # 512 rows of a head: two passes over the pages
    (40, 4, 1, 1, [1 + 5 * i for i in range(40)]),
])
def test_against_64_bits(B, Hq, Hkv, nq, lengths, dh, dv):
    import exact_scaled_dot_gb300 as esd
    c, q, w, lse = _case(B * 10 + nq, B, Hq, Hkv, nq, dh, dv, lengths)
    W = _dev(w)
    got = esd.attn_cache_weigh(_dev(q).to(torch.bfloat16), esd.QuantCache(_dev(c.pool), dh, dv), _dev(c.table),
                               _dev(np.array(c.lengths, np.int32)), _dev(lse), W)
    torch.cuda.synchronize()
    assert got.data_ptr() == W.data_ptr()
    _check(c, q, w, lse, f64(W), dh)


def test_long_and_ragged():
    import exact_scaled_dot_gb300 as esd
    c, q, w, lse = _case(3, 4, 8, 2, 1, 128, 128, [3000, 1, 0, 777], max_pages=120)
    W = _dev(w)
    esd.attn_cache_weigh(_dev(q).to(torch.bfloat16), esd.QuantCache(_dev(c.pool), 128, 128), _dev(c.table),
                         _dev(np.array(c.lengths, np.int32)), _dev(lse), W)
    torch.cuda.synchronize()
    _check(c, q, w, lse, f64(W), 128)
    # every row's weights sum to 1
    assert np.allclose((f64(W) - w).sum(-1)[[0, 1, 3]], 4.0, atol=1e-3)


def test_rows_that_add_nothing_or_nan():
    import exact_scaled_dot_gb300 as esd
    dh = 64
    c, q, w, lse = _case(7, 2, 4, 2, 2, dh, dh, [40, 1])
    lse[0, 0] = -np.inf                     # as a row that saw no key
    lse[0, 1, 1] = np.inf                   # every weight 0
    q[1, 2, 1, 3] = np.nan                  # sees key 0 of sequence 1
    q[1, 0, 0, 0] = np.inf                  # sees nothing
    W = _dev(w)
    esd.attn_cache_weigh(_dev(q).to(torch.bfloat16), esd.QuantCache(_dev(c.pool), dh, dh), _dev(c.table),
                         _dev(np.array(c.lengths, np.int32)), _dev(lse), W)
    torch.cuda.synchronize()
    got = f64(W)
    assert np.isnan(got[1, 1, 0])
    got[1, 1, 0] = 0
    assert not np.isnan(got).any()
    want, err = srv.weigh(np.nan_to_num(q[0]), c.K[0], np.where(lse[0] == np.inf, 1e9, lse[0]), 40, w[0], dh ** -0.5)
    assert_within(got[0], want, err, "weights")


def test_bad_pages_and_lengths_are_left_out_and_reported():
    import exact_scaled_dot_gb300 as esd
    dh = 128
    c, q, w, lse = _case(17, 2, 4, 1, 1, dh, dh, [100, 96], max_pages=4)
    table = c.table.copy()
    table[0, 1], table[1, 2] = -1, len(c.pool)
    W = _dev(w)
    esd.attn_cache_weigh(_dev(q).to(torch.bfloat16), esd.QuantCache(_dev(c.pool), dh, dh), _dev(table),
                         _dev(np.array([100, 96], np.int32)), _dev(lse), W)
    torch.cuda.synchronize()
    assert esd.attn_get_status() == esd.ATTN_ERR_PAGE
    esd.attn_clear_status()
    got = f64(W)
    for b, page in ((0, 1), (1, 2)):
        want, err = srv.weigh(q[b], c.K[b], lse[b].astype(np.float64), c.lengths[b], w[b], dh ** -0.5)
        want[:, page * PAGE:(page + 1) * PAGE] = w[b][:, page * PAGE:(page + 1) * PAGE]
        assert_within(got[b], want, err, "weights")
    W = _dev(w)
    esd.attn_cache_weigh(_dev(q).to(torch.bfloat16), esd.QuantCache(_dev(c.pool), dh, dh), _dev(c.table[:, :3]),
                         _dev(np.array([1 << 30, -4], np.int32)), _dev(lse), _dev(w[:, :, :96]))
    torch.cuda.synchronize()
    assert esd.attn_get_status() == esd.ATTN_ERR_PAGE
    esd.attn_clear_status()


def test_captured_and_repeated():
    """Adds again at every replay, the same each time."""
    import exact_scaled_dot_gb300 as esd
    dh = 128
    c, q, w, lse = _case(27, 5, 8, 2, 2, dh, 64, [300, 2, 64, 31, 150])
    args = (_dev(q).to(torch.bfloat16), esd.QuantCache(_dev(c.pool), dh, 64), _dev(c.table),
            _dev(np.array(c.lengths, np.int32)), _dev(lse))
    W = torch.zeros(w.shape, device="cuda")
    esd.attn_cache_weigh(*args, W)
    one = W.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        esd.attn_cache_weigh(*args, W)
    W.zero_()
    graph.replay()
    assert torch.equal(W, one)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(W, one + one)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    two = torch.zeros_like(W)
    side.wait_stream(torch.cuda.current_stream())
    esd.attn_cache_weigh(*args, two, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(two, one)


def test_lengths_past_the_table_and_below_zero():
    """A length past the table is cut to it; a sequence of negative length is left alone."""
    import exact_scaled_dot_gb300 as esd
    dh = 128
    c, q, w, lse = _case(19, 2, 4, 1, 1, dh, dh, [96, 64], max_pages=3)
    W = _dev(w)
    esd.attn_cache_weigh(_dev(q).to(torch.bfloat16), esd.QuantCache(_dev(c.pool), dh, dh), _dev(c.table),
                         _dev(np.array([1 << 30, -4], np.int32)), _dev(lse), W)
    torch.cuda.synchronize()
    assert esd.attn_get_status() == esd.ATTN_ERR_PAGE
    esd.attn_clear_status()
    want, err = srv.weigh(q[0], c.K[0], lse[0].astype(np.float64), 96, w[0], dh ** -0.5)
    assert_within(f64(W)[0], want, err, "weights")
    assert np.array_equal(W.cpu().numpy()[1], w[1])


@pytest.mark.parametrize("nq", [1, 3])
def test_rows_without_a_log_sum_exp_add_nothing_whatever_they_hold(nq):
    """LSE = -inf beside an infinity or a NaN in the row of Q, at keys that the row sees."""
    import exact_scaled_dot_gb300 as esd
    dh = 64
    c, q, w, lse = _case(23 + nq, 2, 4, 2, nq, dh, dh, [70, 33])
    lse[0, 1, nq - 1] = lse[1, 2] = -np.inf
    want = [srv.weigh(q[b], c.K[b], lse[b].astype(np.float64), c.lengths[b], w[b], dh ** -0.5) for b in range(2)]
    q[0, 1, nq - 1, 7] = np.nan
    q[1, 2, :, 3] = np.inf
    W = _dev(w)
    esd.attn_cache_weigh(_dev(q).to(torch.bfloat16), esd.QuantCache(_dev(c.pool), dh, dh), _dev(c.table),
                         _dev(np.array(c.lengths, np.int32)), _dev(lse), W)
    torch.cuda.synchronize()
    for b in range(2):
        assert_within(f64(W)[b], *want[b], "weights")
