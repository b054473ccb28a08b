"""Host-side tests of the calls that serve from the 4-bit cache (shared prefix,
attention weights, eviction): refusals before any CUDA call, sizes, and the
64-bit forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import exact_scaled_dot_gb300 as esd
from exact_scaled_dot_gb300 import _binding as bnd
from exact_scaled_dot_gb300.build import build

import _qk_cache_ref as ref
import _serving_ref as srv

P = ctypes.c_void_p(256)
F = ctypes.c_float
S, N, A, U = bnd.ATTN_ERR_SHAPE, bnd.ATTN_ERR_NULL, bnd.ATTN_ERR_ALIGN, bnd.ATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build()
    return esd.load()


def _cache(Hkv=2, dh=128, dv=128, pages=8, pool=256):
    return ctypes.byref(bnd.AttnCache(Hkv, dh, dv, pages, pool))


def test_prefix_refuses(lib):
    def call(c=_cache(), B=2, Hq=8, nq=1, pre=4, pages=4, scale=0.1, q=P, pt=P, pl=P, table=P, lengths=P, o=P, lse=P,
             ws=P, n=1 << 40):
        return lib.attn_fwd_prefix_cache(c, B, Hq, nq, pre, pages, F(scale), q, pt, pl, table, lengths, o, lse, ws,
                                         ctypes.c_size_t(n), None)

    assert call(c=None) == N
    for kw in (dict(B=0), dict(Hq=0), dict(Hq=7), dict(nq=0), dict(pre=0), dict(pre=1 << 26), dict(pages=0),
               dict(pages=1 << 26), dict(B=1 << 30), dict(c=_cache(pages=0)), dict(c=_cache(Hkv=0))):
        assert call(**kw) == S, kw
    assert call(nq=17) == U and call(c=_cache(dh=64, dv=128)) == U
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == bnd.ATTN_ERR_SCALE
    for kw in (dict(q=None), dict(pt=None), dict(pl=None), dict(table=None), dict(lengths=None), dict(o=None),
               dict(lse=None), dict(c=_cache(pool=None))):
        assert call(**kw) == N, kw
    for kw in (dict(q=ctypes.c_void_p(264)), dict(pt=ctypes.c_void_p(258)), dict(pl=ctypes.c_void_p(257)),
               dict(table=ctypes.c_void_p(258)), dict(lengths=ctypes.c_void_p(258))):
        assert call(**kw) == A, kw
    for B, nq, pre, pages in ((1, 1, 1, 1), (2, 1, 4, 4), (64, 1, 1024, 64), (300, 16, 1000, 2000)):
        need = lib.attn_fwd_prefix_cache_workspace_bytes(_cache(), B, 8, nq, pre, pages)
        assert need > 0 and need % 256 == 0
        for kw in (dict(ws=None), dict(n=need - 1), dict(ws=ctypes.c_void_p(512 + 16))):
            assert call(B=B, nq=nq, pre=pre, pages=pages, **kw) == bnd.ATTN_ERR_WORKSPACE
    assert lib.attn_fwd_prefix_cache_workspace_bytes(_cache(), 2, 8, 17, 4, 4) == 0
    assert lib.attn_fwd_prefix_cache_workspace_bytes(_cache(), 2, 8, 1, 0, 4) == 0


def test_weigh_refuses(lib):
    def call(c=_cache(), B=2, Hq=8, nq=1, pages=4, scale=0.1, q=P, table=P, lengths=P, lse=P, w=P):
        return lib.attn_cache_weigh(c, B, Hq, nq, pages, F(scale), q, table, lengths, lse, w, None)

    for kw in (dict(B=0), dict(Hq=0), dict(Hq=7), dict(nq=0), dict(pages=0), dict(pages=1 << 26), dict(B=1 << 30)):
        assert call(**kw) == S, kw
    assert call(nq=17) == U and call(c=_cache(dh=96)) == U
    for scale in (0.0, float("nan")):
        assert call(scale=scale) == bnd.ATTN_ERR_SCALE
    for kw in (dict(c=None), dict(q=None), dict(table=None), dict(lengths=None), dict(lse=None), dict(w=None)):
        assert call(**kw) == N, kw
    for kw in (dict(q=ctypes.c_void_p(264)), dict(w=ctypes.c_void_p(258)), dict(lse=ctypes.c_void_p(258))):
        assert call(**kw) == A, kw


def test_evict_refuses(lib):
    def call(c=_cache(), B=2, pages=4, keep=64, first=4, recent=8, table=P, lengths=P, w=P, nl=ctypes.c_void_p(512), nw=P,
             kept=P, ws=P, n=1 << 40):
        return lib.attn_cache_evict(c, B, pages, keep, first, recent, table, lengths, w, nl, nw, kept, ws,
                                    ctypes.c_size_t(n), None)

    for kw in (dict(B=0), dict(pages=0), dict(pages=(1 << 25) + 1), dict(keep=0), dict(keep=-1), dict(first=-1),
               dict(recent=-1), dict(first=60, recent=5), dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), dict(nl=P),
               dict(B=2 ** 31 - 1)):
        assert call(**kw) == S, kw
    assert call(c=_cache(dh=96)) == U
    for kw in (dict(c=None), dict(table=None), dict(lengths=None), dict(w=None), dict(nl=None), dict(nw=None)):
        assert call(**kw) == N, kw
    for kw in (dict(table=ctypes.c_void_p(258)), dict(w=ctypes.c_void_p(258)), dict(kept=ctypes.c_void_p(258))):
        assert call(**kw) == A, kw
    # few tokens that may move need no workspace, many do
    assert lib.attn_cache_evict_workspace_bytes(_cache(), 2, 4, 64, 4, 8) == 0
    need = lib.attn_cache_evict_workspace_bytes(_cache(), 2, 400, 4096, 4, 8)
    assert need > 0 and need % 256 == 0
    for kw in (dict(ws=None), dict(n=need - 1), dict(ws=ctypes.c_void_p(512 + 16))):
        assert call(pages=400, keep=4096, **kw) == bnd.ATTN_ERR_WORKSPACE
    assert lib.attn_cache_evict_workspace_bytes(_cache(), 2, 4, 0, 0, 0) == 0


def test_binding_refuses():
    """Types, shapes and devices are checked before the library is called."""
    pool = torch.zeros((4, 2, 32 * 128 * 9 // 16), dtype=torch.uint8)
    bad = torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        esd.QuantCache(pool, 64, 64)                                             # not on a GPU

    class Fake:                                                                  # the sizes of a cache, on the CPU
        device, Hkv, d_h, d_v, pages = torch.device("cpu"), 2, 64, 64, 4
    t, n = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        esd.attn_cache_weigh(bad[0], Fake, t, n, None, None)
    with pytest.raises(ValueError):
        esd.attn_fwd_prefix_cache(bad, Fake, n, n, t[0], n)
    with pytest.raises(ValueError):
        esd.attn_cache_evict(Fake, n, n, n, 4)


def test_reference_eviction_keeps_what_it_says():
    rng = np.random.default_rng(1)
    for _ in range(200):
        n, keep = int(rng.integers(0, 60)), int(rng.integers(1, 40))
        first = int(rng.integers(0, keep + 1))
        recent = int(rng.integers(0, keep - first + 1))
        w = rng.integers(0, 6, 64).astype(np.float32)
        src, new = srv.evict(w, n, keep, first, recent)
        m = min(n, keep)
        assert (src[m:] == -1).all() and (new[m:] == 0).all() and np.array_equal(new[:m], w[src[:m]])
        stay = sorted(src[:m])
        assert len(set(stay)) == m
        if n <= keep:
            assert stay == list(range(n))
            continue
        assert stay[:first] == list(range(first)) and list(src[keep - recent:]) == list(range(n - recent, n))
        out = sorted(set(range(n)) - set(stay))
        chosen = [j for j in stay if first <= j < n - recent]
        # nothing left out weighs more than what stays, and of equals the lowest places stay
        assert all((w[j], -j) < (w[i], -i) for j in out for i in chosen)
        for p in range(keep - recent):
            assert src[p] == p or (p in out and src[p] >= keep - recent)


def test_reference_prefix_is_one_softmax():
    """Prefix and own keys as one row of keys."""
    rng = np.random.default_rng(2)
    q = rng.normal(size=(4, 2, 64))
    Kp, Vp, K, V = (rng.normal(size=(n, 2, 64)) for n in (7, 7, 5, 5))
    O, L, _, _ = srv.attend_prefix(q, Kp, Vp, K, V, 5, 0.125)
    O2, L2, _, _ = ref.attend(q, np.concatenate([Kp, K]), np.concatenate([Vp, V]), 12, 0.125)
    assert np.allclose(O, O2, atol=1e-14) and np.allclose(L, L2, atol=1e-14)
    # a row that comes before its sequence's own tokens sees the prefix alone
    O3, L3, _, _ = srv.attend_prefix(q, Kp, Vp, K, V, 1, 0.125)
    O4, _, _, _ = ref.attend(q[:, :1], Kp, Vp, 7, 0.125)
    assert np.allclose(O3[:, :1], O4, atol=1e-14)


def test_reference_weights_sum_to_one():
    rng = np.random.default_rng(3)
    q, K = rng.normal(size=(4, 2, 64)), rng.normal(size=(9, 2, 64))
    _, L, _, _ = ref.attend(q, K, K, 9, 0.125)
    w, _ = srv.weigh(q, K, L, 9, np.zeros((2, 32)), 0.125)
    assert np.allclose(w.sum(-1), 4.0) and (w[:, 9:] == 0).all()


@pytest.mark.parametrize("first,recent,keep", [(0, 0, (1 << 30) + 1), (0, 0, 0), ((1 << 32) + 1, 0, 16), (0, -1, 16),
                                               (9, 8, 16), (0, 0, (1 << 32) + 16)])
def test_eviction_sizes_are_checked_before_they_are_32_bits(lib, first, recent, keep):
    class Fake:
        device, Hkv, d_h, d_v, pages = torch.device("cpu"), 2, 64, 64, 4

        @staticmethod
        def arg():
            return _cache()
    t, n = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(esd.AttnError):
        esd.attn_cache_evict(Fake, t, n, torch.zeros((2, 2, 96)), keep, first=first, recent=recent)
    assert esd.attn_cache_evict_workspace_bytes(Fake, 2, 1 << 20, keep, first=first, recent=recent) == 0
    if keep < 1 << 31 and first < 1 << 31:
        assert lib.attn_cache_evict_workspace_bytes(_cache(), 2, 1 << 20, keep, first, recent) == 0


def test_eviction_refuses_outputs_over_its_inputs(lib):
    """An output that shares a byte with an input or with another output, but for the weights in place.
    (Every call here is refused: none reaches a device.)"""
    B, Hkv, pages, keep = 3, 2, 4, 64
    size = dict(table=4 * B * pages, lengths=4 * B, weights=4 * B * Hkv * 32 * pages, new_lengths=4 * B,
                new_weights=4 * B * Hkv * 32 * pages, kept=4 * B * Hkv * keep)
    at, free = {}, 4096
    for name, n in size.items():
        at[name], free = free, free + n                    # one right behind the other

    def call(**moved):
        a = {**at, **moved}
        return lib.attn_cache_evict(_cache(Hkv), B, pages, keep, 4, 8, *(ctypes.c_void_p(a[k]) for k in (
            "table", "lengths", "weights", "new_lengths", "new_weights", "kept")), None, ctypes.c_size_t(0), None)

    outputs = ("new_lengths", "new_weights", "kept")
    for out in outputs:
        for other in size:
            if other == out:
                continue
            for to in (at[other] + 4, at[other] + size[other] - 4, at[other] - size[out] + 4):
                assert call(**{out: to}) == S, (out, other, to)
            if (out, other) != ("new_weights", "weights"):
                assert call(**{out: at[other]}) == S, (out, other)
    # in place, the others are checked as well
    assert call(new_weights=at["weights"], kept=at["weights"]) == S
    assert call(new_weights=at["weights"], new_lengths=at["lengths"] + 4) == S
