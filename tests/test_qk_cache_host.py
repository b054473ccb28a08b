"""Host-side tests of the query/key norm, the rotation over several axes and
the 4-bit cache: refusals (before any CUDA call), sizes, and the 64-bit
reference forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import exact_scaled_dot_gb300 as esd
from exact_scaled_dot_gb300 import _binding as bnd
from exact_scaled_dot_gb300.build import build

import _qk_cache_ref as ref

P = ctypes.c_void_p(256)
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    build()
    return esd.load()


def _axes(sections=(32,), base=10000.0, restart=0, pos=256, axes=None):
    s = (ctypes.c_int32 * 3)(*sections)
    return ctypes.byref(bnd.AttnRotaryAxes(base, len(sections) if axes is None else axes, s, restart, pos))


OK = dict(tokens=10, hq=4, hk=2, d=64, rot=_axes(), inv=0, st=None, xq=P, xk=P, yq=P, yk=P, eps=1e-6, gq=P, gk=P)


def _rope(lib, **kw):
    a = dict(OK, **kw)
    return lib.attn_rope_axes(a["tokens"], a["hq"], a["hk"], a["d"], a["rot"], a["inv"], a["st"], a["xq"], a["xk"],
                              a["yq"], a["yk"], None)


def _norm(lib, **kw):
    a = dict(OK, **kw)
    return lib.attn_qk_norm_rope(a["tokens"], a["hq"], a["hk"], a["d"], F(a["eps"]), a["rot"], a["st"], a["xq"],
                                 a["xk"], a["gq"], a["gk"], a["yq"], a["yk"], None)


def _bwd(lib, ws=P, ws_bytes=1 << 30, dgq=P, dgk=P, dyq=P, dyk=P, **kw):
    a = dict(OK, **kw)
    return lib.attn_qk_norm_rope_bwd(a["tokens"], a["hq"], a["hk"], a["d"], F(a["eps"]), a["rot"], a["st"], a["xq"],
                                     a["xk"], a["gq"], a["gk"], dyq, dyk, a["yq"], a["yk"], dgq, dgk, ws,
                                     ctypes.c_size_t(ws_bytes), None)


@pytest.mark.parametrize("call", [_rope, _norm, _bwd])
def test_row_calls_refuse(lib, call):
    S, N, A, C = bnd.ATTN_ERR_SHAPE, bnd.ATTN_ERR_NULL, bnd.ATTN_ERR_ALIGN, bnd.ATTN_ERR_SCALE
    for kw in (dict(tokens=0), dict(tokens=1 << 31), dict(hq=0), dict(hk=-1), dict(hq=65536), dict(d=60), dict(d=136),
               dict(d=0)):
        assert call(lib, **kw) == S, kw
    # key tensors without key heads, key heads without tensors
    assert call(lib, hk=0) == S
    assert call(lib, xk=None) == N
    assert call(lib, xq=None) == N
    assert call(lib, yq=None) == N
    assert call(lib, xq=ctypes.c_void_p(0x1008)) == A
    # rotations
    for kw in (dict(sections=(33,)), dict(sections=(16, 17)), dict(sections=(16, 0)), dict(sections=(16, -1)),
               dict(axes=0), dict(axes=4), dict(restart=2), dict(sections=(2 ** 31 - 1, 2 ** 31 - 1, 4))):
        assert call(lib, rot=_axes(**kw)) == S, kw
    assert call(lib, rot=_axes(base=1.0)) == C
    assert call(lib, rot=_axes(base=float("nan"))) == C
    assert call(lib, rot=_axes(pos=None)) == N
    assert call(lib, rot=_axes(pos=258)) == A
    # strides: multiples of 8, at least a row
    st = bnd.AttnQkStrides()
    st.q = bnd.AttnTensorStrides(4 * 64 + 4, 64)
    assert call(lib, st=ctypes.byref(st)) == A
    st.q = bnd.AttnTensorStrides(256, 56)
    assert call(lib, st=ctypes.byref(st)) == S


def test_norm_calls_refuse(lib):
    for call in (_norm, _bwd):
        for eps in (0.0, -1e-6, float("nan"), float("inf")):
            assert call(lib, eps=eps) == bnd.ATTN_ERR_SCALE
        assert call(lib, gq=ctypes.c_void_p(0x1008)) == bnd.ATTN_ERR_ALIGN
    assert _rope(lib, rot=None) == bnd.ATTN_ERR_NULL
    assert _rope(lib, inv=2) == bnd.ATTN_ERR_SHAPE
    need = lib.attn_qk_norm_rope_bwd_workspace_bytes(10, 4, 2, 64)
    assert need > 0 and need % 256 == 0
    assert _bwd(lib, ws=None) == bnd.ATTN_ERR_WORKSPACE
    assert _bwd(lib, ws_bytes=need - 1) == bnd.ATTN_ERR_WORKSPACE
    assert _bwd(lib, ws=ctypes.c_void_p(512 + 16)) == bnd.ATTN_ERR_WORKSPACE
    # a weight gradient needs its weight
    assert _bwd(lib, gq=None) == bnd.ATTN_ERR_NULL
    assert _bwd(lib, gk=None) == bnd.ATTN_ERR_NULL
    assert _bwd(lib, hk=0, xk=None, yk=None, dyk=None, gk=None) == bnd.ATTN_ERR_NULL
    assert _bwd(lib, dyq=None) == bnd.ATTN_ERR_NULL
    assert lib.attn_qk_norm_rope_bwd_workspace_bytes(0, 4, 2, 64) == 0
    assert lib.attn_qk_norm_rope_bwd_workspace_bytes(10 ** 9, 3000, 1000, 128) <= 400_000


def _cache(Hkv=2, dh=128, dv=128, pages=8, pool=256):
    return ctypes.byref(bnd.AttnCache(Hkv, dh, dv, pages, pool))


def test_cache_calls_refuse(lib):
    S, N, A = bnd.ATTN_ERR_SHAPE, bnd.ATTN_ERR_NULL, bnd.ATTN_ERR_ALIGN
    for fn in (lib.attn_cache_append, lib.attn_cache_read):
        call = lambda c=_cache(), n=4, st=None, slots=P, K=P, V=P: fn(c, n, st, slots, K, V, None)  # noqa: E731,B023
        assert call(c=None) == N
        assert call(c=_cache(Hkv=0)) == S
        assert call(c=_cache(pages=0)) == S
        assert call(c=_cache(pages=1 << 31)) == S
        assert call(c=_cache(dh=96, dv=96)) == bnd.ATTN_ERR_UNSUPPORTED
        assert call(c=_cache(pool=None)) == N
        assert call(c=_cache(pool=0x1008)) == A
        assert call(n=0) == S
        assert call(slots=None) == N
        assert call(slots=ctypes.c_void_p(260)) == A
        assert call(K=None) == N
        assert call(V=ctypes.c_void_p(0x1008)) == A
        st = bnd.AttnStrides()
        st.k = bnd.AttnTensorStrides(260, 128)
        assert call(st=ctypes.byref(st)) == A


def test_cache_attention_refuses(lib):
    def call(c=_cache(), B=2, Hq=8, nq=1, pages=4, scale=0.1, q=P, table=P, lengths=P, o=P, lse=P, ws=P, n=1 << 40):
        return lib.attn_fwd_decode_cache(c, B, Hq, nq, pages, F(scale), q, table, lengths, o, lse, ws,
                                         ctypes.c_size_t(n), None)

    S, N, A = bnd.ATTN_ERR_SHAPE, bnd.ATTN_ERR_NULL, bnd.ATTN_ERR_ALIGN
    for kw in (dict(B=0), dict(Hq=0), dict(Hq=7), dict(nq=0), dict(pages=0), dict(pages=1 << 26), dict(B=1 << 30)):
        assert call(**kw) == S, kw
    assert call(nq=17) == bnd.ATTN_ERR_UNSUPPORTED
    assert call(c=_cache(dh=64, dv=128)) == bnd.ATTN_ERR_UNSUPPORTED
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == bnd.ATTN_ERR_SCALE
    for kw in (dict(q=None), dict(table=None), dict(lengths=None), dict(o=None), dict(lse=None)):
        assert call(**kw) == N, kw
    assert call(q=ctypes.c_void_p(0x1008)) == A
    assert call(table=ctypes.c_void_p(258)) == A
    # a long table is split: its workspace is checked
    need = lib.attn_fwd_decode_cache_workspace_bytes(_cache(), 2, 8, 1, 1000)
    assert need > 0 and need % 256 == 0
    assert call(pages=1000, ws=None) == bnd.ATTN_ERR_WORKSPACE
    assert call(pages=1000, n=need - 1) == bnd.ATTN_ERR_WORKSPACE
    assert call(pages=1000, ws=ctypes.c_void_p(512 + 16)) == bnd.ATTN_ERR_WORKSPACE
    assert lib.attn_fwd_decode_cache_workspace_bytes(_cache(), 2, 8, 17, 1000) == 0
    # four pages in all are one CTA's: no workspace
    assert lib.attn_fwd_decode_cache_workspace_bytes(_cache(), 1, 8, 1, 4) == 0


def test_page_bytes(lib):
    for Hkv, dh, dv in ((1, 64, 64), (8, 128, 128), (3, 128, 64)):
        assert esd.attn_cache_page_bytes(Hkv, dh, dv) == Hkv * 32 * (dh + dv) * 9 // 16
    assert esd.attn_cache_page_bytes(0, 64, 64) == 0
    assert esd.attn_cache_page_bytes(1, 64, 128) == 0


def test_binding_refuses():
    """The binding checks types, shapes and devices before it calls the library."""
    cpu = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    pos = torch.zeros((4,), dtype=torch.int32)
    with pytest.raises(ValueError):
        esd.attn_rope_axes(cpu, None, esd.RotaryAxes(pos))                       # not on a GPU
    with pytest.raises(ValueError):
        esd.attn_qk_norm_rope(cpu[0], None)                                      # not 3-D
    with pytest.raises(ValueError):
        esd.RotaryAxes(pos, sections=(1, 1, 1, 1)).arg(4, 64, None)
    with pytest.raises(TypeError):
        esd.attn_qk_norm_rope(cpu.float(), None)
    with pytest.raises(ValueError):
        esd.QuantCache(torch.zeros((4, 2, 100), dtype=torch.uint8), 64, 64)
    # a count of blocks that would wrap in the library's 32 bits
    with pytest.raises(ValueError):
        esd._binding._axes_bytes(10000.0, (2 ** 32 + 8,), False)


def test_one_row_expanded_is_refused():
    """Strides {0, 0} mean contiguous to the library: a row that stands for all of them must not reach it."""
    one = torch.zeros((64,), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        esd._binding._stride_arg(esd._binding.AttnQkStrides, ("q",), one.expand(4, 2, 64))
    with pytest.raises(ValueError):
        esd._binding._strides_arg(True, q=one.expand(4, 2, 64))
    with pytest.raises(ValueError):
        esd._binding._strides_arg(False, q=one.expand(3, 4, 2, 64))
    # one zero alone is the library's to refuse; size-1 dimensions are free
    assert esd._binding._packed_strides(one.expand(1, 1, 64)) == (64, 64)


def test_reference_gradient_against_differences():
    """The gradient formula against central differences of the forward, fp64."""
    rng = np.random.default_rng(3)
    T, H, d, eps = 3, 2, 16, 1e-3
    x, g, dy = rng.normal(size=(T, H, d)), rng.normal(size=d), rng.normal(size=(T, H, d))
    a = ref.angles(rng.integers(0, 50, (2, T)), (3, 4), d, 100.0, True)
    f = lambda x, g: float((ref.norm_rope(x, g, a, eps)[0] * dy).sum())  # noqa: E731
    dx, dg, _, _ = ref.norm_rope_bwd(x, g, dy, a, eps)
    h = 1e-6
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, g) - f(x - e, g)) / (2 * h) - dx[at]) < 1e-6
    for k in range(d):
        e = np.zeros_like(g)
        e[k] = h
        assert abs((f(x, g + e) - f(x, g - e)) / (2 * h) - dg[k]) < 1e-6


def test_reference_quantisation():
    """Every element within one step of its value, 0 exact, and the bytes hold what was stored."""
    rng = np.random.default_rng(5)
    x = ref.bf16(rng.normal(size=(40, 2, 128)) * np.exp(2 * rng.normal(size=(40, 2, 1))) + rng.normal(size=(40, 2, 1)))
    x[3] = 0.0
    x[4, :, 64:] = np.abs(x[4, :, 64:])
    c, s, z = ref.quantize(x)
    v = ref.values(c, s, z)
    step = np.repeat(s, 64, -1)
    assert (np.abs(v - x) <= step * (1 + 2.0 ** -7)).all()
    assert (v[3] == 0).all() and (v[x == 0] == 0).all()
    pool = np.full((3, 2, 32 * 256 * 9 // 16), 0xAB, dtype=np.uint8)
    slots = rng.permutation(96)[:40]
    ref.store(pool, slots, x, -x)
    K, V = ref.load(pool, slots, 128, 128)
    assert (K == v).all() and (V == ref.values(*ref.quantize(-x))).all()
