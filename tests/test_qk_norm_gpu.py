"""GPU tests of the query/key RMS norm with rotation, its gradients and the
rotation over several axes, element by element against the 64-bit forms.

Bounds: one rounding to bf16 (half a step, 2^-8 of the value) plus the fp32
arithmetic's share, which scales with the block that a rotation mixes
(_qk_cache_ref)."""
import numpy as np
import pytest
import torch

import _qk_cache_ref as ref
from _qk_cache_ref import assert_within, f64

pytestmark = pytest.mark.gpu
EPS = 1e-6


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


# (tokens, Hq, Hk, d, sections, restart, base, largest position)
CASES = {
    "one_token": (1, 1, 0, 64, (32,), False, 10000.0, 100),
    "gqa": (257, 32, 8, 128, (64,), False, 10000.0, 65536),
    "odd_heads": (33, 9, 5, 128, (16, 24, 24), False, 1e6, 5000),
    "narrow": (70, 3, 1, 8, (1, 2), True, 10.0, 300),
    "width_40": (65, 5, 2, 40, (7, 6, 5), True, 10000.0, 1000),
    "width_96": (130, 17, 3, 96, (48,), False, 500000.0, (1 << 24) - 1),
    "part_turned": (100, 4, 4, 128, (8, 16), False, 10000.0, 4096),
    "many_tokens": (20011, 2, 1, 64, (16, 16), True, 10000.0, 256),
}


def _inputs(name, seed=0, fused=False):
    T, Hq, Hk, d, sections, restart, base, maxpos = CASES[name]
    g = torch.Generator().manual_seed(seed + T + d)
    if fused:
        x = torch.randn((T, Hq + 2 * Hk, d), generator=g).to(torch.bfloat16).cuda()
        Q, K = x[:, :Hq], x[:, Hq:Hq + Hk] if Hk else None
    else:
        Q = (torch.randn((T, Hq, d), generator=g) * torch.exp(torch.randn((T, Hq, 1), generator=g))).to(torch.bfloat16).cuda()
        K = torch.randn((T, Hk, d), generator=g).to(torch.bfloat16).cuda() if Hk else None
    pos = torch.randint(0, maxpos + 1, (len(sections), T), generator=g, dtype=torch.int32)
    gq = (1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda()
    gk = (1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() if Hk else None
    dYq = torch.randn((T, Hq, d), generator=g).to(torch.bfloat16).cuda()
    dYk = torch.randn((T, Hk, d), generator=g).to(torch.bfloat16).cuda() if Hk else None
    a = ref.angles(pos.numpy(), sections, d, base, restart)
    import exact_scaled_dot_gb300 as esd
    return Q, K, gq, gk, dYq, dYk, a, esd.RotaryAxes(pos.cuda(), sections, base=base, restart=restart)


def _weights(g, d):
    return np.ones(d) if g is None else f64(g)


def _check_forward(x, g, y, a, eps, what):
    want, rel, err = ref.norm_rope(f64(x), _weights(g, x.shape[-1]), a, eps)
    assert_within(f64(y), want, rel * np.abs(want) + err, what)


def _check_backward(x, g, dy, dx, dg, a, eps, what):
    want, wdg, err, dgerr = ref.norm_rope_bwd(f64(x), _weights(g, x.shape[-1]), f64(dy), a, eps)
    assert_within(f64(dx), want, ref.BF16 * np.abs(want) + err, f"d{what}")
    if g is not None:
        assert_within(f64(dg), wdg, dgerr, f"dg of {what}")


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_norm_rope(name, fused):
    import exact_scaled_dot_gb300 as esd
    Q, K, gq, gk, _, _, a, rot = _inputs(name, fused=fused)
    Yq, Yk = esd.attn_qk_norm_rope(Q, K, gq, gk, rot, eps=EPS)
    torch.cuda.synchronize()
    _check_forward(Q, gq, Yq, a, EPS, "queries")
    if K is None:
        assert Yk is None
    else:
        _check_forward(K, gk, Yk, a, EPS, "keys")


@pytest.mark.parametrize("name", list(CASES))
def test_norm_rope_backward(name):
    import exact_scaled_dot_gb300 as esd
    Q, K, gq, gk, dYq, dYk, a, rot = _inputs(name, seed=7)
    dQ, dK, dgq, dgk = esd.attn_qk_norm_rope_bwd(Q, K, gq, gk, dYq, dYk, rot, eps=EPS)
    again = esd.attn_qk_norm_rope_bwd(Q, K, gq, gk, dYq, dYk, rot, eps=EPS)
    torch.cuda.synchronize()
    _check_backward(Q, gq, dYq, dQ, dgq, a, EPS, "queries")
    if K is not None:
        _check_backward(K, gk, dYk, dK, dgk, a, EPS, "keys")
    for x, y in zip((dQ, dK, dgq, dgk), again):       # the same bits on every run
        assert (x is None and y is None) or torch.equal(x, y)


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_axes(name, inverse):
    import exact_scaled_dot_gb300 as esd
    Q, K, _, _, _, _, a, rot = _inputs(name, seed=11, fused=True)
    Yq, Yk = esd.attn_rope_axes(Q, K, rot, inverse=inverse)
    torch.cuda.synchronize()
    for x, y, what in ((Q, Yq, "queries"), (K, Yk, "keys")):
        if x is not None:
            want = ref.turn(f64(x), -a if inverse else a)
            assert_within(f64(y), want, ref.BF16 * np.abs(want) + ref.TURN * ref.pair_size(f64(x)), what)


@pytest.mark.parametrize("d,inverse", [(128, False), (64, True), (24, False)])
def test_one_axis_is_the_plain_rotation(d, inverse):
    import exact_scaled_dot_gb300 as esd
    g = torch.Generator().manual_seed(d)
    Q = torch.randn((301, 9, d), generator=g).to(torch.bfloat16).cuda()
    K = torch.randn((301, 2, d), generator=g).to(torch.bfloat16).cuda()
    pos = torch.randint(0, 1 << 20, (301,), generator=g, dtype=torch.int32).cuda()
    want = esd.attn_rope_qk(Q, K, pos, base=500000.0, inverse=inverse)
    got = esd.attn_rope_axes(Q, K, esd.RotaryAxes(pos, base=500000.0), inverse=inverse)
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_blocks_past_the_sections_keep_their_value():
    import exact_scaled_dot_gb300 as esd
    Q, K, _, _, _, _, _, rot = _inputs("part_turned")
    Yq, Yk = esd.attn_rope_axes(Q, K, rot)
    assert torch.equal(Yq[..., 48:], Q[..., 48:]) and torch.equal(Yk[..., 48:], K[..., 48:])


@pytest.mark.parametrize("weights", [False, True])
def test_norm_alone(weights):
    """Without a rotation, and with and without weights."""
    import exact_scaled_dot_gb300 as esd
    Q, K, gq, gk, dYq, dYk, a, _ = _inputs("odd_heads")
    if not weights:
        gq = gk = None
    a = np.zeros_like(a)
    Yq, Yk = esd.attn_qk_norm_rope(Q, K, gq, gk, eps=1e-3)
    dQ, dK, dgq, dgk = esd.attn_qk_norm_rope_bwd(Q, K, gq, gk, dYq, dYk, eps=1e-3)
    torch.cuda.synchronize()
    assert (dgq is None) == (gq is None)
    _check_forward(Q, gq, Yq, a, 1e-3, "queries")
    _check_forward(K, gk, Yk, a, 1e-3, "keys")
    _check_backward(Q, gq, dYq, dQ, dgq, a, 1e-3, "queries")
    _check_backward(K, gk, dYk, dK, dgk, a, 1e-3, "keys")


def test_small_large_and_zero_rows():
    import exact_scaled_dot_gb300 as esd
    Q, K, gq, gk, dYq, dYk, a, rot = _inputs("gqa")
    Q[0], Q[1], Q[2], K[3] = 0.0, Q[1] * 2.0 ** 50, Q[2] * 2.0 ** -70, K[3] * 2.0 ** -9
    Yq, Yk = esd.attn_qk_norm_rope(Q, K, gq, gk, rot, eps=EPS)
    dQ, dK, dgq, dgk = esd.attn_qk_norm_rope_bwd(Q, K, gq, gk, dYq, dYk, rot, eps=EPS)
    torch.cuda.synchronize()
    assert (Yq[0] == 0).all()
    _check_forward(Q, gq, Yq, a, EPS, "queries")
    _check_forward(K, gk, Yk, a, EPS, "keys")
    _check_backward(Q, gq, dYq, dQ, dgq, a, EPS, "queries")
    _check_backward(K, gk, dYk, dK, dgk, a, EPS, "keys")


def test_rows_whose_cubed_norm_passes_fp32():
    """r = 2^62: r^3 is beyond fp32, dx (some 2^68) is not."""
    import exact_scaled_dot_gb300 as esd
    eps = 2.0 ** -125
    Q, K, gq, gk, dYq, dYk, a, rot = _inputs("odd_heads", seed=3)
    Q = (Q.sign().double() * 2.0 ** -62).to(torch.bfloat16)
    dYq = (dYq.double() * 64).to(torch.bfloat16)
    dYq[3] = Q[3] * 2.0 ** 68
    dQ, dK, dgq, dgk = esd.attn_qk_norm_rope_bwd(Q, K, gq, gk, dYq, dYk, rot, eps=eps)
    torch.cuda.synchronize()
    _check_backward(Q, gq, dYq, dQ, dgq, a, eps, "queries")
    _check_backward(K, gk, dYk, dK, dgk, a, eps, "keys")


def test_in_place_and_views_write_nothing_else():
    import exact_scaled_dot_gb300 as esd
    T, Hq, Hk, d = 75, 6, 2, 128
    g = torch.Generator().manual_seed(1)
    x = torch.randn((T, Hq + 2 * Hk, d), generator=g).to(torch.bfloat16).cuda()
    gq = (1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda()
    rot = esd.RotaryAxes(torch.arange(T, dtype=torch.int32).cuda())
    Q, K = x[:, :Hq], x[:, Hq:Hq + Hk]
    want = esd.attn_qk_norm_rope(Q, K, gq, gq, rot)
    turned = esd.attn_rope_axes(Q, K, rot)
    dy = torch.randn((T, Hq + 2 * Hk, d), generator=g).to(torch.bfloat16).cuda()
    grads = esd.attn_qk_norm_rope_bwd(Q, K, gq, gq, dy[:, :Hq], dy[:, Hq:Hq + Hk], rot)
    for op in ("norm", "turn", "grad"):
        y = (dy if op == "grad" else x).clone()
        Y = (y[:, :Hq], y[:, Hq:Hq + Hk])
        if op == "norm":
            esd.attn_qk_norm_rope(*Y, gq, gq, rot, Yq=Y[0], Yk=Y[1])
        elif op == "turn":
            esd.attn_rope_axes(*Y, rot, Yq=Y[0], Yk=Y[1])
        else:                                           # dQ over dYq
            esd.attn_qk_norm_rope_bwd(Q, K, gq, gq, *Y, rot, dQ=Y[0], dK=Y[1])
        torch.cuda.synchronize()
        for got, ref_ in zip(Y, {"norm": want, "turn": turned, "grad": grads}[op]):
            assert torch.equal(got, ref_), op
        assert torch.equal(y[:, Hq + Hk:], (dy if op == "grad" else x)[:, Hq + Hk:]), op


def test_strided_heads():
    """Heads that are slices of wider rows, results into another layout."""
    import exact_scaled_dot_gb300 as esd
    T, H, d = 50, 3, 64
    g = torch.Generator().manual_seed(2)
    Q = torch.randn((H, T, d + 16), generator=g).to(torch.bfloat16).cuda().transpose(0, 1)[..., 8:8 + d]
    rot = esd.RotaryAxes(torch.randint(0, 99, (2, T), generator=g, dtype=torch.int32).cuda(), (10, 12))
    Y = torch.zeros((T, 2 * H, d), dtype=torch.bfloat16, device="cuda")
    esd.attn_qk_norm_rope(Q, None, None, None, rot, Yq=Y[:, ::2])
    want, _ = esd.attn_qk_norm_rope(Q.contiguous(), None, None, None, rot)
    torch.cuda.synchronize()
    assert torch.equal(Y[:, ::2], want) and (Y[:, 1::2] == 0).all()


def test_other_stream_and_replayed_graph():
    import exact_scaled_dot_gb300 as esd
    Q, K, gq, gk, dYq, dYk, a, rot = _inputs("gqa")
    want = (*esd.attn_qk_norm_rope(Q, K, gq, gk, rot), *esd.attn_qk_norm_rope_bwd(Q, K, gq, gk, dYq, dYk, rot))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = (*esd.attn_qk_norm_rope(Q, K, gq, gk, rot, stream=side),
           *esd.attn_qk_norm_rope_bwd(Q, K, gq, gk, dYq, dYk, rot, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    q, pos = Q.clone(), rot.positions
    with torch.cuda.graph(graph):
        y = (*esd.attn_qk_norm_rope(q, K, gq, gk, rot), *esd.attn_qk_norm_rope_bwd(q, K, gq, gk, dYq, dYk, rot))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, z) for x, z in zip(want, y))
    q.mul_(0.5)
    pos.add_(3)
    graph.replay()
    want = (*esd.attn_qk_norm_rope(q, K, gq, gk, rot), *esd.attn_qk_norm_rope_bwd(q, K, gq, gk, dYq, dYk, rot))
    torch.cuda.synchronize()
    assert all(torch.equal(x, z) for x, z in zip(want, y))


def test_training_step_with_packed_attention():
    """norm + rotation -> packed causal attention -> its backward -> the norm's
    backward, against the same step in fp64 (autograd over plain torch)."""
    import exact_scaled_dot_gb300 as esd
    cu, Hq, Hk, d = [0, 150, 200], 4, 2, 64
    T = cu[-1]
    g = torch.Generator().manual_seed(9)
    x = torch.randn((T, Hq + 2 * Hk, d), generator=g).to(torch.bfloat16)
    gq, gk = ((1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) for _ in range(2))
    dO = torch.randn((T, Hq, d), generator=g).to(torch.bfloat16)
    pos = torch.cat([torch.arange(b - a) for a, b in zip(cu, cu[1:])]).to(torch.int32)
    X, Gq, Gk = x.cuda(), gq.cuda(), gk.cuda()
    Q, K, V = X[:, :Hq], X[:, Hq:Hq + Hk], X[:, Hq + Hk:]
    rot = esd.RotaryAxes(pos.cuda())
    Yq, Yk = esd.attn_qk_norm_rope(Q, K, Gq, Gk, rot)
    O, LSE, O_lo = esd.attn_fwd_varlen(Yq, Yk, V, cu, cu, causal=True)
    dYq, dYk, dV = esd.attn_bwd_varlen(Yq, Yk, V, O, dO.cuda(), LSE, cu, cu, O_lo=O_lo, causal=True)
    dQ, dK, dgq, dgk = esd.attn_qk_norm_rope_bwd(Q, K, Gq, Gk, dYq, dYk, rot)
    torch.cuda.synchronize()
    # The same step in fp64.
    xr = x.double().requires_grad_()
    gr = [t.double().requires_grad_() for t in (gq, gk)]
    ang = torch.from_numpy(ref.angles(pos.numpy()[None], (d // 2,), d, 10000.0, False))
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]

    def nr(v, w):
        u = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w
        return torch.stack([u[..., 0::2] * c - u[..., 1::2] * s, u[..., 0::2] * s + u[..., 1::2] * c], -1).flatten(-2)

    yq, yk, v = nr(xr[:, :Hq], gr[0]), nr(xr[:, Hq:Hq + Hk], gr[1]), xr[:, Hq + Hk:]
    outs = []
    for a, b in zip(cu, cu[1:]):
        k, vv = (t[a:b].repeat_interleave(Hq // Hk, 1).transpose(0, 1) for t in (yk, v))
        sc = yq[a:b].transpose(0, 1) @ k.transpose(1, 2) / d ** 0.5
        sc = sc.masked_fill(torch.ones((b - a, b - a)).triu(1).bool(), float("-inf"))
        outs.append((sc.softmax(-1) @ vv).transpose(0, 1))
    (torch.cat(outs) * dO.double()).sum().backward()
    gx = xr.grad
    # The rotated rows pass through bf16 on the GPU (2^-8 each), as do the gradients between
    # the calls: in the 2-norm, where these independent roundings average, 4 of them.
    for got, want in ((dQ, gx[:, :Hq]), (dK, gx[:, Hq:Hq + Hk]), (dV, gx[:, Hq + Hk:]), (dgq, gr[0].grad), (dgk, gr[1].grad)):
        got = got.double().cpu()
        assert float((got - want).norm() / want.norm()) < 4 * ref.BF16
