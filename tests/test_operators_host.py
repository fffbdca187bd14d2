"""Host-side refusals of the norm, balance-loss and 8-bit expert calls: every one returns
before its first CUDA call, so no GPU is touched."""
import math

import pytest


@pytest.fixture(scope="module")
def g():
    import grouped_expert_gemm_gb300 as g
    from grouped_expert_gemm_gb300 import build
    build.build()
    return g


def test_norm_refusals(g):
    L, N = g.abi.lib(), g.NormParams
    ARG, UNS = g.MOE_ERR_INVALID_ARG, g.MOE_ERR_UNSUPPORTED

    def fwd(p, x=16, res=16, w=16, ro=16, y=16, q=None, s=None, rstd=None):
        return L.moe_add_rms_norm(p, x, res, w, ro, y, q, s, rstd, None, None)

    ok = N(0, 64)
    assert fwd(ok) == g.MOE_OK  # no rows: nothing launches
    # an empty batch has no addresses: nothing to refuse, whatever the types
    assert fwd(N(0, 64, x_type=1), x=None, res=None, ro=None, y=None) == g.MOE_OK
    assert L.moe_add_rms_norm(None, 16, 16, 16, 16, 16, None, None, None, None, None) == ARG
    for p in (N(-1, 64), N(1, 0), N(1, -8), N(1, 64, x_type=2), N(1, 64, residual_type=-1),
              N(1, 64, group=64), N(1, 64, eps=0.0), N(1, 64, eps=-1.0), N(1, 64, eps=math.nan),
              N(1, 64, eps=math.inf), N(1, 64, x_stride=63)):
        assert fwd(p) == ARG
    for p in (N(1, 60), N(1, 16392), N(1, 64, x_stride=68), N(1 << 40, 64)):
        assert fwd(p) == UNS
    p = N(1, 64)
    assert fwd(p, x=None) == ARG and fwd(p, w=None) == ARG and fwd(p, ro=None) == ARG
    assert fwd(p, y=None) == ARG                        # no output at all
    assert fwd(p, q=16) == ARG and fwd(p, s=16) == ARG  # codes without scales, scales alone
    assert fwd(N(1, 64, residual_type=1), res=None) == ARG  # h = x has x's type
    assert fwd(N(1, 72), q=16, s=16) == UNS             # codes need d % 16 == 0
    for k in ("x", "res", "w", "ro", "y"):
        assert fwd(p, **{k: 24}) == UNS
    assert fwd(p, q=24, s=16) == UNS and fwd(p, q=16, s=18) == UNS and fwd(p, rstd=18) == UNS

    def bwd(p, t=0, dy=16, h=16, w=16, rstd=16, dro=None, dx=16, dr=None, dw=None, ws=None, nb=0):
        return L.moe_add_rms_norm_backward(p, t, dy, h, w, rstd, dro, dx, dr, dw, ws, nb, None)

    assert bwd(ok) == g.MOE_OK and bwd(ok, dy=None, h=None, rstd=None, dx=None) == g.MOE_OK
    assert bwd(p, t=2) == ARG and bwd(p, dx=None) == ARG
    for k in ("dy", "h", "w", "rstd"):
        assert bwd(p, **{k: None}) == ARG
    for k in ("dy", "h", "w", "dro", "dx", "dr"):
        assert bwd(p, **{k: 24}) == UNS
    assert bwd(p, dw=16, ws=None) == ARG
    assert bwd(p, dw=16, ws=16, nb=255) == g.MOE_ERR_WORKSPACE_TOO_SMALL
    assert g.moe_add_rms_norm_backward_workspace_size(p) == 256
    assert g.moe_add_rms_norm_backward_workspace_size(N(1, 12)) == 0


def test_balance_refusals(g):
    L, P = g.abi.lib(), g.RouteParams
    ARG, UNS = g.MOE_ERR_INVALID_ARG, g.MOE_ERR_UNSUPPORTED
    soft = lambda T=4, E=8, k=2: P(T, E, k, 0, 1, 1, 1.0)  # noqa: E731

    def fwd(p, S=1, off=None, z=16, ids=16, alpha=0.1, c=16, t=16, m=16, loss=16, ws=16, nb=1 << 30):
        return L.moe_balance_loss(p, S, off, z, ids, alpha, c, t, m, loss, ws, nb, None, None)

    for p in (soft(T=-1), soft(E=0), soft(k=0), soft(k=9), P(4, 8, 2, 7, 1, 1, 1.0),
              P(4, 8, 2, 1, 1, 1, 0.0), P(4, 8, 2, 1, 1, 1, math.nan)):
        assert fwd(p) == ARG
    assert fwd(soft(E=513)) == UNS and fwd(soft(E=32, k=17)) == UNS
    assert fwd(soft(T=1 << 30, k=2)) == UNS
    p = soft()
    assert fwd(p, S=0) == ARG and fwd(p, S=2) == ARG and fwd(p, S=65536, off=16) == UNS
    for k in ("z", "ids", "c", "t", "m", "loss", "ws"):
        assert fwd(p, **{k: None}) == ARG
        assert fwd(p, **{k: 18}) == UNS
    assert fwd(p, off=18) == UNS
    assert fwd(p, alpha=math.inf) == ARG and fwd(p, alpha=math.nan) == ARG
    nb = g.moe_balance_loss_workspace_size(p, 1)
    assert nb > 0 and fwd(p, nb=nb - 1) == g.MOE_ERR_WORKSPACE_TOO_SMALL
    assert g.moe_balance_loss_workspace_size(soft(E=513), 1) == 0

    def bwd(p, S=1, off=None, z=16, ids=16, gates=16, dg=16, alpha=0.1, c=16, t=16, dl=None, dz=16):
        return L.moe_route_backward(p, S, off, z, ids, gates, dg, alpha, c, t, dl, dz, None, None)

    assert bwd(soft(T=0)) == g.MOE_OK
    assert bwd(p, c=None) == ARG and bwd(p, t=None) == ARG
    assert bwd(p, c=None, t=None, dg=None) == ARG  # neither part
    for k in ("z", "ids", "gates", "dz"):
        assert bwd(p, **{k: None}) == ARG
        assert bwd(p, **{k: 18}) == UNS
    assert bwd(p, dl=18) == UNS and bwd(p, alpha=math.nan) == ARG


def test_expert_refusals(g):
    L = g.abi.lib()
    ARG, UNS = g.MOE_ERR_INVALID_ARG, g.MOE_ERR_UNSUPPORTED
    names = ("xq", "xs", "b", "c", "g0", "s0", "g1", "s1", "g2", "s2", "y", "ws")

    def call(n=2, d=64, I=128, R=8, nb=1 << 30, **kw):
        a = [kw.get(k, 16) for k in names]
        return L.moe_grouped_swiglu_w8(n, d, I, R, *a, nb, None, None)

    assert call(R=0) == g.MOE_OK
    for kw in (dict(n=0), dict(d=0), dict(I=-16), dict(R=-1)):
        assert call(**kw) == ARG
    for kw in (dict(n=1025), dict(d=72), dict(I=24), dict(d=65552), dict(I=65552)):
        assert call(**kw) == UNS
    for k in names:
        assert call(**{k: None}) == ARG, k
        assert call(**{k: 18}) == UNS, k
    for k in ("xq", "g0", "g1", "g2", "y", "ws"):
        assert call(**{k: 24}) == UNS, k
    nb = g.moe_grouped_swiglu_w8_workspace_size(8, 128)
    assert nb >= 8 * 128 + 8 * 4 and call(nb=nb - 1) == g.MOE_ERR_WORKSPACE_TOO_SMALL
    assert g.moe_grouped_swiglu_w8_workspace_size(8, 24) == 0
    assert g.moe_grouped_swiglu_w8_workspace_size(-1, 128) == 0

    up = lambda **kw: L.moe_grouped_gate_up_w8(2, 64, 128, 8, *[kw.get(k, 16) for k in names[:8]], kw.get("hq", 16), kw.get("hs", 16), None, None)  # noqa: E731,E501
    assert up(hq=None) == ARG and up(hs=None) == ARG and up(hq=24) == UNS and up(hs=18) == UNS
    dn = lambda **kw: L.moe_grouped_down_w8(2, 64, 128, 8, *[kw.get(k, 16) for k in ("xq", "xs", "b", "c", "g0", "s0", "y")], None, None)  # noqa: E731,E501
    for k in ("xq", "xs", "b", "c", "g0", "s0", "y"):
        assert dn(**{k: None}) == ARG and dn(**{k: 18}) == UNS
    q = L.moe_quantize_weights_fp8
    assert q(0, 16, 16, 16, 16, 16, None, None) == ARG and q(1, 16, 16, None, 16, 16, None, None) == ARG
    assert q(1, 24, 16, 16, 16, 16, None, None) == UNS and q(1, 16, 16, 24, 16, 16, None, None) == UNS


def test_balance_token_indexes_stay_in_32_bits(g):
    """A tile past T must not pass 2^31."""
    for T, ok in (((1 << 31) - 1, False), ((1 << 31) - (1 << 23), False), ((1 << 31) - (1 << 23) - 1, True)):
        p = g.RouteParams(T, 8, 1, 0, 1, 1, 1.0)
        assert (g.moe_balance_loss_workspace_size(p, 1) > 0) == ok
        st = g.abi.lib().moe_route_backward(p, 1, None, None, 16, 16, 16, 0.1, 16, 16, None, 16, None, None)
        assert st == (g.MOE_ERR_INVALID_ARG if ok else g.MOE_ERR_UNSUPPORTED)  # (no logits)


@pytest.mark.parametrize("other", [b"\0" * 64, "16", 16.0, (16, 16), [16]],
                         ids=["bytes", "str", "float", "tuple", "list"])
def test_arguments_that_are_neither_tensor_nor_address(g, other):
    """Bytes and strings would pass as the address of their own storage."""
    with pytest.raises(TypeError, match="expected a tensor"):
        g.moe_add_rms_norm(g.NormParams(0, 64), other, None, 16, None, 16)
    with pytest.raises(TypeError, match="expected a tensor"):
        g.moe_quantize_weights_fp8(0, 16, 16, 16, other, 16)
