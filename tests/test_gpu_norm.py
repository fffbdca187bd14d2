"""moe_add_rms_norm and its backward against their definition in 64 bits.

Tolerances: a bf16 result is off by at most half a step (2^-8 of the value), an
E4M3 code by half a step (2^-4 of the value, or 2^-10 of the scale below the
normal range).  The fp32 arithmetic before it: the sum of d squares runs in
chains of at most 64 terms per thread, five shuffle and eight warp steps, so its
relative error is below 80 * 2^-24 < 5e-6, half of it in rstd, and a handful of
products add 2^-24 each: FP = 8e-6 bounds the relative error of v."""
import pytest
import torch

import operator_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FP = 8e-6
BF = 2.0 ** -8
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def G():
    import grouped_expert_gemm_gb300 as g
    return g


def kind(name):
    return G().MOE_DTYPE_BF16 if name == "bf16" else G().MOE_DTYPE_FP32


def make(n, d, xt, rt, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((n, d), generator=gen, device=DEV)
    x = x * torch.exp(torch.randn((n, 1), generator=gen, device=DEV))
    r = 3 * torch.randn((n, d), generator=gen, device=DEV)
    if n >= 4:
        x[0], r[0] = 0, 0                      # a zero row
        x[1], r[1] = x[1] * 1e-20, r[1] * 1e-20  # squares far below eps
        x[2, d // 2] = 3e4                     # one outlier
        r[3] = 0
    w = 1 + 0.3 * torch.randn((d,), generator=gen, device=DEV)
    w[d // 3] = 0
    return x.to(TYPES[xt]), None if rt is None else r.to(TYPES[rt]), w, gen


def half_step(v, t):
    return v.abs() * BF if t is torch.bfloat16 else v.abs() * 2.0 ** -24


def forward(x, res, w, xt, rt, group, stride=None, y=True, q=True, rstd=True):
    g = G()
    n, d = x.shape
    p = g.NormParams(n, d, stride or d, kind(xt), kind(rt or xt), group, EPS)
    o = dict(h=torch.full((n, d), -7.0, device=DEV, dtype=TYPES[rt or xt]) if res is not None else None,
             y=torch.full((n, d), -7.0, device=DEV, dtype=torch.bfloat16) if y else None,
             q=torch.full((n, d), 1, device=DEV, dtype=torch.uint8) if q else None,
             s=torch.full((n, ref.groups(d, group)), -7.0, device=DEV) if q else None,
             rstd=torch.full((n,), -7.0, device=DEV) if rstd else None,
             st=torch.zeros(1, dtype=torch.int32, device=DEV))
    g.moe_add_rms_norm(p, x, res, w, o["h"], o["y"], o["q"], o["s"], o["rstd"], o["st"])
    return p, o


def check_forward(x, res, w, rt, group, o):
    h, rstd, v = ref.norm(x, res, w, EPS, TYPES.get(rt))
    d = x.shape[1]
    if o["h"] is not None:
        assert torch.equal(o["h"].double(), h)
    if o["rstd"] is not None:
        assert ((o["rstd"].double() - rstd).abs() <= FP * rstd).all()
    if o["y"] is not None:
        assert ((o["y"].double() - v).abs() <= v.abs() * (BF + 2 * FP)).all()
    if o["q"] is not None:
        s = ref.scales(v, group)
        assert ((o["s"].double() - s).abs() <= 2 * FP * s).all()
        val = o["q"].view(torch.float8_e4m3fn).double() * ref.spread(o["s"].double(), d, group)
        room = torch.maximum(v.abs() * 2.0 ** -4, ref.spread(s, d, group) * 2.0 ** -10)
        assert ((val - v).abs() <= room * (1 + 1e-3) + 2 * FP * v.abs()).all()
    return h, rstd, v


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"),
                                   ("fp32", "fp32"), ("bf16", None), ("fp32", None)])
@pytest.mark.parametrize("n,d", [(1, 16), (5, 208), (37, 512), (33, 528), (9, 2048), (7, 2064),
                                 (3, 4112), (4, 7168), (2, 8208), (3, 16384)])
def test_forward(n, d, xt, rt, group):
    x, res, w, _ = make(n, d, xt, rt, seed=n * 7 + d)
    _, o = forward(x, res, w, xt, rt, group)
    check_forward(x, res, w, rt, group, o)
    assert int(o["st"].item()) == 0


def test_many_rows_and_optional_outputs():
    x, res, w, _ = make(3001, 256, "fp32", "bf16", seed=5)
    for y, q, rstd in [(True, False, False), (False, True, True)]:
        _, o = forward(x, res, w, "fp32", "bf16", 128, y=y, q=q, rstd=rstd)
        check_forward(x, res, w, "bf16", 128, o)


@pytest.mark.parametrize("n", [0, 1, 6])
def test_row_stride_and_rows_behind_the_last(n):
    g = G()
    wide, _, w, _ = make(8, 1040, "bf16", None, seed=3)
    x = wide[:, 520:520 + 512]
    p = g.NormParams(n, 512, 1040, kind("bf16"), kind("bf16"), 128, EPS)
    y = torch.full((8, 512), -7.0, device=DEV, dtype=torch.bfloat16)
    g.moe_add_rms_norm(p, x, None, w, None, y)
    _, _, v = ref.norm(x[:n].contiguous(), None, w[:512], EPS, None)
    assert ((y[:n].double() - v).abs() <= v.abs() * (BF + 2 * FP)).all()
    assert (y[n:] == -7.0).all()


def test_residual_in_place_equals_out_of_place():
    x, res, w, _ = make(21, 2048, "fp32", "bf16", seed=11)
    p, o = forward(x, res, w, "fp32", "bf16", 0)
    r2 = res.clone()
    y2 = torch.empty_like(o["y"])
    G().moe_add_rms_norm(p, x, r2, w, r2, y2)
    assert torch.equal(r2, o["h"]) and torch.equal(y2, o["y"])


def test_nonfinite_rows_are_reported_and_stay_in_their_row():
    x, res, w, _ = make(6, 256, "bf16", "bf16", seed=2)
    clean = forward(x, res, w, "bf16", "bf16", 128)[1]
    x2 = x.clone()
    x2[4, 9] = float("nan")
    o = forward(x2, res, w, "bf16", "bf16", 128)[1]
    assert int(o["st"].item()) == G().MOE_DEV_NONFINITE_INPUT
    assert o["y"][4].isnan().all()
    keep = [0, 1, 2, 3, 5]
    assert torch.equal(o["q"][keep], clean["q"][keep]) and torch.equal(o["y"][keep], clean["y"][keep])


def backward_bounds(n, d, h, rstd, w, dy, dres, t):
    """Room for dh and dw.  dh: the fp32 products and the mean (a chain of at most 128
    terms) err by at most FP of each term's size, then the result is rounded to t.
    dw: a column is summed over at most n rows in one chain, its blocks in at most
    38 + 8 more steps, each 2^-24 of the sum of magnitudes, and each term errs by FP."""
    xh = (h * rstd[:, None]).abs()
    u = (dy.double() * w.double()).abs()
    dh, _ = ref.norm_backward(h, rstd, w, dy, dres)
    room = 2 * FP * rstd[:, None] * (u + xh * (u * xh).mean(dim=1, keepdim=True))
    if dres is not None:
        room = room + FP * dres.double().abs()
    mass = (dy.double().abs() * xh).sum(dim=0)
    return room + half_step(dh, t) * (1 + 1e-3), mass * ((-(-n // 304) * 4 + 64) * 2.0 ** -24 + FP)


@pytest.mark.parametrize("dyt", ["bf16", "fp32"])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"), ("fp32", None)])
@pytest.mark.parametrize("n,d", [(1, 8), (700, 64), (1300, 512), (33, 520), (401, 2056), (5, 4112),
                                 (611, 7168), (3, 16384)])
def test_backward(n, d, xt, rt, dyt):
    g = G()
    x, res, w, gen = make(n, d, xt, rt, seed=n + 3 * d)
    p, o = forward(x, res, w, xt, rt, 128, q=False)
    h = o["h"] if res is not None else x
    dy = torch.randn((n, d), generator=gen, device=DEV).to(TYPES[dyt])
    for dres in (None, torch.randn((n, d), generator=gen, device=DEV).to(h.dtype)):
        dx = torch.empty((n, d), device=DEV, dtype=TYPES[xt])
        dr = torch.empty((n, d), device=DEV, dtype=h.dtype)
        dw = torch.empty((d,), device=DEV)
        nb = g.moe_add_rms_norm_backward_workspace_size(p)
        ws = torch.empty((nb,), dtype=torch.uint8, device=DEV)
        g.moe_add_rms_norm_backward(p, kind(dyt), dy, h, w, o["rstd"], dres, dx, dr, dw, ws, nb)
        hd, rstd, _ = ref.norm(x, res, w, EPS, TYPES.get(rt))
        dh, dwr = ref.norm_backward(hd, rstd, w, dy, dres)
        for got in (dx, dr):
            room, wroom = backward_bounds(n, d, hd, rstd, w, dy, dres, got.dtype)
            assert ((got.double() - dh).abs() <= room + 1e-30).all()
        assert ((dw.double() - dwr).abs() <= wroom + 1e-30).all()
        dw2 = torch.empty_like(dw)
        g.moe_add_rms_norm_backward(p, kind(dyt), dy, h, w, o["rstd"], dres, None, None, dw2, ws, nb)
        assert torch.equal(dw, dw2)
        if dres is not None:  # in place over the incoming gradient
            g.moe_add_rms_norm_backward(p, kind(dyt), dy, h, w, o["rstd"], dres, None, dres, None,
                                        None, 0)
            assert torch.equal(dres, dr)


def test_backward_of_no_rows_is_zero():
    g = G()
    p = g.NormParams(0, 64, 64, 1, 1, 0, EPS)
    dw = torch.full((64,), 5.0, device=DEV)
    g.moe_add_rms_norm_backward(p, 1, None, None, None, None, None, None, None, dw, None, 0)
    assert (dw == 0).all()


def test_backward_against_differences():
    """L = <c, v(h, w)>: its directional derivative by central differences of the 64-bit
    forward (error of order step^2, 1e-8 here) against the kernel's gradients."""
    g = G()
    n, d = 9, 768
    x, res, w, gen = make(n, d, "fp32", "fp32", seed=77)
    x, res = x[3:], res[3:]  # rows of ordinary size: the difference quotient needs them smooth
    n -= 3
    c = torch.randn((n, d), generator=gen, device=DEV)
    p, o = forward(x, res, w, "fp32", "fp32", 128, q=False)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    nb = g.moe_add_rms_norm_backward_workspace_size(p)
    ws = torch.empty((nb,), dtype=torch.uint8, device=DEV)
    g.moe_add_rms_norm_backward(p, 1, c, o["h"], w, o["rstd"], None, dx, None, dw, ws, nb)

    def loss(h, wt):
        r = (h.square().mean(dim=1) + EPS).pow(-0.5)
        return (c.double() * h * r[:, None] * wt).sum()

    h, wd = o["h"].double(), w.double()
    t = 1e-4
    for _ in range(4):
        a = torch.randn((n, d), generator=gen, device=DEV).double()
        b = torch.randn((d,), generator=gen, device=DEV).double()
        num = (loss(h + t * a, wd + t * b) - loss(h - t * a, wd - t * b)) / (2 * t)
        got = (dx.double() * a).sum() + (dw.double() * b).sum()
        size = (dx.double() * a).abs().sum() + (dw.double() * b).abs().sum()
        assert (num - got).abs() <= 2e-5 * size


def test_captured_replays_and_another_stream():
    x, res, w, _ = make(64, 1024, "bf16", "bf16", seed=8)
    p, want = forward(x, res, w, "bf16", "bf16", 128)
    g = G()
    s = torch.cuda.Stream()
    h, y = torch.empty_like(want["h"]), torch.empty_like(want["y"])
    q, sc = torch.empty_like(want["q"]), torch.empty_like(want["s"])
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            g.moe_add_rms_norm(p, x, res, w, h, y, q, sc, stream=s)
        for _ in range(3):
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want["h"]) and torch.equal(y, want["y"])
    assert torch.equal(q, want["q"]) and torch.equal(sc, want["s"])


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("n", [3, 300])
def test_a_scale_that_underflows_counts_as_zero(n, group):
    """v of about 1e-44 (amax / 448 is 0 in fp32): scale 1 and zero codes, nothing reported;
    zeros among them stay zero."""
    g = G()
    d = 256
    x = torch.ones((n, d), dtype=torch.bfloat16, device=DEV)
    x[:, 5] = 0
    w = torch.full((d,), 1e-44, device=DEV)
    assert (w > 0).all()
    p = g.NormParams(n, d, d, 0, 0, group, EPS)
    q = torch.full((n, d), 0x55, dtype=torch.uint8, device=DEV)
    sc = torch.zeros((n, 1 if group == 0 else 2), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    g.moe_add_rms_norm(p, x, None, w, None, None, q, sc, None, st)
    assert (sc == 1).all() and (q == 0).all() and int(st.item()) == 0


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"),
                                   ("fp32", "fp32"), ("bf16", None), ("fp32", None)])
@pytest.mark.parametrize("n,d", [(153, 16), (155, 7168), (9001, 64), (2500, 512), (2600, 528),
                                 (1300, 2064), (1000, 7168), (480, 12288), (400, 16384)])
def test_forward_of_several_rows_a_block(n, d, xt, rt, group):
    """Rings of one to four slots that wrap, a row to a warp and to a block."""
    x, res, w, _ = make(n, d, xt, rt, seed=n + d)
    _, o = forward(x, res, w, xt, rt, group)
    check_forward(x, res, w, rt, group, o)
    assert int(o["st"].item()) == 0


@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("fp32", "fp32")])
def test_strided_rows_and_residual_in_place_of_several_rows_a_block(xt, rt):
    g = G()
    wide, res, w, _ = make(1500, 2080, xt, rt, seed=41)
    x, res, w = wide[:, 16:1056], res[:, :1040].contiguous(), w[:1040].contiguous()
    x[7, 3] = float("nan")
    _, o = forward(x.contiguous(), res, w, xt, rt, 128)
    assert int(o["st"].item()) == g.MOE_DEV_NONFINITE_INPUT
    p = g.NormParams(1500, 1040, 2080, kind(xt), kind(rt), 128, EPS)
    r2, y2, q2, s2 = res.clone(), torch.empty_like(o["y"]), torch.empty_like(o["q"]), torch.empty_like(o["s"])
    g.moe_add_rms_norm(p, x, r2, w, r2, y2, q2, s2)
    keep = torch.arange(1500, device=DEV) != 7
    for a, b in ((r2, o["h"]), (y2, o["y"]), (q2, o["q"]), (s2, o["s"])):
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("dyt", ["bf16", "fp32"])
@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("fp32", "bf16"), ("bf16", "fp32"), ("fp32", None)])
@pytest.mark.parametrize("n,d", [(1, 8200), (700, 8208), (480, 12288), (330, 16384)])
def test_backward_of_wide_rows(n, d, xt, rt, dyt):
    test_backward(n, d, xt, rt, dyt)


@pytest.mark.parametrize("rt", ["bf16", "fp32"])
def test_backward_of_wide_rows_in_place_and_without_parts(rt):
    g = G()
    n, d = 500, 12288
    x, res, w, gen = make(n, d, "bf16", rt, seed=43)
    p, o = forward(x, res, w, "bf16", rt, 128, q=False)
    dy = torch.randn((n, d), generator=gen, device=DEV).to(torch.bfloat16)
    dres = torch.randn((n, d), generator=gen, device=DEV).to(TYPES[rt])
    nb = g.moe_add_rms_norm_backward_workspace_size(p)
    ws = torch.empty((nb,), dtype=torch.uint8, device=DEV)
    dr, dw, dw2 = torch.empty_like(dres), torch.empty_like(w), torch.empty_like(w)
    g.moe_add_rms_norm_backward(p, 0, dy, o["h"], w, o["rstd"], dres, None, dr, dw, ws, nb)
    g.moe_add_rms_norm_backward(p, 0, dy, o["h"], w, o["rstd"], None, None, None, dw2, ws, nb)
    assert torch.equal(dw, dw2)  # the order of the sums does not depend on dres
    g.moe_add_rms_norm_backward(p, 0, dy, o["h"], w, o["rstd"], dres, None, dres, None, None, 0)
    assert torch.equal(dres, dr)
