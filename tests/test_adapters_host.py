"""Host-side refusals of the projection with adapters and of clipping (every call returns before
its first CUDA call, so no GPU is touched), the plan of a table of gradients, and the gradients'
formulas against differences."""
import ctypes
import math

import pytest
import torch

import adapter_reference as ref


@pytest.fixture(scope="module")
def g():
    import grouped_expert_gemm_gb300 as g
    from grouped_expert_gemm_gb300 import build
    build.build()
    return g


def test_project_refusals(g):
    L, P = g.abi.lib(), g.AdapterParams
    ARG, UNS = g.MOE_ERR_INVALID_ARG, g.MOE_ERR_UNSUPPORTED

    def fwd(p, off=16, adp=16, x=16, w=16, a=16, b=16, s=16, u=16, y=16):
        return L.moe_adapter_project(p, off, adp, x, w, a, b, s, u, y, None, None)

    assert fwd(P(0, 64, 64, 16, 2, 3)) == g.MOE_OK
    assert fwd(P(0, 64, 64, 16, 2, 3), x=None, y=None) == g.MOE_OK
    assert L.moe_adapter_project(None, *[16] * 9, None, None) == ARG
    for p in (P(-1, 64, 64, 16, 2, 3), P(4, 0, 64, 16, 2, 3), P(4, 64, 0, 16, 2, 3),
              P(4, 64, 64, 0, 2, 3), P(4, 64, 64, 16, 0, 3), P(4, 64, 64, 16, 2, 0),
              P(4, 64, 64, 16, 2, 3, y_type=2), P(4, 64, 64, 16, 2, 3, x_stride=56),
              P(4, 64, 64, 16, 2, 3, y_stride=56)):
        assert fwd(p) == ARG
    for p in (P(4, 60, 64, 16, 2, 3), P(4, 64, 60, 16, 2, 3), P(4, 64, 64, 12, 2, 3),
              P(4, 64, 64, 136, 2, 3), P(4, 65544, 64, 16, 2, 3), P(4, 64, 65544, 16, 2, 3),
              P(4, 64, 64, 16, 65536, 3), P(4, 64, 64, 16, 2, 65536),
              P((1 << 31) - 1, 64, 64, 16, 2, 3), P(4, 64, 64, 16, 2, 3, x_stride=68),
              P(4, 64, 64, 16, 2, 3, y_stride=68), P(4, 64, 64, 16, 2, 3, x_stride=(1 << 31) + 8),
              P(1 << 30, 64, 65536, 16, 2, 3)):
        assert fwd(p) == UNS
    p = P(4, 64, 64, 16, 2, 3)
    for k in ("off", "adp", "x", "w", "a", "b", "s", "u", "y"):
        assert fwd(p, **{k: None}) == ARG
    for k in ("x", "w", "a", "b", "u", "y"):
        assert fwd(p, **{k: 24}) == UNS
    for k in ("off", "adp", "s"):
        assert fwd(p, **{k: 18}) == UNS

    def bwd(p, off=16, adp=16, x=16, w=16, a=16, b=16, s=16, u=16, dy=16, dx=16, da=16, db=16,
            acc=0, ws=16, nb=1 << 30):
        return L.moe_adapter_project_backward(p, off, adp, x, w, a, b, s, u, dy, dx, da, db, acc,
                                              ws, nb, None, None)

    for k in ("off", "adp", "x", "w", "a", "b", "s", "u", "dy", "ws"):
        assert bwd(p, **{k: None}) == ARG
    for k in ("x", "w", "a", "b", "u", "dy", "dx", "da", "db", "ws"):
        assert bwd(p, **{k: 24}) == UNS
    assert bwd(p, dx=None, da=None, db=None) == ARG
    assert bwd(p, acc=2) == ARG and bwd(p, acc=-1) == ARG
    nb = g.moe_adapter_project_backward_workspace_size(p)
    assert nb >= 4 * 16 * 4 and bwd(p, nb=nb - 1) == g.MOE_ERR_WORKSPACE_TOO_SMALL
    assert g.moe_adapter_project_backward_workspace_size(P(4, 60, 64, 16, 2, 3)) == 0
    assert bwd(P(0, 64, 64, 16, 2, 3), acc=1, ws=None, nb=0) == g.MOE_OK  # nothing to add


def table(g, rows):
    t = (g.GradTensor * len(rows))()
    for e, (grad, out, count, kind, group) in zip(t, rows):
        e.grad, e.out, e.count, e.type, e.group = grad, out, count, kind, group
    return t


def test_grad_plan(g):
    rows = [(16, 16, 100_000, 1, 0), (None, None, 0, 0, 0), (18, 20, 100_001, 0, 1), (16, 16, 1, 1, 1),
            (16, 16, 5, 0, 4), (None, None, 0, 1, 4)]
    t = table(g, rows)
    n = g.moe_grad_plan(t, 5)
    first = [e.first_chunk for e in t] + [n]
    # whole chunks, none for a tensor without elements, one for a few elements
    assert first[0] == 0 and 0 < first[1] == first[2] < first[3] == first[4] - 1 == first[5] - 2 == n - 2
    assert [(e.group_begin, e.group_end) for e in t] == \
        [(0, first[2])] * 2 + [(first[2], first[4])] * 2 + [(first[4], n)] * 2
    assert g.moe_grad_plan((g.GradTensor * 0)(), 1) == 0
    L, n = g.abi.lib(), ctypes.c_int64()
    ARG, UNS = g.MOE_ERR_INVALID_ARG, g.MOE_ERR_UNSUPPORTED
    plan = lambda rows, groups=2: L.moe_grad_plan(len(rows), table(g, rows), groups, ctypes.byref(n))  # noqa: E731
    good = (16, 16, 10, 1, 0)
    assert plan([good]) == g.MOE_OK
    for bad in ((None, 16, 10, 1, 0), (16, None, 10, 1, 0), (16, 16, -1, 1, 0), (16, 16, 10, 2, 0),
                (16, 16, 10, 1, -1), (16, 16, 10, 1, 2)):
        assert plan([bad]) == ARG
    assert plan([(16, 16, 10, 1, 1), good]) == ARG  # groups out of order
    assert plan([(18, 16, 10, 1, 0)]) == UNS and plan([(16, 17, 10, 0, 0)]) == UNS
    assert plan([(16, 16, (1 << 50) + 1, 0, 0)]) == UNS and plan([good], 1 << 21) == UNS
    assert plan([good], 0) == ARG
    assert L.moe_grad_plan(1, None, 1, ctypes.byref(n)) == ARG
    assert L.moe_grad_plan(-1, table(g, [good]), 1, ctypes.byref(n)) == ARG
    assert L.moe_grad_plan(1, table(g, [good]), 1, None) == ARG


def test_clip_refusals(g):
    L = g.abi.lib()
    ARG, UNS = g.MOE_ERR_INVALID_ARG, g.MOE_ERR_UNSUPPORTED

    def clip(n=1, t=16, c=1, G=1, m=1.0, norms=16, ws=16, nb=1 << 20):
        return L.moe_clip_grads(n, t, c, G, m, norms, ws, nb, None, None)

    for kw in (dict(n=-1), dict(n=0), dict(t=None), dict(c=-1), dict(G=0), dict(m=0.0), dict(m=-1.0),
               dict(m=math.nan), dict(norms=None), dict(ws=None)):
        assert clip(**kw) == ARG
    for kw in (dict(t=20), dict(ws=20), dict(norms=18), dict(G=(1 << 20) + 1), dict(c=(1 << 40) + 1)):
        assert clip(**kw) == UNS
    nb = g.moe_clip_grads_workspace_size(7)
    assert nb > 0 and clip(G=7, nb=nb - 1) == g.MOE_ERR_WORKSPACE_TOO_SMALL
    assert g.moe_clip_grads_workspace_size(0) == 0


def test_objects_refuse(g):
    bf = torch.bfloat16
    w, a, b, s = (torch.zeros(64, 72, dtype=bf), torch.zeros(2, 8, 64, dtype=bf),
                  torch.zeros(2, 8, 72, dtype=bf), torch.zeros(2))
    new = lambda **kw: g.AdapterProjection(4, **{**dict(weight=w, a=a, b=b, scale=s, device="cpu"), **kw})  # noqa: E731
    m = new()
    for kw in (dict(weight=w.float()), dict(a=a[:, :, :56]), dict(b=b[:1]), dict(scale=s[:1]),
               dict(a=a[0]), dict(weight=None), dict(y_dtype=torch.float16),
               dict(a=torch.zeros(2, 12, 64, dtype=bf), b=torch.zeros(2, 12, 72, dtype=bf))):
        with pytest.raises(ValueError):
            new(**kw)
    x = torch.zeros(4, 64, dtype=bf)
    ids, off = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for args in ((x[:3], ids, off), (x.float(), ids, off), (x, ids, None), (x, ids.long(), off),
                 (x, ids, off[:2]), (x, ids[:0], off[:1]), (x, None, off),
                 (torch.zeros(4, 68, dtype=bf)[:, :64], ids, off), (x.t().contiguous().t(), ids, off)):
        with pytest.raises(ValueError):
            m.forward(*args)
    with pytest.raises(ValueError):
        m.forward(x, ids, off, out=torch.zeros(4, 72))
    with pytest.raises(ValueError):
        m.backward(torch.zeros(4, 72, dtype=bf))  # no forward before it
    t = torch.zeros(5)
    for kw in (dict(max_norm=0.0), dict(max_norm=math.nan), dict(out=[]), dict(groups=[0, 1]),
               dict(groups=[1], n_groups=1), dict(groups=[-1]), dict(n_groups=0),
               dict(out=[torch.zeros(4)]), dict(out=[t.double()]), dict(grads=[t.double()]),
               dict(grads=[torch.zeros(4, 4)[:, :2]]), dict(norms=torch.zeros(2))):
        with pytest.raises(ValueError):
            g.GradientClip(**{**dict(grads=[t], max_norm=1.0, device="cpu"), **kw})


def test_clip_refuses_overlapping_tensors(g):
    flat = torch.ones(64)
    make = lambda grads, out=None: g.GradientClip(grads, 1.0, out=out, device="cpu")  # noqa: E731
    make([flat[:32], flat[32:]])  # neighbours
    make([flat[:32]], out=[flat[32:]])
    make([flat[:32], flat[8:8]])  # no elements
    for grads, out in (([flat, flat], None), ([flat[:33], flat[32:]], None),
                       ([flat[:32]], [flat[1:33]]),  # a result behind its own gradient
                       ([flat[:16], flat[16:32]], [flat[16:32], flat[32:48]]),
                       ([flat[:16], flat[16:32]], [flat[40:56], flat[40:56]])):
        with pytest.raises(ValueError, match="overlap"):
            make(grads, out)


def test_formulas_against_differences():
    """The gradients' formulas, by central differences in 64 bits."""
    gen = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    T, d, n, r, N = 9, 6, 5, 3, 3
    x, w, a, b, s, dy = rnd(T, d), rnd(d, n), rnd(N, r, d), rnd(N, r, n), rnd(N).abs(), rnd(T, n)
    segs = ref.segments([0, 2, 2, 3, 7, 9], [1, 0, -1, 2, 1], T)
    loss = lambda: (ref.forward(x, w, a, b, s, segs)[2] * dy).sum()  # noqa: E731
    grads = ref.backward(x, w, a, b, s, segs, dy)
    for t, (g64, _) in zip((x, a, b), grads):
        flat, h = t.view(-1), 1e-5
        for i in range(flat.numel()):
            old = float(flat[i])
            flat[i] = old + h
            up = loss()
            flat[i] = old - h
            down = loss()
            flat[i] = old
            assert abs((up - down) / (2 * h) - g64.reshape(-1)[i]) <= 1e-7
