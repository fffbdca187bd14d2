"""moe_adapter_project and its backward against their definition in 64 bits (the room of the
fp32 arithmetic is derived in adapter_reference), their rows that stay as they are, and the
isolation of one request's values from another's."""
import pytest
import torch

import adapter_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MARK = -7.0  # what rows of no segment hold, before and after


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def G():
    import grouped_expert_gemm_gb300 as g
    return g


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def make(T, d, n, r, N, seed=0, x_stride=None):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    bf = torch.bfloat16
    x = rnd(T, x_stride or d).to(bf)[:, :d]
    w = (rnd(d, n) / d ** 0.5).to(bf)
    a = (rnd(N, r, d) / d ** 0.5).to(bf)
    b = (rnd(N, r, n) / r ** 0.5).to(bf)
    return x, w, a, b, torch.exp(0.5 * rnd(N)), rnd


def project(t, off, ids, y_type=torch.bfloat16, y_stride=None, st=None, stream=None):
    g = G()
    x, w, a, b, scale = t
    T, (d, n), (N, r) = x.shape[0], w.shape, a.shape[:2]
    u = torch.full((T, r), MARK, device=DEV)
    wide = torch.full((T, y_stride or n), MARK, device=DEV, dtype=y_type)
    kind = g.MOE_DTYPE_BF16 if y_type is torch.bfloat16 else g.MOE_DTYPE_FP32
    p = g.AdapterParams(T, d, n, r, N, len(ids), kind, x.stride(0), y_stride or n)
    g.moe_adapter_project(p, None if off is None else i32(off), i32(ids), x, w, a, b, scale, u,
                          wide, st, stream)
    return u, wide, p


def live_rows(segs, T):
    live = torch.zeros(T, dtype=torch.bool, device=DEV)
    for b, e, _ in segs:
        live[b:e] = True
    return live


def check_forward(t, off, ids, y_type=torch.bfloat16, y_stride=None):
    x, w, a, b, scale = t
    T, n = x.shape[0], w.shape[1]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    u, wide, p = project(t, off, ids, y_type, y_stride, st)
    segs = ref.segments(off, ids, T)
    u64, ur, y64, yr = ref.forward(x, w, a, b, scale, segs)
    live = live_rows(segs, T)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert (u[~live] == MARK).all() and (wide[~live] == MARK).all() and (wide[:, n:] == MARK).all()
    y = wide[:, :n].double()
    assert ((u.double() - u64).abs() <= ur + ref.half_step(u64, torch.float32))[live].all()
    assert ((y - y64).abs() <= yr + ref.half_step(y64, y_type) * 1.01)[live].all()
    return u, wide, p


SHAPES = [
    # T, offsets, adapters, d, n, r, N
    (1, None, [0], 64, 8, 8, 1),
    (1, [0, 1], [2], 2048, 768, 16, 3),
    (1, [0, 1], [-1], 136, 264, 128, 1),
    (5, [0, 2, 2, 5], [1, 0, 1], 72, 200, 24, 2),             # an empty segment, one adapter twice
    (17, list(range(18)), [q % 5 - 1 for q in range(17)], 520, 136, 32, 4),
    (33, [0, 33], [0], 1040, 96, 64, 1),
    (128, list(range(129)), [(7 * q) % 13 - 1 for q in range(128)], 512, 1024, 40, 12),
    (128, [0, 3, 90, 120], [3, 1, 0], 8, 4096, 128, 4),       # rows behind the last segment
    (300, [11, 60, 60, 61, 299], [0, 1, 2, 0], 328, 720, 16, 3),  # and before the first
    (1021, [0, 1, 2, 3, 500, 1000, 1021], [4, 0, -1, 2, 2, 1], 256, 256, 104, 5),
    (2048, [0, 2048], [1], 512, 392, 16, 2),
    # tiles of two CTAs, forward and (turned around) backward
    (2290, [3] + list(range(4, 24)) + [700, 701, 1500, 2281], [q % 8 - 1 for q in range(24)], 200, 2040, 72, 7),
    (2290, [0, 9, 1000, 1000, 2290], [2, 1, 0, 1], 2040, 200, 16, 3),
    # runs between rows without an adapter, inside 32 rows
    (2200, [0, 34, 50, 64, 70, 2180], [-1, 1, -1, 0, -1], 200, 2040, 24, 2),
    (100, [1, 4, 9, 40, 60, 97], [-1, 1, -1, 0, -1], 328, 136, 8, 2),
    # single tokens beside long segments in tiles of two CTAs; more segments than are looked over
    # piece by piece; reductions of several fp32 pieces, whole and shared by a cluster
    (2290, list(range(41)) + [400, 1200, 2290], [q % 5 - 1 for q in range(43)], 200, 2040, 128, 4),
    (3500, list(range(2900)) + [3100, 3490], [q % 7 - 1 for q in range(2901)], 64, 72, 16, 6),
    (2290, [0, 700, 1300, 2290], [1, 0, 2], 2056, 2040, 8, 3),
    (40, [0, 5, 39], [1, 0], 6000, 136, 48, 2),
    # whole tiles of two CTAs with one adapter, of 8, 16, 24 and 32 ranks, and beside others
    (2304, [0, 2304], [1], 320, 2048, 16, 2),
    (2304, [0, 1024, 2000, 2304], [0, 1, 0], 320, 1928, 8, 2),
    (2300, [0, 600, 2290], [2, 0], 264, 2048, 24, 3),
    (2304, [0, 256, 512, 1500, 2304], [1, -1, 0, 1], 2048, 264, 32, 2),
    (700, [0] * 300 + [400] * 200 + [700], [q % 3 for q in range(500)], 128, 128, 8, 3),
]


@pytest.mark.parametrize("T,off,ids,d,n,r,N", SHAPES)
@pytest.mark.parametrize("y_type", [torch.bfloat16, torch.float32])
def test_forward(T, off, ids, d, n, r, N, y_type):
    *t, _ = make(T, d, n, r, N, seed=T + d)
    check_forward(t, off, ids, y_type)


@pytest.mark.parametrize("T,off,ids,d,n,r,N", SHAPES)
def test_forward_strided(T, off, ids, d, n, r, N):
    *t, _ = make(T, d, n, r, N, seed=T, x_stride=d + 24)
    check_forward(t, off, ids, y_stride=n + 40)


def project_backward(t, off, ids, u, dy, accumulate=0, da=None, db=None, want="xab"):
    g = G()
    x, w, a, b, scale = t
    T, (d, n), (N, r) = x.shape[0], w.shape, a.shape[:2]
    p = g.AdapterParams(T, d, n, r, N, len(ids), 0, x.stride(0), dy.stride(0))
    nb = g.moe_adapter_project_backward_workspace_size(p)
    ws = torch.full((nb,), 0x7F, dtype=torch.uint8, device=DEV)
    dx = torch.full((T, d), MARK, dtype=torch.bfloat16, device=DEV)
    da = torch.full(a.shape, MARK, device=DEV) if da is None else da
    db = torch.full(b.shape, MARK, device=DEV) if db is None else db
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    g.moe_adapter_project_backward(p, None if off is None else i32(off), i32(ids), x, w, a, b,
                                   scale, u, dy, dx if "x" in want else None,
                                   da if "a" in want else None, db if "b" in want else None,
                                   accumulate, ws, nb, st)
    assert int(st.item()) == 0
    return dx, da, db


@pytest.mark.parametrize("T,off,ids,d,n,r,N", SHAPES)
@pytest.mark.parametrize("stride", [0, 16])
def test_backward(T, off, ids, d, n, r, N, stride):
    x, w, a, b, scale, rnd = make(T, d, n, r, N, seed=T + 1, x_stride=d + stride)
    t = (x, w, a, b, scale)
    dy = rnd(T, n + stride).to(torch.bfloat16)[:, :n]
    u, _, _ = project(t, off, ids)
    dx, da, db = project_backward(t, off, ids, u, dy)
    segs = ref.segments(off, ids, T)
    (dx64, dxr), (da64, dar), (db64, dbr) = ref.backward(x, w, a, b, scale, segs, dy)
    live = live_rows(segs, T)
    assert (dx[~live] == MARK).all()
    assert ((dx.double() - dx64).abs() <= dxr + ref.half_step(dx64, torch.bfloat16) * 1.01)[live].all()
    assert ((da.double() - da64).abs() <= dar).all()
    assert ((db.double() - db64).abs() <= dbr).all()
    # added to what is there
    da0, db0 = rnd(*a.shape), rnd(*b.shape)
    _, da2, db2 = project_backward(t, off, ids, u, dy, 1, da0.clone(), db0.clone())
    assert torch.equal(da2, da0 + da) and torch.equal(db2, db0 + db)
    # a part of the outputs: the same bits
    dx3, da3, db3 = project_backward(t, off, ids, u, dy, want="x")
    assert torch.equal(dx3, dx) and (da3 == MARK).all() and (db3 == MARK).all()
    dx4, da4, db4 = project_backward(t, off, ids, u, dy, want="ab")
    assert (dx4 == MARK).all() and torch.equal(da4, da) and torch.equal(db4, db)


def test_gradient_against_differences():
    """y is linear in each table: the difference of sum(y dy) over a step is the gradient's
    product with the step, without a remainder."""
    T, d, n, r, N, off, ids = 200, 256, 264, 16, 3, [0, 70, 71, 200], [2, 0, 2]
    x, w, a, b, scale, rnd = make(T, d, n, r, N, seed=5)
    dy = rnd(T, n).to(torch.bfloat16)
    u, y, _ = project((x, w, a, b, scale), off, ids, torch.float32)
    dx, da, db = project_backward((x, w, a, b, scale), off, ids, u, dy)
    segs = ref.segments(off, ids, T)
    total = lambda t: (t.double() * dy.double()).sum()  # noqa: E731
    for which in range(3):
        other = [x, a, b]
        other[which] = (other[which].float() + 0.5 * rnd(*other[which].shape)).to(torch.bfloat16)
        step = other[which].double() - (x, a, b)[which].double()
        _, y2, _ = project((other[0], w, other[1], other[2], scale), off, ids, torch.float32)
        got = ((dx, da, db)[which].double() * step).sum()
        _, _, _, r1 = ref.forward(x, w, a, b, scale, segs)
        _, _, _, r2 = ref.forward(other[0], w, other[1], other[2], scale, segs)
        (dx64, dxr), (da64, dar), (db64, dbr) = ref.backward(x, w, a, b, scale, segs, dy)
        room = (((dxr + ref.half_step(dx64, torch.bfloat16)), dar, dbr)[which] * step.abs()).sum() + \
            ((r1 + r2 + y2.double().abs() * 2.0 ** -23) * dy.double().abs()).sum()
        assert abs(total(y2) - total(y) - got) <= room


@pytest.mark.parametrize("T,off,ids", [
    (64, list(range(65)), [q % 4 for q in range(64)]),
    (700, [0, 10, 300, 301, 302, 640, 690], [0, 1, 2, 3, 1, 0]),
    (2000, [0, 700, 1000, 1990], [3, 0, 2]),
])
def test_values_stay_with_their_requests(T, off, ids):
    """NaN and infinities of adapter 0's tables, of one row and of rows behind the last segment
    reach only the rows and the gradients that use them."""
    d, n, r, N = 264, 392, 24, 4
    x, w, a, b, scale, rnd = make(T, d, n, r, N, seed=1)
    dy = rnd(T, n).to(torch.bfloat16)
    u, y, _ = project((x, w, a, b, scale), off, ids)
    dx, da, db = project_backward((x, w, a, b, scale), off, ids, u, dy)
    bad = off[2] - 1  # a row of the second segment
    x2, dy2, a2, b2 = x.clone(), dy.clone(), a.clone(), b.clone()
    x2[bad], dy2[bad] = float("nan"), float("inf")
    x2[off[-1]:], dy2[off[-1]:] = float("nan"), float("nan")
    a2[0, 3], b2[0, :, 5] = float("inf"), float("nan")
    u2, y2, _ = project((x2, w, a2, b2, scale), off, ids)
    dx2, da2, db2 = project_backward((x2, w, a2, b2, scale), off, ids, u2, dy2)
    segs = ref.segments(off, ids, T)
    touched = torch.zeros(T, dtype=torch.bool, device=DEV)
    touched[bad] = True
    for p, q, e in segs:
        if e == 0:
            touched[p:q] = True
    bits = lambda t: t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)  # noqa: E731
    for new, old in ((u2, u), (y2, y), (dx2, dx)):
        assert torch.equal(bits(new[~touched]), bits(old[~touched]))
    clean = [e for e in range(N) if e not in (0, ids[1])]
    assert torch.equal(bits(da2[clean]), bits(da[clean]))
    assert torch.equal(bits(db2[clean]), bits(db[clean]))
    assert torch.isnan(y2[bad].float()).all()


@pytest.mark.parametrize("T,off,ids,d,n,r,N", [SHAPES[1], SHAPES[6], SHAPES[9]])
def test_same_bits_captured_and_on_another_stream(T, off, ids, d, n, r, N):
    g = G()
    x, w, a, b, scale, rnd = make(T, d, n, r, N, seed=3)
    dy = rnd(T, n).to(torch.bfloat16)
    seg, adp = (None if off is None else i32(off)), i32(ids)

    def run(mod, stream=None):
        y = mod.forward(x, adp, seg, stream=stream)
        return (y, mod.u) + mod.backward(dy, stream=stream)

    first = [t.clone() for t in run(g.AdapterProjection(T, w, a, b, scale, device=DEV))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = g.AdapterProjection(T, w, a, b, scale, device=DEV)
    torch.cuda.synchronize()
    got = run(other, side)
    side.synchronize()
    for p, q in zip(first, got):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(other)
    for t in got:
        t.fill_(5.0)
    keep = [t.clone() for t in got]
    graph.replay()
    torch.cuda.synchronize()
    live = live_rows(ref.segments(off, ids, T), T)
    for i, (p, q) in enumerate(zip(first, got)):
        if i < 3:  # y, u, dx: rows of no segment stay
            assert torch.equal(p[live], q[live]) and torch.equal(keep[i][~live], q[~live])
        else:
            assert torch.equal(p, q)


def test_two_streams_at_once():
    """Objects of their own on two streams, their kernels side by side: each gives what it gives
    alone."""
    g = G()
    shapes = [SHAPES[6], SHAPES[9]]
    mods, args, alone = [], [], []
    for i, (T, off, ids, d, n, r, N) in enumerate(shapes):
        x, w, a, b, scale, rnd = make(T, d, n, r, N, seed=20 + i)
        m = g.AdapterProjection(T, w, a, b, scale, device=DEV)
        mods.append(m)
        args.append((x, i32(ids), None if off is None else i32(off), rnd(T, n).to(torch.bfloat16)))
        y = m.forward(*args[i][:3])
        alone.append([t.clone() for t in (y, m.u) + m.backward(args[i][3])])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for m, (x, ids, off, dy), s in zip(mods, args, streams):
            got = (m.forward(x, ids, off, stream=s), m.u) + m.backward(dy, stream=s)
            m.last = got
    torch.cuda.synchronize()
    for m, want in zip(mods, alone):
        assert int(m.dev_status.item()) == 0
        assert all(torch.equal(p, q) for p, q in zip(m.last, want))


def test_results_into_a_slice():
    g = G()
    T, d, n, r, N = 130, 136, 264, 16, 2
    x, w, a, b, scale, _ = make(T, d, n, r, N, seed=9, x_stride=d + 8)
    m = g.AdapterProjection(T, w, a, b, scale, y_dtype=torch.float32, device=DEV)
    off, ids = i32([0, 100, 130]), i32([1, 0])
    want = m.forward(x, ids, off).clone()
    wide = torch.full((T, n + 48), MARK, device=DEV)
    assert m.forward(x, ids, off, out=wide[:, 16:16 + n]).data_ptr() == wide.data_ptr() + 64
    assert torch.equal(wide[:, 16:16 + n], want)
    assert (wide[:, :16] == MARK).all() and (wide[:, 16 + n:] == MARK).all()


def test_bad_tables_are_reported():
    g = G()
    *t, rnd = make(64, 128, 136, 16, 3)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    u, y, _ = project(t, [0, 20, 40, 64], [1, 3, -2], st=st)
    assert int(st.item()) == g.MOE_DEV_BAD_ADAPTER
    u0, y0, _ = project(t, [0, 20, 40, 64], [1, -1, -1])  # such an adapter counts as none
    assert torch.equal(u, u0) and torch.equal(y, y0)
    for off in ([0, 40, 20, 64], [0, 20, 40, 65], [-1, 20, 40, 64], [64, 0, -5, 1 << 30],
                [0, 0, 1 << 30, 5]):
        st.zero_()
        guard = torch.full((66, 136), MARK, device=DEV, dtype=torch.bfloat16)
        x, w, a, b, scale = t
        p = g.AdapterParams(64, 128, 136, 16, 3, 3)
        u = torch.full((66, 16), MARK, device=DEV)
        g.moe_adapter_project(p, i32(off), i32([0, 1, 2]), x, w, a, b, scale, u[1:], guard[1:], st)
        assert int(st.item()) == g.MOE_DEV_BAD_MAP
        assert (guard[0] == MARK).all() and (guard[65] == MARK).all()
        assert (u[0] == MARK).all() and (u[65] == MARK).all()
        dy = rnd(64, 136).to(torch.bfloat16)
        nb = g.moe_adapter_project_backward_workspace_size(p)
        ws = torch.empty((nb,), dtype=torch.uint8, device=DEV)
        da, db = torch.empty_like(a, dtype=torch.float32), torch.empty_like(b, dtype=torch.float32)
        dx = torch.full((66, 128), MARK, device=DEV, dtype=torch.bfloat16)
        g.moe_adapter_project_backward(p, i32(off), i32([0, 1, 2]), x, w, a, b, scale, u[1:], dy,
                                       dx[1:], da, db, 0, ws, nb, st)
        assert (dx[0] == MARK).all() and (dx[65] == MARK).all()


def test_empty_batch():
    g = G()
    x, w, a, b, scale, _ = make(0, 64, 72, 8, 2)
    p = g.AdapterParams(0, 64, 72, 8, 2, 1)
    u, y = torch.empty((0, 8), device=DEV), torch.empty((0, 72), device=DEV, dtype=torch.bfloat16)
    g.moe_adapter_project(p, None, i32([0]), x, w, a, b, scale, u, y)
    da, db = torch.full(a.shape, MARK, device=DEV), torch.full(b.shape, MARK, device=DEV)
    for acc, want in ((1, MARK), (0, 0.0)):
        g.moe_adapter_project_backward(p, None, i32([0]), x, w, a, b, scale, u, y, None, da, db,
                                       acc, None, 0)
        assert (da == want).all() and (db == want).all()
