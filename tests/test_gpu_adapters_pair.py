"""The projection in tiles of two CTAs (256 weight columns by 256 tokens), with the reduction
over the ranks of a tile of one adapter, and batches whose rows outgrow the L2.  Each case makes sure
that its calls take such tiles, so that a changed rule shows.  (The rule takes them where both
sides are a few thousand long; 152 SMs.)"""
import re
import warnings

import pytest
import torch

import adapter_reference as ref
from test_gpu_adapters import (DEV, G, check_forward, i32, live_rows, make, project,
                               project_backward)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def kernels(call, path):
    """The captured call's graph as text, with its kernels' names."""
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        call()
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")  # (says that it is called)
        graph.debug_dump(str(path))
    return path.read_text()


def tile_tokens(names):
    """Tokens of the projections' tiles: the kernel's first template argument."""
    return {int(n) for n in re.findall(r"project_kernel(?:ILi|<)(?:\(int\))?(\d+)", names)}


CASES = [
    # T, offsets, adapters, d, n, r, N
    # one adapter for the whole batch, for whole tiles, and across a tile's border: the ranks that
    # the tensor cores reduce (8 to 32) and more of them
    (2300, [0, 2300], [1], 2056, 2040, 8, 2),
    (2300, [0, 1024, 2000, 2300], [0, 1, 0], 2056, 2040, 16, 2),
    (2300, [0, 600, 2290], [2, 0], 2056, 2040, 24, 3),
    (2304, [0, 256, 512, 1500, 2304], [1, -1, 0, 1], 2056, 2040, 32, 2),
    (2300, [5, 800, 800, 2300], [1, 0, 1], 2056, 2040, 40, 2),
    (2300, [0, 1536, 2300], [1, 0], 2056, 2040, 64, 2),
    (2300, [0, 700, 2290], [0, 2], 2056, 2040, 104, 3),
    (2300, [0, 2300], [0], 2056, 2040, 128, 1),
    # single tokens, short runs and rows without an adapter in front of long segments
    (2300, list(range(41)) + [400, 1200, 2290], [q % 5 - 1 for q in range(43)], 2056, 2040, 16, 4),
    (2300, [3] + list(range(4, 24)) + [700, 701, 1500, 2281], [q % 8 - 1 for q in range(24)], 2056, 2040, 72, 7),
    (2300, [0, 34, 50, 64, 70, 2180], [-1, 1, -1, 0, -1], 2056, 2040, 24, 2),
    (2300, [0] + list(range(3, 123, 3)) + [1000, 2300], [q % 3 for q in range(42)], 2056, 2040, 128, 3),
    # several tiles a pair, tiles of one adapter between others (each pair lays down its ranks anew)
    (4000, [0, 700, 1300, 3990], [1, 0, 2], 2056, 2040, 32, 3),
    (4000, [0, 1500, 1530, 4000], [3, 1, 2], 2056, 2040, 16, 4),
    (4000, [0] + list(range(900, 970)) + [4000], [q % 4 for q in range(71)], 2056, 2040, 8, 4),
]


@pytest.mark.parametrize("T,off,ids,d,n,r,N", CASES)
@pytest.mark.parametrize("stride", [0, 24])
def test_pairs(T, off, ids, d, n, r, N, stride, tmp_path):
    g = G()
    x, w, a, b, scale, rnd = make(T, d, n, r, N, seed=T + r, x_stride=d + stride)
    t = (x, w, a, b, scale)
    dy = rnd(T, n + stride).to(BF)[:, :n]
    mod = g.AdapterProjection(T, w, a, b, scale, device=DEV)
    seg, adp = i32(off), i32(ids)
    assert tile_tokens(kernels(lambda: mod.forward(x, adp, seg), tmp_path / "forward")) == {256}
    assert tile_tokens(kernels(lambda: mod.backward(dy), tmp_path / "backward")) == {256}
    u, _, _ = check_forward(t, off, ids, y_stride=n + stride if stride else None)
    dx, da, db = project_backward(t, off, ids, u, dy)
    segs = ref.segments(off, ids, T)
    (dx64, dxr), (da64, dar), (db64, dbr) = ref.backward(x, w, a, b, scale, segs, dy)
    live = live_rows(segs, T)
    assert (dx[~live] == -7.0).all()
    assert ((dx.double() - dx64).abs() <= dxr + ref.half_step(dx64, BF) * 1.01)[live].all()
    assert ((da.double() - da64).abs() <= dar).all()
    assert ((db.double() - db64).abs() <= dbr).all()


@pytest.mark.parametrize("r", [16, 24, 72])
@pytest.mark.parametrize("off,ids", [
    ([0, 512, 1280, 1290, 2290], [0, 1, 2, 3]),          # whole tiles of one adapter beside others
    (list(range(20)) + [600, 610, 2000, 2290], [q % 4 for q in range(23)])])
def test_values_stay_with_their_requests_in_pairs(off, ids, r):
    """NaN and infinities of adapter 0's tables, of one row and of rows behind the last segment
    reach only the rows and the gradients that use them."""
    T, d, n, N = 2300, 2056, 2040, 4
    x, w, a, b, scale, rnd = make(T, d, n, r, N, seed=r)
    dy = rnd(T, n).to(BF)
    u, y, _ = project((x, w, a, b, scale), off, ids)
    dx, da, db = project_backward((x, w, a, b, scale), off, ids, u, dy)
    bad, q = off[-2] - 1, len(ids) - 2  # a row of the last segment but one
    x2, dy2, a2, b2 = x.clone(), dy.clone(), a.clone(), b.clone()
    x2[bad], dy2[bad] = float("nan"), float("inf")
    x2[off[-1]:], dy2[off[-1]:] = float("nan"), float("nan")
    a2[0, 3], b2[0, :, 5] = float("inf"), float("nan")
    u2, y2, _ = project((x2, w, a2, b2, scale), off, ids)
    dx2, da2, db2 = project_backward((x2, w, a2, b2, scale), off, ids, u2, dy2)
    touched = torch.zeros(T, dtype=torch.bool, device=DEV)
    touched[bad] = True
    for p, e, i in ref.segments(off, ids, T):
        if i == 0:
            touched[p:e] = True
    bits = lambda t: t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)  # noqa: E731
    for new, old in ((u2, u), (y2, y), (dx2, dx)):
        assert torch.equal(bits(new[~touched]), bits(old[~touched]))
    clean = [e for e in range(N) if e not in (0, ids[q])]
    assert torch.equal(bits(da2[clean]), bits(da[clean]))
    assert torch.equal(bits(db2[clean]), bits(db[clean]))
    assert torch.isnan(y2[bad].float()).all()


@pytest.mark.parametrize("case", [CASES[3], CASES[9], CASES[13]])
def test_pairs_captured_and_on_two_streams(case):
    g = G()
    T, off, ids, d, n, r, N = case
    x, w, a, b, scale, rnd = make(T, d, n, r, N, seed=3)
    dy = rnd(T, n).to(BF)
    seg, adp = i32(off), i32(ids)

    def run(mod, stream=None):
        y = mod.forward(x, adp, seg, stream=stream)
        return (y, mod.u) + mod.backward(dy, stream=stream)

    mods = [g.AdapterProjection(T, w, a, b, scale, device=DEV) for _ in range(3)]
    first = [t.clone() for t in run(mods[0])]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        both = [run(m, s) for m, s in zip(mods[1:], streams)]
    torch.cuda.synchronize()
    for got in both:
        assert all(torch.equal(p, q) for p, q in zip(first, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(mods[1])
    for t in got:
        t.fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    live = live_rows(ref.segments(off, ids, T), T)
    for i, (p, q) in enumerate(zip(first, got)):
        assert torch.equal(p[live], q[live]) if i < 3 else torch.equal(p, q)
        if i < 3:  # y, u, dx: rows of no segment stay
            assert (q[~live] == 5.0).all()
    for m in mods:
        assert int(m.dev_status.item()) == 0


@pytest.mark.parametrize("T,off,ids,d,n,r,N,tile", [
    # rows of more than 80 MB beside a small weight: their tiles stay, the columns go round
    (10300, [0, 3000, 10290], [1, 0], 4104, 264, 16, 2, 128),
    (10300, list(range(60)) + [5000, 10300], [q % 3 - 1 for q in range(61)], 4104, 2056, 24, 2, 256)])
def test_rows_that_outgrow_the_l2(T, off, ids, d, n, r, N, tile, tmp_path):
    g = G()
    x, w, a, b, scale, rnd = make(T, d, n, r, N, seed=T)
    mod = g.AdapterProjection(T, w, a, b, scale, device=DEV)
    seg, adp = i32(off), i32(ids)
    assert tile_tokens(kernels(lambda: mod.forward(x, adp, seg), tmp_path / "forward")) == {tile}
    check_forward((x, w, a, b, scale), off, ids)
    if tile == 128:
        check_forward((x, w, a, b, scale), off, ids, torch.float32)
    # turned around: dy is the one that outgrows it
    x2, w2, a2, b2, scale2, rnd = make(T, n, d, r, N, seed=T + 1)
    dy = rnd(T, d).to(BF)
    t = (x2, w2, a2, b2, scale2)
    u, _, _ = project(t, off, ids)
    dx, _, _ = project_backward(t, off, ids, u, dy)
    segs = ref.segments(off, ids, T)
    (dx64, dxr), _, _ = ref.backward(x2, w2, a2, b2, scale2, segs, dy)
    live = live_rows(segs, T)
    assert ((dx.double() - dx64).abs() <= dxr + ref.half_step(dx64, BF) * 1.01)[live].all()
