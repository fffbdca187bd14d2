"""AdapterProjection as a training program uses it: gradients summed over replays of a captured
step, several micro-batches, and what each kind of backward reports."""
import pytest
import torch

import adapter_reference as ref
from test_gpu_adapters import DEV, G, MARK, i32, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


T, D, N_OUT, R, N = 150, 264, 136, 16, 3
OFF, IDS = [4, 30, 31, 140], [2, 0, 2]


def step(seed):
    x, w, a, b, scale, rnd = make(T, D, N_OUT, R, N, seed=seed)
    return x, w, a, b, scale, rnd(T, N_OUT).to(torch.bfloat16)


def gradients(x, w, a, b, scale, dy):
    """da and db of an object of their own that adds nothing up."""
    m = G().AdapterProjection(T, w, a, b, scale, device=DEV)
    m.forward(x, i32(IDS), i32(OFF))
    dx, da, db = m.backward(dy)
    return dx.clone(), da.clone(), db.clone()


def test_replays_of_a_first_backward_add_up():
    """The first backward of an object is captured, with accumulate: K replays hold the sum of K
    gradients, in fp32 additions in that order, and rows of no segment of dx are not written."""
    g = G()
    x, w, a, b, scale, dy = step(11)
    dx1, da1, db1 = gradients(x, w, a, b, scale, dy)
    ids, off = i32(IDS), i32(OFF)
    m = g.AdapterProjection(T, w, a, b, scale, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(x, ids, off)
        dx, da, db = m.backward(dy, accumulate=True)
    torch.cuda.synchronize()
    assert not da.any() and not db.any()  # zeros at first; a capture runs nothing
    dx.fill_(MARK)
    want_a, want_b = torch.zeros_like(da1), torch.zeros_like(db1)
    for _ in range(3):
        graph.replay()
        want_a, want_b = want_a + da1, want_b + db1
    torch.cuda.synchronize()
    assert torch.equal(da, want_a) and torch.equal(db, want_b)
    assert (dx[:OFF[0]] == MARK).all() and (dx[OFF[-1]:] == MARK).all()
    assert torch.equal(dx[OFF[0]:OFF[-1]], dx1[OFF[0]:OFF[-1]])
    # and eagerly onto the same sums
    m.forward(x, ids, off)
    m.backward(dy, accumulate=True)
    assert torch.equal(da, want_a + da1) and torch.equal(db, want_b + db1)


def test_micro_batches_add_up():
    g = G()
    x, w, a, b, scale, _ = step(12)
    m = g.AdapterProjection(T, w, a, b, scale, device=DEV)
    want_a = want_b = 0.0
    for seed in (12, 13, 14):
        x, _, _, _, _, dy = step(seed)
        _, da1, db1 = gradients(x, w, a, b, scale, dy)
        want_a, want_b = want_a + da1, want_b + db1
        m.forward(x, i32(IDS), i32(OFF))
        _, da, db = m.backward(dy, accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(da, want_a) and torch.equal(db, want_b)
    _, da, db = m.backward(dy)  # without it they start again
    assert torch.equal(da, da1) and torch.equal(db, db1)


@pytest.mark.parametrize("want", ["x", "a", "b", "ab", "xab"])
def test_every_backward_reports_bad_tables(want):
    g = G()
    x, w, a, b, scale, dy = step(15)
    u = torch.zeros((T, R), device=DEV)
    out = dict(x=torch.zeros((T, D), dtype=torch.bfloat16, device=DEV),
               a=torch.zeros(a.shape, device=DEV), b=torch.zeros(b.shape, device=DEV))
    p = g.AdapterParams(T, D, N_OUT, R, N, 3)
    nb = g.moe_adapter_project_backward_workspace_size(p)
    ws = torch.zeros((nb,), dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    for off, ids, bit in (([0, 20, 40, T], [0, 1, 2], 0), ([0, 40, 20, T], [0, 1, 2], g.MOE_DEV_BAD_MAP),
                          ([0, 20, 40, T + 1], [0, 1, 2], g.MOE_DEV_BAD_MAP),
                          ([0, 20, 40, T], [0, N, 2], g.MOE_DEV_BAD_ADAPTER),
                          ([0, 20, 40, T], [0, -2, 2], g.MOE_DEV_BAD_ADAPTER)):
        st.zero_()
        g.moe_adapter_project_backward(p, i32(off), i32(ids), x, w, a, b, scale, u, dy,
                                       *(out[k] if k in want else None for k in "xab"), 0, ws, nb, st)
        assert int(st.item()) == bit


def test_gradients_of_a_captured_step_against_the_definition():
    g = G()
    x, w, a, b, scale, dy = step(16)
    m = g.AdapterProjection(T, w, a, b, scale, device=DEV)
    ids, off = i32(IDS), i32(OFF)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(x, ids, off)
        dx, da, db = m.backward(dy, accumulate=True)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    _, (da64, dar), (db64, dbr) = ref.backward(x, w, a, b, scale, ref.segments(OFF, IDS, T), dy)
    assert ((da.double() - 2 * da64).abs() <= 2 * dar).all()
    assert ((db.double() - 2 * db64).abs() <= 2 * dbr).all()


def test_first_forward_on_another_stream():
    """Results do not race with the clearing of the buffers that hold them, which the current stream
    does behind other work."""
    g = G()
    x, w, a, b, scale, dy = step(17)
    busy = torch.empty((1 << 30,), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    ids, off = i32(IDS), i32(OFF)
    torch.cuda.synchronize()
    for _ in range(100):
        busy.fill_(1)
    m = g.AdapterProjection(T, w, a, b, scale, device=DEV)
    y = m.forward(x, ids, off, stream=side)
    dx, da, db = m.backward(dy, stream=side)
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, m.u, dx, da, db)]
    m.forward(x, ids, off)
    m.backward(dy)
    assert all(torch.equal(p, q) for p, q in zip(got, (y, m.u, dx, da, db)))
    assert y[OFF[0]:OFF[-1]].any() and da.any() and int(m.dev_status.item()) == 0


def test_rows_and_results_side_by_side_in_one_buffer():
    g = G()
    x, w, a, b, scale, dy = step(18)
    m = g.AdapterProjection(T, w, a, b, scale, device=DEV)
    ids, off = i32(IDS), i32(OFF)
    want = m.forward(x, ids, off).clone()
    grads = [t.clone() for t in m.backward(dy)]
    wide = torch.full((T, 8 + D + N_OUT), MARK, dtype=torch.bfloat16, device=DEV)
    wide[:, :D] = x
    m.forward(wide[:, :D], ids, off, out=wide[:, D + 8:])
    live = slice(OFF[0], OFF[-1])
    assert torch.equal(wide[live, D + 8:], want[live]) and torch.equal(wide[:, :D], x)
    assert (wide[:, D:D + 8] == MARK).all()
    wide[:, D + 8:] = dy
    assert all(torch.equal(p, q) for p, q in zip(m.backward(wide[:, D + 8:]), grads))


def test_objects_are_refused_inside_a_capture():
    """(and the capture goes on)"""
    g = G()
    x, w, a, b, scale, dy = step(19)
    m = g.AdapterProjection(T, w, a, b, scale, device=DEV)
    ids, off = i32(IDS), i32(OFF)
    want = m.forward(x, ids, off).clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="capture"):
            g.AdapterProjection(T, w, a, b, scale, device=DEV)
        with pytest.raises(ValueError, match="capture"):
            g.GradientClip([scale], 1.0, device=DEV)
        m.forward(x, ids, off)
    m.y.fill_(MARK)
    graph.replay()
    live = slice(OFF[0], OFF[-1])
    assert torch.equal(m.y[live], want[live]) and (m.y[:OFF[0]] == MARK).all()
