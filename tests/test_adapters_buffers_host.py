"""What AdapterProjection owns, and the calls of the adapters' classes that are refused before any CUDA
call (no GPU is touched)."""
import pytest
import torch

BF = torch.bfloat16


@pytest.fixture(scope="module")
def g():
    import grouped_expert_gemm_gb300 as g
    from grouped_expert_gemm_gb300 import build
    build.build()
    return g


def tables(d=64, n=72, r=8, N=2):
    return dict(weight=torch.zeros(d, n, dtype=BF), a=torch.zeros(N, r, d, dtype=BF),
                b=torch.zeros(N, r, n, dtype=BF), scale=torch.zeros(N))


def test_gradient_buffers_are_made_with_the_object(g):
    """A capture of the first backward records no clearing of them."""
    m = g.AdapterProjection(4, **tables(), device="cpu")
    dx, da, db, ws = m._grads
    assert dx.shape == (4, 64) and da.shape == (2, 8, 64) and db.shape == (2, 8, 72)
    assert not (dx.any() or da.any() or db.any()) and ws.numel() == m.ws_bytes
    m = g.AdapterProjection(4, **tables(), device="cpu", gradients=False)
    assert m._grads is None
    with pytest.raises(ValueError, match="without gradients"):
        m.backward(torch.zeros(4, 72, dtype=BF))


def test_overlap_of_rows():
    from grouped_expert_gemm_gb300.adapters import _overlap
    wide = torch.zeros(6, 48, dtype=BF)
    for p, q, want in (
            (wide[:, :16], wide[:, 16:], False), (wide[:, 16:], wide[:, :16], False),
            (wide[:, :16], wide[:, 8:24], True), (wide[:, 8:24], wide[:, :16], True),
            (wide[:, 16:32], wide[:, 16:32], True), (wide[:, :16], wide[:, 40:], False),
            (wide[:3, :16], wide[3:, :16], False), (wide[:3], wide[2:5], True),
            (wide[:, :16], wide[1:, 16:], False), (wide[1:, :24], wide[:5, 16:40], True),
            (wide, wide.view(-1)[5:6], True), (wide[:2], wide.view(-1)[96:], False),
            (wide[0:1, :16], wide[0:1, 16:], False), (wide[0:1], wide[0:1, 40:], True),
            (wide[:, 1:47].view(torch.int16), wide[:, 46:], True), (wide[:0], wide, False),
            (wide[:, :8], torch.zeros(6, 48, dtype=BF), False),
            (wide[::2, :16], wide[:3, 16:], False), (wide[::2, :16], wide[1::2, :16], False),
            (wide[::2, :16], wide[:3, 8:], True), (wide[::3, :16], wide[:4:2, 16:32], False),
            # a row's slice that goes on into the next row of the other
            (wide[:, 40:], wide.view(-1)[44:188].view(3, 48), True)):
        assert _overlap(p, q) == _overlap(q, p) == want


def test_outputs_that_a_call_reads_are_refused(g):
    d = 64
    t = tables(d, d)
    m = g.AdapterProjection(4, **t, device="cpu")
    ids, off = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    wide = torch.zeros(4, 3 * d, dtype=BF)
    for x, out in ((m.y, None),                          # the result of the last call as the next one's rows
                   (wide[:, :d], wide[:, d - 8:2 * d - 8]), (wide[:, :d], wide[:, :d]),
                   (wide[:, :d], t["weight"][8:12]), (wide[:, :d], t["b"][1, 2:6])):
        with pytest.raises(ValueError, match="overlap"):
            m.forward(x, ids, off, out=out)
    f = g.AdapterProjection(4, **tables(d, 8), y_dtype=torch.float32, device="cpu")
    with pytest.raises(ValueError, match="overlap"):
        f.forward(torch.zeros(4, d, dtype=BF), ids, off, out=f.u)
    m._last = (torch.zeros(4, d, dtype=BF), ids, off)
    with pytest.raises(ValueError, match="overlap"):
        m.backward(m._grads[0])                          # the last dx as the next dy
    m._last = (m._grads[0], ids, off)
    with pytest.raises(ValueError, match="overlap"):
        m.backward(torch.zeros(4, d, dtype=BF))


def test_norms_apart_from_the_gradients(g):
    flat = torch.ones(64)
    g.GradientClip([flat[:32]], 1.0, norms=flat[32:33], device="cpu")
    for grads, out, norms in (([flat[:32]], None, flat[31:32]), ([flat[:32]], [flat[32:]], flat[40:41]),
                              ([flat.view(8, 8)], None, flat[:1])):
        with pytest.raises(ValueError, match="overlap"):
            g.GradientClip(grads, 1.0, out=out, norms=norms, device="cpu")
