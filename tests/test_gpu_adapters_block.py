"""A block whose router has adapters, run together as a step uses it: norm, router projection
(fp32 logits), layer, balance loss; then the backward, the adapters' gradients, one norm for each
adapter and the clipped gradients.  Each stage is held to its 64-bit definition on the values that
the stage before it stored, and the captured step gives the eager one's bits."""
import pytest
import torch

import adapter_reference as ref
import operator_reference as op

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


class Step:
    def __init__(self, T, d, E, k, I, r, N, off, ids, seed=0):
        import grouped_expert_gemm_gb300 as g
        gen = torch.Generator(device=DEV).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
        self.rnd, self.T, self.k, self.d, self.E, self.N = rnd, T, k, d, E, N
        w = [(rnd(E, p, q) / p ** 0.5).to(BF) for p, q in ((d, I), (d, I), (I, d))]
        self.layer = g.MoELayer(T, d, E, k, I, *w, device=DEV)
        self.norm = g.TokenNorm(T, d, 1 + 0.2 * rnd(d), device=DEV)
        self.tables = ((rnd(d, E) / d ** 0.5).to(BF), (rnd(N, r, d) / d ** 0.5).to(BF),
                       (rnd(N, r, E) / r ** 0.5).to(BF), torch.exp(0.3 * rnd(N)))
        self.router = g.AdapterProjection(T, *self.tables, y_dtype=torch.float32, device=DEV)
        self.loss = g.RouterLoss(T, E, k, 0.01, device=DEV)
        self.off, self.ids = off, ids
        self.seg = torch.tensor(off, dtype=torch.int32, device=DEV)
        self.adp = torch.tensor(ids, dtype=torch.int32, device=DEV)
        self.x, self.res, self.dout = rnd(T, d).to(BF), rnd(T, d).to(BF), rnd(T, d)
        R = T * k
        self.dy = torch.zeros((max(R, 1), d), dtype=BF, device=DEV)
        self.dgates = torch.empty((T, k), device=DEV)
        self.clip = None
        self.g = g

    def run(self):
        g, T, k, d = self.g, self.T, self.k, self.d
        rows = self.norm.forward(self.x, self.res)
        logits = self.router.forward(rows, self.adp, self.seg)
        out = self.layer.forward(logits, rows)
        self.loss.forward(logits, self.layer.topk_ids)
        g.moe_combine_backward(T, k, d, self.dout, self.layer.y, T * k, self.layer.route_to_row,
                               self.layer.gates, self.dy, self.dgates)
        dz = self.loss.backward(logits, self.layer.topk_ids, None, self.layer.gates, self.dgates)
        self.dz = dz.to(BF)
        dx, da, db = self.router.backward(self.dz)
        if self.clip is None:  # one norm for each adapter; made once, when the gradients are there
            grads = [t[e] for e in range(self.N) for t in (da, db)]
            self.clip = g.GradientClip(grads, 1e-3, out=[torch.empty_like(t) for t in grads],
                                       groups=[e for e in range(self.N) for _ in range(2)], device=DEV)
        norms = self.clip.clip()
        dxn, dres, dw = self.norm.backward(dx)
        return [rows, logits, out, dz, dx, da, db, norms, dxn, dres, dw] + self.clip.out


@pytest.mark.parametrize("T,d,E,k,I,r,N,off,ids", [
    (37, 256, 16, 4, 128, 16, 3, [0, 1, 2, 30, 37], [2, -1, 0, 2]),
    (300, 512, 64, 8, 128, 40, 5, [0, 120, 121, 122, 300], [4, 1, 0, 4])])
def test_block_with_an_adapted_router(T, d, E, k, I, r, N, off, ids):
    s = Step(T, d, E, k, I, r, N, off, ids)
    got = [t.clone() for t in s.run()]
    torch.cuda.synchronize()
    for m in (s.norm, s.router, s.layer, s.loss, s.clip):
        assert int(m.dev_status.item()) == 0
    rows, logits, out, dz, dx, da, db, norms = got[:8]
    segs = ref.segments(off, ids, T)
    _, _, y64, yr = ref.forward(rows, *s.tables, segs)
    assert ((logits.double() - y64).abs() <= yr + ref.half_step(y64, torch.float32)).all()
    want = op.balance_grad(logits, s.layer.topk_ids, [0, T], 0.01, 1.0, E, k, False) + \
        op.gate_grad(logits, s.layer.topk_ids, s.layer.gates, s.dgates, False, 1.0)
    assert ((dz.double() - want).abs() <= 2e-5 * (want.abs().max() + s.dgates.abs().max())).all()
    (dx64, dxr), (da64, dar), (db64, dbr) = ref.backward(rows, *s.tables, segs, s.dz)
    assert ((dx.double() - dx64).abs() <= dxr + ref.half_step(dx64, BF) * 1.01).all()
    assert ((da.double() - da64).abs() <= dar).all() and ((db.double() - db64).abs() <= dbr).all()
    n64, c64 = ref.clip(s.clip.grads, [e for e in range(N) for _ in range(2)], N, 1e-3)
    for a, b in zip(norms.tolist(), n64):
        assert abs(a - float(b)) <= float(b) * 8 * 2.0 ** -24
    for a, b in zip(got[11:], c64):
        assert ((a.double() - b).abs() <= b.abs() * 14 * 2.0 ** -24 + 1e-45).all()
    # captured and replayed: the same bits
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = s.run()
    for t in again[:1] + again[2:]:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(got, again):
        assert torch.equal(p, q)
