"""The adapters' calls at their limits: 65,535 adapters, 65,535 segments."""
import pytest
import torch

import adapter_reference as ref
from test_gpu_adapters import DEV, G, MARK

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def test_65535_adapters_and_segments():
    g = G()
    N, S, d, n, r = 65535, 65535, 64, 72, 8
    gen = torch.Generator(device=DEV).manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    lengths = torch.randint(0, 3, (S,), generator=gen, device=DEV)  # empty ones among them
    lengths[7] = 300
    off = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)])
    live, T = int(off[-1]), int(off[-1]) + 5
    ids = torch.randint(-1, N, (S,), generator=gen, device=DEV)
    ids[-1], ids[7], ids[9] = N - 1, 0, 0
    row = torch.repeat_interleave(ids, lengths)                     # a row's adapter
    x, dy = rnd(T, d).to(BF), rnd(T, n).to(BF)
    w = (rnd(d, n) / d ** 0.5).to(BF)
    a, b = (rnd(N, r, d) / d ** 0.5).to(BF), (rnd(N, r, n) / r ** 0.5).to(BF)
    s = torch.exp(0.5 * rnd(N))
    m = g.AdapterProjection(T, w, a, b, s, device=DEV)
    m.y.fill_(MARK)
    m._grads[0].fill_(MARK)
    y = m.forward(x, ids.int(), off.int())
    dx, da, db = m.backward(dy)
    assert int(m.dev_status.item()) == 0
    assert (y[live:] == MARK).all() and (dx[live:] == MARK).all()

    has, e = (row >= 0).double()[:, None], row.clamp(min=0)
    S64 = s.double()[e][:, None] * has

    def side(p, q, left, right):
        """p left, the part of each row's own adapter and its bound, and the whole with its bound"""
        p = p[:live].double()
        u = torch.einsum("tk,trk->tr", p, left[e].double()) * S64
        ur = torch.einsum("tk,trk->tr", p.abs(), left[e].double().abs()) * S64 * (ref.chain(p.shape[1]) + 2 * ref.STEP)
        out = p @ q.double() + torch.einsum("tr,trk->tk", u, right[e].double())
        size = torch.einsum("tr,trk->tk", u.abs(), right[e].double().abs())
        room = p.abs() @ q.double().abs() * ref.chain(p.shape[1]) + size * (ref.PAIR + ref.chain(2 * r)) + \
            torch.einsum("tr,trk->tk", ur, right[e].double().abs())
        return u, ur, out, room

    u, ur, y64, yr = side(x, w, a, b)
    v, vr, dx64, dxr = side(dy, w.t(), b, a)
    assert ((m.u[:live].double() - u).abs() <= ur + ref.half_step(u, torch.float32)).all()
    assert ((y[:live].double() - y64).abs() <= yr + ref.half_step(y64, BF) * 1.01).all()
    assert ((dx[:live].double() - dx64).abs() <= dxr + ref.half_step(dx64, BF) * 1.01).all()
    k = ref.PAIR + 2 * ref.chain(310) + 64 * ref.STEP
    for p, pr, q, got in ((v, vr, x, da), (u, ur, dy, db)):
        q = q[:live].double()
        terms = torch.einsum("tr,tk->trk", p * has, q)
        want = torch.zeros(got.shape, dtype=torch.float64, device=DEV).index_add_(0, e, terms)
        terms = torch.einsum("tr,tk->trk", (pr + p.abs() * k) * has, q.abs())
        room = torch.zeros(got.shape, dtype=torch.float64, device=DEV).index_add_(0, e, terms)
        assert ((got.double() - want).abs() <= room).all()
