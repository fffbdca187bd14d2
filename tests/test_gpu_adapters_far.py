"""The projection with adapters and clipping where offsets pass 32 bits: rows gigabytes apart, a
table of many adapters, a tensor of more than 2^31 elements."""
import pytest
import torch

import adapter_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def G():
    import grouped_expert_gemm_gb300 as g
    return g


def test_rows_far_apart():
    g = G()
    T, d, n, r, N, far = 4, 72, 136, 16, 2, (1 << 30) + 64
    gen = torch.Generator(device=DEV).manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    x = torch.empty(((T - 1) * far + d,), dtype=BF, device=DEV).as_strided((T, d), (far, 1))
    y = torch.empty(((T - 1) * far + n,), dtype=BF, device=DEV).as_strided((T, n), (far, 1))
    x.copy_(rnd(T, d))
    w, a, b = rnd(d, n).to(BF), rnd(N, r, d).to(BF), rnd(N, r, n).to(BF)
    m = g.AdapterProjection(T, w, a, b, torch.ones(N, device=DEV), device=DEV)
    off = torch.tensor([0, 1, 4], dtype=torch.int32, device=DEV)
    ids = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    near = m.forward(x.contiguous(), ids, off).clone()
    assert torch.equal(m.forward(x, ids, off, out=y), near)
    dy = rnd(T, n).to(BF)
    want = [t.clone() for t in m.backward(dy)]
    y.copy_(dy)
    for p, q in zip(want, m.backward(y)):
        assert torch.equal(p, q)


def test_tables_beyond_two_giga_elements():
    g = G()
    T, d, n, r, N = 40, 8, 65536, 128, 300  # b: 2.5e9 elements
    gen = torch.Generator(device=DEV).manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    x, w, a = rnd(T, d).to(BF), rnd(d, n).to(BF), rnd(N, r, d).to(BF)
    b = torch.zeros((N, r, n), dtype=BF, device=DEV)
    b[N - 1] = rnd(r, n).to(BF)
    b[270] = rnd(r, n).to(BF)
    s = torch.ones(N, device=DEV)
    for off, ids in (([0, 40], [N - 1]), (list(range(41)), [N - 1, 270] * 20)):
        u = torch.empty((T, r), device=DEV)
        y = torch.empty((T, n), dtype=BF, device=DEV)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        g.moe_adapter_project(g.AdapterParams(T, d, n, r, N, len(ids)), i32(off), i32(ids), x, w, a, b,
                              s, u, y)
        segs = ref.segments(off, [1 if e == N - 1 else 0 for e in ids], T)
        pick = lambda t: torch.stack([t[270], t[N - 1]])  # noqa: E731
        u64, ur, y64, yr = ref.forward(x, w, pick(a), pick(b), s[:2], segs)
        assert ((u.double() - u64).abs() <= ur + ref.half_step(u64, torch.float32)).all()
        assert ((y.double() - y64).abs() <= yr + ref.half_step(y64, BF) * 1.01).all()


def test_clip_a_tensor_beyond_two_giga_elements():
    g = G()
    big = torch.zeros(((1 << 31) + 12345,), dtype=BF, device=DEV)
    big[5], big[-1], big[1 << 31] = 3.0, 4.0, 12.0
    small = torch.full((3,), 2.0, device=DEV)
    norms = g.GradientClip([big, small], 1.0, groups=[0, 1], device=DEV).clip()
    assert norms[0].item() == 13.0 and abs(norms[1].item() - 12 ** 0.5) <= 12 ** 0.5 * 2.0 ** -21
    for at, v in ((5, 3.0), (-1, 4.0), (1 << 31, 12.0)):
        assert abs(big[at].item() - v / 13) <= v / 13 * 2.0 ** -8
    assert int((big != 0).sum()) == 3
