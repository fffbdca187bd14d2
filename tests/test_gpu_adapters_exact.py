"""How exact the adapters' fp32 numbers are: sums of long reductions, u and v in products.

Limits for sums, relative to the norm of the result, of zero-mean random terms.  A tensor-core
step adds 16 products and is off by at most one last bit, 2^-23, of the sum so far, whose size
after i of n steps is sqrt(i / n) of the whole: sum over a piece of n steps is (2 n / 3 + 1) 2^-23 of the
piece.  Pieces are independent, so their errors add up as the pieces do, in squares, and the
relative bound is a piece's own.  Each of J fp32 additions that join pieces is off by 2^-24 of the sum so
far, independently: sqrt(J) 2^-24 at most.  An unbroken sum of 7,168 or more, or of 4,096 tokens,
has measured errors of 7e-6 and more; every limit here is below 3.5e-6."""
import pytest
import torch

import adapter_reference as ref
from test_gpu_adapters import DEV, G, i32, make, project, project_backward

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def limit(steps, joins, more=0):
    """Pieces of `steps` steps, `joins` additions of pieces, `more` single roundings."""
    return (2 * steps / 3 + 1) * 2.0 ** -23 + (joins ** 0.5 + more) * 2.0 ** -24


def off_by(got, want):
    want = want.double()
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("T,K,r", [(600, 7168, 16), (300, 16384, 128), (2000, 8192, 40)])
def test_u_of_long_segments(T, K, r):
    """Pieces of 256 values (16 steps), K / 256 joins, the scale."""
    x, w, a, b, scale, _ = make(T, K, 64, r, 2, seed=K)
    u, _, _ = project((x, w, a, b, scale), [0, T // 3, T], [1, 0])
    for rows, e in ((slice(0, T // 3), 1), (slice(T // 3, T), 0)):
        want = x[rows].double() @ a[e].double().T * scale[e].double()
        assert off_by(u[rows], want) <= limit(16, K / 256, 1)


@pytest.mark.parametrize("T,n", [(40, 256), (200, 256), (200, 4096), (1000, 264)])
def test_fp32_results(T, n):
    """Pieces of 512 values (32 steps) and their joins, no adapter's part."""
    K = 16384
    x, w, a, b, scale, _ = make(T, K, n, 8, 1, seed=T + n)
    _, y, _ = project((x, w, a, b, scale), None, [-1], F32)
    assert off_by(y, x.double() @ w.double()) <= limit(32, K / 512, 1)


@pytest.mark.parametrize("r", [8, 24, 64, 128])
def test_gradients_of_many_tokens(r):
    """Pieces of 128 tokens in two halves: four steps of a half's values, then eight with what
    rounding left of them, which cut a sum that no longer grows.  Sizes of the sum at the 24 steps,
    relative to the last one: sqrt(i / 8) for i = 1 to 4, 8 sqrt(4 / 8), sqrt(i / 8) for i = 5 to 8, 8: 19.4 together,
    as 28 steps of a sum that grows.  At most T / 128 + 8 joins.  Against the products of the kernels'
    own u and v, so that nothing but the sums is looked at."""
    T, d, n = 4096, 264, 520
    x, w, a, b, scale, rnd = make(T, d, n, r, 2, seed=r)
    dy = rnd(T, n).to(BF)
    t, off, ids = (x, w, a, b, scale), [0, 96, T], [1, 0]
    u, _, _ = project(t, off, ids)
    _, da, db = project_backward(t, off, ids, u, dy)
    # v: the same rows against the tables turned around
    v, _, _ = project((dy, w.t().contiguous(), b, a, scale), off, ids)
    rows = slice(96, T)
    room = limit(28, T / 128 + 8, 1)
    assert off_by(da[0], v[rows].double().T @ x[rows].double()) <= room
    assert off_by(db[0], u[rows].double().T @ dy[rows].double()) <= room


# 1 + 2^-9 + 2^-17: its bf16 value is 1, what that left rounds to 2^-9, and 2^-17 is left of it
LONG = 1.0 + 2.0 ** -9 + 2.0 ** -17


def exact_u(T, d, n, r, N):
    """Inputs whose u is scale[e] in every rank: one value of a row, times ones."""
    x, w, a, b, scale, rnd = make(T, d, n, r, N, seed=T + r)
    x.zero_()
    x[:, 5] = 1.0
    a[:, :, 5] = 1.0
    w.zero_()
    scale[:] = LONG * 2.0 ** torch.arange(N, device=DEV).float()
    keep = torch.zeros_like(b)
    keep[:, 3] = b[:, 3]  # one rank: y is one product
    return x, w, a, keep, scale, rnd


@pytest.mark.parametrize("T,off,ids", [
    (1, [0, 1], [1]), (40, [0, 40], [2]), (40, [0, 10, 40], [0, 2]),         # whole, few runs
    (64, list(range(65)), [q % 3 for q in range(64)]),                       # many runs
    (300, [0, 300], [1]), (300, [0, 100, 110, 300], [1, -1, 2]),
    (300, list(range(40)) + [300], [q % 3 for q in range(40)])])
@pytest.mark.parametrize("r", [8, 24, 40, 128])
def test_all_of_u_enters_fp32_results(T, off, ids, r):
    """y is one product u b: three parts of u, each added exactly or cut by one last bit."""
    d, n = 72, 136
    x, w, a, b, scale, _ = exact_u(T, d, n, r, 3)
    u, y, _ = project((x, w, a, b, scale), off, ids, F32)
    for p, q, e in ref.segments(off, ids, T):
        if e < 0:
            assert not y[p:q].any()
            continue
        assert (u[p:q] == scale[e]).all()
        want = scale[e].double() * b[e, 3].double()
        assert ((y[p:q].double() - want).abs() <= 4 * 2.0 ** -23 * want.abs()).all()


@pytest.mark.parametrize("r", [8, 24, 64, 128])
def test_all_of_u_and_v_enters_the_gradients(r):
    """One token: db = u^T dy and da = v^T x are single products."""
    T, d, n = 3, 72, 136
    x, w, a, b, scale, rnd = exact_u(T, d, n, r, 3)
    off, ids = [0, 1, 2, 3], [2, 0, 1]
    dy = torch.zeros((T, n), dtype=BF, device=DEV)
    dy[:, 7] = 1.0
    b.zero_()
    b[:, :, 7] = 1.0  # v is scale[e] too
    t = (x, w, a, b, scale)
    u, _, _ = project(t, off, ids)
    x2 = rnd(T, d).to(BF)
    dx, da, db = project_backward((x2, *t[1:]), off, ids, u, dy)
    for q, e in enumerate(ids):
        want = scale[e].double() * x2[q].double()
        assert ((da[e].double() - want).abs() <= 4 * 2.0 ** -23 * want.abs()).all()
        want = scale[e].double() * dy[q].double()
        assert ((db[e].double() - want).abs() <= 4 * 2.0 ** -23 * want.abs()).all()
