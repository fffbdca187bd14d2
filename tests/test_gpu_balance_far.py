"""Balance loss and gradient of finite logits far from zero, of any size.

Tolerances are those of test_gpu_balance.  Its P holds for rows near zero in the form
2^(z log2 e - c), c = fl(m log2 e) for the row's maximum m: an exponent -x (x <= 24 where
z - m >= -16) rounds once (2^-24 x), log2 e is off by 2^-25 of itself (2^-25 x) and c's
rounding is a factor that every term of the row and their sum share, 2^(ulp(c) / 2) at most,
harmless while it is near one.  Together ln 2 * 24 * 1.5 * 2^-24 + 2^-22 + 24 * 2^-24 = 3.2e-6.
Where m is too large for that, e^(z - m) has z - m exact (z and m within a factor of two, or
one of them beyond where the term is 0) and the same roundings after it."""
import pytest
import torch

import test_gpu_balance as near

pytestmark = pytest.mark.gpu
DEV = near.DEV
LEVELS = [2.0 ** 19, 1e6, 2.0 ** 20, 2.0 ** 21, 1.7e7, 2.0 ** 30, 3e9, 5e9, 1.1e10, 2.0 ** 35, 1e20,
          1e30, 9.9e37, 1.1e38, 3.3e38]


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def rows(E, sigmoid):
    """Per level and sign: a row filled with it, one near it, one with it in one place and one
    with it everywhere but there; ordinary rows between them."""
    gen = torch.Generator(device=DEV).manual_seed(E)
    rnd = lambda: torch.randn((E,), generator=gen, device=DEV)  # noqa: E731
    out = []
    for i, level in enumerate(LEVELS):
        for sign in (1.0, -1.0):
            v = sign * level
            one, but = rnd(), torch.full((E,), v, device=DEV)
            one[i % E] = v
            but[i % E] = 0.5
            out += [one, rnd(), but]
            if sign > 0 or not sigmoid:  # (a sum of sigmas that far below zero is 0 in 64 bits)
                out += [torch.full((E,), v, device=DEV), rnd(), v + 4 * rnd()]
    return torch.stack(out)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k", [(6, 2), (8, 2), (16, 4), (31, 3), (40, 4), (100, 6), (150, 3),
                                 (192, 8), (256, 8), (300, 8), (384, 8), (385, 8), (509, 16)])
def test_finite_logits_of_any_size(E, k, sigmoid):
    z = rows(E, sigmoid)
    assert torch.isfinite(z).all()
    T = z.shape[0]
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k]
                       for t in range(T)]).to(torch.int32).to(DEV)
    for off in (list(range(T + 1)), None):  # a token a sequence, and all together
        o = near.run(z, ids, None, None, off, sigmoid)
        assert int(o["st"].item()) == 0
        near.check(z, ids, None, None, off, sigmoid, o)


def test_a_batch_of_mask_constants():
    """Many tokens a block, so that several of them share a warp or follow one another in it."""
    for E in (16, 384):
        z = torch.full((5000, E), -1e30, device=DEV)
        z[::3, 5] = 0.25
        z[1::7] = -1e10
        ids = torch.tensor([5, 1], dtype=torch.int32, device=DEV).repeat(5000, 1)
        o = near.run(z, ids, None, None, None, False)
        near.check(z, ids, None, None, None, False, o)


@pytest.mark.parametrize("E", [8, 300])
def test_every_row_sums_to_one(E):
    """Maxima over the whole range of the type, both signs: a uniform row is 1 / E."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    top = torch.exp2(128 * torch.rand((20000, 1), generator=gen, device=DEV) - 0.01).clamp(max=3.4e38)
    z = (top * torch.where(torch.rand((20000, 1), generator=gen, device=DEV) < 0.5, -1.0, 1.0)).expand(-1, E)
    ids = torch.zeros((20000, 1), dtype=torch.int32, device=DEV)
    o = near.run(z.contiguous(), ids, None, None, [0] + list(range(1, 20001)), False) \
        if E == 8 else near.run(z.contiguous(), ids, None, None, None, False)
    assert (o["probs"] - 1.0 / E).abs().max() <= (near.P + 80 * 2.0 ** -24) / E
    assert torch.isfinite(o["dz"]).all()
