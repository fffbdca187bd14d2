"""moe_clip_grads against its definition in 64 bits.

Tolerances: 32 squares in fp32 in four chains of eight (12 roundings at most, 2^-24 each), the
rest in fp64, half of the error in the norm, and its rounding: 8 * 2^-24.  The factor adds the
sum with 1e-6, a division, and its rounding (3 more); the product and the tensor's type one
rounding each."""
import math

import pytest
import torch

import adapter_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
NORM = 8 * 2.0 ** -24
FACTOR = NORM + 4 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def G():
    import grouped_expert_gemm_gb300 as g
    return g


def make(counts, types, seed=0, offset=0, level=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn((c + offset,), generator=gen, device=DEV) * level).to(t)[offset:]
            for c, t in zip(counts, types)]


def check(grads, groups, n_groups, max_norm, in_place, shift=0):
    g = G()
    before = [x.clone() for x in grads]
    out = None
    if not in_place:
        out = [torch.full((x.numel() + shift,), -7.0, device=DEV, dtype=x.dtype)[shift:].view(x.shape)
               for x in grads]
    clip = g.GradientClip(grads, max_norm, out=out, groups=groups, n_groups=n_groups, device=DEV)
    norms = clip.clip()
    n64, o64 = ref.clip(before, groups, n_groups, max_norm)
    if n_groups == 1 and float(n64[0]) >= 2.0 ** 128:
        # 3e37 / 4 * sqrt(9050) = 7.1e38: norms [n_groups] is fp32, whose largest value is
        # 3.4e38, so the norm is infinite and the formula's factor is zero
        assert int(clip.dev_status.item()) == g.MOE_DEV_NONFINITE_INPUT
        assert math.isinf(float(norms)) and all((t == 0).all() for t in clip.out)
        return clip
    assert int(clip.dev_status.item()) == 0
    for a, b in zip(norms.tolist(), n64):
        assert abs(a - float(b)) <= float(b) * NORM + 1e-45
    for got, want, old in zip(clip.out, o64, before):
        room = want.abs() * (FACTOR + 2.0 ** -24) + ref.half_step(want, got.dtype) * 1.001 + 1e-45
        if got.dtype is BF:
            room += 2.0 ** -134  # half a step below the normal range
        assert ((got.double() - want).abs() <= room).all()
    if not in_place:
        for x, old in zip(grads, before):
            assert torch.equal(x, old)
    return clip


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("counts,groups,n_groups", [
    ([1], [0], 1), ([7, 8, 9], [0, 0, 0], 1), ([8191, 8192, 8193, 1, 20000], [0] * 5, 1),
    ([5000] * 40, [i // 2 for i in range(40)], 20),
    ([30000, 0, 17, 0], [2, 0, 2, 4], 6),                      # empty tensors and groups, unordered
    ([3] * 700, [i % 70 for i in range(700)], 70),
    ([9_000_001, 3, 1_000_000], [0, 1, 1], 2),
])
@pytest.mark.parametrize("types", [(F32,), (BF,), (BF, F32, F32)])
def test_clip(counts, groups, n_groups, types, in_place):
    kinds = [types[i % len(types)] for i in range(len(counts))]
    grads = make(counts, kinds, seed=len(counts))
    check(grads, groups, n_groups, 3.0, in_place)


@pytest.mark.parametrize("kind", [F32, BF])
@pytest.mark.parametrize("offset,shift", [(1, 0), (3, 3), (0, 1), (5, 2)])
def test_odd_addresses(kind, offset, shift):
    grads = make([1, 2, 100, 8192, 16389], [kind] * 5, seed=2, offset=offset)
    check(grads, [0] * 5, 1, 0.5, False, shift)
    check(grads, [0] * 5, 1, 0.5, True)


def test_neighbours_of_a_tensor_stay():
    for kind in (F32, BF):
        flat = torch.full((3000,), -7.0, device=DEV, dtype=kind)
        out = flat.clone()
        g = G()
        g.GradientClip([flat[3:1001], flat[1005:2003]], 0.1, out=[out[3:1001], out[1005:2003]],
                       device=DEV).clip()
        keep = torch.ones(3000, dtype=torch.bool, device=DEV)
        keep[3:1001] = False
        keep[1005:2003] = False
        assert (out[keep] == -7).all() and (out[~keep] > -7).all()


@pytest.mark.parametrize("level", [1e-30, 1e-18, 1e-3, 1e18, 1e30, 3e37])
@pytest.mark.parametrize("kind", [F32, BF])
def test_range_of_fp32(level, kind):
    """Values whose squares leave fp32's range still have their norm."""
    grads = make([50, 9000], [kind] * 2, seed=3, level=level / 4)
    check(grads, [0, 0], 1, level, False)


def test_small_norms_in_place_are_left_alone():
    grads = make([1000, 77], [F32, BF], seed=4, level=1e-3)
    before = [x.clone() for x in grads]
    clip = check(grads, [0, 1], 2, 1.0, True)
    assert all(torch.equal(a, b) for a, b in zip(clip.out, before))
    zeros = [torch.zeros(5, device=DEV), torch.zeros(0, device=DEV)]
    clip = G().GradientClip(zeros, 1.0, groups=[0, 1], device=DEV)
    assert clip.clip().tolist() == [0.0, 0.0] and (zeros[0] == 0).all()
    assert G().GradientClip([], 1.0, n_groups=3, device=DEV).clip().tolist() == [0.0] * 3


def test_infinite_limit_keeps_the_values():
    grads = make([5000], [F32], seed=6, level=1e3)
    out = [torch.empty_like(grads[0])]
    clip = G().GradientClip(grads, math.inf, out=out, device=DEV)
    n64, _ = ref.clip(grads, [0], 1, 1.0)
    assert abs(float(clip.clip()) - float(n64[0])) <= float(n64[0]) * NORM
    assert torch.equal(out[0], grads[0])


def test_values_that_are_not_finite():
    """The formula is followed, in the group that holds them alone."""
    g = G()
    for bad, own in ((math.nan, "nan"), (math.inf, "inf")):
        grads = make([100, 9000, 300], [F32, BF, F32], seed=5)
        keep = [x.clone() for x in grads]
        grads[1][8500] = bad
        clip = g.GradientClip(grads, 1.0, groups=[0, 1, 2], device=DEV)
        norms = clip.clip()
        assert int(clip.dev_status.item()) == g.MOE_DEV_NONFINITE_INPUT
        _, want = ref.clip([keep[0], keep[2]], [0, 1], 2, 1.0)
        for got, w in zip((grads[0], grads[2]), want):
            assert ((got.double() - w).abs() <= w.abs() * 1e-6).all()
        if own == "nan":
            assert torch.isnan(norms[1]) and torch.isnan(grads[1].float()).all()
        else:
            assert torch.isinf(norms[1]) and torch.isnan(grads[1][8500].float())
            rest = torch.cat([grads[1][:8500], grads[1][8501:]])
            assert (rest == 0).all()


def test_same_bits_captured_and_on_another_stream():
    g = G()
    grads = make([100_000, 31, 2_000_000, 5], [F32, BF, BF, F32], seed=7)
    new = lambda: [torch.empty_like(x) for x in grads]  # noqa: E731
    first = g.GradientClip(grads, 1.0, out=new(), groups=[0, 1, 1, 0], device=DEV)
    first.clip()
    side = torch.cuda.Stream()
    second = g.GradientClip(grads, 1.0, out=new(), groups=[0, 1, 1, 0], device=DEV)
    torch.cuda.synchronize()
    second.clip(stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    third = g.GradientClip(grads, 1.0, out=new(), groups=[0, 1, 1, 0], device=DEV)
    with torch.cuda.graph(graph):
        third.clip()
    graph.replay()
    torch.cuda.synchronize()
    for other in (second, third):
        assert torch.equal(first.norms, other.norms)
        assert all(torch.equal(a, b) for a, b in zip(first.out, other.out))
