"""moe_clip_grads at the edges of its arithmetic: the longest chain of fp32 roundings, and a limit
that is infinite."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def G():
    import grouped_expert_gemm_gb300 as g
    return g


@pytest.mark.parametrize("kind", [BF, F32])
def test_norm_where_every_rounding_loses(kind):
    """A thread's squares go through 12 roundings of fp32 at most, each off by 2^-24 of its sum: half
    of that in the norm, and its own rounding, make 8 * 2^-24 with room.  Here each thread has a
    one whose sum every later square of 2^-24, half a last bit, is added to in vain: 32 KB of a tensor
    to a block at a time, 16-byte vectors i of thread t at 256 i + t."""
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    blocks = min(2 * sms, 1024)
    per = 16 // (2 if kind is BF else 4)  # values of a vector
    x = torch.zeros((blocks, 8, 256, per), device=DEV)
    small = 2.0 ** -12
    n = 256  # blocks whose threads hold values: 2^16 threads, whose norm is 2^8 without the small ones
    assert blocks >= n
    x[:n, :, :, 0] = small
    x[:n, 0, :, 0] = 1.0
    if kind is BF:
        x[:n, :, :, 4] = small
    x[:n, 0, :, 1] = small
    x[:n, 0, :, 2] = small
    g = x.view(-1).to(kind)
    assert torch.equal(g.float(), x.view(-1))
    want = float(g.double().square().sum().sqrt())
    norm = float(G().GradientClip([g], math.inf, device=DEV).clip())
    assert abs(norm - want) <= want * 8 * 2.0 ** -24


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", [F32, BF])
@pytest.mark.parametrize("bad", [math.inf, math.nan, None])
def test_infinite_limit_scales_nothing(bad, kind, in_place):
    """Norms alone are asked for: also where one is not finite, for an element's sake or because the
    norm of finite values passes fp32's range, every value stays what it was."""
    gen = torch.Generator(device=DEV).manual_seed(0)
    grads = [torch.randn(c, generator=gen, device=DEV).to(kind) for c in (100, 9000, 300)]
    if bad is None:
        grads[1].fill_(1e37)  # norm 9.5e38
    else:
        grads[1][8500] = bad
    before = [x.clone() for x in grads]
    out = None if in_place else [torch.zeros_like(x) for x in grads]
    clip = G().GradientClip(grads, math.inf, out=out, groups=[0, 1, 2], device=DEV)
    norms = clip.clip()
    bits = lambda t: t.view(torch.int32 if kind is F32 else torch.int16)  # noqa: E731
    for got, want in zip(clip.out, before):
        if bad is not None and math.isnan(bad):
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            keep = ~torch.isnan(want)
            assert torch.equal(got[keep], want[keep])
        else:
            assert torch.equal(bits(got), bits(want))
    assert torch.isfinite(norms[[0, 2]]).all() and not torch.isfinite(norms[1])
    assert int(clip.dev_status.item()) == G().MOE_DEV_NONFINITE_INPUT
