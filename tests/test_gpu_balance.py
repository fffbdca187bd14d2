"""moe_balance_loss and moe_route_backward against their definition in 64 bits.

Tolerances (fp32, 2^-24 per rounding): an exponential e^x is taken as 2^(x log2 e),
whose argument rounds twice (2^-23 |x|, and |x| <= 16 for these logits below their
row's maximum) and whose instruction errs by 2^-22; the row's sum of positive terms
has at most 16 + 5 roundings, the division and the products three more.  Together
16 * 2^-23 + 2^-22 + 24 * 2^-24 = 3.6e-6 < P = 4e-6 of a probability.  A column's sum adds
at most ceil(tile / 16) + 16 + ceil(slots / 16) + 16 roundings of the sum of
(positive) terms.  A gradient p (w - <p, w>) errs by that of p times |w| +
<p, |w|>."""
import pytest
import torch

import operator_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
P = 4e-6
ALPHA = 0.02


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def G():
    import grouped_expert_gemm_gb300 as g
    return g


def make(T, E, k, sigmoid, seed, pad=0.0, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    z = scale * (torch.randn((T, E), generator=gen, device=DEV)
                 + 0.5 * torch.randn((E,), generator=gen, device=DEV))
    top = (torch.sigmoid(z) if sigmoid else z).topk(k, dim=1)
    gates = 2.5 * top.values / top.values.sum(1, keepdim=True) if sigmoid else top.values.softmax(1)
    ids = top.indices.to(torch.int32)
    masked = torch.rand((T,), generator=gen, device=DEV) < pad
    ids[masked], gates[masked] = -1, 0.0
    dg = torch.randn((T, k), generator=gen, device=DEV) / max(T, 1)
    return z, ids.contiguous(), gates.contiguous(), dg


def run(z, ids, gates, dg, off, sigmoid, dloss=None, balance=True, stream=None):
    g = G()
    T, E = z.shape
    k = ids.shape[1]
    S = 1 if off is None else len(off) - 1
    offs = None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)
    p = g.RouteParams(T, E, k, g.MOE_SCORE_SIGMOID_GROUP if sigmoid else g.MOE_SCORE_SOFTMAX, 1, 1, 2.5)
    o = dict(counts=torch.full((S, E), -7, dtype=torch.int32, device=DEV),
             tokens=torch.full((S + 1,), -7, dtype=torch.int32, device=DEV),
             probs=torch.full((S, E), -7.0, device=DEV), loss=torch.full((1,), -7.0, device=DEV),
             dz=torch.full((T, E), -7.0, device=DEV), st=torch.zeros(1, dtype=torch.int32, device=DEV))
    nb = g.moe_balance_loss_workspace_size(p, S)
    ws = torch.full((nb,), 0x7F, dtype=torch.uint8, device=DEV)
    g.moe_balance_loss(p, S, offs, z, ids, ALPHA, o["counts"], o["tokens"], o["probs"], o["loss"], ws,
                       nb, o["st"], stream)
    d = None if dloss is None else torch.tensor([dloss], device=DEV)
    g.moe_route_backward(p, S, offs, z, ids, gates, dg, ALPHA, o["counts"] if balance else None,
                         o["tokens"] if balance else None, d, o["dz"], o["st"], stream)
    torch.cuda.synchronize()
    return o


def check(z, ids, gates, dg, off, sigmoid, o, dloss=1.0):
    T, E = z.shape
    k = ids.shape[1]
    off = [0, T] if off is None else off
    counts, tokens, mean, loss = ref.balance(z, ids, off, ALPHA, E, k, sigmoid)
    assert torch.equal(o["counts"].cpu().long(), counts.cpu())
    assert torch.equal(o["tokens"].cpu().long(), tokens)
    chain = P + (-(-T // 304) + 16 + 60 + 16) * 2.0 ** -24
    assert ((o["probs"].double() - mean).abs() <= chain * mean + 1e-30).all()
    assert (o["loss"].double().cpu() - loss.cpu()).abs() <= (chain + 2.0 ** -23) * loss.cpu().abs()
    bal = ref.balance_grad(z, ids, off, ALPHA, dloss, E, k, sigmoid)
    want, room = bal, torch.zeros_like(bal)
    p, _ = ref.probs(z, sigmoid)
    used = max(int(tokens[-1]), 1)
    for q, (a, b) in enumerate(zip(off[:-1], off[1:])):
        n = max(int(tokens[q]), 1)
        w = abs(dloss) * ALPHA / used * E / (k * n) * counts[q].double().to(z.device) / n
        room[a:b] = 4 * P * p[a:b] * (w + (p[a:b] @ w)[:, None])
    if dg is not None:
        want = want + ref.gate_grad(z, ids, gates, dg, sigmoid, 2.5)
        gd = (gates * dg).abs().double()
        at = ids.long().clamp(min=0)
        size = gates.double() * (dg.abs().double() + gd.sum(1, keepdim=True))
        room = room.scatter_add(1, at, 4 * P * size)
    assert ((o["dz"].double() - want).abs() <= room + want.abs() * 2.0 ** -22 + 1e-30).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 2, 1), (3, 8, 8), (256, 8, 2), (130, 31, 5), (77, 33, 16),
                                   (1000, 100, 6), (611, 128, 8), (5000, 129, 3), (999, 256, 8),
                                   (1500, 300, 8), (777, 384, 8), (650, 509, 16), (333, 512, 1)])
def test_one_sequence(T, E, k, sigmoid):
    z, ids, gates, dg = make(T, E, k, sigmoid, seed=T + E)
    o = run(z, ids, gates, dg, None, sigmoid)
    check(z, ids, gates, dg, None, sigmoid, o)
    assert int(o["st"].item()) == 0


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("off", [[0, 0, 1, 1, 700, 700], [0, 699, 700], [0] + list(range(0, 701)) + [700],
                                 [13, 13, 40, 512], [700, 700]])
def test_ragged_sequences_with_padding(off, sigmoid):
    z, ids, gates, dg = make(700, 64, 4, sigmoid, seed=9, pad=0.2)
    o = run(z, ids, gates, dg, off, sigmoid, dloss=-0.75)
    check(z, ids, gates, dg, off, sigmoid, o, dloss=-0.75)
    assert int(o["st"].item()) == 0


def test_nothing_live():
    z, ids, gates, dg = make(40, 16, 2, False, seed=1, pad=2.0)
    o = run(z, ids, gates, dg, [0, 20, 40], False)
    assert (o["counts"] == 0).all() and (o["tokens"] == 0).all() and (o["dz"] == 0).all()
    assert float(o["loss"]) == 0 and (o["probs"] == 0).all()


def test_no_tokens():
    z, ids, gates, dg = make(0, 16, 2, False, seed=1)
    o = run(z, ids, gates, dg, None, False)
    assert (o["counts"] == 0).all() and float(o["loss"]) == 0 and (o["probs"] == 0).all()


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gates_alone_and_loss_alone(sigmoid):
    z, ids, gates, dg = make(300, 48, 4, sigmoid, seed=4)
    o = run(z, ids, gates, dg, None, sigmoid, balance=False)
    want = ref.gate_grad(z, ids, gates, dg, sigmoid, 2.5)
    assert ((o["dz"].double() - want).abs() <= 2e-5 * gates.abs().max() * dg.abs().max()).all()
    o = run(z, ids, gates, None, None, sigmoid)
    check(z, ids, gates, None, None, sigmoid, o)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("shift", [-300.0, -90.0, 300.0])
def test_far_logits(sigmoid, shift):
    """All logits far from zero: the sums neither underflow nor overflow.  (z + shift is
    rounded to fp32 before either side sees it.)"""
    z, ids, gates, dg = make(64, 40, 4, sigmoid, seed=6)
    z = z + shift
    o = run(z, ids, gates, None, None, sigmoid)
    if sigmoid and shift < 0:  # the definition's own sum underflows in 64 bits only below -700
        assert torch.isfinite(o["dz"]).all()
    check(z, ids, gates, None, None, sigmoid, o)


def test_masked_and_nonfinite_logits():
    z, ids, gates, dg = make(32, 24, 2, False, seed=7)
    z[3, 5] = float("-inf")  # a masked expert: probability 0, nothing reported
    z[4, :] = torch.finfo(torch.float32).min  # the type's lowest value in every place: uniform
    o = run(z, ids, gates, None, None, False)
    assert int(o["st"].item()) == 0
    check(z, ids, gates, None, None, False, o)
    assert float(o["dz"][3, 5]) == 0
    for sigmoid in (False, True):
        z2 = z.clone()
        z2[6, 1], z2[7, 2], z2[8, :] = float("nan"), float("inf"), float("-inf")
        o2 = run(z2, ids, gates, None, None, sigmoid)
        assert int(o2["st"].item()) == G().MOE_DEV_NONFINITE_LOGIT
        assert torch.isfinite(o2["dz"]).all() and torch.isfinite(o2["loss"]).all()
        assert (o2["dz"][8] == 0).all() and float(o2["dz"][6, 1]) == 0


def test_bad_ids_and_offsets_are_reported():
    z, ids, gates, dg = make(50, 16, 2, False, seed=3)
    ids[9, 1] = 16
    o = run(z, ids, gates, dg, None, False)
    assert int(o["st"].item()) == G().MOE_DEV_BAD_EXPERT_ID
    assert int(o["counts"].sum()) == 99
    z, ids, gates, dg = make(50, 16, 2, False, seed=3)
    for off in ([0, 30, 20, 50], [0, 51], [-1, 50]):
        o = run(z, ids, gates, dg, off, False)
        assert int(o["st"].item()) == G().MOE_DEV_BAD_MAP


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gradient_against_differences(sigmoid):
    """The loss (its counts held) and the gates, differenced in 64 bits."""
    z, ids, gates, dg = make(60, 20, 3, sigmoid, seed=12)
    off = [0, 25, 60]
    o = run(z, ids, gates, dg, off, sigmoid)

    def value(zz):
        _, _, _, loss = ref.balance(zz, ids, off, ALPHA, 20, 3, sigmoid)
        s = zz.gather(1, ids.long())
        g = torch.sigmoid(s) * 2.5 / torch.sigmoid(s).sum(1, keepdim=True) if sigmoid else s.softmax(1)
        return loss + (g * dg.double()).sum()

    gen = torch.Generator(device=DEV).manual_seed(1)
    for _ in range(4):
        a = torch.randn(z.shape, generator=gen, device=DEV).double()
        t = 1e-4
        num = (value(z.double() + t * a) - value(z.double() - t * a)) / (2 * t)
        got = (o["dz"].double() * a).sum()
        assert (num - got).abs() <= 2e-5 * (o["dz"].double() * a).abs().sum()


def test_same_bits_on_every_run_and_from_a_graph():
    z, ids, gates, dg = make(4000, 96, 6, True, seed=5, pad=0.1)
    off = [0, 1000, 1000, 2500, 4000]
    a = run(z, ids, gates, dg, off, True)
    b = run(z, ids, gates, dg, off, True)
    for k in ("counts", "tokens", "probs", "loss", "dz"):
        assert torch.equal(a[k], b[k])
    g = G()
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    p = g.RouteParams(4000, 96, 6, g.MOE_SCORE_SIGMOID_GROUP, 1, 1, 2.5)
    nb = g.moe_balance_loss_workspace_size(p, 4)
    ws = torch.empty((nb,), dtype=torch.uint8, device=DEV)
    for k in ("counts", "tokens", "probs", "loss", "dz"):
        b[k].fill_(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.moe_balance_loss(p, 4, offs, z, ids, ALPHA, b["counts"], b["tokens"], b["probs"], b["loss"],
                           ws, nb)
        g.moe_route_backward(p, 4, offs, z, ids, gates, dg, ALPHA, b["counts"], b["tokens"], None,
                             b["dz"])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for k in ("counts", "tokens", "probs", "loss", "dz"):
        assert torch.equal(a[k], b[k])


def test_unaligned_rows_take_the_narrow_loads():
    z, ids, gates, dg = make(200, 64, 4, False, seed=21)
    buf = torch.empty(200 * 64 + 1, device=DEV)
    zo = buf[1:].view(200, 64)
    zo.copy_(z)
    o = run(zo, ids, gates, dg, None, False)
    check(z, ids, gates, dg, None, False, o)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_a_repeated_id_sums_its_slots(sigmoid):
    z, ids, gates, dg = make(40, 16, 4, sigmoid, seed=13)
    ids[5] = torch.tensor([3, 3, 3, 9], dtype=torch.int32)
    ids[6] = 7
    o = run(z, ids, gates, dg, None, sigmoid, balance=False)
    want = ref.gate_grad(z, ids, gates, dg, sigmoid, 2.5)
    assert ((o["dz"].double() - want).abs() <= 2e-5 * gates.abs().max() * dg.abs().max()).all()


SIDE_BY_SIDE = [(4, 2), (8, 8), (12, 3), (16, 16), (20, 5), (32, 16), (36, 7), (64, 16), (68, 4),
                (128, 8), (132, 16), (192, 8), (6, 6), (13, 13)]


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k", SIDE_BY_SIDE)
def test_several_tokens_a_warp(E, k, sigmoid):
    for T in (1, 37, 1500):
        z, ids, gates, dg = make(T, E, k, sigmoid, seed=T + E, pad=0.2)
        for off in (None, [0, min(5, T), min(5, T), T // 2 + 1, T] if T > 9 else [0, 0, T]):
            o = run(z, ids, gates, dg, off, sigmoid, dloss=1.5)
            check(z, ids, gates, dg, off, sigmoid, o, dloss=1.5)
            assert int(o["st"].item()) == 0


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k", [(8, 2), (16, 4), (24, 9), (48, 4), (100, 6), (160, 8), (7, 3)])
def test_nonfinite_logits_beside_other_tokens(E, k, sigmoid):
    """NaN counts as -inf and +inf as the largest finite value; in padding tokens neither is
    reported; the tokens beside them in the warp are as without."""
    z, ids, gates, dg = make(90, E, k, sigmoid, seed=E, pad=0.3)
    pad = ids[:, 0] == -1
    z2 = z.clone()
    z2[pad] = float("nan")
    o = run(z2, ids, gates, dg, None, sigmoid)
    assert int(o["st"].item()) == 0
    check(z, ids, gates, dg, None, sigmoid, o)
    rows = torch.nonzero(~pad)[:, 0]
    free = int(torch.nonzero(~(torch.arange(E, device=DEV)[:, None] == ids[rows[3]]).any(1))[0])
    z2[rows[3], free] = float("nan")   # a place that was not selected
    free = int(torch.nonzero(~(torch.arange(E, device=DEV)[:, None] == ids[rows[10]]).any(1))[0])
    z2[rows[10], free] = float("inf")
    zr = torch.nan_to_num(z2, nan=float("-inf"), posinf=torch.finfo(torch.float32).max)
    zr[pad] = 0
    o = run(z2, ids, gates, dg, None, sigmoid)
    assert int(o["st"].item()) == G().MOE_DEV_NONFINITE_LOGIT
    check(zr, ids, gates, dg, None, sigmoid, o)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k", [(8, 7), (16, 16), (32, 12), (64, 16), (96, 5)])
def test_repeated_and_bad_ids_of_several_tokens_a_warp(E, k, sigmoid):
    z, ids, gates, dg = make(75, E, k, sigmoid, seed=5)
    ids[5] = 3
    ids[6, :2] = 1
    ids[40, -1] = ids[40, 0]
    o = run(z, ids, gates, dg, None, sigmoid, balance=False)
    want = ref.gate_grad(z, ids, gates, dg, sigmoid, 2.5)
    # gates and their gradients as large as their largest, k of them added
    assert ((o["dz"].double() - want).abs() <= 2e-5 * k * gates.abs().max() * dg.abs().max()).all()
    ids[9, 1] = E
    o = run(z, ids, gates, dg, None, sigmoid)
    assert int(o["st"].item()) == G().MOE_DEV_BAD_EXPERT_ID
    assert int(o["counts"].sum()) == 75 * k - 1


def test_unaligned_rows_of_few_experts():
    z, ids, gates, dg = make(333, 8, 2, False, seed=21)
    zo = torch.empty((333 * 8 + 1,), device=DEV)[1:].view(333, 8).copy_(z)
    o = run(zo, ids, gates, dg, None, False)
    check(z, ids, gates, dg, None, False, o)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,k,S", [(64, 4, 130), (100, 6, 200), (40, 3, 1200), (384, 8, 64)])
def test_many_sequences(E, k, S, sigmoid):
    """A block a sequence in the second stage: one long sequence, short and empty ones."""
    T = 3000
    z, ids, gates, dg = make(T, E, k, sigmoid, seed=S, pad=0.1)
    gen = torch.Generator().manual_seed(S)
    cuts = torch.sort(torch.randint(1800, T + 1, (S - 2,), generator=gen)).values.tolist()
    off = [0, 1700] + cuts + [T]
    o = run(z, ids, gates, dg, off, sigmoid)
    check(z, ids, gates, dg, off, sigmoid, o)
    assert int(o["st"].item()) == 0
    again = run(z, ids, gates, dg, off, sigmoid)
    for name in ("loss", "probs", "dz"):
        assert torch.equal(o[name], again[name])
