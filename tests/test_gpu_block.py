"""The norm, the layer with E4M3 experts and the router's loss run together, as a block of a
model runs them: forward, then the backward of everything outside the experts.

Each stage is held to its 64-bit definition on the values that the stage before it stored
(so no stage's rounding is hidden in another's room); the combine's fp32 sum of k + 1 rows
errs by at most (k + 3) 2^-24 of the sum of magnitudes."""
import pytest
import torch

import operator_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def G():
    import grouped_expert_gemm_gb300 as g
    return g


def make(T, d, E, k, I, sigmoid, capacity=-1, shared_I=0, seed=0, payload="fp8_block128"):
    g = G()
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    w = [(rnd(E, a, b) / a ** 0.5).to(torch.bfloat16) for a, b in ((d, I), (d, I), (I, d))]
    q = [g.quantize_weights(t) for t in w]
    sh = None
    if shared_I:
        sh = [g.quantize_weights((rnd(1, a, b) / a ** 0.5).to(torch.bfloat16))
              for a, b in ((d, shared_I), (d, shared_I), (shared_I, d))]
    router = dict(score_fn=g.MOE_SCORE_SIGMOID_GROUP, n_group=4, topk_group=2, route_scale=2.5,
                  sel_bias=0.1 * rnd(E)) if sigmoid else {}
    layer = g.MoELayer(T, d, E, k, I, *q, capacity=capacity, payload=payload,
                       shared_weights=sh, device=DEV, **router)
    norm = g.TokenNorm(T, d, 1 + 0.2 * rnd(d), x_dtype=torch.float32, payload=payload, device=DEV)
    loss = g.RouterLoss(T, E, k, 0.01, layer.params.score_fn, layer.params.route_scale, n_seq=2,
                        device=DEV)
    return layer, norm, loss, rnd, q, sh


def experts_64(q, seg_begin, counts, layer, hq, hs):
    """y rows from the stored codes of H, and the fp32 sums' room: a chain of 128 products a
    block and one addition a block, 2^-24 of the sum of magnitudes each."""
    d, I = layer.d, layer.I
    y = torch.zeros((hq.shape[0], d), dtype=torch.float64, device=DEV)
    room = torch.zeros_like(y)
    for e, (b, c) in enumerate(zip(seg_begin, counts)):
        if c:
            h = hq[b:b + c].view(F8).double() * ref.spread(hs[b:b + c].double(), I, 128)
            w = ref.dequant_blocks(q[2][0][e], q[2][1][e])
            y[b:b + c] = h @ w.T
            room[b:b + c] = (h.abs() @ w.abs().T) * (132 + -(-I // 128)) * 2.0 ** -24
    return y, room


@pytest.mark.parametrize("T,d,E,k,I,sigmoid,capacity,shared_I", [
    (1, 256, 8, 2, 128, False, -1, 0), (37, 208, 16, 4, 144, True, -1, 0),
    (300, 512, 8, 2, 256, False, 60, 0), (130, 256, 16, 4, 128, True, 40, 272)])
def test_block_forward_and_backward(T, d, E, k, I, sigmoid, capacity, shared_I):
    g = G()
    layer, norm, loss, rnd, q, sh = make(T, d, E, k, I, sigmoid, capacity, shared_I, seed=T)
    x, res = rnd(T, d), (3 * rnd(T, d)).to(torch.bfloat16)
    logits = rnd(T, E)
    payload = norm.forward(x, res)
    out = layer.forward(logits, payload)
    offs = torch.tensor([0, T // 3, T], dtype=torch.int32, device=DEV)
    value = loss.forward(logits, layer.topk_ids, offs)
    torch.cuda.synchronize()
    assert int(norm.dev_status.item()) == int(layer.dev_status.item()) == int(loss.dev_status.item()) == 0

    h, rstd, v = ref.norm(x, res, norm.weight, 1e-6, torch.bfloat16)
    assert torch.equal(norm.residual_out.double(), h)
    val = norm.xq.view(F8).double() * ref.spread(norm.xs.double(), d, 128)
    step = torch.maximum(v.abs() * 2.0 ** -4, ref.spread(ref.scales(v, 128), d, 128) * 2.0 ** -10)
    assert ((val - v).abs() <= step * 1.001 + 2e-5 * v.abs()).all()

    # permuted payload rows are the tokens' rows
    offsets, counts = layer.offsets.tolist(), layer.counts.tolist()
    n = offsets[-1]
    tok = (layer.row_to_route[:n] // k).long()
    assert torch.equal(layer.xq_perm[:n], norm.xq[tok]) and torch.equal(layer.xs_perm[:n], norm.xs[tok])

    R = max(T * k, 1)
    hq = torch.empty((R, I), dtype=torch.uint8, device=DEV)
    hs = torch.empty((R, -(-I // 128)), device=DEV)
    g.moe_grouped_gate_up_w8(E, d, I, R, layer.xq_perm, layer.xs_perm, layer.offsets, layer.counts,
                             *q[0], *q[1], hq, hs)
    y, room = experts_64(q, offsets[:-1], counts, layer, hq, hs)
    got = layer.y.double()[:n]
    assert ((got - y[:n]).abs() <= y[:n].abs() * 2.0 ** -8 + 2 * room[:n]).all()

    r2r = layer.route_to_row.long().view(T, k)
    rows = torch.where(r2r[:, :, None] >= 0, layer.y.double()[r2r.clamp(min=0)], 0.0)
    terms = layer.gates.double()[:, :, None] * rows
    want, size = terms.sum(1), terms.abs().sum(1)
    if shared_I:
        want = want + layer.shared_y.double()
        size = size + layer.shared_y.double().abs()
        ys, st = torch.empty_like(layer.shared_y), torch.zeros(1, dtype=torch.int32, device=DEV)
        nb = g.moe_grouped_swiglu_w8_workspace_size(T, shared_I)
        ws = torch.empty((nb,), dtype=torch.uint8, device=DEV)
        g.moe_grouped_swiglu_w8(1, d, shared_I, T, norm.xq, norm.xs, layer.shared_begin,
                                layer.shared_count, *sh[0], *sh[1], *sh[2], ys, ws, nb, st)
        assert torch.equal(ys, layer.shared_y)
    assert ((out.double() - want).abs() <= (k + 3) * 2.0 ** -24 * size + 1e-30).all()

    # backward of everything outside the experts
    dout = rnd(T, d)
    dy = torch.zeros_like(layer.y)
    dg = torch.empty((T, k), device=DEV)
    g.moe_combine_backward(T, k, d, dout, layer.y, R, layer.route_to_row, layer.gates, dy, dg)
    dz = loss.backward(logits, layer.topk_ids, offs, layer.gates, dg)
    dx_perm = rnd(R, d).to(torch.bfloat16)  # (stands for the experts' own backward)
    dv = torch.empty((T, d), device=DEV)
    g.moe_unpermute_grad(T, k, d, dx_perm, R, layer.route_to_row, dv)
    dres_out = rnd(T, d).to(torch.bfloat16)
    dx, dres, dw = norm.backward(dv, dres_out)

    ids, off = layer.topk_ids, offs.tolist()
    c64, t64, m64, l64 = ref.balance(logits, ids, off, 0.01, E, k, sigmoid)
    assert torch.equal(loss.counts.cpu().long(), c64.cpu()) and torch.equal(loss.seq_tokens.cpu().long(), t64)
    assert abs(float(value) - float(l64)) <= 1e-5 * float(l64)
    want = ref.balance_grad(logits, ids, off, 0.01, 1.0, E, k, sigmoid) + \
        ref.gate_grad(logits, ids, layer.gates, dg, sigmoid, layer.params.route_scale)
    assert ((dz.double() - want).abs() <= 2e-5 * (want.abs().max() + dg.abs().max())).all()
    dh, dw64 = ref.norm_backward(h, rstd, norm.weight, dv, dres_out)
    assert ((dx.double() - dh).abs() <= 2e-5 * dh.abs().max()).all()
    assert ((dres.double() - dh).abs() <= dh.abs() * 2.0 ** -8 + 2e-5 * dh.abs().max()).all()
    assert ((dw.double() - dw64).abs() <= 2e-5 * (dv.double().abs() * (h * rstd[:, None]).abs()).sum(0)).all()


def test_bf16_rows_and_payload_pairs_agree():
    """The layer quantizing a bf16 row itself gives the same result as the pair it makes."""
    g = G()
    layer, _, _, rnd, _, _ = make(64, 256, 8, 2, 128, False)
    x = rnd(64, 256).to(torch.bfloat16)
    logits = rnd(64, 8)
    a = layer.forward(logits, x).clone()
    q = torch.empty((64, 256), dtype=torch.uint8, device=DEV)
    s = torch.empty((64, 2), device=DEV)
    g.moe_quantize_fp8(64, 256, g.MOE_SCALE_BLOCK128, x, q, s)
    assert torch.equal(layer.forward(logits, (q, s)), a)
    assert torch.equal(layer.forward(logits, x), a)  # and back to rows


@pytest.mark.parametrize("payload", ["fp8_row", "fp8_block128"])
def test_norm_payload_into_bf16_experts(payload):
    """The dequantizing layer takes the norm's pair too."""
    g = G()
    gen = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    T, d, E, k, I = 50, 256, 8, 2, 128
    w = [(rnd(E, a, b) / a ** 0.5).to(torch.bfloat16) for a, b in ((d, I), (d, I), (I, d))]
    layer = g.MoELayer(T, d, E, k, I, *w, payload=payload, device=DEV)
    norm = g.TokenNorm(T, d, 1 + 0.2 * rnd(d), residual_dtype=None, payload=payload, keep_bf16=False,
                       device=DEV)
    assert norm.y is None
    logits = rnd(T, E)
    out = layer.forward(logits, norm.forward(rnd(T, d).to(torch.bfloat16))).clone()
    rows = torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
    g.moe_dequantize_fp8(T, d, layer.scale_group, norm.xq, norm.xs, rows)
    plain = g.MoELayer(T, d, E, k, I, *w, device=DEV)
    assert torch.equal(plain.forward(logits, rows), out)


def test_block_captured_and_replayed():
    layer, norm, loss, rnd, _, _ = make(48, 256, 16, 4, 128, True, shared_I=128)
    x, res, logits = rnd(48, 256), rnd(48, 256).to(torch.bfloat16), rnd(48, 16)
    offs = torch.tensor([0, 10, 48], dtype=torch.int32, device=DEV)

    def step():
        layer.forward(logits, norm.forward(x, res))
        loss.forward(logits, layer.topk_ids, offs)
        norm.backward(layer.out)
        return loss.backward(logits, layer.topk_ids, offs)

    want_dz = step().clone()
    want, want_dx = layer.out.clone(), norm._grads[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    layer.out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.out, want) and torch.equal(loss.dlogits, want_dz)
    assert torch.equal(norm._grads[0], want_dx)


def test_empty_batch():
    g = G()
    w = torch.ones(64, device=DEV)
    for payload in ("bf16", "fp8_block128"):
        norm = g.TokenNorm(0, 64, w, x_dtype=torch.float32, payload=payload, device=DEV)
        x, res = torch.empty((0, 64), device=DEV), torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
        norm.forward(x, res)
        dx, dres, dw = norm.backward(x, res)
        assert dx.shape == (0, 64) and dres.shape == (0, 64) and (dw == 0).all()
    loss = g.RouterLoss(0, 8, 2, 0.1, device=DEV)
    z, ids = torch.empty((0, 8), device=DEV), torch.empty((0, 2), dtype=torch.int32, device=DEV)
    assert float(loss.forward(z, ids)) == 0 and (loss.counts == 0).all()
    assert loss.backward(z, ids).shape == (0, 8)
    torch.cuda.synchronize()


@pytest.mark.parametrize("shared_I", [0, 128])
def test_empty_batch_through_the_layer(shared_I):
    """No tokens: the norm's empty pair goes into the layer."""
    layer, norm, _, rnd, _, _ = make(0, 256, 8, 2, 128, False, shared_I=shared_I)
    x, res = torch.empty((0, 256), device=DEV), torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)
    logits = torch.empty((0, 8), device=DEV)
    assert layer.forward(logits, norm.forward(x, res)).shape == (0, 256)
    torch.cuda.synchronize()
    assert (layer.counts == 0).all() and (layer.offsets == 0).all()
    assert int(layer.dev_status.item()) == 0


@pytest.mark.parametrize("handle", [False, True])
def test_buffers_made_in_a_call_belong_to_its_stream(handle):
    """The current stream's freed memory, still in use by work queued there, is not taken."""
    g = G()
    gen = torch.Generator(device=DEV).manual_seed(5)
    w = torch.randn((4, 256, 512), generator=gen, device=DEV).to(torch.bfloat16)
    x = torch.randn((64, 512), generator=gen, device=DEV)
    res, dy = x.to(torch.bfloat16), torch.randn((64, 512), generator=gen, device=DEV)
    want = g.quantize_weights(w)
    norms = [g.TokenNorm(64, 512, torch.ones(512, device=DEV), x_dtype=torch.float32, device=DEV)
             for _ in range(2)]
    for n in norms:
        n.forward(x, res)
    want_dx, want_dres, want_dw = norms[0].backward(dy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    stream = s.cuda_stream if handle else s
    torch.cuda._sleep(20_000_000)  # some ms of the current stream's own work
    olds = [torch.empty_like(t) for t in (*want, want_dx, want_dres, want_dw, norms[0]._grads[3])]
    at = {t.data_ptr() for t in olds}
    for t in olds:
        t.view(torch.uint8).fill_(0x33)
    del t, olds
    q, sc = g.quantize_weights(w, stream=stream)
    dx, dres, dw = norms[1].backward(dy, stream=stream)
    assert not at & {t.data_ptr() for t in (q, sc, dx, dres, dw, norms[1]._grads[3])}
    torch.cuda.synchronize()
    assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(sc, want[1])
    assert torch.equal(dx, want_dx) and torch.equal(dres, want_dres) and torch.equal(dw, want_dw)
