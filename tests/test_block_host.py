"""Argument checks of TokenNorm, RouterLoss and the layer with E4M3 experts: each refuses
with ValueError before anything is enqueued (no GPU is touched)."""
import pytest
import torch

import grouped_expert_gemm_gb300 as g

F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_expert_gemm_gb300 import build
    build.build()


def test_norm_arguments():
    w = torch.ones(64)
    n = g.TokenNorm(4, 64, w, device="cpu")
    x, r = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((4, 64), dtype=torch.bfloat16)
    for kw in (dict(payload="fp8"), dict(x_dtype=torch.float16), dict(residual_dtype=torch.float64)):
        with pytest.raises(ValueError):
            g.TokenNorm(4, 64, w, device="cpu", **kw)
    for bad in (torch.ones(63), torch.ones(64, dtype=torch.bfloat16), torch.ones(128)[::2]):
        with pytest.raises(ValueError):
            g.TokenNorm(4, 64, bad, device="cpu")
    for a, b in ((x, None), (x.float(), r), (x[:3], r), (x, r.float()), (x.t().contiguous().t(), r),
                 (x, torch.zeros((4, 128), dtype=torch.bfloat16)[:, :64]), (None, r)):
        with pytest.raises(ValueError):
            n.forward(a, b)
    with pytest.raises(ValueError):
        n.backward(x)  # before any forward
    with pytest.raises(ValueError):
        g.TokenNorm(4, 64, w, residual_dtype=None, device="cpu").forward(x, r)


def test_router_loss_arguments():
    for kw in (dict(E=513, k=8), dict(E=8, k=9), dict(E=8, k=2, n_seq=0),
               dict(E=8, k=2, score_fn=g.MOE_SCORE_SIGMOID_GROUP, route_scale=0.0)):
        with pytest.raises(ValueError):
            g.RouterLoss(4, alpha=0.1, device="cpu", **kw)
    L = g.RouterLoss(4, 8, 2, 0.1, n_seq=2, device="cpu")
    z, ids = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32)
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    for a in ((z, ids, None), (z.double(), ids, off), (z, ids.long(), off), (z[:, :4], ids, off),
              (z, ids, off[:2])):
        with pytest.raises(ValueError):
            L.forward(*a)
    with pytest.raises(ValueError):
        L.backward(z, ids, off, gates=torch.zeros((4, 2)))
    with pytest.raises(ValueError):
        L.backward(z, ids, off, dloss=torch.zeros(2))


def pair(n, N, K):
    return torch.zeros((n, N, K), dtype=F8), torch.ones((n, -(-N // 128), -(-K // 128)))


def test_layer_with_e4m3_experts_arguments():
    d, E, k, I = 256, 4, 2, 128
    w = [pair(E, I, d), pair(E, I, d), pair(E, d, I)]
    ok = dict(payload="fp8_block128", device="cpu")
    g.MoELayer(8, d, E, k, I, *w, **ok)
    for kw in (dict(payload="bf16"), dict(payload="fp8_row"), dict(fp8_loader="fused"),
               dict(gather=True), dict(decode_path="fused"), dict(expert_passes="onepass")):
        with pytest.raises(ValueError):
            g.MoELayer(8, d, E, k, I, *w, **{**ok, **kw})
    for i, bad in ((0, pair(E, d, I)), (2, pair(E, I, d)), (1, (w[1][0], w[1][1][:, :, :1])),
                   (1, (w[1][0].float(), w[1][1])), (0, w[0][0])):
        v = list(w)
        v[i] = bad
        with pytest.raises(ValueError):
            g.MoELayer(8, d, E, k, I, *v, **ok) if isinstance(v[0], tuple) else \
                g.MoELayer(8, d, E, k, I, (v[0],), v[1], v[2], **ok)
    with pytest.raises(ValueError):  # a bf16 shared expert beside E4M3 experts
        g.MoELayer(8, d, E, k, I, *w, shared_weights=[torch.zeros(1, d, I)] * 3, **ok)
    with pytest.raises(ValueError):  # the bucket's calls have no E4M3 form
        g.DecodeBucket(8, d, E, k, I, *w, device="cpu")
    layer = g.MoELayer(8, d, E, k, I, *w, **ok)
    z = torch.zeros((8, E))
    q, s = torch.zeros((8, d), dtype=torch.uint8), torch.ones((8, 2))
    for x in ((q[:4], s), (q, s[:, :1]), (q.float(), s), (q, s.double())):
        with pytest.raises(ValueError):
            layer.forward(z, x)
    with pytest.raises(ValueError):
        g.quantize_weights(torch.zeros((2, 16, 16)))


def test_payload_scales_are_fp32():
    w = [pair(4, 128, 256), pair(4, 128, 256), pair(4, 256, 128)]
    layer = g.MoELayer(8, 256, 4, 2, 128, *w, payload="fp8_block128", device="cpu")
    q, s = torch.zeros((8, 256), dtype=torch.uint8), torch.ones((8, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        layer.forward(torch.zeros((8, 4)), (q, s))


@pytest.mark.parametrize("other", [torch.float8_e5m2, torch.int8, torch.bool])
def test_codes_of_another_one_byte_type_are_refused(other):
    """They would be read as E4M3."""
    d, E, k, I = 256, 4, 2, 128
    w = [pair(E, I, d), pair(E, I, d), pair(E, d, I)]
    sh = [pair(1, I, d), pair(1, I, d), pair(1, d, I)]
    ok = dict(payload="fp8_block128", device="cpu")
    raw = [(q.view(torch.uint8), s) for q, s in w]
    layer = g.MoELayer(8, d, E, k, I, *raw, **ok)  # raw bytes are codes
    for i in range(3):
        v = list(w)
        v[i] = (w[i][0].view(torch.uint8).to(other), w[i][1])
        with pytest.raises(ValueError):
            g.MoELayer(8, d, E, k, I, *v, **ok)
    with pytest.raises(ValueError):
        g.MoELayer(8, d, E, k, I, *w, shared_weights=[(sh[0][0].view(torch.uint8).to(other), sh[0][1]), *sh[1:]], **ok)
    with pytest.raises(ValueError):
        layer.forward(torch.zeros((8, E)), (torch.zeros((8, d), dtype=torch.uint8).to(other), torch.ones((8, 2))))


def test_codes_and_scales_on_another_device_are_refused():
    """Their addresses would go to the kernels as they are.  (The meta device stands for
    another one; the shared expert's pairs and the payload's are looked at too.)"""
    d, E, k, I = 256, 4, 2, 128
    w = [pair(E, I, d), pair(E, I, d), pair(E, d, I)]
    sh = [pair(1, I, d), pair(1, I, d), pair(1, d, I)]
    ok = dict(payload="fp8_block128", device="cpu")
    layer = g.MoELayer(8, d, E, k, I, *w, **ok)

    def away(p, i):
        p = list(p)
        p[i] = p[i].to("meta")
        return tuple(p)

    for i in range(3):
        for part in range(2):
            v = list(w)
            v[i] = away(w[i], part)
            with pytest.raises(ValueError, match="on cpu"):
                g.MoELayer(8, d, E, k, I, *v, **ok)
            v = list(sh)
            v[i] = away(sh[i], part)
            with pytest.raises(ValueError, match="on cpu"):
                g.MoELayer(8, d, E, k, I, *w, shared_weights=v, **ok)
    payload = (torch.zeros((8, d), dtype=torch.uint8), torch.ones((8, 2)))
    for part in range(2):
        with pytest.raises(ValueError, match="on cpu"):
            layer.forward(torch.zeros((8, E)), away(payload, part))
    for bad in ((payload[0], None), (payload[0].numpy(), payload[1])):
        with pytest.raises(ValueError):
            layer.forward(torch.zeros((8, E)), bad)


def test_devices_of_one_name(monkeypatch):
    """"cuda" is the current GPU."""
    from grouped_expert_gemm_gb300 import layer
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    dev = torch.device
    assert layer._same_device(dev("cuda"), dev("cuda", 1)) and layer._same_device(dev("cpu"), dev("cpu"))
    assert not layer._same_device(dev("cuda", 0), dev("cuda")) and not layer._same_device(dev("cpu"), dev("cuda"))


def test_pairs_beside_bf16_weights_are_refused():
    """In the constructor, not in the first forward."""
    d, E, k, I = 256, 4, 2, 128
    w = [pair(E, I, d), pair(E, I, d), pair(E, d, I)]
    bf = [torch.zeros(s, dtype=torch.bfloat16) for s in ((E, d, I), (E, d, I), (E, I, d))]
    for payload in ("bf16", "fp8_block128"):
        for i in range(3):
            for a, b in ((w, bf), (bf, w)):
                v = list(a)
                v[i] = b[i]
                with pytest.raises(ValueError):
                    g.MoELayer(8, d, E, k, I, *v, payload=payload, device="cpu")
        with pytest.raises(ValueError):
            g.MoELayer(8, d, E, k, I, *bf, shared_weights=[pair(1, I, d), pair(1, I, d), pair(1, d, I)],
                       payload=payload, device="cpu")
    for bad in ((), (w[0][0],), (None, w[0][1])):  # a shared gate that is no pair
        with pytest.raises(ValueError):
            g.MoELayer(8, d, E, k, I, *w, shared_weights=[bad, *w[1:]], payload="fp8_block128", device="cpu")


@pytest.mark.parametrize("overlap", [False, True])
def test_pooled_layer_and_buckets_refuse_pairs(overlap):
    d, L, k, I = 256, 4, 2, 128
    w = [pair(L, I, d), pair(L, I, d), pair(L, d, I)]
    with pytest.raises(ValueError, match="E4M3"):
        g.PooledMoELayer(8, d, k, I, 2, L, 1, 16, 16, *w, device="cpu", overlap=overlap)
    with pytest.raises(ValueError, match="E4M3"):
        g.DecodeBucketLadder([1, 4], d, L, k, I, *w, device="cpu")


@pytest.mark.parametrize("T", [0, 1, 3])
def test_payload_has_a_row_of_scales_a_token(T):
    """The empty batch too, whose layer keeps a row of its own."""
    w = [pair(4, 128, 256), pair(4, 128, 256), pair(4, 256, 128)]
    layer = g.MoELayer(T, 256, 4, 2, 128, *w, payload="fp8_block128", device="cpu")
    norm = g.TokenNorm(T, 256, torch.ones(256), payload="fp8_block128", device="cpu")
    layer._check_payload(norm.output)
    for n in {T + 1, max(T - 1, 0)} - {T}:
        with pytest.raises(ValueError):
            layer._check_payload((norm.xq, torch.ones((n, 2))))


def test_calls_allocate_on_their_own_stream(monkeypatch):
    """What a call allocates belongs to the stream it is given: memory of the current one may
    still be in use there."""
    from grouped_expert_gemm_gb300 import block
    asked = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: asked.append(s) or block.contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device: ("external", s, device))
    cuda = torch.device("cuda", 0)
    for stream, want in ((None, []), ("s", ["s"]), (1234, [("external", 1234, cuda)])):
        asked.clear()
        with block._memory_of(stream, cuda):
            pass
        assert asked == want
    with block._memory_of("s", torch.device("cpu")):
        pass
    assert len(asked) == 1


def test_the_current_device_must_be_the_objects(monkeypatch):
    """Kernels go to the current device's stream, whichever GPU the buffers are on."""
    from grouped_expert_gemm_gb300 import abi
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(abi, "_device", lambda: 0)
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    norm = g.TokenNorm(4, 64, torch.ones(64), device="cpu")
    loss = g.RouterLoss(4, 8, 2, 0.1, device="cpu")
    z, ids = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32)
    norm.device = loss.device = torch.device("cuda", 1)
    for call in (lambda: norm.forward(x, x), lambda: norm.backward(x), lambda: loss.forward(z, ids),
                 lambda: loss.backward(z, ids)):
        with pytest.raises(ValueError, match="current device is cuda:0"):
            call()
    abi.check_current_device(torch.device("cuda", 0))
    abi.check_current_device(torch.device("cpu"))
    monkeypatch.setattr(abi, "_device", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    with pytest.raises(ValueError, match="current device is cuda:2"):
        abi.check_current_device(torch.device("cuda", 1))
    abi.check_current_device(torch.device("cuda", 2))

    class Elsewhere:
        device = torch.device("cuda", 1)

    w = [pair(4, 128, 256), pair(4, 128, 256), pair(4, 256, 128)]
    layer = g.MoELayer(8, 256, 4, 2, 128, *w, payload="fp8_block128", device="cpu")
    layer.out = Elsewhere()
    with pytest.raises(ValueError, match="current device is cuda:2"):
        layer.forward(torch.zeros((8, 4)), torch.zeros((8, 256), dtype=torch.bfloat16))
