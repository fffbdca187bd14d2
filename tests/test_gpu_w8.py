"""The grouped SwiGLU product in E4M3 with block scales against its definition in 64 bits.

Tolerances: an fp32 sum of K products in blocks of 128 errs by at most C(K) =
(128 + ceil(K/128) + 4) * 2^-24 of the sum of their magnitudes (a block's chain, the
chain over the blocks, the scales' products).  For H = SiLU(G) U that is at most
1.1 |U| dG + |G| dU, plus (16 + |G|) 2^-23 |H| for the exponential (whose
argument's rounding grows with |G|), division and product; where e^-G overflows
(G < -88) H is below 1e-36 |U|, far inside the first term.  A code is then off by half an E4M3 step (2^-4 of the value, 2^-10 of
the scale below the normal range), y by half a bf16 step (2^-8)."""
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


def C(K):
    return (128 + -(-K // 128) + 4) * 2.0 ** -24


def make(d, I, counts, seed, gaps=0, tail=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = len(counts)
    begin, at = [], gaps
    for c in counts:
        begin.append(at)
        at += c + gaps
    R = at + tail
    x = torch.randn((max(R, 1), d), generator=gen, device=DEV)
    x = x * torch.exp(torch.randn((max(R, 1), 1), generator=gen, device=DEV))
    if R > 2:
        x[R // 2] = 0
    xq, xs = ref.quantize_rows(x)
    w = []
    for N, K in ((I, d), (I, d), (d, I)):
        w.append(ref.quantize_blocks(torch.randn((n, N, K), generator=gen, device=DEV) / K ** 0.5))
    return dict(d=d, I=I, n=n, R=R, begin=begin, counts=counts, xq=xq, xs=xs, w=w,
                b=torch.tensor(begin, dtype=torch.int32, device=DEV),
                c=torch.tensor(counts, dtype=torch.int32, device=DEV))


def gate_up(t, stream=None):
    g = G()
    hq = torch.full((max(t["R"], 1), t["I"]), 0x55, dtype=torch.uint8, device=DEV)
    hs = torch.full((max(t["R"], 1), -(-t["I"] // 128)), -7.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    (g0, s0), (g1, s1) = t["w"][0], t["w"][1]
    g.moe_grouped_gate_up_w8(t["n"], t["d"], t["I"], t["R"], t["xq"], t["xs"], t["b"], t["c"], g0, s0,
                             g1, s1, hq, hs, st, stream)
    return hq, hs, st


def down(t, hq, hs, stream=None):
    g = G()
    y = torch.full((max(t["R"], 1), t["d"]), -7.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    q, s = t["w"][2]
    g.moe_grouped_down_w8(t["n"], t["I"], t["d"], t["R"], hq, hs, t["b"], t["c"], q, s, y, st, stream)
    return y, st


def swiglu(t, stream=None):
    g = G()
    y = torch.full((max(t["R"], 1), t["d"]), -7.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    nb = g.moe_grouped_swiglu_w8_workspace_size(t["R"], t["I"])
    ws = torch.empty((nb,), dtype=torch.uint8, device=DEV)
    (g0, s0), (g1, s1), (g2, s2) = t["w"]
    g.moe_grouped_swiglu_w8(t["n"], t["d"], t["I"], t["R"], t["xq"], t["xs"], t["b"], t["c"], g0, s0, g1,
                            s1, g2, s2, y, ws, nb, st, stream)
    return y, st


def owned(t):
    m = torch.zeros((max(t["R"], 1),), dtype=torch.bool, device=DEV)
    for b, c in zip(t["begin"], t["counts"]):
        m[b:b + c] = True
    return m


def check(t):
    d, I = t["d"], t["I"]
    hq, hs, st = gate_up(t)
    y, st2 = down(t, hq, hs)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and int(st2.item()) == 0
    for e, (b, c) in enumerate(zip(t["begin"], t["counts"])):
        if c == 0:
            continue
        x = t["xq"][b:b + c].double() * ref.spread(t["xs"][b:b + c].double(), d, 128)
        wg, wu, wd = (ref.dequant_blocks(q[e], s[e]) for q, s in t["w"])
        a, u = x @ wg.T, x @ wu.T
        h = a * torch.sigmoid(a) * u
        da, du = C(d) * (x.abs() @ wg.abs().T), C(d) * (x.abs() @ wu.abs().T)
        room = 1.1 * u.abs() * da + a.abs() * du + (16 + a.abs()) * 2.0 ** -23 * h.abs()
        s = ref.scales(h, 128)
        room_s = torch.stack([room[:, j:j + 128].amax(1) for j in range(0, I, 128)], 1) / 448
        got_s = hs[b:b + c].double()
        assert ((got_s - s).abs() <= room_s + 2.0 ** -23 * s).all()
        val = hq[b:b + c].view(F8).double() * ref.spread(got_s, I, 128)
        step = torch.maximum(h.abs() * 2.0 ** -4, ref.spread(s, I, 128) * 2.0 ** -10)
        assert ((val - h).abs() <= step * (1 + 1e-3) + 2 * room).all(), (e, c)
        want = val @ wd.T
        room_y = C(I) * (val.abs() @ wd.abs().T)
        assert ((y[b:b + c].double() - want).abs() <= want.abs() * 2.0 ** -8 + 2 * room_y).all(), (e, c)
    out = ~owned(t)  # rows of no segment are left as they were
    assert (y[out] == -7.0).all() and (hq[out] == 0x55).all() and (hs[out] == -7.0).all()
    y2, st = swiglu(t)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(y, y2)


@pytest.mark.parametrize("d,I", [(16, 16), (64, 128), (208, 144), (512, 400), (1040, 272)])
@pytest.mark.parametrize("counts", [[1], [3, 0, 5], [130, 1, 0, 257], [0, 0, 0]])
def test_small(d, I, counts):
    check(make(d, I, counts, seed=d + I + len(counts)))


@pytest.mark.parametrize("counts", [[0, 1, 2, 3, 15, 16, 17, 31], [33, 0, 63, 64, 65], [128, 127, 129, 255, 256, 300]])
def test_row_counts_around_the_tiles(counts):
    check(make(256, 384, counts, seed=len(counts)))


def test_gapped_segments_leave_other_rows():
    check(make(320, 256, [5, 0, 140, 1, 40], seed=3, gaps=7, tail=200))


@pytest.mark.parametrize("seed", [0, 1])
def test_many_segments(seed):
    gen = torch.Generator().manual_seed(seed)
    check(make(128, 144, torch.randint(0, 12, (200,), generator=gen).tolist(), seed))
    check(make(272, 128, torch.randint(0, 150, (24,), generator=gen).tolist(), seed))


@pytest.mark.parametrize("d,I", [(64, 128), (208, 144), (1040, 272)])
@pytest.mark.parametrize("counts", [[0] * 30 + [40, 17, 1], [9] * 20 + [0, 100], [1] * 75 + [229], [2, 0], [40], [100]])
def test_few_rows_and_uneven_segments(d, I, counts):
    """Row tiles of 16 and 32; segments longer than their tile; the reduction split over two
    and four CTAs with one and with several tiles each."""
    check(make(d, I, counts, seed=d + len(counts), gaps=3, tail=1))


def test_one_token_of_the_decode_shape():
    counts = [0] * 128
    for e in (3, 17, 40, 41, 77, 100, 126, 127):
        counts[e] = 1
    check(make(2048, 768, counts, seed=4))


def test_decode_bucket():
    gen = torch.Generator().manual_seed(9)
    check(make(2048, 768, torch.randint(0, 17, (64,), generator=gen).tolist(), seed=5))


@pytest.mark.parametrize("counts", [[1], [7, 0, 1], [16], [33], [120], [1] * 14 + [150]])
def test_split_reductions(counts):
    """Few tiles and many reduction blocks: clusters of two and four, uneven parts (33
    blocks over four CTAs), segments of several tiles."""
    check(make(4112, 1168, counts, seed=20 + len(counts)))


@pytest.mark.parametrize("d,I", [(2064, 2064), (4112, 1168), (2048, 2192), (1936, 2048)])
@pytest.mark.parametrize("counts", [[33], [128], [129], [300], [40, 0, 200], [64, 70, 1], [17, 9], [500, 12]])
def test_split_reductions_of_long_segments(d, I, counts):
    """128-row tiles few enough for clusters of four or two, beside reductions too short or
    tiles too many for them; 15 to 33 blocks, uneven parts; a tile's last rows and columns."""
    check(make(d, I, counts, seed=d + sum(counts), gaps=2, tail=1))


def test_split_reduction_repeats_bit_for_bit():
    """Two captured calls at once, replayed: the parts are added in one order."""
    cases = [make(4096, 2048, [150], seed=31), make(2048, 4096, [40, 90], seed=32)]
    g = G()
    runs = []
    for v in cases:
        want = swiglu(v)[0]
        nb = g.moe_grouped_swiglu_w8_workspace_size(v["R"], v["I"])
        ws = torch.empty((nb,), dtype=torch.uint8, device=DEV)
        y = torch.full((v["R"], v["d"]), -7.0, dtype=torch.bfloat16, device=DEV)
        (g0, s0), (g1, s1), (g2, s2) = v["w"]
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            g.moe_grouped_swiglu_w8(v["n"], v["d"], v["I"], v["R"], v["xq"], v["xs"], v["b"], v["c"], g0,
                                    s0, g1, s1, g2, s2, y, ws, nb)
        runs.append((graph, stream, y, want, ws))
    for _ in range(20):
        for graph, stream, y, _, _ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, y, want, _ in runs:
        assert torch.equal(y, want)


def test_overlapping_segments_are_reported_where_they_exceed_the_tiles():
    """Two segments of the same 256 rows: four tiles a column block where 256 rows in two
    segments have three."""
    t = make(2048, 2048, [256], seed=33)
    u = dict(t, n=2, w=[(q.repeat(2, 1, 1), s.repeat(2, 1, 1)) for q, s in t["w"]],
             b=t["b"].repeat(2), c=t["c"].repeat(2))
    _, st = swiglu(u)
    torch.cuda.synchronize()
    assert int(st.item()) == G().MOE_DEV_BAD_ROW


def test_long_reduction():
    check(make(4096, 2064, [150, 260], seed=6))


def test_wide_output():
    check(make(7168, 512, [40, 0, 300], seed=7))


def test_no_rows():
    t = make(64, 64, [0], seed=1)
    t["R"] = 0
    y, st = swiglu(t)
    assert (y == -7.0).all()


def test_bad_segments_are_reported_and_skipped():
    t = make(128, 128, [4, 4, 4], seed=8)
    for b, c in ((10, 4), (-1, 3), (4, -2)):
        u = dict(t)
        u["b"], u["c"] = t["b"].clone(), t["c"].clone()
        u["b"][1], u["c"][1] = b, c
        y, st = swiglu(u)
        good, _ = swiglu(t)
        torch.cuda.synchronize()
        assert int(st.item()) == G().MOE_DEV_BAD_ROW
        assert torch.equal(y[:4], good[:4]) and torch.equal(y[8:], good[8:])
        assert (y[4:8] == -7.0).all()


def test_nan_codes_stay_in_their_row():
    t = make(256, 256, [6, 40], seed=10)
    good, _ = swiglu(t)
    t["xq"].view(torch.uint8)[2, 7] = 0x7F
    y, st = swiglu(t)
    torch.cuda.synchronize()
    assert int(st.item()) == G().MOE_DEV_NONFINITE_INPUT
    keep = [i for i in range(46) if i != 2]
    assert torch.equal(y[keep], good[keep])


def test_captured_replays_on_another_stream_and_two_calls_at_once():
    t, u = make(512, 256, [9, 0, 33], seed=11), make(512, 256, [200, 5, 1], seed=12)
    want, want_u = swiglu(t)[0], swiglu(u)[0]
    g = G()
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    for v, s in zip((t, u), streams):
        nb = g.moe_grouped_swiglu_w8_workspace_size(v["R"], v["I"])
        ws = torch.empty((nb,), dtype=torch.uint8, device=DEV)
        y = torch.empty((v["R"], v["d"]), dtype=torch.bfloat16, device=DEV)
        (g0, s0), (g1, s1), (g2, s2) = v["w"]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            g.moe_grouped_swiglu_w8(v["n"], v["d"], v["I"], v["R"], v["xq"], v["xs"], v["b"], v["c"], g0,
                                    s0, g1, s1, g2, s2, y, ws, nb)
        outs.append((y, ws))
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(20):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], want) and torch.equal(outs[1][0], want_u)


@pytest.mark.parametrize("n,K,N", [(1, 16, 16), (3, 144, 208), (2, 256, 128), (1, 1040, 528)])
def test_quantize_weights_bit_exact(n, K, N):
    g = G()
    gen = torch.Generator(device=DEV).manual_seed(K)
    w = (torch.randn((n, K, N), generator=gen, device=DEV) / K ** 0.5).to(torch.bfloat16)
    w[0, : K // 2] = 0
    q = torch.empty((n, N, K), dtype=torch.uint8, device=DEV)
    s = torch.empty((n, -(-N // 128), -(-K // 128)), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    g.moe_quantize_weights_fp8(n, K, N, w, q, s, st)
    rq, rs = ref.quantize_blocks(w.float().transpose(1, 2).contiguous())
    assert torch.equal(s, rs) and torch.equal(q, rq.view(torch.uint8))
    assert int(st.item()) == 0
    w[n - 1, K - 1, N - 1] = float("inf")
    g.moe_quantize_weights_fp8(n, K, N, w, q, s, st)
    assert int(st.item()) == g.MOE_DEV_NONFINITE_INPUT


def test_tiny_and_huge_rows():
    """Scales near the ends of fp32: rows whose H is about 1e-38 and about 1e30."""
    t = make(256, 256, [5, 130], seed=14)
    t["xs"][1] *= 1e-19   # G and U about 1e-19, H about 1e-38: its scale is below 2^-126
    t["xs"][3] *= 1e-10
    t["xs"][7] *= 1e15
    hq, hs, st = gate_up(t)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for i, e in ((1, 0), (3, 0), (7, 1)):
        x = t["xq"][i:i + 1].double() * ref.spread(t["xs"][i:i + 1].double(), 256, 128)
        h = ref.swiglu_hidden(x, *(ref.dequant_blocks(t["w"][j][0][e], t["w"][j][1][e]) for j in (0, 1)))
        s = ref.scales(h, 128)
        val = hq[i:i + 1].view(F8).double() * ref.spread(hs[i:i + 1].double(), 256, 128)
        # fp32 holds values this small to 2^-149 only, the scales among them
        room = torch.maximum(h.abs() * 2.0 ** -4, ref.spread(s, 256, 128) * 2.0 ** -10) * 1.01
        floor = 449 * 2.0 ** -149
        assert ((val - h).abs() <= room + 1e-3 * h.abs().max() + floor).all()


def test_a_scale_that_underflows_counts_as_zero():
    """Rows whose H is below 1e-43 (amax / 448 is 0 in fp32): scale 1 and zero codes."""
    for counts in ([5], [130]):  # a few rows, and the 128-row tiles
        t = make(256, 256, counts, seed=15)
        # G and U so small that H is G U / 2: its largest value set to 2e-43
        x = t["xq"][1:2].double()
        gu = [x @ ref.dequant_blocks(q[0], s[0]).T for q, s in t["w"][:2]]
        top = (gu[0] * gu[1] / 2).abs()
        t["xs"][1] = (2e-43 / top.max()).sqrt().float()
        assert (top[:, :128].max() > 0.1 * top.max()) and (top[:, 128:].max() > 0.1 * top.max())
        hq, hs, st = gate_up(t)
        y, st2 = down(t, hq, hs)
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and int(st2.item()) == 0
        assert (hs[1] == 1).all() and (hq[1] & 0x7F == 0).all() and (y[1] == 0).all()


def test_overlapping_segments_of_more_tiles_than_numbers():
    """1,024 segments of the same 2^28 rows have 2^31 tiles: reported, and nothing is written."""
    g = G()
    n, R, I, d = 1024, 1 << 28, 16, 16
    hq = torch.empty((R, I), dtype=torch.uint8, device=DEV)
    hs = torch.empty((R, 1), device=DEV)
    y = torch.empty((R, d), dtype=torch.bfloat16, device=DEV)
    ends = [y[:4096], y[-4096:]]
    for t in ends:
        t.fill_(-7.0)
    b = torch.zeros((n,), dtype=torch.int32, device=DEV)
    c = torch.full((n,), R, dtype=torch.int32, device=DEV)
    q = torch.zeros((n, d, I), dtype=torch.uint8, device=DEV)
    s = torch.ones((n, 1, 1), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    g.moe_grouped_down_w8(n, I, d, R, hq, hs, b, c, q, s, y, st)
    torch.cuda.synchronize()
    assert int(st.item()) == g.MOE_DEV_BAD_ROW
    assert all((t == -7.0).all() for t in ends)
    del hq, hs, y, ends, t
    torch.cuda.empty_cache()
