"""Low-rank adapters beside a shared projection, and clipping by gradient norm, as measured
work.

Two operators, each in a plain form (elementary torch operations in fp32) and as the calls a
user of this package makes (``own``):

``adapters``  y = x W + s (x A^T) B over ragged segments of token rows, each with an adapter of
              its own or none; with ``train`` also the backward pass (dx, and the gradients of
              every adapter's two tables).  Rows behind the last segment stay as they are.
``clip``      one gradient norm per group of tensors, and the tensors scaled to it.
"""
import math
import random

import torch

own = False
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
MAX_NORM = 1.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one request decodes one token: latency of streaming the projection and its adapter
        dict(name="adapters_one_token", op="adapters", T=1, live=1, singles=1, longs=0, d=7168,
             n=2048, r=16, adapters=8, y="bf16", train=False),
        # a decode batch, every request with a token and mostly an adapter of its own
        dict(name="adapters_decode", op="adapters", T=128, live=128, singles=128, longs=0, d=4096,
             n=4096, r=32, adapters=96, y="bf16", train=False),
        # decoding requests beside pieces of prompts in one step, padding rows behind
        dict(name="adapters_mixed", op="adapters", T=1024, live=1021, singles=61, longs=5, d=4096,
             n=4096, r=64, adapters=24, y="bf16", train=False),
        # fp32 logits of a router of 256 experts, with adapters
        dict(name="adapters_router", op="adapters", T=4096, live=4096, singles=0, longs=16, d=7168,
             n=256, r=8, adapters=16, y="fp32", train=False),
        # prompt processing at the largest sizes
        dict(name="adapters_prefill", op="adapters", T=8192, live=8192, singles=0, longs=5, d=4096,
             n=14336, r=16, adapters=8, y="bf16", train=False),
        # a training step's forward and backward, four adapters trained side by side
        dict(name="adapters_train", op="adapters", T=4096, live=4096, singles=0, longs=8, d=7168,
             n=2048, r=16, adapters=4, y="bf16", train=True),
        # odd sizes, padding rows
        dict(name="adapters_train_odd", op="adapters", T=1021, live=1003, singles=3, longs=7,
             d=1040, n=712, r=24, adapters=5, y="bf16", train=True),
        # a few small gradients (norm weights, a router): latency
        dict(name="clip_small", op="clip", tensors=6, total=300_000, spread=True, type="fp32",
             groups=1),
        # the gradients of 64 adapters' pairs of tables, a norm for each adapter
        dict(name="clip_adapters", op="clip", tensors=128, total=128 * 16 * 4096, spread=False,
             type="fp32", groups=64),
        # everything that a step trains, many sizes, both types, odd counts
        dict(name="clip_mixed", op="clip", tensors=301, total=90_000_001, spread=True,
             type="mixed", groups=1),
        # the expert weights of a layer with 128 experts (3 x 2048 x 768 each)
        dict(name="clip_experts", op="clip", tensors=384, total=128 * 3 * 2048 * 768, spread=False,
             type="bf16", groups=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.35:
        groups = rng.choice([1, 1, _log(rng, 2, 64)])
        tensors = _log(rng, groups, 500)
        total = _log(rng, max(1000, tensors), 400_000_000)
        return dict(op="clip", tensors=tensors, total=total, spread=rng.random() < 0.7,
                    type=rng.choice(["fp32", "bf16", "mixed"]), groups=groups)
    train = rng.random() < 0.35
    T = _log(rng, 1, 8192)
    d, n = 8 * _log(rng, 8, 1792), 8 * _log(rng, 8, 1792)
    cost = T * d * n * (4 if train else 1)
    if cost > 8192 * 4096 * 14336:
        T = max(1, T * 8192 * 4096 * 14336 // cost)
    live = T if rng.random() < 0.5 else max(1, T - rng.randint(0, T // 8))
    singles = 0 if train else rng.choice([0, min(live, 256), rng.randint(0, min(live, 64))])
    longs = _log(rng, 1, 16) if live > singles else 0
    return dict(op="adapters", T=T, live=live, singles=singles, longs=longs, d=d, n=n,
                r=8 * rng.choice([1, 2, 2, 3, 4, 8, 8, 16]), adapters=_log(rng, 1, 128),
                y="bf16" if train else rng.choice(["bf16", "bf16", "fp32"]), train=train)


def _segments(case, seed):
    """Offsets of the segments and the adapter of each (-1: none), on the host: the program
    that plans a step knows its requests."""
    rng = random.Random(7919 * seed + 11)
    ends = list(range(1, case["singles"] + 1))
    left = case["live"] - case["singles"]
    if case["longs"]:
        # a segment may be empty where two cuts fall together
        cuts = sorted(rng.randint(0, left) for _ in range(case["longs"] - 1)) + [left]
        ends += [case["singles"] + c for c in cuts]
    ids = [rng.randrange(case["adapters"]) if rng.random() < 0.95 else -1 for _ in ends]
    if case["T"] == 1:
        ids = [rng.randrange(case["adapters"])]
    return [0] + ends, ids


def _sizes(case):
    """Element counts of the tensors, from the case alone."""
    n, total = case["tensors"], case["total"]
    if not case["spread"]:
        return [total // n] * n
    rng = random.Random(n * 1_000_003 + total)
    w = [math.exp(rng.uniform(0, math.log(1000))) for _ in range(n)]
    return [max(1, int(total * x / sum(w))) for x in w]


def _types(case):
    return [BF16 if case["type"] == "bf16" or (case["type"] == "mixed" and i % 3 == 1) else F32
            for i in range(case["tensors"])]


_NAMES = {F32: "fp32", BF16: "bf16"}


def _lengths(case):
    """Elements of the flat buffer of each type: every tensor starts at 16 bytes."""
    m = {}
    for c, t in zip(_sizes(case), _types(case)):
        m[t] = m.get(t, 0) + -(-c // 8) * 8
    return m


def _views(case, flat):
    at, out = {t: 0 for t in flat}, []
    for c, t in zip(_sizes(case), _types(case)):
        out.append(flat[t][at[t]:at[t] + c])
        at[t] += -(-c // 8) * 8
    return out


def work(case):
    if case["op"] == "clip":
        b = sum(c * (2 if t == BF16 else 4) for c, t in zip(_sizes(case), _types(case)))
        return {"bytes": 2 * b + 4 * case["groups"], "flops": 3 * sum(_sizes(case))}
    d, n, r = case["d"], case["n"], case["r"]
    off, ids = _segments(case, 0)
    T = off[-1]
    with_adapter = sum(e - b for b, e, a in zip(off, off[1:], ids) if a >= 0)
    touched = len({a for b, e, a in zip(off, off[1:], ids) if a >= 0 and e > b})
    tables = 2 * touched * r * (d + n)
    b = 2 * T * d + 2 * d * n + tables + 4 * T * r + T * n * (4 if case["y"] == "fp32" else 2)
    f = 2 * T * d * n + 2 * with_adapter * r * (d + n)
    if case["train"]:
        # dy, x, u, the weight and the tables once more; dx, and every adapter's gradients
        b += 2 * T * (n + d) + 4 * T * r + 2 * d * n + tables + 2 * T * d
        b += 4 * case["adapters"] * r * (d + n)
        f += 2 * T * d * n + 4 * with_adapter * r * (d + n)
    return {"bytes": b, "flops": f}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=F32)


def prepare(case, seed):
    gen = _gen(seed)
    st = {"case": case}
    new = dict(device=DEV)
    if case["op"] == "clip":
        sizes, types = _sizes(case), _types(case)
        n, G = case["tensors"], case["groups"]
        st["groups"] = [i * G // n for i in range(n)]
        # norms on both sides of the limit: some groups keep their gradients
        per_group = sum(sizes) / G
        level = torch.exp(1.0 + 1.5 * torch.randn((G,), generator=gen, device=DEV)) \
            if G > 1 else torch.full((1,), 3.0, device=DEV)
        flat = {t: torch.zeros((m,), dtype=t, **new) for t, m in _lengths(case).items()}
        kept = {t: torch.zeros_like(f) for t, f in flat.items()}
        st["grads"], st["clipped"] = _views(case, flat), _views(case, kept)
        for x, c, t, q in zip(st["grads"], sizes, types, st["groups"]):
            x.copy_(_randn(gen, c) * (level[q] / math.sqrt(per_group)))
        st["out"] = dict(norms=torch.empty((G,), dtype=F32, **new),
                         **{_NAMES[t]: f for t, f in kept.items()})
        if own:
            import grouped_expert_gemm_gb300 as g
            st["clip"] = g.GradientClip(st["grads"], MAX_NORM, out=st["clipped"],
                                        groups=st["groups"], n_groups=G, norms=st["out"]["norms"])
        return st
    T, d, n, r, N = case["T"], case["d"], case["n"], case["r"], case["adapters"]
    st["off"], st["ids"] = _segments(case, seed)
    st["x"] = _randn(gen, T, d).to(BF16)
    st["w"] = (_randn(gen, d, n) / math.sqrt(d)).to(BF16)
    st["a"] = (_randn(gen, N, r, d) / math.sqrt(d)).to(BF16)
    st["b"] = (_randn(gen, N, r, n) * (0.3 / math.sqrt(r))).to(BF16)
    st["scale"] = torch.exp(0.5 * _randn(gen, N))
    # rows behind the last segment hold what they held
    st["out"] = dict(u=torch.zeros((T, r), dtype=F32, **new),
                     y=torch.zeros((T, n), dtype=BF16 if case["y"] == "bf16" else F32, **new))
    if case["train"]:
        st["dy"] = (_randn(gen, T, n) * 0.01).to(BF16)
        st["out"]["dx"] = torch.zeros((T, d), dtype=BF16, **new)
        st["out"]["da"] = torch.empty((N, r, d), dtype=F32, **new)
        st["out"]["db"] = torch.empty((N, r, n), dtype=F32, **new)
    st["seg_offsets"] = torch.tensor(st["off"], dtype=torch.int32, **new)
    st["seg_adapter"] = torch.tensor(st["ids"], dtype=torch.int32, **new)
    if own:
        import grouped_expert_gemm_gb300 as g
        kind = {"bf16": g.MOE_DTYPE_BF16, "fp32": g.MOE_DTYPE_FP32}
        st["params"] = g.AdapterParams(T, d, n, r, N, len(st["ids"]), kind[case["y"]])
        if case["train"]:
            st["ws_bytes"] = g.moe_adapter_project_backward_workspace_size(st["params"])
            st["ws"] = torch.empty((st["ws_bytes"],), dtype=torch.uint8, **new)
    return st


# ------------------------------------------------------------ plain forms

def _plain_clip(st):
    o = st["out"]
    sums = torch.zeros((st["case"]["groups"],), device=DEV, dtype=torch.float64)
    for x, g in zip(st["grads"], st["groups"]):  # long sums
        sums[g] += x.float().square().sum(dtype=torch.float64)
    norm = sums.sqrt()
    coef = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()
    for x, out, g in zip(st["grads"], st["clipped"], st["groups"]):
        out.copy_(x.float() * coef[g])
    o["norms"].copy_(norm)
    return o


def _plain_adapters(st):
    c, o = st["case"], st["out"]
    live = st["off"][-1]
    x, w = st["x"][:live].float(), st["w"].float()
    segs = [(b, e, a) for b, e, a in zip(st["off"], st["off"][1:], st["ids"]) if e > b]
    y = x @ w
    u = torch.zeros((live, c["r"]), device=DEV)
    for b, e, a in segs:
        if a >= 0:
            u[b:e] = (x[b:e] @ st["a"][a].float().T) * st["scale"][a]
            y[b:e] += u[b:e] @ st["b"][a].float()
    o["u"][:live] = u
    o["y"][:live] = y
    if c["train"]:
        dy = st["dy"][:live].float()
        dx = dy @ w.T
        o["da"].zero_()
        o["db"].zero_()
        for b, e, a in segs:
            if a >= 0:
                v = (dy[b:e] @ st["b"][a].float().T) * st["scale"][a]
                dx[b:e] += v @ st["a"][a].float()
                o["da"][a] += v.T @ x[b:e]
                o["db"][a] += u[b:e].T @ dy[b:e]
        o["dx"][:live] = dx
    return o


# -------------------------------------------------------------------- run

def run(st):
    c, o = st["case"], st["out"]
    if not own:
        return _plain_clip(st) if c["op"] == "clip" else _plain_adapters(st)
    if c["op"] == "clip":
        st["clip"].clip()
        return o
    import grouped_expert_gemm_gb300 as g
    head = (st["params"], st["seg_offsets"], st["seg_adapter"], st["x"], st["w"], st["a"],
            st["b"], st["scale"])
    g.moe_adapter_project(*head, o["u"], o["y"])
    if c["train"]:
        g.moe_adapter_project_backward(*head, o["u"], st["dy"], o["dx"], o["da"], o["db"], 0,
                                       st["ws"], st["ws_bytes"])
    return o


# ------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        norms = []
        flat = {t: torch.zeros((m,), dtype=torch.float64, device=DEV)
                for t, m in _lengths(case).items()}
        outs = _views(case, flat)
        for g in range(case["groups"]):
            mine = [i for i, q in enumerate(st["groups"]) if q == g]
            total = sum((torch.linalg.vector_norm(st["grads"][i].double()) ** 2 for i in mine),
                        torch.zeros((), dtype=torch.float64, device=DEV))
            norm = torch.sqrt(total)
            norms.append(norm)
            factor = torch.minimum(torch.ones_like(norm), MAX_NORM / (norm + 1e-6))
            for i in mine:
                outs[i].copy_(st["grads"][i].double() * factor)
        return dict(norms=torch.stack(norms), **{_NAMES[t]: f for t, f in flat.items()})
    T, d, n, r, N = case["T"], case["d"], case["n"], case["r"], case["adapters"]
    f64 = dict(dtype=torch.float64, device=DEV)
    out = dict(u=torch.zeros((T, r), **f64), y=torch.zeros((T, n), **f64))
    w = st["w"].double()
    if case["train"]:
        out.update(dx=torch.zeros((T, d), **f64), da=torch.zeros((N, r, d), **f64),
                   db=torch.zeros((N, r, n), **f64))
    for q, a in enumerate(st["ids"]):
        rows = slice(st["off"][q], st["off"][q + 1])
        x = st["x"][rows].double()
        # the segment's own weight, W + s A^T B, split into its two parts
        out["y"][rows] = torch.einsum("td,dn->tn", x, w)
        dy = st["dy"][rows].double() if case["train"] else None
        if case["train"]:
            out["dx"][rows] = torch.einsum("tn,dn->td", dy, w)
        if a < 0:
            continue
        A, B = st["a"][a].double(), st["b"][a].double() * st["scale"][a].double()
        xa = torch.einsum("td,rd->tr", x, A)
        out["u"][rows] = xa * st["scale"][a].double()
        out["y"][rows] += torch.einsum("tr,rn->tn", xa, B)
        if case["train"]:
            yb = torch.einsum("tn,rn->tr", dy, B)
            out["dx"][rows] += torch.einsum("tr,rd->td", yb, A)
            out["da"][a] += torch.einsum("tr,td->rd", yb, x)
            out["db"][a] += torch.einsum("tr,tn->rn", out["u"][rows], dy)
    return out
