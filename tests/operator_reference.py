"""Plain 64-bit definitions of the norm, balance-loss and 8-bit expert operators (torch
doubles, on the device of their inputs), shared by their tests."""
import torch

E4M3_MAX = 448.0


def groups(d, group):
    return 1 if group == 0 else -(-d // 128)


def spread(s, d, group):
    """Scales [n, G] -> one per value [n, d]."""
    return s.expand(-1, d) if group == 0 else s.repeat_interleave(128, 1)[:, :d]


def norm(x, res, w, eps, res_dtype):
    h = x.double() if res is None else (x.float() + res.float()).to(res_dtype).double()
    rstd = (h.square().mean(dim=1) + eps).pow(-0.5)
    return h, rstd, h * rstd[:, None] * w.double()


def norm_backward(h, rstd, w, dy, dres):
    xh = h * rstd[:, None]
    u = dy.double() * w.double()
    dh = rstd[:, None] * (u - xh * (u * xh).mean(dim=1, keepdim=True))
    if dres is not None:
        dh = dh + dres.double()
    return dh, (dy.double() * xh).sum(dim=0)


def scales(v, group):
    """amax / 448 per group (1 for a zero group)."""
    n, d = v.shape
    a = v.abs()
    if group == 0:
        s = a.amax(dim=1, keepdim=True)
    else:
        s = torch.stack([a[:, j:j + 128].amax(dim=1) for j in range(0, d, 128)], dim=1)
    s = s / E4M3_MAX
    return torch.where(s == 0, torch.ones_like(s), s)


def e4m3(v):
    """The nearest E4M3 value, ties to even, saturating."""
    a = v.abs().clamp(max=E4M3_MAX)
    _, e = torch.frexp(a)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def probs(z, sigmoid):
    z = z.double()
    if not sigmoid:
        return torch.softmax(z, dim=1), torch.ones_like(z)
    s = torch.sigmoid(z)
    return s / s.sum(dim=1, keepdim=True), torch.sigmoid(-z)


def balance(z, ids, offsets, alpha, E, k, sigmoid):
    """(counts [S, E], tokens [S + 1], mean probabilities [S, E], loss)."""
    p, _ = probs(z, sigmoid)
    counts, tokens, mean, terms = [], [], [], []
    for a, b in zip(offsets[:-1], offsets[1:]):
        on = ids[a:b, 0] >= 0
        n = int(on.sum())
        c = torch.bincount(ids[a:b][on].reshape(-1).long(), minlength=E)
        m = p[a:b][on].sum(dim=0) / max(n, 1)
        counts.append(c)
        tokens.append(n)
        mean.append(m)
        if n:
            terms.append((c * m).sum() * E / (k * n))
    used = len(terms)
    loss = alpha / used * sum(terms) if used else torch.zeros((), dtype=torch.float64)
    return (torch.stack(counts), torch.tensor(tokens + [used]), torch.stack(mean),
            torch.as_tensor(loss))


def balance_grad(z, ids, offsets, alpha, dloss, E, k, sigmoid):
    p, slope = probs(z, sigmoid)
    counts, tokens, _, _ = balance(z, ids, offsets, alpha, E, k, sigmoid)
    used = max(int(tokens[-1]), 1)
    dz = torch.zeros_like(p)
    for q, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
        n = int(tokens[q])
        if n == 0:
            continue
        w = dloss * alpha / used * E / (k * n) * counts[q].double() / n
        dz[a:b] = p[a:b] * slope[a:b] * (w - (p[a:b] @ w)[:, None])
    return dz * (ids[:, :1] >= 0)


def gate_grad(z, ids, gates, dgates, sigmoid, route_scale):
    g, dg = gates.double(), dgates.double()
    at = ids.long().clamp(min=0)
    inner = (g * dg).sum(dim=1, keepdim=True)
    if sigmoid:
        d = g * torch.sigmoid(-z.double()).gather(1, at) * (dg - inner / route_scale)
    else:
        d = g * (dg - inner)
    return torch.zeros_like(z, dtype=torch.float64).scatter_add(1, at, d * (ids[:, :1] >= 0))


def dequant_blocks(q, s):
    """Codes [N, K] (float8_e4m3fn) and scales [GN, GK] -> doubles."""
    N, K = q.shape
    return q.double() * s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def quantize_blocks(w):
    """fp32 [E, N, K] -> float8 codes and fp32 scales per 128 x 128 block."""
    E, N, K = w.shape
    gn, gk = -(-N // 128), -(-K // 128)
    p = torch.nn.functional.pad(w, (0, gk * 128 - K, 0, gn * 128 - N)).view(E, gn, 128, gk, 128)
    top = p.abs().amax(dim=(2, 4))
    s = top / torch.full_like(top, E4M3_MAX)  # a tensor: dividing by a number multiplies by 1/448
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = (p / s[:, :, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(E, gn * 128, gk * 128)[:, :N, :K].contiguous(), s


def quantize_rows(x):
    """fp32 [n, d] -> float8 codes and fp32 scales per 128 values."""
    n, d = x.shape
    g = -(-d // 128)
    p = torch.nn.functional.pad(x, (0, g * 128 - d)).view(n, g, 128)
    top = p.abs().amax(dim=2)
    s = top / torch.full_like(top, E4M3_MAX)
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = (p / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(n, g * 128)[:, :d].contiguous(), s


def swiglu_hidden(x, wg, wu):
    """Doubles: x [n, d], weights [I, d] -> H [n, I]."""
    a = x @ wg.T
    return a * torch.sigmoid(a) * (x @ wu.T)
