"""Plain 64-bit definitions of the projection with adapters and of clipping (torch doubles, on
the device of their inputs), and the room of the kernels' fp32 arithmetic, shared by their
tests.

Room: the tensor cores add 16 products at a time into an fp32 sum; each such addition is off by
at most 2^-23 of the sum of magnitudes S so far (the hardware may cut instead of round), and the
joins of partial sums add at most 40 more: (K / 16 + 40) 2^-23 S.  u and v enter products as two
bf16 numbers at worst, which hold them to 2^-16."""
import torch

BF = 2.0 ** -8
STEP = 2.0 ** -23
PAIR = 2.0 ** -16


def chain(K):
    return (K / 16 + 40) * STEP


def segments(off, ids, T):
    """(first row, last row + 1, adapter) of the segments that hold rows."""
    off = [0, T] if off is None else off
    return [(b, e, a) for b, e, a in zip(off, off[1:], ids) if e > b]


def half_step(v, t):
    return v.abs() * (BF if t is torch.bfloat16 else 2.0 ** -24)


def forward(x, w, a, b, scale, segs):
    """(u, its room, y, its room before the rounding to y's type) of the live rows; other rows
    are NaN."""
    x, w, a, b, s = (t.double() for t in (x, w, a, b, scale))
    T, d = x.shape
    nan = float("nan")
    u = x.new_full((T, a.shape[1]), nan)
    y = x.new_full((T, w.shape[1]), nan)
    ur, yr = u.clone(), y.clone()
    for p, q, e in segs:
        rows = slice(p, q)
        u[rows], ur[rows] = 0.0, 0.0
        y[rows] = x[rows] @ w
        yr[rows] = x[rows].abs() @ w.abs() * chain(d)
        if e >= 0:
            u[rows] = x[rows] @ a[e].T * s[e]
            ur[rows] = (x[rows].abs() @ a[e].abs().T * (chain(d) + 2 * STEP)) * s[e].abs()
            y[rows] += u[rows] @ b[e]
            size = u[rows].abs() @ b[e].abs()
            yr[rows] += ur[rows] @ b[e].abs() + size * (PAIR + chain(2 * a.shape[1]))
    return u, ur, y, yr


def backward(x, w, a, b, scale, segs, dy):
    """(dx, room), (da, room), (db, room): the rooms before dx's rounding."""
    # v and dx are the forward's formulas with the tables and the weight turned around
    v, vr, dx, dxr = forward(dy, w.T, b, a, scale, segs)
    u, ur, _, _ = forward(x, w, a, b, scale, segs)
    x, dy = x.double(), dy.double()
    da, db = torch.zeros(a.shape, dtype=torch.float64, device=x.device), \
        torch.zeros(b.shape, dtype=torch.float64, device=x.device)
    dar, dbr = torch.zeros_like(da), torch.zeros_like(db)
    count = sum(q - p for p, q, _ in segs)
    k = PAIR + 2 * chain(count) + 64 * STEP  # pieces of 32 rows, a part of the rows to a block
    for p, q, e in segs:
        if e < 0:
            continue
        rows = slice(p, q)
        da[e] += v[rows].T @ x[rows]
        db[e] += u[rows].T @ dy[rows]
        dar[e] += (vr[rows] + v[rows].abs() * k).T @ x[rows].abs()
        dbr[e] += (ur[rows] + u[rows].abs() * k).T @ dy[rows].abs()
    return (dx, dxr), (da, dar), (db, dbr)


def clip(grads, groups, n_groups, max_norm):
    sums = [0.0] * n_groups
    for x, g in zip(grads, groups):
        sums[g] = sums[g] + x.double().square().sum()
    norms = [torch.as_tensor(s, dtype=torch.float64).sqrt() for s in sums]
    out = [x.double() * torch.clamp(max_norm / (norms[g].to(x.device) + 1e-6), max=1.0)
           for x, g in zip(grads, groups)]
    return norms, out
