"""Plain 64-bit forms of the operators beside the projection (adapters of many
requests, per-head norm and rotation), with the bounds their kernels are held
to.  Elementwise torch on any device.

Bounds.  U16 = 2^-8 is half a step of bf16 relative to the value, U32 = 2^-23 a
whole step of fp32 (tensor cores may truncate a sum, so an addition counts a
step, not half of one).  A product of two bf16 is exact in fp32.  A value kept as
the sum of two bf16 is off by at most U16^2 = 2^-16 of itself.
"""
import torch

U16, U32, USPLIT = 2.0 ** -8, 2.0 ** -23, 2.0 ** -16


def adapter_ranks(count, rank, ranks):
    return [rank] * count if ranks is None else [max(0, min(rank, int(r))) for r in ranks]


def adapters(x, ids, a, b, scale, ranks, base):
    """y = base + s_i B_i (A_i x), and the bound of a kernel's |error|."""
    x, base = x.double(), base.double()
    y, tol = base.clone(), torch.zeros_like(base)  # tokens without an adapter: exactly base
    for i, r in enumerate(adapter_ranks(a.shape[0], a.shape[1], ranks)):
        m = torch.nonzero(ids == i)[:, 0]
        if r == 0 or not len(m):
            continue
        ai, bi = a[i, :r].double(), b[i, :, :r].double()
        s = 1.0 if scale is None else float(scale[i])
        v = s * (x[m] @ ai.t())
        y[m] += v @ bi.t()
        dv = abs(s) * (x.shape[1] + 2) * U32 * (x[m].abs() @ ai.abs().t()) + USPLIT * v.abs()
        dd = dv @ bi.abs().t() + (2 * r + 2) * U32 * (base[m].abs() + v.abs() @ bi.abs().t())
        tol[m] = U16 * y[m].abs() + (1 + U16) * dd
    return y, tol


def adapters_backward(x, dy, ids, a, b, scale, ranks, dx_base):
    """(dx, da, db) and the bounds of a kernel's |error| on each."""
    x, dy, dx = x.double(), dy.double(), dx_base.double().clone()
    da, db = torch.zeros_like(a, dtype=torch.float64), torch.zeros_like(b, dtype=torch.float64)
    tx, ta, tb = torch.zeros_like(dx), torch.zeros_like(da), torch.zeros_like(db)
    for i, r in enumerate(adapter_ranks(a.shape[0], a.shape[1], ranks)):
        m = torch.nonzero(ids == i)[:, 0]
        if r == 0 or not len(m):
            continue
        ai, bi = a[i, :r].double(), b[i, :, :r].double()
        s = 1.0 if scale is None else float(scale[i])
        u, v = s * (dy[m] @ bi), s * (x[m] @ ai.t())
        du = abs(s) * (dy.shape[1] + 2) * U32 * (dy[m].abs() @ bi.abs()) + USPLIT * u.abs()
        dv = abs(s) * (x.shape[1] + 2) * U32 * (x[m].abs() @ ai.abs().t()) + USPLIT * v.abs()
        da[i, :r], db[i, :, :r] = u.t() @ x[m], dy[m].t() @ v
        n = 2 * len(m) + 8
        ta[i, :r] = du.t() @ x[m].abs() + n * U32 * (u.abs().t() @ x[m].abs())
        tb[i, :, :r] = dy[m].abs().t() @ dv + n * U32 * (dy[m].abs().t() @ v.abs())
        base = dx[m].abs()
        dx[m] += u @ ai
        dd = du @ ai.abs() + (2 * r + 2) * U32 * (base + u.abs() @ ai.abs())
        tx[m] = U16 * dx[m].abs() + (1 + U16) * dd
    return (dx, da, db), (tx, ta, tb)


def _pairs(rotary, rotation, device):
    k = torch.arange(rotary // 2, device=device)
    return (k, k + rotary // 2) if rotation == "halves" else (2 * k, 2 * k + 1)


def _rotate(v, positions, inv_freq, rotation, sign):
    if inv_freq is None or len(inv_freq) == 0:
        return v, v.abs()
    lo, hi = _pairs(2 * len(inv_freq), rotation, v.device)
    t = (positions.double()[:, None] * inv_freq.double()[None, :])[:, None, :]
    c, s = t.cos(), sign * t.sin()
    out, size = v.clone(), v.abs()
    x, y = v[..., lo], v[..., hi]
    out[..., lo], out[..., hi] = x * c - y * s, y * c + x * s
    size[..., lo] = size[..., hi] = x.abs() + y.abs()
    return out, size


def heads(x, positions, inv_freq, rotation, weight, eps, head_dim):
    """The norm and rotation of one tensor [tokens, heads * head_dim], and the bound of a kernel's |error|."""
    v = x.double().view(x.shape[0], -1, head_dim)
    if weight is not None:
        v = v / (v.pow(2).mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    out, size = _rotate(v, positions, inv_freq, rotation, 1.0)
    # the sum of squares, rsqrt, the products, and an angle off by 2^-24 of a turn and a few steps
    tol = U16 * out.abs() + (1 + U16) * (head_dim + 32) * U32 * size
    return out.flatten(1), tol.flatten(1)


def heads_backward(x, dout, positions, inv_freq, rotation, weight, eps, head_dim):
    """(din, dweight or None) of one tensor and the bounds of a kernel's |error|."""
    d = dout.double().view(dout.shape[0], -1, head_dim)
    dn, size = _rotate(d, positions, inv_freq, rotation, -1.0)
    k = (2 * head_dim + 64) * U32
    if weight is None:
        tol = U16 * dn.abs() + (1 + U16) * k * size
        return (dn.flatten(1), None), (tol.flatten(1), None)
    v = x.double().view(x.shape[0], -1, head_dim)
    rstd = 1.0 / (v.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    n, w = v * rstd, weight.double()
    g = w * dn
    din = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    mean = (w.abs() * size * n.abs()).mean(-1, keepdim=True)
    tol = U16 * din.abs() + (1 + U16) * k * rstd * (w.abs() * size + n.abs() * mean)
    count = dn.shape[0] * dn.shape[1]
    dw = (dn * n).sum((0, 1))
    tw = (k + count * U32) * (size * n.abs()).sum((0, 1))
    return (din.flatten(1), dw), (tol.flatten(1), tw)


def within(got, exact, tol, what=""):
    """Every element of `got` within `tol` of `exact` (and equal where tol is 0)."""
    off = (got.double() - exact).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst {float((off - tol).max()):.3e} "
                                 f"past its bound at {tuple(int(v) for v in torch.nonzero(bad)[0])}")
