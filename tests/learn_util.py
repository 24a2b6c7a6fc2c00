"""Float64 restatements of the operators for learning with the factor, and the
error bounds that the tests hold the kernels to.

Bounds are of first order in the unit roundoffs: U32 of float32 sums and
products, and UNIT[dtype] of the rounding to the output's type."""
import numpy as np
import torch

U32 = 2.0 ** -24
UNIT = {torch.float32: U32, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
#: the least normal number: below it a type's roundings are absolute
LEAST = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -14, torch.bfloat16: 2.0 ** -126}


def f64(x):
    return None if x is None else x.detach().to(torch.float64).cpu().numpy()


def within(got, want, bound, dtype):
    """|got - want| <= bound + the output's rounding, element by element; NaN
    and infinities where the reference has them."""
    got, want = f64(got), np.asarray(want, np.float64)
    assert got.shape == want.shape, (got.shape, want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    room = bound + UNIT[dtype] * (np.abs(want) + bound) + LEAST[dtype] * UNIT[dtype]
    room = np.broadcast_to(room, want.shape)
    off = np.abs(got[fine] - want[fine])
    worst = off - room[fine]
    assert worst.size == 0 or worst.max() <= 0, \
        f"{int((worst > 0).sum())} of {worst.size} outside, by up to {worst.max():.3g}; " \
        f"there {off[worst.argmax()]:.3g} against {room[fine][worst.argmax()]:.3g}"


# ----------------------------------------------------------------------------
# Norm
# ----------------------------------------------------------------------------
def norm(x, w, res, eps):
    """r, rstd, y in float64 from float64 rows."""
    r = x if res is None else x + res
    rstd = 1.0 / np.sqrt((r * r).mean(-1) + eps)
    y = r * rstd[..., None]
    return r, rstd, y if w is None else y * w


def norm_rounds(d):
    """Relative error of rstd and of y, in units of U32: the sum of d squares,
    r's own rounding (twice: in the sum and in y), and a few operations more."""
    return d + 16


def norm_adj(dy, r, rstd, w, dr):
    """adj_in, adj_w and their bounds before the outputs are rounded."""
    d = r.shape[-1]
    n = r * rstd[..., None]
    u = dy if w is None else dy * w
    c = (u * n).mean(-1, keepdims=True)
    k = (d + 16) * U32
    a = rstd[..., None] * (u - n * c)
    size = rstd[..., None] * (np.abs(u) + np.abs(n) * np.abs(u * n).mean(-1, keepdims=True))
    if dr is not None:
        a, size = a + dr, size + np.abs(dr)
    rows = int(np.prod(r.shape[:-1]))
    flat = (dy * n).reshape(-1, d)
    return a, k * size, flat.sum(0), (rows + 16) * U32 * np.abs(flat).sum(0)


# ----------------------------------------------------------------------------
# Recurrence
# ----------------------------------------------------------------------------
def gates(g, kind):
    """a, 1 - a, da/dg and the relative error of a and 1 - a in units of U32
    (an exponential's own, and that of its scaled argument)."""
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "linear":
            return g, 1.0 - g, np.ones_like(g), np.full_like(g, 2.0)
        if kind == "log":
            a = np.exp(g)
            return a, -np.expm1(g), a, 8.0 + 3.0 * np.abs(g)
        a, c = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
        return a, c, a * c, 8.0 + 3.0 * np.abs(g)


def spans(shape, offsets):
    """(row of the batch, state, lo, hi) of each sequence."""
    if offsets is None:
        return [(b, b, 0, shape[1]) for b in range(shape[0])]
    off = [int(v) for v in offsets]
    return [(0, s, lo, hi) for s, (lo, hi) in enumerate(zip(off, off[1:]))]


def linrec(g, x, state, offsets, kind, comp):
    """h, final states and bounds of both; g, x are [B, T, D] in float64.

    The bound carries every rounding along the recurrence of magnitudes: with
    M_t = |a| M_{t-1} + |b|, each step adds at most its units of M_t."""
    a, c, _, rel = gates(g, kind)
    b = c * x if comp else x
    n = state.shape[0]
    h, eh = np.zeros_like(b), np.zeros_like(b)
    last, elast = state.copy(), np.zeros_like(state)
    for row, s, lo, hi in spans(g.shape, offsets):
        cur, m, e = state[s], np.abs(state[s]), np.zeros_like(state[s])
        for t in range(lo, hi):
            mag = np.abs(a[row, t]) * m + np.abs(b[row, t])
            e = np.abs(a[row, t]) * e + (8.0 + rel[row, t]) * U32 * mag
            cur = a[row, t] * cur + b[row, t]
            m = mag
            h[row, t], eh[row, t] = cur, e
        last[s], elast[s] = cur, e
    assert n == len(spans(g.shape, offsets))
    return h, last, eh, elast


def linrec_adj(g, x, h, dh, state, dlast, offsets, kind, comp):
    """adj_g, adj_x, adj_state0 and bounds, from the forward's own h."""
    a, c, da_dg, rel = gates(g, kind)
    dg, dx, eg, ex = (np.zeros_like(g) for _ in range(4))
    d0, e0 = dlast.copy(), np.zeros_like(dlast)
    for row, s, lo, hi in spans(g.shape, offsets):
        carry, m, e = dlast[s], np.abs(dlast[s]), np.zeros_like(dlast[s])
        for t in reversed(range(lo, hi)):
            lam, mag = dh[row, t] + carry, np.abs(dh[row, t]) + m
            err = e + 2.0 * U32 * mag
            before = h[row, t - 1] if t > lo else state[s]
            diff = before - x[row, t] if comp else before
            size = np.abs(before) + (np.abs(x[row, t]) if comp else 0.0)
            units = (8.0 + 2.0 * rel[row, t]) * U32
            dg[row, t] = lam * diff * da_dg[row, t]
            eg[row, t] = (err + units * mag) * size * np.abs(da_dg[row, t])
            cv = c[row, t] if comp else 1.0
            dx[row, t], ex[row, t] = lam * cv, (err + units * mag) * np.abs(cv)
            carry = a[row, t] * lam
            m = np.abs(a[row, t]) * mag
            e = np.abs(a[row, t]) * err + (8.0 + rel[row, t]) * U32 * m
        d0[s], e0[s] = carry, e
    return dg, dx, d0, eg, ex, e0


# ----------------------------------------------------------------------------
# AdamW, with float32's roundings one by one
# ----------------------------------------------------------------------------
def e4m3(x):
    return torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn)


def encode(x, keep):
    """(e4m3 values, scales) of float32 x in blocks of 256."""
    n = x.size
    pad = np.zeros(-(-n // 256) * 256, np.float32)
    pad[:n] = x
    blocks = pad.reshape(-1, 256)
    scale = np.maximum(np.abs(blocks).max(1) * np.float32(1.0 / 448.0), np.float32(2.0 ** -100))
    q = blocks * (np.float32(1.0) / scale)[:, None]
    if keep:
        q = np.where(blocks > 0, np.maximum(q, np.float32(2.0 ** -9)), q)
    return e4m3(q.reshape(-1)[:n].astype(np.float32)), torch.from_numpy(scale.astype(np.float32))


def decode(q, scale):
    return (q.float() * scale.repeat_interleave(256)[:q.numel()]).numpy()


def adamw(p, g, m, r_or_v, bits, lr, b1, b2, eps, wd, step, scale):
    """p (float64 or float32 array), float32 g and m, and sqrt(v) (8 bits) or v:
    new p, m, v, sqrt(v)."""
    f = np.float32
    g = (g * f(scale)).astype(f)
    v = (r_or_v * r_or_v).astype(f) if bits == 8 else r_or_v
    m = m * f(b1) + g * f(1.0 - b1)
    v = v * f(b2) + (g * g) * f(1.0 - b2)
    r = np.sqrt(v)
    upd = (m / (r * f(1.0 / np.sqrt(1.0 - b2 ** step)) + f(eps))) * f(lr / (1.0 - b1 ** step))
    assert m.dtype == v.dtype == r.dtype == upd.dtype == f
    decay = 1.0 - lr * wd
    p = p * decay - upd.astype(np.float64) if p.dtype == np.float64 else p * f(decay) - upd
    return p, m, v, r
