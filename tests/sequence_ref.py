"""The sequence operators from their definitions, token by token in 64 bits, and
bounds on what fp32 arithmetic may differ from them by.

Bounds.  u = 2^-24 is half a step of fp32.  Each output is rounded once to the io
type (half a step, eps / 2 of its size).  Inside, every fp32 operation is off by at
most u of its result; exp by 2^-22 = 4 u of itself and by its argument's error
(the argument is a product rounded twice, log2(e) among them: 3 u of its size, so
3 |arg| u of the exp); the reciprocal by 2 u.  The recursions below carry these
along with the values, so that each element has a bound of its own.
"""
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _silu(v, bound):
    """silu in 64 bits, and its bound for an argument off by `bound`: the slope is under
    1.1; exp(-v) is off by (5 + 3 |v|) u of itself, the sum, the reciprocal and the
    product by 4 u more."""
    y = v * torch.sigmoid(v)
    return y, 1.1 * bound + (9 + 3 * v.abs()) * U * y.abs()


def _cast(y, bound, dtype):
    """The bound of y after its rounding to dtype (whose smallest step is absolute)."""
    return bound + half_step(dtype) * (y.abs() + bound) + torch.finfo(dtype).tiny * torch.finfo(dtype).eps


def causal_conv(x, w, bias, silu, window):
    """One sequence x [L, C] after window [K-1, C]: (out, bound of out, new window)."""
    L, k = x.shape[0], w.shape[1]
    rows = torch.cat([window.double(), x.double()])
    wd = w.double()
    y = torch.zeros(L, x.shape[1], dtype=torch.float64)
    size = torch.zeros_like(y)
    if bias is not None:
        y += bias.double()
        size += bias.double().abs()
    for j in range(k):
        y += rows[j:j + L] * wd[:, j]
        size += (rows[j:j + L] * wd[:, j]).abs()
    bound = k * U * size
    if silu:
        y, bound = _silu(y, bound)
    return y, _cast(y, bound, x.dtype), torch.cat([window, x])[L:]


def scan(x, dt, a, b, c, d, z, dt_bias, softplus, h, bound_h=None):
    """One sequence x, dt, z [L, D], b, c [L, G, S] from h [D, S]:
    (out, bound of out, h, bound of h)."""
    L, dim = x.shape
    g, s = b.shape[1:]
    xd, a = x.double(), a.double()
    delta = dt.double()
    off = torch.zeros_like(delta)
    if dt_bias is not None:
        delta = delta + dt_bias.double()
        off = U * delta.abs()
    if softplus:
        # log1p's series and its quotient: 12 u; t = exp(-|delta|) off by (4 + 3 |delta|) u
        # of itself, which the result follows by at most its own relative size; the slope is under 1
        soft = torch.nn.functional.softplus(delta, threshold=1e9)
        off = off + (16 + 3 * delta.abs()) * U * soft
        delta = soft
    h = h.double().clone()
    e = torch.zeros_like(h) if bound_h is None else bound_h.clone()
    y = torch.zeros(L, dim, dtype=torch.float64)
    bound = torch.zeros_like(y)
    for t in range(L):
        bt = b[t].double().repeat_interleave(dim // g, 0)
        ct = c[t].double().repeat_interleave(dim // g, 0)
        arg = delta[t][:, None] * a
        decay = torch.exp(arg)
        # exp's own error, its argument's, delta's in the argument
        rel = (4 + 3 * arg.abs()) * U + a.abs() * off[t][:, None]
        add = (delta[t] * xd[t])[:, None] * bt
        add_off = 2 * U * add.abs() + (off[t] * xd[t].abs())[:, None] * bt.abs()
        # a cut sequence also multiplies exp(a sum of delta): its error is below that of the product of the tokens' own
        e = decay * (e + rel * h.abs()) + add_off
        h = decay * h + add
        e = e + 2 * U * h.abs()
        y[t] = (ct * h).sum(1)
        bound[t] = (ct.abs() * e).sum(1) + (s + 1) * U * (ct.abs() * (h.abs() + e)).sum(1)
    if d is not None:
        y = y + d.double() * xd
        bound = bound + 2 * U * (y.abs() + (d.double() * xd).abs())
    if z is not None:
        gate, gate_off = _silu(z.double(), torch.zeros_like(y))
        bound = bound * gate.abs() + (y.abs() + bound) * gate_off + U * (y * gate).abs()
        y = y * gate
    return y, _cast(y, bound, x.dtype), h, e


def assert_within(got, want, bound, what=""):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{what}: off by {(got - want).abs().max():.3e}, {int((over > 0).sum())} values over their bound, " \
                              f"worst {((got - want).abs() / bound.clamp(min=1e-300)).max():.2f} times"
