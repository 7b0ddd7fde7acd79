"""The experts' FFN and its gradients from their formulas, in 64 bits, with bounds on what the
kernels' roundings may add; and values kept in 8 bits.

Every function works on one expert: x [n,H], w13 [2I,H], w2 [H,I], dy [n,H], h [n,2I] (double).
Bounds are element by element.  e = 2^-24 is one fp32 rounding, b = 2^-8 one bf16 rounding
(both half a step, relative to the value).  A sum of n products in fp32 is off by at most
(n + 1) e sum |products|, in any order of its additions.
"""
import torch

E24 = 2.0 ** -24
B8 = 2.0 ** -8


def sigmoid(g):
    return 1 / (1 + torch.exp(-g))


def forward(x, w13, w2):
    """h = (g, u), a and y"""
    h = x @ w13.T
    g, u = h.chunk(2, 1)
    a = g * sigmoid(g) * u
    return h, a, a @ w2.T


def backward(dy, x, w13, w2, h):
    """dh = (dg, du), a, dx, dw13 and dw2 at the gate and up values h"""
    g, u = h.chunk(2, 1)
    s = sigmoid(g)
    a = g * s * u
    da = dy @ w2
    dh = torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
    return dh, a, dh @ w13, dh.T @ x, dy.T @ a


def silu_error(g):
    """of g s(g) in fp32: exp is off by some e (4 + |g|) of itself (its argument's rounding grows
    with it), and s by no more than that; the other operations add 4 e"""
    return 2 * E24 * (8 + g.abs()) * (g * sigmoid(g)).abs()


def slope_error(g):
    """of s (1 + g (1 - s)) in fp32: s is off by e (8 + |g|) s as above; 1 - s by as much and a
    rounding, times |g|"""
    s = sigmoid(g)
    return 2 * E24 * (8 + g.abs()) * s * (1 + g.abs()) * 2


def forward_bounds(x, w13, w2):
    """of h (before it is rounded to be kept) and of y (its own rounding included)"""
    h, a, y = forward(x, w13, w2)
    g, u = h.chunk(2, 1)
    err_h = (x.shape[1] + 1) * E24 * (x.abs() @ w13.abs().T)
    eg, eu = err_h.chunk(2, 1)
    # the slope of silu is below 1.1 in size
    err_a = (1.1 * eg + silu_error(g)) * (u.abs() + eu) + (g * sigmoid(g)).abs() * eu
    err_a = err_a + (B8 + E24) * (a.abs() + err_a)
    err_y = err_a @ w2.abs().T + (w2.shape[1] + 1) * E24 * ((a.abs() + err_a) @ w2.abs().T)
    return err_h, err_y + B8 * (y.abs() + err_y)


def backward_bounds(dy, x, w13, w2, h, out):
    """of dx, dw13 and dw2, rounded to bf16, bf16 and half a step `out` of theirs"""
    n, H = dy.shape
    I = w2.shape[1]
    g, u = h.chunk(2, 1)
    dh, a, dx, dw13, dw2 = backward(dy, x, w13, w2, h)
    s = sigmoid(g)
    da = dy @ w2
    err_da = (H + 1) * E24 * (dy.abs() @ w2.abs())
    slope = (s * (1 + g * (1 - s))).abs()
    err_dg = err_da * u.abs() * slope + (da.abs() + err_da) * u.abs() * (slope_error(g) + 3 * E24 * slope)
    err_du = err_da * (g * s).abs() + (da.abs() + err_da) * (silu_error(g) + E24 * (g * s).abs())
    err_dh = torch.cat([err_dg, err_du], 1)
    err_dh = err_dh + B8 * (dh.abs() + err_dh)
    err_a = silu_error(g) * u.abs() + E24 * a.abs()
    err_a = err_a + B8 * (a.abs() + err_a)
    err_dx = err_dh @ w13.abs() + (2 * I + 1) * E24 * ((dh.abs() + err_dh) @ w13.abs())
    err_w13 = err_dh.T @ x.abs() + (n + 1) * E24 * ((dh.abs() + err_dh).T @ x.abs())
    err_w2 = dy.abs().T @ err_a + (n + 1) * E24 * (dy.abs().T @ (a.abs() + err_a))
    return (err_dx + B8 * (dx.abs() + err_dx), err_w13 + out * (dw13.abs() + err_w13),
            err_w2 + out * (dw2.abs() + err_w2))


# 2^e, -300 <= e <= 300
_TABLE = torch.tensor([2.0 ** k for k in range(-300, 301)], dtype=torch.float64)


def power(e):
    return _TABLE.to(e.device)[e.long() + 300]


def e4m3_values():
    """The value of each of the 256 codes, from the format's definition"""
    v = []
    for c in range(256):
        s, k, m = -1.0 if c & 128 else 1.0, c >> 3 & 15, c & 7
        v.append(float("nan") if k == 15 and m == 7 else
                 s * (m / 8 * 2.0 ** -6 if k == 0 else (1 + m / 8) * 2.0 ** (k - 7)))
    return torch.tensor(v, dtype=torch.float64)


def scale_exponents(v):
    """e [.., N/32] of rows v [.., N]: the least e >= -127 with max |v| <= 448 * 2^e, over the
    finite values"""
    b = v.double().unflatten(-1, (-1, 32)).abs()
    most = torch.where(torch.isfinite(b), b, torch.zeros_like(b)).amax(-1)
    e = torch.full(most.shape, -127, dtype=torch.int64, device=v.device)
    for k in range(-127, 128):
        e = torch.where(most > 448.0 * 2.0 ** k, k + 1, e)
    return e


def nearest_codes(v, e):
    """The values that v / 2^e rounds to among e4m3's, ties to the even code; NaN for what is not
    finite"""
    q = (v.double().unflatten(-1, (-1, 32)) / power(e)[..., None]).flatten(-2)
    grid = e4m3_values()[:127].to(v.device)        # ascending, from 0 to 448
    a = q.abs().clamp(max=448.0)
    a = torch.where(torch.isfinite(q), a, torch.zeros_like(a))
    hi = torch.searchsorted(grid, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - grid[lo], grid[hi] - a
    pick = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    r = torch.copysign(grid[pick], q)
    return torch.where(torch.isfinite(q), r, torch.full_like(r, float("nan")))


def kept_values(codes, scales):
    """What uint8 codes [.., N] and scales [.., N/32] stand for, in 64 bits"""
    v = e4m3_values().to(codes.device)[codes.long()]
    return (v.unflatten(-1, (-1, 32)) * power(scales.long() - 127)[..., None]).flatten(-2)
