"""Plain fp64 implementations (torch, CPU) of the operators of include/mamba2_proj.h, for the
tests."""
import math

import torch


def scale_exponent(top):
    """The smallest whole e >= -127 with top <= 448 * 2^e, by trying."""
    if top == 0:
        return -127
    e = max(-127, math.floor(math.log2(top)) - 10)
    while top > 448 * 2.0 ** e:
        e += 1
    return e


def e4m3(v):
    """fp64 values of magnitude at most 448 to the nearest e4m3 number, ties to even; what is not
    finite to NaN."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.where(v.isfinite(), torch.round(v / step) * step, float("nan"))


def quant(x, rows, cols):
    """x [m, n] fp64 in groups of rows x cols -> (q [m, n], s [m / rows, n / cols]) as fp64 values."""
    m, n = x.shape
    q, s = torch.empty_like(x), torch.empty(-(-m // rows), -(-n // cols), dtype=torch.float64)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = slice(i * rows, (i + 1) * rows), slice(j * cols, (j + 1) * cols)
            part = x[at]
            finite = part[part.isfinite()].abs()
            s[i, j] = 2.0 ** scale_exponent(finite.max().item() if finite.numel() else 0.0)
            q[at] = e4m3(part / s[i, j])
    return q, s


def dequant(q, s, rows, cols):
    wide = s.repeat_interleave(rows, 0)[:q.shape[0]].repeat_interleave(cols, 1)[:, :q.shape[1]]
    return q * wide


def add_norm(total, w, eps):
    """y of the sum (in whatever precision it is kept)."""
    r = 1 / (total.square().mean(-1, keepdim=True) + eps).sqrt()
    return total * r * (w if w is not None else 1.0)


def add_norm_bwd(total, w, eps, dy, dtotal):
    v = w if w is not None else torch.ones_like(total[0])
    r = 1 / (total.square().mean(-1, keepdim=True) + eps).sqrt()
    n, g = total * r, dy * v
    d = r * (g - n * (g * n).mean(-1, keepdim=True))
    return (d if dtotal is None else d + dtotal), (dy * n).flatten(0, -2).sum(0)


def add_norm_bwd_size(total, w, eps, dy, dtotal):
    """The sum of the magnitudes of dx's three terms."""
    v = w if w is not None else torch.ones_like(total[0])
    r = 1 / (total.square().mean(-1, keepdim=True) + eps).sqrt()
    n, g = total * r, dy * v
    return r * (g.abs() + n.abs() * (g * n).mean(-1, keepdim=True).abs()) + (0 if dtotal is None else dtotal.abs())


def proj_bwd(dy, x, w):
    """dx and dw of y = x w^T in 8 bits, for x and w as the values that they stand for."""
    return dequant(*quant(dy, 1, 128), 1, 128) @ w, \
        dequant(*quant(dy, 128, 1), 128, 1).t() @ dequant(*quant(x, 128, 1), 128, 1)
