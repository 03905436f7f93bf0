"""Plain fp64 implementations (torch, CPU) of the layer operators of
include/mamba2_layer.h, forward and backward, token by token, for the tests."""
import torch


def silu(v):
    g = torch.sigmoid(v)
    return v * g, g + v * g * (1 - g)


def _ends(lengths, b, T):
    return [T] * b if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def conv(x, w, bias, init, lengths, act=True, dy=None, dfinal=None):
    """(y, final_state), or the gradients when dy is given."""
    b, T, D = x.shape
    W = w.shape[1]
    init_ = init if init is not None else x.new_zeros(b, W - 1, D)
    y, final = x.new_zeros(b, T, D), init_.clone()
    g = dict(dx=x.new_zeros(b, T, D), dw=torch.zeros_like(w), dbias=w.new_zeros(D), dinit=torch.zeros_like(init_))
    for i, n in enumerate(_ends(lengths, b, T)):
        seen = torch.cat([init_[i], x[i, :n]])
        dseen = torch.zeros_like(seen)
        for t in range(n):
            near = seen[t:t + W]
            s = (near * w.t()).sum(0) + (bias if bias is not None else 0)
            v, slope = silu(s) if act else (s, torch.ones_like(s))
            y[i, t] = v
            if dy is not None:
                ds = dy[i, t] * slope
                g["dw"] += (ds * near).t()
                g["dbias"] += ds
                dseen[t:t + W] += ds * w.t()
        final[i] = seen[n:]
        if dfinal is not None:
            dseen[n:] += dfinal[i]
        g["dinit"][i], g["dx"][i, :n] = dseen[:W - 1], dseen[W - 1:]
    return (y, final) if dy is None else g


def scan(x, dt, A, B, C, D, z, dt_bias, init, lengths, softplus=True, dy=None, dfinal=None):
    """(y, final_state), or the gradients when dy is given."""
    b, T, ch = x.shape
    N, G = A.shape[1], B.shape[2]
    size = ch // G
    y, final = x.new_zeros(b, T, ch), x.new_zeros(b, ch, N)
    skip = D if D is not None else x.new_zeros(ch)
    g = dict(dx=torch.zeros_like(x), ddt=torch.zeros_like(x), dA=torch.zeros_like(A), dB=torch.zeros_like(B),
             dC=torch.zeros_like(C), dD=x.new_zeros(ch), dz=torch.zeros_like(x), ddt_bias=x.new_zeros(ch),
             dinit=torch.zeros_like(final))
    for i, n in enumerate(_ends(lengths, b, T)):
        h = init[i] if init is not None else x.new_zeros(ch, N)
        hs = [h]
        raw = [dt[i, t] + (dt_bias if dt_bias is not None else 0) for t in range(n)]
        step = [torch.logaddexp(r, torch.zeros_like(r)) if softplus else r for r in raw]
        for t in range(n):
            Bt, Ct = (v[i, t].repeat_interleave(size, 0) for v in (B, C))
            h = torch.exp(step[t][:, None] * A) * h + (step[t] * x[i, t])[:, None] * Bt
            hs.append(h)
            core = (h * Ct).sum(1) + skip * x[i, t]
            y[i, t] = core * silu(z[i, t])[0] if z is not None else core
        final[i] = h
        if dy is None:
            continue
        a = dfinal[i].clone() if dfinal is not None else x.new_zeros(ch, N)
        for t in range(n - 1, -1, -1):
            Bt, Ct = (v[i, t].repeat_interleave(size, 0) for v in (B, C))
            dY, d, xt = dy[i, t], step[t], x[i, t]
            if z is not None:
                gate, slope = silu(z[i, t])
                g["dz"][i, t] = dY * ((hs[t + 1] * Ct).sum(1) + skip * xt) * slope
                dY = dY * gate
            a = a + dY[:, None] * Ct
            g["dC"][i, t] = (hs[t + 1] * dY[:, None]).view(G, size, N).sum(1)
            g["dB"][i, t] = (a * (d * xt)[:, None]).view(G, size, N).sum(1)
            q = (a * Bt).sum(1)
            a = a * torch.exp(d[:, None] * A)
            e = a * hs[t]
            g["dA"] += e * d[:, None]
            g["dx"][i, t] = d * q + skip * dY
            dd = (xt * q + (e * A).sum(1)) * (torch.sigmoid(raw[t]) if softplus else 1)
            g["ddt"][i, t] = dd
            g["ddt_bias"] += dd
            g["dD"] += dY * xt
        g["dinit"][i] = a
    return (y, final) if dy is None else g


def norm(x, w, z, G, eps, gate_first=True, dy=None):
    """y, or the gradients when dy is given."""
    S = x.shape[-1] // G
    gate, slope = silu(z) if z is not None else (torch.ones_like(x), torch.zeros_like(x))
    v = (x * gate if gate_first else x).unflatten(-1, (G, S))
    r = 1 / (v.square().mean(-1, keepdim=True) + eps).sqrt()
    n = (v * r).flatten(-2)
    ww = w if w is not None else torch.ones_like(x[0, 0]) if x.numel() else x.new_ones(x.shape[-1])
    if dy is None:
        return n * ww if gate_first else n * ww * gate
    out = {}
    if not gate_first:
        out["dz"] = dy * n * ww * slope
        dy = dy * gate
    out["dw"] = (dy * n).sum((0, 1))
    q = (dy * ww).unflatten(-1, (G, S))
    dv = (r * q - v * r ** 3 * (q * v).mean(-1, keepdim=True)).flatten(-2)
    if gate_first:
        out["dz"] = dv * x * slope
        dv = dv * gate
    out["dx"] = dv
    return out
