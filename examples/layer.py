"""A layer out of this package's operators: prompts, single tokens and a training step.

    python examples/layer.py            # on a CUDA device

Two layers are shown.  SSDLayer: projection -> conv -> chunked scan (one decay per head)
-> gated group norm -> projection.  ScanLayer: projection -> conv -> selective scan (a
decay per channel and state, gated) -> projection.  Both take padded prompts of
different lengths and then go on token by token from the states that the prompt left;
main() checks that this gives what the whole sequence gives, and takes a training step
whose gradients are chained by hand through the operators' backward calls.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mamba_ssd_chunked_02_gb300 as m2  # noqa: E402


def _randn(*shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, device="cuda") * scale).to(dtype)


class SSDLayer:
    def __init__(self, width, heads, headdim=64, dstate=128, conv_width=4, groups=1, dtype=torch.bfloat16):
        self.h, self.p, self.n, self.g = heads, headdim, dstate, groups
        inner = heads * headdim
        self.inner, self.conv_dim = inner, inner + 2 * groups * dstate
        self.w_in = _randn(inner + self.conv_dim + heads, width, scale=width ** -0.5, dtype=dtype)
        self.w_out = _randn(width, inner, scale=inner ** -0.5, dtype=dtype)
        self.w_conv, self.b_conv = _randn(self.conv_dim, conv_width, scale=0.5), _randn(self.conv_dim, scale=0.1)
        self.A = -torch.exp(torch.rand(heads, device="cuda") * math.log(16))
        self.D, self.dt_bias = torch.ones(heads, device="cuda"), _randn(heads, scale=0.5) - 3
        self.w_norm = torch.ones(inner, device="cuda")

    def _project(self, u):
        """z, the convolution's input and the raw step sizes: column slices of one product."""
        return (u @ self.w_in.t()).split([self.inner, self.conv_dim, self.h], -1)

    def _steps(self, raw, lengths=None):
        dt = torch.nn.functional.softplus(raw.float() + self.dt_bias)
        if lengths is not None:      # a step of 0 leaves the state as it is, whatever the padding holds
            dt = torch.where((torch.arange(dt.shape[1], device="cuda")[None] < lengths[:, None])[..., None], dt, 0.0)
        return dt

    def _heads(self, xbc):
        x, B, C = xbc.split([self.inner, self.g * self.n, self.g * self.n], -1)
        return x.unflatten(-1, (self.h, self.p)), B.unflatten(-1, (self.g, self.n)), C.unflatten(-1, (self.g, self.n))

    def forward(self, u, lengths=None, keep=None):
        """u [b,T,width] -> (output, (conv window, state)); `keep`: a dict for the backward."""
        z, xbc, raw = self._project(u)
        a, window = m2.conv_fwd(xbc, self.w_conv, self.b_conv, None, lengths)
        x, B, C = self._heads(a)
        dt = self._steps(raw, lengths)
        y, state = m2.ssd_fwd(x, dt, self.A, B, C, self.D)
        v = m2.norm_fwd(y.flatten(2), self.w_norm, z)
        if keep is not None:
            keep.update(u=u, z=z, xbc=xbc, raw=raw, a=a, dt=dt, y=y, v=v)
        return v @ self.w_out.t(), (window, state)

    def step(self, u, cache):
        """u [b,width], one token; the cache moves on in place."""
        window, state = cache
        z, xbc, raw = self._project(u)
        x, B, C = self._heads(m2.conv_step(window, xbc, self.w_conv, self.b_conv))
        y = m2.ssd_decode(state, x.contiguous(), self._steps(raw), self.A, B.contiguous(), C.contiguous(), self.D)
        return m2.norm_fwd(y.flatten(1)[:, None], self.w_norm, z[:, None])[:, 0] @ self.w_out.t()

    def backward(self, dout, k):
        """Gradients for dL/d(output) = dout, from what forward kept (no lengths)."""
        io = dout.dtype
        g = {"w_out": torch.einsum("btw,bti->wi", dout.float(), k["v"].float())}
        n = m2.norm_bwd(k["y"].flatten(2), self.w_norm, k["z"], (dout @ self.w_out).contiguous())
        x, B, C = (t.contiguous() for t in self._heads(k["a"]))
        s = m2.ssd_bwd(x, k["dt"], self.A, B, C, self.D, None, n["dx"].view_as(x))
        da = torch.cat([s[name].flatten(2) for name in ("dx", "dB", "dC")], -1).to(io)
        c = m2.conv_bwd(k["xbc"], self.w_conv, self.b_conv, None, da)
        draw = s["ddt"] * torch.sigmoid(k["raw"].float() + self.dt_bias)
        dproj = torch.cat([n["dz"], c["dx"], draw.to(io)], -1)
        g.update(w_norm=n["dw"], A=s["dA"], D=s["dD"], w_conv=c["dw"], b_conv=c["dbias"], dt_bias=draw.sum((0, 1)),
                 w_in=torch.einsum("btp,btw->pw", dproj.float(), k["u"].float()))
        return dproj @ self.w_in, g


class ScanLayer:
    def __init__(self, width, inner, dstate=16, rank=None, conv_width=4, dtype=torch.bfloat16):
        rank = rank or max(1, width // 16)
        self.inner, self.n, self.rank = inner, dstate, rank
        self.w_in = _randn(2 * inner, width, scale=width ** -0.5, dtype=dtype)
        self.w_x = _randn(rank + 2 * dstate, inner, scale=inner ** -0.5, dtype=dtype)
        self.w_dt = _randn(inner, rank, scale=rank ** -0.5, dtype=dtype)
        self.w_out = _randn(width, inner, scale=inner ** -0.5, dtype=dtype)
        self.w_conv, self.b_conv = _randn(inner, conv_width, scale=0.5), _randn(inner, scale=0.1)
        self.A = -torch.arange(1, dstate + 1, device="cuda").float().repeat(inner, 1)
        self.D, self.dt_bias = torch.ones(inner, device="cuda"), _randn(inner, scale=0.5) - 3

    def _inputs(self, x):
        low, B, C = (x @ self.w_x.t()).split([self.rank, self.n, self.n], -1)
        return low @ self.w_dt.t(), B.unflatten(-1, (1, self.n)), C.unflatten(-1, (1, self.n)), low

    def forward(self, u, lengths=None, keep=None):
        xin, z = (u @ self.w_in.t()).chunk(2, -1)
        x, window = m2.conv_fwd(xin, self.w_conv, self.b_conv, None, lengths)
        dt, B, C, low = self._inputs(x)
        y, state = m2.scan_fwd(x, dt, self.A, B, C, self.D, z, self.dt_bias, None, lengths, dt_softplus=True)
        if keep is not None:
            keep.update(u=u, xin=xin, z=z, x=x, dt=dt, B=B, C=C, low=low, y=y)
        return y @ self.w_out.t(), (window, state)

    def step(self, u, cache):
        window, state = cache
        xin, z = (u @ self.w_in.t()).chunk(2, -1)
        x = m2.conv_step(window, xin, self.w_conv, self.b_conv)
        dt, B, C, _ = self._inputs(x)
        y = m2.scan_step(state, x, dt, self.A, B, C, self.D, z, self.dt_bias, dt_softplus=True)
        return y @ self.w_out.t()

    def backward(self, dout, k):
        g = {"w_out": torch.einsum("btw,bti->wi", dout.float(), k["y"].float())}
        s = m2.scan_bwd(k["x"], k["dt"], self.A, k["B"], k["C"], self.D, k["z"], self.dt_bias, None,
                        dout @ self.w_out, dt_softplus=True)
        dlow = torch.cat([s["ddt"] @ self.w_dt, s["dB"].flatten(2), s["dC"].flatten(2)], -1)
        c = m2.conv_bwd(k["xin"], self.w_conv, self.b_conv, None, s["dx"] + dlow @ self.w_x)
        dproj = torch.cat([c["dx"], s["dz"]], -1)
        g.update(A=s["dA"], D=s["dD"], dt_bias=s["ddt_bias"], w_conv=c["dw"], b_conv=c["dbias"],
                 w_dt=torch.einsum("bti,btr->ir", s["ddt"].float(), k["low"].float()),
                 w_x=torch.einsum("btr,bti->ri", dlow.float(), k["x"].float()),
                 w_in=torch.einsum("btp,btw->pw", dproj.float(), k["u"].float()))
        return dproj @ self.w_in, g


def generate(layer, u, prompt, lengths):
    """The padded prompts u[:, :prompt] in one call, then each sequence's next tokens one by one.
    Returns the outputs [b, T, width] as the whole sequence would have them, and the cache."""
    out, cache = layer.forward(u[:, :prompt], lengths)
    out = [out[i, :n] for i, n in enumerate(lengths.tolist())]
    steps = u.shape[1] - prompt
    at = torch.arange(len(out), device="cuda")
    for t in range(steps):
        y = layer.step(u[at, lengths.long() + t], cache)
        out = [torch.cat([o, y[i:i + 1]]) for i, o in enumerate(out)]
    return out, cache


def main():
    torch.manual_seed(0)
    with torch.no_grad():
        for name, layer in (("chunked scan", SSDLayer(256, heads=8)), ("selective scan", ScanLayer(256, 512))):
            u = _randn(3, 200, 256, dtype=torch.bfloat16)
            lengths = torch.tensor([190, 3, 77], dtype=torch.int32, device="cuda")
            got, _ = generate(layer, u, 190, lengths)
            whole, _ = layer.forward(u)
            far = max((g - whole[i, :len(g)]).float().norm().item() / whole[i, :len(g)].float().norm().item()
                      for i, g in enumerate(got))
            keep = {}
            out, _ = layer.forward(u, keep=keep)
            _, grads = layer.backward(out, keep)         # of |out|^2 / 2
            torch.cuda.synchronize()
            print(f"{name}: prompt and tokens differ from the whole sequence by {far:.1e}; gradients: "
                  + ", ".join(f"{k} {v.norm().item():.3g}" for k, v in sorted(grads.items())))


if __name__ == "__main__":
    main()
