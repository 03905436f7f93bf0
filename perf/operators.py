"""Measured cases of the layer operators: the short causal convolution (conv), the
selective scan with a decay per channel and state (scan) and the gated group norm
(norm), each forward, backward and, where it carries state, for single tokens.

`run` computes the plain form in elementary torch operations in fp32 (own = False)
or calls the package (own = True); `exact` computes the definition in fp64, token
by token.
"""
import math

import torch

own = False

# The 2.7B layer of this repository: H P = 80 * 64 = 5120 channels, N = 128, G = 1.
INNER = 80 * 64
XBC = INNER + 2 * 128            # channels the convolution sees: x, B and C side by side
PROJ = INNER + XBC + 80          # columns of the projection they are sliced from: z, x, B, C, dt


def listed():
    return [
        # The 2.7B layer's prompts: x, B and C convolved as one slice of the projection.
        dict(name="conv fwd layer", op="conv", dir="fwd", b=8, T=4096, D=XBC, W=4, pitch=PROJ,
             dtype="bf16", ragged=False, init=False),
        # Prompts of different lengths after a cached prefix, odd channel count, fp32.
        dict(name="conv fwd ragged f32", op="conv", dir="fwd", b=3, T=1021, D=1095, W=3, pitch=1095,
             dtype="f32", ragged=True, init=True),
        # Training the same layer.
        dict(name="conv bwd layer", op="conv", dir="bwd", b=8, T=4096, D=XBC, W=4, pitch=PROJ,
             dtype="bf16", ragged=False, init=False),
        # Generation: one token of 64 sequences.
        dict(name="conv step", op="conv", dir="step", b=64, T=1, D=XBC, W=4, pitch=PROJ,
             dtype="bf16", ragged=False, init=True),
        # The layer's width and prompts with a decay per channel and 16 states each.
        dict(name="scan fwd layer", op="scan", dir="fwd", b=8, T=4096, D=INNER, N=16, G=1,
             dtype="bf16", ragged=False, init=False, gate=True),
        # One long prompt: little to do beside the token axis.
        dict(name="scan fwd long", op="scan", dir="fwd", b=1, T=16384, D=1280, N=16, G=1,
             dtype="bf16", ragged=False, init=False, gate=True),
        # Padded prompts continued from a state, groups, more states, odd sizes, fp32.
        dict(name="scan fwd ragged f32", op="scan", dir="fwd", b=3, T=777, D=1002, N=32, G=2,
             dtype="f32", ragged=True, init=True, gate=False),
        # Training at the layer's width.
        dict(name="scan bwd layer", op="scan", dir="bwd", b=4, T=4096, D=INNER, N=16, G=1,
             dtype="bf16", ragged=False, init=False, gate=True),
        # Generation: one token of eight sequences, where latency counts.
        dict(name="scan step", op="scan", dir="step", b=8, T=1, D=INNER, N=16, G=1,
             dtype="bf16", ragged=False, init=True, gate=True),
        # The norm between the scan and the output projection, prompts.
        dict(name="norm fwd layer", op="norm", dir="fwd", b=8, T=4096, D=INNER, G=1,
             dtype="bf16", gate="first"),
        # ... and its gradient, groups of 640 channels.
        dict(name="norm bwd layer", op="norm", dir="bwd", b=8, T=4096, D=INNER, G=8,
             dtype="bf16", gate="first"),
        # ... and for one token of 64 sequences in fp32, gate after the norm.
        dict(name="norm fwd token f32", op="norm", dir="fwd", b=64, T=1, D=INNER, G=1,
             dtype="f32", gate="after"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, way = rng.choice([("conv", "fwd"), ("conv", "bwd"), ("conv", "step"), ("scan", "fwd"), ("scan", "fwd"),
                          ("scan", "bwd"), ("scan", "step"), ("norm", "fwd"), ("norm", "bwd")])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 4 if dtype == "f32" else 2
    init, ragged = rng.random() < 0.5, rng.random() < 0.4
    b = _log_int(rng, 1, 256) if way == "step" else _log_int(rng, 1, 8)
    T = 1 if way == "step" else _log_int(rng, 1, 16384)
    D = _log_int(rng, 64, XBC)
    if rng.random() < 0.5:
        D = max(80, D // 80 * 80)
    if op == "conv":
        while b * T * D * size > 8 * 4096 * XBC * 2:
            T = max(1, T // 2)
        return dict(op=op, dir=way, b=b, T=T, D=D, W=rng.choice([2, 3, 4]), pitch=D + rng.choice([0, 0, 8, 64, 33]),
                    dtype=dtype, ragged=ragged and way != "step", init=init or way == "step")
    G = rng.choice([1, 1, 2, 4])
    D = max(G, D // G * G)
    if op == "scan":
        N = rng.choice([8, 16, 16, 32, 64])
        most = (4 if way == "bwd" else 8) * 4096 * INNER * 16
        while b * T * D * N > most:
            T = max(1, T // 2)
        return dict(op=op, dir=way, b=b, T=T, D=D, N=N, G=G, dtype=dtype, ragged=ragged and way != "step",
                    init=init or way == "step", gate=rng.random() < 0.6)
    while b * T * D * size > 8 * 4096 * INNER * 2:
        T = max(1, T // 2)
    return dict(op=op, dir=way, b=b, T=T, D=D, G=G, dtype=dtype, gate=rng.choice(["first", "first", "after", "none"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    io = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    f32 = torch.float32

    def randn(*shape, dtype=f32, scale=1.0):
        return torch.randn(*shape, device="cuda", dtype=f32, generator=gen).mul_(scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", dtype=f32, generator=gen)

    b, T, D, way = case["b"], case["T"], case["D"], case["dir"]
    s = dict(case=case)
    if case.get("ragged"):
        # prompts of any part of the padded length, some of them empty, one of them full
        s["lengths"] = (T * (1.1 * uniform(b) - 0.1)).ceil().to(torch.int32).clamp(0, T)
        s["lengths"][0] = T
    else:
        s["lengths"] = None
    if case["op"] == "conv":
        W = case["W"]
        if way == "step":
            s["x"] = randn(b, case["pitch"], dtype=io)[:, :D]
        else:
            s["x"] = randn(b, T, case["pitch"], dtype=io)[:, :, :D]
        s["w"] = (uniform(D, W) * 2 - 1) / math.sqrt(W)
        s["bias"] = (uniform(D) * 2 - 1) / math.sqrt(W)
        s["init"] = randn(b, W - 1, D, dtype=io) if case["init"] else None
        if way == "bwd":
            s["dy"] = randn(b, T, D, dtype=io)
            s["dfinal"] = randn(b, W - 1, D, dtype=io) if case["init"] else None
        return s
    if case["op"] == "norm":
        s["x"] = randn(b, T, D, dtype=io)
        s["z"] = randn(b, T, D, dtype=io) if case["gate"] != "none" else None
        s["w"] = 1.0 + randn(D, scale=0.1)
        if way == "bwd":
            s["dy"] = randn(b, T, D, dtype=io)
        return s
    N, G = case["N"], case["G"]
    lead = (b,) if way == "step" else (b, T)
    s["x"] = randn(*lead, D, dtype=io)
    s["dt"] = randn(*lead, D, dtype=io, scale=0.5)
    # steps of 1e-3 to 1e-1 after the softplus, decays near -1 .. -N
    step = torch.exp(uniform(D) * (math.log(1e-1) - math.log(1e-3)) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=f32) * torch.exp(randn(D, N, scale=0.1))
    s["B"] = randn(*lead, G, N, dtype=io)
    s["C"] = randn(*lead, G, N, dtype=io)
    s["D"] = 1.0 + randn(D, scale=0.1)
    s["z"] = randn(*lead, D, dtype=io) if case["gate"] else None
    s["init"] = randn(b, D, N, scale=0.1) if case["init"] else None
    if way == "bwd":
        s["dy"] = randn(b, T, D, dtype=io)
        s["dfinal"] = randn(b, D, N, scale=0.1) if case["init"] else None
    return s


def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"], case["dir"]](state)
    return _PLAIN[case["op"], case["dir"]](state)


# --- the package's operators, called as a program calls them ---------------------------------

def _own_conv_fwd(s):
    import mamba_ssd_chunked_02_gb300 as m2
    return m2.conv_fwd(s["x"], s["w"], s["bias"], s["init"], s["lengths"], silu=True)


def _own_conv_bwd(s):
    import mamba_ssd_chunked_02_gb300 as m2
    g = m2.conv_bwd(s["x"], s["w"], s["bias"], s["init"], s["dy"], s["dfinal"], s["lengths"], silu=True)
    return {k: v for k, v in g.items() if v is not None}


def _own_conv_step(s):
    import mamba_ssd_chunked_02_gb300 as m2
    return m2.conv_step(s["init"], s["x"], s["w"], s["bias"], silu=True), s["init"]


def _own_scan_fwd(s):
    import mamba_ssd_chunked_02_gb300 as m2
    return m2.scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["init"],
                       s["lengths"], dt_softplus=True)


def _own_scan_bwd(s):
    import mamba_ssd_chunked_02_gb300 as m2
    g = m2.scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["init"], s["dy"],
                    s["dfinal"], s["lengths"], dt_softplus=True)
    return {k: v for k, v in g.items() if v is not None}


def _own_scan_step(s):
    import mamba_ssd_chunked_02_gb300 as m2
    return m2.scan_step(s["init"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                        dt_softplus=True), s["init"]


def _own_norm_fwd(s):
    import mamba_ssd_chunked_02_gb300 as m2
    return m2.norm_fwd(s["x"], s["w"], s["z"], ngroups=s["case"]["G"], eps=EPS, gate_first=s["case"]["gate"] != "after")


def _own_norm_bwd(s):
    import mamba_ssd_chunked_02_gb300 as m2
    g = m2.norm_bwd(s["x"], s["w"], s["z"], s["dy"], ngroups=s["case"]["G"], eps=EPS,
                    gate_first=s["case"]["gate"] != "after")
    return {k: v for k, v in g.items() if v is not None}


_OWN = {("conv", "fwd"): _own_conv_fwd, ("conv", "bwd"): _own_conv_bwd, ("conv", "step"): _own_conv_step,
        ("scan", "fwd"): _own_scan_fwd, ("scan", "bwd"): _own_scan_bwd, ("scan", "step"): _own_scan_step,
        ("norm", "fwd"): _own_norm_fwd, ("norm", "bwd"): _own_norm_bwd}


# --- the plain forms: elementary torch operations in fp32 ------------------------------------

EPS = 1e-5


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _valid(s):
    """[b, T, 1] truth values of the tokens below each sequence's length, or None."""
    if s["lengths"] is None:
        return None
    return (torch.arange(s["x"].shape[1], device="cuda")[None] < s["lengths"][:, None])[..., None]


def _keep(v, valid):
    return v if valid is None else torch.where(valid, v, torch.zeros((), device="cuda"))


def _window(s, x):
    """x (fp32, zero past the lengths) behind its carried window: [b, W - 1 + T, D]."""
    b, _, D = x.shape
    W = s["w"].shape[1]
    init = s["init"].float() if s["init"] is not None else torch.zeros(b, W - 1, D, device="cuda")
    return torch.cat([init, x], 1)


def _last_rows(s, W):
    """Row indices [b, W - 1] of the final window inside _window's result."""
    b, T, _ = s["x"].shape
    ends = s["lengths"].long() if s["lengths"] is not None else torch.full((b,), T, device="cuda")
    return ends[:, None] + torch.arange(W - 1, device="cuda")[None]


def _plain_conv_fwd(s):
    io, W, T = s["x"].dtype, s["w"].shape[1], s["x"].shape[1]
    valid = _valid(s)
    xp = _window(s, _keep(s["x"].float(), valid))
    v = s["bias"] + sum(xp[:, k:k + T] * s["w"][:, k] for k in range(W))
    y = _keep(v * _sigmoid(v), valid).to(io)
    rows = _last_rows(s, W)
    final = xp[torch.arange(len(xp), device="cuda")[:, None], rows].to(io)
    return y, final


def _plain_conv_bwd(s):
    io, W, (b, T, D) = s["x"].dtype, s["w"].shape[1], s["x"].shape
    valid = _valid(s)
    xp = _window(s, _keep(s["x"].float(), valid))
    v = s["bias"] + sum(xp[:, k:k + T] * s["w"][:, k] for k in range(W))
    g = _sigmoid(v)
    dv = _keep(s["dy"].float() * g * (1.0 + v * (1.0 - g)), valid)
    dw = torch.stack([(dv * xp[:, k:k + T]).sum((0, 1)) for k in range(W)], 1)
    padded = torch.nn.functional.pad(dv, (0, 0, W - 1, W - 1))
    dxp = sum(padded[:, W - 1 - k:W - 1 - k + T + W - 1] * s["w"][:, k] for k in range(W))
    if s["dfinal"] is not None:
        at = torch.arange(b, device="cuda")[:, None], _last_rows(s, W)
        dxp[at] += s["dfinal"].float()
    out = dict(dx=_keep(dxp[:, W - 1:], valid).to(io), dw=dw, dbias=dv.sum((0, 1)))
    if s["init"] is not None:
        out["dinit"] = dxp[:, :W - 1].to(io)
    return out


def _plain_conv_step(s):
    xp = torch.cat([s["init"].float(), s["x"].float()[:, None]], 1)
    v = s["bias"] + (xp * s["w"].t()).sum(1)
    s["init"].copy_(xp[:, 1:])
    return (v * _sigmoid(v)).to(s["x"].dtype), s["init"]


def _linear_scan(a, v):
    """h[:, t] = a[:, t] h[:, t - 1] + v[:, t] by doubling, in place (v becomes h)."""
    k, T = 1, a.shape[1]
    while k < T:
        v[:, k:] += a[:, k:] * v[:, :-k]
        a[:, k:] *= a[:, :-k].clone()
        k *= 2
    return v


def _step_sizes(s, valid):
    """dt + dt_bias and its softplus, 0 past the lengths."""
    v = _keep(s["dt"].float(), valid) + s["dt_bias"]
    return v, _keep(torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v))), valid)


def _per_channel(v, D):
    """[.., G, N] -> [.., D, N] fp32: channel d reads group d / (D / G)."""
    return v.float().repeat_interleave(D // v.shape[-2], -2)


def _plain_scan_fwd(s):
    io, (b, T, D), N = s["x"].dtype, s["x"].shape, s["A"].shape[1]
    valid = _valid(s)
    x = _keep(s["x"].float(), valid)
    _, d = _step_sizes(s, valid)
    a = torch.exp(d[..., None] * s["A"])
    u = (d * x)[..., None] * _per_channel(_keep(s["B"].float(), None if valid is None else valid[..., None]), D)
    if s["init"] is not None:
        u[:, 0] += a[:, 0] * s["init"]
    h = _linear_scan(a, u)
    y = (h * _per_channel(_keep(s["C"].float(), None if valid is None else valid[..., None]), D)).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = _keep(s["z"].float(), valid)
        y = y * z * _sigmoid(z)
    return _keep(y, valid).to(io), h[:, -1].clone()


def _plain_scan_bwd(s):
    io, (b, T, D), (_, N) = s["x"].dtype, s["x"].shape, s["A"].shape
    G = s["B"].shape[2]
    valid = _valid(s)
    deep = None if valid is None else valid[..., None]
    x, dy = _keep(s["x"].float(), valid), _keep(s["dy"].float(), valid)
    B, C = _keep(s["B"].float(), deep), _keep(s["C"].float(), deep)
    v, d = _step_sizes(s, valid)
    a = torch.exp(d[..., None] * s["A"])
    u = (d * x)[..., None] * _per_channel(B, D)
    if s["init"] is not None:
        u[:, 0] += a[:, 0] * s["init"]
    h = _linear_scan(a.clone(), u)
    out = {}
    if s["z"] is not None:
        z = _keep(s["z"].float(), valid)
        gz = _sigmoid(z)
        core = (h * _per_channel(C, D)).sum(-1) + s["D"] * x
        out["dz"] = (dy * core * gz * (1.0 + z * (1.0 - gz))).to(io)
        dy = dy * z * gz
    out["dC"] = (dy[..., None] * h).view(b, T, G, D // G, N).sum(3).to(io)
    # the adjoint runs backwards: g_t = C_t dy_t + a_{t + 1} g_{t + 1}
    g = dy[..., None] * _per_channel(C, D)
    if s["dfinal"] is not None:
        g[:, -1] += s["dfinal"]
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1).flip(1)
    g = _linear_scan(later, g.flip(1)).flip(1)
    out["dB"] = ((d * x)[..., None] * g).view(b, T, G, D // G, N).sum(3).to(io)
    q = (g * _per_channel(B, D)).sum(-1)
    if s["init"] is not None:
        out["dinit"] = g[:, 0] * a[:, 0]
    first = s["init"][:, None] if s["init"] is not None else torch.zeros(b, 1, D, N, device="cuda")
    e = g.mul_(a).mul_(torch.cat([first, h[:, :-1]], 1))
    out["dA"] = (e * d[..., None]).sum((0, 1))
    dd = x * q + (e * s["A"]).sum(-1)
    dv = _keep(dd * _sigmoid(v), valid)
    out["dx"] = _keep(d * q + s["D"] * dy, valid).to(io)
    out["ddt"] = dv.to(io)
    out["ddt_bias"] = dv.sum((0, 1))
    out["dD"] = (dy * x).sum((0, 1))
    return out


def _plain_scan_step(s):
    x, D = s["x"].float(), s["x"].shape[1]
    v = s["dt"].float() + s["dt_bias"]
    d = torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))
    h = s["init"]
    h.mul_(torch.exp(d[..., None] * s["A"])).add_((d * x)[..., None] * _per_channel(s["B"], D))
    y = (h * _per_channel(s["C"], D)).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return y.to(s["x"].dtype), h


def _plain_norm_fwd(s):
    x, case = s["x"].float(), s["case"]
    gate = s["z"].float() * _sigmoid(s["z"].float()) if s["z"] is not None else None
    v = x * gate if case["gate"] == "first" else x
    vg = v.view(*v.shape[:-1], case["G"], -1)
    y = (vg * torch.rsqrt((vg * vg).mean(-1, keepdim=True) + EPS)).view_as(v) * s["w"]
    return (y * gate if case["gate"] == "after" else y).to(s["x"].dtype)


def _plain_norm_bwd(s):
    io, x, dy, case = s["x"].dtype, s["x"].float(), s["dy"].float(), s["case"]
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sg = _sigmoid(z)
        gate, dgate = z * sg, sg * (1.0 + z * (1.0 - sg))
    v = x * gate if case["gate"] == "first" else x
    vg = v.view(*v.shape[:-1], case["G"], -1)
    r = torch.rsqrt((vg * vg).mean(-1, keepdim=True) + EPS)
    n = (vg * r).view_as(v)
    if case["gate"] == "after":
        out["dz"] = (dy * n * s["w"] * dgate).to(io)
        dy = dy * gate
    out["dw"] = (dy * n).sum((0, 1))
    wg, ng = (dy * s["w"]).view_as(vg), n.view_as(vg)
    dv = (r * (wg - ng * (wg * ng).mean(-1, keepdim=True))).view_as(v)
    if case["gate"] == "first":
        out["dz"] = (dv * x * dgate).to(io)
        dv = dv * gate
    out["dx"] = dv.to(io)
    return out


_PLAIN = {("conv", "fwd"): _plain_conv_fwd, ("conv", "bwd"): _plain_conv_bwd, ("conv", "step"): _plain_conv_step,
          ("scan", "fwd"): _plain_scan_fwd, ("scan", "bwd"): _plain_scan_bwd, ("scan", "step"): _plain_scan_step,
          ("norm", "fwd"): _plain_norm_fwd, ("norm", "bwd"): _plain_norm_bwd}


# --- what a pass cannot do without -----------------------------------------------------------

def work(case):
    E = 4 if case["dtype"] == "f32" else 2
    b, T, D, way = case["b"], case["T"], case["D"], case["dir"]
    rows = b * T * D
    if case["op"] == "conv":
        W = case["W"]
        state = E * b * (W - 1) * D
        par = 4 * D * (W + 1)
        if way == "bwd":
            ends = 3 * state if case["init"] else 0
            return {"bytes": 3 * E * rows + 2 * par + ends, "flops": rows * (6 * W + 12)}
        return {"bytes": 2 * E * rows + par + state * (2 if case["init"] else 1), "flops": rows * (2 * W + 5)}
    if case["op"] == "norm":
        gate = case["gate"] != "none"
        if way == "bwd":
            return {"bytes": E * rows * (3 + 2 * gate) + 8 * D, "flops": rows * (10 + 12 * gate)}
        return {"bytes": E * rows * (2 + gate) + 4 * D, "flops": rows * (4 + 6 * gate)}
    N, G = case["N"], case["G"]
    bc = 2 * E * b * T * G * N
    par = 4 * D * (N + 2)
    state = 4 * b * D * N
    each = rows * N
    if way == "bwd":
        return {"bytes": E * rows * (5 + 2 * case["gate"]) + 2 * bc + 2 * par + (3 * state if case["init"] else 0),
                "flops": each * 20}
    return {"bytes": E * rows * (3 + case["gate"]) + bc + par + state * (2 if case["init"] else 1), "flops": each * 7}


# --- the definitions in fp64, token by token -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](case, s)


def _f64(v):
    return v.double() if v is not None else None


def _silu64(v):
    """silu and its derivative."""
    g = torch.sigmoid(v)
    return v * g, g + v * g * (1.0 - g)


def _exact_conv(case, s):
    W, way = case["W"], case["dir"]
    x = _f64(s["x"])[:, None] if way == "step" else _f64(s["x"])
    b, T, D = x.shape
    w, bias = _f64(s["w"]), _f64(s["bias"])
    ends = s["lengths"].tolist() if s["lengths"] is not None else [T] * b
    init = _f64(s["init"]) if s["init"] is not None else x.new_zeros(b, W - 1, D)
    y, final = x.new_zeros(b, T, D), torch.empty_like(init)
    dx, dinit = x.new_zeros(b, T, D), torch.zeros_like(init)
    dw, dbias = torch.zeros_like(w), torch.zeros_like(bias)
    for i, n in enumerate(ends):                       # one sequence at a time
        seen = torch.cat([init[i], x[i, :n]])          # [W - 1 + n, D]
        near = seen.unfold(0, W, 1)                    # [n, D, W]
        out, slope = _silu64((near * w).sum(-1) + bias)
        y[i, :n], final[i] = out, seen[n:]
        if way == "bwd":
            ds = _f64(s["dy"][i, :n]) * slope
            dw += (near * ds[..., None]).sum(0)
            dbias += ds.sum(0)
            dseen = torch.zeros_like(seen)
            for k in range(W):
                dseen[k:k + n] += ds * w[:, k]
            if s["dfinal"] is not None:
                dseen[n:] += _f64(s["dfinal"][i])
            dinit[i], dx[i, :n] = dseen[:W - 1], dseen[W - 1:]
    if way == "step":
        return y[:, 0], final
    if way == "fwd":
        return y, final
    out = dict(dx=dx, dw=dw, dbias=dbias)
    if s["init"] is not None:
        out["dinit"] = dinit
    return out


def _exact_scan(case, s):
    way, N, G, D = case["dir"], case["N"], case["G"], case["D"]
    names = ("x", "dt", "B", "C", "z") + (("dy",) if way == "bwd" else ())
    t = {k: (_f64(s[k])[:, None] if way == "step" else _f64(s[k])) if s[k] is not None else None for k in names}
    b, T = t["x"].shape[:2]
    if s["lengths"] is not None:
        past = torch.arange(T, device="cuda")[None] >= s["lengths"][:, None]
        for k in names:
            if t[k] is not None:
                t[k][past] = 0.0
    A, skip, bias = _f64(s["A"]), _f64(s["D"]), _f64(s["dt_bias"])
    raw = t["dt"] + bias
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    if s["lengths"] is not None:
        step[past] = 0.0
    size = D // G

    def wide(v):                                       # [b, G, N] -> [b, D, N]
        return v[:, :, None].expand(b, G, size, N).reshape(b, D, N)

    h = _f64(s["init"]) if s["init"] is not None else A.new_zeros(b, D, N)
    states = [h] if way == "bwd" else None
    core = torch.empty_like(t["x"])
    for i in range(T):
        d, x = step[:, i, :, None], t["x"][:, i, :, None]
        h = torch.exp(d * A) * h + d * x * wide(t["B"][:, i])
        core[:, i] = (h * wide(t["C"][:, i])).sum(-1)
        if states is not None:
            states.append(h)
    core += skip * t["x"]
    gate, slope = _silu64(t["z"]) if t["z"] is not None else (None, None)
    if way != "bwd":
        y = core * gate if gate is not None else core
        if s["lengths"] is not None:
            y[past] = 0.0
        return (y[:, 0], h) if way == "step" else (y, h)
    out = {}
    dy = t["dy"]
    if gate is not None:
        out["dz"] = dy * core * slope
        dy = dy * gate
    g = _f64(s["dfinal"]) if s["dfinal"] is not None else torch.zeros_like(h)
    dA = torch.zeros_like(A)
    dB, dC = torch.zeros_like(t["B"]), torch.zeros_like(t["C"])
    dstep, dx = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    for i in range(T - 1, -1, -1):
        d, x, h = step[:, i, :, None], t["x"][:, i, :, None], states.pop()
        g = g + dy[:, i, :, None] * wide(t["C"][:, i])
        dC[:, i] = (h * dy[:, i, :, None]).view(b, G, size, N).sum(2)
        dB[:, i] = (g * d * x).view(b, G, size, N).sum(2)
        q = (g * wide(t["B"][:, i])).sum(-1)
        g = g * torch.exp(d * A)
        e = g * states[-1]
        dA += (e * d).sum(0)
        dstep[:, i] = x[..., 0] * q + (e * A).sum(-1)
        dx[:, i] = d[..., 0] * q
    dx += skip * dy
    draw_ = dstep * torch.sigmoid(raw)
    if s["lengths"] is not None:
        draw_[past] = 0.0
    out.update(dx=dx, ddt=draw_, dA=dA, dB=dB, dC=dC, dD=(dy * t["x"]).sum((0, 1)), ddt_bias=draw_.sum((0, 1)))
    if s["init"] is not None:
        out["dinit"] = g
    return out


def _exact_norm(case, s):
    """By autograd of the definition in fp64, a slice of the rows at a time."""
    G, D = case["G"], case["D"]
    flat = {k: s[k].view(-1, D) for k in ("x", "z", "dy") if s.get(k) is not None}
    w = _f64(s["w"]).requires_grad_()
    ys, dxs, dzs, dw = [], [], [], torch.zeros_like(w)
    for at in range(0, flat["x"].shape[0], 4096):
        x = _f64(flat["x"][at:at + 4096]).requires_grad_()
        z = _f64(flat["z"][at:at + 4096]).requires_grad_() if "z" in flat else None
        gate = torch.nn.functional.silu(z) if z is not None else 1.0
        v = (x * gate if case["gate"] == "first" else x).reshape(-1, G, D // G)
        y = (v / (v.square().mean(-1, keepdim=True) + EPS).sqrt()).reshape(-1, D) * w
        y = y * gate if case["gate"] == "after" else y
        if case["dir"] == "fwd":
            ys.append(y.detach())
            continue
        inputs = [x, w] + ([z] if z is not None else [])
        got = torch.autograd.grad(y, inputs, _f64(flat["dy"][at:at + 4096]))
        dxs.append(got[0])
        dw += got[1]
        dzs += got[2:]
    if case["dir"] == "fwd":
        return torch.cat(ys).view(s["x"].shape)
    out = dict(dx=torch.cat(dxs).view(s["x"].shape), dw=dw.detach())
    if s["z"] is not None:
        out["dz"] = torch.cat(dzs).view(s["x"].shape)
    return out
