"""Measured cases of the operators around a layer's projections: the norm that takes the
residual in (add_norm), e4m3 values with power-of-two scales (quant8) and the matrix
product of such values (proj8), forward and backward, for prompts and for single tokens.

`run` computes the plain form in elementary torch operations in fp32 (own = False)
or calls the package (own = True); `exact` computes the definition in fp64.

Quantising a group of values: s = 2^e with the smallest whole e >= -127 for which
max|x| <= 448 s, q = x / s rounded to e4m3.  Groups are 128 neighbours of a row
("row"), or 128 x 128 blocks ("block"); the backward product also takes 128 rows of
one column.
"""
import math

import torch

own = False

# The 2.7B layer of this repository: 80 heads of 64 channels, N = 128, G = 1, in a model half as wide.
INNER = 80 * 64
WIDTH = INNER // 2
PROJ = 2 * INNER + 2 * 128 + 80  # columns of the input projection: z, x, B, C, dt
TOKENS = 8 * 4096
EPS = 1e-5


def listed():
    return [
        # Before the layer's input projection, prompts: residual kept in fp32, output as the product takes it.
        dict(name="add_norm fwd layer 8bit", op="add_norm", dir="fwd", b=8, T=4096, D=WIDTH, dtype="bf16",
             res="f32", quant=True),
        # The same for one token of one sequence: the smallest call.
        dict(name="add_norm fwd token 8bit", op="add_norm", dir="fwd", b=1, T=1, D=WIDTH, dtype="bf16",
             res="f32", quant=True),
        # Odd width, everything fp32, no 8 bits (the last norm before the output head).
        dict(name="add_norm fwd odd f32", op="add_norm", dir="fwd", b=3, T=1021, D=1095, dtype="f32",
             res="f32", quant=False),
        # Training the layer.
        dict(name="add_norm bwd layer", op="add_norm", dir="bwd", b=8, T=4096, D=WIDTH, dtype="bf16",
             res="f32", quant=False),
        # The gated norm's output before the output projection, prompts.
        dict(name="quant8 rows layer", op="quant8", group="row", M=TOKENS, D=INNER, dtype="bf16"),
        # The input projection's weights after an optimizer's step.
        dict(name="quant8 blocks weight", op="quant8", group="block", M=PROJ, D=WIDTH, dtype="f32"),
        # The input projection of prompts.
        dict(name="proj8 fwd layer", op="proj8", dir="fwd", M=TOKENS, K=WIDTH, N=PROJ, dtype="bf16"),
        # Odd sizes everywhere, fp32 results (logits).
        dict(name="proj8 fwd odd f32", op="proj8", dir="fwd", M=777, K=1095, N=5003, dtype="f32"),
        # Generation: the input projection of one token.
        dict(name="proj8 fwd token", op="proj8", dir="fwd", M=1, K=WIDTH, N=PROJ, dtype="bf16"),
        # Generation: the output projection of one token of 64 sequences.
        dict(name="proj8 fwd 64 tokens", op="proj8", dir="fwd", M=64, K=INNER, N=WIDTH, dtype="bf16"),
        # Training the input projection.
        dict(name="proj8 bwd layer", op="proj8", dir="bwd", M=TOKENS, K=WIDTH, N=PROJ, dtype="bf16"),
        # Training a narrow odd layer on short sequences, gradients in fp32.
        dict(name="proj8 bwd odd f32", op="proj8", dir="bwd", M=1500, K=1095, N=1002, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    n = _log_int(rng, lo, hi)
    return max(lo, n // 16 * 16) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["add_norm", "add_norm", "quant8", "proj8", "proj8", "proj8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "add_norm":
        way = rng.choice(["fwd", "fwd", "bwd"])
        b, T, D = _log_int(rng, 1, 64), _log_int(rng, 1, 16384), _width(rng, 64, 8192)
        while b * T * D > TOKENS * WIDTH:
            b, T = max(1, b // 2), max(1, T // 2)
        return dict(op=op, dir=way, b=b, T=T, D=D, dtype=dtype, res="f32" if dtype == "f32" else rng.choice(["f32", "bf16"]),
                    quant=way == "fwd" and rng.random() < 0.6)
    if op == "quant8":
        M, D = _log_int(rng, 1, TOKENS), _width(rng, 64, PROJ)
        while M * D > TOKENS * INNER:
            M //= 2
        return dict(op=op, group=rng.choice(["row", "row", "block"]), M=M, D=D, dtype=dtype)
    way = rng.choice(["fwd", "fwd", "bwd"])
    M, K, N = _log_int(rng, 1, TOKENS), _width(rng, 64, PROJ), _width(rng, 64, PROJ)
    while M * K * N > TOKENS * WIDTH * PROJ:
        M //= 2
    return dict(op=op, dir=way, M=M, K=K, N=N, dtype=dtype)


# --- inputs ----------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    types = dict(f32=torch.float32, bf16=torch.bfloat16)
    io = types[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(*shape, device="cuda", generator=gen).mul_(scale).to(dtype)

    def channels(n):
        """Sizes of a hidden state's channels: alike but for a few large ones."""
        return torch.where(torch.rand(n, device="cuda", generator=gen) < 0.01, 30.0, 1.0) * (1 + randn(n, scale=0.2))

    def pitched(q):
        """8-bit operands have rows of whole 16 bytes."""
        room = torch.zeros(q.shape[0], -(-q.shape[1] // 16) * 16, dtype=q.dtype, device="cuda")
        room[:, :q.shape[1]].view(torch.uint8).copy_(q.view(torch.uint8))
        return room[:, :q.shape[1]]

    s = dict(case=case)
    if case["op"] == "add_norm":
        b, T, D = case["b"], case["T"], case["D"]
        s["x"] = (randn(b, T, D) * channels(D)).to(io)
        s["residual"] = (randn(b, T, D, scale=3.0) * channels(D)).to(types[case["res"]])
        s["w"] = 1.0 + randn(D, scale=0.2)
        if case["dir"] == "bwd":
            s["dy"], s["dtotal"] = randn(b, T, D, dtype=io), randn(b, T, D, dtype=types[case["res"]])
        return s
    if case["op"] == "quant8":
        M, D = case["M"], case["D"]
        s["x"] = randn(M, D, scale=D ** -0.5, dtype=io) if case["group"] == "block" else (randn(M, D) * channels(D)).to(io)
        return s
    M, K, N = case["M"], case["K"], case["N"]
    q, s["xs"] = _plain_quant(randn(M, K) * channels(K), 1, 128)
    s["xq"] = pitched(q)
    q, s["ws"] = _plain_quant(randn(N, K, scale=K ** -0.5), 128, 128)
    s["wq"] = pitched(q)
    if case["dir"] == "bwd":
        s["dy"] = (randn(M, N) * torch.exp(randn(M, 1))).mul_(1e-3).to(io)
    return s


def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"], case.get("dir")](state)
    return _PLAIN[case["op"], case.get("dir")](state)


# --- the package's operators, called as a program calls them ---------------------------------

def _own_add_norm_fwd(s):
    import mamba_ssd_chunked_02_gb300 as m2
    if s["case"]["quant"]:
        q, scale, total = m2.add_norm_fwd(s["x"], s["residual"], s["w"], eps=EPS, quant=True)
        return dict(q=q, s=scale, total=total)
    y, total = m2.add_norm_fwd(s["x"], s["residual"], s["w"], eps=EPS)
    return dict(y=y, total=total)


def _own_add_norm_bwd(s):
    import mamba_ssd_chunked_02_gb300 as m2
    g = m2.add_norm_bwd(s["residual"], s["w"], s["dy"], s["dtotal"], eps=EPS)
    return dict(dx=g["dx"], dresidual=g["dresidual"], dw=g["dw"])


def _own_quant8(s):
    import mamba_ssd_chunked_02_gb300 as m2
    q, scale = m2.quant8(s["x"], group=s["case"]["group"])
    return dict(q=q, s=scale)


def _own_proj8_fwd(s):
    import mamba_ssd_chunked_02_gb300 as m2
    return m2.proj8_fwd(s["xq"], s["xs"], s["wq"], s["ws"],
                        dtype=torch.float32 if s["case"]["dtype"] == "f32" else torch.bfloat16)


def _own_proj8_bwd(s):
    import mamba_ssd_chunked_02_gb300 as m2
    g = m2.proj8_bwd(s["dy"], s["xq"], s["xs"], s["wq"], s["ws"])
    return dict(dx=g["dx"], dw=g["dw"])


_OWN = {("add_norm", "fwd"): _own_add_norm_fwd, ("add_norm", "bwd"): _own_add_norm_bwd, ("quant8", None): _own_quant8,
        ("proj8", "fwd"): _own_proj8_fwd, ("proj8", "bwd"): _own_proj8_bwd}


# --- the plain forms: elementary torch operations in fp32 ------------------------------------

def _blocks(x, rows, cols):
    """x [m, n] as [m / rows, rows, n / cols, cols], zeros behind its ends."""
    m, n = x.shape
    x = torch.nn.functional.pad(x, (0, -n % cols, 0, -m % rows))
    return x.view(x.shape[0] // rows, rows, x.shape[1] // cols, cols)


def _plain_quant(x, rows, cols):
    """x [m, n] fp32 -> (q [m, n], s [m / rows, n / cols])."""
    parts = _blocks(x, rows, cols)
    top = parts.abs().amax((1, 3))
    part, e = torch.frexp(top)                       # 448 = 0.875 * 2^9
    e = torch.where(top > 0, torch.where(part > 0.875, e - 8, e - 9), -127).clamp(min=-127)
    q = torch.ldexp(parts, -e[:, None, :, None]).view(parts.shape[0] * rows, -1)[:x.shape[0], :x.shape[1]]
    return q.contiguous().to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_dequant(q, s, rows, cols):
    scale = torch.exp2(s.view(torch.uint8).float() - 127.0)
    return (_blocks(q.float(), rows, cols) * scale[:, None, :, None]).view(scale.shape[0] * rows, -1)[:q.shape[0], :q.shape[1]]


def _plain_add_norm_fwd(s):
    total = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    v = total.float()
    y = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["w"]
    if not s["case"]["quant"]:
        return dict(y=y.to(s["x"].dtype), total=total)
    q, scale = _plain_quant(y.flatten(0, 1), 1, 128)
    return dict(q=q.view(y.shape), s=scale.view(*y.shape[:2], -1), total=total)


def _plain_add_norm_bwd(s):
    v, dy = s["residual"].float(), s["dy"].float()
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    n, g = v * r, dy * s["w"]
    d = r * (g - n * (g * n).mean(-1, keepdim=True)) + s["dtotal"].float()
    return dict(dx=d.to(s["dy"].dtype), dresidual=d.to(s["residual"].dtype), dw=(dy * n).sum((0, 1)))


def _plain_quant8(s):
    q, scale = _plain_quant(s["x"].float(), *((1, 128) if s["case"]["group"] == "row" else (128, 128)))
    return dict(q=q, s=scale)


def _plain_proj8_fwd(s):
    x, w = _plain_dequant(s["xq"], s["xs"], 1, 128), _plain_dequant(s["wq"], s["ws"], 128, 128)
    return (x @ w.t()).to(torch.float32 if s["case"]["dtype"] == "f32" else torch.bfloat16)


def _plain_proj8_bwd(s):
    x, w, dy = _plain_dequant(s["xq"], s["xs"], 1, 128), _plain_dequant(s["wq"], s["ws"], 128, 128), s["dy"].float()
    along, across = _plain_dequant(*_plain_quant(dy, 1, 128), 1, 128), _plain_dequant(*_plain_quant(dy, 128, 1), 128, 1)
    seen = _plain_dequant(*_plain_quant(x, 128, 1), 128, 1)
    return dict(dx=(along @ w).to(s["dy"].dtype), dw=across.t() @ seen)


_PLAIN = {("add_norm", "fwd"): _plain_add_norm_fwd, ("add_norm", "bwd"): _plain_add_norm_bwd,
          ("quant8", None): _plain_quant8, ("proj8", "fwd"): _plain_proj8_fwd, ("proj8", "bwd"): _plain_proj8_bwd}


# --- what a pass cannot do without -----------------------------------------------------------

def work(case):
    E = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "add_norm":
        R = 4 if case["res"] == "f32" else 2
        D, rows = case["D"], case["b"] * case["T"]
        if case["dir"] == "bwd":
            return {"bytes": rows * D * (R + E + R + E + (R if R != E else 0)) + 8 * D, "flops": rows * D * 12}
        out = rows * (D + -(-D // 128)) if case["quant"] else rows * D * E
        return {"bytes": rows * D * (E + 2 * R) + out + 4 * D, "flops": rows * D * (7 if case["quant"] else 5)}
    if case["op"] == "quant8":
        M, D = case["M"], case["D"]
        groups = M * -(-D // 128) if case["group"] == "row" else -(-M // 128) * -(-D // 128)
        return {"bytes": M * D * (E + 1) + groups, "flops": 2 * M * D}
    M, K, N = case["M"], case["K"], case["N"]
    kb, nb = -(-K // 128), -(-N // 128)
    operands = M * (K + kb) + N * K + nb * kb
    if case["dir"] == "bwd":
        return {"bytes": operands + E * M * (N + K) + 4 * N * K, "flops": 4 * M * N * K}
    return {"bytes": operands + E * M * N, "flops": 2 * M * N * K}


# --- the definitions in fp64 -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"add_norm": _exact_add_norm, "quant8": _exact_quant8, "proj8": _exact_proj8}[case["op"]](case, s)


def _group_top(v, dim):
    """max|v| over each 128 neighbours along dim, for every value of v."""
    tops = torch.cat([c.abs().amax(dim, keepdim=True) for c in v.split(128, dim)], dim)
    return tops


def _exact_round(v, dims):
    """v [m, n] fp64 in groups of 128 along each of dims -> (q, s) as fp64 values."""
    top = v
    for d in (0, 1):
        top = _group_top(top, d) if d in dims else top
    part, e = torch.frexp(top.abs() / 448.0)         # part in [1/2, 1)
    scale = torch.exp2((e - (part <= 0.5).int()).clamp(min=-127).double())
    scale = torch.where(top == 0, 2.0 ** -127, scale)
    wide = scale
    for d in dims:
        wide = wide.repeat_interleave(128, d).narrow(d, 0, v.shape[d])
    u = v / wide
    # e4m3: 4 significant bits down to 2^-6, steps of 2^-9 below; torch.round takes ties to even
    step = torch.exp2(torch.frexp(u.abs().clamp(min=2.0 ** -6))[1].double() - 4.0)
    return torch.round(u / step) * step, scale


def _spread(q, s, dims):
    s = s.double()
    for d in dims:
        s = s.repeat_interleave(128, d).narrow(d, 0, q.shape[d])
    return q.double() * s


def _exact_add_norm(case, s):
    """The backward by autograd of the definition."""
    if case["dir"] == "fwd":
        total = (s["x"].double() + s["residual"].double()).to(s["residual"].dtype).double()
        y = total / (total.square().mean(-1, keepdim=True) + EPS).sqrt() * s["w"].double()
        if not case["quant"]:
            return dict(y=y, total=total)
        q, scale = _exact_round(y.flatten(0, 1), (1,))
        return dict(q=q.view(y.shape), s=scale.view(*y.shape[:2], -1), total=total)
    total, w = s["residual"].double().requires_grad_(), s["w"].double().requires_grad_()
    y = total / (total.square().mean(-1, keepdim=True) + EPS).sqrt() * w
    d, dw = torch.autograd.grad([y, total * 1.0], [total, w], [s["dy"].double(), s["dtotal"].double()])
    return dict(dx=d, dresidual=d, dw=dw)


def _exact_quant8(case, s):
    q, scale = _exact_round(s["x"].double(), (1,) if case["group"] == "row" else (0, 1))
    return dict(q=q, s=scale)


def _exact_proj8(case, s):
    x, w = _spread(s["xq"], s["xs"], (1,)), _spread(s["wq"], s["ws"], (0, 1))
    if case["dir"] == "fwd":
        return x @ w.t()
    dy = s["dy"].double()
    dx = _spread(*_exact_round(dy, (1,)), (1,)) @ w
    return dict(dx=dx, dw=_spread(*_exact_round(dy, (0,)), (0,)).t() @ _spread(*_exact_round(x, (0,)), (0,)))
