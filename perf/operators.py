"""Measured cases of the transformer-block operators around a microscaled 4-bit linear layer: the
norms before and after a block with its gate and residual scale, MXFP4 quantization, the MXFP4 +
low-rank linear layer, and a norm that quantizes its result for the next layer.

``run`` computes each operator in plain torch operations (``own`` false) or by the package's calls
(``own`` true). Sizes are those of the synthetic workloads (1024^2 and 2048^2 images of 16x16-pixel
tokens plus 512 text tokens, hidden size 3072, MLP width 12288, branch rank 32) and generic ones.
"""
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TYPES = {"bf16": BF16, "f32": F32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token's norm (a text token, a pooled embedding): launch latency
        dict(name="norm_token", op="norm", B=1, T=1, D=3072, kind="rms", affine=True, mod=False, x="bf16", mods="bf16"),
        # the modulated LayerNorm in front of the fused QKV layer of a 1024^2 image
        dict(name="norm_1024", op="norm", B=1, T=4608, D=3072, kind="layer", affine=False, mod=True, x="bf16",
             mods="bf16"),
        # end of a 2048^2 attention block for two guidance branches: post-norm, gate, residual and the MLP's norm
        dict(name="residual_2048", op="residual", B=2, T=16896, D=3072, post="rms", kind="layer", packed=False,
             x="bf16", y="bf16", mods="bf16", res=1.0),
        # packed images of several sizes, fp32 residual stream, a width that fills no power of two, rows behind the
        # last image that stay as they were
        dict(name="residual_packed", op="residual", B=5, T=1201, D=1544, post="", kind="rms", packed=True, x="f32",
             y="bf16", mods="f32", res=0.5),
        # MXFP4 activations of the MLP's down layer at 1024^2 and the values they stand for (calibration error)
        dict(name="quantize_down_1024", op="quantize", M=4608, K=12288),
        # a short odd-sized batch
        dict(name="quantize_odd", op="quantize", M=333, K=1000),
        # one token through the QKV layer (the conditioning path): weight traffic and latency
        dict(name="linear_token", op="linear", M=1, K=3072, N=9216, r=32, bias=True, swiglu=False),
        # the 2048^2 QKV layer
        dict(name="linear_qkv_2048", op="linear", M=16896, K=3072, N=9216, r=32, bias=False, swiglu=False),
        # the 1024^2 gate/up layer with its SwiGLU
        dict(name="linear_gate_up_1024", op="linear", M=4608, K=3072, N=24576, r=32, bias=True, swiglu=True),
        # sizes that fill no tile
        dict(name="linear_odd", op="linear", M=777, K=1608, N=2344, r=16, bias=True, swiglu=False),
        # a block's end and the next layer without a branch, 1024^2: gate + residual + norm quantized in one pass, then
        # the product
        dict(name="block_qkv_1024", op="block", B=1, T=4608, D=3072, N=9216, post="rms", kind="layer"),
        # the same for a few tokens of two samples
        dict(name="block_few", op="block", B=2, T=12, D=3072, N=3072, post="", kind="rms"),
    ]


def _log(rng, lo, hi, step=1):
    import math
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(("norm", "residual", "quantize", "linear", "linear", "block"))
    if op == "norm":
        D = _log(rng, 64, 8192, rng.choice((1, 8, 64)))
        return dict(op=op, B=rng.randint(1, 4), T=_log(rng, 1, min(16896, 25_000_000 // D)), D=D,
                    kind=rng.choice(("rms", "layer")), affine=rng.random() < 0.5, mod=rng.random() < 0.7,
                    x=rng.choice(("bf16", "f32")), mods=rng.choice(("bf16", "f32")))
    if op == "residual":
        D = _log(rng, 64, 8192, rng.choice((1, 8, 64)))
        return dict(op=op, B=rng.randint(1, 6), T=_log(rng, 1, min(8448, 16_000_000 // D)), D=D,
                    post=rng.choice(("", "rms", "layer")), kind=rng.choice(("rms", "layer")),
                    packed=rng.random() < 0.4, x=rng.choice(("bf16", "f32")), y=rng.choice(("bf16", "bf16", "f32")),
                    mods=rng.choice(("bf16", "f32")), res=rng.choice((1.0, 0.5)))
    if op == "quantize":
        K = _log(rng, 64, 12288, 8)
        return dict(op=op, M=_log(rng, 1, min(16896, 50_000_000 // K)), K=K)
    K = _log(rng, 256, 6144, rng.choice((8, 64, 256)))
    if op == "linear":
        swiglu = rng.random() < 0.35
        N = _log(rng, 128, 12288, rng.choice((16, 128, 768)))
        return dict(op=op, M=_log(rng, 1, min(16896, 300_000_000_000 // (K * N))), K=K, N=N,
                    r=rng.choice((0, 16, 32, 64)), bias=rng.random() < 0.6, swiglu=swiglu)
    N = _log(rng, 128, 9216, rng.choice((8, 128, 768)))
    return dict(op=op, B=rng.randint(1, 3), T=_log(rng, 1, min(4096, 100_000_000_000 // (K * N))), D=K, N=N, post=rng.choice(("", "rms", "layer")),
                kind=rng.choice(("rms", "layer")))


# ---------------------------------------------------------------- inputs

def _normal(g, *shape, std=1.0, dtype=BF16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32).mul_(std).to(dtype)


def _stream(g, rows, D, dtype):
    """Activations with 1 % outlier channels, as the diffusion transformer's layers see them."""
    x = torch.randn(rows, D, generator=g, device="cuda", dtype=F32)
    n = max(1, D // 100)
    x[:, torch.randperm(D, generator=g, device="cuda")[:n]] *= 50.0
    return x.to(dtype)


def _norm_inputs(g, s, case, D):
    s["eps"] = 1e-6
    s["w"] = s["b"] = s["pw"] = s["pb"] = None
    if case.get("affine", True):
        s["w"] = _normal(g, D, std=0.1, dtype=F32).add_(1.0)
        s["b"] = _normal(g, D, std=0.1, dtype=F32) if case["kind"] == "layer" else None
    if case.get("post"):
        s["pw"] = _normal(g, D, std=0.1, dtype=F32).add_(1.0)
        s["pb"] = _normal(g, D, std=0.1, dtype=F32) if case["post"] == "layer" else None
    dt = TYPES[case.get("mods", "bf16")]
    # gate, scale and shift are thirds of one conditioning output, as a modulation layer writes them
    m = _normal(g, case["B"], 3 * D, std=0.5, dtype=dt)
    s["gate"], s["scale"], s["shift"] = m[:, :D], m[:, D:2 * D], m[:, 2 * D:]
    if not case.get("mod", True):
        s["scale"] = s["shift"] = None


def _weight_inputs(g, s, K, N, r, bias):
    """A prepared layer: smoothing reciprocals of channels with outliers, a smoothed residual, a branch."""
    lam = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 7.0, 1.0) * K ** 0.25
    s["inv_lambda"] = (1.0 / lam).to(F32)
    s["R"] = _normal(g, N, K, std=K ** -0.5, dtype=F32) * lam
    s["L1s"] = _normal(g, K, r, std=K ** -0.5) if r else None
    s["L2"] = _normal(g, r, N, std=0.05) if r else None
    s["bias"] = _normal(g, N, std=0.14) if bias else None


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("norm", "residual", "block"):
        B, T, D = case["B"], case["T"], case["D"]
        packed = case.get("packed", False)
        rows = B * T + (7 if packed else 0)
        x = _stream(g, rows, D, TYPES[case.get("x", "bf16")])
        s["x"] = x if packed else x.view(B, T, D)
        _norm_inputs(g, s, case, D)
        if op != "norm":
            y = _normal(g, rows, D, std=2.0, dtype=TYPES[case.get("y", "bf16")])
            s["y"] = y if packed else y.view(B, T, D)
        s["offsets"] = None
        if packed:  # sample lengths from the seed (an empty one among them where B allows), then 7 rows of nothing
            cuts = torch.randint(0, B * T + 1, (B - 1,), generator=g, device="cuda").sort().values
            end = torch.tensor([B * T], device="cuda")
            s["offsets"] = torch.cat([end - end, cuts, end]).to(torch.int32)
            s["out"], s["h"] = torch.zeros_like(x), torch.zeros(rows, D, device="cuda", dtype=BF16)
    if op == "block":
        _weight_inputs(g, s, case["D"], case["N"], 0, False)
    if op in ("quantize", "linear"):
        s["X"] = _stream(g, case["M"], case["K"], BF16)
        _weight_inputs(g, s, case["K"], case.get("N", 128), case.get("r", 0), case.get("bias", False))
    if own:
        _handles(s, case)
    elif "R" in s and op != "quantize":
        s["Wq"] = _mx_values(s["R"])  # the packed weight's values: packing is no part of a call
    return s


def _handles(s, case):
    """What a program keeps between calls: the norms, the packed weight, the quantized-activation buffer."""
    import bit_diffusion_transformer_svdquant_b200 as svdq
    s["lib"] = svdq
    if "kind" in case:
        s["norm"] = svdq.Norm(case["kind"], s["w"], s["b"], s["eps"])
        s["post"] = svdq.Norm(case["post"], s["pw"], s["pb"], s["eps"]) if case.get("post") else None
    if "R" in s:
        s["weight"] = svdq.MxWeight(s["R"], s["L1s"], s["L2"], s["inv_lambda"], swiglu=case.get("swiglu", False))
        M, K = (case["M"], case["K"]) if "M" in case else (case["B"] * case["T"], case["D"])
        s["act"] = svdq.MxAct(M, K, case.get("r", 0), "cuda")


# ---------------------------------------------------------------- plain forms, 32 bits

def _normed(v, kind, w, b, eps):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)
    if w is not None:
        v = v * w
    return v if b is None else v + b


def _per_row(m, s, rows):
    """A per-sample vector for every row: by the packed rows' samples, or broadcast over a sample's rows."""
    if s["offsets"] is None:
        return m.float()[:, None, :]
    at = torch.searchsorted(s["offsets"], torch.arange(rows, device="cuda", dtype=torch.int32), right=True) - 1
    return m.float()[at.clamp(max=m.shape[0] - 1)]


def _plain_norm(s, v):
    case, rows = s["case"], v.shape[0]
    h = _normed(v, case["kind"], s["w"], s["b"], s["eps"])
    if s["scale"] is not None:
        h = h * (1.0 + _per_row(s["scale"], s, rows)) + _per_row(s["shift"], s, rows)
    return h


def _plain_residual(s):
    case, y = s["case"], s["y"].float()
    if case["post"]:
        y = _normed(y, case["post"], s["pw"], s["pb"], s["eps"])
    return s["x"].float() + case.get("res", 1.0) * _per_row(s["gate"], s, y.shape[0]) * y


def _mx_values(v):
    """fp32 values -> the MXFP4 values they round to: blocks of 32 along the last axis share the scale
    2^(floor(log2(max)) - 2), elements round to {0, .5, 1, 1.5, 2, 3, 4, 6} with ties to the even code."""
    rows, K = v.shape
    b = torch.nn.functional.pad(v, (0, -K % 32)).view(rows, -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top).exponent - 3).clamp(min=-127)
    e = torch.where(top > 0, e, -127)
    a = torch.ldexp(b, -e)
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(-6.0, 6.0)
    return torch.ldexp(q, e).view(rows, -1)[:, :K]


def _plain_product(s, X, Xq):
    case = s["case"]
    y = Xq @ s["Wq"].T
    if s["L1s"] is not None:
        y = y + (X.float() @ s["L1s"].float()) @ s["L2"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if case.get("swiglu"):
        gate, up = y.chunk(2, dim=-1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y


# ---------------------------------------------------------------- one pass

def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        return _own(s, case, op)
    if op == "norm":
        return _plain_norm(s, s["x"].float()).to(BF16)
    if op == "residual":
        xo = _plain_residual(s)
        h = _plain_norm(s, xo)
        if not case["packed"]:
            return xo.to(s["x"].dtype), h.to(BF16)
        n = case["B"] * case["T"]
        s["out"][:n], s["h"][:n] = xo[:n].to(s["x"].dtype), h[:n].to(BF16)
        return s["out"], s["h"]
    if op == "quantize":
        return _mx_values(s["X"].float() * s["inv_lambda"]).to(BF16)
    if op == "linear":
        return _plain_product(s, s["X"], _mx_values(s["X"].float() * s["inv_lambda"])).to(BF16)
    xo = _plain_residual(s)
    h = _plain_norm(s, xo).to(BF16).view(-1, case["D"])
    y = _plain_product(s, h, _mx_values(h.float() * s["inv_lambda"]))
    return xo.to(BF16), y.to(BF16)


def _own(s, case, op):
    svdq = s["lib"]
    if op == "norm":
        return svdq.block_norm(s["x"], s["norm"], s["scale"], s["shift"], out_dtype=BF16)
    if op == "residual":
        return svdq.gated_residual(s["x"], s["y"], gate=s["gate"], post=s["post"], res_scale=case["res"],
                                   norm=s["norm"], scale=s["scale"], shift=s["shift"], offsets=s["offsets"],
                                   out=s.get("out"), h=s.get("h"), h_dtype=BF16)
    if op == "quantize":
        return svdq.dequantize_act_mx(svdq.quantize_act_mx(s["X"], s["weight"], s["act"]))
    if op == "linear":
        return svdq.linear_mx(s["X"], s["weight"], s["bias"], s["act"])
    xo, act = svdq.gated_residual_quantize_mx(s["x"], s["y"], s["norm"], s["weight"], s["act"], gate=s["gate"],
                                              post=s["post"], scale=s["scale"], shift=s["shift"])
    return xo, svdq.gemm_mx(act, s["weight"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("norm", "residual", "block"):
        n, D, B = case["B"] * case["T"], case["D"], case["B"]
        size = {"bf16": 2, "f32": 4}
        xb, yb, mb = size[case.get("x", "bf16")], size[case.get("y", "bf16")], size[case.get("mods", "bf16")]
        if op == "norm":
            return {"bytes": n * D * (xb + 2) + (2 * B * D * mb if case["mod"] else 0) + 8 * D * case["affine"],
                    "flops": 8 * n * D}
        byte = n * D * (2 * xb + yb) + 3 * B * D * mb + 8 * D
        if op == "residual":
            return {"bytes": byte + 2 * n * D, "flops": 16 * n * D}
        N = case["N"]
        return {"bytes": byte + N * D * 17 // 32 + 2 * n * N, "flops": 2 * n * N * D + 16 * n * D}
    M, K = case["M"], case["K"]
    if op == "quantize":
        return {"bytes": 4 * M * K + 4 * K, "flops": 4 * M * K}
    N, r = case["N"], case["r"]
    n_out = N // 2 if case["swiglu"] else N
    return {"bytes": 2 * M * K + 4 * K + N * K * 17 // 32 + 2 * r * (K + N) + 2 * N * case["bias"] + 2 * M * n_out,
            "flops": 2 * M * N * K + 2 * M * r * (K + N)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm(v, kind, w, b, eps):
    mean = v.sum(-1, keepdim=True) / v.shape[-1] if kind == "layer" else torch.zeros_like(v[..., :1])
    var = ((v - mean) ** 2).sum(-1, keepdim=True) / v.shape[-1]
    n = (v - mean) * (var + eps) ** -0.5
    n = n if w is None else n * w.double()
    return n if b is None else n + b.double()


def _exact_rows(s, m):
    """One modulation row per row of x, sample by sample."""
    case = s["case"]
    if s["offsets"] is None:
        return torch.repeat_interleave(m.double(), case["T"], dim=0)
    n = (s["offsets"][1:] - s["offsets"][:-1]).long()
    return torch.repeat_interleave(m.double(), n, dim=0)


def _exact_mx(v):
    """float64 values [rows, K] -> MXFP4 values, by comparison with the midpoints of the element grid."""
    rows, K = v.shape
    b = torch.zeros(rows, (K + 31) // 32 * 32, device=v.device, dtype=F64)
    b[:, :K] = v
    b = b.view(rows, -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140)))
    e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e))
    scale = torch.exp2((e - 2).clamp(min=-127))
    a = b.abs() / scale
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=v.device, dtype=F64)
    code = torch.zeros(a.shape, device=v.device, dtype=torch.int64)
    for i in range(7):
        mid = (float(grid[i]) + float(grid[i + 1])) / 2
        code += (a >= mid) if i % 2 else (a > mid)
    return (torch.sign(b) * grid[code] * scale).view(rows, -1)[:, :K]


def _exact_product(s, X, Xq):
    y = Xq @ _exact_mx(s["R"].double()).T
    if s["L1s"] is not None:
        y += X.double() @ s["L1s"].double() @ s["L2"].double()
    if s["bias"] is not None:
        y += s["bias"].double()
    if s["case"].get("swiglu"):
        half = y.shape[1] // 2
        y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
    return y


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    s.pop("Wq", None)
    op = case["op"]
    smoothed = lambda X: (X.double() * s["inv_lambda"].double()).float().double()  # the operator rounds it to fp32
    if op in ("quantize", "linear"):
        Xq = _exact_mx(smoothed(s["X"]))
        return Xq if op == "quantize" else _exact_product(s, s["X"], Xq)
    n, D = case["B"] * case["T"], case["D"]
    v = s["x"].reshape(-1, D)[:n].double()
    if op != "norm":
        y = s["y"].reshape(-1, D)[:n].double()
        if case["post"]:
            y = _exact_norm(y, case["post"], s["pw"], s["pb"], s["eps"])
        v = v + case.get("res", 1.0) * _exact_rows(s, s["gate"]) * y
    h = _exact_norm(v, case["kind"], s["w"], s["b"], s["eps"])
    if s["scale"] is not None:
        h = h * (1.0 + _exact_rows(s, s["scale"])) + _exact_rows(s, s["shift"])
    if op == "norm":
        return h.view(s["x"].shape)
    if op == "block":
        hb = h.to(BF16)  # the quantizer takes the activation in bf16
        return v.view(s["x"].shape), _exact_product(s, hb, _exact_mx(smoothed(hb)))
    if case["packed"]:
        pad = torch.zeros(s["x"].shape[0] - n, D, device="cuda", dtype=F64)
        return torch.cat([v, pad]), torch.cat([h, pad])
    return v.view(s["x"].shape), h.view(s["x"].shape)
