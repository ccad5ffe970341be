"""Operators of a dense block with biases and of its weights' update, in plain
torch and through this package's own calls:

  ln          layer norm with the residual's addition
  ln_bwd      its backward pass with the weight's and bias's gradients
  linear      matrix product with bias, activation and residual in its epilogue
  linear_dx   gradient of its input, times the derivative of the activation
              that made that input
  linear_dw   gradients of its weight and bias
  orth        orthogonalisation of a batch of matrices by Newton-Schulz products
  muon        an optimiser step on such matrices: momentum, orthogonalisation,
              weight decay and update of the fp32 weights and their bf16 copy
"""
import math

import torch

own = False

EPS = 1e-5
ORTH_EPS = 1e-7
COEF = (3.4445, -4.7750, 2.0315)
STEPS = 5
MOMENTUM, DECAY, LR = 0.95, 0.1, 2e-4
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of one request
        dict(name="ln_token_bf16", op="ln", T=1, d=2048, dtype="bf16", residual=True),
        # a packed 32k-token microbatch of training
        dict(name="ln_32k_bf16", op="ln", T=32768, d=2048, dtype="bf16", residual=True),
        # backward pass of an fp32 layer on an odd number of tokens, no residual
        dict(name="ln_bwd_7001_f32", op="ln_bwd", T=7001, d=1024, dtype="f32", residual=False),
        # backward pass of a packed microbatch at the larger hidden size, with the residual stream's gradient
        dict(name="ln_bwd_32k_bf16", op="ln_bwd", T=32768, d=4096, dtype="bf16", residual=True),
        # one token: reading the weight is all there is
        dict(name="linear_token_bf16", op="linear", T=1, K=2048, N=8192, act="gelu", bias=True, residual=False, save=False),
        # 48 requests decode one token each: the product that ends a block, into the residual stream
        dict(name="linear_decode_48", op="linear", T=48, K=8192, N=2048, act="none", bias=True, residual=True, save=False),
        # training, forward: the product that opens a block, its input to the activation kept
        dict(name="linear_16k_gelu", op="linear", T=16384, K=2048, N=8192, act="gelu", bias=True, residual=False, save=True),
        # training, backward: from a block's output gradient to the gradient before its activation, an uneven microbatch
        dict(name="linear_dx_7001", op="linear_dx", T=7001, K=8192, N=2048, act="gelu", add=False),
        # training, backward: weight and bias gradients of a packed microbatch
        dict(name="linear_dw_32k", op="linear_dw", T=32768, K=2048, N=1408, bias=True),
        # a few odd-sized bf16 matrices
        dict(name="orth_odd_bf16", op="orth", batch=3, rows=1001, cols=333, dtype="bf16"),
        # the weight of one dense layer, taller than wide
        dict(name="muon_dense_8192", op="muon", batch=1, rows=8192, cols=2048, nesterov=True),
        # gate and up weights of 32 experts
        dict(name="muon_experts_gate_up", op="muon", batch=64, rows=1408, cols=2048, nesterov=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["ln", "ln", "ln_bwd", "ln_bwd", "linear", "linear", "linear", "linear_dx", "linear_dw", "orth", "muon", "muon"])
    if op in ("ln", "ln_bwd"):
        return dict(op=op, T=_log(rng, 1, 32768), d=64 * _log(rng, 1, 64), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.random() < 0.6)
    if op.startswith("linear"):
        K, N = 64 * _log(rng, 1, 128), 64 * _log(rng, 1, 128)
        T = _log(rng, 1, max(1, min(32768, 16384 * 2048 * 8192 // (K * N))))
        case = dict(op=op, T=T, K=K, N=N)
        if op != "linear_dw":
            case["act"] = rng.choice(ACTS)
        if op == "linear":
            case.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5, save=rng.random() < 0.5)
        elif op == "linear_dx":
            case["add"] = rng.random() < 0.5
        else:
            case["bias"] = rng.random() < 0.7
        return case
    rows, cols = _log(rng, 8, 4096), _log(rng, 8, 4096)
    small, large = min(rows, cols), max(rows, cols)
    most = 64 * 1408 * 1408 * 2048 // (2 * small * small * large)
    batch = _log(rng, 1, max(1, min(64, most)))
    if op == "orth":
        return dict(op=op, batch=batch, rows=rows, cols=cols, dtype=rng.choice(["bf16", "f32"]))
    return dict(op=op, batch=batch, rows=rows, cols=cols, nesterov=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev) * std + mean).to(dtype)

    op = case["op"]
    s = dict(case)
    if op in ("ln", "ln_bwd"):
        T, d, t = case["T"], case["d"], TYPES[case["dtype"]]
        s["x"] = normal(T, d, mean=0.3, dtype=t)
        s["w"] = normal(d, std=0.1, mean=1.0, dtype=t)
        if op == "ln":
            s["b"] = normal(d, std=0.1, dtype=t)
            s["residual_in"] = normal(T, d, std=2.0, dtype=t) if case["residual"] else None
        else:  # x is the row that the forward normalised
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt()
            s["dy"] = normal(T, d, std=0.1, dtype=t)
            s["dres"] = normal(T, d, std=0.1, dtype=t) if case["residual"] else None
        return s
    if op.startswith("linear"):
        T, K, N = case["T"], case["K"], case["N"]
        if op == "linear_dw":
            s.update(x=normal(T, K), dz=normal(T, N, std=0.1))
            return s
        s["w"] = normal(N, K, std=K ** -0.5)
        if op == "linear":
            s["x"] = normal(T, K)
            s["b"] = normal(N, std=0.1) if case["bias"] else None
            s["residual_in"] = normal(T, N) if case["residual"] else None
        else:
            s["dz"] = normal(T, N, std=0.1)
            s["z_in"] = normal(T, K) if case["act"] != "none" else None
            s["add_in"] = normal(T, K, std=0.05) if case["add"] else None
        return s
    B, R, C = case["batch"], case["rows"], case["cols"]

    def gradient():  # rows and columns of uneven size, and a few directions that stand out
        g = torch.randn(B, R, C, generator=gen, device=dev)
        g *= torch.exp(0.5 * torch.randn(B, R, 1, generator=gen, device=dev))
        g *= torch.exp(0.5 * torch.randn(B, 1, C, generator=gen, device=dev))
        u = torch.randn(B, R, 8, generator=gen, device=dev) * torch.logspace(0, -1, 8, device=dev)
        return g.baddbmm_(u, torch.randn(B, 8, C, generator=gen, device=dev)).mul_(1e-3)

    if op == "orth":
        s["x"] = gradient().to(TYPES[case["dtype"]])
        return s
    s["grad"] = gradient()
    s["momentum"] = gradient().mul_(4.0)
    s["param"] = normal(B, R, C, std=0.02, dtype=torch.float32)
    s["param_bf16"] = s["param"].to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _act(act, z):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(act, z):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _orthogonal(u):
    """[batch, rows, cols] fp32, on the shorter side's products."""
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2).contiguous() if tall else u
    x = x / ((x.double() ** 2).sum((1, 2), keepdim=True).sqrt() + ORTH_EPS).float()
    for _ in range(STEPS):
        a = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = COEF[0] * x + torch.bmm(COEF[1] * a + COEF[2] * torch.bmm(a, a), x)
    return x.transpose(1, 2) if tall else x


def _scale(s):
    return 0.2 * math.sqrt(max(s["rows"], s["cols"]))


def _plain(s):
    op = s["op"]
    if op == "ln":
        t = s["x"].dtype
        r = s["x"]
        if s["residual"]:
            r = (s["x"].float() + s["residual_in"].float()).to(t)
        rf = r.float()
        mean = rf.mean(1)
        c = rf - mean.unsqueeze(1)
        rstd = 1 / torch.sqrt((c * c).mean(1) + EPS)
        out = dict(y=(c * rstd.unsqueeze(1) * s["w"].float() + s["b"].float()).to(t), mean=mean, rstd=rstd)
        if s["residual"]:
            out["r"] = r
        return out
    if op == "ln_bwd":
        t = s["x"].dtype
        dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(1)
        n = (s["x"].float() - s["mean"].unsqueeze(1)) * rstd
        g = dy * s["w"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
        if s["residual"]:
            dx = dx + s["dres"].float()
        return dict(dx=dx.to(t), dw=(dy * n).sum(0), db=dy.sum(0))
    if op == "linear":
        z = s["x"].float() @ s["w"].float().T
        if s["bias"]:
            z = z + s["b"].float()
        y = _act(s["act"], z)
        if s["residual"]:
            y = y + s["residual_in"].float()
        out = dict(y=y.bfloat16())
        if s["save"]:
            out["z"] = z.bfloat16()
        return out
    if op == "linear_dx":
        dx = s["dz"].float() @ s["w"].float()
        if s["act"] != "none":
            dx = dx * _act_grad(s["act"], s["z_in"].float())
        if s["add"]:
            dx = dx + s["add_in"].float()
        return dict(dx=dx.bfloat16())
    if op == "linear_dw":
        dz = s["dz"].float()
        out = dict(dw=dz.T @ s["x"].float())
        if s["bias"]:
            out["db"] = dz.sum(0)
        return out
    if op == "orth":
        return dict(o=_orthogonal(s["x"].float()).contiguous().bfloat16())
    m, g, w = s["momentum"], s["grad"], s["param"]
    m.mul_(MOMENTUM).add_(g)
    o = _orthogonal(g + MOMENTUM * m if s["nesterov"] else m)
    w.mul_(1 - LR * DECAY).sub_(LR * _scale(s) * o)
    s["param_bf16"].copy_(w)
    return dict(momentum=m, param=w, param_bf16=s["param_bf16"])


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------
def _buffers(s, moe):
    """Shape, workspace and outputs, as a program makes them once."""
    op, dev = s["op"], "cuda"
    new = lambda *shape, t=torch.bfloat16: torch.empty(*shape, dtype=t, device=dev)  # noqa: E731
    f32 = torch.float32
    if op in ("ln", "ln_bwd"):
        T, d, t = s["T"], s["d"], TYPES[s["dtype"]]
        dt = moe.MOE_DTYPE_BF16 if s["dtype"] == "bf16" else moe.MOE_DTYPE_F32
        b = dict(shape=moe.make_norm_shape(T, d, dt, EPS, moe.MOE_NORM_OVERWRITE_DW))
        if op == "ln":
            b.update(y=new(T, d, t=t), r=new(T, d, t=t) if s["residual"] else None, mean=new(T, t=f32), rstd=new(T, t=f32))
        else:
            b.update(dx=new(T, d, t=t), dw=new(d, t=f32), db=new(d, t=f32))
            b["ws"] = new(max(1, moe.moe_layernorm_workspace_size(b["shape"])), t=torch.uint8)
        return b
    if op.startswith("linear"):
        T, K, N = s["T"], s["K"], s["N"]
        acts = dict(none=moe.MOE_ACT_NONE, relu=moe.MOE_ACT_RELU, gelu=moe.MOE_ACT_GELU, gelu_tanh=moe.MOE_ACT_GELU_TANH,
                    silu=moe.MOE_ACT_SILU)
        b = dict(act=acts[s.get("act", "none")])
        if op == "linear":
            b["shape"] = moe.make_linear_shape(T, K, N, moe.MOE_DTYPE_BF16, b["act"])
            b.update(y=new(T, N), z=new(T, N) if s["save"] else None)
        else:
            b["shape"] = moe.make_linear_shape(T, K, N, moe.MOE_DTYPE_BF16, flags=moe.MOE_LINEAR_OVERWRITE_DW)
        if op == "linear_dx":
            b["dx"] = new(T, K)
        if op == "linear_dw":
            b.update(dw=new(N, K, t=f32), db=new(N, t=f32) if s["bias"] else None)
            b["ws"] = new(max(1, moe.moe_linear_workspace_size(b["shape"])), t=torch.uint8)
        return b
    B, R, C = s["batch"], s["rows"], s["cols"]
    dt = moe.MOE_DTYPE_BF16 if s.get("dtype") == "bf16" else moe.MOE_DTYPE_F32
    b = dict(shape=moe.make_orth_shape(B, R, C, dt, STEPS, COEF, ORTH_EPS))
    b["ws"] = new(max(1, moe.moe_orthogonalize_workspace_size(b["shape"])), t=torch.uint8)
    if op == "orth":
        b["o"] = new(B, R, C)
    else:
        b["cfg"] = moe.make_muon_config(LR, MOMENTUM, DECAY, _scale(s), nesterov=s["nesterov"])
    return b


def _own(s):
    import token_dispatch_grouped_amd as moe
    b = s.get("buffers")
    if b is None:
        b = s["buffers"] = _buffers(s, moe)
    op = s["op"]
    if op == "ln":
        moe.moe_layernorm_fwd(b["shape"], s["x"], s["residual_in"], s["w"], s["b"], b["r"], b["y"], b["mean"], b["rstd"])
        return {k: b[k] for k in ("y", "mean", "rstd", "r") if b[k] is not None}
    if op == "ln_bwd":
        moe.moe_layernorm_bwd(b["shape"], s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["dres"], b["dx"], b["dw"], b["db"],
                              b["ws"], b["ws"].numel())
        return dict(dx=b["dx"], dw=b["dw"], db=b["db"])
    if op == "linear":
        moe.moe_linear_fwd(b["shape"], s["x"], s["w"], s["b"], s["residual_in"], b["z"], b["y"])
        return {k: b[k] for k in ("y", "z") if b[k] is not None}
    if op == "linear_dx":
        moe.moe_linear_dgrad(b["shape"], s["dz"], s["w"], s["z_in"], b["act"], s["add_in"], b["dx"])
        return dict(dx=b["dx"])
    if op == "linear_dw":
        moe.moe_linear_wgrad(b["shape"], s["dz"], s["x"], b["dw"], b["db"], b["ws"], b["ws"].numel())
        return {k: b[k] for k in ("dw", "db") if b[k] is not None}
    if op == "orth":
        moe.moe_orthogonalize(b["shape"], s["x"], b["o"], b["ws"], b["ws"].numel())
        return dict(o=b["o"])
    moe.moe_muon_step(b["cfg"], b["shape"], s["param"], s["grad"], s["momentum"], s["param_bf16"], b["ws"], b["ws"].numel())
    return dict(momentum=s["momentum"], param=s["param"], param_bf16=s["param_bf16"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("ln", "ln_bwd"):
        T, d, z = case["T"], case["d"], BYTES[case["dtype"]]
        res = 1 if case["residual"] else 0
        if op == "ln":
            return dict(bytes=T * d * z * (2 + 2 * res) + 2 * z * d + 8 * T, flops=8.0 * T * d)
        return dict(bytes=T * d * z * (3 + res) + (z + 8) * d + 8 * T, flops=14.0 * T * d)
    if op.startswith("linear"):
        T, K, N = case["T"], case["K"], case["N"]
        flops = 2.0 * T * K * N
        if op == "linear":
            return dict(bytes=2 * (T * K + N * K + T * N * (1 + case["residual"] + case["save"]) + (N if case["bias"] else 0)), flops=flops)
        if op == "linear_dx":
            return dict(bytes=2 * (T * N + N * K + T * K * (1 + case["add"] + (case["act"] != "none"))), flops=flops)
        return dict(bytes=2 * T * (K + N) + 4 * N * K + (4 * N if case["bias"] else 0), flops=flops)
    B, R, C = case["batch"], case["rows"], case["cols"]
    S, L = min(R, C), max(R, C)
    flops = STEPS * B * (3.0 * S * S * L + 1.0 * S * S * S)  # the two symmetric products by half
    if op == "orth":
        return dict(bytes=B * R * C * (BYTES[case["dtype"]] + 2), flops=flops)
    return dict(bytes=B * R * C * (4 * 5 + 2), flops=flops)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _polar64(u):
    """a X + b (X X') X + c (X X')^2 X, five times, with the products on whichever side is shorter."""
    a, b, c = COEF
    y = u / (torch.linalg.vector_norm(u.flatten(1), dim=1)[:, None, None] + ORTH_EPS)
    for _ in range(STEPS):
        if y.shape[1] <= y.shape[2]:
            gy = torch.matmul(torch.matmul(y, y.mT), y)
            y = a * y + b * gy + c * torch.matmul(torch.matmul(y, y.mT), gy)
        else:
            gram = torch.matmul(y.mT, y)
            y = a * y + torch.matmul(y, b * gram + c * torch.matrix_power(gram, 2))
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    D = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if op == "ln":
        r = D["x"]
        out = {}
        if case["residual"]:
            out["r"] = r = (D["x"] + D["residual_in"]).to(s["x"].dtype).double()
        mu = torch.sum(r, dim=1, keepdim=True) / case["d"]
        inv = torch.rsqrt(torch.sum((r - mu) ** 2, dim=1, keepdim=True) / case["d"] + EPS)
        out.update(y=torch.addcmul(D["b"], (r - mu) * inv, D["w"]), mean=mu.squeeze(1), rstd=inv.squeeze(1))
        return out
    if op == "ln_bwd":
        d = case["d"]
        hat = (D["x"] - D["mean"][:, None]) * D["rstd"][:, None]
        gw = D["dy"] * D["w"]
        total, proj = torch.sum(gw, dim=1, keepdim=True), torch.sum(gw * hat, dim=1, keepdim=True)
        dx = (d * gw - total - hat * proj) * D["rstd"][:, None] / d
        if case["residual"]:
            dx += D["dres"]
        return dict(dx=dx, dw=torch.einsum("td,td->d", D["dy"], hat), db=torch.sum(D["dy"], dim=0))
    act = case.get("act", "none")
    if op == "linear":
        z = torch.mm(D["x"], D["w"].t())
        if case["bias"]:
            z += D["b"]
        y = {"none": lambda v: v.clone(), "relu": lambda v: v.clamp(min=0), "silu": lambda v: v * torch.sigmoid(v),
             "gelu": lambda v: v * torch.special.ndtr(v),
             "gelu_tanh": lambda v: v * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3))}[act](z)
        if case["residual"]:
            y += D["residual_in"]
        return dict(y=y, z=z) if case["save"] else dict(y=y)
    if op == "linear_dx":
        dx = torch.mm(D["dz"], D["w"])
        if act != "none":
            v = D["z_in"]
            if act == "relu":
                slope = torch.gt(v, 0).double()
            elif act == "silu":
                slope = torch.sigmoid(v) + v * torch.sigmoid(v) * torch.sigmoid(-v)
            elif act == "gelu":
                slope = torch.special.ndtr(v) + v * torch.exp(-v ** 2 / 2) / (2 * math.pi) ** 0.5
            else:
                k = 2 * (2 / math.pi) ** 0.5
                q = torch.sigmoid(k * (v + 0.044715 * v ** 3))
                slope = q + v * q * (1 - q) * k * (1 + 0.134145 * v ** 2)
            dx *= slope
        if case["add"]:
            dx += D["add_in"]
        return dict(dx=dx)
    if op == "linear_dw":
        out = dict(dw=torch.mm(D["dz"].t(), D["x"]))
        if case["bias"]:
            out["db"] = torch.sum(D["dz"], dim=0)
        return out
    if op == "orth":
        return dict(o=_polar64(D["x"]))
    moved = MOMENTUM * D["momentum"] + D["grad"]
    o = _polar64(MOMENTUM * moved + D["grad"] if case["nesterov"] else moved)
    w = D["param"] - LR * (DECAY * D["param"] + 0.2 * max(case["rows"], case["cols"]) ** 0.5 * o)
    return dict(momentum=moved, param=w, param_bf16=w)
