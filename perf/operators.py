"""The operators that stand before and beside the routed experts of an MoE
layer, in plain torch and through this package's own calls:

  norm    RMS norm with the residual's addition, in the layer's type or in
          8 bits with block scales, and its backward pass
  quant   the 8-bit form of a matrix (weights, or rows that no norm made)
  ffn     the gated feed-forward block that every token takes (the shared
          expert): forward, gradient of its input, gradient of its weights
  ffn8    the same block on 8-bit rows and 8-bit weights (serving)

The 8-bit form: e4m3 elements and, for 32 consecutive ones of a row, one
power of two (e8m0), the smallest S with max|v| <= 448 S.
"""
import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of one request: the norm in front of an 8-bit block
        dict(name="norm_token_mx8", op="norm", T=1, d=2048, dtype="bf16", residual=True, mx8=True),
        # a packed 32k-token microbatch of training
        dict(name="norm_32k_bf16", op="norm", T=32768, d=2048, dtype="bf16", residual=True, mx8=False),
        # an fp32 layer, an odd number of tokens, no residual (the first norm of a model)
        dict(name="norm_odd_f32", op="norm", T=7001, d=1024, dtype="f32", residual=False, mx8=False),
        # the backward pass of a packed microbatch at the larger hidden size, with the residual stream's gradient
        dict(name="norm_bwd_32k_bf16", op="norm_bwd", T=32768, d=4096, dtype="bf16", residual=True),
        # a few fp32 rows on their way into the 8-bit block
        dict(name="quant_rows_f32", op="quant", T=129, d=1024, dtype="f32"),
        # a gate/up weight on loading: 2 x 2816 rows
        dict(name="quant_weight_bf16", op="quant", T=5632, d=4096, dtype="bf16"),
        # one token through the block: reading the weights is all there is
        dict(name="ffn_token_bf16", op="ffn", T=1, d=2048, F=1408, add=True, save=False),
        # training, forward: keeps h and a, adds to the routed experts' output
        dict(name="ffn_16k_bf16", op="ffn", T=16384, d=2048, F=1408, add=True, save=True),
        # training, backward: the input's gradient on an uneven microbatch, added to the routed experts' gradient
        dict(name="ffn_dgrad_7001_bf16", op="ffn_dgrad", T=7001, d=2048, F=1408, add=True),
        # training, backward: the weights' gradient of a packed microbatch (fp32)
        dict(name="ffn_wgrad_32k_bf16", op="ffn_wgrad", T=32768, d=2048, F=1408),
        # 48 requests decode one token each
        dict(name="ffn8_decode_48", op="ffn8", T=48, d=4096, F=2816, add=True),
        # prompts: enough rows to fill the card
        dict(name="ffn8_prompt_8k", op="ffn8", T=8192, d=4096, F=2816, add=False),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "quant", "ffn", "ffn", "ffn_dgrad", "ffn_wgrad", "ffn8", "ffn8"])
    if op in ("norm", "norm_bwd", "quant"):
        case = dict(op=op, T=_log(rng, 1, 32768), d=64 * _log(rng, 1, 64), dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op != "quant":
            case["residual"] = rng.random() < 0.7
        if op == "norm":
            case["mx8"] = rng.random() < 0.4
        return case
    step = 128 if op == "ffn8" else 64
    d, F = step * _log(rng, 1, 4096 // step), step * _log(rng, 1, 2816 // step)
    most = 32768 * 2048 * 1408 if op != "ffn8" else 8192 * 4096 * 2816
    case = dict(op=op, T=_log(rng, 1, max(1, min(32768, most // (d * F)))), d=d, F=F)
    if op != "ffn_wgrad":
        case["add"] = rng.random() < 0.5
    if op == "ffn":
        case["save"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    T, d, op = case["T"], case["d"], case["op"]
    s = dict(case)
    if op in ("norm", "norm_bwd", "quant"):
        t = TYPES[case["dtype"]]
        s["x"] = normal(T, d, dtype=t)
        if op != "quant":
            s["w"] = (1 + 0.1 * torch.randn(d, generator=gen, device=dev)).to(t)
        if op == "norm":
            s["residual_in"] = normal(T, d, std=2.0, dtype=t) if case["residual"] else None
        if op == "norm_bwd":  # x is the row that the forward normalised
            s["rstd"] = (s["x"].float().square().mean(1) + EPS).rsqrt()
            s["dy"] = normal(T, d, std=0.1, dtype=t)
            s["dres"] = normal(T, d, std=0.1, dtype=t) if case["residual"] else None
        return s
    F = case["F"]
    if case.get("add"):
        s["addend"] = normal(T, d, std=0.5)
    if op == "ffn_wgrad":
        s.update(x=normal(T, d), dy=normal(T, d, std=0.1), a=normal(T, F, std=0.4), dh=normal(T, 2 * F, std=0.05))
        return s
    s["w_gu"], s["w_down"] = normal(2 * F, d, std=0.02), normal(d, F, std=0.02)
    if op == "ffn_dgrad":
        s.update(dy=normal(T, d, std=0.1), h=normal(T, 2 * F, std=0.02 * d ** 0.5))
    else:
        s["x"] = normal(T, d)
    if op == "ffn8":  # a program holds the weights in their 8-bit form, and the norm hands the rows over in it
        for k in ("x", "w_gu", "w_down"):
            s[k], s[k + "_s"] = _quantize(s[k].float())
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _quantize(v):
    """[n, m] fp32 -> e4m3 elements [n, m] and e8m0 scales [n, m / 32]."""
    b = v.reshape(v.shape[0], -1, 32)
    m, e = torch.frexp(b.abs().amax(2))  # max|v| = m 2^e with m in [0.5, 1), and 448 = 0.875 * 2^9
    e = torch.where(m > 0, e - 9 + (m > 0.875), -127).clamp(-127, 127)
    q = torch.ldexp(b, -e.unsqueeze(2)).to(torch.float8_e4m3fn).reshape(v.shape)
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(q, scale):
    return (q.float().reshape(*scale.shape, 32) * scale.float().unsqueeze(2)).reshape(q.shape)


def _swiglu(h):
    g, u = h.chunk(2, 1)
    return g / (1 + torch.exp(-g)) * u


def _plain(s):
    op = s["op"]
    if op == "norm":
        t = s["x"].dtype
        r = s["x"]
        if s["residual"]:
            r = (s["x"].float() + s["residual_in"].float()).to(t)
        rf = r.float()
        rstd = 1 / torch.sqrt((rf * rf).mean(1) + EPS)
        y = rf * rstd.unsqueeze(1) * s["w"].float()
        out = dict(rstd=rstd)
        if s["residual"]:
            out["r"] = r
        if s["mx8"]:
            out["y"], out["y_scale"] = _quantize(y)
        else:
            out["y"] = y.to(t)
        return out
    if op == "norm_bwd":
        t = s["x"].dtype
        dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(1)
        n = s["x"].float() * rstd
        g = dy * s["w"].float()
        dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
        if s["residual"]:
            dx = dx + s["dres"].float()
        return dict(dx=dx.to(t), dw=(dy * n).sum(0))
    if op == "quant":
        q, scale = _quantize(s["x"].float())
        return dict(q=q, scale=scale)
    if op == "ffn":
        h = s["x"].float() @ s["w_gu"].float().T
        a = _swiglu(h)
        y = a @ s["w_down"].float().T
        if s["add"]:
            y = y + s["addend"].float()
        out = dict(y=y.bfloat16())
        if s["save"]:
            out.update(h=h.bfloat16(), a=a.bfloat16())
        return out
    if op == "ffn_dgrad":
        g, u = s["h"].float().chunk(2, 1)
        da = s["dy"].float() @ s["w_down"].float()
        sg = 1 / (1 + torch.exp(-g))
        dh = torch.cat([da * u * sg * (1 + g * (1 - sg)), da * g * sg], 1)
        dx = dh @ s["w_gu"].float()
        if s["add"]:
            dx = dx + s["addend"].float()
        return dict(dh=dh.bfloat16(), dx=dx.bfloat16())
    if op == "ffn_wgrad":
        return dict(dw_gu=s["dh"].float().T @ s["x"].float(), dw_down=s["dy"].float().T @ s["a"].float())
    # ffn8
    a = _swiglu(_values(s["x"], s["x_s"]) @ _values(s["w_gu"], s["w_gu_s"]).T)
    y = _values(*_quantize(a)) @ _values(s["w_down"], s["w_down_s"]).T
    if s["add"]:
        y = y + s["addend"].float()
    return dict(y=y.bfloat16())


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------
def _buffers(s, moe):
    """Shape, workspace and outputs, as a program makes them once."""
    op, T, d, dev = s["op"], s["T"], s["d"], "cuda"
    new = lambda *shape, t=torch.bfloat16: torch.empty(*shape, dtype=t, device=dev)  # noqa: E731
    f32, e4m3, e8m0 = torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu
    b = {}
    if op in ("norm", "norm_bwd", "quant"):
        t = TYPES[s["dtype"]]
        dt = moe.MOE_DTYPE_BF16 if s["dtype"] == "bf16" else moe.MOE_DTYPE_F32
        if op == "quant":
            return dict(dt=dt, q=new(T, d, t=e4m3), scale=new(T, d // 32, t=e8m0))
        b["shape"] = moe.make_norm_shape(T, d, dt, EPS, moe.MOE_NORM_OVERWRITE_DW)
        if op == "norm":
            b["rstd"] = new(T, t=f32)
            b["r"] = new(T, d, t=t) if s["residual"] else None
            b["y"] = new(T, d, t=e4m3 if s["mx8"] else t)
            b["y_scale"] = new(T, d // 32, t=e8m0) if s["mx8"] else None
        else:
            b.update(dx=new(T, d, t=t), dw=new(d, t=f32))
            b["ws"] = new(max(1, moe.moe_rmsnorm_workspace_size(b["shape"])), t=torch.uint8)
        return b
    F = s["F"]
    b["shape"] = moe.make_ffn_shape(T, d, F, moe.MOE_DTYPE_MX8 if op == "ffn8" else moe.MOE_DTYPE_BF16,
                                    moe.MOE_FFN_OVERWRITE_DW)
    fwd, wgrad = moe.moe_ffn_workspace_size(b["shape"])
    if op in ("ffn", "ffn8"):
        b.update(ws=new(max(1, fwd), t=torch.uint8), y=new(T, d))
        save = s.get("save", False)
        b.update(h=new(T, 2 * F) if save else None, a=new(T, F) if save else None)
    elif op == "ffn_dgrad":
        b.update(dh=new(T, 2 * F), dx=new(T, d))
    else:
        b.update(ws=new(max(1, wgrad), t=torch.uint8), dw_gu=new(2 * F, d, t=f32), dw_down=new(d, F, t=f32))
    return b


def _own(s):
    import token_dispatch_grouped_amd as moe
    b = s.get("buffers")
    if b is None:
        b = s["buffers"] = _buffers(s, moe)
    op = s["op"]
    if op == "norm":
        moe.moe_rmsnorm_fwd(b["shape"], s["x"], s["residual_in"], s["w"], b["r"], b["y"], b["y_scale"], b["rstd"])
        return {k: b[k] for k in ("rstd", "r", "y", "y_scale") if b[k] is not None}
    if op == "norm_bwd":
        moe.moe_rmsnorm_bwd(b["shape"], s["dy"], s["x"], s["w"], s["rstd"], s["dres"], b["dx"], b["dw"], b["ws"],
                            b["ws"].numel())
        return dict(dx=b["dx"], dw=b["dw"])
    if op == "quant":
        moe.moe_mx8_quantize(s["T"], s["d"], b["dt"], s["x"], b["q"], b["scale"])
        return dict(q=b["q"], scale=b["scale"])
    if op in ("ffn", "ffn8"):
        moe.moe_ffn_fwd(b["shape"], s["x"], s.get("x_s"), s["w_gu"], s.get("w_gu_s"), s["w_down"], s.get("w_down_s"),
                        s.get("addend"), b["h"], b["a"], b["y"], b["ws"], b["ws"].numel())
        return {k: b[k] for k in ("y", "h", "a") if b[k] is not None}
    if op == "ffn_dgrad":
        moe.moe_ffn_dgrad(b["shape"], s["dy"], s["h"], s["w_gu"], s["w_down"], s.get("addend"), b["dh"], b["dx"])
        return dict(dh=b["dh"], dx=b["dx"])
    moe.moe_ffn_wgrad(b["shape"], s["dy"], s["x"], s["a"], s["dh"], b["dw_gu"], b["dw_down"], b["ws"], b["ws"].numel())
    return dict(dw_gu=b["dw_gu"], dw_down=b["dw_down"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    T, d, op = case["T"], case["d"], case["op"]
    if op in ("norm", "norm_bwd", "quant"):
        z = BYTES[case["dtype"]]
        if op == "quant":
            return dict(bytes=T * d * z + T * d * 33 / 32, flops=2.0 * T * d)
        res = 1 if case["residual"] else 0
        if op == "norm":
            out = 33 / 32 if case["mx8"] else z
            return dict(bytes=T * d * (z * (1 + 2 * res) + out) + z * d + 4 * T, flops=5.0 * T * d)
        return dict(bytes=T * d * z * (3 + res) + (z + 4) * d + 4 * T, flops=10.0 * T * d)
    F = case["F"]
    add = T * d * 2 if case.get("add") else 0
    flops = 6.0 * T * d * F
    if op == "ffn":
        return dict(bytes=2 * (2 * T * d + 3 * d * F) + add + (6 * T * F if case["save"] else 0), flops=flops)
    if op == "ffn_dgrad":
        return dict(bytes=2 * (2 * T * d + 3 * d * F + 4 * T * F) + add, flops=flops)
    if op == "ffn_wgrad":
        return dict(bytes=2 * (2 * T * d + 3 * T * F) + 4 * 3 * d * F, flops=flops)
    return dict(bytes=(T * d + 3 * d * F) * 33 / 32 + 2 * T * d + add, flops=flops)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _mx8_64(v):
    """The 8-bit form of fp64 rows, by the definition: the power of two from the block's largest value, then the nearest
    e4m3 number (3 fraction bits, exponents from -6, ties to even)."""
    n, m = v.shape
    blocks = v.reshape(n, m // 32, 32)
    top = blocks.abs().max(dim=2, keepdim=True).values
    p = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0))
    p = torch.where(448.0 * torch.exp2(p - 1) >= top, p - 1, p)  # log2's own rounding next to a power of two
    p = torch.where(448.0 * torch.exp2(p) < top, p + 1, p)
    p = torch.where(top > 0, p, torch.full_like(p, -127.0)).clamp(-127, 127)
    w = blocks / torch.exp2(p)
    step = torch.exp2(torch.floor(torch.log2(w.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(w / step) * step).reshape(n, m), torch.exp2(p).squeeze(2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    D = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and not k.endswith("_s") and "float8" not in str(v.dtype)}
    if op == "norm":
        r = D["x"]
        out = {}
        if case["residual"]:
            r = (D["x"] + D["residual_in"]).to(s["x"].dtype).double()
            out["r"] = r
        inv = torch.rsqrt(torch.sum(r ** 2, dim=1) / case["d"] + EPS)
        y = torch.einsum("td,t,d->td", r, inv, D["w"])
        out["rstd"] = inv
        if case["mx8"]:
            out["y"], out["y_scale"] = _mx8_64(y)
        else:
            out["y"] = y
        return out
    if op == "norm_bwd":
        inv, x, gy = D["rstd"][:, None], D["x"], D["dy"]
        proj = torch.sum(gy * D["w"] * x, dim=1, keepdim=True) * inv ** 3 / case["d"]
        dx = gy * D["w"] * inv - x * proj
        if case["residual"]:
            dx += D["dres"]
        return dict(dx=dx, dw=torch.sum(gy * x * inv, dim=0))
    if op == "quant":
        q, scale = _mx8_64(D["x"])
        return dict(q=q, scale=scale)
    if op == "ffn_wgrad":
        return dict(dw_gu=torch.mm(D["dh"].t(), D["x"]), dw_down=torch.mm(D["dy"].t(), D["a"]))
    F = case["F"]
    if op == "ffn_dgrad":
        gate, up = D["h"][:, :F], D["h"][:, F:]
        da = torch.mm(D["dy"], D["w_down"])
        sig = torch.sigmoid(gate)
        dh = torch.empty_like(D["h"])
        dh[:, F:] = da * gate * sig
        dh[:, :F] = da * up * (sig + gate * sig * (1 - sig))
        dx = torch.mm(dh, D["w_gu"])
        return dict(dh=dh, dx=dx + D["addend"] if case["add"] else dx)
    if op == "ffn8":
        for k in ("x", "w_gu", "w_down"):
            scale = torch.exp2(s[k + "_s"].view(torch.uint8).double() - 127)
            D[k] = s[k].float().double() * scale.repeat_interleave(32, dim=1)
    gate, up = torch.mm(D["x"], D["w_gu"][:F].t()), torch.mm(D["x"], D["w_gu"][F:].t())
    a = gate * torch.sigmoid(gate) * up
    kept = a
    if op == "ffn8":
        q, scale = _mx8_64(a)
        kept = q * scale.repeat_interleave(32, dim=1)
    y = torch.mm(kept, D["w_down"].t())
    out = dict(y=y + D["addend"] if case["add"] else y)
    if op == "ffn" and case["save"]:
        out.update(h=torch.cat((gate, up), dim=1), a=a)
    return out
