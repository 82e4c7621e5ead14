"""The dense half of a mixture-of-experts block, measured operator by operator:

* norm / norm_bwd: the residual stream's addition with the root-mean-square norm in
  front of the router and the experts, its output in bf16 and, or, in 8 bits (MXFP8:
  e4m3 codes with one e8m0 scale per 32), and its backward pass;
* ffn / ffn_bwd: the gated feed-forward block that every token passes beside its
  routed experts (a shared expert), on bf16 or MXFP8 weights, with the residual in the
  epilogue of its second product, and its backward pass;
* mxq: the MXFP8 quantiser for weights and for activations that no norm quantised;
* clip: the global norm of the adapters' gradients, and clipping by it.

``run`` computes them in their plain form, or with ``own`` by the framework's calls;
``exact`` computes them from their definitions in 64 bits. Codes are returned as e4m3
values and scales as e8m0 values (dtypes that hold what the bytes stand for).
"""
import math

import torch

own = False

EPS = 1e-6
ALPHA, LIMIT = 1.702, 7.0
CLIP_EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step, residual stream in bf16: latency alone
        {"name": "norm_decode", "op": "norm", "T": 1, "H": 2048, "x": "bf16", "mx": False,
         "bf16": True},
        # a prefill chunk: the combine's fp32 output joins the stream, the norm feeds the router
        # and the 4-bit experts (bf16) and an MXFP8 shared expert (codes and scales)
        {"name": "norm_prefill_mx", "op": "norm", "T": 4096, "H": 2880, "x": "f32", "mx": True,
         "bf16": True},
        # a training step of a ragged batch: gradients of the stream and of the norm's weight
        {"name": "norm_backward", "op": "norm_bwd", "T": 8191, "H": 2880, "dy": "bf16"},
        # one token through a small shared expert: latency and the weights' bytes
        {"name": "ffn_decode", "op": "ffn", "T": 1, "H": 2048, "I": 768, "mx": False,
         "clamped": False, "bias": False, "train": False},
        # a prefill batch through a large dense block: matrix rate
        {"name": "ffn_prefill", "op": "ffn", "T": 4096, "H": 4096, "I": 8192, "mx": False,
         "clamped": False, "bias": False, "train": False},
        # a decode batch through an MXFP8 shared expert with biases and the clamped activation
        {"name": "ffn_mx_decode", "op": "ffn", "T": 16, "H": 2880, "I": 2880, "mx": True,
         "clamped": True, "bias": True, "train": False},
        # a prefill chunk of the same block
        {"name": "ffn_mx_prefill", "op": "ffn", "T": 2048, "H": 2880, "I": 2880, "mx": True,
         "clamped": True, "bias": True, "train": False},
        # a training step: every gradient of the block, biases among them
        {"name": "ffn_backward", "op": "ffn_bwd", "T": 8192, "H": 2880, "I": 2880,
         "clamped": True, "bias": True},
        # activations of a decode batch that come from no norm
        {"name": "quantize_decode", "op": "mxq", "R": 16, "K": 2880, "x": "bf16"},
        # a weight stack taken to MXFP8 once, from bf16
        {"name": "quantize_weights", "op": "mxq", "R": 16384, "K": 4096, "x": "bf16"},
        # the two adapter gradients of one small layer: launches alone
        {"name": "clip_layer", "op": "clip", "layers": 1, "E": 8, "r": 8, "H": 256, "I": 512,
         "g": "f32"},
        # the adapter gradients of a 24-layer model, 128 experts to a layer
        {"name": "clip_model", "op": "clip", "layers": 24, "E": 128, "r": 8, "H": 2048, "I": 768,
         "g": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _step(v, m):
    return max(m, v // m * m)


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_bwd", "ffn", "ffn", "ffn", "ffn_bwd", "ffn_bwd", "mxq",
                     "clip"))
    if op == "norm":
        mx = rng.random() < 0.5
        return {"op": op, "T": _log(rng, 1, 16384), "H": _step(_log(rng, 64, 8192), 32 if mx else 8),
                "x": rng.choice(("bf16", "f32")), "mx": mx, "bf16": not mx or rng.random() < 0.7}
    if op == "norm_bwd":
        return {"op": op, "T": _log(rng, 1, 16384), "H": _step(_log(rng, 64, 8192), 8),
                "dy": rng.choice(("bf16", "f32"))}
    if op == "mxq":
        return {"op": op, "R": _log(rng, 1, 32768), "K": _step(_log(rng, 32, 8192), 32),
                "x": rng.choice(("bf16", "f32"))}
    if op == "clip":
        return {"op": op, "layers": rng.randint(1, 24), "E": _log(rng, 4, 128),
                "r": rng.choice((4, 8, 16)), "H": _step(_log(rng, 128, 4096), 8),
                "I": _step(_log(rng, 128, 2048), 8), "g": rng.choice(("f32", "f32", "bf16"))}
    mx = op == "ffn" and rng.random() < 0.4
    m = 32 if mx else 8
    most = 4096 * 4096 * 8192 // (2 if op == "ffn_bwd" else 1)
    while True:
        T, H, I = _log(rng, 1, 16384), _step(_log(rng, 64, 6144), m), _step(_log(rng, 64, 8192), m)
        if T * H * I <= most:
            break
    c = {"op": op, "T": T, "H": H, "I": I, "clamped": rng.random() < 0.5, "bias": rng.random() < 0.5}
    if op == "ffn":
        c["mx"] = mx
        c["train"] = not mx and rng.random() < 0.3
    return c


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["H"]
        b = n * ((2 if case["x"] == "bf16" else 4) + 2 + 2) + 2 * case["H"] + 4 * case["T"]
        b += (2 * n if case["bf16"] else 0) + (n + n // 32 if case["mx"] else 0)
        return {"bytes": b, "flops": 5 * n}
    if op == "norm_bwd":
        n = case["T"] * case["H"]
        return {"bytes": n * ((2 if case["dy"] == "bf16" else 4) + 2 + 2 + 2) + 4 * case["T"]
                + 6 * case["H"], "flops": 9 * n}
    if op == "mxq":
        n = case["R"] * case["K"]
        return {"bytes": n * (2 if case["x"] == "bf16" else 4) + n + n // 32, "flops": 2 * n}
    if op == "clip":
        n = case["layers"] * case["E"] * case["r"] * (case["H"] + 2 * case["I"])
        return {"bytes": 2 * n * (4 if case["g"] == "f32" else 2), "flops": 3 * n}
    T, H, I = case["T"], case["H"], case["I"]
    if op == "ffn":
        w = 3 * H * I
        b = w + w // 32 + T * H + T * H // 32 if case["mx"] else 2 * (w + T * H)
        b += 2 * T * H + 2 * T * H + (2 * (2 * I + H) if case["bias"] else 0)
        return {"bytes": b + (8 * T * I if case["train"] else 0), "flops": 6 * T * H * I}
    # weights and their gradients, x, dy, dx, the saved pre-activations
    return {"bytes": 2 * 2 * 3 * H * I + 3 * 2 * T * H + 8 * T * I
            + (2 * (2 * I + H) if case["bias"] else 0), "flops": 12 * T * H * I}


# ------------------------------------------------------------------ inputs

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    """The tensors of one call; with `own` also what a program keeps beside them: output
    buffers, the workspace and the descriptor of the weights or of the gradient list."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        s["w"] = (1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        # a stream whose rows differ in size, as they do from layer to layer and token to token
        size = torch.exp(torch.randn(T, 1, generator=g, device="cuda"))
        stream = torch.randn(T, H, generator=g, device="cuda") * size
        if op == "norm":
            s["x"], s["res"] = normal(T, H, dtype=_DT[case["x"]]), stream.to(torch.bfloat16)
        else:
            s["s"] = stream.to(torch.bfloat16)
            s["rstd"] = torch.rsqrt(s["s"].double().square().mean(1) + EPS).float()
            s["dy"], s["dres"] = normal(T, H, std=0.1, dtype=_DT[case["dy"]]), normal(T, H, std=0.1)
    elif op == "mxq":
        # rows of weights or activations, each block of its own size
        R, K = case["R"], case["K"]
        size = torch.exp2(2 * torch.randn(R, K // 32, 1, generator=g, device="cuda"))
        s["x"] = (torch.randn(R, K // 32, 32, generator=g, device="cuda") * size).reshape(R, K).to(
            _DT[case["x"]])
    elif op == "clip":
        E, r, H, I = case["E"], case["r"], case["H"], case["I"]
        s["grads"] = []
        for _ in range(case["layers"]):
            s["grads"] += [normal(E, r, H, std=1e-2, dtype=_DT[case["g"]]),
                           normal(E, 2 * I, r, std=1e-2, dtype=_DT[case["g"]])]
        s["max_norm"] = 1.0
    else:
        T, H, I = case["T"], case["H"], case["I"]
        # gpt-oss's activation is clamped at 7: pre-activations that reach it
        wgu = normal(2 * I, H, std=(2.5 if case["clamped"] else 1.0) / math.sqrt(H))
        wdn = normal(H, I, std=1.0 / math.sqrt(I))
        s["x"] = normal(T, H)
        s["bgu"] = normal(2 * I, std=0.1) if case["bias"] else None
        s["bdn"] = normal(H, std=0.1) if case["bias"] else None
        s["wgu"], s["wdn"] = wgu, wdn
        if op == "ffn":
            s["res"] = normal(T, H)
            if case["mx"]:
                s["wgu"], s["wgu_s"] = _mx_quantize(wgu)
                s["wdn"], s["wdn_s"] = _mx_quantize(wdn)
                s["x"], s["x_s"] = _mx_quantize(s["x"])
        else:
            s["dy"] = normal(T, H, std=0.1)
            gu = s["x"].float() @ wgu.float().t()
            s["gu"] = gu + s["bgu"].float() if case["bias"] else gu
    if own:
        _handles(s, case)
    return s


def _handles(s, case):
    from bit_mixture_experts_amd import moe4
    op = case["op"]

    def new(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    def bytes_(n):
        return new(max(n, 256), dtype=torch.uint8)

    if op == "norm":
        T, H = case["T"], case["H"]
        s["sum"], s["rstd"] = new(T, H), new(T, dtype=torch.float32)
        s["out"] = new(T, H) if case["bf16"] else None
        s["q"] = new(T, H, dtype=torch.uint8) if case["mx"] else None
        s["qs"] = new(T, H // 32, dtype=torch.uint8) if case["mx"] else None
    elif op == "norm_bwd":
        T, H = case["T"], case["H"]
        s["dx"], s["dw"] = new(T, H), new(H, dtype=torch.float32)
        s["ws"] = bytes_(moe4.moe4_add_rmsnorm_workspace_size(T, H))
    elif op == "mxq":
        s["q"] = new(case["R"], case["K"], dtype=torch.uint8)
        s["qs"] = new(case["R"], case["K"] // 32, dtype=torch.uint8)
    elif op == "clip":
        s["outs"] = [torch.empty_like(t) for t in s["grads"]]
        s["list"] = moe4.GradList(s["grads"], s["outs"])
        s["norm"] = new(1, dtype=torch.float32)
        s["ws"] = bytes_(moe4.moe4_grad_workspace_size(s["list"]))
    else:
        T, H, I = case["T"], case["H"], case["I"]
        mx = case.get("mx", False)
        s["ffn"] = moe4.Ffn(
            moe4.MOE4_FFN_MXFP8 if mx else moe4.MOE4_FFN_BF16, s["wgu"], s["wdn"],
            gu_s=s.get("wgu_s"), dn_s=s.get("wdn_s"), gu_bias=s["bgu"], dn_bias=s["bdn"], H=H, I=I,
            gu_layout=moe4.MOE4_GU_INTERLEAVED if case["clamped"] else moe4.MOE4_GU_HALVES,
            act=moe4.MOE4_ACT_SWIGLU_CLAMPED if case["clamped"] else moe4.MOE4_ACT_SWIGLU,
            act_alpha=ALPHA, act_limit=LIMIT)
        s["ws"] = bytes_(moe4.moe4_ffn_workspace_size(s["ffn"], T, backward=op == "ffn_bwd"))
        if op == "ffn":
            s["out"] = new(T, H)
            s["gu"] = new(T, 2 * I, dtype=torch.float32) if case["train"] else None
        else:
            s["dx"], s["dwgu"], s["dwdn"] = new(T, H), new(2 * I, H), new(H, I)
            s["dbgu"] = new(2 * I) if case["bias"] else None
            s["dbdn"] = new(H) if case["bias"] else None


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from bit_mixture_experts_amd import moe4
    op = s["case"]["op"]
    if op == "norm":
        moe4.moe4_add_rmsnorm(s["x"], s["w"], EPS, residual=s["res"], sum_out=s["sum"], out=s["out"],
                              out_q=s["q"], out_s=s["qs"], rstd=s["rstd"])
        return _norm_outputs(s["sum"], s["rstd"], s["out"], s["q"], s["qs"])
    if op == "norm_bwd":
        moe4.moe4_add_rmsnorm_backward(s["dy"], s["s"], s["w"], s["rstd"], s["dx"], dres=s["dres"],
                                       dweight=s["dw"], ws=s["ws"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "mxq":
        moe4.moe4_quantize_mxfp8(s["x"], s["q"], s["qs"])
        return _mx_views(s["q"], s["qs"])
    if op == "clip":
        moe4.moe4_clip_grads(s["list"], s["max_norm"], s["norm"], s["ws"])
        return {"norm": s["norm"], "grads": s["outs"]}
    if op == "ffn":
        moe4.moe4_ffn_forward(s["ffn"], s["x"], s["out"], x_s=s.get("x_s"), residual=s["res"],
                              save_gu=s["gu"], ws=s["ws"])
        return {"y": s["out"], "gu": s["gu"]}
    moe4.moe4_ffn_backward(s["ffn"], s["x"], s["gu"], s["dy"], s["dx"], dw_gu=s["dwgu"],
                           dw_dn=s["dwdn"], db_gu=s["dbgu"], db_dn=s["dbdn"], ws=s["ws"])
    return {"dx": s["dx"], "dwgu": s["dwgu"], "dwdn": s["dwdn"], "dbgu": s["dbgu"],
            "dbdn": s["dbdn"]}


def _mx_views(q, e):
    return {"q": q.view(torch.float8_e4m3fn), "scale": e.view(torch.float8_e8m0fnu)}


def _norm_outputs(sum_, rstd, out, q, e):
    r = {"sum": sum_, "rstd": rstd, "out": out}
    if q is not None:
        r.update(_mx_views(q, e))
    return r


# the plain forms: elementary operations in 32 bits, rounded at the end

def _mx_quantize(v):
    """e4m3 codes and e8m0 scales of the last axis' blocks of 32: the scale is the smallest
    power of two that brings the block's largest magnitude to at most 448."""
    b = v.float().unflatten(-1, (-1, 32))
    m, ex = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = (ex - 9 + (m > 0.875).int()).clamp_(-127, 127)
    e = torch.where(m == 0, -127, e)
    q = torch.ldexp(b, -e).to(torch.float8_e4m3fn)
    return q.flatten(-2).view(torch.uint8), (e.squeeze(-1) + 127).to(torch.uint8)


def _mx_values(q, e):
    b = q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return torch.ldexp(b, e.int().unsqueeze(-1) - 127).flatten(-2)


def _plain_norm(s):
    c = s["case"]
    t = (s["x"].float() + s["res"].float()).to(torch.bfloat16)
    f = t.float()
    rstd = torch.rsqrt(f.square().mean(1) + EPS)
    y = f * rstd[:, None] * s["w"].float()
    q, e = _mx_quantize(y) if c["mx"] else (None, None)
    return _norm_outputs(t, rstd, y.to(torch.bfloat16) if c["bf16"] else None, q, e)


def _plain_norm_bwd(s):
    f = s["s"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    p = dy * s["w"].float()
    dx = (p - f * (p * f).mean(1, keepdim=True)) * s["rstd"][:, None] + s["dres"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * f).sum(0)}


def _plain_mxq(s):
    return _mx_views(*_mx_quantize(s["x"]))


def _plain_clip(s):
    total = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
    coef = (s["max_norm"] / (total + CLIP_EPS)).clamp(max=1.0)
    return {"norm": total.reshape(1), "grads": [(t.float() * coef).to(t.dtype) for t in s["grads"]]}


def _split(gu, clamped):
    """gate and up pre-activations: interleaved rows in the clamped block, halves in the other"""
    return (gu[..., 0::2], gu[..., 1::2]) if clamped else gu.chunk(2, -1)


def _join(g, u, clamped):
    return torch.stack((g, u), -1).flatten(-2) if clamped else torch.cat((g, u), -1)


def _act(g, u, clamped):
    if not clamped:
        return g * torch.sigmoid(g) * u
    g, u = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
    return (u + 1) * g * torch.sigmoid(ALPHA * g)


def _act_backward(g, u, dh, clamped):
    if not clamped:
        sg = torch.sigmoid(g)
        return dh * u * sg * (1 + g * (1 - sg)), dh * g * sg
    gc, uc = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
    sg = torch.sigmoid(ALPHA * gc)
    dg = dh * (uc + 1) * sg * (1 + ALPHA * gc * (1 - sg))
    return dg * (g <= LIMIT), dh * gc * sg * (u.abs() <= LIMIT)


def _plain_ffn(s):
    c = s["case"]
    if c["mx"]:
        x, wgu, wdn = (_mx_values(s[k], s[k + "_s"]) for k in ("x", "wgu", "wdn"))
    else:
        x, wgu, wdn = s["x"].float(), s["wgu"].float(), s["wdn"].float()
    gu = x @ wgu.t()
    if c["bias"]:
        gu += s["bgu"].float()
    h = _act(*_split(gu, c["clamped"]), c["clamped"])
    if c["mx"]:
        h = _mx_values(*_mx_quantize(h))
    y = h @ wdn.t()
    if c["bias"]:
        y += s["bdn"].float()
    return {"y": (y + s["res"].float()).to(torch.bfloat16), "gu": gu if c["train"] else None}


def _plain_ffn_bwd(s):
    c = s["case"]
    x, wgu, wdn, dy = (s[k].float() for k in ("x", "wgu", "wdn", "dy"))
    g, u = _split(s["gu"], c["clamped"])
    h = _act(g, u, c["clamped"])
    dgu = _join(*_act_backward(g, u, dy @ wdn, c["clamped"]), c["clamped"])
    r = {"dx": dgu @ wgu, "dwgu": dgu.t() @ x, "dwdn": dy.t() @ h,
         "dbgu": dgu.sum(0) if c["bias"] else None, "dbdn": dy.sum(0) if c["bias"] else None}
    return {k: None if v is None else v.to(torch.bfloat16) for k, v in r.items()}


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "mxq": _plain_mxq, "clip": _plain_clip,
          "ffn": _plain_ffn, "ffn_bwd": _plain_ffn_bwd}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_mx(v):
    """(codes as values, scales as values) by logarithms and steps, in 64 bits"""
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    top = b.abs().max(dim=-1, keepdim=True).values
    e = torch.ceil(torch.log2(top / 448))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top == 0, torch.full_like(e, -127.0), e.clamp(-127, 127))
    q = b * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(q / step) * step).reshape(v.shape), torch.exp2(e.squeeze(-1))


def _exact_deq(q, e):
    """e4m3 bytes times powers of two, from the fields of the bytes"""
    b = q.to(torch.int64)
    ex, man = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(ex == 0, man * 2.0 ** -9, (8 + man) * torch.exp2((ex - 10).double()))
    val = torch.where(b >= 128, -mag, mag)
    return val * torch.exp2(e.double() - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    op = case["op"]
    if op == "norm":
        t = (s["x"].double() + s["res"].double()).to(torch.bfloat16)
        d = t.double()
        rstd = 1 / torch.sqrt((d * d).sum(1) / case["H"] + EPS)
        y = torch.einsum("th,t,h->th", d, rstd, s["w"].double())
        q, e = _exact_mx(y) if case["mx"] else (None, None)
        r = {"sum": t, "rstd": rstd, "out": y if case["bf16"] else None}
        return {**r, "q": q, "scale": e} if case["mx"] else r
    if op == "norm_bwd":
        n = s["s"].double() * s["rstd"].double().unsqueeze(1)
        p = s["dy"].double() * s["w"].double()
        inner = (p * n).sum(1, keepdim=True) / case["H"]
        return {"dx": s["rstd"].double().unsqueeze(1) * (p - inner * n) + s["dres"].double(),
                "dw": torch.einsum("th,th->h", s["dy"].double(), n)}
    if op == "mxq":
        q, e = _exact_mx(s["x"].double())
        return {"q": q, "scale": e}
    if op == "clip":
        total = math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in s["grads"]))
        k = min(1.0, s["max_norm"] / (total + CLIP_EPS))
        return {"norm": torch.tensor([total], dtype=torch.float64),
                "grads": [t.double() * k for t in s["grads"]]}
    T, H, I = case["T"], case["H"], case["I"]
    gi = torch.arange(I, device="cuda")
    gate, up = (2 * gi, 2 * gi + 1) if case["clamped"] else (gi, I + gi)
    lim, al = (LIMIT, ALPHA) if case["clamped"] else (math.inf, 1.0)
    if op == "ffn":
        if case["mx"]:
            x, wgu, wdn = (_exact_deq(s[k], s[k + "_s"]) for k in ("x", "wgu", "wdn"))
        else:
            x, wgu, wdn = (s[k].double() for k in ("x", "wgu", "wdn"))
        gu = torch.matmul(x, wgu.T.contiguous())
        if case["bias"]:
            gu = gu + s["bgu"].double()
    else:
        x, wgu, wdn, gu = s["x"].double(), s["wgu"].double(), s["wdn"].double(), s["gu"].double()
    g, u = gu[:, gate], gu[:, up]
    gm, um = torch.minimum(g, torch.full_like(g, lim)), u.clamp(min=-lim, max=lim)
    sig = 1 / (1 + torch.exp(-al * gm))
    lin = um + 1 if case["clamped"] else um
    h = gm * sig * lin
    if op == "ffn":
        if case["mx"]:
            q, e = _exact_mx(h)
            h = q * e.repeat_interleave(32, dim=-1)
        y = torch.matmul(h, wdn.T.contiguous()) + s["res"].double()
        if case["bias"]:
            y = y + s["bdn"].double()
        return {"y": y, "gu": gu if case["train"] else None}
    dy = s["dy"].double()
    dh = torch.matmul(dy, wdn)
    dgu = torch.zeros_like(gu)
    dgu[:, gate] = torch.where(g > lim, 0.0, dh * lin * (sig + al * gm * sig * (1 - sig)))
    dgu[:, up] = torch.where(u.abs() > lim, 0.0, dh * gm * sig)
    return {"dx": torch.matmul(dgu, wgu), "dwgu": torch.matmul(dgu.T.contiguous(), x),
            "dwdn": torch.matmul(dy.T.contiguous(), h),
            "dbgu": dgu.sum(0) if case["bias"] else None,
            "dbdn": dy.sum(0) if case["bias"] else None}
