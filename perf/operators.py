"""Cases of the operators around a W8A8 transformer block: the 8-bit integer linear layer (per-token and per-channel
scales), the (modulated) layer norm with its backward pass, and rotary positions over several axes.

Every case is measured in its plain form (elementary torch operations) and through the public calls of
``w4a4_diffusion_model_b200.svdq``. ``prepare`` holds what a user's program holds before the call: activations, prepared
weights, position ids and the rotary frequencies; ``run`` makes one pass.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # The modulation linear of a transformer block: the timestep embedding of a guided pair (two rows) gives shifts,
        # scales and gates for six places. Nothing but the weights is read: bandwidth and latency.
        {"name": "int8_modulation", "op": "int8", "M": 2, "K": 4096, "N": 24576, "dtype": "bf16", "smooth": False, "bias": True},
        # A caption of odd length through a projection whose sizes are no multiple of any tile, in fp32.
        {"name": "int8_text", "op": "int8", "M": 333, "K": 1360, "N": 2305, "dtype": "fp32", "smooth": True, "bias": False},
        # A merged QKV projection over 4096 image and 512 text tokens, smoothed.
        {"name": "int8_qkv", "op": "int8", "M": 4608, "K": 4096, "N": 12288, "dtype": "bf16", "smooth": True, "bias": True},
        # The second feed-forward projection over the tokens of a video clip, a ragged row count: the largest product.
        {"name": "int8_mlp_down", "op": "int8", "M": 9001, "K": 13824, "N": 5120, "dtype": "bf16", "smooth": True, "bias": True},
        # The norm of one pooled embedding: latency.
        {"name": "ln_token", "op": "ln", "M": 1, "C": 1152, "groups": 1, "dtype": "fp16", "wtype": "fp16", "add_one": False},
        # The modulated norm before a block's projections, two images of 4608 tokens, each with its own scale and shift.
        {"name": "ln_modulated", "op": "ln", "M": 9216, "C": 4096, "groups": 2, "dtype": "bf16", "wtype": "bf16", "add_one": True},
        # Backward of a caption's norm in fp32 with an odd width.
        {"name": "ln_backward_text", "op": "ln_backward", "M": 226, "C": 1151, "groups": 1, "dtype": "fp32", "wtype": "fp32", "add_one": False},
        # Backward of the modulated norm: the gradients of two images' scales and shifts.
        {"name": "ln_backward_modulated", "op": "ln_backward", "M": 9216, "C": 4096, "groups": 2, "dtype": "bf16", "wtype": "bf16", "add_one": True},
        # Backward of an affine norm over a video clip's tokens, with fp32 weights: the largest reduction over rows.
        {"name": "ln_backward_video", "op": "ln_backward", "M": 32760, "C": 5120, "groups": 1, "dtype": "bf16", "wtype": "fp32", "add_one": False},
        # A few tokens with shared key heads and a small head: latency.
        {"name": "rope_tokens", "op": "rope", "F": 1, "H": 1, "W": 7, "text": 0, "heads": 40, "parts": 1, "D": 80, "axes": "16,32,32", "dtype": "fp16", "interleaved": True, "inverse": False, "ids": "int32", "start": 1000},
        # The query and key heads inside a merged QKV activation: 64 x 64 image tokens after 512 text tokens at position 0.
        {"name": "rope_image", "op": "rope", "F": 1, "H": 64, "W": 64, "text": 512, "heads": 48, "parts": 3, "D": 128, "axes": "16,56,56", "dtype": "bf16", "interleaved": True, "inverse": False, "ids": "fp32", "start": 0},
        # The gradient through the rotation for a video latent of 21 x 30 x 52 tokens, halves rotated against each other.
        {"name": "rope_video_gradient", "op": "rope", "F": 21, "H": 30, "W": 52, "text": 0, "heads": 40, "parts": 1, "D": 128, "axes": "44,42,42", "dtype": "bf16", "interleaved": False, "inverse": True, "ids": "int32", "start": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["int8", "int8", "ln", "ln_backward", "rope"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "int8":
        while True:   # rows from one token to a clip's; K in steps of 16; N of any size, mostly in steps of 8
            M, K, N = _log(rng, 1, 9216), 16 * _log(rng, 24, 896), _log(rng, 200, 24576)
            N = N if rng.random() < 0.3 else (N + 7) // 8 * 8
            if M * K * N <= 4608 * 4096 * 12288:
                break
        return {"op": op, "M": M, "K": K, "N": N, "dtype": dtype, "smooth": rng.random() < 0.5, "bias": rng.random() < 0.5}
    if op in ("ln", "ln_backward"):
        while True:
            M, C = _log(rng, 1, 65536), _log(rng, 48, 16384)
            if M * C * SIZES[dtype] <= 9216 * 4096 * 4:
                break
        C = C if rng.random() < 0.4 else (C + 15) // 16 * 16
        groups = rng.choice([1, 1, 2, 4])
        return {"op": op, "M": (M + groups - 1) // groups * groups, "C": C, "groups": groups, "dtype": dtype,
                "wtype": rng.choice([dtype, "fp32"]), "add_one": rng.random() < 0.5}
    D = rng.choice([64, 80, 96, 128, 256])
    rot = D if rng.random() < 0.7 else D // 2          # the whole head, or its first half only
    a = 2 * rng.randint(1, rot // 4)
    b = 2 * rng.randint(1, (rot - a) // 2 - 1) if rot - a > 2 else 0
    axes = [a, b, rot - a - b] if b else [a, rot - a]
    while True:
        F, H, W, text, heads = rng.choice([1, 1, 3, 13]), _log(rng, 1, 96), _log(rng, 1, 96), rng.choice([0, 0, 77, 512]), _log(rng, 1, 64)
        if (F * H * W + text) * heads * D * SIZES[dtype] <= 4608 * 48 * 128 * 4:
            break
    return {"op": op, "F": F, "H": H, "W": W, "text": text, "heads": heads, "parts": rng.choice([1, 1, 3]), "D": D,
            "axes": ",".join(str(x) for x in axes), "dtype": dtype, "interleaved": rng.random() < 0.5,
            "inverse": rng.random() < 0.5, "ids": rng.choice(["int32", "fp32"]), "start": rng.choice([0, 0, 17, 100000])}


def _activations(M, C, dtype, g):
    """Token activations: a few channels are many times larger than the rest, and every channel has its own mean."""
    dev = g.device
    size = torch.exp(0.5 * torch.randn(C, generator=g, device=dev))
    size = torch.where(torch.rand(C, generator=g, device=dev) < 0.01, size * 20, size)
    x = torch.randn(M, C, generator=g, device=dev)
    x.add_(0.3 * torch.randn(C, generator=g, device=dev)).mul_(size)
    return x.to(DTYPES[dtype])


def _rope_inputs(case, g):
    dev = g.device
    T, axes = case["F"] * case["H"] * case["W"] + case["text"], [int(x) for x in case["axes"].split(",")]
    t = torch.arange(T - case["text"], device=dev)
    grid = torch.stack([t // (case["H"] * case["W"]), t // case["W"] % case["H"], t % case["W"]], 1)[:, 3 - len(axes):] + case["start"]
    ids = torch.cat([torch.zeros(case["text"], len(axes), dtype=grid.dtype, device=dev), grid])
    ids = ids.to(torch.int32 if case["ids"] == "int32" else torch.float32).contiguous()
    # with three parts the heads are the first two thirds (query and key) of a merged projection's output
    per = case["heads"] if case["parts"] == 1 else (case["heads"] + 1) // 2 * 3
    x = torch.randn(T, per, case["D"], generator=g, device=dev).to(DTYPES[case["dtype"]])[:, :case["heads"]]
    return x, ids, axes


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "int8":
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = _activations(M, K, case["dtype"], g)
        w = (torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)).to(torch.bfloat16)
        s["bias"] = torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        lam = torch.exp(0.4 * torch.randn(K, generator=g, device="cuda")) if case["smooth"] else None
        s["inv_lam"] = 1.0 / lam if case["smooth"] else None
        # the weights' codes are laid out once, as the model is loaded
        what = w.float() * lam if case["smooth"] else w.float()
        sw = what.abs().amax(1) / 127.0
        qw = torch.round(what.double() / sw.double()[:, None]).clamp_(-127, 127).to(torch.int8)
        s["qw"], s["sw"] = qw, sw
        if own:
            from w4a4_diffusion_model_b200 import svdq
            s["weights"] = svdq.Int8Weights(N, K, qw, sw, s["inv_lam"], s["bias"])
        return s
    if case["op"] in ("ln", "ln_backward"):
        M, C, G = case["M"], case["C"], case["groups"]
        s["x"] = _activations(M, C, case["dtype"], g)
        w = 0.3 * torch.randn(G, C, generator=g, device="cuda")
        s["weight"] = (w if case["add_one"] else w + 1).to(DTYPES[case["wtype"]])
        s["bias"] = (0.3 * torch.randn(G, C, generator=g, device="cuda")).to(DTYPES[case["wtype"]])
        s["eps"] = 1e-6
        if case["op"] == "ln_backward":   # the forward pass kept its rows' statistics
            s["dy"] = torch.randn(M, C, generator=g, device="cuda").to(DTYPES[case["dtype"]])
            s["mean"], s["rstd"] = _statistics(s["x"].float(), s["eps"])
        return s
    s["x"], s["ids"], s["axes"] = _rope_inputs(case, g)
    s["freqs"] = torch.cat([torch.exp(-math.log(10000.0) * torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
                            for d in s["axes"]])
    if own:
        from w4a4_diffusion_model_b200 import svdq
        s["table"] = svdq.RopeTable(tuple(s["axes"]), s["freqs"])
    return s


def _statistics(xf, eps):
    mean = xf.mean(1)
    var = (xf - mean[:, None]).square_().mean(1)
    return mean, torch.rsqrt(var + eps)


def _plain_int8(s):
    x = s["x"].float()
    if s["inv_lam"] is not None:
        x = x * s["inv_lam"]
    sx = x.abs().amax(1) / 127.0
    # codes next to a midpoint: the quotient of two fp32 values, rounded in 64 bits, has the exact quotient's code
    qx = torch.where(sx[:, None] > 0, torch.round(x.double() / sx.double()[:, None]), 0).clamp_(-127, 127)
    acc = qx.float() @ s["qw"].float().t()
    y = acc * sx[:, None] * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["x"].dtype), qx.to(torch.int8), sx


def _effective(s):
    w = s["weight"].float()
    return w + 1 if s["case"]["add_one"] else w


def _plain_ln(s):
    G, x = s["case"]["groups"], s["x"].float()
    mean, rstd = _statistics(x, s["eps"])
    xhat = ((x - mean[:, None]) * rstd[:, None]).view(G, -1, x.shape[1])
    y = xhat * _effective(s)[:, None] + s["bias"].float()[:, None]
    return y.view_as(x).to(s["x"].dtype), mean, rstd


def _plain_ln_backward(s):
    G, C = s["case"]["groups"], s["case"]["C"]
    x, dy = s["x"].float(), s["dy"].float()
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gy = (dy.view(G, -1, C) * _effective(s)[:, None]).view(-1, C)
    dx = s["rstd"][:, None] * (gy - gy.mean(1, keepdim=True) - xhat * (gy * xhat).mean(1, keepdim=True))
    dw = (dy * xhat).view(G, -1, C).sum(1)
    db = dy.view(G, -1, C).sum(1)
    return dx.to(s["x"].dtype), dw, db


def _rotate(x, cos, sin, interleaved, rot):
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(s):
    case, axes = s["case"], s["axes"]
    which = torch.cat([torch.full((d // 2,), i, device=s["ids"].device) for i, d in enumerate(axes)])
    angle = s["ids"].double()[:, which] * s["freqs"]      # far positions: 64 bits
    if case["inverse"]:
        angle = -angle
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return _rotate(s["x"].float(), cos, sin, case["interleaved"], sum(axes)).to(s["x"].dtype)


def run(s):
    case = s["case"]
    if not own:
        plain = {"int8": _plain_int8, "ln": _plain_ln, "ln_backward": _plain_ln_backward, "rope": _plain_rope}
        return plain[case["op"]](s)
    from w4a4_diffusion_model_b200 import svdq
    if case["op"] == "int8":
        qx, sx = svdq.svdq_int8_quantize_act(s["x"], s["inv_lam"])
        return svdq.svdq_int8_linear(qx, sx, s["weights"], dtype=s["x"].dtype), qx, sx
    if case["op"] == "ln":
        return svdq.svdq_layernorm(s["x"], s["weight"], s["bias"], eps=s["eps"], add_one=case["add_one"])
    if case["op"] == "ln_backward":
        return svdq.svdq_layernorm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], add_one=case["add_one"])
    return svdq.svdq_rope(s["x"], s["ids"], s["table"], interleaved=case["interleaved"], inverse=case["inverse"])


def work(case):
    es = SIZES[case["dtype"]]
    if case["op"] == "int8":
        M, K, N = case["M"], case["K"], case["N"]
        once = 4 * N + (4 * N if case["bias"] else 0) + (4 * K if case["smooth"] else 0)
        return {"bytes": M * K * es + M * K + 4 * M + N * K + M * N * es + once, "flops": 2 * M * N * K}
    if case["op"] in ("ln", "ln_backward"):
        M, C, G = case["M"], case["C"], case["groups"]
        ws = SIZES[case["wtype"]]
        if case["op"] == "ln":
            return {"bytes": 2 * M * C * es + 8 * M + 2 * G * C * ws, "flops": 8 * M * C}
        return {"bytes": 3 * M * C * es + 8 * M + G * C * ws + 8 * G * C, "flops": 15 * M * C}
    T, n = case["F"] * case["H"] * case["W"] + case["text"], len(case["axes"].split(","))
    return {"bytes": 2 * T * case["heads"] * case["D"] * es + 4 * n * T, "flops": 3 * T * case["heads"] * case["D"]}


def exact(case, seed):
    """The same outputs in 64 bits, from the operators' definitions."""
    s = prepare(case, seed)
    x = s["x"].to(torch.float64)
    if case["op"] == "int8":
        # the definition rounds the smoothed activation and its scale to fp32 once
        if case["smooth"]:
            x = (x * s["inv_lam"].to(torch.float64)).to(torch.float32).to(torch.float64)
        scale = (x.abs().max(dim=1).values / 127).to(torch.float32).to(torch.float64)
        safe = torch.where(scale == 0, torch.ones_like(scale), scale)
        codes = torch.clamp(torch.round(x / safe.unsqueeze(1)), -127, 127)
        codes[scale == 0] = 0
        y = torch.empty(case["M"], case["N"], dtype=torch.float64, device=x.device)
        for n in range(0, case["N"], 4096):
            w = s["qw"][n:n + 4096].to(torch.float64) * s["sw"][n:n + 4096].to(torch.float64).unsqueeze(1)
            y[:, n:n + 4096] = torch.matmul(codes * scale.unsqueeze(1), w.T)
        if case["bias"]:
            y += s["bias"].to(torch.float64)
        return y, codes.to(torch.int8), scale
    if case["op"] in ("ln", "ln_backward"):
        group = torch.arange(case["M"], device=x.device) // (case["M"] // case["groups"])
        gain = s["weight"].to(torch.float64) + (1.0 if case["add_one"] else 0.0)
        if case["op"] == "ln":
            centre = x.sum(1) / case["C"]
            x -= centre.unsqueeze(1)
            inv = 1.0 / torch.sqrt((x * x).sum(1) / case["C"] + s["eps"])
            return x * inv.unsqueeze(1) * gain[group] + s["bias"].to(torch.float64)[group], centre, inv
        dy = s["dy"].to(torch.float64)
        inv = s["rstd"].to(torch.float64).unsqueeze(1)
        x = (x - s["mean"].to(torch.float64).unsqueeze(1)) * inv
        dw = torch.zeros(case["groups"], case["C"], dtype=torch.float64, device=x.device).index_add_(0, group, dy * x)
        db = torch.zeros_like(dw).index_add_(0, group, dy)
        h = dy * gain[group]
        dx = inv * (h - h.sum(1, keepdim=True) / case["C"] - x * ((h * x).sum(1, keepdim=True) / case["C"]))
        return dx, dw, db
    y, at = x.clone(), 0
    rot = sum(s["axes"])
    for axis, d in enumerate(s["axes"]):
        for i in range(d // 2):
            turn = s["ids"][:, axis].to(torch.float64) * s["freqs"][at]
            if case["inverse"]:
                turn = -turn
            c, n = torch.cos(turn).unsqueeze(1), torch.sin(turn).unsqueeze(1)
            p, q = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + rot // 2)
            y[:, :, p] = x[:, :, p] * c - x[:, :, q] * n
            y[:, :, q] = x[:, :, p] * n + x[:, :, q] * c
            at += 1
    return y
