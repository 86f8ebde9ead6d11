"""Operators of a training step's end, as measured work: norms with their gradients, and gradient clipping.

* ``ln_fwd``: layer norm over the last axis with weight and bias, which also returns each row's mean and 1 / deviation;
* ``ln_bwd``: its gradient for the input (on top of a residual stream's gradient, where there is one), weight and bias;
* ``mod_bwd``: the gradient of the block's modulated RMSNorm for its input and for each element's shift and scale;
* ``clip``: the 2-norm over many gradient tensors, and the gradients scaled down to a largest norm.

``listed()`` and ``draw(rng)`` give the cases, ``prepare(case, seed)`` a case's tensors, ``run(state)``
one pass: with ``own`` false in elementary torch operations, with ``own`` true through the library.
``exact(case, seed)`` is the same in 64 bits, from the definitions.
"""
import math
import random

import torch

own = False

EPS = 1e-6       # of both norms
CLIP_EPS = 1e-6  # added to the gradients' norm before it divides
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a tiny picture (8 x 8 tokens behind 10 prompt rows): the latency of a forward
        {"name": "ln_tiny", "op": "ln_fwd", "rows": 74, "width": 256, "type": "bf16", "weights": "bf16"},
        # features of an odd width in 32 bits, as a head in front of a classifier has them: rows at every alignment
        {"name": "ln_ragged", "op": "ln_fwd", "rows": 9237, "width": 1155, "type": "f32", "weights": "f32"},
        # a 2048 x 2048 picture (128 x 128 tokens behind 34 prompt rows) at the largest width of a block
        {"name": "ln_long", "op": "ln_fwd", "rows": 16418, "width": 4096, "type": "bf16", "weights": "bf16"},
        # the tiny picture's gradient: launches and one row's latency
        {"name": "lnb_tiny", "op": "ln_bwd", "rows": 74, "width": 256, "type": "bf16", "weights": "bf16", "residual": False},
        # ragged rows of an odd width in fp16 under 32-bit weights
        {"name": "lnb_ragged", "op": "ln_bwd", "rows": 4503, "width": 1283, "type": "f16", "weights": "f32", "residual": False},
        # a batch of two 1024 x 1024 pictures, 20 heads wide, with the gradient that comes past the norm
        {"name": "lnb_picture", "op": "ln_bwd", "rows": 8260, "width": 2560, "type": "bf16", "weights": "bf16",
         "residual": True},
        # the tiny block's modulated norm
        {"name": "mod_tiny", "op": "mod_bwd", "batch": 1, "seq": 74, "hidden": 256, "residual": True},
        # a batch of two 1024 x 1024 pictures at the block's width
        {"name": "mod_picture", "op": "mod_bwd", "batch": 2, "seq": 4130, "hidden": 3072, "residual": True},
        # three video elements of 10,571 tokens, 14 heads wide
        {"name": "mod_video", "op": "mod_bwd", "batch": 3, "seq": 10571, "hidden": 1792, "residual": False},
        # the gradients of one tiny block (six tensors), below the limit: the latency of a step that changes nothing
        {"name": "clip_tiny", "op": "clip", "layout": "blocks", "blocks": 1, "hidden": 256, "inter": 1024, "clipped": False},
        # the gradients of four blocks of the 1024 x 1024 model, over the limit, scaled into a second set
        {"name": "clip_blocks", "op": "clip", "layout": "blocks", "blocks": 4, "hidden": 3072, "inter": 8192,
         "clipped": True},
        # 700 tensors of odd sizes back to back in one bucket of each type, as a flattened optimizer keeps them
        {"name": "clip_bucket", "op": "clip", "layout": "bucket", "tensors": 700, "largest": 400000, "sizes": 11,
         "f32_share": 0.3, "clipped": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "mod_bwd", "clip"])
    if op in ("ln_fwd", "ln_bwd"):
        kind = rng.choice(["bf16", "bf16", "f16", "f32"])
        width = _log_int(rng, 24, 8192)
        if rng.random() < 0.6:
            width = max(8, width // 8 * 8)
        most = 16418 * 4096 // (width * (2 if kind == "f32" else 1)) // (2 if op == "ln_bwd" else 1)
        case = {"op": op, "rows": _log_int(rng, 1, min(100000, most)), "width": width, "type": kind,
                "weights": rng.choice([kind, "f32"])}
        return case if op == "ln_fwd" else {**case, "residual": rng.random() < 0.5}
    if op == "mod_bwd":
        batch, hidden = rng.randint(1, 4), 256 * rng.randint(1, 16)
        most = 2 * 4130 * 3072 // (batch * hidden)
        return {"op": op, "batch": batch, "seq": _log_int(rng, 1, min(16418, most)), "hidden": hidden,
                "residual": rng.random() < 0.5}
    clipped = rng.random() < 0.6
    if rng.random() < 0.4:
        hidden = 128 * rng.randint(2, 20)
        return {"op": op, "layout": "blocks", "blocks": rng.randint(1, 4), "hidden": hidden, "inter": 128 * rng.randint(4, 60),
                "clipped": clipped}
    return {"op": op, "layout": "bucket", "tensors": _log_int(rng, 1, 1500), "largest": _log_int(rng, 10, 300000),
            "sizes": rng.randint(0, 1 << 30), "f32_share": rng.choice([0.0, 0.3, 1.0]), "clipped": clipped}


def _block_shapes(case):
    """A block's weights (16 bits) and gains (32 bits), as the training pass gives their gradients."""
    h, i = case["hidden"], case["inter"]
    one = [(3 * h, h, torch.bfloat16), (h, h, torch.bfloat16), (2 * i, h, torch.bfloat16), (h, i, torch.bfloat16),
           (1, 128, torch.float32), (1, 128, torch.float32)]
    return one * case["blocks"]


def _bucket_sizes(case):
    """Elements and type of every tensor of a bucket, sizes spread over their logarithm."""
    rng = random.Random(case["sizes"])
    return [(_log_int(rng, 1, case["largest"]), torch.float32 if rng.random() < case["f32_share"] else torch.bfloat16)
            for _ in range(case["tensors"])]


def _size(dtype):
    return 4 if dtype == torch.float32 else 2


def work(case):
    if case["op"] == "clip":
        if case["layout"] == "blocks":
            sizes = [(r * c, t) for r, c, t in _block_shapes(case)]
        else:
            sizes = _bucket_sizes(case)
        elements, size = sum(n for n, _ in sizes), sum(n * _size(t) for n, t in sizes)
        return {"bytes": (2 if case["clipped"] else 1) * size + 4, "flops": (3 if case["clipped"] else 2) * elements}
    if case["op"] == "mod_bwd":
        h, b = case["hidden"], case["batch"]
        n = b * case["seq"] * h
        return {"bytes": 2 * n * (4 if case["residual"] else 3) + b * h * (2 + 8), "flops": 13 * n}
    n, w = case["rows"] * case["width"], case["width"]
    e, p = _size(TYPES[case["type"]]), _size(TYPES[case["weights"]])
    if case["op"] == "ln_fwd":
        return {"bytes": 2 * n * e + 8 * case["rows"] + 2 * w * p, "flops": 8 * n}
    return {"bytes": n * e * (4 if case["residual"] else 3) + 8 * case["rows"] + w * (p + 8), "flops": 13 * n}


# ----------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    def stream(rows, width, dtype):
        """A residual stream: every channel around a mean of its own, rows of different size."""
        x = torch.randn(rows, width, generator=gen, device="cuda")
        x.add_(torch.randn(1, width, generator=gen, device="cuda"))
        return x.mul_(0.5 + torch.rand(rows, 1, generator=gen, device="cuda")).to(dtype)

    s = {"case": dict(case)}
    if case["op"] in ("ln_fwd", "ln_bwd"):
        rows, width, t, p = case["rows"], case["width"], TYPES[case["type"]], TYPES[case["weights"]]
        s["x"] = stream(rows, width, t)
        s["weight"] = normal(width, std=0.1, mean=1.0, dtype=p)
        if case["op"] == "ln_fwd":
            s["bias"] = normal(width, std=0.1, dtype=p)
            s["y"] = torch.empty_like(s["x"])
            s["mean"] = torch.empty(rows, device="cuda")
            s["rstd"] = torch.empty(rows, device="cuda")
            return s
        _, s["mean"], s["rstd"] = _layer_norm(s["x"], s["weight"], torch.zeros_like(s["weight"]))
        s["dy"] = normal(rows, width, std=0.02, dtype=t)
        s["residual"] = normal(rows, width, std=0.02, dtype=t) if case["residual"] else None
        s["dx"] = torch.empty_like(s["x"])
        s["dweight"] = torch.empty(width, device="cuda")
        s["dbias"] = torch.empty(width, device="cuda")
        return s
    if case["op"] == "mod_bwd":
        batch, seq, hidden = case["batch"], case["seq"], case["hidden"]
        s["x"] = stream(batch * seq, hidden, torch.bfloat16)
        s["mod"] = normal(batch, 6, hidden, std=0.1)
        s["dy"] = normal(batch * seq, hidden, std=0.02)
        s["residual"] = normal(batch * seq, hidden, std=0.02) if case["residual"] else None
        s["dx"] = torch.empty_like(s["x"])
        s["dmod"] = torch.zeros(batch, 6, hidden, device="cuda")
        return s
    if case["layout"] == "blocks":
        s["grads"] = [normal(r, c, std=0.01, dtype=t) for r, c, t in _block_shapes(case)]
        s["outs"] = [torch.empty_like(g) for g in s["grads"]] if case["clipped"] else s["grads"]
        s["whole"] = s["outs"]
    else:
        sizes = _bucket_sizes(case)
        s["grads"], s["outs"], s["whole"] = [None] * len(sizes), [None] * len(sizes), []
        for t in (torch.bfloat16, torch.float32):
            mine = [i for i, (_, kind) in enumerate(sizes) if kind == t]
            if not mine:
                continue
            lengths = [sizes[i][0] for i in mine]
            flat = normal(sum(lengths), std=0.01, dtype=t)
            out = torch.empty_like(flat) if case["clipped"] else flat
            s["whole"].append(out)
            for i, g, o in zip(mine, flat.split(lengths), out.split(lengths)):
                s["grads"][i], s["outs"][i] = g, o
    count = sum(g.numel() for g in s["grads"])
    s["limit"] = 0.01 * math.sqrt(count) * (0.3 if case["clipped"] else 4.0)  # the norm is near 0.01 sqrt(count)
    s["norm"] = torch.empty(1, device="cuda")
    return s


# ------------------------------------------------------------------------------------- plain forms
def _layer_norm(x, weight, bias):
    f = x.float()
    mean = f.mean(1, keepdim=True)
    f = f - mean
    rstd = (f.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = (f * rstd * weight.float() + bias.float()).to(x.dtype)
    return y, mean.squeeze(1), rstd.squeeze(1)


def _layer_norm_backward(s):
    x, dy, rstd = s["x"], s["dy"].float(), s["rstd"].unsqueeze(1)
    n = (x.float() - s["mean"].unsqueeze(1)) * rstd
    dweight, dbias = (dy * n).sum(0, dtype=torch.float64).float(), dy.sum(0, dtype=torch.float64).float()  # long sums
    g = dy * s["weight"].float()
    dx = (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True)) * rstd
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return dx.to(x.dtype), dweight, dbias


def _mod_backward(s):
    case = s["case"]
    shape = (case["batch"], case["seq"], case["hidden"])
    x, dy = s["x"].view(shape).float(), s["dy"].view(shape).float()
    r = (x.square().mean(2, keepdim=True) + EPS).rsqrt()
    n = x * r
    dscale, dshift = (dy * n).sum(1, dtype=torch.float64).float(), dy.sum(1, dtype=torch.float64).float()  # long sums
    g = dy * (1.0 + s["mod"][:, 1:2].float())
    dx = (g - n * (g * n).mean(2, keepdim=True)) * r
    if s["residual"] is not None:
        dx = dx + s["residual"].view(shape).float()
    return dx.bfloat16().view_as(s["x"]), dshift, dscale


def _by_type(grads):
    """A bucket's tensors of one type in one piece: the elementary operations then run once for each type."""
    return [torch.cat(part) for t in (torch.bfloat16, torch.float32) if (part := [g for g in grads if g.dtype == t])]


def _clip(s):
    grads = s["grads"] if s["case"]["layout"] == "blocks" else _by_type(s["grads"])
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum()  # a long sum
    norm = total.sqrt().float().view(1)
    c = (s["limit"] / (norm + CLIP_EPS)).clamp(max=1.0)
    return norm, [(g.float() * c).to(g.dtype) for g in grads]


# ----------------------------------------------------------------------------------- the operators
def _own(s):
    import diffusion_transformer_denoiser_gb300 as mi

    case = s["case"]
    op = case["op"]
    if op == "ln_fwd":
        mi.layer_norm(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], eps=EPS)
        return s["y"], s["mean"], s["rstd"]
    if "ws" not in s:  # a program plans its workspaces, and which gradients it clips, once
        if op == "clip":
            s["set"] = mi.GradSet(s["grads"], s["outs"] if case["clipped"] else None)
            size = s["set"].workspace_size()
        elif op == "ln_bwd":
            size = mi.layer_norm_backward_workspace_size(case["rows"], case["width"])
        else:
            size = mi.mod_rmsnorm_backward_workspace_size(case["batch"], case["seq"], case["hidden"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if op == "ln_bwd":
        mi.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"], s["ws"],
                               residual=s["residual"])
        return s["dx"], s["dweight"], s["dbias"]
    if op == "mod_bwd":
        mi.mod_rmsnorm_backward(s["dy"], s["x"], s["mod"], 0, 1, s["dx"], s["dmod"], case["batch"], case["seq"], s["ws"],
                                eps=EPS, residual=s["residual"])
        return s["dx"], s["dmod"][:, 0], s["dmod"][:, 1]
    s["set"].clip_norm(s["limit"], s["norm"], s["ws"])
    return s["norm"], s["whole"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "ln_fwd":
        return _layer_norm(state["x"], state["weight"], state["bias"])
    return {"ln_bwd": _layer_norm_backward, "mod_bwd": _mod_backward, "clip": _clip}[op](state)


# ----------------------------------------------------------------------------------------- 64 bits
def _exact_norm(x, dy, factor, shift, root):
    """The chain rule on y = factor (x - shift) / root, row by row: the part of dx that the row's own statistics
    leave, from the projections on them.  Returns the normalised rows and dx (without the mean's part)."""
    n = (x - shift) / root
    g = dy * factor
    return n, (g - n * ((g * n).sum(-1, keepdim=True) / x.shape[-1])) / root


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ln_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        deviation = torch.sqrt(var + EPS)
        y = (x - mean[:, None]) / deviation[:, None]
        return torch.addcmul(s["bias"].double(), y, s["weight"].double()), mean, 1.0 / deviation
    if case["op"] == "ln_bwd":
        # the gradient for the statistics that are given, so that they need not be x's to the last bit
        n, dx = _exact_norm(s["x"].double(), s["dy"].double(), s["weight"].double(), s["mean"].double()[:, None],
                            1.0 / s["rstd"].double()[:, None])
        dx -= (s["dy"].double() @ s["weight"].double() / case["width"] * s["rstd"].double())[:, None]
        if s["residual"] is not None:
            dx += s["residual"]
        return dx, torch.einsum("rw,rw->w", s["dy"].double(), n), s["dy"].double().sum(0)
    if case["op"] == "mod_bwd":
        parts = []
        for x, dy, mod in zip(s["x"].chunk(case["batch"]), s["dy"].chunk(case["batch"]), s["mod"].double()):
            x, dy = x.double(), dy.double()
            root = torch.sqrt((x * x).sum(1, keepdim=True) / case["hidden"] + EPS)
            n, dx = _exact_norm(x, dy, 1.0 + mod[1], 0.0, root)
            parts.append((dx, dy.sum(0), torch.einsum("rw,rw->w", dy, n)))
        dx = torch.cat([p[0] for p in parts])
        if s["residual"] is not None:
            dx += s["residual"]
        return dx, torch.stack([p[1] for p in parts]), torch.stack([p[2] for p in parts])
    sources = s["grads"] if case["layout"] == "blocks" else _by_type(s["grads"])
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in sources))
    c = min(1.0, s["limit"] / (norm + CLIP_EPS))
    return torch.tensor([norm], dtype=torch.float64, device="cuda"), [g.double() * c for g in sources]
