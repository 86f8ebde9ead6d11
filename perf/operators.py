"""Operators of the attention section's training pass, as measured work.

Four operators that a program calls between the QKV projection and its gradient:

* ``rope_axes``: rotary tables for tokens with several position axes (time, row, column);
* ``attn_fwd``: attention that also returns each row's log-sum-exp;
* ``attn_bwd``: attention's gradient, which recomputes the probabilities from the log-sum-exp;
* ``qk_bwd``: the gradient of the per-head q/k RMSNorm and the rotation behind it.

``listed()`` and ``draw(rng)`` give the cases, ``prepare(case, seed)`` a case's tensors, ``run(state)``
one pass: with ``own`` false in elementary torch operations, with ``own`` true through the library.
``exact(case, seed)`` is the same in 64 bits, from the definitions.
"""
import math

import torch

own = False

HEAD = 128          # head dimension
PAIRS = HEAD // 2   # rotary pairs of a head
EPS = 1e-6
SCALE = 1.0 / math.sqrt(HEAD)


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a small picture with a short prompt in one batch: the tables of a preview, launch-bound
        {"name": "rope_small", "op": "rope_axes", "rows": 420, "pairs": "32,32", "far": 0.0, "frac": False},
        # a video clip of 21 latent frames of 45 x 80 tokens behind a 226-row prompt, 16/24/24 pairs
        {"name": "rope_video", "op": "rope_axes", "rows": 75826, "pairs": "16,24,24", "far": 0.0, "frac": True},
        # two small elements, the second with a padded prompt: the latency of a training forward
        {"name": "fwd_small", "op": "attn_fwd", "batch": 2, "heads": 4, "seq": 210, "pad": 13, "empty": 0},
        # one 1024 x 1024 picture (64 x 64 tokens) behind a 34-row prompt
        {"name": "fwd_picture", "op": "attn_fwd", "batch": 1, "heads": 24, "seq": 4130, "pad": 0, "empty": 0},
        # a batch of ragged sequences with padded keys and one element without any valid key
        {"name": "fwd_padded", "op": "attn_fwd", "batch": 3, "heads": 10, "seq": 1501, "pad": 300, "empty": 1},
        # a tiny picture (8 x 8 tokens, 10 prompt rows) of two heads: the latency of a gradient
        {"name": "bwd_tiny", "op": "attn_bwd", "batch": 1, "heads": 2, "seq": 74, "pad": 0, "empty": 0},
        # the padded batch of above, one element of it empty: masked keys, zero gradients, odd length
        {"name": "bwd_padded", "op": "attn_bwd", "batch": 3, "heads": 10, "seq": 1501, "pad": 300, "empty": 1},
        # one 1024 x 1024 picture: the ordinary training step
        {"name": "bwd_picture", "op": "attn_bwd", "batch": 1, "heads": 24, "seq": 4130, "pad": 0, "empty": 0},
        # one 2048 x 2048 picture (128 x 128 tokens): the longest sequence
        {"name": "bwd_long", "op": "attn_bwd", "batch": 1, "heads": 24, "seq": 16418, "pad": 0, "empty": 0},
        # the tiny picture's norm and rotation, tables shared by the batch
        {"name": "qk_tiny", "op": "qk_bwd", "batch": 1, "heads": 2, "seq": 74, "tables": "shared"},
        # a batch of two 1024 x 1024 pictures, tables shared by the batch
        {"name": "qk_picture", "op": "qk_bwd", "batch": 2, "heads": 24, "seq": 4130, "tables": "shared"},
        # ragged video elements with tables of their own each
        {"name": "qk_video", "op": "qk_bwd", "batch": 3, "heads": 14, "seq": 10571, "tables": "own"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope_axes", "attn_fwd", "attn_bwd", "attn_bwd", "qk_bwd"])
    if op == "rope_axes":
        n = rng.randint(1, 4)
        cuts = sorted(rng.sample(range(1, PAIRS), n - 1))
        pairs = [b - a for a, b in zip([0] + cuts, cuts + [PAIRS])]
        return {"op": op, "rows": _log_int(rng, 33, 75826), "pairs": ",".join(map(str, pairs)),
                "far": rng.choice([0.0, 0.0, 1000.0, 100000.0]), "frac": rng.random() < 0.5}
    batch = rng.choice([1, 1, 2, 3, 4])
    if op == "qk_bwd":
        heads = rng.randint(1, 32)
        top = 3 * 14 * 10571 // (batch * heads)
        return {"op": op, "batch": batch, "heads": heads, "seq": _log_int(rng, 17, max(18, min(16418, top))),
                "tables": rng.choice(["shared", "own"])}
    heads = _log_int(rng, 1, 30)
    top = int(16418 * math.sqrt(24.0 / max(24, batch * heads)))
    seq = _log_int(rng, 17, top)
    pad = rng.choice([0, 0, rng.randint(1, max(1, min(seq - 16, seq // 2)))])
    return {"op": op, "batch": batch, "heads": heads, "seq": seq, "pad": pad,
            "empty": 1 if batch > 1 and rng.random() < 0.3 else 0}


def _valid_keys(case):
    """Keys that may be attended to, over the batch (see _mask)."""
    total = case["batch"] * case["seq"]
    if case["empty"]:
        total -= case["seq"]
    return total - case["pad"]


def work(case):
    if case["op"] == "rope_axes":
        axes = len(case["pairs"].split(","))
        return {"bytes": case["rows"] * (4 * axes + 2 * 4 * PAIRS), "flops": case["rows"] * PAIRS * 4}
    rows, heads = case["batch"] * case["seq"], case["heads"]
    width = 2 * heads * HEAD  # bytes of one row of all heads
    if case["op"] == "qk_bwd":
        table_rows = rows if case["tables"] == "own" else case["seq"]
        return {"bytes": 6 * rows * width + table_rows * 2 * 4 * PAIRS + 2 * HEAD * 6, "flops": rows * heads * 2 * HEAD * 12}
    mask = rows if case["pad"] or case["empty"] else 0
    pairs = case["seq"] * _valid_keys(case) * heads
    if case["op"] == "attn_fwd":
        return {"bytes": 4 * rows * width + 4 * rows * heads + mask, "flops": 2 * 2 * HEAD * pairs}
    return {"bytes": 8 * rows * width + 4 * rows * heads + mask, "flops": 5 * 2 * HEAD * pairs}


# ----------------------------------------------------------------------------------------- inputs
def _mask(case):
    """uint8 [batch, seq] or None: `pad` keys from row 5 on of the last element are padding, and the
    first element of a batch marked `empty` has no valid key."""
    if not case["pad"] and not case["empty"]:
        return None
    m = torch.ones(case["batch"], case["seq"], dtype=torch.uint8, device="cuda")
    if case["pad"]:
        m[-1, 5:5 + case["pad"]] = 0
    if case["empty"]:
        m[0] = 0
    return m


def _positions(case, gen):
    """fp32 [rows, axes]: a row-major walk over a box of tokens, from `far` on; rows of the last axes
    change fastest.  `frac`: positions between the whole ones, as interpolated grids have them."""
    axes = len(case["pairs"].split(","))
    side = max(2, int(math.ceil(case["rows"] ** (1.0 / axes))))
    i = torch.arange(case["rows"], device="cuda")
    cols = [(i // side ** (axes - 1 - a)) % side if a else i // side ** (axes - 1) for a in range(axes)]
    pos = torch.stack(cols, 1).float()
    shift = torch.randint(0, 64, (1, axes), generator=gen, device="cuda").float()
    if case["frac"]:
        pos = pos * (0.5 + torch.rand(1, axes, generator=gen, device="cuda"))
    return (pos + shift + case["far"]).contiguous()


def _tables(rows, gen):
    angle = torch.rand(rows, PAIRS, generator=gen, device="cuda") * 60.0
    return torch.cos(angle), torch.sin(angle)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).bfloat16()

    s = {"case": dict(case)}
    if case["op"] == "rope_axes":
        s["pos"] = _positions(case, gen)
        s["pairs"] = tuple(int(p) for p in case["pairs"].split(","))
        s["cos"] = torch.empty(case["rows"], PAIRS, device="cuda")
        s["sin"] = torch.empty_like(s["cos"])
        return s
    batch, heads, seq = case["batch"], case["heads"], case["seq"]
    rows, width = batch * seq, heads * HEAD
    s["qkv"] = normal(rows, 3 * width)
    if case["op"] == "qk_bwd":
        s["gq"], s["gk"] = normal(HEAD, std=0.02, mean=1.0), normal(HEAD, std=0.02, mean=1.0)
        s["cos"], s["sin"] = _tables(rows if case["tables"] == "own" else seq, gen)
        s["dq"], s["dk"] = normal(batch, heads, seq, HEAD, std=0.5), normal(batch, heads, seq, HEAD, std=0.5)
        s["dqkv"] = torch.zeros_like(s["qkv"])
        s["dgq"] = torch.empty(HEAD, device="cuda")
        s["dgk"] = torch.empty(HEAD, device="cuda")
        return s
    s["q"], s["k"] = normal(batch, heads, seq, HEAD), normal(batch, heads, seq, HEAD)
    s["mask"] = _mask(case)
    s["o"] = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(batch, heads, seq, device="cuda")
    if case["op"] == "attn_bwd":
        o, lse = _attention(s)
        s["o"], s["lse"] = o, lse
        s["do"] = normal(rows, width)
        s["dq"], s["dk"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["dqkv"] = torch.zeros_like(s["qkv"])
    return s


# ------------------------------------------------------------------------------------- plain forms
def _rope_axes(s):
    cols = []
    for axis, n in enumerate(s["pairs"]):
        freq = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n)
        cols.append(s["pos"][:, axis:axis + 1].double() * freq)
    angle = torch.cat(cols, 1)
    return angle.cos().float(), angle.sin().float()


def _heads_of(t, case):
    """[batch * seq, heads * 128] -> fp32 [batch, heads, seq, 128]"""
    return t.view(case["batch"], case["seq"], case["heads"], HEAD).permute(0, 2, 1, 3).float()


def _rows_of(t):
    """[batch, heads, seq, 128] -> bf16 [batch * seq, heads * 128]"""
    b, h, n, d = t.shape
    return t.permute(0, 2, 1, 3).reshape(b * n, h * d).bfloat16()


def _scores(s):
    z = torch.matmul(s["q"].float(), s["k"].float().transpose(2, 3)).mul_(SCALE)
    if s["mask"] is not None:
        z.masked_fill_((s["mask"] == 0)[:, None, None, :], -math.inf)
    return z


def _values(s):
    width = s["case"]["heads"] * HEAD
    return _heads_of(s["qkv"][:, 2 * width:], s["case"])


def _attention(s):
    z = _scores(s)
    top = z.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = z.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, _values(s)) / torch.where(total > 0, total, torch.ones_like(total))
    return _rows_of(o), (top + total.log()).squeeze(3)


def _attention_backward(s):
    case = s["case"]
    v, do = _values(s), _heads_of(s["do"], case)
    lse = s["lse"].unsqueeze(3)
    p = _scores(s).sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)).exp_()
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3))
    ds.sub_((ds * p).sum(3, keepdim=True)).mul_(p).mul_(SCALE)
    del p
    dq = torch.matmul(ds, s["k"].float())
    dk = torch.matmul(ds.transpose(2, 3), s["q"].float())
    return dq.bfloat16(), dk.bfloat16(), _rows_of(dv)


def _qk_backward_one(x, gain, cos, sin, dy, case):
    """x: raw [batch * seq, heads * 128] columns; dy [batch, heads, seq, 128]."""
    x = _heads_of(x, case)
    dy = dy.float()
    a, b = dy[..., 0::2], dy[..., 1::2]
    dn = torch.stack([a * cos + b * sin, b * cos - a * sin], 4).flatten(3)  # rotated back
    r = (x.square().mean(3, keepdim=True) + EPS).rsqrt()
    n = x * r
    dgain = (dn * n).double().sum((0, 1, 2)).float()  # a long sum
    dn = dn * gain.float()
    dx = (dn - n * (dn * n).mean(3, keepdim=True)) * r
    return _rows_of(dx), dgain


def _qk_backward(s):
    case = s["case"]
    width = case["heads"] * HEAD
    shape = (case["batch"] if case["tables"] == "own" else 1, 1, case["seq"], PAIRS)
    cos, sin = s["cos"].view(shape), s["sin"].view(shape)
    dq, dgq = _qk_backward_one(s["qkv"][:, :width], s["gq"], cos, sin, s["dq"], case)
    dk, dgk = _qk_backward_one(s["qkv"][:, width:2 * width], s["gk"], cos, sin, s["dk"], case)
    return torch.cat([dq, dk], 1), dgq, dgk


# ----------------------------------------------------------------------------------- the operators
def _own(s):
    import diffusion_transformer_denoiser_gb300 as mi

    case = s["case"]
    op = case["op"]
    if op == "rope_axes":
        mi.rope_axes_tables(s["pos"], s["pairs"], s["cos"], s["sin"])
        return s["cos"], s["sin"]
    batch, heads, seq = case["batch"], case["heads"], case["seq"]
    if "ws" not in s:  # a program plans its workspaces once
        size = {"attn_fwd": mi.attention_workspace_size, "attn_bwd": mi.attention_backward_workspace_size,
                "qk_bwd": mi.qk_norm_rope_backward_workspace_size}[op](batch, seq, heads)
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    width = heads * HEAD
    if op == "attn_fwd":
        mi.attention_lse(s["q"], s["k"], s["qkv"], s["mask"], s["o"], s["lse"], batch, seq, heads, ws=s["ws"])
        return s["o"], s["lse"]
    if op == "attn_bwd":
        mi.attention_backward(s["q"], s["k"], s["qkv"], s["mask"], s["o"], s["lse"], s["do"], s["dq"], s["dk"], s["dqkv"],
                              batch, seq, heads, s["ws"])
        return s["dq"], s["dk"], s["dqkv"][:, 2 * width:]
    mi.qk_norm_rope_backward(s["qkv"], s["gq"], s["gk"], s["cos"], s["sin"], s["dq"], s["dk"], s["dqkv"], s["dgq"], s["dgk"],
                             batch, seq, heads, s["ws"], eps=EPS,
                             rope_bstride=seq * PAIRS if case["tables"] == "own" else 0)
    return s["dqkv"][:, :2 * width], s["dgq"], s["dgk"]


def run(state):
    if own:
        return _own(state)
    return {"rope_axes": _rope_axes, "attn_fwd": _attention, "attn_bwd": _attention_backward,
            "qk_bwd": _qk_backward}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------------------- 64 bits
def _exact_attention(s, backward):
    """One head of one element at a time: softmax from its definition, and its Jacobian."""
    case = s["case"]
    batch, heads, seq = case["batch"], case["heads"], case["seq"]
    width = heads * HEAD
    f = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(batch * seq, width, **f), torch.full((batch, heads, seq), -math.inf, **f)
    dq, dk, dv = torch.zeros(batch, heads, seq, HEAD, **f), torch.zeros(batch, heads, seq, HEAD, **f), torch.zeros_like(o)
    for b in range(batch):
        keys = torch.arange(seq, device="cuda") if s["mask"] is None else s["mask"][b].nonzero().flatten()
        if not len(keys):
            continue
        at = slice(b * seq, (b + 1) * seq)
        for h in range(heads):
            cols = slice(h * HEAD, (h + 1) * HEAD)
            q, k = s["q"][b, h].double(), s["k"][b, h][keys].double()
            v = s["qkv"][at, 2 * width + h * HEAD:2 * width + (h + 1) * HEAD][keys].double()
            z = q @ k.T / HEAD ** 0.5
            lse[b, h] = torch.logsumexp(z, 1)
            p = torch.softmax(z, 1)
            if not backward:
                o[at, cols] = p @ v
                continue
            g = s["do"][at, cols].double()
            dp = g @ v.T
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) / HEAD ** 0.5
            dq[b, h] = ds @ k
            dk[b, h, keys] = ds.T @ q
            t = torch.zeros(seq, HEAD, **f)
            t[keys] = p.T @ g
            dv[at, cols] = t
    return (dq, dk, dv) if backward else (o, lse)


def _exact_qk(s):
    """The chain rule on y = rotate(x / sqrt(mean x^2 + eps) * gain), by rows; pairs as complex numbers."""
    case = s["case"]
    batch, heads, seq = case["batch"], case["heads"], case["seq"]
    width = heads * HEAD
    turn = torch.complex(s["cos"].double(), s["sin"].double()).view(-1, seq, 1, PAIRS)
    grads, gains = [], []
    for x, gain, dy in ((s["qkv"][:, :width], s["gq"], s["dq"]), (s["qkv"][:, width:2 * width], s["gk"], s["dk"])):
        x = x.reshape(batch, seq, heads, HEAD).double()
        pairs = torch.view_as_complex(dy.permute(0, 2, 1, 3).double().reshape(batch, seq, heads, PAIRS, 2).contiguous())
        dz = torch.view_as_real(pairs * turn.conj()).reshape(batch, seq, heads, HEAD)
        size = torch.sqrt((x * x).sum(3, keepdim=True) / HEAD + EPS)
        gains.append((dz * x / size).sum((0, 1, 2)))
        dz = dz * gain.double()
        dx = dz / size - x * (dz * x).sum(3, keepdim=True) / (HEAD * size ** 3)
        grads.append(dx.reshape(batch * seq, width))
    return torch.cat(grads, 1), gains[0], gains[1]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope_axes":
        n = [int(p) for p in case["pairs"].split(",")]
        axis = torch.tensor([a for a, c in enumerate(n) for _ in range(c)], device="cuda")
        power = torch.tensor([j / c for c in n for j in range(c)], dtype=torch.float64, device="cuda")
        angle = s["pos"].double()[:, axis] / torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"), power)
        return torch.cos(angle), torch.sin(angle)
    if case["op"] == "qk_bwd":
        return _exact_qk(s)
    return _exact_attention(s, case["op"] == "attn_bwd")
