"""What is measured of the layer norm, dropout and 8-bit linear operators.

layer_norm    s = r + drop(x), y = (s - mean(s)) / sqrt(var(s) + eps) * w + b, and its gradients
dropout       y = r + drop(x), drop(x) = x / (1 - p) where a counter-based generator keeps it, else 0
              (the mask is made again in the backward pass, never stored)
linear_int8   rows of x to 8 bits (one scale a row), their product with weights in 8 bits
              (one scale a channel), bias, residual, activation

Tokens (or images) are rows.  An element's random number is 16 bits of Philox4x32-10 with
counter (column / 8, row, offset) and key seed; it is kept where they are at least p 2^16.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("identity", "relu", "silu", "gelu", "gelu_tanh")
EPS = 1e-5
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------------ cases

def _norm(name, dtype, m, n, res=False, drop=0.0, keep=False, pad=0, back=False):
    return {"name": name, "op": "layer_norm_backward" if back else "layer_norm", "dtype": dtype,
            "m": m, "n": n, "res": res, "drop": drop, "keep": keep, "pad": pad}


def _drop(name, dtype, m, n, drop=0.1, res=False, pad=0, back=False):
    return {"name": name, "op": "dropout_backward" if back else "dropout", "dtype": dtype, "m": m,
            "n": n, "drop": drop, "res": res, "pad": pad}


def _int8(name, dtype, m, n, k, act="identity", bias=False, res="none", pad=0):
    return {"name": name, "op": "linear_int8", "dtype": dtype, "m": m, "n": n, "k": k, "act": act,
            "bias": bias, "res": res, "pad": pad}


def listed():
    return [
        # the norm before a block, one new token: latency
        _norm("norm_token_f16", "f16", 1, 2048),
        # a norm over whole feature maps (256 channels of 14 x 14), a batch of 32
        _norm("norm_images_f32", "f32", 32, 50176),
        # training: a block's output dropped and added to the stream, and the next norm
        _norm("norm_block_bf16", "bf16", 8192, 4096, res=True, drop=0.1, keep=True),
        # its gradients, with the gradient that comes down the stream
        _norm("norm_grads_bf16", "bf16", 8192, 4096, res=True, drop=0.1, back=True),
        # gradients at an odd width, rows of a wider buffer
        _norm("norm_odd_grads_f16", "f16", 777, 1001, res=True, pad=5, back=True),
        # the hidden activations of a block in training
        _drop("dropout_long_bf16", "bf16", 8192, 11008),
        # scores of a small head in single precision, added to a residual, odd rows
        _drop("dropout_odd_f32", "f32", 1000, 1001, drop=0.5, res=True),
        # the gradient of a block's hidden activations
        _drop("dropout_grads_f16", "f16", 4096, 5632, drop=0.2, back=True),
        # one new token through an expanding projection: the weights' stream
        _int8("int8_token_f16", "f16", 1, 5632, 2048, act="silu"),
        # the down projection, 16 sequences of one new token each
        _int8("int8_tokens_bf16", "bf16", 16, 2048, 5632, res="after"),
        # a long batch (a prompt) through an expanding projection
        _int8("int8_long_bf16", "bf16", 8192, 11008, 4096, act="gelu_tanh", bias=True),
        # odd sizes, a residual before the activation
        _int8("int8_odd_f16", "f16", 777, 1001, 1531, act="relu", bias=True, res="before"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm", "layer_norm_backward", "layer_norm_backward",
                     "dropout", "dropout_backward", "linear_int8", "linear_int8", "linear_int8"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    size = 4 if dtype == "f32" else 2
    pad = rng.choice([0, 0, 0, 8, 5])
    if op == "linear_int8":
        m = _log(rng, 1, 16384)
        k, n = _log(rng, 64, 8192), _log(rng, 64, 11008)
        if rng.random() < 0.6:  # most sizes are the usual multiples
            k, n = (k + 63) // 64 * 64, (n + 63) // 64 * 64
        m = max(1, min(m, int(3.6e11 / (n * k))))
        return {"op": op, "dtype": dtype, "m": m, "n": n, "k": k, "act": rng.choice(ACTS),
                "bias": rng.random() < 0.5, "res": rng.choice(["none", "before", "after"]),
                "pad": pad}
    n = _log(rng, 8, 131072) if op.startswith("layer") else _log(rng, 1, 16384)
    if rng.random() < 0.5:
        n = (n + 63) // 64 * 64
    most = 6.7e7 if op.startswith("layer") else 1.8e8  # bytes of a matrix
    m = max(1, min(_log(rng, 1, 65536), int(most / (n * size))))
    drop = rng.choice([0.0, 0.1, 0.5]) if op.startswith("layer") else rng.choice([0.1, 0.5, 0.9])
    case = {"op": op, "dtype": dtype, "m": m, "n": n, "drop": drop, "res": rng.random() < 0.5,
            "pad": pad}
    if op.startswith("layer"):
        case["keep"] = rng.random() < 0.5
    return case


# ----------------------------------------------------------------------- inputs

def prepare(case, seed):
    t = TYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    m, n, pad = case["m"], case["n"], case["pad"]

    def normal(scale, *shape, pad=0, shift=0.0):
        full = (*shape[:-1], shape[-1] + pad)
        v = (torch.randn(full, generator=gen, device="cuda") * scale + shift).to(t)
        return v[..., :shape[-1]] if pad else v

    s = {"case": case, "t": t, "seed": (seed * 0x9E3779B97F4A7C15 + 0x1234) % (1 << 64)}
    if case["op"] == "linear_int8":
        k = case["k"]
        s["x"] = normal(1.0, m, k, pad=pad)
        # weights laid out once in 8 bits: the nearest of 127 steps to either side
        w = torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5
        s["ws"] = w.abs().amax(1) / 127
        s["w"] = torch.round(w / s["ws"][:, None]).to(torch.int8)
        s["b"] = normal(0.5, n) if case["bias"] else None
        s["r"] = normal(1.0, m, n, pad=pad) if case["res"] != "none" else None
    else:
        # the number of the training step, on the device: a captured step moves it on
        s["step"] = torch.randint(0, 1 << 40, (1,), generator=gen, device="cuda")
        s["offset"] = seed % 1000 << 33
        if case["op"].startswith("layer"):
            # a stream with a few channels that stand out
            col = torch.randn(n, generator=gen, device="cuda")
            scale = torch.where(col.abs() > 2.5, 8.0, 1.0)
            wide = torch.cat([scale, scale.new_ones(pad)])
            stream = normal(1.0, m, n + pad, shift=0.3) * wide.to(t)
            stream = stream[:, :n]
            s["w"], s["b"] = normal(0.2, n, shift=1.0), normal(0.2, n)
        if case["op"] == "layer_norm":
            s["x"] = normal(1.0, m, n, pad=pad) if case["res"] else stream
            s["r"] = stream if case["res"] else None
        elif case["op"] == "layer_norm_backward":
            # what the forward pass kept, and the gradients that arrive
            s["s"] = stream
            f = stream.float()
            s["mean"] = f.mean(1)
            s["rstd"] = 1 / torch.sqrt(((f - s["mean"][:, None]) ** 2).mean(1) + EPS)
            s["dy"] = normal(1.0, m, n, pad=pad)
            s["ds"] = normal(1.0, m, n, pad=pad) if case["res"] else None
        elif case["op"] == "dropout":
            s["x"] = normal(1.0, m, n, pad=pad)
            s["r"] = normal(1.0, m, n, pad=pad) if case["res"] else None
        else:
            s["dy"] = normal(1.0, m, n, pad=pad)
    if own:
        _plan(s)
    return s


def _plan(s):
    """The problem, the outputs and the scratch that a program keeps beside its weights."""
    import convolution_forward_amd as cf
    c, t, d = s["case"], s["t"], s["case"]["dtype"]
    m, n = c["m"], c["n"]
    empty = lambda *shape, t=t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
    ld = lambda v: 0 if v is None else v.stride(0)  # noqa: E731
    s["cf"] = cf
    size = 0
    if c["op"] == "linear_int8":
        k = c["k"]
        s["q"], s["xs"], s["y"] = empty(m, k, t=torch.int8), empty(m, t=torch.float32), empty(m, n)
        s["quant"] = cf.make_quantize_problem(m, k, ldx=ld(s["x"]))
        s["p"] = cf.make_linear_int8_problem(m, n, k, act=c["act"], bias=c["bias"],
                                             residual=c["res"], ldr=ld(s["r"]))
        size = cf.linear_int8_scratch_size(s["p"], d)
    elif c["op"].startswith("dropout"):
        back = c["op"] == "dropout_backward"
        s["p"] = cf.make_dropout_problem(
            m, n, c["drop"], seed=s["seed"], offset=s["offset"], residual=not back and c["res"],
            ldx=0 if back else ld(s["x"]), ldr=0 if back else ld(s["r"]),
            ldy=ld(s["dy"]) if back else 0)
        s["dx" if back else "y"] = empty(m, n)
    else:
        back = c["op"] == "layer_norm_backward"
        s["p"] = cf.make_layer_norm_problem(
            m, n, eps=EPS, residual=c["res"], drop=c["drop"], seed=s["seed"], offset=s["offset"],
            ldx=0 if back else ld(s["x"]), ldr=0 if back else ld(s["r"]),
            lds=ld(s["s"]) if back else 0, ldy=ld(s["dy"]) if back else 0,
            ldds=ld(s["ds"]) if back else 0)
        if back:
            s["dx"], s["dw"], s["db"] = empty(m, n), empty(n), empty(n)
            s["dr"] = empty(m, n) if c["res"] else None
            size = cf.layer_norm_backward_scratch_size(s["p"], d)
        else:
            s["y"] = empty(m, n)
            s["s"] = empty(m, n) if c["keep"] else None
            s["mean"], s["rstd"] = (empty(m, t=torch.float32) if c["keep"] else None
                                    for _ in range(2))
            size = cf.layer_norm_scratch_size(s["p"], d)
    s["bytes"] = size
    s["scratch"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None


# ---------------------------------------------------------------- the plain form

def _keeps(m, n, drop, seed, offset):
    """Which elements stay; offset: a tensor (the call's offset with the step added)."""
    at = torch.arange((n + 7) // 8, device="cuda")[None, :].expand(m, -1)
    c = [at, torch.arange(m, device="cuda")[:, None], offset & M32, (offset >> 32) & M32]
    k = [seed & M32, seed >> 32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & M32) ^ c[1] ^ k[0], b & M32, ((a >> 32) & M32) ^ c[3] ^ k[1], a & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    words = torch.stack([q.expand(at.shape) for q in c], dim=2)
    bits = torch.stack([words & 0xFFFF, words >> 16], dim=3).reshape(m, -1)[:, :n]
    return bits >= round(drop * 65536)


def _dropped(v, s):
    """v in 32 bits, scaled where kept, 0 elsewhere."""
    c = s["case"]
    if c["drop"] == 0:
        return v
    keep = _keeps(c["m"], c["n"], c["drop"], s["seed"], s["step"] + s["offset"])
    return torch.where(keep, v * (65536 / (65536 - round(c["drop"] * 65536))), torch.zeros_like(v))


def _act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _run_plain(s):
    c, t = s["case"], s["t"]
    if c["op"] == "linear_int8":
        x = s["x"].float()
        top = x.abs().amax(1)
        most = torch.full_like(top, 127.0)  # a tensor: divisions by a number are products
        xs = top / most
        q = torch.round(x * (most / top)[:, None])
        y = (q @ s["w"].float().t()) * (xs[:, None] * s["ws"])
        if c["bias"]:
            y = y + s["b"].float()
        if c["res"] == "before":
            y = y + s["r"].float()
        y = _act(y, c["act"])
        if c["res"] == "after":
            y = y + s["r"].float()
        return {"y": y.to(t), "xs": xs}
    if c["op"] == "dropout":
        y = _dropped(s["x"].float(), s)
        return {"y": (y + s["r"].float() if c["res"] else y).to(t)}
    if c["op"] == "dropout_backward":
        return {"dx": _dropped(s["dy"].float(), s).to(t)}
    w = s["w"].float()
    if c["op"] == "layer_norm":
        v = _dropped(s["x"].float(), s)
        if c["res"]:
            v = v + s["r"].float()
        mean = v.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt(((v - mean) ** 2).mean(1, keepdim=True) + EPS)
        out = {"y": ((v - mean) * rstd * w + s["b"].float()).to(t)}
        if c["keep"]:
            out |= {"s": v.to(t), "mean": mean[:, 0], "rstd": rstd[:, 0]}
        return out
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (s["s"].float() - s["mean"][:, None]) * rstd
    g = dy * w
    d = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if c["res"]:
        d = d + s["ds"].float()
    out = {"dx": _dropped(d, s).to(t), "dw": (dy * xhat).sum(0).to(t), "db": dy.sum(0).to(t)}
    return out | ({"dr": d.to(t)} if c["res"] else {})


# ------------------------------------------------------------- the framework's calls

def _run_own(s):
    c, cf, p, d = s["case"], s["cf"], s["p"], s["case"]["dtype"]
    stream = torch.cuda.current_stream().cuda_stream
    if c["op"] == "linear_int8":
        cf.quantize_rows(s["quant"], d, s["x"], s["q"], s["xs"], stream)
        cf.linear_int8_forward(p, d, s["q"], s["xs"], s["w"], s["ws"], s["b"], s["r"], s["y"],
                               s["scratch"], s["bytes"], stream)
        return {"y": s["y"], "xs": s["xs"]}
    if c["op"] == "dropout":
        cf.dropout_forward(p, d, s["x"], s["r"], s["y"], s["step"], stream)
        return {"y": s["y"]}
    if c["op"] == "dropout_backward":
        cf.dropout_backward(p, d, s["dy"], s["dx"], s["step"], stream)
        return {"dx": s["dx"]}
    if c["op"] == "layer_norm":
        cf.layer_norm_forward(p, d, s["x"], s["r"], s["w"], s["b"], s["y"], s["s"], s["mean"],
                              s["rstd"], s["step"], s["scratch"], s["bytes"], stream)
        out = {"y": s["y"]}
        if c["keep"]:
            out |= {"s": s["s"], "mean": s["mean"], "rstd": s["rstd"]}
        return out
    cf.layer_norm_backward(p, d, s["s"], s["w"], s["mean"], s["rstd"], s["dy"], s["ds"], s["dx"],
                           s["dr"], s["dw"], s["db"], s["step"], s["scratch"], s["bytes"], stream)
    out = {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    return out | ({"dr": s["dr"]} if c["res"] else {})


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------- work

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    m, n, op = case["m"], case["n"], case["op"]
    if op == "linear_int8":
        k, r = case["k"], int(case["res"] != "none")
        return {"bytes": size * (m * k + (1 + r) * m * n + case["bias"] * n) + n * k + 4 * (m + n),
                "flops": 2 * m * n * k}
    r, d = int(case["res"]), int(case["drop"] > 0)
    if op == "dropout":
        return {"bytes": size * (2 + r) * m * n, "flops": (1 + r) * m * n}
    if op == "dropout_backward":
        return {"bytes": size * 2 * m * n, "flops": m * n}
    if op == "layer_norm":
        kept = (size * m * n + 8 * m) * case["keep"]
        return {"bytes": size * ((2 + r) * m * n + 2 * n) + kept, "flops": (7 + r + d) * m * n}
    return {"bytes": size * ((3 + 2 * r) * m * n + 3 * n) + 8 * m, "flops": (15 + r + d) * m * n}


# ------------------------------------------------------------ in 64 bits, written apart

def _philox(m, n, drop, seed, offset):
    """1 / (1 - p) where an element stays and 0 elsewhere, on the host, word by word."""
    low, shift = np.uint64(M32), np.uint64(32)
    groups = -(-n // 8)
    x = [np.broadcast_to(np.arange(groups, dtype=np.uint64), (m, groups)),
         np.broadcast_to(np.arange(m, dtype=np.uint64)[:, None], (m, groups)),
         np.uint64(offset & M32), np.uint64(offset >> 32)]
    for i in range(10):
        key = [np.uint64((seed + i * 0x9E3779B9) & M32), np.uint64(((seed >> 32) + i * 0xBB67AE85) & M32)]
        one, two = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(two >> shift) ^ x[1] ^ key[0], two & low, (one >> shift) ^ x[3] ^ key[1], one & low]
    out = np.empty((m, groups, 8), dtype=np.uint16)
    for i, word in enumerate(x):
        out[:, :, 2 * i], out[:, :, 2 * i + 1] = word & np.uint64(0xFFFF), word >> np.uint64(16)
    below = round(65536 * drop)
    keep = torch.from_numpy(out.reshape(m, -1)[:, :n] >= below).cuda()
    return keep.double() * (1 / (1 - below / 65536))


def exact(case, seed):
    saved = own
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = saved
    f = torch.nn.functional
    d = {key: v.double() for key, v in s.items() if torch.is_tensor(v)}
    if case["op"] == "linear_int8":
        # the steps of x are the definition's, taken in float32
        top = torch.max(torch.abs(s["x"].float()), dim=1).values
        q = torch.mul(s["x"].float(), torch.div(127.0, top).unsqueeze(1)).round().double()
        xs = top.double() / 127
        z = torch.mm(q, d["w"].transpose(0, 1)).mul(xs.unsqueeze(1)).mul(d["ws"].unsqueeze(0))
        z = z + d.get("b", 0.0) + (d["r"] if case["res"] == "before" else 0.0)
        act = {"relu": f.relu, "silu": f.silu, "gelu": f.gelu, "identity": lambda v: v,
               "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[case["act"]]
        return {"y": act(z) + (d["r"] if case["res"] == "after" else 0.0), "xs": xs}
    scale = 1.0
    if case["drop"]:
        offset = (int(s["step"]) + s["offset"]) % (1 << 64)
        scale = _philox(case["m"], case["n"], case["drop"], s["seed"], offset)
    if case["op"] == "dropout":
        return {"y": d["x"] * scale + d.get("r", 0.0)}
    if case["op"] == "dropout_backward":
        return {"dx": d["dy"] * scale}
    n = case["n"]
    if case["op"] == "layer_norm":
        v = d["x"] * scale + d.get("r", 0.0)
        var, mean = torch.var_mean(v, dim=1, correction=0)
        root = torch.sqrt(var + EPS)
        out = {"y": (v - mean.unsqueeze(1)) / root.unsqueeze(1) * d["w"] + d["b"]}
        return out | ({"s": v, "mean": mean, "rstd": 1 / root} if case["keep"] else {})
    # d/ds of sum(dy y) with the statistics as they were kept: Jacobian of the norm, row by row
    u = (d["s"] - d["mean"].unsqueeze(1)) * d["rstd"].unsqueeze(1)
    e = d["dy"] * d["w"]
    along, level = torch.sum(e * u, dim=1, keepdim=True), torch.sum(e, dim=1, keepdim=True)
    ds = (n * e - level - u * along) * (d["rstd"].unsqueeze(1) / n) + d.get("ds", 0.0)
    out = {"dx": ds * scale, "dw": torch.sum(d["dy"] * u, dim=0), "db": torch.sum(d["dy"], dim=0)}
    return out | ({"dr": ds} if case["res"] else {})
