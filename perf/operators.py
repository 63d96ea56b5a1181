"""The 8-bit activation checkpoints and the backward operators that read them,
as they are timed: cases, inputs, one pass of each, and exact results.

A pass is one of
  pack   an activation matrix packed into an 8-bit checkpoint and restored;
  norm   RMS norm of x + residual with its packed output: forward alone (with
         the packed output restored), or forward and backward;
  wgrad  weight (and bias) gradient of a linear layer from a packed input;
  block  norm forward, the weight gradient of the layer behind it from the
         norm's packed output, and the norm's backward.

Format of a checkpoint: codes int8 [rows][pitch], pitch = cols rounded up to
32, and scales uint8 [rows][pitch / 32].  A block of 32 columns of a row holds
q * 2^(s - 127): s the lowest scale at which the block's largest magnitude is
at most 127 quanta (0 for a block of zeros, 255 for a block with an infinity
or a NaN).
"""

import math

import numpy as np
import torch

own = False

BLOCK = 32
EPS = float(np.float32(1e-5))
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------- cases


def _pack(name, rows, cols, dtype, pad=0):
    return {"name": name, "op": "pack", "rows": rows, "cols": cols, "dtype": dtype, "pad": pad}


def _norm(name, rows, cols, dtype, backward, residual=True, pad=0):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "backward": backward,
            "residual": residual, "pad": pad}


def _wgrad(name, rows, n_in, n_out, dtype, gain=False, bias=False, pad=0):
    return {"name": name, "op": "wgrad", "rows": rows, "cols": n_in, "out": n_out, "dtype": dtype, "gain": gain,
            "bias": bias, "pad": pad}


def _block(name, rows, cols, n_out, dtype):
    return {"name": name, "op": "block", "rows": rows, "cols": cols, "out": n_out, "dtype": dtype, "pad": 0}


def listed():
    return [
        # one token of the 2048-wide layout: latency of the two launches
        _pack("pack_token", 1, 2048, "bf16"),
        # the GPT layout's MLP activation, 8 sequences of 1024, rows inside a wider buffer
        _pack("pack_mlp_fp16", 8192, 4096, "fp16", pad=64),
        # the largest activation of a layer: the 1.8B layout's FFN, 8 sequences of 2048
        _pack("pack_ffn", 16384, 5632, "bf16"),
        # evaluation of one token: forward alone
        _norm("norm_token", 1, 2048, "bf16", backward=False),
        # one sequence of 4096 tokens at the 500M layout's width, fp16
        _norm("norm_step_fp16", 4096, 1280, "fp16", backward=True),
        # a ragged batch at an odd width, fp32, no residual
        _norm("norm_odd_fp32", 1531, 777, "fp32", backward=True, residual=False, pad=3),
        # a training step's norm at the 1.8B layout's width, 8 sequences of 2048
        _norm("norm_step", 16384, 2048, "bf16", backward=True),
        # a short micro-batch through a square projection (wq of the 500M layout)
        _wgrad("wgrad_short", 256, 1280, 1280, "bf16"),
        # the GPT layout's first MLP product, with its bias, fp16 gradients
        _wgrad("wgrad_mlp_fp16", 8192, 1024, 4096, "fp16", bias=True),
        # odd everything, fp32 gradients
        _wgrad("wgrad_odd_fp32", 999, 777, 1531, "fp32", gain=True, bias=True, pad=1),
        # the 1.8B layout's gate product from the norm's packed output, 8 sequences of 2048
        _wgrad("wgrad_ffn", 16384, 2048, 5632, "bf16", gain=True),
        # norm, wq's weight gradient and the norm's backward: 2 sequences of 4096 at the 500M layout
        _block("block_attention", 8192, 1280, 1280, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pack", "norm", "wgrad", "block"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    pad = rng.choice([0, 0, 1, 8, 40])
    # wider types take more bytes and more products an element
    rows = _log_int(rng, 1, {"bf16": 16384, "fp16": 8192, "fp32": 4096}[dtype])
    if op == "pack":
        return {"op": op, "rows": rows, "cols": _log_int(rng, 32, 5632), "dtype": dtype, "pad": pad}
    cols = _log_int(rng, 64, 2048)
    if op == "norm":
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "backward": rng.random() < 0.7,
                "residual": rng.random() < 0.7, "pad": pad}
    out = _log_int(rng, 64, 5632)
    if op == "wgrad":
        return {"op": op, "rows": rows, "cols": cols, "out": out, "dtype": dtype, "gain": rng.random() < 0.5,
                "bias": rng.random() < 0.5, "pad": pad}
    return {"op": op, "rows": min(rows, 8192), "cols": min(cols, 1280), "out": min(out, 1280), "dtype": dtype,
            "pad": 0}


# ------------------------------------------------------------------ inputs


def _gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + stream) & 0x7FFFFFFFFFFFFFFF)
    return g


def _matrix(rows, cols, pad, dtype):
    """An empty [rows][cols] matrix whose rows lie cols + pad elements apart."""
    return torch.empty((rows, cols + pad), dtype=dtype, device=DEV)[:, :cols]


def _activation(case, seed, stream, dtype):
    """Activations: channels of unequal spread, a few outlier channels of
    about 20 times the rest, and some padded tokens that are all zero."""
    rows, cols = case["rows"], case["cols"]
    g = _gen(seed, stream)
    chan = torch.exp(0.5 * torch.randn(cols, generator=g, device=DEV))
    chan = chan * torch.where(torch.rand(cols, generator=g, device=DEV) < 0.005, 20.0, 1.0)
    x = torch.randn((rows, cols), generator=g, device=DEV) * chan
    if rows > 8:
        x *= (torch.rand((rows, 1), generator=g, device=DEV) >= 0.02).float()
    out = _matrix(rows, cols, case["pad"], dtype)
    out.copy_(x)
    return out


def _gradient(case, cols, seed, stream, dtype):
    """Gradients of a layer's output: tokens of unequal weight, tokens whose
    loss is masked (zero rows).  fp16 gradients carry a loss scale."""
    rows = case["rows"]
    g = _gen(seed, stream)
    tok = 1e-3 * torch.exp(torch.randn((rows, 1), generator=g, device=DEV))
    if dtype == torch.float16:
        tok = tok * 128.0
    if rows > 8:
        tok = tok * (torch.rand((rows, 1), generator=g, device=DEV) >= 0.05).float()
    out = _matrix(rows, cols, case["pad"], dtype)
    out.copy_(torch.randn((rows, cols), generator=g, device=DEV) * tok)
    return out


def _weight(cols, seed, stream):
    """A norm's weight: near one, a few channels far from it."""
    g = _gen(seed, stream)
    return 1.0 + 0.3 * torch.randn(cols, generator=g, device=DEV)


def _inputs(case, seed):
    dt = DTYPES[case["dtype"]]
    op, rows, cols = case["op"], case["rows"], case["cols"]
    s = {"case": case, "dtype": dt}
    if op == "pack":
        s["x"] = _activation(case, seed, 1, dt)
    elif op == "wgrad":
        # the packed input as the forward pass left it
        codes, scales = _quantise(_activation(case, seed, 1, dt).float())
        s["codes"], s["scales"] = codes.to(torch.int8), scales.to(torch.uint8)
        s["dy"] = _gradient(case, case["out"], seed, 2, dt)
        s["gain"] = _weight(cols, seed, 3) if case["gain"] else None
    else:
        s["x"] = _activation(case, seed, 1, dt)
        s["residual"] = _activation(case, seed, 2, dt) if case.get("residual", True) else None
        s["weight"] = _weight(cols, seed, 3)
        if op == "block" or case["backward"]:
            s["dy"] = _gradient(case, cols, seed, 4, dt)
            s["dres"] = _gradient(case, cols, seed, 5, dt) if s["residual"] is not None else None
        if op == "block":
            s["dout"] = _gradient(case, case["out"], seed, 6, dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    # the buffers a training program keeps: outputs, checkpoint, workspaces,
    # and the gradient rows' parts that the weight gradients go to
    from sparse_communication_distributed_amd import scape as S
    op, rows, cols, dt = case["op"], case["rows"], case["cols"], s["dtype"]
    if op == "pack":
        s["act"] = S.act_alloc(rows, cols, DEV)
        s["restored"] = torch.empty((rows, cols), dtype=dt, device=DEV)
        return s
    if op == "wgrad":
        s["act"] = S.ActCheckpoint(s["codes"], s["scales"], cols)
    else:
        s["act"] = S.act_alloc(rows, cols, DEV)
        s["rstd"] = torch.empty(rows, device=DEV)
        s["h"] = torch.empty((rows, cols), dtype=dt, device=DEV) if s["residual"] is not None else None
        s["y"] = torch.empty((rows, cols), dtype=dt, device=DEV)
        if "dy" in s:
            s["dh"] = torch.empty((rows, cols), dtype=dt, device=DEV)
            s["dweight"] = torch.empty(cols, device=DEV)
            s["norm_ws"] = torch.empty(S.rmsnorm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEV)
        else:
            s["restored"] = torch.empty((rows, cols), dtype=dt, device=DEV)
    if op in ("wgrad", "block"):
        s["dw"] = torch.empty((case["out"], cols), device=DEV)
        s["db"] = torch.empty(case["out"], device=DEV) if case.get("bias") else None
        s["wgrad_ws"] = torch.empty(S.wgrad_workspace_bytes(rows, cols, case["out"]), dtype=torch.uint8, device=DEV)
    return s


# -------------------------------------------------------------- plain form


def _blocks(x):
    """[rows][cols] as zero-filled blocks [rows][blocks][32]."""
    rows, cols = x.shape
    nb = (cols + BLOCK - 1) // BLOCK
    if nb * BLOCK != cols:
        x = torch.cat([x, torch.zeros((rows, nb * BLOCK - cols), dtype=x.dtype, device=x.device)], dim=1)
    return x.reshape(rows, nb, BLOCK)


def _quantise(x):
    """Codes [rows][pitch] and scale bytes [rows][blocks] (as int32) of an
    fp32 matrix."""
    b = _blocks(x)
    amax = b.abs().amax(dim=2)
    bits = amax.view(torch.int32)
    s = (bits >> 23) - 6 + ((bits & 0x7FFFFF) > 0x7E0000).to(torch.int32)
    s = torch.where(amax == 0, torch.zeros_like(s), s.clamp(min=1))
    bad = ~torch.isfinite(amax)
    inv = ((254 - s) << 23).view(torch.float32)  # 2^(127 - s)
    q = torch.round(b * inv[:, :, None])
    q = torch.where((bad | (s == 0))[:, :, None], torch.zeros_like(q), q)
    s = torch.where(bad, torch.full_like(s, 255), s)
    return q.reshape(x.shape[0], -1), s


def _restore(codes, scales, cols):
    """fp32 values [rows][cols] of codes and scale bytes."""
    rows = codes.shape[0]
    scale = (scales.to(torch.int32) << 23).view(torch.float32)
    v = codes.float().reshape(rows, -1, BLOCK) * scale[:, :, None]
    return v.reshape(rows, -1)[:, :cols]


def _plain_forward(s):
    dt = s["dtype"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    # 64 bits: the packed values lie next to rounding borders, where the
    # order of a 32-bit sum would decide
    hd = h.double()
    rstd = (1.0 / torch.sqrt((hd * hd).mean(dim=1) + EPS)).float()
    xhat = h * rstd[:, None]
    y = (xhat * s["weight"]).to(dt)
    hat8 = _restore(*_quantise(xhat), s["case"]["cols"])
    return h.to(dt), y, hat8, rstd


def _plain_backward(s, hat8, rstd):
    dy = s["dy"].float()
    g = dy * s["weight"]
    c = (g * hat8).mean(dim=1, keepdim=True)
    dh = rstd[:, None] * (g - hat8 * c)
    if s["dres"] is not None:
        dh = dh + s["dres"].float()
    return dh.to(s["dtype"]), (dy * hat8).sum(dim=0)


def _plain(s):
    case = s["case"]
    op, cols = case["op"], case["cols"]
    if op == "pack":
        return _restore(*_quantise(s["x"].float()), cols).to(s["dtype"])
    if op == "wgrad":
        dy = s["dy"].float()
        dw = dy.t() @ _restore(s["codes"], s["scales"], cols)
        if s["gain"] is not None:
            dw = dw * s["gain"]
        return (dw, dy.sum(dim=0)) if case["bias"] else (dw,)
    h, y, hat8, rstd = _plain_forward(s)
    out = {"y": y, "rstd": rstd}
    if s["residual"] is not None:
        out["h"] = h
    if op == "norm" and not case["backward"]:
        out["xhat"] = hat8.to(s["dtype"])
        return out
    if op == "block":
        out["dw"] = (s["dout"].float().t() @ hat8) * s["weight"]
    out["dh"], out["dweight"] = _plain_backward(s, hat8, rstd)
    return out


def _framework(s):
    from sparse_communication_distributed_amd import scape as S
    case = s["case"]
    op = case["op"]
    if op == "pack":
        S.act_pack(s["x"], s["act"])
        S.act_unpack(s["act"], s["restored"])
        return s["restored"]
    if op == "wgrad":
        S.wgrad(s["dy"], s["act"], s["dw"], s["wgrad_ws"], gain=s["gain"], dbias=s["db"])
        return (s["dw"], s["db"]) if case["bias"] else (s["dw"],)
    S.rmsnorm_pack(s["x"], s["weight"], EPS, s["y"], xhat=s["act"], rstd=s["rstd"], residual=s["residual"], h=s["h"])
    out = {"y": s["y"], "rstd": s["rstd"]}
    if s["residual"] is not None:
        out["h"] = s["h"]
    if op == "norm" and not case["backward"]:
        S.act_unpack(s["act"], s["restored"])
        out["xhat"] = s["restored"]
        return out
    if op == "block":
        S.wgrad(s["dout"], s["act"], s["dw"], s["wgrad_ws"], gain=s["weight"])
        out["dw"] = s["dw"]
    S.rmsnorm_backward(s["dy"], s["act"], s["rstd"], s["weight"], s["dh"], s["dweight"], s["norm_ws"],
                       dres=s["dres"])
    out["dh"], out["dweight"] = s["dh"], s["dweight"]
    return out


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------- work and exact


def work(case):
    """The checkpoint counts where it is written and again where it is read:
    it exists to be kept from the forward pass to the backward pass."""
    rows, cols, size = case["rows"], case["cols"], DTYPES[case["dtype"]].itemsize
    nb = (cols + BLOCK - 1) // BLOCK
    packed = rows * (cols + nb)
    mat = rows * cols * size
    op = case["op"]
    if op == "pack":
        return {"bytes": 2 * mat + 2 * packed, "flops": 5 * rows * cols}
    total, flops = 0, 0
    if op in ("norm", "block"):
        res = case.get("residual", True)
        total += mat * (4 if res else 2) + packed + 4 * rows + 4 * cols  # x, residual, h, y, codes, rstd, weight
        flops += 9 * rows * cols
        if op == "block" or case["backward"]:
            total += mat * (3 if res else 2) + packed + 4 * rows + 8 * cols
            flops += 9 * rows * cols
        else:
            total += packed + mat
            flops += rows * cols
    if op in ("wgrad", "block"):
        out = case["out"]
        total += rows * out * size + packed + 4 * out * cols
        total += 4 * cols if case.get("gain", op == "block") else 0
        flops += 2 * rows * cols * out
        if case.get("bias"):
            total += 4 * out
            flops += rows * out
    return {"bytes": total, "flops": flops}


def _power(e):
    """2^e in 64 bits, for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_pack(v):
    """The nearest multiples of the block's quantum (half to even), in 64
    bits: the quantum is the least power of two of which 127 cover the
    block's largest magnitude."""
    rows, cols = v.shape
    out = torch.zeros_like(v)
    for c0 in range(0, cols, BLOCK):
        blk = v[:, c0:c0 + BLOCK]
        top = blk.abs().max(dim=1, keepdim=True).values
        _, ex = torch.frexp(top)  # top = m * 2^ex, 1/2 <= m < 1
        quantum = _power(ex - 7)
        quantum = torch.where(127.0 * quantum < top, 2.0 * quantum, quantum).clamp(min=2.0 ** -126)
        out[:, c0:c0 + BLOCK] = torch.where(top > 0, torch.round(blk / quantum) * quantum, torch.zeros_like(blk))
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    op, cols = case["op"], case["cols"]
    f64 = torch.float64
    if op == "pack":
        return _exact_pack(s["x"].to(f64))
    if op == "wgrad":
        step = _power(s["scales"].to(torch.int64) - 127) * (s["scales"] > 0)
        x8 = (s["codes"].to(f64) * step.repeat_interleave(BLOCK, dim=1))[:, :cols]
        dy = s["dy"].to(f64)
        dw = torch.matmul(x8.t().contiguous(), dy).t()
        if s["gain"] is not None:
            dw = dw * s["gain"].to(f64)[None, :]
        return (dw.contiguous(), dy.sum(0)) if case["bias"] else (dw.contiguous(),)
    h = s["x"].to(f64)
    if s["residual"] is not None:
        h = h + s["residual"].to(f64)
    h32 = h.float()  # the sum that the norm is of, in 32 bits
    ms = (h32.to(f64) ** 2).sum(1) / cols
    rstd = (ms + EPS).rsqrt()
    w = s["weight"].to(f64)
    y = h * rstd[:, None] * w
    # the checkpoint holds the codes of the 32-bit number x_hat, made of the
    # 32-bit h and rstd
    hat8 = _exact_pack((h32 * rstd.float()[:, None]).to(f64))
    out = {"y": y, "rstd": rstd}
    if s["residual"] is not None:
        out["h"] = h
    if op == "norm" and not case["backward"]:
        out["xhat"] = hat8
        return out
    if op == "block":
        out["dw"] = torch.matmul(hat8.t().contiguous(), s["dout"].to(f64)).t().contiguous() * w
    r32 = rstd.float().to(f64)[:, None]
    dy = s["dy"].to(f64)
    inner = (dy * w * hat8).sum(1, keepdim=True) / cols
    dh = r32 * (dy * w - inner * hat8)
    if s["dres"] is not None:
        dh = dh + s["dres"].to(f64)
    out["dh"], out["dweight"] = dh, (dy * hat8).sum(0)
    return out
