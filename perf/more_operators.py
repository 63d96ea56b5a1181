"""The operators at the ends of a training step, as they are timed: cases,
inputs, one pass of each, and exact results.

A pass is one of
  embed     rows of an embedding table by token (scaled, with a second table's
            rows by position added): forward, or forward and the gradient of
            each table;
  logprobs  log probabilities of given tokens, with the entropy of each row
            and the likeliest alternatives, and the gradient of the logits, in
            the same pass or in one of its own;
  clip      the norm of the gradients of one or several workers and the
            gradients clipped by it, written to the optimizer's fp32 rows.

A token (target) outside the table (vocabulary) has no row, no log probability
(0) and no gradient.  Alternatives are ordered by logit, ties by index.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"
INDEX = {"int64": torch.int64, "int32": torch.int32}
MIXED = (1531, 64, 2903, 1, 777, 4099, 250, 17, 1024, 3)  # tensor sizes of every alignment


# ------------------------------------------------------------------- cases


def _embed(name, tokens, vocab, cols, dtype, backward, table="fp32", positions=0, scale=1.0, ids="int64", pad=0):
    return {"name": name, "op": "embed", "tokens": tokens, "vocab": vocab, "cols": cols, "dtype": dtype,
            "backward": backward, "table": table, "positions": positions, "scale": scale, "ids": ids, "pad": pad}


def _logprobs(name, rows, vocab, dtype, top=0, entropy=False, grad="none", scale=1.0, ids="int64", pad=0):
    return {"name": name, "op": "logprobs", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top,
            "entropy": entropy, "grad": grad, "scale": scale, "ids": ids, "pad": pad}


def _clip(name, dtype, workers, scale, max_norm, flat=0, mixed=0, layers=0, hidden=0, ffn=0, vocab=0):
    return {"name": name, "op": "clip", "dtype": dtype, "workers": workers, "scale": scale, "max_norm": max_norm,
            "flat": flat, "mixed": mixed, "layers": layers, "hidden": hidden, "ffn": ffn, "vocab": vocab}


def listed():
    return [
        # one token of the 1.8B layout from the fp32 parameters: latency of the launch
        _embed("embed_token", 1, 32000, 2048, "bf16", False),
        # a micro-batch of the 1.8B layout: 8 sequences of 2048
        _embed("embed_step", 16384, 32000, 2048, "bf16", True),
        # the GPT layout's two tables, 8 sequences of 1024, fp16 activations
        _embed("embed_gpt_fp16", 8192, 50257, 1024, "fp16", True, positions=1024),
        # a ragged batch at an odd width, scaled, rows inside a wider buffer
        _embed("embed_odd_fp32", 1531, 4099, 777, "fp32", True, scale=27.875, ids="int32", pad=3),
        # one sampled token of a 32000-word vocabulary with its 20 likeliest alternatives
        _logprobs("logp_token", 1, 32000, "bf16", top=20, entropy=True, scale=1.25),
        # a batch of sampled tokens at the GPT layout's odd vocabulary, fp16 logits
        _logprobs("logp_batch_fp16", 61, 50257, "fp16", top=5, entropy=True, ids="int32", pad=7),
        # cross-entropy of 4 sequences of 2048 with its gradient: the weight of each token is known before
        _logprobs("logp_loss", 8192, 32000, "bf16", grad="fused"),
        # a policy step on fp32 logits: gradients of log probability and entropy once the advantages are known
        _logprobs("logp_policy_fp32", 1999, 32000, "fp32", entropy=True, grad="separate"),
        # two workers' rows of the smallest layout
        _clip("clip_tiny", "fp32", 2, 1.0, 1.0, flat=1 << 20),
        # three workers with many small tensors, fp16 with a loss scale
        _clip("clip_mixed_fp16", "fp16", 3, 1.0 / 1024, 0.5, mixed=131),
        # the bf16 gradients of the 500M layout, tensor by tensor, to a worker's fp32 row
        _clip("clip_gather", "bf16", 1, 0.25, 1.0, layers=24, hidden=1280, ffn=3456, vocab=32000),
        # one rank's fp32 row of the GPT layout
        _clip("clip_row", "fp32", 1, 1.0, 1.0, flat=354823168),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "logprobs", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    ids = rng.choice(["int64", "int64", "int32"])
    pad = rng.choice([0, 0, 1, 8, 40])
    if op == "embed":
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "vocab": _log_int(rng, 256, 50257),
                "cols": _log_int(rng, 64, 1280), "dtype": dtype, "backward": rng.random() < 0.75,
                "table": rng.choice(["fp32", "fp32", dtype]), "positions": rng.choice([0, 0, _log_int(rng, 64, 4096)]),
                "scale": rng.choice([1.0, 1.0, rng.uniform(0.25, 48.0)]), "ids": ids, "pad": pad}
    if op == "logprobs":
        vocab = _log_int(rng, 64, 131072)
        top = rng.choice([0, rng.randint(1, 32)])
        rows = _log_int(rng, 1, min(1024 if top else 8192, (1 << 27) // vocab))
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "top": top, "entropy": rng.random() < 0.6,
                "grad": "none" if top else rng.choice(["none", "fused", "separate"]),
                "scale": rng.choice([1.0, rng.uniform(0.5, 2.0)]), "ids": ids, "pad": pad}
    case = {"op": op, "dtype": dtype, "workers": rng.randint(1, 4),
            "scale": rng.choice([1.0, 0.125, rng.uniform(0.001, 1.0)]),
            "max_norm": rng.choice([0.1, 1.0, 1e6]), "flat": 0, "mixed": 0, "layers": 0, "hidden": 0, "ffn": 0,
            "vocab": 0}
    kind = rng.choice(["flat", "mixed", "layers"])
    if kind == "flat":
        case["flat"] = _log_int(rng, 1, 1 << 26)
    elif kind == "mixed":
        case["mixed"] = _log_int(rng, 1, 300)
    else:
        case.update(layers=rng.randint(1, 12), hidden=8 * _log_int(rng, 8, 128), vocab=_log_int(rng, 256, 32000))
        case["ffn"] = 4 * case["hidden"]
    return case


# ------------------------------------------------------------------ inputs


def _gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + stream) & 0x7FFFFFFFFFFFFFFF)
    return g


def _matrix(rows, cols, pad, dtype):
    """An empty [rows][cols] matrix whose rows lie cols + pad elements apart."""
    return torch.empty((rows, cols + pad), dtype=dtype, device=DEV)[:, :cols]


def _tokens(count, vocab, seed, stream, dtype, none):
    """Token ids: the n-th likeliest word about 1/n as frequent as the first,
    likely and rare words in any order in the table.  A share `none` of them
    is padding (-100)."""
    g = _gen(seed, stream)
    rank = torch.exp(torch.rand(count, generator=g, device=DEV, dtype=torch.float64) * math.log(vocab + 1.0)) - 1.0
    word = torch.randperm(vocab, generator=g, device=DEV)
    ids = word[rank.long().clamp(0, vocab - 1)]
    if count > 8:
        ids = torch.where(torch.rand(count, generator=g, device=DEV) < none, -100, ids)
    return ids.to(dtype)


def _gradient(rows, cols, pad, seed, stream, dtype):
    """Gradients of activations: tokens of unequal weight, masked tokens (zero
    rows).  fp16 gradients carry a loss scale."""
    g = _gen(seed, stream)
    tok = 1e-3 * torch.exp(torch.randn((rows, 1), generator=g, device=DEV))
    if dtype == torch.float16:
        tok = tok * 128.0
    if rows > 8:
        tok = tok * (torch.rand((rows, 1), generator=g, device=DEV) >= 0.05).float()
    out = _matrix(rows, cols, pad, dtype)
    out.copy_(torch.randn((rows, cols), generator=g, device=DEV) * tok)
    return out


def _sizes(case):
    """Numbers of elements of one worker's tensors, in the layout's order."""
    if case["flat"]:
        return [case["flat"]]
    if case["mixed"]:
        return [MIXED[i % len(MIXED)] for i in range(case["mixed"])]
    h, f, v = case["hidden"], case["ffn"], case["vocab"]
    return [v * h] + [h, h * h, h * h, h * h, h * h, h, f * h, f * h, f * h] * case["layers"] + [h, v * h]


def _inputs(case, seed):
    dt = DTYPES[case["dtype"]]
    s = {"case": case, "dtype": dt}
    if case["op"] == "embed":
        tokens, vocab, cols = case["tokens"], case["vocab"], case["cols"]
        s["ids"] = _tokens(tokens, vocab, seed, 1, INDEX[case["ids"]], 0.02)
        s["table"] = (0.02 * torch.randn((vocab, cols), generator=_gen(seed, 2), device=DEV)).to(DTYPES[case["table"]])
        s["pos"] = s["pos_table"] = None
        if case["positions"]:
            s["pos"] = (torch.arange(tokens, device=DEV) % case["positions"]).to(INDEX[case["ids"]])
            s["pos_table"] = (0.02 * torch.randn((case["positions"], cols), generator=_gen(seed, 3),
                                                 device=DEV)).to(DTYPES[case["table"]])
        if case["backward"]:
            s["dy"] = _gradient(tokens, cols, case["pad"], seed, 4, dt)
    elif case["op"] == "logprobs":
        rows, vocab = case["rows"], case["vocab"]
        g = _gen(seed, 1)
        s["targets"] = _tokens(rows, vocab, seed, 2, INDEX[case["ids"]], 0.05)
        x = 2.0 * torch.randn((rows, vocab), generator=g, device=DEV) + torch.randn((rows, 1), generator=g, device=DEV)
        # most targets are likely, some rows are all but decided
        rise = 12.0 * torch.rand(rows, generator=g, device=DEV) ** 2 + 3.0
        x.scatter_add_(1, s["targets"].long().clamp(min=0)[:, None], rise[:, None])
        # one row in eight may only be continued by some of the words (the target among them)
        barred = torch.rand(vocab, generator=g, device=DEV) < 0.9
        few = torch.rand(rows, generator=g, device=DEV) < 0.125
        kept = x.gather(1, s["targets"].long().clamp(min=0)[:, None])
        x.masked_fill_(few[:, None] & barred[None, :], -math.inf)
        x.scatter_(1, s["targets"].long().clamp(min=0)[:, None], kept)
        s["logits"] = _matrix(rows, vocab, case["pad"], dt)
        s["logits"].copy_(x)
        if case["grad"] != "none":
            unit = (65536.0 if dt == torch.float16 else 1.0) / rows  # fp16 gradients carry a loss scale
            s["dlogp"] = -unit * (0.5 + torch.rand(rows, generator=g, device=DEV))
            s["dentropy"] = torch.full((rows,), -0.01 * unit, device=DEV) if case["entropy"] else None
    else:
        sizes, workers = _sizes(case), case["workers"]
        total = sum(sizes)
        g = _gen(seed, 1)
        # tensors of unequal spread; the norm lies above max_norm for some workers, below it for others
        level = case["max_norm"] / (case["scale"] * math.sqrt(total))
        level = min(level, 1e3 if dt == torch.float16 else 1e9)
        s["grads"] = []
        for w in range(workers):
            flat = torch.randn(total, generator=g, device=DEV)
            at = 0
            for size in sizes:
                spread = level * (2.0 if w % 2 == 0 else 0.4) * (0.7 + 0.6 * ((at * 7 + w) % 11) / 11.0)
                s["grads"].append((flat[at:at + size] * spread).to(dt))
                at += size
            del flat
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    # the buffers a training or serving program keeps: outputs (parts of its
    # gradient rows among them), workspaces, the list of its gradients
    from sparse_communication_distributed_amd import scape as S
    dt = s["dtype"]

    def scratch(size):
        return torch.empty(size, dtype=torch.uint8, device=DEV)

    if case["op"] == "embed":
        tokens, cols = case["tokens"], case["cols"]
        s["out"] = torch.empty((tokens, cols), dtype=dt, device=DEV)
        if case["backward"]:
            s["dtable"] = torch.empty((case["vocab"], cols), device=DEV)
            s["ws"] = scratch(S.embed_workspace_bytes(tokens, cols))
            if case["positions"]:
                s["dpos"] = torch.empty((case["positions"], cols), device=DEV)
    elif case["op"] == "logprobs":
        rows, vocab, top = case["rows"], case["vocab"], case["top"]
        s["logp"] = torch.empty(rows, device=DEV)
        s["entropy"] = torch.empty(rows, device=DEV) if case["entropy"] else None
        s["stats"] = torch.empty((rows, 2), device=DEV) if case["grad"] == "separate" else None
        s["top_logp"] = torch.empty((rows, top), device=DEV) if top else None
        s["top_ids"] = torch.empty((rows, top), dtype=torch.int32, device=DEV) if top else None
        s["dlogits"] = torch.empty((rows, vocab), dtype=dt, device=DEV) if case["grad"] != "none" else None
        s["ws"] = scratch(S.token_logprobs_workspace_bytes(rows, vocab, top))
    else:
        sizes, workers = _sizes(case), case["workers"]
        s["row"] = torch.empty((workers, sum(sizes)), device=DEV)
        s["norm"] = torch.empty(workers, device=DEV)
        parts = [p for w in range(workers) for p in s["row"][w].split(sizes)]
        s["list"] = S.GradList(s["grads"], out=parts, groups=workers)
        s["ws"] = scratch(S.grad_workspace_bytes(s["list"]))
    return s


# -------------------------------------------------------------- plain form


def _plain_rows(table, ids):
    """fp32 rows of a table; zeros where there is no such row."""
    there = (ids >= 0) & (ids < table.shape[0])
    return torch.where(there[:, None], table[torch.where(there, ids, 0).long()].float(), 0.0)


def _plain_scatter(dy, ids, rows, scale):
    """The gradient of a table from that of its rows; those of no row go to
    one more, which is dropped."""
    there = (ids >= 0) & (ids < rows)
    acc = torch.zeros((rows + 1, dy.shape[1]), device=DEV)
    acc.index_add_(0, torch.where(there, ids, rows).long(), dy.float())
    return acc[:rows] * scale


def _plain_embed(s):
    case = s["case"]
    out = _plain_rows(s["table"], s["ids"]) * case["scale"]
    if case["positions"]:
        out = out + _plain_rows(s["pos_table"], s["pos"])
    res = {"out": out.to(s["dtype"])}
    if case["backward"]:
        res["dtable"] = _plain_scatter(s["dy"], s["ids"], case["vocab"], case["scale"])
        if case["positions"]:
            res["dpos"] = _plain_scatter(s["dy"], s["pos"], case["positions"], 1.0)
    return res


def _plain_logprobs(s):
    case = s["case"]
    x = s["logits"].float()
    z = x * case["scale"]
    best = z.argmax(dim=1, keepdim=True)
    z = z - z.gather(1, best)
    e = torch.exp(z)
    # the sum over the other words: where it is small against 1, the log
    # probability of the likeliest word and the entropy are of its size
    others = e.scatter(1, best, 0.0).sum(dim=1, keepdim=True)
    logs = torch.log1p(others)
    there = (s["targets"] >= 0) & (s["targets"] < case["vocab"])
    y = torch.where(there, s["targets"], 0).long()[:, None]
    logp = z.gather(1, y) - logs
    res = {"logp": torch.where(there, logp[:, 0], 0.0)}
    if case["entropy"]:
        ez = torch.where(e > 0, e * z, 0.0)  # e^z * z -> 0 as z -> -inf
        h = logs - ez.sum(dim=1, keepdim=True) / (1.0 + others)
        res["entropy"] = h[:, 0]
    if case["top"]:
        # one whole number orders by logit, then by the lower index (-0 as 0)
        bits = (x + 0.0).view(torch.int32)
        key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
        key = key + (case["vocab"] - 1 - torch.arange(case["vocab"], device=DEV))
        ids = case["vocab"] - 1 - (torch.topk(key, case["top"], dim=1).values & 0xFFFFFFFF)
        res["top_ids"] = ids.to(torch.int32)
        res["top_logp"] = z.gather(1, ids) - logs
    if case["grad"] != "none":
        p = e / (1.0 + others)
        w = torch.where(there, s["dlogp"], 0.0)[:, None]
        d = (-w * p).scatter(1, y, -w * torch.expm1(logp))  # 1 - p at the target
        if case["entropy"]:
            d = d - s["dentropy"][:, None] * torch.where(p > 0, p * (z - logs + h), 0.0)
        res["dlogits"] = (d * case["scale"]).to(s["dtype"])
    return res


def _plain_clip(s):
    case = s["case"]
    flat = torch.cat(s["grads"]).view(case["workers"], -1).float()
    # 64 bits: a sum over the whole model
    norm = (flat * flat).sum(dim=1, dtype=torch.float64).sqrt() * case["scale"]
    factor = case["scale"] * torch.where(norm > case["max_norm"], case["max_norm"] / norm, 1.0)
    return {"norm": norm.float(), "row": flat * factor.float()[:, None]}


def _plain(s):
    return {"embed": _plain_embed, "logprobs": _plain_logprobs, "clip": _plain_clip}[s["case"]["op"]](s)


def _framework(s):
    from sparse_communication_distributed_amd import scape as S
    case = s["case"]
    if case["op"] == "embed":
        S.embed(s["ids"], s["table"], s["out"], scale=case["scale"], pos=s["pos"], pos_table=s["pos_table"])
        res = {"out": s["out"]}
        if case["backward"]:
            S.embed_backward(s["ids"], s["dy"], s["dtable"], s["ws"], scale=case["scale"])
            res["dtable"] = s["dtable"]
            if case["positions"]:
                S.embed_backward(s["pos"], s["dy"], s["dpos"], s["ws"])
                res["dpos"] = s["dpos"]
        return res
    if case["op"] == "logprobs":
        fused, separate = case["grad"] == "fused", case["grad"] == "separate"
        S.token_logprobs(s["logits"], s["targets"], s["logp"], s["ws"], stats=s["stats"], entropy=s["entropy"],
                         top_logp=s["top_logp"], top_ids=s["top_ids"], scale=case["scale"],
                         dlogp=s["dlogp"] if fused else None, dentropy=s["dentropy"] if fused else None,
                         dlogits=s["dlogits"] if fused else None)
        if separate:
            S.token_logprobs_backward(s["logits"], s["targets"], s["stats"], s["dlogits"], dlogp=s["dlogp"],
                                      entropy=s["entropy"], dentropy=s["dentropy"], scale=case["scale"])
        return {k: s[k] for k in ("logp", "entropy", "top_ids", "top_logp", "dlogits") if s[k] is not None}
    S.clip_grads(s["list"], case["max_norm"], s["norm"], s["ws"], scale=case["scale"])
    return {"norm": s["norm"], "row": s["row"]}


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------- work and exact


def work(case):
    size = DTYPES[case["dtype"]].itemsize
    if case["op"] == "embed":
        tokens, vocab, cols = case["tokens"], case["vocab"], case["cols"]
        wide = DTYPES[case["table"]].itemsize
        index = tokens * INDEX[case["ids"]].itemsize * (2 if case["positions"] else 1)
        # rows are read once each, however many tokens share them
        total = index + min(tokens, vocab) * cols * wide + tokens * cols * size
        total += min(tokens, case["positions"]) * cols * wide
        flops = tokens * cols * (2 if case["positions"] else 1)
        if case["backward"]:
            total += index + tokens * cols * size + (vocab + case["positions"]) * cols * 4
            flops += tokens * cols * (2 if case["positions"] else 1)
        return {"bytes": total, "flops": flops}
    if case["op"] == "logprobs":
        rows, vocab = case["rows"], case["vocab"]
        # the logits count once, also where the gradient is a call of its own
        total = rows * vocab * size * (1 if case["grad"] == "none" else 2)
        total += rows * (INDEX[case["ids"]].itemsize + 4 + (4 if case["entropy"] else 0) + 8 * case["top"])
        flops = rows * vocab * (5 + (2 if case["entropy"] else 0))
        if case["grad"] != "none":
            total += rows * (8 if case["entropy"] else 4)
            flops += rows * vocab * (4 + (3 if case["entropy"] else 0))
        return {"bytes": total, "flops": flops}
    n = case["workers"] * sum(_sizes(case))
    # the gradients count once, though the norm has to be known before the first is clipped
    return {"bytes": n * (size + 4) + 4 * case["workers"], "flops": 3 * n}


def _exact_embed(s):
    case = s["case"]
    f64 = torch.float64

    def pick(table, ids):
        wide = torch.cat([table.to(f64), torch.zeros((1, table.shape[1]), dtype=f64, device=DEV)])
        row = ids.long()
        return wide[torch.where((row < 0) | (row >= table.shape[0]), table.shape[0], row)]

    def gradient(ids, rows, scale):
        order = torch.argsort(ids.long(), stable=True)
        row = ids.long()[order]
        # prefix sums of the rows in the order of their tokens; a token's sum is a difference of two
        out = torch.zeros((rows, case["cols"]), dtype=f64, device=DEV)
        edges = torch.searchsorted(row, torch.arange(rows + 1, device=DEV))
        for c in range(0, case["cols"], 256):
            run = torch.cumsum(s["dy"][order, c:c + 256].to(f64), dim=0)
            run = torch.cat([torch.zeros_like(run[:1]), run])
            out[:, c:c + 256] = scale * (run[edges[1:]] - run[edges[:-1]])
        return out

    out = case["scale"] * pick(s["table"], s["ids"])
    if case["positions"]:
        out = out + pick(s["pos_table"], s["pos"])
    res = {"out": out}
    if case["backward"]:
        res["dtable"] = gradient(s["ids"], case["vocab"], case["scale"])
        if case["positions"]:
            res["dpos"] = gradient(s["pos"], case["positions"], 1.0)
    return res


def _exact_logprobs(s):
    case = s["case"]
    f64 = torch.float64
    rows, vocab = case["rows"], case["vocab"]
    res = {"logp": torch.zeros(rows, dtype=f64, device=DEV)}
    if case["entropy"]:
        res["entropy"] = torch.zeros(rows, dtype=f64, device=DEV)
    if case["top"]:
        res["top_ids"] = torch.zeros((rows, case["top"]), dtype=torch.int32, device=DEV)
        res["top_logp"] = torch.zeros((rows, case["top"]), dtype=f64, device=DEV)
    if case["grad"] != "none":
        res["dlogits"] = torch.zeros((rows, vocab), dtype=f64, device=DEV)
    step = max(1, (1 << 26) // vocab)
    words = torch.arange(vocab, device=DEV)[None, :]
    for r in range(0, rows, step):
        part = slice(r, r + step)
        x = s["logits"][part].to(f64)
        lp = x * case["scale"]
        lp = lp - torch.logsumexp(lp, dim=1, keepdim=True)
        p = lp.exp()
        hit = words == s["targets"][part].long()[:, None]
        res["logp"][part] = torch.where(hit, lp, 0.0).sum(dim=1)
        plogp = torch.where(p > 0, p * lp, 0.0)
        h = -plogp.sum(dim=1)
        if case["entropy"]:
            res["entropy"][part] = h
        if case["top"]:
            best = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            res["top_ids"][part] = best.to(torch.int32)
            res["top_logp"][part] = lp.gather(1, best)
        if case["grad"] != "none":
            w = s["dlogp"][part].to(f64) * hit.any(dim=1)
            d = w[:, None] * (hit.to(f64) - p)
            if case["entropy"]:
                d = d - s["dentropy"][part].to(f64)[:, None] * (plogp + p * h[:, None])
            res["dlogits"][part] = case["scale"] * d
    return res


def _exact_clip(s):
    case = s["case"]
    per = len(s["grads"]) // case["workers"]
    norms, rows = [], []
    for w in range(case["workers"]):
        flat = torch.cat([g.reshape(-1) for g in s["grads"][w * per:(w + 1) * per]]).to(torch.float64)
        flat *= case["scale"]
        norm = math.sqrt(float(torch.dot(flat, flat)))
        if norm > case["max_norm"]:
            flat *= case["max_norm"] / norm
        norms.append(norm)
        rows.append(flat)
    return {"norm": torch.tensor(norms, dtype=torch.float64, device=DEV), "row": torch.stack(rows)}


def exact(case, seed):
    s = _inputs(case, seed)
    return {"embed": _exact_embed, "logprobs": _exact_logprobs, "clip": _exact_clip}[case["op"]](s)
