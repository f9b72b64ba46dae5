"""Cases and plain forms of the operators at the two ends of a language model and
before the optimizer's step: embedding lookup with its gradient by tokens, log
probabilities of given tokens with entropy, alternatives and gradient (and the
loss that takes its gradient in the same pass), and the global gradient norm over
many tensors with clipping.

`own` false: elementary torch operations in 32 bits (64 for the squares' sum over
a whole model), rounded once at the end.  `own` true: the calls of
sparse_communication_sharded_gb300.layers.

A token or target below 0 stands for none: its embedding row is zeros and it has
no gradient; its log probability is 0 and its row of the logits' gradient zeros.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-6  # beside the norm, in the clipping coefficient


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # one token looked up while a Llama-1.8B-shaped model answers: pure latency
        dict(name="embed_one_token", op="embed", tokens=1, vocab=32000, cols=2048, table="bf16",
             out="bf16", scale=1.0, index="i64", spread="uniform"),
        # a ragged batch from a float32 table with an odd width, scaled, padding among it
        dict(name="embed_odd_f32", op="embed", tokens=16381, vocab=50304, cols=1283, table="f32",
             out="bf16", scale=35.8, index="i32", spread="padded"),
        # its gradient for eight GPT-345M sequences: words of a text, few of them most of it
        dict(name="embed_bwd_gpt345m", op="embed_bwd", tokens=8192, vocab=50304, cols=1024, dtype="bf16",
             grad="bf16", scale=1.0, index="i64", spread="text", offset=0, gap=0),
        # four Llama-500M sequences of 4K padded at their ends, into a flat vector at an odd place
        dict(name="embed_bwd_llama500m_padded", op="embed_bwd", tokens=16384, vocab=32000, cols=1280,
             dtype="bf16", grad="bf16", scale=2.0, index="i64", spread="padded", offset=3, gap=0),
        # one row of logits while a model answers: the chosen token's, entropy, five alternatives
        dict(name="logprob_one_token", op="logprob", rows=1, vocab=32000, dtype="bf16", entropy=True,
             top=5, gap=0, mask="none"),
        # scoring four 2K sequences of the Llama-1.8B shape
        dict(name="logprob_llama1p8b_8k", op="logprob", rows=8192, vocab=32000, dtype="bf16",
             entropy=True, top=0, gap=0, mask="none"),
        # float32 logits of an odd vocabulary, part of it masked, rows of a wider buffer
        dict(name="logprob_odd_f32_top20", op="logprob", rows=333, vocab=50301, dtype="f32",
             entropy=True, top=20, gap=3, mask="inf"),
        # a policy's gradient: through log probability and entropy, Llama-500M
        dict(name="logprob_bwd_llama500m", op="logprob_bwd", rows=4096, vocab=32000, dtype="bf16",
             entropy=True, gap=0, mask="none"),
        # loss and gradient of eight GPT-345M sequences, as pretrained
        dict(name="loss_gpt345m_8k", op="loss", rows=8192, vocab=50304, dtype="bf16", gap=0, mask="none"),
        # the gradients of a small stack of blocks, before its step: latency
        dict(name="clip_small_stack", op="clip", shapes="blocks", parts=13, largest=65536, dtype="bf16",
             out="bf16", over=2.0, offset=0),
        # the norm of one worker's flat Llama-500M gradient, tensor by tensor, for the log
        dict(name="norm_llama500m", op="norm", shapes="llama500m", parts=0, largest=0, dtype="bf16",
             offset=0),
        # GPT-345M gradients gathered in float32 over small batches, clipped into a worker's
        # flat bfloat16 vector
        dict(name="clip_gpt345m_f32", op="clip", shapes="gpt345m", parts=0, largest=0, dtype="f32",
             out="bf16", over=3.0, offset=0),
    ]


MAX_TABLE = 50304 * 2048    # elements of an embedding table
MAX_ROWS = 16384 * 2048     # elements of its looked-up rows
MAX_LOGITS = 8192 * 50304   # elements of logits (bfloat16; half of it in float32)
MAX_GRADS = 250_000_000     # elements of a set of gradients


def _size(rng, lo, hi):
    """A size spread over its logarithm: any number, or a multiple of 8 or of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    step = rng.choice([1, 1, 8, 64])
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(["embed", "embed_bwd", "embed_bwd", "logprob", "logprob", "logprob_bwd", "loss",
                     "loss", "norm", "clip"])
    if op in ("embed", "embed_bwd"):
        cols, vocab = _size(rng, 64, 8192), _size(rng, 256, 131072)
        vocab = max(256, min(vocab, MAX_TABLE // cols))
        tokens = max(1, min(_size(rng, 1, 65536), MAX_ROWS // cols))
        c = dict(op=op, tokens=tokens, vocab=vocab, cols=cols, scale=rng.choice([1.0, 1.0, math.sqrt(cols)]),
                 index=rng.choice(["i64", "i32"]), spread=rng.choice(["text", "text", "uniform", "padded"]))
        if op == "embed":
            c.update(table=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["bf16", "bf16", "f32"]))
        else:
            c.update(dtype=rng.choice(["bf16", "bf16", "f32"]), grad=rng.choice(["bf16", "bf16", "f32"]),
                     offset=rng.choice([0, 0, 8, 3]), gap=rng.choice([0, 0, 16, 3]))
        return c
    if op in ("logprob", "logprob_bwd", "loss"):
        vocab, dtype = _size(rng, 256, 262144), rng.choice(["bf16", "bf16", "f32"])
        most = MAX_LOGITS // (2 if dtype == "f32" else 1) // vocab
        c = dict(op=op, rows=max(1, min(_size(rng, 1, 16384), most)), vocab=vocab, dtype=dtype,
                 gap=rng.choice([0, 0, 8, 3]), mask=rng.choice(["none", "none", "inf", "lowest"]))
        if op == "logprob":
            c.update(entropy=rng.random() < 0.6, top=rng.choice([0, 0, 1, 5, 20]))
            if c["top"]:  # the plain form looks through a row once for each alternative
                c["rows"] = max(1, min(c["rows"], most // (1 + c["top"])))
        if op == "logprob_bwd":
            c.update(entropy=rng.random() < 0.5)
        return c
    parts, dtype = _size(rng, 1, 400), rng.choice(["bf16", "bf16", "f32"])
    largest = max(256, min(_size(rng, 256, 1 << 27), MAX_GRADS // parts))
    c = dict(op=op, shapes="blocks", parts=parts, largest=largest, dtype=dtype, offset=rng.choice([0, 0, 8, 3]))
    if op == "clip":
        c.update(out=rng.choice(["bf16", "bf16", "f32"]), over=rng.choice([0.5, 2.0, 30.0]))
    return c


def _sizes(case):
    """Elements of each tensor of a set of gradients."""
    if case["shapes"] == "llama500m":  # 24 layers, hidden 1280, feed-forward 3584, vocabulary 32000
        h, f = 1280, 3584
        return [32000 * h] + [h, h * h, h * h, h * h, h * h, h, h * f, h * f, f * h] * 24 + [h, 32000 * h]
    if case["shapes"] == "gpt345m":  # 24 layers, hidden 1024, feed-forward 4096, vocabulary 50304
        h, f = 1024, 4096
        layer = [h, h] + [h * h, h] * 4 + [h, h, f * h, f, h * f, h]
        return [50304 * h, 1024 * h] + layer * 24 + [h, h]
    # vectors and matrices in turn, the matrices up to the largest
    n, top = case["parts"], case["largest"]
    return [max(1, top // (1 + i % 5) - i % 3) if i % 2 == 0 else 1 + (top // 64 + 7 * i) % 5000
            for i in range(n)]


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    """Tokens with the frequencies of words in a text (or padded, or spread evenly), small
    tables and gradients, logits of a trained model: a few large ones a row, the target's
    often among them."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device=DEV, generator=g)

    op, s = case["op"], {"case": dict(case)}
    if op in ("embed", "embed_bwd"):
        n, v, c = case["tokens"], case["vocab"], case["cols"]
        if case["spread"] == "uniform":
            t = (uniform(n) * v).long().clamp_max(v - 1)
        else:
            # the k-th commonest of a text's words is 1/k as common as the first
            rank = (torch.exp(uniform(n) * math.log(v)) - 1).long().clamp_max(v - 1)
            t = torch.randperm(v, device=DEV, generator=g)[rank]
        if case["spread"] == "padded":
            # ends of sequences: one padding token, and a few positions that stand for none
            t = torch.where(uniform(n) < 0.2, 2 % v, t)
            t = torch.where(uniform(n) < 0.02, -1, t)
        s["tokens"] = t.to(torch.int64 if case["index"] == "i64" else torch.int32)
        if op == "embed":
            s["w"] = (normal(v, c) * 0.02).to(_dt(case["table"]))
        else:
            s["dy"] = (normal(n, c + case["gap"]) * 1e-3).to(_dt(case["dtype"]))[:, :c]
            s["grad"] = torch.zeros(case["offset"] + v * c, device=DEV, dtype=_dt(case["grad"]))
        return s
    if op in ("logprob", "logprob_bwd", "loss"):
        n, v = case["rows"], case["vocab"]
        x = normal(n, v + case["gap"]).mul_(2.5).add_(normal(n, 1), alpha=3.0)
        # vocabulary that may not be chosen: its last part, and every 11th column
        allowed = torch.ones(v, dtype=torch.bool, device=DEV)
        if case["mask"] != "none":
            allowed[v - v // 10:] = False
            allowed[torch.arange(v, device=DEV) % 11 == 10] = False
        options = torch.nonzero(allowed).flatten()
        t = options[(uniform(n) * options.numel()).long().clamp_max(options.numel() - 1)]
        x.scatter_add_(1, t[:, None], uniform(n, 1) * 14.0)
        x = x.to(_dt(case["dtype"]))[:, :v]
        if case["mask"] != "none":
            x.masked_fill_(~allowed, -math.inf if case["mask"] == "inf" else torch.finfo(x.dtype).min)
        s["logits"] = x
        if n > 8:
            t = torch.where(uniform(n) < 0.02, -1, t)
        s["targets"] = t
        if op == "loss":
            s["weight"] = (0.5 + uniform(n)) / n
        if op == "logprob_bwd":
            s["dlogprob"] = normal(n) / n
            s["dentropy"] = normal(n) * (0.01 / n) if case["entropy"] else None
            f = x.float()
            lse = torch.logsumexp(f, 1)
            s["lse"] = lse
            s["entropy"] = None
            if case["entropy"]:
                d = (f - lse[:, None]).clamp_min(-200.0)
                s["entropy"] = -(torch.exp(d) * d).sum(1)
        return s
    sizes, dt = _sizes(case), _dt(case["dtype"])
    flat = torch.empty(case["offset"] + sum(sizes), device=DEV, dtype=dt)[case["offset"]:]
    s["grads"] = list(torch.split(flat, sizes))
    for i, t in enumerate(s["grads"]):
        t.copy_(normal(t.numel()) * (1e-4 * (1 + i % 7)))
    if op == "clip":
        total = torch.stack([(t.float() ** 2).sum(dtype=torch.float64) for t in s["grads"]]).sum().sqrt()
        s["max_norm"] = float(total) / case["over"]
        into = torch.empty(case["offset"] + sum(sizes), device=DEV, dtype=_dt(case["out"]))
        s["flat"] = into[case["offset"]:]
        s["into"] = list(torch.split(s["flat"], sizes))
    return s


# ------------------------------------------------------------------- plain forms
def _log_softmax(x):
    """(largest, log of the sum of exponentials), rows of -inf giving -inf."""
    top = x.amax(1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    return (top + torch.log(torch.exp(x - top).sum(1, keepdim=True))).squeeze(1)


def _taken(x, targets):
    """The targets' logits; 0 where there is no target."""
    t = torch.gather(x, 1, targets.long().clamp_min(0)[:, None]).squeeze(1)
    return torch.where(targets < 0, 0.0, t)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "embed":
        t = s["tokens"].long()
        y = s["w"][t.clamp_min(0)].float() * c["scale"]
        return {"y": torch.where(t[:, None] < 0, 0.0, y).to(_dt(c["out"]))}
    if op == "embed_bwd":
        t, v = s["tokens"].long(), c["vocab"]
        sums = torch.zeros(v + 1, c["cols"], device=DEV)
        sums.index_add_(0, torch.where(t < 0, v, t), s["dy"].float())
        dw = s["grad"][c["offset"]:].view(v, c["cols"])
        dw.copy_(sums[:v] * c["scale"])
        return {"dw": dw}
    if op in ("logprob", "logprob_bwd", "loss"):
        x, t = s["logits"].float(), s["targets"]
        if op == "logprob":
            lse = _log_softmax(x)
            out = {"logprob": torch.where(t < 0, 0.0, _taken(x, t) - lse), "lse": lse}
            if c["entropy"]:
                d = (x - lse[:, None]).clamp_min(-200.0)
                out["entropy"] = -(torch.exp(d) * d).sum(1)
            if c["top"]:
                column = torch.arange(c["vocab"], device=DEV)[None]
                left, best, which = x.clone(), [], []
                for _ in range(c["top"]):
                    m = left.amax(1, keepdim=True)
                    i = torch.where(left == m, column, c["vocab"]).amin(1, keepdim=True)
                    left.scatter_(1, i, -math.inf)
                    best.append(m - lse[:, None])
                    which.append(i)
                out["top_logprob"], out["top_token"] = torch.cat(best, 1), torch.cat(which, 1)
            return out
        if op == "loss":
            lse = _log_softmax(x)
            w = torch.where(t < 0, 0.0, s["weight"])
            loss = torch.where(t < 0, 0.0, w * (lse - _taken(x, t)))
        else:
            lse, w = s["lse"], torch.where(t < 0, 0.0, -s["dlogprob"])
        d = (x - lse[:, None]).clamp_min(-200.0)
        p = torch.exp(d)
        dx = p * w[:, None]
        dx.scatter_add_(1, t.clamp_min(0)[:, None], -w[:, None])
        if op == "loss":
            return {"loss": loss, "dlogits": dx.to(s["logits"].dtype)}
        if c["entropy"]:
            dx = dx - p * (d + s["entropy"][:, None]) * s["dentropy"][:, None]
        return {"dlogits": dx.to(s["logits"].dtype)}
    total = torch.stack([(t.float() * t.float()).sum(dtype=torch.float64) for t in s["grads"]]).sum().sqrt()
    if op == "norm":
        return {"norm": total.float()}
    factor = (s["max_norm"] / (total + EPS)).clamp_max(1.0).float()
    for t, o in zip(s["grads"], s["into"]):
        o.copy_(t.float() * factor)
    return {"norm": total.float(), "grads": s["flat"]}


def _framework(s):
    from sparse_communication_sharded_gb300 import layers as L

    c = s["case"]
    op = c["op"]
    if op == "embed":
        return {"y": L.embedding(s["tokens"], s["w"], scale=c["scale"], dtype=_dt(c["out"]))}
    if op == "embed_bwd":
        dw = s["grad"][c["offset"]:].view(c["vocab"], c["cols"])
        return {"dw": L.embedding_backward(s["dy"], s["tokens"], dw, scale=c["scale"])}
    if op == "logprob":
        r = L.token_logprobs(s["logits"], s["targets"], entropy=c["entropy"], top=c["top"])
        out = {"logprob": r.logprob, "lse": r.lse}
        if c["entropy"]:
            out["entropy"] = r.entropy
        if c["top"]:
            out["top_logprob"], out["top_token"] = r.top_logprob, r.top_token
        return out
    if op == "logprob_bwd":
        return {"dlogits": L.token_logprobs_backward(s["logits"], s["targets"], s["lse"], s["dlogprob"],
                                                     entropy=s["entropy"], dentropy=s["dentropy"])}
    if op == "loss":
        loss, dx = L.token_loss(s["logits"], s["targets"], s["weight"])
        return {"loss": loss, "dlogits": dx}
    if op == "norm":
        return {"norm": L.grad_norm(s["grads"])}
    return {"norm": L.clip_grad_norm(s["grads"], s["max_norm"], out=s["into"], eps=EPS), "grads": s["flat"]}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------------- sizes
def _bytes(name):
    return 4 if name == "f32" else 2


def work(case):
    """Bytes with every input read once (of a table, the rows looked up) and every output
    written once; flops of the arithmetic, a few operations a value."""
    op = case["op"]
    if op in ("embed", "embed_bwd"):
        n, v, c = case["tokens"], case["vocab"], case["cols"]
        i = n * (8 if case["index"] == "i64" else 4)
        if op == "embed":
            rows = min(n, v)
            return {"bytes": i + rows * c * _bytes(case["table"]) + n * c * _bytes(case["out"]), "flops": n * c}
        return {"bytes": i + n * c * _bytes(case["dtype"]) + v * c * _bytes(case["grad"]), "flops": 2 * n * c}
    if op in ("logprob", "logprob_bwd", "loss"):
        n, el = case["rows"], case["rows"] * case["vocab"]
        e = _bytes(case["dtype"])
        if op == "logprob":
            b = el * e + n * (8 + 8 + (4 if case["entropy"] else 0) + 12 * case["top"])
            return {"bytes": b, "flops": el * (6 if case["entropy"] else 4)}
        if op == "loss":
            return {"bytes": 2 * el * e + n * 16, "flops": 7 * el}
        return {"bytes": 2 * el * e + n * (16 + (8 if case["entropy"] else 0)), "flops": el * (7 if case["entropy"] else 4)}
    el = sum(_sizes(case))
    if op == "norm":
        return {"bytes": el * _bytes(case["dtype"]) + 4, "flops": 2 * el}
    return {"bytes": el * (_bytes(case["dtype"]) + _bytes(case["out"])) + 4, "flops": 3 * el}


# ---------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        t = s["tokens"].long()
        rows = torch.nn.functional.pad(s["w"], (0, 0, 0, 1))  # a row of zeros for no token
        return {"y": rows[torch.where(t < 0, case["vocab"], t)].double() * case["scale"]}
    if op == "embed_bwd":
        t, dy = s["tokens"].long(), s["dy"]
        order = torch.argsort(torch.where(t < 0, case["vocab"], t), stable=True)
        dw = torch.zeros(case["vocab"], case["cols"], dtype=torch.float64, device=DEV)
        for a in range(0, t.numel(), 4096):  # in pieces, in the order of the tokens
            part = order[a:a + 4096]
            part = part[t[part] >= 0]
            dw.index_put_((t[part],), dy[part].double(), accumulate=True)
        return {"dw": dw.mul_(case["scale"])}
    if op in ("logprob", "logprob_bwd", "loss"):
        parts = []
        for a in range(0, case["rows"], 1024):  # 64-bit copies of all rows would not fit beside the rest
            parts.append(_exact_rows(case, {k: v[a:a + 1024] if torch.is_tensor(v) else v for k, v in s.items()}))
        return {k: None if parts[0][k] is None else torch.cat([p[k] for p in parts]) for k in parts[0]}
    squares = 0.0
    for t in s["grads"]:
        for piece in t.split(1 << 26):
            squares = squares + piece.double().pow(2).sum()
    norm = squares.sqrt()
    if op == "norm":
        return {"norm": norm}
    factor = min(1.0, s["max_norm"] / (float(norm) + EPS))
    return {"norm": norm, "grads": torch.cat([t.double() * factor for t in s["grads"]])}


def _exact_rows(case, s):
    x, t = s["logits"].double(), s["targets"]
    n, none = x.shape[0], t < 0
    at = (torch.arange(n, device=x.device), t.clamp_min(0))
    if case["op"] == "logprob_bwd":
        lse = s["lse"].double()  # an input
    else:
        lse = torch.logsumexp(x, 1)
    logp = x - lse[:, None]
    p = logp.exp()
    chosen = torch.where(none, 0.0, logp[at])
    if case["op"] == "logprob":
        out = {"logprob": chosen, "lse": lse}
        if case["entropy"]:
            out["entropy"] = -torch.where(p > 0, p * logp, 0.0).sum(1)
        if case["top"]:
            # all of a row in order, equal ones by their place
            value, place = torch.sort(x, dim=1, descending=True, stable=True)
            out["top_logprob"] = value[:, :case["top"]] - lse[:, None]
            out["top_token"] = place[:, :case["top"]]
        return out
    one = torch.zeros_like(x)
    one[at] = 1.0
    if case["op"] == "loss":
        w = torch.where(none, 0.0, s["weight"].double())
        return {"loss": -w * chosen, "dlogits": w[:, None] * (p - one)}
    dx = torch.where(none, 0.0, s["dlogprob"].double())[:, None] * (one - p)
    if case["entropy"]:
        slope = torch.where(p > 0, p * (logp + s["entropy"].double()[:, None]), 0.0)
        dx = dx - slope * s["dentropy"].double()[:, None]
    return {"dlogits": dx}
