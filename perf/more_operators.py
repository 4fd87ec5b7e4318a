"""Cases of the rest of a language model's training step: the embedding at its
start, the residual stream between its layers (addition with gate and scale,
norms before and after a block) and the cross entropy over the vocabulary at
its end, each forward alone or with its gradients.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` makes one pass (the framework's calls where ``own`` is true,
elementary torch operations in 32 bits otherwise), ``work`` counts the bytes
and operations of a pass and ``exact`` gives the outputs in 64 bits.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
IDS = {"i32": torch.int32, "i64": torch.int64}
EPS = 1e-5
# Logits held at once by the plain form and by the 64-bit one.
PLAIN_BLOCK = 1 << 30
EXACT_BLOCK = 1 << 27


def _embed(op, name, tokens, vocab, d, dtype, ids, padded, scale):
    return dict(name=name, op=op, tokens=tokens, vocab=vocab, d=d, dtype=dtype, ids=ids,
                padded=padded, scale=scale)


def _norm(op, name, rows, d, dtype, gate, post, scale):
    return dict(name=name, op=op, rows=rows, d=d, dtype=dtype, gate=gate, post=post, scale=scale)


def _xent(op, name, tokens, vocab, d, dtype, ids, kept, tied):
    return dict(name=name, op=op, tokens=tokens, vocab=vocab, d=d, dtype=dtype, ids=ids,
                kept=kept, tied=tied)


def listed():
    return [
        # The one new token of a generated text: what a call costs at the least.
        _embed("embed_fwd", "embed_fwd_one", 1, 50257, 768, "bf16", "i64", 0.0, 1.0),
        # A training step's sixteen contexts of 1024 tokens at GPT-2-small size.
        _embed("embed_train", "embed_train_gpt2", 16384, 50257, 768, "bf16", "i64", 0.0, 1.0),
        # The long-sequence workload's tokens and width, 32-bit storage, scaled by sqrt(d), an
        # eighth of the batch padding.
        _embed("embed_train", "embed_train_long_f32", 65536, 32003, 1024, "f32", "i32", 0.125,
               32.0),
        # One token's row between two layers.
        _norm("norm_fwd", "norm_fwd_one", 1, 768, "bf16", "channel", True, 1.0),
        # A training step at GPT-2-small width, norms on both sides of the block and a gate a
        # channel.
        _norm("norm_train", "norm_train_gpt2", 16384, 768, "bf16", "channel", True, 0.7),
        # The long-sequence workload's tokens and width: a gate of its own for each element, no
        # norm behind the block.
        _norm("norm_train", "norm_train_long_f32", 65536, 1024, "f32", "row", False, 1.0),
        # A forward pass over the long-sequence workload in bf16, the plain residual addition.
        _norm("norm_fwd", "norm_fwd_long", 65536, 1024, "bf16", "none", False, 1.0),
        # A tiny model's loss over a few tokens, 32-bit storage.
        _xent("xent_fwd", "xent_fwd_tiny", 17, 1003, 64, "f32", "i64", 1.0, False),
        # Scoring one context at GPT-2-small size.
        _xent("xent_fwd", "xent_fwd_gpt2", 1024, 50257, 768, "bf16", "i64", 1.0, False),
        # The loss of a training step at GPT-2-small size, its weights tied to the embedding.
        _xent("xent_train", "xent_train_gpt2", 16384, 50257, 768, "bf16", "i64", 1.0, True),
        # Masked language modelling: a sixth of the tokens has a target.
        _xent("xent_train", "xent_train_masked", 16384, 50257, 768, "bf16", "i32", 0.15, False),
        # A 32-bit training step of a small model, odd vocabulary.
        _xent("xent_train", "xent_train_f32", 2048, 32003, 512, "f32", "i64", 0.9, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_train", "norm_fwd", "norm_train", "xent_fwd",
                     "xent_train", "xent_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    ids = rng.choice(["i32", "i64"])
    d = rng.choice([_log_int(rng, 16, 1024), 8 * _log_int(rng, 2, 128)])
    if op.startswith("norm"):
        d = rng.choice([d, _log_int(rng, 16, 4096)])
        case = _norm(op, None, _log_int(rng, 1, min(100000, 65536 * 1024 // d)), d, dtype,
                     rng.choice(["none", "channel", "row"]), rng.random() < 0.5,
                     rng.choice([0.5, 0.7, 1.0]))
    elif op.startswith("embed"):
        case = _embed(op, None, _log_int(rng, 1, 65536), _log_int(rng, 100, 60000), d, dtype, ids,
                      rng.choice([0.0, 0.0, 0.1, 0.5]), rng.choice([1.0, math.sqrt(d)]))
    else:
        most = 3.7e12 if dtype == "bf16" else 2.0e11
        while True:
            case = _xent(op, None, _log_int(rng, 1, 16384), _log_int(rng, 100, 60000), d, dtype,
                         ids, rng.choice([1.0, 0.9, 0.15]), op == "xent_train" and
                         rng.random() < 0.3)
            if work(case)["flops"] <= most:
                break
    del case["name"]
    return case


def _distinct(vocab, n):
    """How many different ids n tokens have on average (log-uniform ids)."""
    k = np.arange(1, vocab + 1, dtype=np.float64)
    p = np.log1p(1 / k) / math.log(vocab + 1)
    return float((1 - np.exp(n * np.log1p(-np.minimum(p, 1 - 1e-12)))).sum())


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    d = case["d"]
    if case["op"].startswith("norm"):
        n, w = case["rows"] * d, d * es
        row, chan = case["gate"] == "row", case["gate"] == "channel"
        vectors = 2 + (2 if case["post"] else 0) + (1 if chan else 0)
        fwd = (4 + row) * n * es + vectors * w + (4 if case["post"] else 2) * 4 * case["rows"]
        if case["op"] == "norm_fwd":
            return {"bytes": fwd, "flops": (20 if case["post"] else 12) * n}
        # The step as one: R, B, the gate, dH, dY read; H, Y, dR, dB, the gate's gradient written.
        return {"bytes": fwd + (4 + row) * n * es + vectors * w,
                "flops": (50 if case["post"] else 32) * n}
    tokens, vocab = case["tokens"], case["vocab"]
    ib = 4 if case["ids"] == "i32" else 8
    if case["op"].startswith("embed"):
        live = tokens * (1 - case["padded"])
        fwd = tokens * ib + (_distinct(vocab, live) + tokens) * d * es
        if case["op"] == "embed_fwd":
            return {"bytes": fwd, "flops": tokens * d}
        return {"bytes": fwd + (live + vocab) * d * es, "flops": (tokens + live) * d}
    live = tokens * case["kept"]
    fwd = (live + vocab) * d * es + tokens * (ib + 8)
    if case["op"] == "xent_fwd":
        return {"bytes": fwd, "flops": 2 * live * vocab * d}
    tied = tokens * (ib + d * es) if case["tied"] else 0
    return {"bytes": fwd + (tokens + vocab) * d * es + tied, "flops": 6 * live * vocab * d}


def _tokens(g, n, vocab, kind):
    """Ids as frequent as a text's: the k-th in proportion to 1/k, in a random order of ids."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    k = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)
    # A step that shares no factor with the vocabulary spreads the frequent ids.
    step = vocab // 3 * 2 + 1
    while math.gcd(step, vocab) != 1:
        step += 1
    return (k * step % vocab).to(IDS[kind])


def _inputs(case, seed):
    """The case's inputs on the GPU."""
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t, d = TYPES[case["dtype"]], case["d"]
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    if case["op"].startswith("norm"):
        rows = case["rows"]
        # A residual stream: an offset, and a few channels much larger than the rest.
        r = randn(rows, d) * (0.5 + torch.rand((1, d), generator=g, device=dev))
        r[:, ::61] *= 12.0
        r += 0.4
        b = randn(rows, d) * 0.8 + 0.1
        s = dict(r=r.to(t), b=b.to(t), gamma=(1 + 0.2 * randn(d)).to(t),
                 beta=(0.1 * randn(d)).to(t), gate=None, pg=None, pb=None)
        if case["gate"] == "channel":
            s["gate"] = (0.3 + 0.2 * randn(d)).to(t)
        elif case["gate"] == "row":
            s["gate"] = torch.sigmoid(randn(rows, d)).to(t)
        if case["post"]:
            s["pg"], s["pb"] = (1 + 0.2 * randn(d)).to(t), (0.1 * randn(d)).to(t)
        if case["op"] == "norm_train":
            s["dh"], s["dy"] = randn(rows, d).to(t), randn(rows, d).to(t)
        return s
    tokens, vocab = case["tokens"], case["vocab"]
    ids = _tokens(g, tokens, vocab, case["ids"])
    if case["op"].startswith("embed"):
        # Padding at the ends of the batch's contexts.
        if case["padded"]:
            length = min(tokens, 512)
            at = torch.arange(tokens, device=dev) % length
            ids[at >= length - int(round(case["padded"] * length))] = -1
        s = dict(ids=ids, w=(0.02 * randn(vocab, d)).to(t))
        if case["op"] == "embed_train":
            s["dy"] = (1e-2 * randn(tokens, d)).to(t)
        return s
    # A normalised hidden state that points to its target by more or less: probabilities of the
    # target from 1/vocab to nearly one.
    w = randn(vocab, d) * (1.5 / math.sqrt(d))
    x = randn(tokens, d)
    pull = 10.0 * torch.rand((tokens, 1), generator=g, device=dev)
    x += (pull / 1.5 ** 2) * w[ids.long()]
    if case["kept"] < 1:
        drop = torch.rand(tokens, generator=g, device=dev) >= case["kept"]
        ids = torch.where(drop, torch.full_like(ids, -100), ids)
    s = dict(x=x.to(t), w=w.to(t), targets=ids)
    if case["op"] == "xent_train":
        # The mean over the tokens that have a target.
        s["dloss"] = 1.0 / (ids >= 0).sum().clamp(min=1).float()
    if case["tied"]:
        s["ids"] = _tokens(g, tokens, vocab, case["ids"])
        s["dy"] = (1e-4 * randn(tokens, d)).to(t)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import fft_circulant_attention_gb300 as cat
        if case["op"].startswith("norm"):
            s["plan"] = cat.ResNormPlan(case["rows"], case["d"], case["dtype"], eps=EPS,
                                        scale=case["scale"], post=case["post"])
        elif case["op"].startswith("embed"):
            s["plan"] = cat.EmbedPlan(case["tokens"], case["vocab"], case["d"], case["dtype"],
                                      scale=case["scale"])
        else:
            s["plan"] = cat.XentPlan(case["tokens"], case["vocab"], case["d"], case["dtype"],
                                     grad=case["op"] == "xent_train")
            if case["tied"]:
                s["embed"] = cat.EmbedPlan(case["tokens"], case["vocab"], case["d"], case["dtype"])
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    op, plan = s["case"]["op"], s["plan"]
    if op.startswith("norm"):
        h, y, stats = plan.forward(s["r"], s["b"], s["gate"], s["gamma"], s["beta"], s["pg"],
                                   s["pb"])
        if op == "norm_fwd":
            return h, y, stats
        grads = plan.backward(h, s["b"], s["gate"], s["gamma"], s["pg"], s["pb"], stats, s["dh"],
                              s["dy"])
        return (h, y, stats) + tuple(v for v in grads if v is not None)
    if op.startswith("embed"):
        y = plan.forward(s["ids"], s["w"])
        return y if op == "embed_fwd" else (y, plan.backward(s["ids"], s["dy"]))
    loss, lse = plan.forward(s["x"], s["w"], s["targets"])
    if op == "xent_fwd":
        return loss, lse
    dx, dw = plan.backward(s["x"], s["w"], s["targets"], lse, s["dloss"])
    if s["case"]["tied"]:
        s["embed"].backward(s["ids"], s["dy"], dW=dw, accumulate=True)
    return loss, lse, dx, dw


def _run_plain(s):
    op = s["case"]["op"]
    if op.startswith("norm"):
        return _plain_norm(s)
    if op.startswith("embed"):
        return _plain_embed(s)
    return _plain_xent(s)


def _plain_stats(x):
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
    return c * rstd, mean, rstd


def _plain_norm_bwd(g, xh, rstd):
    return rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))


def _plain_norm(s):
    case = s["case"]
    t, scale = s["r"].dtype, case["scale"]
    f = {k: v.float() for k, v in s.items() if torch.is_tensor(v)}
    u = f["b"]
    if case["post"]:
        bh, bmean, brstd = _plain_stats(u)
        u = bh * f["pg"] + f["pb"]
    gate = f.get("gate")
    su = scale * u
    h = f["r"] + (su if gate is None else gate * su)
    xh, mean, rstd = _plain_stats(h)
    y = xh * f["gamma"] + f["beta"]
    stats = [mean, rstd] + ([bmean, brstd] if case["post"] else [])
    out = (h.to(t), y.to(t), torch.cat(stats, -1).T.contiguous())
    if case["op"] == "norm_fwd":
        return out
    dy = f["dy"]
    dh = f["dh"] + _plain_norm_bwd(dy * f["gamma"], xh, rstd)
    du = scale * (dh if gate is None else gate * dh)
    db = _plain_norm_bwd(du * f["pg"], bh, brstd) if case["post"] else du
    grads = [dh, db]
    if gate is not None:
        grads.append(su * dh if case["gate"] == "row" else (su * dh).sum(0))
    grads += [(dy * xh).sum(0), dy.sum(0)]
    if case["post"]:
        grads += [(du * bh).sum(0), du.sum(0)]
    return out + tuple(v.to(t) for v in grads)


def _plain_embed(s):
    case, ids, w = s["case"], s["ids"].long(), s["w"]
    held = (ids >= 0)[:, None]
    at = ids.clamp(min=0)
    y = torch.where(held, case["scale"] * w[at].float(), 0.0).to(w.dtype)
    if case["op"] == "embed_fwd":
        return y
    dw = torch.zeros(w.shape, dtype=torch.float32, device=w.device)
    dw.index_add_(0, at, torch.where(held, case["scale"] * s["dy"].float(), 0.0))
    return y, dw.to(w.dtype)


def _plain_xent(s):
    case, x, targets = s["case"], s["x"], s["targets"].long()
    train, tokens = case["op"] == "xent_train", case["tokens"]
    w = s["w"].float()
    loss, lse = (torch.empty(tokens, dtype=torch.float32, device=w.device) for _ in range(2))
    if train:
        dx, dw = torch.empty_like(x), torch.zeros_like(w)
    step = max(1, PLAIN_BLOCK // case["vocab"])
    for a in range(0, tokens, step):
        rows = slice(a, min(tokens, a + step))
        xs, at = x[rows].float(), targets[rows]
        held, at = at >= 0, at.clamp(min=0)[:, None]
        p = torch.matmul(xs, w.T)
        hit = p.gather(1, at)[:, 0]
        top = p.amax(1, keepdim=True)
        p = torch.exp(p - top)
        total = p.sum(1, keepdim=True)
        z = (top + total.log())[:, 0]
        lse[rows] = torch.where(held, z, 0.0)
        loss[rows] = torch.where(held, z - hit, 0.0)
        if not train:
            continue
        p /= total
        p.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
        p *= (held * s["dloss"])[:, None]
        dx[rows] = torch.matmul(p, w).to(x.dtype)
        dw += torch.matmul(p.T, xs)
    if not train:
        return loss, lse
    if case["tied"]:
        dw.index_add_(0, s["ids"].long(), s["dy"].float())
    return loss, lse, dx, dw.to(x.dtype)


def exact(case, seed):
    """The outputs of ``run`` from the definitions, in 64 bits."""
    s = _inputs(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, s)
    if case["op"].startswith("embed"):
        held = s["ids"] >= 0
        y = torch.zeros((case["tokens"], case["d"]), dtype=torch.float64, device="cuda")
        y[held] = s["w"].double()[s["ids"][held].long()] * case["scale"]
        if case["op"] == "embed_fwd":
            return y
        return y, _exact_rows(case, s["ids"], s["dy"]) * case["scale"]
    return _exact_xent(case, s)


def _exact_rows(case, ids, dy):
    """Sums of the rows of each id, one block of columns at a time."""
    held = ids >= 0
    dw = torch.zeros((case["vocab"], case["d"]), dtype=torch.float64, device="cuda")
    dw.index_put_((ids[held].long(),), dy[held].double(), accumulate=True)
    return dw


def _exact_norm(case, s):
    d, k = case["d"], case["scale"]
    a = {n: v.double() for n, v in s.items() if v is not None}
    rows = a["r"].shape[0]

    def centred(x):
        m = x.sum(1) / d
        c = x - m[:, None]
        return m, c, 1 / torch.sqrt(torch.einsum("rd,rd->r", c, c) / d + EPS)

    def back(c, r, dout):
        """Through x -> c(x)·r(x): the centring and the variance by the chain rule."""
        dvar = -0.5 * r ** 3 * torch.einsum("rd,rd->r", dout, c)
        dc = dout * r[:, None] + (2.0 / d) * dvar[:, None] * c
        return dc - dc.sum(1, keepdim=True) / d

    u = a["b"]
    if case["post"]:
        mb, cb, rb = centred(u)
        u = cb * (rb[:, None] * a["pg"][None]) + a["pb"][None]
    gate = a["gate"].expand(rows, d) if "gate" in a else torch.ones_like(u)
    h = a["r"] + k * gate * u
    mh, ch, rh = centred(h)
    y = ch * (rh[:, None] * a["gamma"][None]) + a["beta"][None]
    out = (h, y, torch.stack([mh, rh] + ([mb, rb] if case["post"] else [])))
    if case["op"] == "norm_fwd":
        return out
    dh = a["dh"] + back(ch, rh, a["dy"] * a["gamma"][None])
    du = dh * gate * k
    db = back(cb, rb, du * a["pg"][None]) if case["post"] else du
    grads = [dh, db]
    if case["gate"] == "row":
        grads.append(dh * u * k)
    elif case["gate"] == "channel":
        grads.append(torch.einsum("rd,rd->d", dh, u) * k)
    grads += [torch.einsum("rd,rd,r->d", a["dy"], ch, rh), a["dy"].sum(0)]
    if case["post"]:
        grads += [torch.einsum("rd,rd,r->d", du, cb, rb), du.sum(0)]
    return out + tuple(grads)


def _exact_xent(case, s):
    """One block of the tokens that have a target at a time."""
    vocab, train = case["vocab"], case["op"] == "xent_train"
    held = torch.nonzero(s["targets"] >= 0)[:, 0]
    w = s["w"].double()
    loss, lse = (torch.zeros(case["tokens"], dtype=torch.float64, device="cuda") for _ in "ab")
    dx, dw = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda"), torch.zeros_like(w)
    step = max(1, EXACT_BLOCK // vocab)
    for at in held.split(step):
        x, t = s["x"][at].double(), s["targets"][at].long()
        logits = x @ w.T
        z = torch.logsumexp(logits, 1)
        lse[at] = z
        loss[at] = z - (x * w[t]).sum(1)
        if train:
            q = torch.exp(logits - z[:, None])
            q[torch.arange(len(t), device=q.device), t] -= 1
            q *= s["dloss"].double()
            dx[at] = q @ w
            dw += q.T @ x
    if not train:
        return loss, lse
    if case["tied"]:
        dw += _exact_rows(case, s["ids"], s["dy"])
    return loss, lse, dx, dw
