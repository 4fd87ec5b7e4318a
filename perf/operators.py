"""Cases of the operators around a CAT layer in a training step: softmax
attention over packed sequences (the other layer of a CAT-Alter stack), layer
norm, and the global gradient norm with clipping.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` makes one pass (the framework's calls where ``own`` is true,
elementary torch operations in 32 bits otherwise), ``work`` counts the bytes
and operations of a pass and ``exact`` gives the outputs in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
# Scores of one block of the plain form and of the 64-bit one: elements held at once.
PLAIN_BLOCK = 1 << 30
EXACT_BLOCK = 1 << 26


def _attn(op, name, lens, hq, hkv, dh, dtype, causal, fused):
    return dict(name=name, op=op, lens=lens, hq=hq, hkv=hkv, dh=dh, dtype=dtype, causal=causal,
                fused=fused)


def _ragged(count, longest, seed):
    """`count` lengths up to `longest`, the first of them that long, as text."""
    import random
    r = random.Random(seed)
    n = [longest] + [max(1, int(longest * r.random())) for _ in range(count - 1)]
    return ",".join(str(v) for v in n)


def listed():
    return [
        # One short prompt beside a single token and a few: what a call costs at the least.
        _attn("attn_fwd", "attn_fwd_tiny", "1,17,64", 2, 1, 32, "bf16", True, False),
        # GPT-2-small width, sixteen packed documents up to its 1024 tokens, q, k and v as
        # columns of one projection's output.
        _attn("attn_fwd", "attn_fwd_gpt2", _ragged(16, 1024, 1), 12, 12, 64, "bf16", True, True),
        # The long-sequence workload's width with grouped heads: two whole contexts and a rest.
        _attn("attn_fwd", "attn_fwd_long16k", "16384,16384,4999", 16, 4, 64, "bf16", True, False),
        # ViT patches, not causal, 32-bit storage.
        _attn("attn_fwd", "attn_fwd_vit196_f32", ",".join(["196"] * 64), 6, 6, 64, "f32", False,
              False),
        # The attention layer of one training step at GPT-2-small width.
        _attn("attn_train", "attn_train_gpt2", _ragged(16, 1024, 2), 12, 12, 64, "bf16", True,
              True),
        # Wide heads, four query heads to a key head, documents of very different lengths.
        _attn("attn_train", "attn_train_grouped", "8192,4095,2049,1000,511,129,64,3,1", 16, 4, 128,
              "bf16", True, False),
        # A 32-bit training step, causal, few sequences.
        _attn("attn_train", "attn_train_f32", "1024,777,300,2", 12, 12, 64, "f32", True, False),
        # Layer norm in front of a tiny layer: one small call.
        dict(name="ln_fwd_tiny", op="ln_fwd", rows=256, d=64, dtype="f32"),
        # A training step's norm at GPT-2-small width over its sixteen contexts.
        dict(name="ln_train_gpt2", op="ln_train", rows=16384, d=768, dtype="bf16"),
        # The long-sequence workload's tokens and width, 32-bit storage.
        dict(name="ln_train_long_f32", op="ln_train", rows=65536, d=1024, dtype="f32"),
        # The gradients of one small CAT layer.
        dict(name="clip_layer", op="clip", layers=1, d=64, heads=2, vocab=0, dtype="f32",
             bound=0.5),
        # The gradients of a GPT-2-small-shaped CAT-Alter stack: bf16 matrices, 32-bit vectors.
        dict(name="clip_gpt2", op="clip", layers=12, d=768, heads=12, vocab=50257, dtype="bf16",
             bound=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_train", "attn_train", "ln_fwd", "ln_train",
                     "clip"])
    if op.startswith("attn"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        longest = {"attn_fwd": 16384, "attn_train": 8192}[op] if dtype == "bf16" else 2048
        flops = {"attn_fwd": 1.0e12, "attn_train": 7.0e11}[op] if dtype == "bf16" else 2.0e10
        while True:
            hkv = rng.choice([1, 2, 4, 6, 12])
            hq = hkv * rng.choice([1, 1, 2, 4])
            dh = rng.choice([16, 32, 64, 64, 80, 96, 128])
            top = _log_int(rng, 16, longest)
            count = _log_int(rng, 1, 64)
            lens = [max(1, int(top * rng.random())) for _ in range(count - 1)] + [top]
            case = _attn(op, None, ",".join(map(str, lens)), hq, hkv, dh, dtype,
                         rng.random() < 0.75, rng.random() < 0.5)
            del case["name"]
            w = work(case)
            if w["flops"] <= flops and w["bytes"] <= 6e8:
                return case
    if op.startswith("ln"):
        dtype = rng.choice(["bf16", "f32"])
        d = rng.choice([_log_int(rng, 16, 8192), 8 * _log_int(rng, 8, 1024)])
        most = 65536 * 1024 // d
        return dict(op=op, rows=_log_int(rng, 1, min(most, 100000)), d=d, dtype=dtype)
    heads = rng.choice([1, 2, 4, 6])
    d = heads * _log_int(rng, 5, 128)
    return dict(op="clip", layers=_log_int(rng, 1, 12), d=d, heads=heads,
                vocab=rng.choice([0, _log_int(rng, 100, 50257)]), dtype=rng.choice(["bf16", "f32"]),
                bound=rng.choice([0.1, 0.5, 1.0, 2.0]))


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def _shapes(case):
    """(shape, type) of every gradient of a CAT-Alter stack: matrices in the case's type,
    vectors in 32 bits."""
    d, h, t = case["d"], case["heads"], case["dtype"]
    out = [((case["vocab"], d), t)] if case["vocab"] else []
    for i in range(case["layers"]):
        out += [((d,), "f32")] * 4                          # two norms
        if i % 2 == 0:
            out += [((d, h), t), ((d, d), t)]               # CAT: scores and values
        else:
            out += [((d, 3 * d), t), ((3 * d,), "f32"), ((d, d), t), ((d,), "f32")]
        out += [((d, 2 * d), t), ((2 * d,), "f32"), ((2 * d, d), t), ((d,), "f32")]
    return out


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("attn"):
        lens, hq, hkv, dh = _lens(case), case["hq"], case["hkv"], case["dh"]
        tokens = sum(lens)
        pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
        nbytes = (2 * hq + 2 * hkv) * dh * tokens * es + 4 * hq * tokens
        flops = 4 * dh * hq * pairs
        if case["op"] == "attn_train":     # and dO read, dQ, dK, dV written; five products more
            nbytes += (2 * hq + 2 * hkv) * dh * tokens * es
            flops += 10 * dh * hq * pairs
        return {"bytes": nbytes, "flops": flops}
    if case["op"].startswith("ln"):
        n = case["rows"] * case["d"]
        if case["op"] == "ln_fwd":
            return {"bytes": 2 * n * es + 8 * case["rows"] + 2 * case["d"] * es, "flops": 8 * n}
        return {"bytes": 4 * n * es + 8 * case["rows"] + 4 * case["d"] * es, "flops": 19 * n}
    total = [(math.prod(s), 2 if t == "bf16" else 4) for s, t in _shapes(case)]
    return {"bytes": 2 * sum(n * e for n, e in total) + 4, "flops": 3 * sum(n for n, _ in total)}


def _inputs(case, seed):
    """The case's inputs on the GPU."""
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = TYPES[case["dtype"]]
    if case["op"].startswith("attn"):
        lens, hq, hkv, dh = _lens(case), case["hq"], case["hkv"], case["dh"]
        tokens = sum(lens)
        # A projection's output: unit variance, heads of somewhat different sharpness.
        rows = torch.randn((tokens, hq + 2 * hkv, dh), generator=g, device=dev)
        rows[:, :hq] *= torch.linspace(0.7, 1.6, hq, device=dev)[None, :, None]
        rows = rows.to(t)
        q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        if not case["fused"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s = dict(q=q, k=k, v=v, cu=torch.tensor(cu, dtype=torch.int32, device=dev))
        if case["op"] == "attn_train":
            s["do"] = torch.randn((tokens, hq, dh), generator=g, device=dev).to(t)
        return s
    if case["op"].startswith("ln"):
        rows, d = case["rows"], case["d"]
        # A residual stream: a common offset, and a few channels much larger than the rest.
        x = torch.randn((rows, d), generator=g, device=dev)
        x *= 0.5 + torch.rand((1, d), generator=g, device=dev)
        x[:, ::61] *= 12.0
        x += 0.7
        s = dict(x=x.to(t), gamma=(1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(t),
                 beta=(0.1 * torch.randn(d, generator=g, device=dev)).to(t))
        if case["op"] == "ln_train":
            s["dy"] = torch.randn((rows, d), generator=g, device=dev).to(t)
        return s
    grads = []
    for shape, kind in _shapes(case):
        a = torch.randn(shape, generator=g, device=dev) * (1e-3 * math.exp(len(grads) % 5 - 2))
        grads.append(a.to(TYPES[kind]))
    # The gradients' norm to expect, so that a bound below one clips and one above does not.
    norm = math.sqrt(sum(math.prod(s) * (1e-3 * math.exp(i % 5 - 2)) ** 2
                         for i, (s, _) in enumerate(_shapes(case))))
    return dict(grads=grads, max_norm=case["bound"] * norm)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"].startswith("attn"):
        s["lens"] = _lens(case)
        if own:
            import fft_circulant_attention_gb300 as cat
            s["plan"] = cat.AttnPlan(sum(s["lens"]), len(s["lens"]), case["hq"], case["hkv"],
                                     case["dh"], case["dtype"], causal=case["causal"])
    elif case["op"].startswith("ln"):
        if own:
            import fft_circulant_attention_gb300 as cat
            s["plan"] = cat.LayerNormPlan(case["rows"], case["d"], case["dtype"], eps=EPS)
    else:
        # The clipped gradients: parts of one flat buffer for each type, one after the other.
        s["flat"], s["out"] = [], [None] * len(s["grads"])
        for t in TYPES.values():
            at = [i for i, a in enumerate(s["grads"]) if a.dtype == t]
            if not at:
                continue
            flat = torch.empty(sum(s["grads"][i].numel() for i in at), dtype=t, device="cuda")
            s["flat"].append(flat)
            pos = 0
            for i in at:
                a = s["grads"][i]
                s["out"][i] = flat[pos:pos + a.numel()].view(a.shape)
                pos += a.numel()
        if own:
            import fft_circulant_attention_gb300 as cat
            s["plan"] = cat.ClipPlan([a.numel() for a in s["grads"]],
                                     [a.dtype for a in s["grads"]])
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    op, plan = s["case"]["op"], s["plan"]
    if op == "attn_fwd":
        return plan.forward(s["q"], s["k"], s["v"], s["cu"])
    if op == "attn_train":
        o, lse = plan.forward(s["q"], s["k"], s["v"], s["cu"])
        grads = plan.backward(s["q"], s["k"], s["v"], o, lse, s["do"], s["cu"])
        return (o, lse) + tuple(grads)
    if op == "ln_fwd":
        return plan.forward(s["x"], s["gamma"], s["beta"])
    if op == "ln_train":
        y, mean, rstd = plan.forward(s["x"], s["gamma"], s["beta"])
        grads = plan.backward(s["x"], s["gamma"], mean, rstd, s["dy"])
        return (y, mean, rstd) + tuple(grads)
    norm = plan.clip(s["grads"], s["max_norm"], out=s["out"])
    return [norm] + s["flat"]


def _run_plain(s):
    op = s["case"]["op"]
    if op.startswith("attn"):
        return _plain_attn(s)
    if op.startswith("ln"):
        return _plain_ln(s)
    total = None
    for a in s["grads"]:
        v = a.float()
        part = (v * v).sum()
        total = part if total is None else total + part
    norm = total.sqrt()
    coef = torch.clamp(s["max_norm"] / norm, max=1.0)
    coef = torch.where(torch.isfinite(norm), coef, torch.ones_like(coef))
    for a, o in zip(s["grads"], s["out"]):
        o.copy_(a.float() * coef)
    return [norm] + s["flat"]


def _plain_attn(s):
    case = s["case"]
    hq, hkv, dh = case["hq"], case["hkv"], case["dh"]
    rep, scale, train = hq // hkv, 1.0 / math.sqrt(dh), case["op"] == "attn_train"
    q, k, v = s["q"], s["k"], s["v"]
    o, lse = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty(
        (hq, q.shape[0]), dtype=torch.float32, device=q.device)
    if train:
        dq, dk, dv = (torch.empty_like(a, memory_format=torch.contiguous_format)
                      for a in (q, k, v))
    at = 0
    for n in s["lens"]:
        rows = slice(at, at + n)
        at += n
        mask = None
        if case["causal"]:
            mask = torch.ones((n, n), dtype=torch.bool, device=q.device).tril()
        step = max(1, PLAIN_BLOCK // (n * n * rep))         # key heads at once
        for g0 in range(0, hkv, step):
            g1 = min(hkv, g0 + step)
            heads = slice(g0 * rep, g1 * rep)
            qs = q[rows, heads].float().transpose(0, 1)
            ks = k[rows, g0:g1].float().transpose(0, 1).repeat_interleave(rep, 0)
            vs = v[rows, g0:g1].float().transpose(0, 1).repeat_interleave(rep, 0)
            p = torch.matmul(qs, ks.transpose(1, 2)) * scale
            if mask is not None:
                p = p.masked_fill_(~mask, float("-inf"))
            top = p.amax(-1, keepdim=True)
            p = torch.exp(p - top)
            total = p.sum(-1, keepdim=True)
            p = p / total
            out = torch.matmul(p, vs)
            o[rows, heads] = out.transpose(0, 1).to(o.dtype)
            lse[heads, rows] = (top + total.log()).squeeze(-1)
            if not train:
                continue
            ds = s["do"][rows, heads].float().transpose(0, 1)
            dvs = torch.matmul(p.transpose(1, 2), ds)
            dp = torch.matmul(ds, vs.transpose(1, 2))
            dp = p * (dp - (ds * out).sum(-1, keepdim=True)) * scale
            dq[rows, heads] = torch.matmul(dp, ks).transpose(0, 1).to(dq.dtype)
            dks = torch.matmul(dp.transpose(1, 2), qs)
            dk[rows, g0:g1] = dks.view(g1 - g0, rep, n, dh).sum(1).transpose(0, 1).to(dk.dtype)
            dv[rows, g0:g1] = dvs.view(g1 - g0, rep, n, dh).sum(1).transpose(0, 1).to(dv.dtype)
    return (o, lse, dq, dk, dv) if train else (o, lse)


def _plain_ln(s):
    x, t = s["x"].float(), s["x"].dtype
    gamma = s["gamma"].float()
    mean = x.mean(-1, keepdim=True)
    cent = x - mean
    rstd = torch.rsqrt((cent * cent).mean(-1, keepdim=True) + EPS)
    xh = cent * rstd
    y = (xh * gamma + s["beta"].float()).to(t)
    if s["case"]["op"] == "ln_fwd":
        return y, mean.squeeze(-1), rstd.squeeze(-1)
    dy = s["dy"].float()
    g = dy * gamma
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return (y, mean.squeeze(-1), rstd.squeeze(-1), dx.to(t), (dy * xh).sum(0).to(t),
            dy.sum(0).to(t))


def exact(case, seed):
    """The outputs of ``run`` from the definitions, in 64 bits."""
    s = _inputs(case, seed)
    if case["op"].startswith("attn"):
        return _exact_attn(case, s)
    if case["op"].startswith("ln"):
        x, gamma, beta = s["x"].double(), s["gamma"].double(), s["beta"].double()
        d = case["d"]
        mean = x.sum(1) / d
        var = ((x - mean[:, None]) ** 2).sum(1) / d
        rstd = 1 / torch.sqrt(var + EPS)
        y = (x - mean[:, None]) * (rstd[:, None] * gamma[None]) + beta[None]
        if case["op"] == "ln_fwd":
            return y, mean, rstd
        # dx by the chain rule through the mean and the variance.
        dy = s["dy"].double()
        c = x - mean[:, None]
        dc = dy * gamma[None] * rstd[:, None]
        dvar = -0.5 * rstd ** 3 * (dy * gamma[None] * c).sum(1)
        dc = dc + (2.0 / d) * dvar[:, None] * c
        dx = dc - dc.sum(1, keepdim=True) / d
        return y, mean, rstd, dx, torch.einsum("rd,rd,r->d", dy, c, rstd), dy.sum(0)
    norm = math.sqrt(sum(float(a.double().pow(2).sum()) for a in s["grads"]))
    coef = min(1.0, s["max_norm"] / norm)
    parts = ([a.double().flatten() * coef for a in s["grads"] if a.dtype == t]
             for t in TYPES.values())
    return [torch.tensor(norm, dtype=torch.float64)] + [torch.cat(p) for p in parts if p]


def _exact_attn(case, s):
    """One head and one block of query rows at a time, over the keys that the rows see."""
    hq, hkv, dh = case["hq"], case["hkv"], case["dh"]
    scale, train = dh ** -0.5, case["op"] == "attn_train"
    tokens, dev = s["q"].shape[0], s["q"].device
    new = lambda h: torch.zeros((h, tokens, dh), dtype=torch.float64, device=dev)  # noqa: E731
    q, k, v = (s[n].permute(1, 0, 2).double().contiguous() for n in "qkv")
    out, lse = new(hq), torch.zeros((hq, tokens), dtype=torch.float64, device=dev)
    if train:
        g, dq, dk, dv = s["do"].permute(1, 0, 2).double().contiguous(), new(hq), new(hkv), new(hkv)
    start = 0
    for n in _lens(case):
        block = max(1, min(n, EXACT_BLOCK // n))
        for h in range(hq):
            j = h * hkv // hq
            kk, vv = k[j, start:start + n], v[j, start:start + n]
            for r0 in range(0, n, block):
                r1 = min(n, r0 + block)
                seen = r1 if case["causal"] else n
                rows = slice(start + r0, start + r1)
                keys = slice(start, start + seen)
                a = scale * (q[h, rows] @ kk[:seen].T)
                if case["causal"]:
                    i = torch.arange(r0, r1, device=dev)[:, None]
                    a = torch.where(torch.arange(seen, device=dev)[None] <= i, a, -math.inf)
                z = torch.logsumexp(a, 1)
                w = torch.exp(a - z[:, None])
                out[h, rows] = w @ vv[:seen]
                lse[h, rows] = z
                if train:
                    u = g[h, rows] @ vv[:seen].T
                    u = w * (u - (w * u).sum(1, keepdim=True))
                    dq[h, rows] = scale * (u @ kk[:seen])
                    dk[j, keys] += scale * (u.T @ q[h, rows])
                    dv[j, keys] += w.T @ g[h, rows]
        start += n
    back = lambda a: a.permute(1, 0, 2).contiguous()  # noqa: E731
    return (back(out), lse) + ((back(dq), back(dk), back(dv)) if train else ())
