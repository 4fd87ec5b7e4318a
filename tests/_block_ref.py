"""64-bit references of the operators around a CAT layer (softmax attention
over packed sequences, layer norm, gradient clipping), with elementwise error
bounds counted in rounding steps.

Half a step relative to the value: H for fp32, U[dtype] for the storage type.
A sum of n products accumulated in fp32 is off by at most (n + 1)·H times the
sum of the absolute products.
"""
import math

import torch

H = 2.0 ** -24
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def attn_inputs(lens, hq, hkv, dh, dtype, seed=0, extra=0, sharp=1.0):
    """q, k, v, dO on the CPU for these sequence lengths, `extra` rows behind."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + extra
    mk = lambda h, f=1.0: (torch.randn((T, h, dh), generator=g) * f).to(TORCH[dtype])  # noqa: E731
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return mk(hq, sharp), mk(hkv), mk(hkv), mk(hq), torch.tensor(cu, dtype=torch.int32)


def attention(q, k, v, do, cu, causal, dtype, scale=None, rounds=None):
    """Per output (o, lse, dq, dk, dv) the pair (value, bound), each fp64;
    rows outside the sequences are NaN (no value).  `rounds`: relative half
    step of the probabilities and of ds as the second products' operands
    (default: the storage type's, which both may be rounded to)."""
    T, hq, dh = q.shape
    hkv = k.shape[1]
    rep = hq // hkv
    scale = scale if scale is not None else 1 / math.sqrt(dh)
    u = U[dtype]
    up = u if rounds is None else rounds
    q, k, v, do = (t.double() for t in (q, k, v, do))
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.float64)  # noqa: E731
    o, lse, dq, dk, dv = nan(T, hq, dh), nan(hq, T), nan(T, hq, dh), nan(T, hkv, dh), nan(T, hkv, dh)
    bo, bl, bq, bk, bv = (torch.zeros_like(t) for t in (o, lse, dq, dk, dv))
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        n = b - a
        if n == 0:
            continue
        mask = torch.ones((n, n), dtype=torch.bool)
        if causal:
            mask = mask.tril()
        for t in (dk, dv):
            t[a:b] = 0.0
        for h in range(hq):
            g = h // rep
            Q, K, V, D = q[a:b, h], k[a:b, g], v[a:b, g], do[a:b, h]
            s = scale * (Q @ K.T)
            s = torch.where(mask, s, torch.tensor(-math.inf, dtype=torch.float64))
            L = torch.logsumexp(s, 1)
            p = torch.exp(s - L[:, None])
            out = p @ V
            # Scores: dh products, the scaling, the exponent's own roundings
            # (of s, of lse, and two steps of exp2).
            es = torch.where(mask, (dh + 4) * H * scale * (Q.abs() @ K.abs().T) +
                             4 * H * s.abs() + 4 * H, torch.zeros((), dtype=torch.float64))
            el = es.amax(1) + (n + 4) * H
            ep = es + el[:, None] + 2 * H * L.abs()[:, None]
            acc = (n + dh + 8) * H
            e_o = (p * (ep + up + acc)) @ V.abs() + u * out.abs()
            delta = (D * out).sum(1)
            e_d = (D.abs() * (e_o + acc * out.abs())).sum(1)
            dp = D @ V.T
            ds = p * (dp - delta[:, None])
            e_dp = acc * (D.abs() @ V.abs().T)
            # p moves by ep·p, the bracket by e_dp + e_d, and ds is rounded.
            e_s = p * (e_dp + e_d[:, None]) + (ep + up + 4 * H) * \
                p * (dp.abs() + delta.abs()[:, None])
            rows = slice(a, b)
            o[rows, h], lse[h, rows] = out, L
            bo[rows, h], bl[h, rows] = e_o, el + 2 * H * L.abs()
            dq[rows, h] = scale * (ds @ K)
            bq[rows, h] = scale * ((e_s + acc * ds.abs()) @ K.abs())
            dk[rows, g] += scale * (ds.T @ Q)
            # A key head's sums run over the rows of all its query heads.
            big = acc * rep
            bk[rows, g] += scale * ((e_s + big * ds.abs()).T @ Q.abs())
            dv[rows, g] += p.T @ D
            bv[rows, g] += (p * (ep + up + big)).T @ D.abs()
    bq += u * dq.abs().nan_to_num(0.0) + 2 * H * dq.abs().nan_to_num(0.0)
    bk += u * dk.abs().nan_to_num(0.0) + 2 * H * dk.abs().nan_to_num(0.0)
    bv += u * dv.abs().nan_to_num(0.0) + 2 * H * dv.abs().nan_to_num(0.0)
    return dict(o=(o, bo), lse=(lse, bl), dq=(dq, bq), dk=(dk, bk), dv=(dv, bv))


def check(name, got, ref, tiny=1e-30):
    """|got - value| <= bound wherever the reference has a value."""
    val, bound = ref
    g = got.detach().double().cpu()
    has = ~val.isnan()
    err = (g - val).abs()
    bad = has & ~(err <= bound + tiny)
    if bad.any():
        ratio = torch.where(has, err / (bound + tiny), torch.zeros_like(err)).nan_to_num(math.inf)
        i = int(ratio.argmax())
        raise AssertionError("%s: %d of %d values out of bounds; worst at flat %d: %r for %r, "
                             "bound %.3e" % (name, int(bad.sum()), int(has.sum()), i,
                                             g.flatten()[i].item(), val.flatten()[i].item(),
                                             bound.flatten()[i].item()))


# Terms that one thread or one tree of the layer norm's row sums adds up:
# 32 elements, five shuffles, eight warps, and the division.
ROW_TERMS = 48


def layernorm(x, gamma, beta, dy, eps, dtype):
    """Per output (y, mean, rstd, dx, dgamma, dbeta) the pair (value, bound).
    The backward's bounds hold for mean and rstd given as the fp32 roundings
    of their values."""
    u = U[dtype]
    D, rows = x.shape[-1], x.shape[0]
    x, dy = x.double(), dy.double()
    gm = gamma.double() if gamma is not None else torch.ones(D, dtype=torch.float64)
    bt = beta.double() if beta is not None else torch.zeros(D, dtype=torch.float64)
    mean = x.mean(-1)
    c = x - mean[:, None]
    var = (c * c).mean(-1)
    rstd = 1 / torch.sqrt(var + eps)
    xh = c * rstd[:, None]
    e_mean = ROW_TERMS * H * x.abs().mean(-1) + H * mean.abs()
    # The centred values carry the mean's error and a rounding; in the sum of
    # squares the mean's error enters squared.
    e_var = (ROW_TERMS + 4) * H * var + e_mean ** 2 + 2 * H * (c.abs() * x.abs()).mean(-1)
    e_rstd = 0.5 * rstd ** 3 * e_var + 4 * H * rstd
    e_c = e_mean[:, None] + H * c.abs()
    e_xh = e_c * rstd[:, None] + c.abs() * e_rstd[:, None] + H * xh.abs()
    y = xh * gm + bt
    e_y = e_xh * gm.abs() + 3 * H * ((xh * gm).abs() + bt.abs()) + u * y.abs()
    # Backward, from the rounded mean and rstd.
    f_xh = rstd[:, None] * (H * mean.abs()[:, None] + H * c.abs()) + 3 * H * xh.abs()
    g = dy * gm
    s1, s2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    t1 = (ROW_TERMS + 4) * H * g.abs().mean(-1, keepdim=True)
    t2 = (ROW_TERMS + 4) * H * (g * xh).abs().mean(-1, keepdim=True) + \
        (g.abs() * f_xh).mean(-1, keepdim=True)
    dx = rstd[:, None] * (g - s1 - xh * s2)
    e_dx = rstd[:, None] * (6 * H * (g.abs() + s1.abs() + (xh * s2).abs()) + t1 + xh.abs() * t2 +
                            f_xh * s2.abs()) + u * dx.abs()
    n = (rows + 64) * H
    dgamma, dbeta = (dy * xh).sum(0), dy.sum(0)
    e_dg = n * (dy * xh).abs().sum(0) + (dy.abs() * f_xh).sum(0) + u * dgamma.abs()
    e_db = n * dy.abs().sum(0) + u * dbeta.abs()
    return dict(y=(y, e_y), mean=(mean, e_mean), rstd=(rstd, e_rstd), dx=(dx, e_dx),
                dgamma=(dgamma, e_dg), dbeta=(dbeta, e_db))


def clip(grads, max_norm):
    """(norm, bound) and per tensor (value, bound)."""
    norm = math.sqrt(sum(float(a.double().pow(2).sum()) for a in grads))
    coef = min(1.0, max_norm / norm) if norm > 0 else 1.0
    # A thread adds at most 16 squares a chunk, a few chunks, then fp64: the
    # sum of squares is off by 64 H at most, its root by half of that.
    rel = 32 * H + 2 * H
    outs = []
    for a in grads:
        u = U["bf16" if a.dtype == torch.bfloat16 else "f32"]
        v = a.double() * coef
        outs.append((v, v.abs() * (rel + 2 * H + u)))
    return (torch.tensor(norm, dtype=torch.float64), torch.tensor(norm * rel)), outs
