"""64-bit references of the rest of a language model's training step (embedding,
residual addition with its norms, cross entropy over a vocabulary), with
elementwise error bounds counted in rounding steps.

Half a step relative to the value: H for fp32, U[dtype] for the storage type.
A sum of n terms in fp32 is off by at most n·H times the sum of their absolute
values; the tensor core's accumulator cuts instead of rounding, 2·H a term.
"""
import torch

from _block_ref import H, ROW_TERMS, TORCH, U

F64 = torch.float64


def rnd(g, *shape, scale=1.0, dtype="f32"):
    return (torch.randn(*shape, generator=g) * scale).to(TORCH[dtype])


# ------------------------------------------------------------------ embedding
def embed_forward(ids, w, scale, dtype):
    held = (ids >= 0) & (ids < w.shape[0])
    y = torch.zeros(tuple(ids.shape) + (w.shape[1],), dtype=F64)
    y[held] = w.double()[ids[held].long()] * scale
    return y, (U[dtype] + H) * y.abs()


def embed_backward(ids, dy, V, scale, dtype, base=None):
    held = (ids >= 0) & (ids < V)
    at, rows = ids[held].long(), dy[held].double() * scale
    dw = torch.zeros((V, dy.shape[-1]), dtype=F64).index_add_(0, at, rows)
    mass = torch.zeros_like(dw).index_add_(0, at, rows.abs())
    n = torch.bincount(at, minlength=V).double()[:, None]
    bound = (n + 2) * H * mass
    if base is not None:
        dw = torch.where(n > 0, dw + base.double(), base.double())
        bound = bound + H * dw.abs()
        return dw, torch.where(n > 0, bound + U[dtype] * dw.abs(), torch.zeros_like(dw))
    return dw, bound + U[dtype] * dw.abs()


# ------------------------------------------------- residual addition with norms
def _stats(x, ex, eps):
    """Centred values, rstd, x̂ and mean with the bounds of each, for x off by ex."""
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    var = (c * c).mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    e_mean = ROW_TERMS * H * x.abs().mean(-1, keepdim=True) + ex.mean(-1, keepdim=True) + \
        H * mean.abs()
    e_c = ex + e_mean + H * c.abs()
    e_var = (ROW_TERMS + 4) * H * var + (2 * c.abs() * e_c + e_c * e_c).mean(-1, keepdim=True)
    # (1 + t)^-1/2 is off by t/2 to first order; twice that covers t up to 1/2.
    rel = 0.5 * rstd ** 2 * e_var
    e_rstd = rstd * (rel * torch.where(rel < 0.02, 1.05, 2.0) + 4 * H)
    xh = c * rstd
    e_xh = e_c * rstd + c.abs() * e_rstd + e_c * e_rstd + 2 * H * xh.abs()
    return (mean, e_mean), (rstd, e_rstd), (xh, e_xh)


def resnorm_forward(r, b, gate, gamma, beta, pg, pb, post, eps, scale, dtype):
    """(h, y, stats) as pairs of value and bound."""
    u = U[dtype]
    d = lambda t, fill: torch.full((b.shape[-1],), fill, dtype=F64) if t is None else t.double()  # noqa: E731,E501
    r, b, gate, gamma, beta, pg, pb = (r.double(), b.double(), d(gate, 1.0), d(gamma, 1.0),
                                       d(beta, 0.0), d(pg, 1.0), d(pb, 0.0))
    stats = []
    x, ex = b, torch.zeros_like(b)
    if post:
        mb, rb, (bh, e_bh) = _stats(b, ex, eps)
        x = bh * pg + pb
        ex = e_bh * pg.abs() + 3 * H * ((bh * pg).abs() + pb.abs())
        stats = [mb, rb]
    k = scale * gate
    h = r + k * x
    eh = k.abs() * ex + 4 * H * ((k * x).abs() + r.abs())
    mh, rh, (xh, e_xh) = _stats(h, eh, eps)
    y = xh * gamma + beta
    e_y = e_xh * gamma.abs() + 3 * H * ((xh * gamma).abs() + beta.abs()) + u * y.abs()
    stats = [mh, rh] + stats
    pair = tuple(torch.stack([s[i][..., 0] for s in stats]) for i in (0, 1))
    return dict(h=(h, eh + u * h.abs()), y=(y, e_y), stats=pair)


def resnorm_backward(h, b, gate, gamma, pg, pb, stats, dh_up, dy, post, scale, dtype):
    """Gradients as pairs, from these very h, b and stats."""
    u, D = U[dtype], b.shape[-1]
    rows = b.numel() // D
    d = lambda t, fill: torch.full((D,), fill, dtype=F64) if t is None else t.double()  # noqa: E731
    per_row = gate is not None and gate.dim() > 1
    has_gate = gate is not None
    h, b, dy = (t.double().reshape(rows, D) for t in (h, b, dy))
    dh_up = torch.zeros_like(h) if dh_up is None else dh_up.double().reshape(rows, D)
    gate = gate.double().reshape(rows, D) if per_row else d(gate, 1.0)
    gamma, pg, pb = d(gamma, 1.0), d(pg, 1.0), d(pb, 0.0)
    stats = stats.double().reshape(stats.shape[0], rows, 1)

    def hat(x, mean, rstd):
        v = (x - mean) * rstd
        return v, 2.1 * H * v.abs()

    def through(w, e_w, xh, f_xh, rstd):
        """rstd·(w - mean(w) - x̂·mean(w·x̂))."""
        m1, m2 = w.mean(-1, keepdim=True), (w * xh).mean(-1, keepdim=True)
        t1 = e_w.mean(-1, keepdim=True) + (ROW_TERMS + 4) * H * w.abs().mean(-1, keepdim=True)
        t2 = (e_w * xh.abs() + w.abs() * f_xh).mean(-1, keepdim=True) + \
            (ROW_TERMS + 8) * H * (w * xh).abs().mean(-1, keepdim=True)
        v = rstd * (w - m1 - xh * m2)
        e = rstd * (e_w + 8 * H * (w.abs() + m1.abs() + (xh * m2).abs()) + t1 + xh.abs() * t2 +
                    f_xh * m2.abs())
        return v, e

    def column(v, e):
        total = v.sum(0)
        return total, e.sum(0) + (rows + 64) * H * v.abs().sum(0) + u * total.abs()

    xh, f_xh = hat(h, stats[0], stats[1])
    g = dy * gamma
    v, e = through(g, H * g.abs(), xh, f_xh, stats[1])
    dh = dh_up + v
    e_dh = e + 2 * H * (dh.abs() + dh_up.abs())
    out = dict(dr=(dh, e_dh + u * dh.abs()))
    x, ex = b, torch.zeros_like(b)
    if post:
        bh, f_bh = hat(b, stats[2], stats[3])
        x = bh * pg + pb
        ex = f_bh * pg.abs() + 2 * H * ((bh * pg).abs() + pb.abs())
    k = scale * gate
    du = k * dh
    e_du = k.abs() * e_dh + 3 * H * du.abs()
    if has_gate:
        q = scale * x * dh
        e_q = abs(scale) * (x.abs() * e_dh + dh.abs() * ex + e_dh * ex) + 3 * H * q.abs()
        out["dgate"] = (q, e_q + u * q.abs()) if per_row else column(q, e_q)
    if post:
        w = du * pg
        db, e_db = through(w, e_du * pg.abs() + H * w.abs(), bh, f_bh, stats[3])
        out["db"] = (db, e_db + u * db.abs())
        out["dpg"] = column(du * bh, e_du * bh.abs() + du.abs() * f_bh + H * (du * bh).abs())
        out["dpb"] = column(du, e_du)
    else:
        out["db"] = (du, e_du + u * du.abs())
    out["dgamma"] = column(dy * xh, dy.abs() * f_xh + H * (dy * xh).abs())
    out["dbeta"] = column(dy, torch.zeros_like(dy))
    return out


# --------------------------------------------------------------- cross entropy
def _logits(x, w):
    """The logits and their bounds: exact products of bf16 terms, accumulators
    that cut; fp32 operands are three terms, of whose nine products six are
    taken (the others and what three terms leave: 8·H)."""
    D = x.shape[1]
    return x @ w.T, (2 * D + 16) * H * (x.abs() @ w.abs().T)


def xent_forward(x, w, targets):
    """(loss, lse) as pairs; 0 where there is no target."""
    x, w = x.double(), w.double()
    V = w.shape[0]
    held = (targets >= 0) & (targets < V)
    l, el = _logits(x, w)
    z = torch.logsumexp(l, 1)
    p = torch.exp(l - z[:, None])
    # Each exponential: its argument's roundings and four steps of exp2; the sum:
    # at most this many terms one after another; the logarithm and the addition.
    chain = min(V, 1024 + V // 64) + 64
    top = l.amax(1, keepdim=True)
    e_z = (p * (el + 4 * H * (l - top).abs())).sum(1) + (chain + 8) * H + \
        4 * H * z.abs() + 2 * H * (z - top[:, 0]).abs()
    at = targets.long().clamp(0, V - 1)[:, None]
    hit, e_hit = l.gather(1, at)[:, 0], el.gather(1, at)[:, 0]
    loss = z - hit
    zero = torch.zeros_like(z)
    pick = lambda t: torch.where(held, t, zero)  # noqa: E731
    return dict(loss=(pick(loss), pick(e_z + e_hit + 2 * H * (z.abs() + hit.abs()))),
                lse=(pick(z), pick(e_z)))


def xent_backward(x, w, targets, lse, dloss, dtype):
    """(dx, dw) as pairs, from this very lse; and for each the norm that fp32
    sums stay within: d's own errors (p - [v = t] cancels where p is near one, so
    they are not small beside d) meet at random, as do two half steps for each
    term of the sums; four standard deviations of these."""
    u = U[dtype]
    x, w = x.double(), w.double()
    V, T = w.shape[0], x.shape[0]
    held = (targets >= 0) & (targets < V)
    x = torch.where(held[:, None], x, torch.zeros_like(x))
    g = torch.where(held, dloss.double().expand(T), torch.zeros(T, dtype=F64))[:, None]
    z = torch.where(held, lse.double(), torch.zeros(T, dtype=F64))[:, None]
    l, el = _logits(x, w)
    p = torch.exp(l - z)
    ep = p * (el + 2 * H * (l.abs() + z.abs()) + 6 * H)
    hot = torch.zeros_like(p)
    hot[torch.arange(T)[held], targets[held].long()] = 1.0
    d = g * (p - hot)
    # d is an operand of the products: one rounding to bf16, or three bf16 terms.
    e_d = g.abs() * (ep + H * (p - hot).abs()) + (u + 3 * H) * d.abs()
    dx, dw = d @ w, d.T @ x
    m_dx, m_dw = d.abs() @ w.abs(), d.abs().T @ x.abs()
    b_dx = e_d @ w.abs() + (2 * V + 32) * H * m_dx + u * dx.abs()
    b_dw = e_d.T @ x.abs() + (2 * T + 32) * H * m_dw + u * dw.abs()
    n_dx = (e_d ** 2 @ w ** 2).sum().sqrt() + 8 * H * (V + 16) ** 0.5 * m_dx.norm()
    n_dw = ((e_d ** 2).T @ x ** 2).sum().sqrt() + 8 * H * (T + 16) ** 0.5 * m_dw.norm()
    return dict(dx=(dx, b_dx), dw=(dw, b_dw)), n_dx, n_dw
