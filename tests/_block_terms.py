"""The attention backward in 64 bits from given o and lse, with P and dS rounded
as the tensor-core kernels round them, and the relative error of a result that is
otherwise exact: what one bf16 term of dS costs against two."""
import math

import torch


def bf16(x):
    return x.float().bfloat16().double()


def one_term(x):
    return bf16(x)


def two_terms(x):
    a = bf16(x)
    return a + bf16(x - a)


def exact(x):
    return x


def forward(q, k, v, causal):
    """o in the inputs' type and lse in fp32, each rounded once from 64 bits."""
    T, hq, dh = q.shape
    o, lse = torch.empty_like(q), torch.empty((hq, T))
    for h in range(hq):
        g = h * k.shape[1] // hq
        s = dh ** -0.5 * (q[:, h].double() @ k[:, g].double().T)
        if causal:
            s = s.masked_fill(~torch.ones((T, T), dtype=torch.bool).tril(), -math.inf)
        lse[h] = torch.logsumexp(s, 1).float()
        o[:, h] = (torch.softmax(s, 1) @ v[:, g].double()).to(o.dtype)
    return o, lse


def backward(q, k, v, do, o, lse, causal, of_p=exact, of_ds=exact):
    """(dq, dk, dv) of one sequence."""
    T, hq, dh = q.shape
    q, k, v, do, o, lse = (t.double() for t in (q, k, v, do, o, lse))
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for h in range(hq):
        g = h * k.shape[1] // hq
        p = torch.exp(dh ** -0.5 * (q[:, h] @ k[:, g].T) - lse[h][:, None])
        if causal:
            p = p.tril()
        ds = of_ds(p * (do[:, h] @ v[:, g].T - (do[:, h] * o[:, h]).sum(1, keepdim=True)))
        dq[:, h] = dh ** -0.5 * (ds @ k[:, g])
        dk[:, g] += dh ** -0.5 * (ds.T @ q[:, h])
        dv[:, g] += of_p(p).T @ do[:, h]
    return dq, dk, dv


def error(a, b):
    """The root mean square of a - b relative to b's."""
    return float((a.double() - b).norm() / b.norm())


# A result rounded once to bf16 is off by some 0.0017 (a half step of 2^-8 at the
# most).  With two terms of dS (2^-16) dq and dk are no further off; with one they
# are by 1.4 times, as the roundings of its many terms add up in squares.  The
# limit lies between; fp32 sums of a few hundred terms are 2^-20 and do not count.
LIMIT = 1.15
CASES = [(400, 4, 2, 64, True), (400, 4, 2, 64, False), (700, 2, 1, 128, True),
         (300, 2, 2, 40, True)]
