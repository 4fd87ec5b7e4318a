"""The references of the training step's operators agree with autograd and with
differences of their own forwards (CPU, 64 bits)."""
import pytest
import torch

import _step_ref as ref


def _g(seed):
    return torch.Generator().manual_seed(seed)


def differences(f, x, direction, step=1e-5):
    return (f(x + step * direction) - f(x - step * direction)) / (2 * step)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
def test_resnorm_gradients(gate, post):
    g = _g(3)
    rows, D, scale, eps = 5, 12, 0.7, 1e-5
    mk = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    t = dict(r=mk(rows, D), b=mk(rows, D), gamma=mk(D), beta=mk(D), gate=None, pg=None, pb=None)
    if gate != "none":
        t["gate"] = mk(D) if gate == "channel" else mk(rows, D)
    if post:
        t["pg"], t["pb"] = mk(D), mk(D)
    uh, uy = mk(rows, D), mk(rows, D)

    def loss(**k):
        a = {**t, **k}
        o = ref.resnorm_forward(a["r"], a["b"], a["gate"], a["gamma"], a["beta"], a["pg"],
                                a["pb"], post, eps, scale, "f32")
        return (o["h"][0] * uh).sum() + (o["y"][0] * uy).sum()

    o = ref.resnorm_forward(t["r"], t["b"], t["gate"], t["gamma"], t["beta"], t["pg"], t["pb"],
                            post, eps, scale, "f32")
    got = ref.resnorm_backward(o["h"][0], t["b"], t["gate"], t["gamma"], t["pg"], t["pb"],
                               o["stats"][0], uh, uy, post, scale, "f32")
    for name, v in t.items():
        if v is None:
            continue
        grad = got["d" + name][0].reshape(v.shape)
        leaf = v.clone().requires_grad_()
        loss(**{name: leaf}).backward()
        assert torch.allclose(leaf.grad, grad, rtol=1e-9, atol=1e-9), name
        way = mk(*v.shape)
        want = differences(lambda x: loss(**{name: x}), v, way)
        assert abs(float(want - (grad * way).sum())) <= 1e-6 * (1 + abs(float(want))), name


def test_xent_gradients():
    g = _g(4)
    T, V, D = 7, 33, 6
    x, w = (torch.randn(n, D, generator=g, dtype=torch.float64) for n in (T, V))
    targets = torch.tensor([0, 32, -100, 5, 5, -1, 17])
    up = torch.randn(T, generator=g, dtype=torch.float64)
    loss = lambda a, b: (ref.xent_forward(a, b, targets)["loss"][0] * up).sum()  # noqa: E731
    out = ref.xent_forward(x, w, targets)
    got, _, _ = ref.xent_backward(x, w, targets, out["lse"][0], up, "f32")
    a, b = x.clone().requires_grad_(), w.clone().requires_grad_()
    t = torch.where(targets < 0, torch.full_like(targets, -100), targets)
    want = torch.nn.functional.cross_entropy(a @ b.T, t, reduction="none")
    assert torch.allclose(out["loss"][0], want.detach(), rtol=1e-12, atol=1e-12)
    (want * up).sum().backward()
    assert torch.allclose(got["dx"][0], a.grad, rtol=1e-10, atol=1e-12)
    assert torch.allclose(got["dw"][0], b.grad, rtol=1e-10, atol=1e-12)
    for name, v, f in (("dx", x, lambda q: loss(q, w)), ("dw", w, lambda q: loss(x, q))):
        way = torch.randn(*v.shape, generator=g, dtype=torch.float64)
        d = float(differences(f, v, way))
        assert abs(d - float((got[name][0] * way).sum())) <= 1e-7 * (1 + abs(d)), name


def test_embed_gradient():
    g = _g(5)
    ids = torch.tensor([[3, 0, -1], [3, 3, 9]])
    w = torch.randn(10, 4, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(2, 3, 4, generator=g, dtype=torch.float64)
    y = 1.5 * torch.nn.functional.embedding(ids.clamp(min=0), w) * (ids >= 0)[..., None]
    assert torch.equal(y.detach(), ref.embed_forward(ids, w.detach(), 1.5, "f32")[0])
    (y * dy).sum().backward()
    got = ref.embed_backward(ids, dy, 10, 1.5, "f32")[0]
    assert torch.allclose(got, w.grad, rtol=1e-12, atol=1e-12)
    base = torch.randn(10, 4, generator=g, dtype=torch.float64)
    more = ref.embed_backward(ids, dy, 10, 1.5, "f32", base)[0]
    assert torch.allclose(more, w.grad + base, rtol=1e-12, atol=1e-12)
