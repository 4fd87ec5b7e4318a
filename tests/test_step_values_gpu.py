"""GPU tests of the values that the training step's operators return where they are
easily lost: differences of large logits, infinities, sums over very many tokens."""
import math

import pytest
import torch

import fft_circulant_attention_gb300 as cat
import _step_ref as ref
from _block_ref import H, TORCH, U, check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _built(cuda_device):
    from fft_circulant_attention_gb300 import build
    build.build()
    cat.lib()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ embedding
def zipf(n, V, g):
    u = torch.rand(n, device=DEV, generator=g, dtype=torch.float64)
    return (torch.exp(u * math.log(V + 1)) - 1).long().clamp(0, V - 1)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V,D,kind", [
    (16385, 200, 16, "one"), (16385, 5000, 16, "zipf"), (50001, 3, 24, "zipf"),
    (50001, 60000, 16, "one"), (300001, 70, 8, "zipf"), (300001, 2, 16, "one"),
    (30000, 5000, 768, "zipf"), (40000, 900, 768, "padded"), (20001, 300, 1024, "zipf"),
    (20001, 40, 1000, "one"), (9000, 100, 513, "zipf"), (12000, 100, 8192, "zipf"),
    (12000, 7, 8192, "one"),
])
def test_embed_gradient_counts_every_token(n, V, D, kind, dtype, accumulate):
    # Gradients of small integers: sums in fp32 are exact in any order, below 2^24, so
    # that no part of a run that many pieces hold can be lost or counted twice.
    g = torch.Generator(DEV).manual_seed(n + D)
    ids = torch.full((n,), V - 1, device=DEV) if kind == "one" else zipf(n, V, g)
    if kind == "padded":
        ids[torch.rand(n, device=DEV, generator=g) < 0.3] = -1
    draw = lambda *shape: torch.randint(-8, 9, shape, device=DEV, generator=g)  # noqa: E731
    dy, base = draw(n, D), draw(V, D)
    held = ids >= 0
    want = torch.zeros((V, D), device=DEV, dtype=torch.float64)
    want.index_add_(0, ids[held], dy[held].double())
    want *= 2.0
    assert want.abs().max() < 2 ** 24
    there = torch.bincount(ids[held], minlength=V) > 0
    if accumulate:
        want += base
    with cat.EmbedPlan(n, V, D, dtype, scale=2.0) as plan:
        dw = plan.backward(ids, dy.to(TORCH[dtype]),
                           dW=base.to(TORCH[dtype]) if accumulate else None,
                           accumulate=accumulate)
        plan.sync()
    assert there.any() and torch.equal(dw, want.float().to(TORCH[dtype]))


# --------------------------------------------------------------- cross entropy
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,D", [(1, 8), (700, 64), (300, 33)])
def test_xent_of_a_single_id_is_zero(T, D, dtype):
    # One id has probability one, whatever its logit (up to some 100 here).
    g = gen(T)
    x = (torch.randn(T, D, generator=g) * 4).to(TORCH[dtype])
    w = torch.randn(1, D, generator=g).to(TORCH[dtype])
    with cat.XentPlan(T, 1, D, dtype) as plan:
        loss, lse = plan.forward(x.to(DEV), w.to(DEV), torch.zeros(T, dtype=torch.int64,
                                                                  device=DEV))
        assert (loss == 0).all()
        assert lse.abs().max() > 4


def separate_logits(T, V, dtype, seed):
    """Logits that the products make exactly: W's rows are powers of two in columns of
    their own.  Each row has its largest, 40 to 100, at its target or beside it, and
    others from close behind it to far below."""
    g = gen(seed)
    targets = torch.randint(0, V, (T,), generator=g)
    top = 0.5 * torch.randint(80, 201, (T, 1), generator=g).double()
    down = 0.5 * torch.randint(0, 60, (T, V), generator=g).double()
    logits = top - down.clamp(min=0.5) - 20 * (torch.rand(T, 1, generator=g) < 0.3)
    at = torch.where(torch.rand(T, generator=g) < 0.8, targets, (targets + 1) % V)
    logits[torch.arange(T), at] = top[:, 0]
    c = 2.0 ** (torch.arange(V) % 3 - 1).double()
    D = (V + 7) // 8 * 8
    x, w = torch.zeros(T, D, dtype=torch.float64), torch.zeros(V, D, dtype=torch.float64)
    x[:, :V] = logits / c
    w[torch.arange(V), torch.arange(V)] = c
    xt, wt = x.to(TORCH[dtype]), w.to(TORCH[dtype])
    assert torch.equal(xt.double(), x) and torch.equal(wt.double(), w)
    return xt, wt, targets, logits, c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(2000, 2), (2000, 8), (500, 40), (500, 300)])
def test_xent_of_confident_tokens(T, V, dtype):
    # Where one logit rules its row the loss is a small difference of large numbers:
    # it keeps its own size's accuracy all the same, and is never negative.
    x, w, targets, l, c = separate_logits(T, V, dtype, V)
    with cat.XentPlan(T, V, x.shape[1], dtype) as plan:
        ins = [t.to(DEV) for t in (x, w, targets)]
        loss, lse = plan.forward(*ins)
        dx, _ = plan.backward(*ins, lse, torch.ones((), device=DEV))
        plan.sync()
    z = torch.logsumexp(l, 1)
    down = l.amax(1, keepdim=True) - l
    p = torch.exp(l - z[:, None])
    # An exponential: its argument's factor and product are off by half a step each, the
    # function by four; so is each of at most four scalings of a part's sum.  The sum:
    # half a step for each addition one after another.  The logarithm two half steps.
    e = torch.where(down > 0, p * (2 * down + 20) * H, torch.zeros_like(p)).sum(1) + \
        (min(V, 32 + V // 64) + 4) * H
    hit = l.gather(1, targets[:, None])[:, 0]
    want = z - hit
    e = e + 2 * H * (z - l.amax(1))
    assert (loss >= 0).all()
    check("loss", loss, (want, e + H * want))
    check("lse", lse, (z, e + H * z.abs()))
    # The gradients, from this very lse: l - lse and its product are off by three half
    # steps, p by four; d and the result are rounded to the storage type.
    z = lse.double().cpu()[:, None]
    p = torch.exp(l - z)
    hot = torch.zeros_like(p)
    hot[torch.arange(T), targets] = 1.0
    d = p - hot
    e = p * (3 * (l - z).abs() + 4) * H + (4 * H + (2.1 * U[dtype] if dtype == "bf16" else 0)) * \
        d.abs()
    check("dx", dx[:, :V], (d * c, e * c))


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 64), ("bf16", 36)])
def test_xent_infinite_weights(dtype, D):
    # Logits of plus and minus infinity, and NaN where an infinity meets a zero: loss and
    # lse are what the definition makes of them.
    T, V = 400, 700
    g = gen(D)
    x = torch.randn(T, D, generator=g).to(TORCH[dtype])
    w = (0.2 * torch.randn(V, D, generator=g)).to(TORCH[dtype])
    targets = torch.randint(0, V, (T,), generator=g)
    sign = torch.randint(-1, 2, (T, 3), generator=g)
    sign[:200] = torch.tensor([-1, 1, -1])             # (all three are minus infinity)
    x[:, :3] = sign.to(x.dtype) * x[:, :3].abs().clamp(min=0.1)
    odd = {5: math.inf, 130: -math.inf, 699: math.inf}
    for k, (v, value) in enumerate(odd.items()):
        w[v, k] = value
        targets[201 + k] = targets[k] = v
    with cat.XentPlan(T, V, D, dtype) as plan:
        loss, lse = (t.cpu() for t in plan.forward(*(t.to(DEV) for t in (x, w, targets))))
        plan.sync()
    l = (x.double()[:, None] * w.double()).sum(-1)
    z = torch.logsumexp(l, 1)
    want = z - l.gather(1, targets[:, None])[:, 0]
    kinds = lambda t: (t.isnan(), t == math.inf, t == -math.inf)  # noqa: E731
    for a, b in zip(kinds(z) + kinds(want), kinds(lse) + kinds(loss)):
        assert torch.equal(a, b)
    assert z[:200].isfinite().all()
    assert (z == math.inf).any() and z.isnan().any() and (want[:3] == math.inf).all()
    keep = [v for v in range(V) if v not in odd]
    rows = torch.arange(3, 200)
    rows = rows[torch.isin(targets[rows], torch.tensor(keep))]
    assert len(rows) > 150 and want[rows].isfinite().all()
    new = torch.zeros(V, dtype=torch.int64)
    new[keep] = torch.arange(len(keep))
    for n, v in ref.xent_forward(x[rows], w[keep], new[targets[rows]]).items():
        check(n, dict(loss=loss, lse=lse)[n][rows], v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_xent_infinite_hidden_states_stay_in_their_tokens(dtype):
    T, V, D = 300, 500, 64
    g = gen(3)
    x = torch.randn(T, D, generator=g).to(TORCH[dtype])
    w = (0.2 * torch.randn(V, D, generator=g)).to(TORCH[dtype])
    targets = torch.randint(0, V, (T,), generator=g)
    bad = [7, 140, 299]
    dirty = x.clone()
    for i in bad:
        dirty[i, i % D] = math.inf
    other = [i for i in range(T) if i not in bad]
    one = torch.ones((), device=DEV)
    with cat.XentPlan(T, V, D, dtype) as plan:
        wd, td = w.to(DEV), targets.to(DEV)
        got = []
        for v in (x, dirty):
            v = v.to(DEV)
            loss, lse = plan.forward(v, wd, td)
            got.append((loss, lse, plan.backward(v, wd, td, lse, one)[0]))
        plan.sync()
    for a, b in zip(*got):
        assert torch.equal(a[other], b[other])
    loss, lse, dx = got[1]
    assert (lse[bad] == math.inf).all()
    for i in bad:
        up = float(w[targets[i], i % D]) > 0
        assert loss[i].isnan() if up else loss[i] == math.inf
        assert not dx[i].isfinite().any()


@pytest.mark.parametrize("T", [65536, 600000])
def test_xent_weights_gradient_over_many_tokens_has_no_drift(T):
    # bf16 sums run in an accumulator that cuts instead of rounding: of summands of one
    # sign it loses up to a step (2^-23) twice for every 16 of them, 4096 times before
    # it is read out, far below half a step of the result however many tokens there are.
    V, D = 40, 72
    g = torch.Generator(DEV).manual_seed(T)
    x = (0.5 + torch.rand(T, D, device=DEV, generator=g)).bfloat16()
    w = (0.05 * torch.randn(V, D, device=DEV, generator=g)).bfloat16()
    t = torch.zeros(T, dtype=torch.int64, device=DEV)
    with cat.XentPlan(T, V, D, "bf16") as plan:
        _, lse = plan.forward(x, w, t)
        _, dw = plan.backward(x, w, t, lse, torch.ones((), device=DEV), dX=False)
        plan.sync()
    d = torch.exp(x.double() @ w.double().T - lse.double()[:, None])
    d[:, 0] -= 1
    want = d.float().bfloat16().double().T @ x.double()
    off = (dw.double() - want) / want
    drift = 2 * 4096 * 2.0 ** -23
    assert off.abs().max() <= U["bf16"] + drift
    # (The results' own rounding goes both ways; four standard deviations of its mean.)
    assert off[1:].mean().abs() <= drift + 4 * 0.42 * U["bf16"] / (39 * 72) ** 0.5


def spoiled(t, rows):
    """Rows with infinities of one and of both signs, NaN, both, and values whose
    products overflow, in the first, the last and other places."""
    inf, nan = math.inf, math.nan
    kinds = ({0: inf}, {0: inf, -1: inf}, {20: -inf}, {7: inf, -1: -inf}, {-1: nan},
             {0: nan, 150: -inf}, {5: 1e30, -1: 1e30}, {5: -1e30})
    for r, kind in zip(rows, kinds):
        for k, value in kind.items():
            t[r, k] = value
    return t


def test_xent_f32_logits_that_are_not_finite():
    # Each kind of row of X meets each of W: their logits are those of the definition.
    T, V, D = 130, 300, 300
    g = gen(21)
    xs, ws = [0, 3, 31, 32, 77, 100, 128, 129], [0, 63, 64, 128, 191, 200, 298, 299]
    x = spoiled(torch.randn(T, D, generator=g), xs)
    w = spoiled(0.2 * torch.randn(V, D, generator=g), ws)
    w[63, 20] = 0.0
    l = (x.double()[:, None] * w.double()).sum(-1)
    l = torch.where(l.abs() > 3.4e38, l * math.inf, l)
    x, target = x.to(DEV), torch.zeros(T, dtype=torch.int64, device=DEV)

    def agrees(rows, logits):
        with cat.XentPlan(T, len(rows), D, "f32") as plan:
            lse = plan.forward(x, rows.to(DEV), target)[1].cpu()
            plan.sync()
        want = torch.logsumexp(logits, 1)
        assert torch.equal(lse.isnan(), want.isnan())
        assert torch.equal(lse.isinf(), want.isinf()) and torch.equal(lse > 0, want > 0)

    # Each row of W alone with an ordinary one, then all of a tile, without those that
    # hold NaN and with them.
    for v in ws:
        agrees(w[[v, 1]], l[:, [v, 1]])
    part = [v for v in range(V) if v not in ws[4:6]]
    agrees(w[part], l[:, part])
    agrees(w, l)


@pytest.mark.parametrize("where", ["x", "w", "ruled out"])
def test_xent_f32_of_values_that_are_not_finite_takes_no_age(where):
    # Training that has diverged (NaN everywhere), or ids ruled out by the thousand: no
    # sum of its own for every logit (50 and 100 times the clean call; 5 to 7 without).
    T, V, D = 512, 4096, 512
    g = torch.Generator(DEV).manual_seed(22)
    x, w = (torch.randn(n, D, device=DEV, generator=g) for n in (T, V))
    w *= 0.05
    targets = torch.randint(0, V, (T,), device=DEV, generator=g) // 2 * 2
    x[:, 0], w[:, 0] = 1.0, 0.0
    dirty = dict(x=x, w=w)
    if where == "ruled out":
        dirty["w"] = w.clone()
        dirty["w"][1::2, 0] = -math.inf
    else:
        dirty[where] = torch.full_like(dirty[where], math.nan)
    with cat.XentPlan(T, V, D, "f32") as plan, cat.XentPlan(T, V // 2, D, "f32") as half:
        def took(x, w):
            times = []
            for _ in range(5):
                a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
                a.record()
                lse = plan.forward(x, w, targets)[1]
                b.record()
                b.synchronize()
                times.append(a.elapsed_time(b))
            plan.sync()
            return sorted(times)[2], lse
        clean, _ = took(x, w)
        spoilt, lse = took(**dirty)
        if where == "ruled out":
            want = half.forward(x, w[::2].contiguous(), targets // 2)[1]
            assert torch.allclose(lse, want, rtol=1e-6)
        else:
            assert lse.isnan().all()
        assert spoilt <= 25 * clean, (spoilt, clean)


def test_xent_workspace_of_a_plan_for_the_loss_alone():
    # The rows of X once more, three words a token, and the parts of the longest call.
    T, V, D = 131072, 128256, 64
    with cat.XentPlan(T, V, D, "bf16", grad=False) as plan:
        size = int(plan.describe().split("workspace=")[1].split()[0])
    assert size <= T * (2 * D + 3 * 4) + 40 * 10 ** 6, size


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_xent_calls_of_any_length_in_one_plan(dtype):
    # As each in a plan of its own, and the largest plan's rows never run into each other.
    T, V, D = 20000, 3000, 16
    g = gen(23)
    x, w = torch.randn(T, D, generator=g).to(TORCH[dtype]).to(DEV), \
        torch.randn(V, D, generator=g).to(TORCH[dtype]).to(DEV)
    t = torch.randint(0, V, (T,), generator=g).to(DEV)
    with cat.XentPlan(T, V, D, dtype, grad=False) as plan:
        for n in (20000, 1, 31, 257, 1300, 5000, 9999, 19999):
            with cat.XentPlan(n, V, D, dtype, grad=False) as own:
                a, b = plan.forward(x[:n], w, t[:n]), own.forward(x[:n], w, t[:n])
                own.sync()
            assert all(torch.equal(p, q) for p, q in zip(a, b)), n
        plan.sync()


@pytest.mark.parametrize("each", [False, True])
@pytest.mark.parametrize("T,V,D,kept", [(300, 2500, 256, 1.0), (1000, 777, 96, 0.9),
                                        (2100, 9001, 64, 0.3), (40, 5000, 768, 1.0),
                                        (65537, 300, 40, 1.0), (140000, 40, 200, 0.9),
                                        (65600, 300, 64, 0.01), (70001, 40, 64, 0.0)])
def test_xent_bf16_gradients_round_twice(T, V, D, kept, each):
    # d once and each result once, to the nearest, all else in fp32: the error's norm is
    # that of these two roundings made in 64 bits (the products' own errors, about 2^-20
    # of the values, turn a rounding round now and then: a twentieth more).
    g = gen(T)
    x = torch.randn(T, D, generator=g).bfloat16()
    w = (2 / math.sqrt(D) * torch.randn(V, D, generator=g)).bfloat16()
    targets = torch.randint(0, V, (T,), generator=g)
    targets[torch.rand(T, generator=g) >= kept] = -1
    up = torch.rand(T if each else (), generator=g) + 0.1
    with cat.XentPlan(T, V, D, "bf16") as plan:
        ins = [t.to(DEV) for t in (x, w, targets)]
        _, lse = plan.forward(*ins)
        got = plan.backward(*ins, lse, up.to(DEV))
        plan.sync()
    held = targets >= 0
    x, w, z = x.double()[held], w.double(), lse.double().cpu()[held]
    d = torch.exp(x @ w.T - z[:, None])
    d[torch.arange(len(d)), targets[held]] -= 1.0
    f = up.double()
    if each:
        d, f = d * f[held][:, None], torch.ones(())
    near = lambda t: t.float().bfloat16().double()  # noqa: E731
    dx = got[0].double().cpu()
    assert (dx[~held] == 0).all()
    for a, exact, twice in ((dx[held], f * (d @ w), near(f * (near(d) @ w))),
                            (got[1].double().cpu(), f * (d.T @ x), near(f * (near(d).T @ x)))):
        assert (a - exact).norm() <= 1.05 * (twice - exact).norm()
