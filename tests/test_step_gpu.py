"""GPU tests of the rest of a language model's training step: embedding, residual
addition with its norms, cross entropy over a vocabulary, each against a plain
64-bit implementation with bounds counted in rounding steps, and together."""
import math

import pytest
import torch

import fft_circulant_attention_gb300 as cat
import _step_ref as ref
from _block_ref import check

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


def dev(t):
    return None if t is None else t.to(DEV)


def graphed(step, *changing):
    """step's outputs replayed from a graph, after other values in between."""
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    kept = [t.clone() for t in changing]
    for t in changing:
        t.zero_()
    graph.replay()
    for t, k in zip(changing, kept):
        t.copy_(k)
    graph.replay()
    torch.cuda.synchronize()
    return held


# ------------------------------------------------------------------ embedding
def ids_of(kind, n, V, g):
    if kind == "one":
        return torch.full((n,), V - 1)
    if kind == "sorted":
        return torch.arange(n) % V
    if kind == "zipf":
        u = torch.rand(n, generator=g, dtype=torch.float64)
        return (torch.exp(u * math.log(V + 1)) - 1).long().clamp(0, V - 1)
    ids = torch.randint(0, V, (n,), generator=g)
    if kind == "padded":
        ids[torch.rand(n, generator=g) < 0.4] = -7
    return ids


def embed_parity(n, V, D, dtype, kind, wide=True, scale=1.25, seed=0, accumulate=False):
    g = gen(seed)
    ids = ids_of(kind, n, V, g).to(torch.int64 if wide else torch.int32)
    w, dy = ref.rnd(g, V, D, dtype=dtype), ref.rnd(g, n, D, dtype=dtype)
    base = ref.rnd(g, V, D, dtype=dtype) if accumulate else None
    with cat.EmbedPlan(n, V, D, dtype, scale=scale) as plan:
        y = plan.forward(dev(ids), dev(w))
        dw = plan.backward(dev(ids), dev(dy), dW=dev(base), accumulate=accumulate)
        plan.sync()
    check("y", y, ref.embed_forward(ids, w, scale, dtype))
    check("dw", dw, ref.embed_backward(ids, dy, V, scale, dtype, base))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 3, 8, 24, 64, 77, 100, 256, 513, 768, 1000, 1024, 2048, 2050,
                               4096, 8192])
def test_embed_widths(D, dtype):
    embed_parity(333, 50, D, dtype, "zipf", seed=D)


@pytest.mark.parametrize("dtype,wide", [("f32", False), ("bf16", True)])
@pytest.mark.parametrize("kind", ["zipf", "one", "sorted", "padded"])
@pytest.mark.parametrize("n,V", [(1, 1), (1, 50257), (2, 3), (31, 7), (1000, 1), (1023, 5000),
                                 (4096, 333), (16384, 1009), (16385, 200), (40000, 3),
                                 (50001, 60000)])
def test_embed_tokens(n, V, kind, dtype, wide):
    embed_parity(n, V, 16, dtype, kind, wide, seed=n + V)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V,D", [(5, 9, 40), (3000, 40, 64), (20000, 11, 24), (700, 3000, 33)])
def test_embed_adds_to_a_gradient(n, V, D, dtype):
    embed_parity(n, V, D, dtype, "padded", seed=n, accumulate=True)
    embed_parity(n, V, D, dtype, "one", seed=n + 1, accumulate=True)


def test_embed_many_tokens():
    # More tokens than blocks of the sort with a thread for each.
    embed_parity(300001, 70, 8, "f32", "zipf", seed=5)
    embed_parity(270000, 5000, 4, "bf16", "padded", False, seed=6, accumulate=True)


def test_embed_large_vocabulary():
    # More ids than one sorting CTA an SM takes at its largest share.
    embed_parity(3000, 400001, 8, "bf16", "padded", seed=2)
    embed_parity(3000, 400001, 4, "f32", "zipf", seed=3, accumulate=True)


def test_embed_values_and_padding():
    g = gen(1)
    ids = torch.tensor([4, -1, 2, 4, -100, 0], device=DEV)
    w = ref.rnd(g, 5, 32, dtype="bf16").to(DEV)
    w[2, 3], w[4, 1] = math.nan, math.inf
    dy = ref.rnd(g, 6, 32, dtype="bf16").to(DEV)
    dy[1] = math.nan                        # a row that no id has
    dy[4] = math.inf
    with cat.EmbedPlan(6, 5, 32, "bf16") as plan:
        y = plan.forward(ids, w)
        assert torch.equal(y[0], w[4]) and torch.equal(y[5], w[0])
        assert y[2, 3].isnan() and y[2, 4].isfinite()
        assert (y[1] == 0).all() and (y[4] == 0).all()
        dw = plan.backward(ids, dy)
        assert dw.isfinite().all() and (dw[[1, 3]] == 0).all()
        base = torch.full((5, 32), 3.0, dtype=torch.bfloat16, device=DEV)
        base[1, 0], base[3, 1] = math.nan, -0.0
        want = base.clone()
        plan.backward(ids, dy, dW=base, accumulate=True)
        for a, b in ((base[1], want[1]), (base[3], want[3])):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        plan.sync()


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_embed_ids_outside(kind):
    g = gen(2)
    ids = torch.tensor([1, 8, 2**31 - 1, 3], dtype=kind, device=DEV)
    if kind == torch.int64:
        ids[2] = 2**40 + 1                  # (1 in its low 32 bits)
    w = ref.rnd(g, 8, 16).to(DEV)
    dy = ref.rnd(g, 4, 16).to(DEV)
    with cat.EmbedPlan(4, 8, 16, "f32") as plan:
        for call in (lambda: plan.forward(ids, w), lambda: plan.backward(ids, dy)):
            out = call()
            with pytest.raises(cat.CatError) as e:
                plan.sync()
            assert e.value.status == cat.CAT_ERR_DEVICE_STATUS
            if out.shape[0] == 4:
                assert torch.equal(out[[0, 3]], w[[1, 3]]) and (out[1:3] == 0).all()
            else:
                assert torch.equal(out[[1, 3]], dy[[0, 3]])
                assert (out[[0, 2, 4, 5, 6, 7]] == 0).all()


def test_embed_no_tokens_and_shapes():
    g = gen(3)
    w = ref.rnd(g, 6, 8).to(DEV)
    with cat.EmbedPlan(12, 6, 8, "f32") as plan:
        none = torch.empty((0,), dtype=torch.int64, device=DEV)
        assert plan.forward(none, w).shape == (0, 8)
        full = torch.ones_like(w)
        plan.backward(none, torch.empty((0, 8), device=DEV), dW=full, accumulate=True)
        assert (full == 1).all()
        plan.backward(none, torch.empty((0, 8), device=DEV), dW=full)
        assert (full == 0).all()
        ids = torch.arange(6, device=DEV).view(3, 2)
        assert torch.equal(plan.forward(ids, w), w.view(3, 2, 8))
        assert torch.equal(plan.forward(torch.tensor(3, device=DEV), w), w[3])
        plan.sync()


def test_embed_repeats_and_graph():
    g = gen(4)
    n, V, D = 20000, 300, 128
    ids = ids_of("zipf", n, V, g).to(DEV)
    dy, w = ref.rnd(g, n, D, dtype="bf16").to(DEV), ref.rnd(g, V, D, dtype="bf16").to(DEV)
    plan = cat.EmbedPlan(n, V, D, "bf16", scale=11.3)
    step = lambda: (plan.forward(ids, w), plan.backward(ids, dy))  # noqa: E731
    first = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    for a, b, c, d in zip(first, step(), other, graphed(step, ids)):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)
    plan.close()


def test_embed_refusals():
    lib = cat.lib()
    n, V, D = 8, 10, 16
    ids = torch.zeros(n, dtype=torch.int64, device=DEV)
    w, y = torch.zeros((V, D), device=DEV), torch.zeros((n, D), device=DEV)
    dw = torch.zeros((V, D), device=DEV)
    p = cat.cat_plan_create_embed(n, V, D, "f32")
    a = lambda x: x.data_ptr() if torch.is_tensor(x) else x  # noqa: E731

    def fwd(ids=ids, kind=cat.CAT_I64, w=w, y=y, n=n):
        return lib.cat_embed_forward(p, a(ids), kind, a(w), a(y), n)

    def bwd(ids=ids, kind=cat.CAT_I64, dy=y, dw=dw, add=0, n=n):
        return lib.cat_embed_backward(p, a(ids), kind, a(dy), a(dw), add, n)

    assert fwd() == cat.CAT_OK and bwd() == cat.CAT_OK and fwd(n=0) == cat.CAT_OK
    for f in (fwd, bwd):
        assert f(n=n + 1) == cat.CAT_ERR_PLAN_MISMATCH
        assert f(n=-1) == cat.CAT_ERR_INVALID_ARG and f(kind=1) == cat.CAT_ERR_INVALID_ARG
        assert f(ids=None) == cat.CAT_ERR_INVALID_ARG
        assert f(ids=ids.data_ptr() + 4) == cat.CAT_ERR_MISALIGNED
    for k in ("w", "y"):
        assert fwd(**{k: None}) == cat.CAT_ERR_INVALID_ARG
        assert fwd(**{k: dict(w=w, y=y)[k].data_ptr() + 4}) == cat.CAT_ERR_MISALIGNED
    for k in ("dy", "dw"):
        assert bwd(**{k: None}) == cat.CAT_ERR_INVALID_ARG
        assert bwd(**{k: dict(dy=y, dw=dw)[k].data_ptr() + 8}) == cat.CAT_ERR_MISALIGNED
    assert bwd(add=2) == cat.CAT_ERR_INVALID_ARG
    assert fwd(y=w) == cat.CAT_ERR_ALIAS and fwd(w=ids) == cat.CAT_OK
    assert fwd(y=ids) == cat.CAT_ERR_ALIAS and bwd(dw=y) == cat.CAT_ERR_ALIAS
    norm = cat.cat_plan_create_layernorm(n, D, "f32")
    assert lib.cat_embed_forward(norm, a(ids), 3, a(w), a(y), n) == cat.CAT_ERR_PLAN_MISMATCH
    for h in (p, norm):
        cat.cat_plan_destroy(h)
    with cat.EmbedPlan(n, V, D, "f32") as plan:
        for bad in (ids.int().float(), ids.short(), torch.zeros((4, 4), dtype=torch.int64,
                                                                device=DEV).t()[:2]):
            with pytest.raises(ValueError):
                plan.forward(bad, w)
        with pytest.raises(ValueError):
            plan.forward(ids, w.bfloat16())
        with pytest.raises(ValueError):
            plan.forward(ids, w[:9])
        with pytest.raises(ValueError):
            plan.forward(ids.cpu(), w)
        with pytest.raises(ValueError):
            plan.backward(ids, y, accumulate=True)
        with pytest.raises(ValueError):
            plan.backward(ids[:4], y)
        with pytest.raises(TypeError):
            plan.forward([1, 2], w)
        with pytest.raises(cat.CatError):
            plan.forward(torch.zeros(n + 1, dtype=torch.int64, device=DEV), w)


# ------------------------------------------------- residual addition with norms
def norm_inputs(rows, D, dtype, gate, post, weights=True, seed=0):
    g = gen(seed)
    mk = lambda *s, f=1.0: ref.rnd(g, *s, scale=f, dtype=dtype)  # noqa: E731
    t = dict(r=mk(rows, D, f=2.0) + 0.5, b=mk(rows, D), gate=None, gamma=None, beta=None, pg=None,
             pb=None, dh=mk(rows, D), dy=mk(rows, D))
    if gate != "none":
        t["gate"] = mk(D) if gate == "channel" else mk(rows, D)
    if weights:
        t["gamma"], t["beta"] = 1 + mk(D, f=0.2), mk(D, f=0.2)
        if post:
            t["pg"], t["pb"] = 1 + mk(D, f=0.2), mk(D, f=0.2)
    return t


NAMES = ("dr", "db", "dgate", "dgamma", "dbeta", "dpg", "dpb")


def norm_step(plan, d, dh=True):
    h, y, stats = plan.forward(d["r"], d["b"], d["gate"], d["gamma"], d["beta"], d["pg"], d["pb"])
    grads = plan.backward(h, d["b"], d["gate"], d["gamma"], d["pg"], d["pb"], stats,
                          d["dh"] if dh else None, d["dy"])
    return dict(h=h, y=y, stats=stats), dict(zip(NAMES, grads))


def norm_parity(rows, D, dtype, gate, post, weights=True, seed=0, dh=True, scale=0.7, eps=1e-5):
    t = norm_inputs(rows, D, dtype, gate, post, weights, seed)
    with cat.ResNormPlan(rows, D, dtype, eps=eps, scale=scale, post=post) as plan:
        out, grads = norm_step(plan, {k: dev(v) for k, v in t.items()}, dh)
        plan.sync()
    want = ref.resnorm_forward(t["r"], t["b"], t["gate"], t["gamma"], t["beta"], t["pg"], t["pb"],
                               post, eps, scale, dtype)
    for n, v in want.items():
        check(n, out[n], v)
    want = ref.resnorm_backward(out["h"].cpu(), t["b"], t["gate"], t["gamma"], t["pg"], t["pb"],
                                out["stats"].cpu(), t["dh"] if dh else None, t["dy"], post, scale,
                                dtype)
    assert {n for n in NAMES if grads[n] is not None} == set(want)
    for n, v in want.items():
        check(n, grads[n], v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("D", [1, 2, 3, 8, 31, 64, 77, 256, 260, 500, 768, 1000, 1021, 1024, 1032,
                               2048, 2052, 3000, 4096, 5001, 8192])
def test_resnorm_widths(D, post, dtype):
    # (eps large where a row of one or two elements has next to no variance.)
    eps = 1e-5 if D > 3 else 0.5
    norm_parity(37, D, dtype, "channel", post, seed=D, eps=eps)
    norm_parity(5, D, dtype, "row", post, seed=D + 1, eps=eps)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("rows", [1, 2, 7, 9, 300, 5000])
def test_resnorm_rows(rows, gate, dtype):
    norm_parity(rows, 128, dtype, gate, True, seed=rows)
    norm_parity(rows, 96, dtype, gate, False, seed=rows + 1)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
def test_resnorm_missing_weights(gate, post):
    norm_parity(33, 200, "f32", gate, post, weights=False, seed=1)
    norm_parity(33, 200, "bf16", gate, post, weights=False, seed=2, dh=False)


def test_resnorm_agrees_with_the_layer_norm():
    # No gate, no norm behind the block, fp32: the sum and its layer norm.
    t = {k: dev(v) for k, v in norm_inputs(70, 320, "f32", "none", False, seed=5).items()}
    with cat.ResNormPlan(70, 320, "f32") as plan, cat.LayerNormPlan(70, 320, "f32") as ln:
        out, grads = norm_step(plan, t)
        s = t["r"] + t["b"]
        assert torch.equal(out["h"], s)
        y, mean, rstd = ln.forward(s, t["gamma"], t["beta"])
        dx, dg, db = ln.backward(s, t["gamma"], mean, rstd, t["dy"])
    for a, b in ((out["y"], y), (out["stats"][0], mean), (out["stats"][1], rstd),
                 (grads["dr"], dx + t["dh"]), (grads["dgamma"], dg), (grads["dbeta"], db)):
        assert torch.allclose(a, b, rtol=1e-5, atol=1e-5)
    assert torch.equal(grads["dr"], grads["db"])


def test_resnorm_no_rows_batches_and_one_row():
    with cat.ResNormPlan(24, 64, "f32", post=True) as plan:
        z = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
        h, y, stats = plan.forward(z(0, 64), z(0, 64), z(64))
        assert h.shape == (0, 64) and stats.shape == (4, 0)
        outs = [torch.ones(64, device=DEV) for _ in range(5)]
        got = plan.backward(h, z(0, 64), z(64), None, None, None, stats, None, y, dgate=outs[0],
                            dgamma=outs[1], dbeta=outs[2], dpost_gamma=outs[3],
                            dpost_beta=outs[4])
        assert got[2] is not None and all((t == 0).all() for t in outs)
        t = {k: dev(v) for k, v in norm_inputs(24, 64, "f32", "row", True, seed=6).items()}
        flat, fg = norm_step(plan, t)
        cube, cg = norm_step(plan, {k: v.view(2, 3, 4, 64) if v.dim() == 2 else v
                                    for k, v in t.items()})
        assert cube["stats"].shape == (4, 2, 3, 4) and cg["dgate"].shape == (2, 3, 4, 64)
        for a, b in list(zip(flat.values(), cube.values())) + list(zip(fg.values(), cg.values())):
            assert torch.equal(a.flatten(), b.flatten())
        one, _ = norm_step(plan, {k: v[3] if v.dim() == 2 else v for k, v in t.items()})
        assert one["stats"].shape == (4,) and torch.equal(one["y"], flat["y"][3])
        plan.sync()


@pytest.mark.parametrize("dtype,D", [("bf16", 768), ("f32", 3001)])
def test_resnorm_repeats_and_graph(dtype, D):
    t = {k: dev(v) for k, v in norm_inputs(3001, D, dtype, "channel", True, seed=7).items()}
    plan = cat.ResNormPlan(3001, D, dtype, post=True)

    def step():
        out, grads = norm_step(plan, t)
        return list(out.values()) + list(grads.values())

    first = step()
    for a, b, c in zip(first, step(), graphed(step, t["b"], t["dy"])):
        assert torch.equal(a, b) and torch.equal(a, c)
    plan.close()


def test_resnorm_nan_stays_in_its_row():
    t = {k: dev(v) for k, v in norm_inputs(17, 200, "bf16", "row", True, seed=8).items()}
    with cat.ResNormPlan(17, 200, "bf16", post=True) as plan:
        clean, cg = norm_step(plan, t)
        for n, v in (("r", math.nan), ("b", math.inf), ("gate", math.nan), ("dh", math.inf)):
            u = dict(t)
            u[n] = t[n].clone()
            u[n][6, 11] = v
            out, grads = norm_step(plan, u)
            keep = [i for i in range(17) if i != 6]
            for k in ("h", "y"):
                assert torch.equal(out[k][keep], clean[k][keep])
            for k in ("dr", "db", "dgate"):
                assert torch.equal(grads[k][keep], cg[k][keep])
            if n == "r":
                assert out["y"][6].isnan().all() and out["h"][6, 12:].isfinite().all()


def test_resnorm_refusals():
    lib = cat.lib()
    rows, D = 8, 64
    mk = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    f = dict(r=mk(rows, D), b=mk(rows, D), gate=mk(D), each=0, pg=mk(D), pb=mk(D), g=mk(D),
             be=mk(D), h=mk(rows, D), y=mk(rows, D), stats=mk(4, rows), n=rows)
    k = dict(h=mk(rows, D), b=mk(rows, D), gate=mk(D), each=0, pg=mk(D), pb=mk(D), g=mk(D),
             stats=mk(4, rows), dh=mk(rows, D), dy=mk(rows, D), dr=mk(rows, D), db=mk(rows, D),
             dgate=mk(D), dpg=mk(D), dpb=mk(D), dg=mk(D), dbe=mk(D), n=rows)
    a = lambda x: x.data_ptr() if torch.is_tensor(x) else x  # noqa: E731
    p = cat.cat_plan_create_resnorm(rows, D, "f32", True)
    q = cat.cat_plan_create_resnorm(rows, D, "f32", False)
    fwd = lambda plan=p, **c: lib.cat_resnorm_forward(plan, *map(a, {**f, **c}.values()))  # noqa: E731,E501
    bwd = lambda plan=p, **c: lib.cat_resnorm_backward(plan, *map(a, {**k, **c}.values()))  # noqa: E731,E501
    assert fwd() == cat.CAT_OK and bwd() == cat.CAT_OK
    assert fwd(n=0) == cat.CAT_OK and bwd(n=0) == cat.CAT_OK
    for call, args, need, may in (
            (fwd, f, ("r", "b", "h", "y", "stats"), ("gate", "pg", "pb", "g", "be")),
            (bwd, k, ("h", "b", "stats", "dy", "dr", "db"), ("dh", "dgate", "dpg", "dpb", "dg",
                                                            "dbe", "pg", "pb", "g"))):
        assert call(n=-1) == cat.CAT_ERR_INVALID_ARG
        assert call(n=rows + 1) == cat.CAT_ERR_PLAN_MISMATCH
        assert call(each=2) == cat.CAT_ERR_INVALID_ARG
        assert call(each=1, gate=None) == cat.CAT_ERR_INVALID_ARG
        for n in need:
            assert call(**{n: None}) == cat.CAT_ERR_INVALID_ARG, n
        for n in may:
            assert call(**{n: None}) == cat.CAT_OK, n
        for n in need + may:
            off = 1 if n == "stats" else 8
            assert call(**{n: args[n].data_ptr() + off}) == cat.CAT_ERR_MISALIGNED, n
        assert call(q) == cat.CAT_ERR_INVALID_ARG          # weights of a norm it does not have
    assert fwd(q, pg=None, pb=None) == cat.CAT_OK
    assert bwd(q, pg=None, pb=None, dpg=None, dpb=None) == cat.CAT_OK
    assert bwd(gate=None) == cat.CAT_ERR_INVALID_ARG       # dgate without a gate
    assert fwd(h=f["r"]) == cat.CAT_ERR_ALIAS and fwd(y=f["h"]) == cat.CAT_ERR_ALIAS
    assert bwd(dr=k["dh"]) == cat.CAT_ERR_ALIAS and bwd(db=k["dr"]) == cat.CAT_ERR_ALIAS
    assert bwd(dg=k["dbe"]) == cat.CAT_ERR_ALIAS and bwd(dgate=k["gate"]) == cat.CAT_ERR_ALIAS
    e = cat.cat_plan_create_embed(4, 4, D, "f32")
    assert fwd(e) == cat.CAT_ERR_PLAN_MISMATCH and bwd(e) == cat.CAT_ERR_PLAN_MISMATCH
    for h in (p, q, e):
        cat.cat_plan_destroy(h)
    with cat.ResNormPlan(rows, D, "f32") as plan:
        r, b = mk(rows, D), mk(rows, D)
        for bad in (dict(R=r[:4]), dict(R=r.bfloat16()), dict(B=b.cpu()), dict(gate=mk(D + 1)),
                    dict(gate=mk(4, D)), dict(gamma=mk(D, 1)), dict(H=mk(D, rows).t()),
                    dict(stats=mk(4, rows))):
            with pytest.raises(ValueError):
                plan.forward(**{**dict(R=r, B=b), **bad})
        h, y, stats = plan.forward(r, b)
        with pytest.raises(ValueError):
            plan.backward(h, b, None, None, None, None, stats, None, y, dgate=mk(D))
        with pytest.raises(ValueError):
            plan.backward(h, b, None, None, None, None, stats, None, y, dpost_beta=mk(D))
        with pytest.raises(cat.CatError):
            plan.forward(r, b, post_gamma=mk(D))


# --------------------------------------------------------------- cross entropy
def xent_inputs(T, V, D, dtype, kept=1.0, seed=0, sharp=2.0):
    g = gen(seed)
    x = ref.rnd(g, T, D, dtype=dtype)
    w = ref.rnd(g, V, D, scale=sharp / math.sqrt(D), dtype=dtype)
    targets = torch.randint(0, V, (T,), generator=g)
    targets[torch.rand(T, generator=g) >= kept] = -100
    return x, w, targets


def near(got, want, norm):
    err = (got.detach().double().cpu() - want).norm()
    assert err <= norm, (float(err), float(norm))


def xent_parity(T, V, D, dtype, kept=1.0, seed=0, each=True, sharp=2.0, wide=True):
    x, w, targets = xent_inputs(T, V, D, dtype, kept, seed, sharp)
    up = torch.rand(T if each else (), generator=gen(seed + 1)) + 0.1
    t = targets if wide else targets.int()
    with cat.XentPlan(T, V, D, dtype) as plan:
        loss, lse = plan.forward(dev(x), dev(w), dev(t))
        dx, dw = plan.backward(dev(x), dev(w), dev(t), lse, dev(up))
        plan.sync()
    for n, v in ref.xent_forward(x, w, targets).items():
        check(n, dict(loss=loss, lse=lse)[n], v)
    want, n_dx, n_dw = ref.xent_backward(x, w, targets, lse.cpu(), up, dtype)
    check("dx", dx, want["dx"])
    check("dw", dw, want["dw"])
    if dtype == "f32":
        near(dx, want["dx"][0], n_dx)
        near(dw, want["dw"][0], n_dw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D", [
    (1, 1, 1), (1, 2, 8), (2, 1, 16), (1, 1000, 64), (3, 257, 64), (17, 100, 24), (63, 64, 33),
    (64, 256, 64), (65, 300, 72), (127, 511, 128), (128, 512, 100), (129, 513, 200),
    (255, 1023, 7), (256, 1024, 256), (257, 1025, 264), (300, 2500, 520), (1000, 777, 96),
    (40, 5000, 768),
])
def test_xent_sizes(T, V, D, dtype):
    xent_parity(T, V, D, dtype, seed=T + V + D, each=T % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kept", [0.0, 0.05, 0.5, 0.97])
@pytest.mark.parametrize("T,V,D", [(5, 40, 16), (700, 600, 64), (1500, 300, 40)])
def test_xent_without_targets(T, V, D, kept, dtype):
    xent_parity(T, V, D, dtype, kept, seed=T, wide=T > 10)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_xent_long(dtype):
    # More than one piece of the vocabulary; more tokens than one block of the list.
    xent_parity(2100, 9001, 64, dtype, 0.9, seed=5)
    xent_parity(260, 20011, 128, dtype, seed=6)


def test_xent_many_tokens():
    # More tokens than a preparing CTA's 128 for each of its most CTAs.
    xent_parity(270001, 40, 8, "bf16", 0.6, seed=18)
    xent_parity(263000, 20, 12, "f32", 1.0, seed=19, each=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,D,kept,room", [
    (300, 20011, 64, 1.0, 65536), (700, 9000, 520, 0.9, 65536), (5, 17000, 40, 1.0, 65536),
    (1300, 8193, 72, 0.3, 66000), (64, 16384, 96, 0.0, 65536),
])
def test_xent_pieces(T, V, D, kept, room, dtype):
    # A plan for many tokens takes its vocabulary in several pieces, here with few.
    x, w, targets = xent_inputs(T, V, D, dtype, kept, seed=T)
    up = torch.rand(T, generator=gen(T + 1)) + 0.1
    with cat.XentPlan(room, V, D, dtype) as plan:
        piece = int(plan.describe().split("piece=")[1].split()[0])
        assert piece < V
        for _ in range(2):
            loss, lse = plan.forward(dev(x), dev(w), dev(targets))
            dx, dw = plan.backward(dev(x), dev(w), dev(targets), lse, dev(up))
        only = plan.backward(dev(x), dev(w), dev(targets), lse, dev(up), dX=False)[1]
        assert torch.equal(only, dw)
        only = plan.backward(dev(x), dev(w), dev(targets), lse, dev(up), dW=False)[0]
        assert torch.equal(only, dx)
        plan.sync()
    for n, v in ref.xent_forward(x, w, targets).items():
        check(n, dict(loss=loss, lse=lse)[n], v)
    want, n_dx, n_dw = ref.xent_backward(x, w, targets, lse.cpu(), up, dtype)
    check("dx", dx, want["dx"])
    check("dw", dw, want["dw"])
    if dtype == "f32":
        near(dx, want["dx"][0], n_dx)
        near(dw, want["dw"][0], n_dw)


@pytest.mark.parametrize("sharp", [0.0, 30.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_xent_flat_and_sharp(sharp, dtype):
    xent_parity(130, 700, 64, dtype, seed=7, sharp=sharp)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_xent_rows_without_targets_are_not_read(dtype, value):
    T, V, D = 400, 300, 64
    x, w, targets = xent_inputs(T, V, D, dtype, 0.6, seed=8)
    clean, up = x.clone(), torch.rand(T, generator=gen(9))
    x[targets < 0] = value
    up[targets < 0] = math.nan
    with cat.XentPlan(T, V, D, dtype) as plan:
        a = plan.forward(dev(x), dev(w), dev(targets))
        b = plan.forward(dev(clean), dev(w), dev(targets))
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        lse = a[1].clone()
        lse[dev(targets) < 0] = math.nan
        g = plan.backward(dev(x), dev(w), dev(targets), lse, dev(up))
        h = plan.backward(dev(clean), dev(w), dev(targets), a[1], dev(up).nan_to_num(0.0))
        for p, q in zip(g, h):
            assert p.isfinite().all() and torch.equal(p, q)
        assert (g[0][dev(targets) < 0] == 0).all()


def test_xent_a_nan_stays_in_its_token():
    T, V, D = 300, 400, 64
    x, w, targets = xent_inputs(T, V, D, "bf16", seed=10)
    up = torch.full((), 1.0 / T)
    bad = x.clone()
    bad[77, 5] = math.nan
    keep = [i for i in range(T) if i != 77]
    with cat.XentPlan(T, V, D, "bf16") as plan:
        a, b = (plan.forward(dev(v), dev(w), dev(targets)) for v in (x, bad))
        for p, q in zip(a, b):
            assert torch.equal(p[keep], q[keep]) and q[77].isnan()
        g, h = (plan.backward(dev(v), dev(w), dev(targets), s[1], dev(up))
                for v, s in ((x, a), (bad, b)))
        assert torch.equal(g[0][keep], h[0][keep]) and h[0][77].isnan().all()
        # A weight that is not finite reaches every token's sum.
        w[3, 0] = math.inf
        loss, _ = plan.forward(dev(x), dev(w), dev(targets))
        assert not (loss.isfinite() & (dev(x)[:, 0] > 0)).any()


@pytest.mark.parametrize("where", ["x", "w"])
def test_xent_f32_values_that_are_not_finite(where):
    # fp32 operands go as terms: logits with an infinity or a NaN are those of their
    # definition all the same, in every place of a tile.
    T, V, D = 300, 600, 48
    x, w, targets = xent_inputs(T, V, D, "f32", seed=17)
    for i, v in ((3, math.inf), (130, -math.inf), (299, math.nan)):
        (x if where == "x" else w)[i, i % D] = v
    with cat.XentPlan(T, V, D, "f32") as plan:
        loss, lse = plan.forward(dev(x), dev(w), dev(targets))
        plan.sync()
    if where == "w":
        # Every token meets the NaN; without its row the infinities decide.
        assert lse.isnan().all()
        w[299] = 0.0
        keep = (x[:, 3] < 0) & (x[:, 130 % D] > 0)      # both of them minus infinity
        assert keep.any() and not keep.all()
        rest = [i for i in range(V) if i not in (3, 130)]
        with cat.XentPlan(T, V, D, "f32") as plan:
            loss, lse = plan.forward(dev(x), dev(w), dev(targets))
        val, bound = ref.xent_forward(x, w[rest], torch.zeros(T, dtype=torch.int64))["lse"]
        check("lse", lse[dev(keep)], (val[keep], bound[keep]))
        assert not lse[dev(~keep)].isfinite().any()
    else:
        bad = torch.zeros(T, dtype=torch.bool)
        bad[[3, 130, 299]] = True
        val, bound = ref.xent_forward(x[~bad], w, targets[~bad])["lse"]
        check("lse", lse[dev(~bad)], (val, bound))
        assert not lse[dev(bad)].isfinite().any()


def test_xent_minus_infinity_is_a_logit_of_its_own():
    # Ids that the weights rule out (logits of minus infinity) take no part.
    T, V, D = 70, 300, 16
    x, w, targets = xent_inputs(T, V, D, "f32", seed=11)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    targets %= 200
    keep = ref.xent_forward(x, w[:200], targets)
    w[200:] = 0.0
    w[200:, 0] = -math.inf
    with cat.XentPlan(T, V, D, "f32") as plan:
        loss, lse = plan.forward(dev(x), dev(w), dev(targets))
        check("loss", loss, keep["loss"])
        check("lse", lse, keep["lse"])


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_xent_targets_outside(kind):
    T, V, D = 6, 50, 32
    x, w, targets = xent_inputs(T, V, D, "f32", seed=12)
    targets = targets.to(kind)
    targets[1], targets[4] = V, 2**31 - 1
    with cat.XentPlan(T, V, D, "f32") as plan:
        loss, lse = plan.forward(dev(x), dev(w), dev(targets))
        with pytest.raises(cat.CatError) as e:
            plan.sync()
        assert e.value.status == cat.CAT_ERR_DEVICE_STATUS
        for n, v in ref.xent_forward(x, w, targets).items():
            check(n, dict(loss=loss, lse=lse)[n], v)
        dx, _ = plan.backward(dev(x), dev(w), dev(targets), lse, torch.ones((), device=DEV))
        with pytest.raises(cat.CatError):
            plan.sync()
        assert (dx[[1, 4]] == 0).all() and dx[0].abs().sum() > 0


def test_xent_outputs_not_wanted_no_tokens_and_shapes():
    T, V, D = 24, 90, 40
    x, w, targets = (dev(t) for t in xent_inputs(T, V, D, "bf16", seed=13))
    one = torch.ones((), device=DEV)
    with cat.XentPlan(T, V, D, "bf16") as plan, cat.XentPlan(T, V, D, "bf16", grad=False) as fwd:
        loss, lse = plan.forward(x, w, targets)
        l2, _ = fwd.forward(x, w, targets)
        assert torch.equal(loss, l2)
        with pytest.raises(cat.CatError) as e:
            fwd.backward(x, w, targets, lse, one)
        assert e.value.status == cat.CAT_ERR_PLAN_MISMATCH
        dx, dw = plan.backward(x, w, targets, lse, one)
        a, none = plan.backward(x, w, targets, lse, one, dW=False)
        assert none is None and torch.equal(a, dx)
        none, b = plan.backward(x, w, targets, lse, one, dX=False)
        assert none is None and torch.equal(b, dw)
        cube = plan.forward(x.view(2, 12, D), w, targets.view(2, 12))[0]
        assert cube.shape == (2, 12) and torch.equal(cube.flatten(), loss)
        each = torch.ones((2, 12), device=DEV)
        c, _ = plan.backward(x.view(2, 12, D), w, targets.view(2, 12), lse.view(2, 12), each)
        assert c.shape == (2, 12, D) and torch.equal(c.view(T, D), dx)
        z = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
        no = torch.zeros(0, dtype=torch.int64, device=DEV)
        assert plan.forward(x[:0], w, no)[0].shape == (0,)
        d0, dw0 = plan.backward(x[:0], w, no, z(0), one, dW=torch.ones_like(w))
        assert d0.shape == (0, D) and (dw0 == 0).all()
        gone = torch.full_like(targets, -1)
        d0, dw0 = plan.backward(x, w, gone, lse, one, dX=torch.ones_like(x),
                                dW=torch.ones_like(w))
        assert (d0 == 0).all() and (dw0 == 0).all()
        # Fewer tokens than the plan's, after more of them.
        s, _ = plan.forward(x[:5], w, targets[:5])
        assert torch.equal(s, loss[:5])
        plan.sync()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_xent_repeats_streams_and_graph(dtype):
    T, V, D = 700, 5000, 96
    x, w, targets = (dev(t) for t in xent_inputs(T, V, D, dtype, 0.8, seed=14))
    up = torch.full((), 0.01, device=DEV)
    plan = cat.XentPlan(T, V, D, dtype)

    def step():
        loss, lse = plan.forward(x, w, targets)
        return (loss, lse) + tuple(plan.backward(x, w, targets, lse, up))

    first = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    for a, b, c, d in zip(first, step(), other, graphed(step, x, targets)):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)
    plan.close()


def test_xent_one_factor_for_all_tokens_loses_nothing():
    # With one upstream value for all tokens dx and dw are scaled by it in fp32: as
    # near as with the value 1, whatever its own rounding to bf16 would be; and
    # gradients of no tokens are zero, whatever it is.
    T, V, D = 400, 700, 64
    x, w, targets = xent_inputs(T, V, D, "bf16", seed=16, sharp=0.5)
    with cat.XentPlan(T, V, D, "bf16") as plan:
        _, lse = plan.forward(dev(x), dev(w), dev(targets))
        off = []
        for up in (1.0, 2.0 ** -7 * (1 + 2.0 ** -8)):       # (half a step from a bf16 value)
            up = torch.tensor(up)
            got = plan.backward(dev(x), dev(w), dev(targets), lse, dev(up))
            want, _, _ = ref.xent_backward(x, w, targets, lse.cpu(), up, "bf16")
            for n, t in zip(("dx", "dw"), got):
                check(n, t, want[n])
                off.append(float((t.double().cpu() - want[n][0]).norm() / want[n][0].norm()))
        # A rounding to bf16 is off by an even spread within 2^-8 / x of a value of
        # mantissa x in 1 .. 2: in the root mean square, over mantissas spread by their
        # logarithm, 2^-8 / sqrt(3) · sqrt(3 / (8 ln 2)) = 0.42 · 2^-8.  Two of them
        # meet, d's and the result's: 0.60 · 2^-8.  The factor's own would add all of
        # its 2^-8, the same way everywhere.
        assert max(off) <= 0.75 * 2.0 ** -8, off
        for up in (math.nan, math.inf):
            dx, dw = plan.backward(dev(x), dev(w), torch.full_like(dev(targets), -1), lse,
                                   torch.full((), up, device=DEV))
            assert (dx == 0).all() and (dw == 0).all()
        assert plan.backward(dev(x), dev(w), dev(targets), lse,
                             torch.full((), math.nan, device=DEV))[1].isnan().all()


def test_xent_two_plans_on_two_streams():
    T, V, D = 300, 3001, 64
    x, w, targets = (dev(t) for t in xent_inputs(T, V, D, "bf16", 0.8, seed=15))
    up = torch.full((), 0.01, device=DEV)
    streams = [torch.cuda.Stream() for _ in range(2)]
    plans = [cat.XentPlan(T, V, D, "bf16", stream=s) for s in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s, plan in zip(streams, plans):
            with torch.cuda.stream(s):
                loss, lse = plan.forward(x, w, targets)
                got.append((loss, lse) + tuple(plan.backward(x, w, targets, lse, up)))
    torch.cuda.synchronize()
    for r in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, got[0]))
    for plan in plans:
        plan.close()


def test_xent_refusals():
    lib = cat.lib()
    T, V, D = 8, 20, 16
    mk = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    t = torch.zeros(T, dtype=torch.int64, device=DEV)
    f = dict(x=mk(T, D), w=mk(V, D), t=t, kind=3, loss=mk(T), lse=mk(T), n=T)
    k = dict(x=f["x"], w=f["w"], t=t, kind=3, lse=mk(T), up=mk(T), each=1, dx=mk(T, D),
             dw=mk(V, D), n=T)
    a = lambda v: v.data_ptr() if torch.is_tensor(v) else v  # noqa: E731
    p = cat.cat_plan_create_xent(T, V, D, "f32")
    fwd = lambda plan=p, **c: lib.cat_xent_forward(plan, *map(a, {**f, **c}.values()))  # noqa: E731
    bwd = lambda plan=p, **c: lib.cat_xent_backward(plan, *map(a, {**k, **c}.values()))  # noqa: E731
    assert fwd() == cat.CAT_OK and bwd() == cat.CAT_OK and bwd(each=0) == cat.CAT_OK
    assert fwd(n=0) == cat.CAT_OK and bwd(n=0) == cat.CAT_OK
    for call, args, need in ((fwd, f, ("x", "w", "t", "loss", "lse")),
                             (bwd, k, ("x", "w", "t", "lse", "up"))):
        assert call(n=-1) == cat.CAT_ERR_INVALID_ARG
        assert call(n=T + 1) == cat.CAT_ERR_PLAN_MISMATCH
        assert call(kind=0) == cat.CAT_ERR_INVALID_ARG
        for n in need:
            assert call(**{n: None}) == cat.CAT_ERR_INVALID_ARG, n
            off = 8 if n in "xw" else 4 if n == "t" else 2
            assert call(**{n: args[n].data_ptr() + off}) == cat.CAT_ERR_MISALIGNED, n
    assert bwd(each=2) == cat.CAT_ERR_INVALID_ARG
    for n in ("dx", "dw"):
        assert bwd(**{n: None}) == cat.CAT_OK
        assert bwd(**{n: k[n].data_ptr() + 8}) == cat.CAT_ERR_MISALIGNED
    assert bwd(dx=None, dw=None) == cat.CAT_OK
    assert fwd(loss=f["x"]) == cat.CAT_ERR_ALIAS and fwd(lse=f["loss"]) == cat.CAT_ERR_ALIAS
    assert bwd(dx=k["x"]) == cat.CAT_ERR_ALIAS and bwd(dw=k["w"]) == cat.CAT_ERR_ALIAS
    e = cat.cat_plan_create_embed(T, V, D, "f32")
    assert fwd(e) == cat.CAT_ERR_PLAN_MISMATCH and bwd(e) == cat.CAT_ERR_PLAN_MISMATCH
    for h in (p, e):
        cat.cat_plan_destroy(h)
    with cat.XentPlan(T, V, D, "f32") as plan:
        x, w = f["x"], f["w"]
        for bad in ((x[:4], w, t), (x, w[:4], t), (x, w, t.float()), (x, w, t[:4]),
                    (x.bfloat16(), w, t), (x, w.t().contiguous().t(), t), (x.cpu(), w, t)):
            with pytest.raises(ValueError):
                plan.forward(*bad)
        loss, lse = plan.forward(x, w, t)
        for up in (mk(2), mk(T, 1), mk(T).double(), mk(2 * T)[::2]):
            with pytest.raises(ValueError):
                plan.backward(x, w, t, lse, up)


# --------------------------------------------------------------------- together
def test_plans_with_a_stream_of_their_own():
    # All calls on the plans' stream, the default stream busy; outputs that a call
    # allocates belong to that stream.
    g = gen(30)
    T, V, D = 500, 900, 64
    ids = ids_of("zipf", T, V, g).to(DEV)
    w = ref.rnd(g, V, D, dtype="bf16").to(DEV)
    t = {k: dev(v) for k, v in norm_inputs(T, D, "bf16", "channel", True, seed=31).items()}
    up = torch.full((), 0.01, device=DEV)

    def step(embed, res, xent):
        x = embed.forward(ids, w)
        h, y, stats = res.forward(x, t["b"], t["gate"], t["gamma"], t["beta"], t["pg"], t["pb"])
        loss, lse = xent.forward(y, w, ids)
        dy, dw = xent.backward(y, w, ids, lse, up)
        grads = res.backward(h, t["b"], t["gate"], t["gamma"], t["pg"], t["pb"], stats, None, dy)
        embed.backward(ids, grads[0], dW=dw, accumulate=True)
        return (x, h, y, stats, loss, lse, dy, dw) + tuple(grads)

    def plans(stream):
        return (cat.EmbedPlan(T, V, D, "bf16", stream=stream),
                cat.ResNormPlan(T, D, "bf16", post=True, stream=stream),
                cat.XentPlan(T, V, D, "bf16", stream=stream))

    want = step(*plans(None))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    own = plans(side)
    for _ in range(5):
        torch.cuda._sleep(3_000_000)
        scratch = [torch.randn(T * D, device=DEV) for _ in range(4)]
        del scratch
        got = step(*own)
        side.synchronize()
        for p in own:
            p.sync()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    for p in own:
        p.close()
    with pytest.raises(ValueError):
        own[0].forward(ids, w)                  # closed


def test_a_step_in_one_graph():
    # Captured once, replayed with other ids, targets and weights.
    T, V, D = 640, 1200, 96
    g = gen(32)
    ids = torch.randint(0, V, (T,), generator=g).to(DEV)
    targets = torch.randint(0, V, (T,), generator=g).to(DEV)
    w = ref.rnd(g, V, D, scale=0.3, dtype="bf16").to(DEV)
    b = ref.rnd(g, T, D, dtype="bf16").to(DEV)
    up = torch.full((), 0.01, device=DEV)
    embed, res = cat.EmbedPlan(T, V, D, "bf16"), cat.ResNormPlan(T, D, "bf16", scale=0.5)
    xent = cat.XentPlan(T, V, D, "bf16")

    def step():
        x = embed.forward(ids, w)
        h, y, stats = res.forward(x, b)
        loss, lse = xent.forward(y, w, targets)
        dy, dw = xent.backward(y, w, targets, lse, up)
        dr, db = res.backward(h, b, None, None, None, None, stats, None, dy)[:2]
        return loss, dw, db, embed.backward(ids, dr)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(3):
        h = gen(40 + seed)
        ids.copy_(ids_of("zipf", T, V, h))
        kept = torch.randint(0, V, (T,), generator=h)
        kept[torch.rand(T, generator=h) < (0.0, 0.5, 1.0)[seed]] = -1
        targets.copy_(kept)
        w.copy_(ref.rnd(h, V, D, scale=0.3, dtype="bf16"))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(held, step()):
            assert torch.equal(a, c), seed
    for p in (embed, res, xent):
        p.sync()


@pytest.mark.parametrize("tied", [False, True])
def test_training_step_of_a_small_language_model(tied):
    """Embedding, a CAT layer and an attention layer with the residual stream
    between them, cross entropy; all gradients by the framework's calls, against
    64-bit autograd.

    Every operator is within some 1e-6 of its values in fp32 and the chain is a
    dozen operators long with weights of norm about one, so 1e-4 of each
    gradient's largest value bounds the whole.
    """
    B, N, D, heads, V = 2, 64, 64, 4, 101
    dh, scale, eps = D // heads, 1.5, 1e-5
    g = gen(20)
    r64 = lambda *s, f=1.0: (torch.randn(*s, generator=g, dtype=torch.float64) * f).float().double()  # noqa: E731,E501
    p = dict(emb=r64(V, D, f=0.5), g0=1 + r64(D, f=0.1), b0=r64(D, f=0.1), wa=r64(D, heads, f=0.1),
             wv=r64(D, D, f=D ** -0.5), gate=r64(D, f=0.5), g1=1 + r64(D, f=0.1),
             b1=r64(D, f=0.1), wqkv=r64(D, 3 * D, f=D ** -0.5), pg=1 + r64(D, f=0.1),
             pb=r64(D, f=0.1), g2=1 + r64(D, f=0.1), b2=r64(D, f=0.1))
    if not tied:
        p["head"] = r64(V, D, f=0.3)
    ids = torch.randint(0, V, (B, N), generator=g)
    ids[1, -9:] = -1
    targets = torch.randint(0, V, (B, N), generator=g)
    targets[torch.rand(B, N, generator=g) < 0.3] = -100
    targets[ids < 0] = -100

    q = {n: t.clone().requires_grad_() for n, t in p.items()}
    ln = lambda t, w, b: torch.nn.functional.layer_norm(t, (D,), w, b, eps)  # noqa: E731
    x0 = scale * torch.nn.functional.embedding(ids.clamp(min=0), q["emb"]) * (ids >= 0)[..., None]
    n0 = ln(x0, q["g0"], q["b0"])
    zs = torch.softmax(n0 @ q["wa"], 1)
    v0 = n0 @ q["wv"]
    at = (torch.arange(N)[:, None] - torch.arange(N)[None]) % N
    blk = torch.einsum("bijh,bjhc->bihc", zs[:, at], v0.view(B, N, heads, dh)).reshape(B, N, D)
    x1 = x0 + 0.8 * q["gate"] * blk
    n1 = ln(x1, q["g1"], q["b1"])
    qkv = (n1 @ q["wqkv"]).view(B, N, 3, heads, dh)
    s = torch.einsum("bihc,bjhc->bhij", qkv[:, :, 0], qkv[:, :, 1]) / math.sqrt(dh)
    s = s.masked_fill(~torch.ones(N, N, dtype=torch.bool).tril(), -math.inf)
    att = torch.einsum("bhij,bjhc->bihc", torch.softmax(s, -1), qkv[:, :, 2]).reshape(B, N, D)
    x2 = x1 + ln(att, q["pg"], q["pb"])
    n2 = ln(x2, q["g2"], q["b2"])
    head = q["emb"] if tied else q["head"]
    count = int((targets >= 0).sum())
    want_loss = torch.nn.functional.cross_entropy((n2 @ head.T).view(-1, V), targets.view(-1),
                                                  reduction="none")
    (want_loss.sum() / count).backward()

    d = {n: t.float().to(DEV) for n, t in p.items()}
    I, Tg = ids.to(DEV), targets.to(DEV)
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV) * N
    embed = cat.EmbedPlan(B * N, V, D, "f32", scale=scale)
    norm0 = cat.LayerNormPlan(B * N, D, "f32", eps=eps)
    layer = cat.Plan(B, N, D, heads, "f32")
    res1 = cat.ResNormPlan(B * N, D, "f32", eps=eps, scale=0.8)
    attn = cat.AttnPlan(B * N, B, heads, heads, dh, "f32")
    res2 = cat.ResNormPlan(B * N, D, "f32", eps=eps, post=True)
    xent = cat.XentPlan(B * N, V, D, "f32")
    X0 = embed.forward(I, d["emb"])
    N0, m0, r0 = norm0.forward(X0, d["g0"], d["b0"])
    V0 = N0 @ d["wv"]
    B0 = layer.forward(N0, d["wa"], V0)
    X1, N1, s1 = res1.forward(X0, B0, d["gate"], d["g1"], d["b1"])
    QKV = (N1 @ d["wqkv"]).view(B * N, 3 * heads, dh)
    parts = (QKV[:, :heads], QKV[:, heads:2 * heads], QKV[:, 2 * heads:])
    O, olse = attn.forward(*parts, cu)
    A = O.view(B, N, D)
    X2, N2, s2 = res2.forward(X1, A, None, d["g2"], d["b2"], d["pg"], d["pb"])
    W = d["emb"] if tied else d["head"]
    loss, lse = xent.forward(N2, W, Tg)
    assert (loss.double().cpu().flatten() - want_loss.detach()).abs().max() <= 1e-4

    got = {}
    dN2, dWt = xent.backward(N2, W, Tg, lse, torch.full((), 1.0 / count, device=DEV))
    dX1, dA, _, got["g2"], got["b2"], got["pg"], got["pb"] = res2.backward(
        X2, A, None, d["g2"], d["pg"], d["pb"], s2, None, dN2)
    dQKV = torch.empty_like(QKV)
    attn.backward(*parts, O, olse, dA.view(B * N, heads, dh), cu, dQ=dQKV[:, :heads],
                  dK=dQKV[:, heads:2 * heads], dV=dQKV[:, 2 * heads:])
    flat = dQKV.view(B * N, 3 * D)
    got["wqkv"] = N1.view(B * N, D).t() @ flat
    dN1 = (flat @ d["wqkv"].t()).view(B, N, D)
    dX0, dB0, got["gate"], got["g1"], got["b1"], _, _ = res1.backward(
        X1, B0, d["gate"], d["g1"], None, None, s1, dX1, dN1)
    dN0, got["wa"], dV0 = layer.backward(N0, d["wa"], V0, dB0)
    got["wv"] = N0.view(B * N, D).t() @ dV0.view(B * N, D)
    dN0 = dN0 + dV0 @ d["wv"].t()
    more, got["g0"], got["b0"] = norm0.backward(X0, d["g0"], m0, r0, dN0)
    if tied:
        got["emb"] = embed.backward(I, dX0 + more, dW=dWt, accumulate=True)
    else:
        got["emb"], got["head"] = embed.backward(I, dX0 + more), dWt
    for n in p:
        want = q[n].grad
        err = (got[n].double().cpu() - want).abs().max()
        assert err <= 1e-4 * want.abs().max(), (n, float(err), float(want.abs().max()))
    for plan in (embed, norm0, res1, attn, res2, xent):
        plan.sync()
