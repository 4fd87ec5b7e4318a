"""GPU tests of the operator plans' life around their kernels: what a plan holds
when its creation returns, on which streams, and what it keeps of its callers'
arguments."""
import numpy as np
import pytest
import torch

import fft_circulant_attention_gb300 as cat
import _block_ref as ref
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


def test_a_new_plan_does_not_wait_for_the_default_stream():
    # A plan is complete when its creation returns, even while the default
    # stream is busy: its status word is not cleared behind a first call that
    # reported into it (sequences that do not ascend).
    q, k, v, _, _ = ref.attn_inputs([100], 2, 2, 64, "bf16", 7)
    ins = [t.to(DEV) for t in (q, k, v)]
    bad = torch.tensor([0, 50, 20, 100], dtype=torch.int32, device=DEV)
    with cat.AttnPlan(100, 3, 2, 2, 64, "bf16") as warm:      # kernels loaded, outputs cached
        warm.forward(*ins, torch.tensor([0, 100], dtype=torch.int32, device=DEV))
        warm.sync()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                            # the default stream: 0.1 s
    plan = cat.AttnPlan(100, 3, 2, 2, 64, "bf16", stream=side)
    plan.forward(*ins, bad)
    side.synchronize()
    torch.cuda.synchronize()
    with pytest.raises(cat.CatError) as e:
        plan.sync()
    assert e.value.status == cat.CAT_ERR_DEVICE_STATUS
    plan.sync()
    plan.close()


@pytest.mark.parametrize("count", [3, 700])
def test_clip_plans_are_ready_at_once_on_a_side_stream(count):
    # Made and used without a wait in between, the default stream idle or busy.
    r = np.random.default_rng(count)
    sizes = [int(n) for n in r.integers(1, 40000 if count < 10 else 400, count)]
    host = [torch.randn(n, generator=torch.Generator().manual_seed(n)) for n in sizes]
    want, outs = ref.clip(host, 0.5)
    grads = [t.to(DEV) for t in host]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for busy in (False, True) * 4:
        if busy:
            torch.cuda._sleep(2_000_000)
        with cat.ClipPlan(sizes, ["f32"] * count, stream=side) as plan:
            to = [torch.empty_like(t) for t in grads]
            got = plan.clip(grads, 0.5, out=to)
            plan.sync()
            check("norm", got, want)
            for t, o in zip(to, outs):
                check("out", t, o)


@pytest.mark.parametrize("B,N,D,H,dtype", [(2, 196, 64, 2, "f32"), (1, 16384, 128, 2, "bf16"),
                                           (1, 1000, 24, 3, "f32")])
def test_cat_plans_are_ready_at_once_on_a_side_stream(B, N, D, H, dtype):
    # A CAT plan's tables as well: made and used while the default stream is busy.
    g = torch.Generator().manual_seed(N)
    X, V = (torch.randn((B, N, D), generator=g).to(ref.TORCH[dtype]).to(DEV) for _ in range(2))
    W = (0.1 * torch.randn((D, H), generator=g)).to(ref.TORCH[dtype]).to(DEV)
    with cat.Plan(B, N, D, H, dtype) as plan:
        torch.cuda.synchronize()
        want = plan.forward(X, W, V)
        plan.sync()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        torch.cuda._sleep(2_000_000)
        O = torch.empty_like(V)
        with cat.Plan(B, N, D, H, dtype, stream=side) as plan:
            plan.forward(X, W, V, O)
            plan.sync()
        assert torch.equal(O, want)


def test_2d_plans_are_ready_at_once_on_a_side_stream():
    g = torch.Generator().manual_seed(2)
    B, h, w, D, H = 1, 16, 16, 64, 2
    Q, K, V = (torch.randn((B, h * w, D), generator=g).to(DEV) for _ in range(3))
    with cat.Plan2D(B, h, w, D, H, "f32") as plan:
        torch.cuda.synchronize()
        want = plan.forward(Q, K, V)
        plan.sync()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        torch.cuda._sleep(2_000_000)
        O = torch.empty_like(V)
        with cat.Plan2D(B, h, w, D, H, "f32", stream=side) as plan:
            plan.forward(Q, K, V, O)
            plan.sync()
        assert torch.equal(O, want)


def test_a_status_is_reported_once_and_again():
    # Reported, cleared, and reported again by the next call.
    q, k, v, _, _ = ref.attn_inputs([100], 2, 2, 64, "bf16", 7)
    ins = [t.to(DEV) for t in (q, k, v)]
    bad = torch.tensor([0, 50, 20, 100], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with cat.AttnPlan(100, 3, 2, 2, 64, "bf16", stream=side) as plan:
        for _ in range(20):
            plan.forward(*ins, bad)
            with pytest.raises(cat.CatError) as e:
                plan.sync()
            assert e.value.status == cat.CAT_ERR_DEVICE_STATUS
        plan.sync()


@pytest.mark.parametrize("hq,hkv,dh", [(4, 2, 64), (4, 1, 128)])
def test_backward_calls_one_after_another(hq, hkv, dh):
    # Calls of one plan without a wait in between, with other inputs, other
    # sequences and other widths of the row statistics each time: none sees
    # what the one before it left in the plan's workspace.
    sets = []
    T = 900
    plan = cat.AttnPlan(T, 8, hq, hkv, dh, "bf16")
    for i, lens in enumerate(([900], [1, 898, 1], [300, 299, 301], [113] * 7 + [109])):
        q, k, v, do, cu = (t.to(DEV) for t in ref.attn_inputs(lens, hq, hkv, dh, "bf16", i))
        o, lse = plan.forward(q, k, v, cu)
        sets.append((q, k, v, o, lse, do * (1.0 + 3 * i), cu))
    want = []
    for s in sets:
        torch.cuda.synchronize()
        want.append(plan.backward(*s))
        plan.sync()
    got = [plan.backward(*sets[i % len(sets)]) for i in range(60)]
    plan.sync()
    for i, r in enumerate(got):
        for a, b in zip(r, want[i % len(sets)]):
            assert torch.equal(a, b), i
    plan.close()


@pytest.mark.parametrize("hq,n,which", [
    (1, 16384, "v"), (1, 16384, "do"), (32, 4096, "v"), (32, 4096, "do"), (32, 4096, None),
])
def test_f32_waits_last_as_long_as_the_work(monkeypatch, hq, n, which):
    # Rows that meet a NaN are computed one by one, and the role that finds the
    # work waits for a whole block of it: with a limit of 2048 polls (8 ms) in
    # place of two million, both take far longer than one wait, and no wait is
    # lost as long as there is progress.
    dh, at, last, c = 64, n - 70, n - 128, 3       # `last`: the first row of the last tile
    g = torch.Generator(device=DEV).manual_seed(n + hq)
    q, k, v, do = (torch.randn((n, h, dh), generator=g, device=DEV) for h in (hq, 1, 1, hq))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    with cat.AttnPlan(n, 1, hq, 1, dh, "f32") as plan:
        o, lse = plan.forward(q, k, v, cu)
        dq, dk, dv = plan.backward(q, k, v, o, lse, do, cu)
        plan.sync()
    if which == "v":
        v = v.clone()
        v[at, :, c] = float("nan")
    elif which == "do":
        do = do.clone()
        do[at, :, c] = float("nan")
    monkeypatch.setenv("CAT_ATTN_POLLS", "2048")
    with cat.AttnPlan(n, 1, hq, 1, dh, "f32") as plan:
        o2, lse2 = plan.forward(q, k, v, cu)
        plan.sync()
        dq2, dk2, dv2 = plan.backward(q, k, v, o2, lse2, do, cu)
        plan.sync()
    assert torch.equal(lse2[:, :last], lse[:, :last])
    assert torch.equal(o2[:last], o[:last]) and torch.equal(dq2[:last], dq[:last])
    if which is None:
        for a, b in ((o2, o), (lse2, lse), (dq2, dq), (dk2, dk), (dv2, dv)):
            assert torch.equal(a, b)
        return
    keep = [x for x in range(dh) if x != c]
    # Some rows and keys that were computed one by one, against 64 bits.  A score
    # is off by (dh + 4) steps of its absolute products, an exponential by four
    # steps of its exponent's terms more, a sum of N products by N + 8 steps.
    H, sc = 2.0 ** -24, dh ** -0.5
    if which == "v":
        assert o2[at:, :, c].isnan().all() and dk2.isnan().all()
        for i in (last, last + 31, at - 1, n - 1):
            Q, K, V = q[i].double(), k[:i + 1, 0].double(), v[:i + 1, 0].double()[:, keep]
            s = sc * (Q @ K.T)
            p = torch.softmax(s, 1)
            es = (dh + 4) * H * sc * (Q.abs() @ K.abs().T) + 4 * H * (s.abs() + 1)
            ep = es + es.amax(1, keepdim=True) + 8 * H
            out = p @ V
            bound = (p * (ep + 2 * (n + 8) * H)) @ V.abs() + H * out.abs()
            assert ((o2[i][:, keep].double() - out).abs() <= bound).all(), i
    else:
        assert torch.equal(o2, o)
        assert dv2[:at + 1, :, c].isnan().all() and dk2[:at + 1].isnan().all()
        assert dk2[at + 1:].isfinite().all()
        for j in (5, last, at, n - 1):
            Q, D = q[j:].double(), do[j:].double()[:, :, keep]
            s = sc * (Q @ k[j, 0].double())                             # [rows, hq]
            L = lse[:, j:].T.double()
            p = torch.exp(s - L)
            ep = (dh + 4) * H * sc * (Q.abs() @ k[j, 0].double().abs()) + \
                4 * H * (s.abs() + L.abs() + 1)
            want = (p[:, :, None] * D).sum((0, 1))
            bound = ((p * (ep + (hq * n + 8) * H))[:, :, None] * D.abs()).sum((0, 1)) + \
                H * want.abs()
            assert ((dv2[j, 0, keep].double() - want).abs() <= bound).all(), j


def test_clip_holds_the_tensors_of_a_generator():
    # The tensors that a generator makes live until the call has used them: the
    # norm that the call allocates does not take their place.
    sizes = [5, 100, 3, 77]
    host = [torch.randn(n, generator=torch.Generator().manual_seed(n)) for n in sizes]
    want, outs = ref.clip(host, 0.5)
    grads = [t.to(DEV) for t in host]
    to = [torch.empty_like(t) for t in grads]
    with cat.ClipPlan(sizes, ["f32"] * 4) as plan:
        for _ in range(3):
            check("norm", plan.norm(t * 1.0 for t in grads), want)
            n = plan.clip((t * 1.0 for t in grads), 0.5, out=(t for t in to))
            plan.sync()
            check("norm", n, want)
            for t, o in zip(to, outs):
                check("out", t, o)
                t.zero_()
        with pytest.raises(TypeError):
            plan.norm(3)
        with pytest.raises(ValueError):
            plan.norm(t for t in grads[:2])
