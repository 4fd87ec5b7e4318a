"""GPU tests of the operators around a CAT layer: softmax attention over
packed sequences, layer norm, gradient norm and clipping, each against a plain
64-bit implementation with bounds counted in rounding steps, and together in
a training step of a CAT-Alter pair of layers."""
import math

import numpy as np
import pytest
import torch

import fft_circulant_attention_gb300 as cat
import _block_ref as ref
from _block_ref import TORCH, check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _built(cuda_device):
    from fft_circulant_attention_gb300 import build
    build.build()
    cat.lib()
    yield
    torch.cuda.synchronize()


def run_attn(q, k, v, do, cu, causal, dtype, scale=None, backward=True):
    T, hq, dh = q.shape
    hkv = k.shape[1]
    qd, kd, vd, dd, cd = (t.to(DEV) for t in (q, k, v, do, cu))
    with cat.AttnPlan(T, len(cu) - 1, hq, hkv, dh, dtype, causal=causal, scale=scale) as plan:
        o, lse = plan.forward(qd, kd, vd, cd)
        out = dict(o=o, lse=lse)
        if backward:
            out["dq"], out["dk"], out["dv"] = plan.backward(qd, kd, vd, o, lse, dd, cd)
        plan.sync()
    return out


def attn_parity(lens, hq, hkv, dh, dtype, causal, seed=0, scale=None, sharp=1.0, extra=0):
    q, k, v, do, cu = ref.attn_inputs(lens, hq, hkv, dh, dtype, seed, extra, sharp)
    got = run_attn(q, k, v, do, cu, causal, dtype, scale)
    want = ref.attention(q, k, v, do, cu, causal, dtype, scale)
    for n, r in want.items():
        check(n, got[n], r)


LENS = [
    [1], [2, 1, 3], [64], [63, 65], [128], [127, 129, 1], [256], [255, 257], [300, 0, 17, 0],
    [513, 2, 200],
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=lambda v: "-".join(map(str, v)))
def test_attn_lengths(lens, dtype, causal):
    attn_parity(lens, 4, 2, 64, dtype, causal, seed=sum(lens))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv,dh", [
    (1, 1, 1), (3, 1, 5), (2, 2, 8), (4, 4, 16), (2, 1, 24), (2, 1, 33), (6, 3, 40), (2, 2, 72),
    (2, 1, 80), (3, 3, 96), (2, 1, 100), (4, 1, 128), (8, 2, 128), (12, 12, 64),
])
def test_attn_heads(hq, hkv, dh, dtype):
    attn_parity([150, 61], hq, hkv, dh, dtype, True, seed=dh)
    attn_parity([150, 61], hq, hkv, dh, dtype, False, seed=dh + 1)


@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_attn_longer(dtype, dh, causal):
    attn_parity([1111, 640, 383], 2, 1, dh, dtype, causal, seed=5)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,dh", [
    ([4096], 64), ([4097], 64), ([4351], 64), ([5003, 3200], 64), ([4500], 40), ([4200, 4000], 8),
], ids=str)
def test_attn_long_sequences(lens, dh, causal):
    # From 4096 rows a sequence (on average) a CTA of the bf16 forward takes
    # two tiles of rows; sequences that end in either tile.
    attn_parity(lens, 2, 1, dh, "bf16", causal, seed=sum(lens) + dh)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("at", [3, 4100, 4239, 4299])
def test_attn_long_masked_values_do_not_leak(value, at):
    # As in short sequences: a value of one token reaches the rows that see it.
    n = 4300
    q, k, v, do, cu = ref.attn_inputs([n], 1, 1, 64, "bf16", 12, extra=30)
    val, b = ref.attention(q, k, v, do, cu, True, "bf16")["o"]
    for which in ("k", "v"):
        t = dict(k=k.clone(), v=v.clone())
        for x in t.values():
            x[n:] = value
        t[which][at, :, 3] = value
        got = run_attn(q, t["k"], t["v"], do, cu, True, "bf16", backward=False)
        check("o", got["o"][:at], (val[:at], b[:at]))
        if which == "v":
            assert not got["o"][at:n, 0, 3].isfinite().any()
            check("o", got["o"][at:n, 0, 4:], (val[at:n, 0, 4:], b[at:n, 0, 4:]))


@pytest.mark.parametrize("lens", [[300], [4400]])
def test_attn_full_masked_tail(lens):
    # Not causal: what lies behind the sequence, in its last block, is not read.
    n = lens[0]
    q, k, v, do, cu = ref.attn_inputs(lens, 2, 2, 64, "bf16", 13, extra=200)
    want = ref.attention(q, k, v, do, cu, False, "bf16")
    for t in (q, k, v, do):
        t[n:] = math.inf
    got = run_attn(q, k, v, do, cu, False, "bf16")
    for name in want:
        check(name, got[name], want[name])


def test_attn_f32_wide_heads_masked_values_do_not_leak():
    # fp32 rows wider than 64, forward and backward.
    n, at = 200, 130
    q, k, v, do, cu = ref.attn_inputs([n, 40], 2, 1, 96, "f32", 14)
    want = ref.attention(q, k, v, do, cu, True, "f32")
    for which in ("k", "v"):
        t = dict(k=k.clone(), v=v.clone())
        t[which][at, :, 70] = math.nan
        got = run_attn(q, t["k"], t["v"], do, cu, True, "f32")
        for name in ("o", "dq"):
            for rows in (slice(0, at), slice(n, None)):
                check(name, got[name][rows], tuple(x[rows] for x in want[name]))
        for name in ("dk", "dv"):
            check(name, got[name][n:], tuple(x[n:] for x in want[name]))
        assert not got["o"][at:n, :, 70 if which == "v" else 0].isfinite().any()


@pytest.mark.parametrize("dh", [3, 33, 40, 64])
@pytest.mark.parametrize("causal", [True, False])
def test_attn_f32_odd_widths_with_a_nan(dh, causal):
    # Rows that are computed again by the definition, whatever their alignment:
    # those that do not see the token's value keep theirs.
    n, at = 300, 170
    lens = [n, 50]
    q, k, v, do, cu = ref.attn_inputs(lens, 2, 1, dh, "f32", 15)
    want = ref.attention(q, k, v, do, cu, causal, "f32")
    c = dh - 1
    for which in ("v", "do"):
        t = dict(v=v.clone(), do=do.clone())
        t[which][at, :, c] = math.nan
        got = run_attn(q, k, t["v"], t["do"], cu, causal, "f32")
        if which == "v":
            rows = torch.ones(350, dtype=torch.bool)
            rows[at if causal else 0:n] = False
            for name in ("o", "dq"):
                check(name, got[name][rows.to(DEV)], tuple(x[rows] for x in want[name]))
            # The other columns of o are as they were in every row.
            check("o", got["o"][..., :c], tuple(x[..., :c] for x in want["o"]))
            assert got["o"][at:n, :, c].isnan().all()
        else:
            check("o", got["o"], want["o"])
            rows = torch.ones(350, dtype=torch.bool)
            rows[at] = False
            check("dq", got["dq"][rows.to(DEV)], tuple(x[rows] for x in want["dq"]))
            check("dv", got["dv"][..., :c], tuple(x[..., :c] for x in want["dv"]))
            assert got["dv"][:at + 1, :, c].isnan().all()
        for name in ("dk", "dv"):
            check(name, got[name][n:], tuple(x[n:] for x in want[name]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_two_plans_on_two_streams(dtype):
    # Each plan has its own workspace: calls that run at the same time.
    lens = [333, 90, 257]
    q, k, v, do, cu = ref.attn_inputs(lens, 4, 2, 64, dtype, 15)
    ins = [t.to(DEV) for t in (q, k, v, do)]
    cd = cu.to(DEV)
    want = run_attn(q, k, v, do, cu, True, dtype)
    T = q.shape[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    plans = [cat.AttnPlan(T, 3, 4, 2, 64, dtype, stream=s) for s in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s, plan in zip(streams, plans):
            with torch.cuda.stream(s):
                o, lse = plan.forward(*ins[:3], cd)
                got.append((o, lse) + tuple(plan.backward(*ins[:3], o, lse, ins[3], cd)))
    torch.cuda.synchronize()
    for r in got:
        for name, t in zip(("o", "lse", "dq", "dk", "dv"), r):
            assert torch.equal(t, want[name]), name
    for plan in plans:
        plan.close()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [31, 128, 129, 300])
def test_attn_many_sequences(S, dtype, causal):
    # Blocks are taken largest first up to 128 sequences, as they lie beyond;
    # empty sequences among them, and lengths either side of a block.
    r = np.random.default_rng(S)
    lens = r.integers(0, 90, S)
    lens[r.integers(0, S, S // 8)] = 0
    lens[r.integers(0, S, 4)] = [127, 128, 129, 260]
    attn_parity([int(n) for n in lens], 2, 1, 64, dtype, causal, seed=S)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_many_wide_heads(dtype):
    attn_parity([40, 0, 130, 3] * 40, 2, 2, 128, dtype, True, seed=6)


def test_plans_with_a_stream_of_their_own():
    # Outputs that a call allocates belong to the plan's stream.
    n = 1 << 22
    s = torch.cuda.Stream()
    x = torch.randn(n // 64, 64, device=DEV)
    g = [torch.randn(1000, device=DEV)]
    torch.cuda.synchronize()
    with cat.LayerNormPlan(n // 64, 64, "f32", stream=s) as plan, \
            cat.ClipPlan([1000], ["f32"], stream=s.cuda_stream) as clip:
        want = torch.nn.functional.layer_norm(x, (64,))
        ok = []
        for _ in range(10):
            # Work on the default stream whose memory is free again behind it.
            t = x * 3.0
            for _ in range(4):
                t = t * 0.5
            del t
            y, _, _ = plan.forward(x)
            total = clip.norm(g)
            s.synchronize()
            ok.append(torch.allclose(y, want, atol=1e-4))
            assert abs(float(total) - float(g[0].norm())) < 1e-3
            plan.sync()
        assert all(ok)
    with cat.ClipPlan([1000], ["f32"], stream=0) as clip:      # the default stream
        assert abs(float(clip.norm(g)) - float(g[0].norm())) < 1e-3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_peaked_and_scaled(dtype):
    # Near one-hot rows: scores of some tens; and a scale of the caller's own.
    attn_parity([200, 77], 2, 2, 64, dtype, True, seed=3, sharp=8.0)
    attn_parity([200, 77], 2, 2, 64, dtype, False, seed=4, scale=0.7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_rising_scores(dtype):
    # Keys whose scores grow along the sequence, and ones that fall: the
    # running maximum moves at every block, or never again.
    n = 700
    q, k, v, do, cu = ref.attn_inputs([n], 2, 2, 64, dtype, 9)
    ramp = torch.linspace(-12, 12, n)[:, None]
    for sign in (1.0, -1.0):
        q[:, :, 0] = 8.0
        k[:, :, 0] = (sign * ramp).to(k.dtype)
        for causal in (True, False):
            got = run_attn(q, k, v, do, cu, causal, dtype)
            for name, r in ref.attention(q, k, v, do, cu, causal, dtype).items():
                check(name, got[name], r)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_rows_outside_the_sequences(dtype):
    # NaN in every row that no sequence holds, before, behind: no result
    # changes, and the outputs' rows there keep what they held.
    q, k, v, do, cu = ref.attn_inputs([70, 130], 2, 1, 64, dtype, 1, extra=45)
    cu = cu + 13
    for t in (q, k, v, do):
        t[:13] = math.nan
        t[213:] = math.nan
    T = q.shape[0]
    ins = [t.to(DEV) for t in (q, k, v, do)]
    cd = cu.to(DEV)
    mark = 7.0
    o = torch.full((T, 2, 64), mark, dtype=TORCH[dtype], device=DEV)
    lse = torch.full((2, T), mark, device=DEV)
    dq, dk, dv = (torch.full_like(t, mark) for t in ins[:3])
    with cat.AttnPlan(T + 50, 7, 2, 1, 64, dtype) as plan:
        plan.forward(*ins[:3], cd, O=o, lse=lse)
        # (what a layer in front would leave in O's other rows is not read)
        o2 = o.clone()
        o2[:13] = math.nan
        o2[213:] = math.nan
        l2 = lse.clone()
        l2[:, :13] = math.nan
        l2[:, 213:] = math.nan
        plan.backward(*ins[:3], o2, l2, ins[3], cd, dQ=dq, dK=dk, dV=dv)
        plan.sync()
    q, k, v, do = (t.nan_to_num(0.0) for t in (q, k, v, do))
    want = ref.attention(q, k, v, do, cu, True, dtype)
    for name, t in dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv).items():
        check(name, t, want[name])
        rows = t if name != "lse" else t.T
        assert (rows[:13] == mark).all() and (rows[213:] == mark).all(), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [5, 64, 100, 130, 199])
def test_attn_masked_values_do_not_leak(dtype, value, at):
    # A value of one token reaches only the rows that see the token, whichever
    # block it shares with rows that do not.
    lens = [200, 90]
    q, k, v, do, cu = ref.attn_inputs(lens, 2, 1, 64, dtype, 2)
    clean = ref.attention(q, k, v, do, cu, True, dtype)
    for which in ("k", "v", "q", "do"):
        t = dict(q=q.clone(), k=k.clone(), v=v.clone(), do=do.clone())
        t[which][at, :, 3] = value
        got = run_attn(t["q"], t["k"], t["v"], t["do"], cu, True, dtype)
        val, b = clean["o"]
        # Query rows before `at` do not see it (and q or dO of a later row is
        # not theirs), rows of the second sequence neither.
        rows = torch.ones(290, dtype=torch.bool)
        rows[at:200] = False
        if which in ("q", "do"):
            rows[at:200] = True
            rows[at] = which == "do"
        check("o", got["o"][rows.to(DEV)], (val[rows], b[rows]))
        # dq of the unaffected rows.
        rows = torch.ones(290, dtype=torch.bool)
        rows[at:200] = which in ("q", "do")
        rows[at] = False
        val, b = clean["dq"]
        check("dq", got["dq"][rows.to(DEV)], (val[rows], b[rows]))
        # dk and dv: a query row at `at` reaches keys up to `at` only; a bad
        # key row reaches every key through the rows that see it.
        keys = torch.ones(290, dtype=torch.bool)
        keys[:200] = False
        if which in ("q", "do"):
            keys[at + 1:200] = True
        for name in ("dk", "dv"):
            val, b = clean[name]
            check(name, got[name][keys.to(DEV)], (val[keys], b[keys]))
        # What does see the value is not finite: nothing was dropped on the way.
        if which == "v":
            assert not got["o"][at:200, :, 3].isfinite().any()
            assert got["o"][at:200, :, 4].isfinite().all()
        if which == "do":
            assert not got["dv"][:at + 1, 0, 3].isfinite().any()
            assert got["dv"][:at + 1, 0, 4].isfinite().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_columns_of_one_buffer(dtype):
    # q, k, v and their gradients as columns of one wide row, as a fused
    # projection lays them out.
    hq, hkv, dh = 4, 2, 64
    lens = [100, 33, 160]
    q, k, v, do, cu = ref.attn_inputs(lens, hq, hkv, dh, dtype, 8)
    T = q.shape[0]
    wide = torch.cat([q, k, v], 1).to(DEV)
    grad = torch.full_like(wide, 5.0)
    sl = (slice(0, hq), slice(hq, hq + hkv), slice(hq + hkv, None))
    cd = cu.to(DEV)
    with cat.AttnPlan(T, len(lens), hq, hkv, dh, dtype) as plan:
        o, lse = plan.forward(wide[:, sl[0]], wide[:, sl[1]], wide[:, sl[2]], cd)
        plan.backward(*(wide[:, s] for s in sl), o, lse, do.to(DEV), cd,
                      dQ=grad[:, sl[0]], dK=grad[:, sl[1]], dV=grad[:, sl[2]])
        plan.sync()
    want = ref.attention(q, k, v, do, cu, True, dtype)
    check("o", o, want["o"])
    for name, s in zip(("dq", "dk", "dv"), sl):
        check(name, grad[:, s], want[name])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attn_rows_at_odd_addresses(dtype):
    # Rows that start on no 16-byte boundary (a view one element in, an odd
    # row stride) give the same values.
    q, k, v, do, cu = ref.attn_inputs([97, 40], 2, 2, 64, dtype, 6)
    T = q.shape[0]

    def odd(t, lead=1, pad=3):
        w = t.shape[1] * t.shape[2]
        buf = torch.zeros(T * (w + pad) + lead, dtype=t.dtype, device=DEV)
        view = torch.as_strided(buf, t.shape, (w + pad, t.shape[2], 1), lead)
        view.copy_(t)
        return view

    with cat.AttnPlan(T, 2, 2, 2, 64, dtype) as plan:
        args = [odd(t) for t in (q, k, v)]
        o, lse = plan.forward(*args, cu.to(DEV))
        grads = plan.backward(*args, o, lse, do.to(DEV), cu.to(DEV), dQ=odd(q, 1, 5),
                              dK=odd(k, 3, 1), dV=odd(v, 5, 7))
        plan.sync()
    want = ref.attention(q, k, v, do, cu, True, dtype)
    for name, t in zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + grads):
        check(name, t, want[name])


def test_attn_long_rows_pass_32_bits():
    # Row offsets beyond 2^31 elements: three short sequences in a tall buffer
    # of wide rows, the last one near its end.
    hq, dh, ld = 1, 64, 65536
    T = 33000
    buf = torch.empty((T, ld), dtype=torch.bfloat16, device=DEV)
    q, k, v = (torch.as_strided(buf, (T, 1, 64), (ld, 64, 1), 64 * i) for i in range(3))
    n = 200
    cq, ck, cv, cdo, _ = ref.attn_inputs([n], 1, 1, 64, "bf16", 4)
    start = T - n - 3
    for t, c in ((q, cq), (k, ck), (v, cv)):
        t[start:start + n] = c.to(DEV)
    do = torch.zeros((T, 1, 64), dtype=torch.bfloat16, device=DEV)
    do[start:start + n] = cdo.to(DEV)
    cu = torch.tensor([start, start + n], dtype=torch.int32, device=DEV)
    with cat.AttnPlan(T, 1, hq, 1, dh, "bf16") as plan:
        o, lse = plan.forward(q, k, v, cu)
        grads = plan.backward(q, k, v, o, lse, do, cu)
        plan.sync()
    want = ref.attention(cq, ck, cv, cdo, torch.tensor([0, n]), True, "bf16")
    rows = slice(start, start + n)
    check("o", o[rows], want["o"])
    for name, t in zip(("dq", "dk", "dv"), grads):
        check(name, t[rows], want[name])


def test_attn_repeats_and_streams():
    # Bit-identical on repetition, on another stream, and replayed from a
    # graph whose sequences change between replays.
    q, k, v, do, cu = ref.attn_inputs([300, 212, 88], 4, 2, 64, "bf16", 12)
    ins = [t.to(DEV) for t in (q, k, v, do)]
    cd = cu.to(DEV)
    T = q.shape[0]
    plan = cat.AttnPlan(T, 3, 4, 2, 64, "bf16")

    def step(c):
        o, lse = plan.forward(*ins[:3], c)
        return (o, lse) + plan.backward(*ins[:3], o, lse, ins[3], c)

    first = step(cd)
    for a, b in zip(first, step(cd)):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = step(cd)
    side.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    cu_g = cd.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(cu_g)
    for lens in ([300, 212, 88], [1, 598, 1], [0, 600, 0]):
        c = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32)
        cu_g.copy_(c.to(DEV))
        graph.replay()
        torch.cuda.synchronize()
        want = step(c.to(DEV))
        plan.sync()
        for a, b in zip(held, want):
            assert torch.equal(a, b)
    plan.close()


@pytest.mark.parametrize("bad", [[0, 50, 20, 100], [0, 50, 101, 100], [-4, 20, 60, 100],
                                 [0, 40, 80, 120]])
def test_attn_bad_sequences_are_reported(bad):
    q, k, v, do, _ = ref.attn_inputs([100], 2, 2, 64, "bf16", 7)
    ins = [t.to(DEV) for t in (q, k, v, do)]
    cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
    plan = cat.AttnPlan(100, 3, 2, 2, 64, "bf16")
    plan.forward(*ins[:3], cu)
    with pytest.raises(cat.CatError) as e:
        plan.sync()
    assert e.value.status == cat.CAT_ERR_DEVICE_STATUS
    plan.sync()                                   # reported once, then clear
    good = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    o, lse = plan.forward(*ins[:3], good)
    plan.sync()
    want = ref.attention(q, k, v, do, torch.tensor([0, 100]), True, "bf16")
    check("o", o, want["o"])
    plan.close()


def test_attn_refusals():
    lib = cat.lib()
    T, hq, hkv, dh = 32, 4, 2, 64
    t = lambda h: torch.zeros((T, h, dh), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    q, k, v, o, do, dq, dk, dv = t(4), t(2), t(2), t(4), t(4), t(4), t(2), t(2)
    lse = torch.zeros((hq, T), device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    p = cat.cat_plan_create_attn(T, 2, hq, hkv, dh, "bf16")
    a = lambda x: x.data_ptr() if torch.is_tensor(x) else x  # noqa: E731

    def fwd(q=q, k=k, v=v, o=o, lse=lse, cu=cu, T=T, S=1, l=(256, 128, 128)):
        return lib.cat_attn_forward(p, a(q), a(k), a(v), a(o), a(lse), a(cu), T, S, *l)

    def bwd(q=q, k=k, v=v, o=o, lse=lse, do=do, dq=dq, dk=dk, dv=dv, cu=cu, T=T, S=1,
            l=(256, 128, 128, 256, 128, 128)):
        return lib.cat_attn_backward(p, a(q), a(k), a(v), a(o), a(lse), a(do), a(dq), a(dk),
                                     a(dv), a(cu), T, S, *l)

    assert fwd() == cat.CAT_OK and bwd() == cat.CAT_OK
    assert fwd(T=0) == cat.CAT_OK and fwd(S=0) == cat.CAT_OK and bwd(T=0) == cat.CAT_OK
    assert fwd(T=T + 1) == cat.CAT_ERR_PLAN_MISMATCH and fwd(S=3) == cat.CAT_ERR_PLAN_MISMATCH
    assert fwd(T=-1) == cat.CAT_ERR_INVALID_ARG and fwd(S=-1) == cat.CAT_ERR_INVALID_ARG
    for n in ("q", "k", "v", "o", "lse", "cu"):
        assert fwd(**{n: None}) == cat.CAT_ERR_INVALID_ARG, n
        x = dict(q=q, k=k, v=v, o=o, lse=lse, cu=cu)[n]
        assert fwd(**{n: x.data_ptr() + 1}) == cat.CAT_ERR_MISALIGNED, n
    for n in ("o", "lse", "do", "dq", "dk", "dv"):
        assert bwd(**{n: None}) == cat.CAT_ERR_INVALID_ARG, n
    assert bwd(dq=dq.data_ptr() + 1) == cat.CAT_ERR_MISALIGNED
    assert fwd(l=(255, 128, 128)) == cat.CAT_ERR_INVALID_ARG
    assert fwd(l=(256, 127, 128)) == cat.CAT_ERR_INVALID_ARG
    assert fwd(l=(256, 128, 2**62)) == cat.CAT_ERR_INVALID_ARG
    assert bwd(l=(256, 128, 128, 256, 128, 1)) == cat.CAT_ERR_INVALID_ARG
    assert fwd(o=q) == cat.CAT_ERR_ALIAS and fwd(lse=v) == cat.CAT_ERR_ALIAS
    assert fwd(o=q.data_ptr() + 128) == cat.CAT_ERR_ALIAS
    assert bwd(dq=do) == cat.CAT_ERR_ALIAS and bwd(dk=dv) == cat.CAT_ERR_ALIAS
    assert bwd(dk=k) == cat.CAT_ERR_ALIAS
    # The other families' calls refuse this plan, and this one's refuse theirs.
    mm = cat.CAT_ERR_PLAN_MISMATCH
    x = a(q)
    assert lib.cat_forward(p, x, x, x, x, 0, 0, 0, 0, 1) == mm
    assert lib.cat_backward(p, x, x, x, x, x, x, x, 0, 0, 0, 0, 1) == mm
    assert lib.cat2d_forward(p, x, x, x, x, 0, 0, 0, 0, 0, 1) == mm
    assert lib.cat_plan_timing(p, 4) == mm
    assert lib.cat_layernorm_forward(p, x, None, None, x, x, x, 1) == mm
    assert lib.cat_grad_norm(p, None, x) == mm
    cat.cat_plan_destroy(p)
    p = cat.cat_plan_create(1, 64, 64, 1, "f32")
    assert fwd() == mm and bwd() == mm
    cat.cat_plan_destroy(p)
    with cat.AttnPlan(T, 2, hq, hkv, dh, "bf16") as plan:
        with pytest.raises(ValueError):
            plan.forward(q.float(), k, v, cu)
        with pytest.raises(ValueError):
            plan.forward(q[:, :, ::2], k, v, cu)
        with pytest.raises(ValueError):
            plan.forward(q, k[:-1], v, cu)
        with pytest.raises(ValueError):
            plan.forward(q, k, v, cu.long())
        with pytest.raises(ValueError):
            plan.forward(q, k, v, cu.cpu())
        with pytest.raises(ValueError):
            plan.forward(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, cu)


# ---------------------------------------------------------------- layer norm


def ln_inputs(rows, D, dtype, seed, offset=0.7):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, D), generator=g) * 1.3 + offset
    w = 1 + 0.3 * torch.randn(D, generator=g)
    b = 0.2 * torch.randn(D, generator=g)
    dy = torch.randn((rows, D), generator=g)
    return tuple(t.to(TORCH[dtype]) for t in (x, w, b, dy))


def ln_parity(rows, D, dtype, seed=0, offset=0.7, eps=1e-5, weights=True):
    x, w, b, dy = ln_inputs(rows, D, dtype, seed, offset)
    if not weights:
        w = b = None
    want = ref.layernorm(x, w, b, dy, eps, dtype)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    with cat.LayerNormPlan(rows, D, dtype, eps=eps) as plan:
        y, mean, rstd = plan.forward(dev(x), dev(w), dev(b))
        m, r = want["mean"][0].float().to(DEV), want["rstd"][0].float().to(DEV)
        dx, dg, db = plan.backward(dev(x), dev(w), m, r, dev(dy))
        plan.sync()
    for n, t in dict(y=y, mean=mean, rstd=rstd, dx=dx, dgamma=dg, dbeta=db).items():
        check(n, t, want[n])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 31, 64, 77, 250, 256, 257, 768, 1000, 1021, 1024,
                               1025, 1026, 2048, 2049, 2056, 4100, 8191, 8192])
def test_layernorm_widths(D, dtype):
    # (A single column normalises to zero: the variance is zero, eps counts.)
    ln_parity(37, D, dtype, seed=D)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 300, 5000])
def test_layernorm_rows(rows, dtype):
    ln_parity(rows, 96, dtype, seed=rows)
    ln_parity(rows, 1030, dtype, seed=rows)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layernorm_offsets_and_missing_weights(dtype):
    # A mean a thousand times the spread: centred before squaring.
    ln_parity(20, 512, dtype, seed=1, offset=1000.0, eps=1e-6)
    ln_parity(20, 512, dtype, seed=2, weights=False)
    ln_parity(20, 1536, dtype, seed=2, weights=False, eps=0.0)


def test_layernorm_one_weight_only():
    x, w, b, dy = (t.to(DEV) for t in ln_inputs(9, 64, "f32", 3))
    with cat.LayerNormPlan(9, 64, "f32") as plan:
        full, mean, rstd = plan.forward(x, w, b)
        only_w = plan.forward(x, w, None)[0]
        only_b = plan.forward(x, None, b)[0]
        dx, dg, db = plan.backward(x, w, mean, rstd, dy)
        g = torch.empty_like(w)
        d2 = torch.empty_like(x)
        cat.cat_layernorm_backward(plan.handle, x, w, mean, rstd, dy, d2, g, None, 9)
        d3 = torch.empty_like(x)
        cat.cat_layernorm_backward(plan.handle, x, w, mean, rstd, dy, d3, None, None, 9)
        plan.sync()
    assert torch.equal(g, dg) and torch.equal(d2, dx) and torch.equal(d3, dx)
    x64, w64, b64 = (t.double().cpu() for t in (x, w, b))
    xh = (x64 - x64.mean(-1, keepdim=True)) / torch.sqrt(
        x64.var(-1, unbiased=False, keepdim=True) + 1e-5)
    assert (only_w.double().cpu() - xh * w64).abs().max() < 1e-5
    assert (only_b.double().cpu() - (xh + b64)).abs().max() < 1e-5


def test_layernorm_no_rows_and_batches():
    with cat.LayerNormPlan(24, 48, "bf16") as plan:
        x = torch.empty((0, 48), dtype=torch.bfloat16, device=DEV)
        w = torch.ones(48, dtype=torch.bfloat16, device=DEV)
        y, mean, rstd = plan.forward(x, w, w)
        dx, dg, db = plan.backward(x, w, mean, rstd, y)
        assert y.shape == (0, 48) and (dg == 0).all() and (db == 0).all()
        x = torch.randn((2, 3, 4, 48), device=DEV).bfloat16()
        y, mean, rstd = plan.forward(x, w, w)
        assert y.shape == x.shape and mean.shape == (2, 3, 4)
        flat = plan.forward(x.view(24, 48), w, w)[0]
        plan.sync()
        assert torch.equal(flat.view_as(y), y)


def test_layernorm_repeats_and_graph():
    x, w, b, dy = (t.to(DEV) for t in ln_inputs(3001, 768, "bf16", 5))
    plan = cat.LayerNormPlan(3001, 768, "bf16")

    def step():
        y, mean, rstd = plan.forward(x, w, b)
        return (y,) + plan.backward(x, w, mean, rstd, dy)

    first = step()
    for a, c in zip(first, step()):
        assert torch.equal(a, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, c in zip(first, held):
        assert torch.equal(a, c)
    plan.close()


def test_layernorm_nan_stays_in_its_row():
    x, w, b, dy = (t.to(DEV) for t in ln_inputs(17, 200, "f32", 6))
    with cat.LayerNormPlan(17, 200, "f32") as plan:
        clean = plan.forward(x, w, b)[0]
        x[4, 7] = math.nan
        x[9, 0] = math.inf
        y = plan.forward(x, w, b)[0]
        plan.sync()
    rows = [r for r in range(17) if r not in (4, 9)]
    assert torch.equal(y[rows], clean[rows])
    assert not y[4].isfinite().any() and not y[9].isfinite().any()


def test_layernorm_refusals():
    lib = cat.lib()
    x, w, b, dy = (t.to(DEV) for t in ln_inputs(8, 64, "f32", 0))
    y, dx, dg, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    mean, rstd = torch.empty(8, device=DEV), torch.empty(8, device=DEV)
    p = cat.cat_plan_create_layernorm(8, 64, "f32")
    a = lambda t: t.data_ptr() if torch.is_tensor(t) else t  # noqa: E731

    def fwd(x=x, w=w, b=b, y=y, mean=mean, rstd=rstd, rows=8):
        return lib.cat_layernorm_forward(p, a(x), a(w), a(b), a(y), a(mean), a(rstd), rows)

    def bwd(x=x, w=w, mean=mean, rstd=rstd, dy=dy, dx=dx, dg=dg, db=db, rows=8):
        return lib.cat_layernorm_backward(p, a(x), a(w), a(mean), a(rstd), a(dy), a(dx), a(dg),
                                          a(db), rows)

    assert fwd() == cat.CAT_OK and bwd() == cat.CAT_OK and fwd(rows=0) == cat.CAT_OK
    assert fwd(rows=9) == cat.CAT_ERR_PLAN_MISMATCH and fwd(rows=-1) == cat.CAT_ERR_INVALID_ARG
    for n in ("x", "y", "mean", "rstd"):
        assert fwd(**{n: None}) == cat.CAT_ERR_INVALID_ARG
    for n in ("x", "mean", "rstd", "dy", "dx"):
        assert bwd(**{n: None}) == cat.CAT_ERR_INVALID_ARG
    assert fwd(x=x.data_ptr() + 4) == cat.CAT_ERR_MISALIGNED
    assert fwd(w=w.data_ptr() + 8) == cat.CAT_ERR_MISALIGNED
    assert bwd(dg=dg.data_ptr() + 4) == cat.CAT_ERR_MISALIGNED
    assert fwd(mean=mean.data_ptr() + 2) == cat.CAT_ERR_MISALIGNED
    assert fwd(y=x) == cat.CAT_ERR_ALIAS and fwd(mean=rstd) == cat.CAT_ERR_ALIAS
    assert bwd(dx=dy) == cat.CAT_ERR_ALIAS and bwd(dg=db) == cat.CAT_ERR_ALIAS
    assert bwd(dg=w) == cat.CAT_ERR_ALIAS
    cat.cat_plan_destroy(p)
    with cat.LayerNormPlan(8, 64, "f32") as plan:
        for bad in (x.bfloat16(), x[:, :32], x.cpu(), x.t().contiguous().t()):
            with pytest.raises(ValueError):
                plan.forward(bad, w, b)
        with pytest.raises(ValueError):
            plan.forward(x, w[:32], b)


# ------------------------------------------------------------------- clipping


def clip_inputs(shapes, seed=0, scale=1e-2):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * scale * 10 ** (i % 3)).to(TORCH[d])
            for i, (s, d) in enumerate(shapes)]


SHAPES = {
    "one": [((1,), "f32")],
    "odd": [((3,), "bf16"), ((17, 5), "f32"), ((1001,), "bf16"), ((0,), "f32"), ((4097,), "f32")],
    "chunks": [((16384,), "bf16"), ((16385,), "bf16"), ((8192,), "f32"), ((8191,), "f32"),
               ((300, 517), "bf16"), ((700, 333), "f32")],
    "many": [((7 + i % 40,), "f32" if i % 3 else "bf16") for i in range(130)],
    "more": [((1 + i % 9,), "f32" if i % 2 else "bf16") for i in range(2300)],
}


@pytest.mark.parametrize("bound", [0.0, 0.25, 3.0, math.inf])
@pytest.mark.parametrize("shapes", sorted(SHAPES))
def test_clip(shapes, bound):
    host = clip_inputs(SHAPES[shapes], seed=len(shapes))
    norm = math.sqrt(sum(float(t.double().pow(2).sum()) for t in host))
    most = bound * norm
    want_norm, want = ref.clip(host, most)
    grads = [t.to(DEV) for t in host]
    with cat.ClipPlan([t.numel() for t in host], [t.dtype for t in host]) as plan:
        check("norm", plan.norm(grads), want_norm)
        outs = [torch.empty_like(t) for t in grads]
        n = plan.clip(grads, most, out=outs)
        check("norm", n, want_norm)
        for i, (t, r) in enumerate(zip(outs, want)):
            check("out %d" % i, t, r)
        for t, h in zip(grads, host):
            assert torch.equal(t.cpu(), h)               # the inputs are as they were
        plan.clip(grads, most)                           # in place
        plan.sync()
        for t, o in zip(grads, outs):
            assert torch.equal(t, o)


def test_clip_views_at_odd_addresses():
    flat = torch.randn(5000, device=DEV).bfloat16()
    out = torch.zeros(5000, device=DEV).bfloat16()
    cuts = [1, 8, 23, 1024, 1031, 4999]
    grads = [flat[a:b] for a, b in zip(cuts[:-1], cuts[1:])]
    outs = [out[a:b] for a, b in zip(cuts[:-1], cuts[1:])]
    want_norm, want = ref.clip([t.cpu() for t in grads], 2.0)
    with cat.ClipPlan([t.numel() for t in grads], ["bf16"] * 5) as plan:
        n = plan.clip(grads, 2.0, out=outs)
        plan.sync()
    check("norm", n, want_norm)
    for t, r in zip(outs, want):
        check("out", t, r)
    assert out[0] == 0 and out[4999] == 0


@pytest.mark.parametrize("size", [1e-25, 1e-12, 1e12, 1e25])
def test_clip_far_from_one(size):
    # Squares outside fp32's range, tiny and huge values side by side.
    host = [torch.randn(1000) * size, torch.randn(33) * size * 1e-6]
    want_norm, want = ref.clip(host, size)
    with cat.ClipPlan([1000, 33], ["f32", "f32"]) as plan:
        grads = [t.to(DEV) for t in host]
        check("norm", plan.clip(grads, size), want_norm, tiny=0)
        plan.sync()
    for t, r in zip(grads, want):
        check("out", t, r, tiny=1e-37)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_clip_not_finite(value):
    g = torch.randn(20000, device=DEV)
    g[17777] = value
    before = g.clone()
    with cat.ClipPlan([20000], ["f32"]) as plan:
        out = [torch.empty_like(g)]
        n = plan.clip([g], 0.5, out=out)
        m = plan.clip([g], 0.5)
        plan.sync()
    assert not n.isfinite() and not m.isfinite()
    assert torch.equal(g.view(torch.int32), before.view(torch.int32))
    assert torch.equal(out[0].view(torch.int32), before.view(torch.int32))


def test_clip_zero_gradients_and_empty_lists():
    with cat.ClipPlan([100, 0], ["bf16", "f32"]) as plan:
        g = [torch.zeros(100, device=DEV).bfloat16(), torch.zeros(0, device=DEV)]
        n = plan.clip(g, 0.0)
        plan.sync()
        assert n == 0 and (g[0] == 0).all()
    with cat.ClipPlan([], []) as plan:
        n = torch.full((), 5.0, device=DEV)
        plan.clip([], 1.0, norm=n)
        plan.sync()
        assert n == 0
        n.fill_(5.0)
        plan.norm([], norm=n)
        plan.sync()
        assert n == 0


def test_clip_refusals():
    g = [torch.ones(64, device=DEV), torch.ones(64, device=DEV).bfloat16()]
    plan = cat.ClipPlan([64, 64], ["f32", "bf16"])
    n = torch.zeros((), device=DEV)

    def status(grads, outs, most=1.0, norm=n):
        with pytest.raises(cat.CatError) as e:
            cat.cat_grad_clip(plan.handle, grads, outs, most, norm)
        return e.value.status

    assert status(g, g, -1.0) == cat.CAT_ERR_INVALID_ARG
    assert status(g, g, math.nan) == cat.CAT_ERR_INVALID_ARG
    assert status([g[0], None], g) == cat.CAT_ERR_INVALID_ARG
    assert status(g, [g[0], None]) == cat.CAT_ERR_INVALID_ARG
    assert status(g, g, norm=None) == cat.CAT_ERR_INVALID_ARG
    assert status([g[0].data_ptr() + 2, g[1]], g) == cat.CAT_ERR_MISALIGNED
    assert status(g, [g[1], g[0]]) == cat.CAT_ERR_ALIAS
    assert status([g[0], g[0]], [g[0], g[0]]) == cat.CAT_ERR_ALIAS
    assert status(g, g, norm=g[0]) == cat.CAT_ERR_ALIAS
    big = torch.ones(200, device=DEV)
    assert status([big, g[1]], [big[4:], g[1]]) == cat.CAT_ERR_ALIAS
    with pytest.raises(ValueError):
        plan.clip(g[:1], 1.0)
    with pytest.raises(ValueError):
        plan.clip([g[1], g[0]], 1.0)
    with pytest.raises(ValueError):
        plan.clip([g[0][::2], g[1]], 1.0)
    with pytest.raises(cat.CatError) as e:
        plan.norm(g, norm=g[0].view(-1)[3])
    assert e.value.status == cat.CAT_ERR_ALIAS
    # Two tensors of one list may be the same for reading.
    same = cat.ClipPlan([64, 64], ["f32", "f32"])
    assert abs(float(same.norm([g[0], g[0]])) - math.sqrt(128)) < 1e-5
    same.close()
    plan.close()


def test_clip_repeats_and_graph():
    host = clip_inputs(SHAPES["chunks"], seed=3)
    grads = [t.to(DEV) for t in host]
    outs = [torch.empty_like(t) for t in grads]
    plan = cat.ClipPlan([t.numel() for t in host], [t.dtype for t in host])
    n0 = plan.clip(grads, 0.1, out=outs)
    keep = [t.clone() for t in outs]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n1 = plan.clip(grads, 0.1, out=outs)
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n0, n1)
        for a, b in zip(keep, outs):
            assert torch.equal(a, b)
    plan.close()


# ------------------------------------------------------- a CAT-Alter train step


def test_training_step_of_a_cat_alter_pair():
    """x + CAT(LN(x)), then x + attention(LN(x)) over packed documents, a
    linear loss, all gradients through the framework's backward calls and
    clipped together, against 64-bit autograd.

    Every operator is within some 1e-6 of its values in fp32 and the chain is
    ten operators long with weights of norm about one, so 1e-4 of each
    gradient's largest value bounds the whole.
    """
    B, N, D, H = 2, 128, 64, 4
    hkv, dh = 2, 16
    g = torch.Generator().manual_seed(0)
    rnd = lambda *s, f=1.0: (torch.randn(*s, generator=g, dtype=torch.float64) * f).float().double()  # noqa: E731,E501
    x = rnd(B, N, D)
    p = dict(g1=1 + rnd(D, f=0.1), b1=rnd(D, f=0.1), wa=rnd(D, H, f=D ** -0.5),
             wv=rnd(D, D, f=D ** -0.5), g2=1 + rnd(D, f=0.1), b2=rnd(D, f=0.1),
             wqkv=rnd(D, (H + 2 * hkv) * dh, f=D ** -0.5), wo=rnd(H * dh, D, f=D ** -0.5))
    r = rnd(B, N, D)
    lens = [100, 28, 1, 127]
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32)

    # 64-bit autograd.
    q = {n: t.clone().requires_grad_() for n, t in p.items()}
    ln = lambda t, w, b: torch.nn.functional.layer_norm(t, (D,), w, b, 1e-5)  # noqa: E731
    n1 = ln(x, q["g1"], q["b1"])
    zs = torch.softmax(n1 @ q["wa"], 1)                                  # [B, N, H]
    v = (n1 @ q["wv"]).view(B, N, H, D // H)
    idx = (torch.arange(N)[:, None] - torch.arange(N)[None]) % N
    x1 = x + torch.einsum("bijh,bjhc->bihc", zs[:, idx], v).reshape(B, N, D)
    n2 = ln(x1, q["g2"], q["b2"]).reshape(B * N, D)
    qkv = (n2 @ q["wqkv"]).view(B * N, H + 2 * hkv, dh)
    outs = []
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        Q = qkv[a:b, :H].transpose(0, 1)
        K = qkv[a:b, H:H + hkv].repeat_interleave(H // hkv, 1).transpose(0, 1)
        V = qkv[a:b, H + hkv:].repeat_interleave(H // hkv, 1).transpose(0, 1)
        s = Q @ K.transpose(1, 2) / math.sqrt(dh)
        s = s.masked_fill(~torch.ones(b - a, b - a, dtype=torch.bool).tril(), -math.inf)
        outs.append((torch.softmax(s, -1) @ V).transpose(0, 1))
    x2 = x1 + (torch.cat(outs).reshape(B * N, H * dh) @ q["wo"]).view(B, N, D)
    (x2 * r).sum().backward()
    names = list(p)
    want = {n: q[n].grad for n in names}
    norm = math.sqrt(sum(float(t.pow(2).sum()) for t in want.values()))

    # The framework's calls (dense projections by torch).
    d = {n: t.float().to(DEV) for n, t in p.items()}
    X, R, cd = x.float().to(DEV), r.float().to(DEV), cu.to(DEV)
    norm1, norm2 = (cat.LayerNormPlan(B * N, D, "f32") for _ in range(2))
    layer = cat.Plan(B, N, D, H, "f32")
    attn = cat.AttnPlan(B * N, len(lens), H, hkv, dh, "f32")
    y1, m1, r1 = norm1.forward(X, d["g1"], d["b1"])
    V = y1 @ d["wv"]
    X1 = X + layer.forward(y1, d["wa"], V)
    y2, m2, r2 = norm2.forward(X1, d["g2"], d["b2"])
    y2f = y2.view(B * N, D)
    fused = (y2f @ d["wqkv"]).view(B * N, H + 2 * hkv, dh)
    parts = (fused[:, :H], fused[:, H:H + hkv], fused[:, H + hkv:])
    O, lse = attn.forward(*parts, cd)
    X2 = X1 + (O.view(B * N, H * dh) @ d["wo"]).view(B, N, D)
    assert (X2.double().cpu() - x2.detach()).abs().max() <= 1e-4 * x2.detach().abs().max()
    got = {}
    Rf = R.view(B * N, D)
    got["wo"] = O.view(B * N, -1).t() @ Rf
    dO = (Rf @ d["wo"].t()).view(B * N, H, dh)
    dF = torch.empty_like(fused)
    attn.backward(*parts, O, lse, dO, cd, dQ=dF[:, :H], dK=dF[:, H:H + hkv], dV=dF[:, H + hkv:])
    dFf = dF.view(B * N, -1)
    got["wqkv"] = y2f.t() @ dFf
    dX1, got["g2"], got["b2"] = norm2.backward(X1, d["g2"], m2, r2,
                                               (dFf @ d["wqkv"].t()).view(B, N, D))
    dX1 = dX1 + R
    dy1, got["wa"], dV = layer.backward(y1, d["wa"], V, dX1.contiguous())
    got["wv"] = y1.view(-1, D).t() @ dV.view(-1, D)
    dy1 = dy1 + dV @ d["wv"].t()
    _, got["g1"], got["b1"] = norm1.backward(X, d["g1"], m1, r1, dy1)
    for n in names:
        e = (got[n].double().cpu() - want[n]).abs().max() / want[n].abs().max()
        assert e <= 1e-4, (n, float(e))
    grads = [got[n].contiguous() for n in names]
    with cat.ClipPlan([t.numel() for t in grads], [t.dtype for t in grads]) as clip:
        total = clip.clip(grads, 0.3 * norm)
        clip.sync()
    assert abs(float(total) / norm - 1) <= 1e-4
    for n, t in zip(names, grads):
        e = (t.double().cpu() - 0.3 * want[n]).abs().max() / want[n].abs().max()
        assert e <= 1e-4, (n, float(e))
    for plan in (norm1, norm2, layer, attn):
        plan.sync()
        plan.close()
