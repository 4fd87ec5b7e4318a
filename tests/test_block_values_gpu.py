"""GPU tests of what the operators around a CAT layer do with values and rows
that must not count: values that are not finite behind a mask, in long and in
many sequences, and rows that no sequence holds."""
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


def run(q, k, v, do, cu, causal, dtype, scale=None):
    T, hq, dh = q.shape
    ins = [t.to(DEV) for t in (q, k, v, do)]
    cd = cu.to(DEV)
    with cat.AttnPlan(T, len(cu) - 1, hq, k.shape[1], dh, dtype, causal=causal,
                      scale=scale) as plan:
        o, lse = plan.forward(*ins[:3], cd)
        grads = plan.backward(*ins[:3], o, lse, ins[3], cd)
        plan.sync()
    return dict(zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + grads))


@pytest.mark.parametrize("dh,hkv", [(64, 2), (128, 1)])
def test_values_behind_the_mask_after_many_blocks(dh, hkv):
    # Blocks that the mask cuts come after whole turns of the ring of key (query)
    # blocks, in every sequence and head: each is looked through.  A value of v
    # (of dO) that is not finite changes nothing, not a bit, in the rows (the
    # keys) that do not see it, and every one that does.
    lens = [1500, 700, 2049, 130, 1111, 300, 4100, 64, 900, 1023]
    hq = 4
    q, k, v, do, cu = ref.attn_inputs(lens, hq, hkv, dh, "bf16", 21)
    clean = run(q, k, v, do, cu, True, "bf16")
    r = np.random.default_rng(3)
    at = [int(s + r.integers(n // 2, n)) for s, n in zip(cu[:-1].tolist(), lens)]
    hidden = torch.zeros(sum(lens), dtype=torch.bool)         # rows before their sequence's value
    after = torch.zeros(sum(lens), dtype=torch.bool)
    for a, s, e in zip(at, cu[:-1].tolist(), cu[1:].tolist()):
        hidden[s:a] = True
        after[a + 1:e] = True
    c = 5
    for value in (math.nan, math.inf):
        bad = v.clone()
        bad[at, :, c] = value
        got = run(q, k, bad, do, cu, True, "bf16")
        for name in ("o", "dq"):
            assert torch.equal(got[name][hidden], clean[name][hidden]), name
        assert torch.equal(got["lse"], clean["lse"])
        seen = ~hidden
        assert not got["o"][seen][:, :, c].isfinite().any()
        keep = [i for i in range(dh) if i != c]
        assert torch.equal(got["o"][:, :, keep], clean["o"][:, :, keep])
        bad = do.clone()
        bad[at, :, c] = value
        got = run(q, k, v, bad, cu, True, "bf16")
        assert torch.equal(got["o"], clean["o"])
        rows = torch.ones(sum(lens), dtype=torch.bool)
        rows[at] = False
        assert torch.equal(got["dq"][rows], clean["dq"][rows])
        for name in ("dk", "dv"):
            assert torch.equal(got[name][after], clean[name][after]), name
        assert not got["dv"][~after][:, :, c].isfinite().any()
        assert torch.equal(got["dv"][:, :, keep], clean["dv"][:, :, keep])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dh", [64, 128])
def test_dv_of_values_in_the_first_and_the_last_cut_block(dh, causal):
    # Rows of dO that are not finite at the diagonal, between, and in a last
    # block that is cut or full: each reaches the dv of the keys its row sees,
    # in its column, and no other; many query heads to the key head.
    lens = [647, 640, 1281, 64, 65]
    hq, T = 16, sum(lens)
    q, k, v, do, cu = ref.attn_inputs(lens, hq, 1, dh, "bf16", 8)
    clean = run(q, k, v, do, cu, causal, "bf16")
    starts = cu[:-1].tolist()
    for back in (1, 5, 70, 200, 639):                          # rows from the end
        bad = do.clone()
        want = torch.zeros((T, dh), dtype=torch.bool)
        for x, (s, n) in enumerate(zip(starts, lens)):
            if back > n:
                continue
            i = n - back
            bad[s + i, (3 * x) % hq, 7 + x] = math.inf
            want[s:s + (i + 1 if causal else n), 7 + x] = True
        got = run(q, k, v, bad, cu, causal, "bf16")["dv"][:, 0].cpu()
        assert not got[want].isfinite().any()
        assert torch.equal(got[~want], clean["dv"][:, 0].cpu()[~want])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_behind_a_sequence_do_not_touch_a_bit(dtype, dh, causal):
    # The rows behind a sequence (padding, or the next sequence) share its last
    # tile: whatever they hold, its results are the same bit for bit.
    lens = [356, 227, 700, 33]
    extra = 64
    q, k, v, do, cu = ref.attn_inputs(lens, 2, 1, dh, dtype, 11, extra=extra)
    want = run(q, k, v, do, cu, causal, dtype)
    n = sum(lens)
    for f in (0.0, 40.0, math.inf):
        pad = [t.clone() for t in (q, k, v, do)]
        for t in pad:
            t[n:] = t[n:] * f if f != math.inf else math.inf
        got = run(*pad, cu, causal, dtype)
        for name in want:
            a, b = (r[name][:, :n] if name == "lse" else r[name][:n] for r in (got, want))
            assert torch.equal(a, b), (name, f)
    # Another sequence behind the first one.
    one = [t.clone() for t in (q, k, v, do)]
    for t in one:
        t[lens[0]:] *= 17.0
    got = run(*one, cu, causal, dtype)
    for name in want:
        a, b = (r[name][:, :lens[0]] if name == "lse" else r[name][:lens[0]] for r in (got, want))
        assert torch.equal(a, b), name


@pytest.mark.parametrize("S", [100, 150])
@pytest.mark.parametrize("causal", [True, False])
def test_f32_values_in_some_of_many_sequences(S, causal):
    # Blocks that are computed again are found like the others, largest first or
    # as they lie: the sequences that hold a NaN have it where their rows see it,
    # the others keep every bit.
    r = np.random.default_rng(S)
    lens = [int(n) for n in r.integers(1, 300, S)]
    hq, hkv, dh, c = 4, 2, 40, 11
    T = sum(lens)
    q, k, v, do, cu = ref.attn_inputs(lens, hq, hkv, dh, "f32", S)
    clean = run(q, k, v, do, cu, causal, "f32")
    struck = sorted(int(s) for s in r.choice(S, 7, replace=False))
    starts = cu[:-1].tolist()
    at = [starts[s] + int(r.integers(0, lens[s])) for s in struck]
    whole = torch.ones(T, dtype=torch.bool)
    sees = torch.zeros(T, dtype=torch.bool)
    for s, i in zip(struck, at):
        whole[starts[s]:starts[s] + lens[s]] = False
        sees[(i if causal else starts[s]):starts[s] + lens[s]] = True
    bad = v.clone()
    bad[at, :, c] = math.nan
    got = run(q, k, bad, do, cu, causal, "f32")
    for name in ("o", "dq", "dk", "dv"):
        assert torch.equal(got[name][whole], clean[name][whole]), name
    assert got["o"][sees][:, :, c].isnan().all() and got["dq"][sees].isnan().all()
    want = ref.attention(q, k, v, do, cu, causal, "f32")
    hidden = ~sees
    for name in ("o", "dq"):
        check(name, got[name].cpu()[hidden], tuple(t[hidden] for t in want[name]))
    keep = [x for x in range(dh) if x != c]
    check("o", got["o"][:, :, keep], tuple(t[:, :, keep] for t in want["o"]))
    check("dv", got["dv"], want["dv"])
