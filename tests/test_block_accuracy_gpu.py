"""GPU tests of how near the attention kernels come to their definition: the two
terms of dS in the bf16 backward, and kernels over lengths of a thousand and more."""
import pytest
import torch

import fft_circulant_attention_gb300 as cat
import _block_ref as ref
import _block_terms as t
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


def off_boundary(x):
    """The same rows, starting one element off a 16-byte boundary."""
    w = x.shape[1] * x.shape[2]
    buf = torch.zeros(x.shape[0] * (w + 3) + 1, dtype=x.dtype, device=DEV)
    view = torch.as_strided(buf, x.shape, (w + 3, x.shape[2], 1), 1)
    view.copy_(x)
    return view


@pytest.mark.parametrize("pipe", ["tensor", "fp32"])
@pytest.mark.parametrize("n,hq,hkv,dh,causal", t.CASES)
def test_ds_keeps_two_terms(n, hq, hkv, dh, causal, pipe):
    # dq and dk from o and lse that are rounded from 64 bits: no further off than
    # their own rounding, on the tensor cores and (rows off a boundary) on the
    # FP32 pipe; dv by its one term of P; and every value within its bound.
    q, k, v, do, cu = ref.attn_inputs([n], hq, hkv, dh, "bf16", 31)
    o, lse = t.forward(q, k, v, causal)
    put = off_boundary if pipe == "fp32" else lambda x: x.to(DEV)
    with cat.AttnPlan(n, 1, hq, hkv, dh, "bf16", causal=causal) as plan:
        got = plan.backward(put(q), put(k), put(v), o.to(DEV), lse.to(DEV), do.to(DEV), cu.to(DEV))
        plan.sync()
    got = [x.cpu() for x in got]
    want = t.backward(q, k, v, do, o, lse, causal)
    for name, g, w in zip(("dq", "dk"), got, want):
        assert t.error(g, w) <= t.LIMIT * t.error(t.bf16(w), w), name
    one = t.backward(q, k, v, do, o, lse, causal, t.one_term)[2]
    assert t.error(got[2], want[2]) <= t.LIMIT * t.error(t.bf16(one), want[2])
    bounds = ref.attention(q, k, v, do, cu, causal, "bf16", rounds=2.0 ** -16)
    for name, g in zip(("dq", "dk"), got):
        check(name, g, bounds[name])


def parity(lens, hq, hkv, dh, dtype, causal, seed, put=lambda x: x.to(DEV)):
    q, k, v, do, cu = ref.attn_inputs(lens, hq, hkv, dh, dtype, seed)
    ins = [put(x) for x in (q, k, v)]
    with cat.AttnPlan(q.shape[0], len(lens), hq, hkv, dh, dtype, causal=causal) as plan:
        o, lse = plan.forward(*ins, cu.to(DEV))
        grads = plan.backward(*ins, o, lse, do.to(DEV), cu.to(DEV))
        plan.sync()
    want = ref.attention(q, k, v, do, cu, causal, dtype)
    for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + grads):
        check(name, x, want[name])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,dh", [([1111, 640, 383], 128), ([2049, 130], 96), ([1500], 72),
                                     ([1025, 1024, 7], 100)], ids=str)
def test_f32_wide_heads_over_long_sequences(lens, dh, causal):
    parity(lens, 2, 1, dh, "f32", causal, sum(lens) + dh)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,dh", [([1111, 640, 383], 64), ([2049, 130], 128), ([1500], 33),
                                     ([1025, 1024, 7], 5)], ids=str)
def test_bf16_rows_off_a_boundary_over_long_sequences(lens, dh, causal):
    parity(lens, 2, 1, dh, "bf16", causal, sum(lens) + dh, off_boundary)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dh", [72, 80, 96, 120])
def test_bf16_padded_heads_over_long_sequences(dh, causal):
    parity([1111, 640, 383], 4, 2, dh, "bf16", causal, dh)
