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
