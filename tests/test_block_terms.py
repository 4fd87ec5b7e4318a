"""The limit of the bf16 backward's errors tells two terms of dS from one: both
forms emulated in 64 bits on the CPU."""
import pytest

import _block_ref as ref
import _block_terms as t


@pytest.mark.parametrize("n,hq,hkv,dh,causal", t.CASES)
def test_one_term_of_ds_is_beyond_the_limit(n, hq, hkv, dh, causal):
    q, k, v, do, _ = ref.attn_inputs([n], hq, hkv, dh, "bf16", 31)
    o, lse = t.forward(q, k, v, causal)
    want = t.backward(q, k, v, do, o, lse, causal)
    one = t.backward(q, k, v, do, o, lse, causal, t.one_term, t.one_term)
    two = t.backward(q, k, v, do, o, lse, causal, t.one_term, t.two_terms)
    for a, b, w in zip(one[:2], two[:2], want[:2]):
        limit = t.LIMIT * t.error(t.bf16(w), w)
        assert t.error(t.bf16(b), w) <= limit < t.error(t.bf16(a), w) / 1.15
