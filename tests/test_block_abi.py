"""Refusals of the operators around a CAT layer that need no device: bad plan
shapes and missing plans return the documented status codes."""
import ctypes
import math

import pytest

import fft_circulant_attention_gb300 as cat

INV = cat.CAT_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    from fft_circulant_attention_gb300 import build
    build.build()
    return cat.lib()


@pytest.mark.parametrize("args", [
    (-1, 4, 4, 4, 64, 0, 1, 0.0),           # max_tokens < 0
    (16, -1, 4, 4, 64, 0, 1, 0.0),          # max_seqs < 0
    (16, 4, 0, 4, 64, 0, 1, 0.0),           # no query heads
    (16, 4, 4, 0, 64, 0, 1, 0.0),           # no key heads
    (16, 4, 4, 3, 64, 0, 1, 0.0),           # Hq % Hkv != 0
    (16, 4, 2, 4, 64, 0, 1, 0.0),           # fewer query heads than key heads
    (16, 4, 4, 4, 0, 0, 1, 0.0),            # dh = 0
    (16, 4, 4, 4, 129, 0, 1, 0.0),          # dh above the limit
    (16, 4, 1 << 20, 1, 64, 0, 1, 0.0),     # rows too wide
    (16, 4, 4, 4, 64, 2, 1, 0.0),           # dtype
    (16, 4, 4, 4, 64, 0, 2, 0.0),           # causal neither 0 nor 1
    (16, 4, 4, 4, 64, 0, 1, -1.0),          # scale
    (16, 4, 4, 4, 64, 0, 1, math.nan),
    (16, 4, 4, 4, 64, 0, 1, math.inf),
    (2**31 - 1, 4, 64, 4, 64, 0, 1, 0.0),   # max_tokens·Hq past 2^31
    (2**30 + 1, 4, 1, 1, 64, 0, 1, 0.0),    # max_tokens above the limit
    (16, 2**31 - 1, 4, 4, 64, 0, 1, 0.0),   # blocks past 2^31
])
def test_attn_plan_refuses(lib, args):
    h = ctypes.c_void_p()
    assert lib.cat_plan_create_attn(ctypes.byref(h), *args, None) == INV
    assert not h.value
    assert lib.cat_plan_create_attn(None, *args, None) == INV


@pytest.mark.parametrize("args", [
    (-1, 64, 0, 1e-5), (4, 0, 0, 1e-5), (4, 8193, 0, 1e-5), (4, 64, 5, 1e-5), (4, 64, 0, -1e-5),
    (4, 64, 0, math.nan), (4, 64, 0, math.inf), (2**30 + 1, 1, 0, 1e-5),
])
def test_layernorm_plan_refuses(lib, args):
    h = ctypes.c_void_p()
    assert lib.cat_plan_create_layernorm(ctypes.byref(h), *args, None) == INV
    assert not h.value


@pytest.mark.parametrize("count,sizes,dtypes", [
    (-1, [1], [0]), (1, [-1], [0]), (1, [4], [7]), (2, [4, 1 << 41], [0, 0]),
    ((1 << 20) + 1, [], []),
])
def test_clip_plan_refuses(lib, count, sizes, dtypes):
    h = ctypes.c_void_p()
    sz = (ctypes.c_longlong * max(1, len(sizes)))(*sizes)
    dt = (ctypes.c_int * max(1, len(dtypes)))(*dtypes)
    assert lib.cat_plan_create_clip(ctypes.byref(h), count, sz, dt, None) == INV
    assert not h.value
    assert lib.cat_plan_create_clip(ctypes.byref(h), 1, None, dt, None) == INV
    assert lib.cat_plan_create_clip(ctypes.byref(h), 1, sz, None, None) == INV


def test_missing_plans(lib):
    n = None
    assert lib.cat_attn_forward(n, n, n, n, n, n, n, 1, 1, 64, 64, 64) == INV
    assert lib.cat_attn_backward(n, n, n, n, n, n, n, n, n, n, n, 1, 1, *[64] * 6) == INV
    assert lib.cat_layernorm_forward(n, n, n, n, n, n, n, 1) == INV
    assert lib.cat_layernorm_backward(n, n, n, n, n, n, n, n, n, 1) == INV
    assert lib.cat_grad_norm(n, n, n) == INV
    assert lib.cat_grad_clip(n, n, n, 1.0, n) == INV


def test_python_lists_must_match(lib):
    with pytest.raises(ValueError):
        cat.cat_plan_create_clip([1, 2], ["f32"])
