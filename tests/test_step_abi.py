"""Refusals of the training step's other operators that need no device: bad plan
shapes and missing plans return the documented status codes."""
import ctypes
import math

import pytest
import torch

import fft_circulant_attention_gb300 as cat

INV = cat.CAT_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    from fft_circulant_attention_gb300 import build
    build.build()
    return cat.lib()


@pytest.mark.parametrize("create,args", [
    ("embed", (-1, 10, 8, 0, 1.0)), ("embed", (2**24 + 1, 10, 8, 0, 1.0)),
    ("embed", (4, 0, 8, 0, 1.0)), ("embed", (4, 2**20 + 1, 8, 0, 1.0)),
    ("embed", (4, 10, 0, 0, 1.0)), ("embed", (4, 10, 8193, 0, 1.0)), ("embed", (4, 10, 8, 2, 1.0)),
    ("embed", (4, 10, 8, 0, math.nan)), ("embed", (4, 10, 8, 0, math.inf)),
    ("resnorm", (-1, 8, 0, 0, 1e-5, 1.0)), ("resnorm", (2**30 + 1, 8, 0, 0, 1e-5, 1.0)),
    ("resnorm", (4, 0, 0, 0, 1e-5, 1.0)), ("resnorm", (4, 8193, 0, 0, 1e-5, 1.0)),
    ("resnorm", (4, 8, 3, 0, 1e-5, 1.0)), ("resnorm", (4, 8, 0, 2, 1e-5, 1.0)),
    ("resnorm", (4, 8, 0, 0, -1e-5, 1.0)), ("resnorm", (4, 8, 0, 0, math.nan, 1.0)),
    ("resnorm", (4, 8, 0, 1, 1e-5, math.inf)),
    ("xent", (-1, 10, 8, 0, 1)), ("xent", (2**20 + 1, 10, 8, 0, 1)), ("xent", (4, 0, 8, 0, 1)),
    ("xent", (4, 2**20 + 1, 8, 0, 1)), ("xent", (4, 10, 0, 0, 1)), ("xent", (4, 10, 8193, 0, 1)),
    ("xent", (4, 10, 8, 7, 1)), ("xent", (4, 10, 8, 0, 2)),
])
def test_plans_refuse(lib, create, args):
    h = ctypes.c_void_p()
    f = getattr(lib, "cat_plan_create_" + create)
    assert f(ctypes.byref(h), *args, None) == INV
    assert not h.value
    assert f(None, *args, None) == INV


def test_missing_plans(lib):
    n = None
    assert lib.cat_embed_forward(n, n, 2, n, n, 1) == INV
    assert lib.cat_embed_backward(n, n, 2, n, n, 0, 1) == INV
    assert lib.cat_resnorm_forward(n, n, n, n, 0, *[n] * 7, 1) == INV
    assert lib.cat_resnorm_backward(n, n, n, n, 0, *[n] * 13, 1) == INV
    assert lib.cat_xent_forward(n, n, n, n, 2, n, n, 1) == INV
    assert lib.cat_xent_backward(n, n, n, n, 2, n, n, 0, n, n, 1) == INV


def test_id_codes():
    assert cat.id_code(torch.int32) == cat.CAT_I32 and cat.id_code(torch.int64) == cat.CAT_I64
    assert cat.id_code(cat.CAT_I64) == cat.CAT_I64
    for t in (torch.int16, torch.uint8, torch.float32):
        with pytest.raises(ValueError):
            cat.id_code(t)
