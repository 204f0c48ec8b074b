"""The dense serving path at the ends of its arguments' ranges and over data that reaches its rarer
paths, against the plain 64-bit forms."""
import math

import pytest
import torch

import serving_plain as sp
from test_gpu_serving import BF16, F32, NAN, _close, _tag, _tree_inputs, _tree_ref, _tree_run, sala  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = [(BF16, "same"), (BF16, "int8"), (BF16, "e4m3"), (F32, "int8")]


@pytest.mark.parametrize("scale", [1e-9, 1e-20, 1e-40])
@pytest.mark.parametrize("dtype,fmt", FORMS)
@pytest.mark.parametrize("H,Hkv,T", [(32, 2, 1), (8, 4, 8), (32, 2, 8)])
def test_tree_decode_small_queries_and_tiny_scales(sala, H, Hkv, T, dtype, fmt, scale):  # noqa: F811
    # A row that is zero or nearly so gives equal weights, whatever the scale, also beside slots
    # and drafts that it does not see.
    ctx = [70, 190, 0]
    q, cache, tree = _tree_inputs(H, Hkv, 128, dtype, fmt, T, ctx, seed=31, fill=NAN)
    q[0] = 0
    q[1] *= 2.0 ** -110
    out = _tree_run(sala, q, cache, ctx, tree, scale=scale)
    sala.check_status()
    _close(out, *_tree_ref(q, cache, ctx, tree, scale), max(ctx) + T, _tag(dtype, "tiny scale"))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H,Hkv,T", [(32, 2, 1), (8, 4, 8), (32, 2, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_tree_decode_large_keys_and_small_queries(sala, H, Hkv, T, d, fmt):  # noqa: F811
    # keys near the top of the type's range, queries that bring the logits back to ordinary ones
    ctx = [300, 61]
    q, cache, tree = _tree_inputs(H, Hkv, d, BF16, fmt, T, ctx, seed=32, fill=NAN)
    q *= 2.0 ** -116
    cache.ks *= 2.0 ** 116
    out = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    _close(out, *_tree_ref(q, cache, ctx, tree), max(ctx) + T, _tag(BF16, "large keys"))
