"""The dense serving path at the ends of its arguments' ranges and over data that reaches its rarer
paths, against the plain 64-bit forms."""
import math

import pytest
import torch

import serving_plain as sp
from test_gpu_serving import (BF16, F32, NAN, _close, _packed_inputs, _tag, _tree_inputs, _tree_ref,  # noqa: F401
                              _tree_run, sala)

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


@pytest.mark.parametrize("H,Hkv,d,top,n", [(4, 4, 64, 300, 300), (4, 4, 128, 300, 250), (4, 2, 64, 300, 300),
                                           (6, 2, 64, 300, 250), (6, 2, 128, 700, 60), (8, 2, 64, 200, 400)])
def test_packed_prefill_several_units_per_block(sala, H, Hkv, d, top, n):  # noqa: F811
    # many short units after one another in every block, the second tile of rows longer, as long or without
    # a row; groups of one, two, three and four query heads
    g = torch.Generator().manual_seed(33)
    lens = [int(x) for x in torch.randint(0, top, (n,), generator=g)]
    q, k, v = _packed_inputs(H, Hkv, d, BF16, sum(lens), seed=34)
    args = q.cuda(), k.cuda(), v.cuda(), sp.offsets(lens).cuda()
    a, b = (sala.packed_prefill(*args) for _ in range(2))
    sala.check_status()
    assert torch.equal(a, b)
    _close(a, *sp.packed64(q, k, v, lens), top, "bf16 units")
