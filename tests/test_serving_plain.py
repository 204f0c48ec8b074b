"""The plain 64-bit forms that the serving kernels are tested against are themselves pinned, and
the serving calls refuse bad arguments on the host.  No GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import serving_plain as sp


def test_packed_plain_equals_the_oracles_dense_causal_attention():
    g = torch.Generator().manual_seed(0)
    lens = [5, 0, 1, 17]
    q, k, v = (torch.randn((h, sum(lens), 8), generator=g, dtype=torch.float64) for h in (4, 2, 2))
    o, A, _ = sp.packed64(q, k, v, lens)
    at = 0
    for n in lens:
        if n:
            r = slice(at, at + n)
            ref = oracle.dense_causal_attention(q[None, :, r].numpy(), k[None, :, r].numpy(), v[None, :, r].numpy())
            np.testing.assert_allclose(o[:, r].numpy(), ref[0], atol=1e-12)
        at += n
    assert bool((A >= o.abs() - 1e-12).all())


def test_tree_plain_with_a_chain_is_the_causal_tail():
    g = torch.Generator().manual_seed(1)
    c, T = 9, 4
    q = torch.randn((1, 4, c + T, 8), generator=g, dtype=torch.float64)
    k, v = (torch.randn((2, c + T, 8), generator=g, dtype=torch.float64) for _ in range(2))
    tree = torch.tensor([sp.ancestors([-1, 0, 1, 2])])
    o, _, _ = sp.tree64(q[:, :, c:], [k], [v], [c], tree)
    ref, _, _ = sp.packed64(q[0], k, v, [c + T])
    np.testing.assert_allclose(o[0].numpy(), ref[:, c:].numpy(), atol=1e-12)


def test_tree_plain_sees_its_bits_only():
    k = torch.zeros((1, 3, 4), dtype=torch.float64)
    v = torch.tensor([[[1.0] * 4, [10.0] * 4, [100.0] * 4]], dtype=torch.float64)
    q = torch.zeros((1, 1, 3, 4), dtype=torch.float64)
    o, _, _ = sp.tree64(q, [k], [v], [0], torch.tensor([[0b001, 0b101, 0b000]]))
    assert o[0, 0, :, 0].tolist() == [1.0, 50.5, 0.0]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_quantiser_is_within_half_a_step(fmt):
    g = torch.Generator().manual_seed(2)
    x = torch.randn((50, 64), generator=g) * torch.exp(torch.randn((50, 1), generator=g) * 3)
    x[0] = 0
    code, scale = sp.quantise64(x, fmt)
    a = x.double().abs().amax(-1)
    err = (code * scale[:, None] - x.double()).abs()
    if fmt == "int8":
        assert float(code.abs().max()) == 127
        assert bool((err <= 0.5001 * a[:, None] / 127 + 1e-38).all())
    else:
        assert bool((scale.log2() == scale.log2().round()).all())
        assert bool((a[1:] / scale[1:] <= 448).all()) and bool((a[1:] / scale[1:] > 224).all())
        assert bool((code == code.float().to(torch.float8_e4m3fn).double()).all())  # e4m3 values
        assert bool((err <= x.double().abs() * 2.0 ** -4 + scale[:, None] * 2.0 ** -10).all())
    bad = x[:3].clone()
    bad[1, 5] = math.inf
    code, scale = sp.quantise64(bad, fmt)
    assert bool(torch.isnan(scale[1])) and bool(torch.isfinite(scale[[0, 2]]).all()) and not code[1].any()


def test_e4m3_codes_equal_torchs_conversion():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((40, 128), generator=g).bfloat16()
    code, scale = sp.quantise64(x, "e4m3")
    y = (x.float() / scale[:, None].float()).to(torch.float8_e4m3fn)
    assert bool((code == y.double()).all())


# ---------------------------------------------------------------------------------------------
# Refusals

@pytest.fixture(scope="module")
def sala():
    from hybrid_sparse_linear_b200 import sala as s
    return s


GOOD = 1 << 20  # never dereferenced: every call below fails validation first


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _packed(sala, q=GOOD, k=GOOD, v=GOOD, cu=GOOD, o=GOOD, B=1, H=4, Hkv=2, total=8, d=128,
            scale=0.0, dt=1):
    return sala.raw.sala_packed_prefill(_p(q), _p(k), _p(v), _p(cu), _p(o), B, H, Hkv, total, d,
                                        scale, dt, None)


def _write(sala, read=False, k=GOOD, v=GOOD, cu=GOOD, pos=GOOD, table=GOOD, max_pages=2, kp=GOOD,
           vp=GOOD, ks=None, vs=None, n_pages=4, B=1, Hkv=2, total=8, d=128, block=64, fmt=0, dt=1):
    if read:
        return sala.raw.sala_kv_read(_p(kp), _p(vp), _p(ks), _p(vs), n_pages, _p(table), max_pages,
                                     _p(cu), _p(pos), _p(k), _p(v), B, Hkv, total, d, block, fmt, dt,
                                     None)
    return sala.raw.sala_kv_write(_p(k), _p(v), _p(cu), _p(pos), _p(table), max_pages, _p(kp), _p(vp),
                                  _p(ks), _p(vs), n_pages, B, Hkv, total, d, block, fmt, dt, None)


def _tree(sala, q=GOOD, kp=GOOD, vp=GOOD, ks=None, vs=None, n_pages=4, table=GOOD, max_pages=2,
          ctx=GOOD, max_ctx=60, tree=GOOD, o=GOOD, B=1, H=4, Hkv=2, T=4, d=128, block=64, scale=0.0,
          ws=GOOD, ws_bytes=1 << 40, fmt=0, dt=1):
    return sala.raw.sala_tree_decode_paged(_p(q), _p(kp), _p(vp), _p(ks), _p(vs), n_pages, _p(table),
                                           max_pages, _p(ctx), max_ctx, _p(tree), _p(o), B, H, Hkv, T,
                                           d, block, scale, _p(ws), ws_bytes, fmt, dt, None)


@pytest.mark.parametrize("bad,code,word", [
    (dict(d=96), 2, b"head dim"), (dict(H=5), 1, b"multiple"), (dict(Hkv=0), 1, b"Hkv"),
    (dict(B=-1), 1, b"negative"), (dict(total=-1), 1, b"negative"), (dict(dt=2), 1, b"dtype"),
    (dict(q=None), 1, b"q must"), (dict(v=GOOD + 8), 1, b"v must"), (dict(cu=None), 1, b"cu_seqlens"),
    (dict(scale=math.nan), 1, b"scale"), (dict(scale=-1.0), 1, b"scale"),
])
def test_packed_prefill_refuses(sala, bad, code, word):
    assert _packed(sala, **bad) == code
    assert word in sala.raw.sala_last_error()


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("bad,code,word", [
    (dict(d=32), 2, b"head dim"), (dict(block=16), 2, b"block"), (dict(fmt=3), 1, b"format"),
    (dict(fmt=1), 1, b"k_scale"), (dict(fmt=1, ks=GOOD), 1, b"v_scale"),
    (dict(ks=GOOD, vs=GOOD), 1, b"8-bit"), (dict(n_pages=-1), 1, b"page"),
    (dict(n_pages=1 << 25), 2, b"rows"), (dict(table=None), 1, b"page_table"),
    (dict(pos=None), 1, b"pos"), (dict(kp=GOOD + 4), 1, b"k_pages"), (dict(k=None), 1, b"k must"),
])
def test_cache_calls_refuse(sala, read, bad, code, word):
    assert _write(sala, read, **bad) == code
    assert word in sala.raw.sala_last_error()


@pytest.mark.parametrize("bad,code,word", [
    (dict(T=65), 2, b"64 bits"), (dict(T=-1), 1, b"negative"), (dict(H=3), 1, b"multiple"),
    (dict(max_ctx=125), 1, b"page table"), (dict(max_ctx=-1), 1, b"page table"),
    (dict(max_ctx=(1 << 31) - 1), 1, b"page table"), (dict(ws_bytes=16), 1, b"workspace"),
    (dict(ws=None), 1, b"workspace"), (dict(tree=GOOD + 4), 1, b"tree"), (dict(ctx=None), 1, b"ctx"),
    (dict(B=40000), 2, b"65535"), (dict(fmt=2), 1, b"k_scale"), (dict(o=None), 1, b"o must"),
])
def test_tree_decode_refuses(sala, bad, code, word):
    assert _tree(sala, **bad) == code
    assert word in sala.raw.sala_last_error()


def test_empty_serving_problems_are_noops(sala):
    assert _packed(sala, q=None, k=None, v=None, cu=None, o=None, total=0) == 0
    assert _packed(sala, B=0) == 0
    assert _write(sala, k=None, v=None, total=0) == 0
    assert _write(sala, True, k=None, v=None, B=0) == 0
    assert _tree(sala, T=0) == 0 and _tree(sala, B=0) == 0
    assert sala.raw.sala_tree_decode_paged_workspace(0, 4, 2, 1, 10, 128) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes(sala):
    q = torch.zeros((4, 8, 64))
    with pytest.raises(ValueError, match="CUDA"):
        sala.packed_prefill(q, q[:2], q[:2], torch.tensor([0, 8], dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        sala.kv_write(q, q, torch.tensor([0, 8], dtype=torch.int32), None, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        sala.tree_decode_paged(q[None], None, None, None, None, 0, None)
