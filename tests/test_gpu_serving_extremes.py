"""The dense serving path at the ends of its arguments' ranges and over data that reaches its rarer
paths, against the plain 64-bit forms."""
import math

import pytest
import torch

import serving_plain as sp
from test_gpu_serving import (BF16, F32, NAN, PACKED, TREE, _close, _packed_inputs, _tag, _tree_inputs, _tree_ref,  # noqa: F401
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


@pytest.mark.parametrize("scale", [1e10, 2e38])
@pytest.mark.parametrize("dtype,fmt", FORMS)
@pytest.mark.parametrize("H,Hkv,T", [(32, 2, 1), (8, 4, 8), (32, 2, 8)])
def test_tree_decode_zero_queries_and_large_scales(sala, H, Hkv, T, dtype, fmt, scale):  # noqa: F811
    ctx = [70, 190, 0]
    q, cache, tree = _tree_inputs(H, Hkv, 128, dtype, fmt, T, ctx, seed=31, fill=NAN)
    q[:] = 0
    # keys as large as the logits' factor allows (more rows than 16) or as large as they come
    if cache.ks is not None and H // Hkv * T <= 16:
        cache.ks *= 2.0 ** 120
    out = _tree_run(sala, q, cache, ctx, tree, scale=scale)
    sala.check_status()
    _close(out, *_tree_ref(q, cache, ctx, tree, scale), max(ctx) + T, _tag(dtype, "large scale"))


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


# ---------------------------------------------------------------------------------------------
# At most 16 rows per KV head: special values, empty rows and missing pages

FEW = [(4, 4, 8), (8, 4, 8), (8, 2, 4), (16, 1, 1)]  # H, Hkv, T
CODES = [(64, "same"), (64, "int8"), (64, "e4m3"), (128, "same"), (128, "int8"), (128, "e4m3")]


def _floor(fmt, kv, n):
    """What the bound gets on top over 8-bit caches with at most 16 rows per KV head.  There the weight of a
    key times V's scale is held in fp16, a warp's largest at 2^7 or above, so half of fp16's smallest step,
    2^-25, is 2^-32 of it.  Each of n keys is off by at most that part of max_j p_j s_j times its own code, p <= 1:
    s times the largest code is the row's largest |v| in int8 (127 s = a), at most twice it in e4m3
    (a / s > 224, codes up to 448).  It shows in a column where the key with nearly all of the weight has the
    code 0 and the sum is what the far smaller ones leave."""
    if fmt == "same":
        return 0.0
    return n * 2.0 ** -32 * max(float(v.abs().max()) for _, v in kv) * (2 if fmt == "e4m3" else 1)


def _close_few(out, o, A, e, n, floor, what):
    over = (out.double().cpu() - o).abs() - sp.bound(A, e, n, True) - floor
    assert bool((over <= 0).all()), f"{what}: {float(over.max()):.3e} over the bound"


def _few(sala, q, cache, ctx, tree, fmt, what, scale=0.0):  # noqa: F811
    out = _tree_run(sala, q, cache, ctx, tree, scale=scale)
    sala.check_status()
    kv = [cache.dense64(b, 0, c + q.shape[2]) for b, c in enumerate(ctx)]
    n = max(ctx) + q.shape[2]
    _close_few(out, *_tree_ref(q, cache, ctx, tree, scale), n, _floor(fmt, kv, n), what)
    return out


@pytest.mark.parametrize("H,Hkv,T", FEW)
@pytest.mark.parametrize("d,fmt", CODES)
def test_few_rows_peaked_and_a_scale(sala, H, Hkv, T, d, fmt):  # noqa: F811
    for ctx in ([600, 90], [3000, 62]):
        q, cache, tree = _tree_inputs(H, Hkv, d, BF16, fmt, T, ctx, seed=41, mul=3.0, fill=NAN)
        _few(sala, q, cache, ctx, tree, fmt, "few peaked", 0.11)


@pytest.mark.parametrize("H,Hkv,T", FEW)
@pytest.mark.parametrize("d,fmt", CODES)
def test_few_rows_that_see_nothing(sala, H, Hkv, T, d, fmt):  # noqa: F811
    for ctx in ([0, 200, 0], [0, 2900, 61]):
        q, cache, tree = _tree_inputs(H, Hkv, d, BF16, fmt, T, ctx, seed=42, fill=NAN)
        tree[0] = 0
        if T > 1:
            tree[0, 1] = 2
            tree[0, T - 1] = -(1 << T)  # bits at and above T only, which count for nothing
        tree[1] = 0
        out = _few(sala, q, cache, ctx, tree, fmt, "few empty")
        assert not out[0, :, [t for t in range(T) if t != 1]].any()


@pytest.mark.parametrize("H,Hkv,T", FEW[:3])
@pytest.mark.parametrize("d,fmt", CODES)
@pytest.mark.parametrize("ctx", [[190, 0, 60, 63], [2622, 60, 0, 190]])  # a block per item; runs with partials
def test_few_rows_hidden_infinities(sala, H, Hkv, T, d, fmt, ctx):  # noqa: F811
    # drafts on both sides of a page's end; what one of them holds reaches the rows that see it alone
    a, t_a, b, t_b, c = (2, 5, 4, 7, 6) if T == 8 else (0, 3, 1, 1, 2)
    q, cache, tree = _tree_inputs(H, Hkv, d, BF16, fmt, T, ctx, seed=43, fill=NAN)
    tree[:] = torch.tensor([1 << t for t in range(T)])
    tree[:, t_a] |= 1 << a
    tree[:, t_b] |= 1 << b
    o, A, e = _tree_ref(q, cache, ctx, tree)
    floor = _floor(fmt, [cache.dense64(s, 0, n + T) for s, n in enumerate(ctx)], max(ctx) + T)
    for s, n in enumerate(ctx):
        for j, col, val, what in ((a, 3, NAN, "v"), (b, 9, -math.inf, "v"), (c, 0, NAN, "k")):
            page, slot = int(cache.table[s, (n + j) // 64]), (n + j) % 64
            if fmt == "same":
                (cache.v if what == "v" else cache.k)[page, :, slot, col] = val
            else:
                (cache.vs if what == "v" else cache.ks)[page, :, slot] = NAN
    out = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    got = out.double().cpu()
    hit = torch.zeros(got.shape, dtype=torch.bool)
    for t, col in ((a, 3), (t_a, 3), (b, 9), (t_b, 9)):
        hit[:, :, t, [col] if fmt == "same" else list(range(d))] = True
    hit[:, :, c] = True
    assert bool(((got - o).abs() <= sp.bound(A, e, max(ctx) + T, True) + floor)[~hit].all())
    assert not bool(torch.isfinite(got[hit]).any())
    if fmt == "same":
        assert bool(torch.isnan(got[:, :, a, 3]).all()) and bool((got[:, :, b, 9] == -math.inf).all())
        assert bool(torch.isnan(got[:, :, c]).all())


@pytest.mark.parametrize("H,Hkv,T", FEW[:3])
@pytest.mark.parametrize("d,fmt", CODES)
def test_few_rows_missing_pages(sala, H, Hkv, T, d, fmt):  # noqa: F811
    # Enough items that each has a block of its own and a warp several pages (every twelfth, or every
    # sixth): a warp's first, a middle one, the last, neighbours, and all of them are missing.
    base, B = [2500, 700], 112 // Hkv
    ctx = [base[b % 2] for b in range(B)]
    _, cache, _ = _tree_inputs(H, Hkv, d, BF16, fmt, T, base, seed=44, fill=NAN)
    g = torch.Generator().manual_seed(45)
    q = torch.randn((B, H, T, d), generator=g).to(BF16)
    tree = torch.tensor([sp.ancestors(range(-1, T - 1))] * B)
    own = cache.table.clone()
    cache.table = own[[b % 2 for b in range(B)]].contiguous()
    good = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    (k, v), n = cache.dense64(0, 0, 2500 + T), 2500 + T
    for missing in ([0], [12], [0, 12], [12, 24], [0, 6, 12, 18, 24, 30, 36], [5, 17, 18, 39], list(range(40))):
        cache.table[0, missing] = -1
        cache.table[B - 2, missing] = cache.n_pages
        out = _tree_run(sala, q, cache, ctx, tree)
        with pytest.raises(sala.SalaError) as err:
            sala.check_status()
        assert err.value.code == sala.ERR_BOUNDS
        cache.table[[0, B - 2]] = own[0]
        assert torch.equal(out[1:B - 2], good[1:B - 2]) and torch.equal(out[B - 1], good[B - 1])
        keep = torch.ones((T, n), dtype=torch.bool)
        keep[:, 2500:] = torch.ones((T, T), dtype=torch.bool).tril()
        for j in missing:
            keep[:, 64 * j:64 * j + 64] = False
        for b in (0, B - 2):
            for h in (0, H - 1):
                o, A, e = sp.attention64(q[b, h], k[h // (H // Hkv)], v[h // (H // Hkv)], keep)
                _close_few(out[b, h], o, A, e, n, _floor(fmt, [(k, v)], n), "few missing pages")


# ---------------------------------------------------------------------------------------------
# Small weights and small components beside large ones

@pytest.mark.parametrize("dtype,fmt", [(BF16, "int8"), (BF16, "e4m3"), (BF16, "same"), (F32, "int8")])
@pytest.mark.parametrize("T", [1, 16, 33])
@pytest.mark.parametrize("below", [20.5, 25.5, 26.0, 31.0])
def test_small_weights_beside_a_peak_in_every_warp(sala, dtype, fmt, T, below):  # noqa: F811
    # 16 pages in one block: each of the first twelve begins with a key of weight 1, all other keys weigh
    # 2^-below.  The peaks' values are zero in the even columns, so those hold the small weights' sum alone
    # and the bound there is relative to it.
    n, d, w = 1024, 64, 2.0 ** -below
    kind = {"same": dtype, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt]
    k, v = torch.zeros((2, 1, 64, d)), torch.full((2, 1, 64, d), 64.0)
    k[0, 0, 0, 0] = 64.0
    v[0, 0, 0] = -64.0
    v[0, 0, 0, ::2] = 0.0
    ks, vs = (None, None) if fmt == "same" else (torch.ones((2, 1, 64)).cuda() for _ in range(2))
    q = torch.zeros((1, 1, T, d), dtype=dtype)
    q[..., 0] = 1.0
    table = torch.tensor([[0] * 12 + [1] * 4], dtype=torch.int32)
    tree = torch.tensor([sp.signed([1 << t for t in range(T)])])  # a row sees the context and itself
    out = sala.tree_decode_paged(q.cuda(), k.to(kind).cuda(), v.to(kind).cuda(), table.cuda(),
                                 torch.tensor([n - T], dtype=torch.int32).cuda(), n - T, tree.cuda(), ks, vs,
                                 scale=below * math.log(2.0) / 64)
    sala.check_status()
    tail = (n - T - 12 + 1) * w
    peak = v[0, 0, 0].double()
    o, A = ((12 * x + tail * 64.0) / (12 + tail) for x in (peak, peak.abs()))
    # the scale is rounded to 32 bits: 2^-24 of a logit of below ln 2 on top of the product's error
    e = torch.full((1, 1, T), below * math.log(2.0) * (d + 5) * 2.0 ** -24, dtype=torch.float64)
    _close(out, o.expand(1, 1, T, d), A.expand(1, 1, T, d), e, n, _tag(dtype, "small weights"))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H,Hkv,T", [(16, 1, 1), (8, 4, 8), (32, 2, 8)])
def test_small_query_components_with_large_keys(sala, H, Hkv, T, fmt):  # noqa: F811
    # a component 2^-30 of its row's largest, against keys that are large there and zero in the large one
    ctx, d = [200, 33], 128
    q, cache, tree = _tree_inputs(H, Hkv, d, BF16, fmt, T, ctx, seed=46)
    q[..., 0] = 1.0
    q[..., 1:] *= 2.0 ** -30
    raw = cache.k.view(torch.uint8)
    raw[..., 0] = 0
    cache.ks *= 2.0 ** 30
    out = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    _close(out, *_tree_ref(q, cache, ctx, tree), max(ctx) + T, "bf16 small components")


# ---------------------------------------------------------------------------------------------
# The cache with the framework's sparse decode

@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pages_written_here_are_read_by_the_sparse_decode(sala, dtype):  # noqa: F811
    # the blocks that the sparse decode names, attended over the pages that kv_write filled
    H, Hkv, d, N, topk = 32, 2, 128, 1000, 8
    g = torch.Generator().manual_seed(47)
    q = torch.randn((1, H, d), generator=g).to(dtype)
    k, v = (torch.randn((Hkv, N, d), generator=g).to(dtype) for _ in range(2))
    cache = sp.Cache([N], Hkv, d, dtype, "same", seed=48).cuda()
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    sala.kv_write(k.cuda(), v.cuda(), sp.offsets([N]).cuda(), zero, cache.table, cache.k, cache.v)
    kbar = sala.block_compress(k[None].cuda())
    idx = torch.full((1, Hkv, 1 + 2 + topk), -7, dtype=torch.int32).cuda()
    o = sala.sparse_decode_paged(q.cuda(), cache.k, cache.v, cache.table, kbar, zero + N - 1, N - 1, topk, 1, 2,
                                 idx_out=idx)
    sala.check_status()
    idx = idx.cpu()
    for kv in range(Hkv):
        blocks = sorted(set(idx[0, kv].tolist()) - {-1})
        assert len(blocks) == 1 + 2 + topk and {0, 15} <= set(blocks), blocks
        seen = torch.zeros((1, N), dtype=torch.bool)
        for b in blocks:
            seen[:, 64 * b:64 * b + 64] = True
        for h in range(kv * H // Hkv, (kv + 1) * H // Hkv):
            ref = sp.attention64(q[0, h:h + 1], k[kv], v[kv], seen)
            _close(o[0, h:h + 1], *ref, 64 * len(blocks), _tag(dtype, "sparse decode over written pages"))


@pytest.mark.parametrize("B", [4, 1500])  # offsets in shared memory, and too many for it
@pytest.mark.parametrize("at,off", [(1, 60), (2, 3), (0, -5), (-1, 140), (-2, 140)])
def test_cache_calls_flag_offsets_out_of_order(sala, B, at, off):  # noqa: F811
    # a pair that descends, also where no row can tell; a first offset below 0, a last one behind total
    Hkv, d, total = 2, 64, 100
    k, v = (torch.randn((Hkv, total, d), generator=torch.Generator().manual_seed(51)).to(BF16).cuda() for _ in range(2))
    cu = torch.full((B + 1,), total, dtype=torch.int32)
    cu[:4] = torch.tensor([0, 20, 40, 70])
    good = cu.cuda()
    cu[at] = off
    table = torch.arange(4 * B, dtype=torch.int32).reshape(B, 4).cuda()
    pos = torch.zeros(B, dtype=torch.int32).cuda()
    kp, vp = (torch.zeros((4 * B, Hkv, 64, d), dtype=BF16).cuda() for _ in range(2))
    for c, bad in ((cu.cuda(), True), (good, False)):
        for call in (lambda: sala.kv_write(k, v, c, pos, table, kp, vp),
                     lambda: sala.kv_read(kp, vp, table, c, pos, total, BF16)):
            call()
            if bad:
                with pytest.raises(sala.SalaError) as err:
                    sala.check_status()
                assert err.value.code == sala.ERR_BOUNDS
            else:
                sala.check_status()
    rk, rv = sala.kv_read(kp, vp, table, good, pos, total, BF16)
    assert torch.equal(rk, k) and torch.equal(rv, v)


# ---------------------------------------------------------------------------------------------
# The main cases of the bf16 kernels at the bound of the instructions that they use

def _instruction_bound(A, e, n):
    """serving_plain.bound for bf16 with its 1e-4 for the exponential replaced by what the kernels' own steps
    cost: ex2.approx 2^-22 of a weight, lg2.approx (V's scales in exponents) 2^-22 of an exponent, both once more
    in the normaliser, together at most 2^-20; and n + 8 additions in 32 bits, 2^-24 each."""
    return A * (2 * e[..., None] + 2.0 ** -7 + 2.0 ** -20 + (n + 8) * 2.0 ** -24) + 1e-30


@pytest.mark.parametrize("H,Hkv,d,dtype,lens", [c for c in PACKED if c[3] == BF16])
def test_packed_cases_at_the_instructions_bound(sala, H, Hkv, d, dtype, lens):  # noqa: F811
    q, k, v = _packed_inputs(H, Hkv, d, dtype, sum(lens), seed=61)
    out = sala.packed_prefill(q.cuda(), k.cuda(), v.cuda(), sp.offsets(lens).cuda())
    sala.check_status()
    o, A, e = sp.packed64(q, k, v, lens)
    assert bool(((out.double().cpu() - o).abs() <= _instruction_bound(A, e, max(lens))).all())


@pytest.mark.parametrize("H,Hkv,d,dtype,fmt,T,ctx", [c for c in TREE if c[3] == BF16])
def test_tree_cases_at_the_instructions_bound(sala, H, Hkv, d, dtype, fmt, T, ctx):  # noqa: F811
    q, cache, tree = _tree_inputs(H, Hkv, d, dtype, fmt, T, ctx, seed=62, fill=NAN)
    out = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    o, A, e = _tree_ref(q, cache, ctx, tree)
    n = max(ctx) + T
    floor = _floor(fmt, [cache.dense64(b, 0, c + T) for b, c in enumerate(ctx)], n) if H // Hkv * T <= 16 else 0.0
    assert bool(((out.double().cpu() - o).abs() <= _instruction_bound(A, e, n) + floor).all())
