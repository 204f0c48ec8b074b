"""The dense serving path on the GPU against its plain 64-bit forms: packed prompt attention, the
quantised paged cache and the attention of new tokens over it, each alone and in a run."""
import math

import pytest
import torch

import serving_plain as sp
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def sala():
    from hybrid_sparse_linear_b200 import sala as s
    return s


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(g, shape, dtype, mul=1.0):
    return (torch.randn(shape, generator=g) * mul).to(dtype)


def _close(out, o, A, e, n_keys, what=""):
    out = out.double().cpu()
    tol = sp.bound(A, e, n_keys, bf16=n_keys is not None and what.startswith("bf16"))
    assert bool(torch.isfinite(out).all()), f"{what}: non-finite"
    over = (out - o).abs() - tol
    assert float(over.max()) <= 0, f"{what}: off by {float((out - o).abs().max()):.3e}, {float(over.max()):.3e} over the bound"


def _tag(dtype, what):
    return ("bf16 " if dtype == BF16 else "fp32 ") + what


# ---------------------------------------------------------------------------------------------
# Packed prompts

PACKED = [
    (32, 2, 128, BF16, [37]),
    (32, 2, 128, BF16, [1]),
    (32, 2, 128, BF16, [517, 1, 0, 129, 64, 15, 300]),
    (16, 1, 128, BF16, [0, 130, 0, 255, 256, 257, 0]),
    (8, 2, 64, BF16, [200, 3, 128]),
    (4, 4, 128, BF16, [300, 129, 1, 127]),   # one query head per KV head
    (6, 2, 64, BF16, [70, 260]),             # three
    (12, 4, 128, BF16, [33, 190]),
    (24, 1, 128, BF16, [5, 140]),            # twenty-four
    (64, 2, 64, BF16, [45, 150]),            # thirty-two
    (2, 1, 128, BF16, [400, 100]),
    (32, 2, 128, F32, [37, 0, 200, 1, 65]),
    (8, 2, 64, F32, [130, 64, 63]),
    (6, 2, 128, F32, [150]),
]


def _packed_inputs(H, Hkv, d, dtype, n, seed=0, mul=1.0):
    g = _gen(seed)
    return _rand(g, (H, n, d), dtype, mul), _rand(g, (Hkv, n, d), dtype, mul), _rand(g, (Hkv, n, d), dtype)


@pytest.mark.parametrize("H,Hkv,d,dtype,lens", PACKED)
def test_packed_prefill(sala, H, Hkv, d, dtype, lens):
    n = sum(lens)
    q, k, v = _packed_inputs(H, Hkv, d, dtype, n)
    out = Guarded((H, n, d), dtype)
    sala.packed_prefill(q.cuda(), k.cuda(), v.cuda(), sp.offsets(lens).cuda(), o=out.t)
    sala.check_status()
    out.check("packed_prefill")
    _close(out.t, *sp.packed64(q, k, v, lens), max(lens), _tag(dtype, "packed"))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_prefill_peaked_rows_and_a_scale(sala, dtype):
    # logits up to about 100: rows settle on one key, the running maximum moves by many steps
    lens = [400, 77]
    q, k, v = _packed_inputs(32, 2, 128, dtype, sum(lens), seed=1, mul=3.0)
    k[:, 0::50] *= 2
    out = sala.packed_prefill(q.cuda(), k.cuda(), v.cuda(), sp.offsets(lens).cuda(), scale=0.11)
    sala.check_status()
    _close(out, *sp.packed64(q, k, v, lens, 0.11), max(lens), _tag(dtype, "peaked"))


@pytest.mark.parametrize("H,Hkv,d,dtype", [(32, 2, 128, BF16), (4, 4, 128, BF16), (8, 2, 64, BF16), (8, 2, 64, F32)])
def test_packed_prefill_hidden_infinities(sala, H, Hkv, d, dtype):
    # An infinity or a NaN in a later token, another sequence or behind the last one reaches only
    # the rows that see it.
    lens, spare = [150, 40, 129], 70
    n = sum(lens)
    q, k, v = _packed_inputs(H, Hkv, d, dtype, n + spare, seed=2)
    base = [x.clone() for x in (q, k, v)]
    v[:, 100, 3] = NAN                  # sequence 0, token 100
    v[:, 140, 5] = math.inf
    k[:, 145] = NAN
    v[:, 189, 7] = -math.inf            # the last token of sequence 1
    for x in (q, k, v):
        x[:, n:] = NAN
    out = torch.full((H, n + spare, d), 7.0, dtype=dtype, device="cuda")
    sala.packed_prefill(q.cuda(), k.cuda(), v.cuda(), sp.offsets(lens).cuda(), o=out)
    sala.check_status()
    got = out.double().cpu()
    assert bool((got[:, n:] == 7.0).all()), "rows behind the last sequence were written"
    o, A, e = sp.packed64(*base, lens)
    clean = torch.ones((H, n, d), dtype=torch.bool)
    clean[:, 100:150, 3] = False
    clean[:, 140:150, 5] = False
    clean[:, 145:150] = False
    clean[:, 189, 7] = False
    tol = sp.bound(A, e, max(lens), dtype == BF16)
    assert bool(((got[:, :n] - o).abs() <= tol)[clean].all())
    assert bool(torch.isnan(got[:, 100:145, 3]).all())
    assert bool((got[:, 140:145, 5] == math.inf).all())
    assert bool(torch.isnan(got[:, 145:150]).all())
    assert bool((got[:, 189, 7] == -math.inf).all())


def test_packed_prefill_many_sequences_and_order(sala):
    # more sequences than a warp has lanes, many of them empty; equal bits on a second run
    g = _gen(3)
    lens = [int(x) for x in torch.randint(0, 40, (150,), generator=g)]
    lens[::3] = [0] * len(lens[::3])
    n = sum(lens)
    q, k, v = _packed_inputs(32, 2, 128, BF16, n, seed=4)
    args = q.cuda(), k.cuda(), v.cuda(), sp.offsets(lens).cuda()
    a, b = sala.packed_prefill(*args), sala.packed_prefill(*args)
    sala.check_status()
    assert torch.equal(a, b)
    _close(a, *sp.packed64(q, k, v, lens), max(lens), "bf16 many")


def test_packed_prefill_long_rows_sampled(sala):
    # one sequence long enough that every CTA takes several units, checked at sampled rows
    n, H, Hkv, d = 64 * 130 + 11, 32, 2, 128
    q, k, v = _packed_inputs(H, Hkv, d, BF16, n, seed=5)
    out = sala.packed_prefill(q.cuda(), k.cuda(), v.cuda(), sp.offsets([n]).cuda()).cpu()
    sala.check_status()
    for i in (0, 1, 127, 128, 4095, 4096, n - 2, n - 1, 6001):
        for h in (0, 15, 16, 31):
            seen = torch.ones((1, i + 1), dtype=torch.bool)
            o, A, e = sp.attention64(q[h, i:i + 1], k[h // 16, :i + 1], v[h // 16, :i + 1], seen)
            _close(out[h, i:i + 1], o, A, e, i + 1, "bf16 long")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_prefill_bad_offsets_are_flagged(sala, dtype):
    q, k, v = (x.cuda() for x in _packed_inputs(32, 2, 128, dtype, 100, seed=6))
    for cu in ([0, 60, 40, 100], [0, 60, 140], [-5, 60, 100]):
        sala.packed_prefill(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
        with pytest.raises(sala.SalaError) as err:
            sala.check_status()
        assert err.value.code == sala.ERR_BOUNDS
    sala.packed_prefill(q, k, v, sp.offsets([60, 40]).cuda())
    sala.check_status()


# ---------------------------------------------------------------------------------------------
# The cache

@pytest.mark.parametrize("fmt", ["same", "int8", "e4m3"])
@pytest.mark.parametrize("dtype,d,Hkv", [(BF16, 128, 2), (BF16, 64, 3), (F32, 64, 2), (F32, 128, 1)])
def test_cache_write_and_read(sala, fmt, dtype, d, Hkv):
    pos, new, spare = [0, 63, 130, 5, 0, 64], [130, 2, 0, 1, 1, 64], 9
    g = _gen(7)
    n = sum(new)
    k, v = (_rand(g, (Hkv, n + spare, d), dtype) for _ in range(2))
    k *= torch.exp(torch.randn((Hkv, n + spare, 1), generator=g) * 4).to(dtype)
    k[:, 3] = 0
    v[0, 5, 1] = math.inf
    v[0, 6] = NAN
    k[0, 7] = 1e-38                     # below the floor of a scale
    end = [a + b for a, b in zip(pos, new)]
    want = sp.Cache(end, Hkv, d, dtype, fmt, seed=1, fill=3)
    have = sp.Cache(end, Hkv, d, dtype, fmt, seed=1, fill=3).cuda()
    cu = sp.offsets(new)
    at = 0
    for b in range(len(new)):
        want.put(b, pos[b], k[:, at:at + new[b]], v[:, at:at + new[b]])
        at += new[b]
    p32 = torch.tensor(pos, dtype=torch.int32)
    sala.kv_write(k.cuda(), v.cuda(), cu.cuda(), p32.cuda(), have.table, have.k, have.v, have.ks, have.vs)
    sala.check_status()
    have.cpu()
    raw = (lambda x: x.view(torch.uint8)) if fmt == "e4m3" else (lambda x: x)
    for a, b in ((have.k, want.k), (have.v, want.v)):
        torch.testing.assert_close(raw(a), raw(b), rtol=0, atol=0, equal_nan=True)
    if fmt != "same":
        for a, b in ((have.ks, want.ks), (have.vs, want.vs)):
            torch.testing.assert_close(a, b, rtol=0, atol=0, equal_nan=True)
    # read the tail of each sequence back, across the old tokens too
    back = [min(e, 70) for e in end]
    start = [e - m for e, m in zip(end, back)]
    m = sum(back)
    ko, vo = Guarded((Hkv, m + 2, d), dtype), Guarded((Hkv, m + 2, d), dtype)
    have.cuda()
    sala.kv_read(have.k, have.v, have.table, sp.offsets(back).cuda(),
                 torch.tensor(start, dtype=torch.int32).cuda(), m + 2, dtype, have.ks, have.vs,
                 k=ko.t, v=vo.t)
    sala.check_status()
    ko.check("kv_read k", all_written=False)
    vo.check("kv_read v", all_written=False)
    fill = torch.full((Hkv, 2, d * ko.t.element_size()), 0xA5, dtype=torch.uint8)
    for x in (ko, vo):
        assert torch.equal(x.t[:, m:].contiguous().view(torch.uint8).cpu(), fill), "rows behind the last sequence"
    at = 0
    for b in range(len(back)):
        rk, rv = want.dense64(b, start[b], back[b])
        for x, ref in ((ko.t, rk), (vo.t, rv)):
            torch.testing.assert_close(x[:, at:at + back[b]].cpu(), ref.to(F32).to(dtype), rtol=0, atol=0,
                                       equal_nan=True)
        at += back[b]


def test_cache_bad_pages_and_positions_are_flagged_and_skipped(sala):
    Hkv, d = 2, 128
    g = _gen(8)
    k, v = (_rand(g, (Hkv, 100, d), BF16).cuda() for _ in range(2))
    cu = sp.offsets([70, 30]).cuda()
    for table, pos in (([[0, 9], [1, 2]], [0, 0]), ([[0, -1], [1, 2]], [0, 0]), ([[0, 3], [1, 2]], [0, 200]),
                       ([[0, 3], [1, 2]], [0, -1])):
        kp, vp = (torch.zeros((4, Hkv, 64, d), dtype=torch.int8, device="cuda") for _ in range(2))
        ks, vs = (torch.ones((4, Hkv, 64), device="cuda") for _ in range(2))
        t = torch.tensor(table, dtype=torch.int32, device="cuda")
        p = torch.tensor(pos, dtype=torch.int32, device="cuda")
        sala.kv_write(k, v, cu, p, t, kp, vp, ks, vs)
        with pytest.raises(sala.SalaError) as err:
            sala.check_status()
        assert err.value.code == sala.ERR_BOUNDS
        assert bool(kp[0].any())                       # the rows whose page is named are written
        out = torch.full((Hkv, 100, d), 7.0, dtype=BF16, device="cuda")
        out2 = out.clone()
        sala.kv_read(kp, vp, t, cu, p, 100, BF16, ks, vs, k=out, v=out2)
        with pytest.raises(sala.SalaError):
            sala.check_status()
        bad = slice(64, 70) if pos[1] == 0 else slice(70, 100)
        assert bool((out[:, bad] == 7.0).all())
        assert bool((out[:, :64] != 7.0).any())


# ---------------------------------------------------------------------------------------------
# New tokens over the cache

TREE = [
    # H, Hkv, d, dtype, fmt, T, ctx
    (32, 2, 128, BF16, "same", 1, [1000]),
    (32, 2, 128, BF16, "int8", 1, [0, 63, 64, 65, 700]),
    (32, 2, 128, BF16, "e4m3", 8, [300, 0, 1, 127, 128, 60]),
    (32, 2, 128, BF16, "same", 64, [130, 0, 500]),
    (16, 1, 128, BF16, "int8", 33, [77, 250]),
    (8, 2, 64, BF16, "same", 5, [190, 3]),
    (8, 2, 64, BF16, "int8", 16, [100]),
    (8, 2, 64, BF16, "e4m3", 2, [129]),
    (4, 4, 128, BF16, "same", 7, [200, 64]),
    (6, 2, 64, BF16, "e4m3", 64, [90, 10]),
    (12, 4, 128, BF16, "int8", 3, [255]),
    (24, 1, 128, BF16, "same", 11, [140]),
    (32, 2, 128, F32, "same", 1, [500, 0]),
    (8, 2, 64, F32, "int8", 9, [100, 64]),
    (6, 2, 128, F32, "e4m3", 64, [70]),
    # contexts long enough to be split over CTAs, and CTAs with several items
    (32, 2, 128, BF16, "same", 1, [5000, 0, 1700, 64, 2999]),
    (32, 2, 128, BF16, "int8", 1, [4000, 1, 2111]),
    (32, 2, 128, BF16, "e4m3", 1, [63, 7000]),
    (8, 2, 64, BF16, "int8", 4, [6000, 0, 33]),
    (16, 1, 128, BF16, "e4m3", 8, [5000, 700, 0, 0, 129]),
    (32, 2, 128, BF16, "same", 5, [3000, 64, 1000, 2, 0, 511]),
    (32, 2, 128, BF16, "int8", 40, [1500, 0, 300]),
    (8, 2, 64, BF16, "same", 64, [2500]),
    (32, 2, 128, F32, "int8", 2, [2000, 0, 100]),
]


def _tree_inputs(H, Hkv, d, dtype, fmt, T, ctx, seed=0, mul=1.0, fill=0):
    g = _gen(seed)
    B = len(ctx)
    cache = sp.Cache([c + T for c in ctx], Hkv, d, dtype, fmt, seed=seed, fill=fill)
    for b, c in enumerate(ctx):
        cache.put(b, 0, _rand(g, (Hkv, c + T, d), dtype, mul), _rand(g, (Hkv, c + T, d), dtype))
    q = _rand(g, (B, H, T, d), dtype, mul)
    parents = [[int(torch.randint(-1, max(i, 1), (1,), generator=g)) if i else -1 for i in range(T)] for _ in range(B)]
    tree = torch.tensor([sp.signed(sp.ancestors(p)) for p in parents], dtype=torch.int64)
    return q, cache, tree


def _tree_run(sala, q, cache, ctx, tree, **kw):
    c = cache.cuda()
    out = sala.tree_decode_paged(q.cuda(), c.k, c.v, c.table, torch.tensor(ctx, dtype=torch.int32).cuda(),
                                 max(ctx), tree.cuda(), c.ks, c.vs, **kw)
    cache.cpu()
    return out


def _tree_ref(q, cache, ctx, tree, scale=0.0):
    kv = [cache.dense64(b, 0, c + q.shape[2]) for b, c in enumerate(ctx)]
    return sp.tree64(q, [x[0] for x in kv], [x[1] for x in kv], ctx, tree, scale)


@pytest.mark.parametrize("H,Hkv,d,dtype,fmt,T,ctx", TREE)
def test_tree_decode(sala, H, Hkv, d, dtype, fmt, T, ctx):
    # slots behind the last token hold NaN (in the 8-bit formats: codes 0 with scale NaN)
    q, cache, tree = _tree_inputs(H, Hkv, d, dtype, fmt, T, ctx, fill=NAN)
    out = Guarded(q.shape, dtype)
    _tree_run(sala, q, cache, ctx, tree, o=out.t)
    sala.check_status()
    out.check("tree_decode_paged")
    _close(out.t, *_tree_ref(q, cache, ctx, tree), max(ctx) + T, _tag(dtype, "tree"))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fmt", ["same", "int8", "e4m3"])
@pytest.mark.parametrize("T,ctx", [(1, [0, 65, 130, 63]), (8, [1, 100, 128]), (64, [70])])
def test_tree_decode_any_bytes_in_unused_slots(sala, dtype, fmt, T, ctx):
    # slots behind the last token and pages no one owns hold every byte, and scales of every kind
    q, cache, tree = _tree_inputs(32, 2, 128, dtype, fmt, T, ctx, seed=6)
    used = torch.zeros((cache.n_pages, 64), dtype=torch.bool)
    for b, c in enumerate(ctx):
        p = torch.arange(c + T)
        used[cache.table[b][p // 64].long(), p % 64] = True
    free = ~used[:, None, :].expand(-1, 2, -1)
    g = _gen(7)
    for x in (cache.k, cache.v):
        raw = x.view(torch.uint8)
        noise = torch.randint(0, 256, raw.shape, generator=g, dtype=torch.uint8)
        noise[..., ::7] = 0x7f  # e4m3's NaN; in the wider types' upper bytes NaN and infinities
        noise[..., 1::7] = 0xff
        raw[free] = noise[free]
    if cache.ks is not None:
        odd = torch.tensor([NAN, math.inf, -math.inf, -1.0, 0.0, 1e30, 1e-40])
        for x in (cache.ks, cache.vs):
            x[free] = odd[torch.randint(0, 7, x.shape, generator=g)][free]
    out = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    _close(out, *_tree_ref(q, cache, ctx, tree), max(ctx) + T, _tag(dtype, "any bytes"))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("T", [1, 8])
def test_tree_decode_scales_far_apart(sala, fmt, T):
    # V rows whose scales differ by 2^80, one row of zeros, and queries far from 1
    ctx = [300, 40]
    q, cache, tree = _tree_inputs(32, 2, 128, BF16, fmt, T, ctx, seed=8)
    q[0] *= 2.0 ** 40
    q[1, :, ::3] *= 2.0 ** -30
    cache.ks[cache.table[0, :5].long()] *= 2.0 ** -40   # the logits stay as they were
    e = torch.randint(-40, 41, cache.vs.shape, generator=_gen(9)).float()
    cache.vs.mul_(torch.exp2(e))
    cache.vs[int(cache.table[0, 0]), :, 5] = 0.0
    out = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    _close(out, *_tree_ref(q, cache, ctx, tree), 310, _tag(BF16, "far scales"))


@pytest.mark.parametrize("dtype,fmt,T", [(BF16, "int8", 1), (BF16, "e4m3", 1), (BF16, "same", 1), (BF16, "int8", 16),
                                         (F32, "int8", 1)])
def test_tree_decode_one_key_above_a_long_flat_tail(sala, dtype, fmt, T):
    # One key of 700032 weighs 1, each other 2^-25.5, which together is 1.5 % of it: nearly twice the bound.
    # Every tail page of the table is the same page; the result follows from the two kinds of keys.
    n, d, w = 700032, 64, 2.0 ** -25.5
    kind = {"same": dtype, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[fmt]
    k, v = torch.zeros((2, 1, 64, d)), torch.full((2, 1, 64, d), 64.0)
    k[0, 0, 0, 0] = 64.0
    v[0, 0, 0] = -64.0
    v[0, 0, 0, ::2] = 0.0
    ks, vs = (None, None) if fmt == "same" else (torch.full((2, 1, 64), x).cuda() for x in (1.0, 1.0))
    q = torch.zeros((1, 1, T, d), dtype=dtype)
    q[..., 0] = 1.0
    table = torch.ones((1, n // 64), dtype=torch.int32)
    table[0, 0] = 0
    tree = torch.tensor([sp.signed([1 << t for t in range(T)])])  # a row sees the context and itself
    out = sala.tree_decode_paged(q.cuda(), k.to(kind).cuda(), v.to(kind).cuda(), table.cuda(),
                                 torch.tensor([n - T], dtype=torch.int32).cuda(), n - T, tree.cuda(), ks, vs,
                                 scale=25.5 * math.log(2.0) / 64)
    sala.check_status()
    tail = (n - T) * w  # the context's keys but one, and the row's own
    peak = v[0, 0, 0].double()
    o, A = ((x + tail * 64.0) / (1.0 + tail) for x in (peak, peak.abs()))
    # the scale is rounded to 32 bits: 2^-24 of a logit of 17.7 on top of the product's error
    e = torch.full((1, 1, T), 17.7 * (d + 5) * 2.0 ** -24, dtype=torch.float64)
    _close(out, o.expand(1, 1, T, d), A.expand(1, 1, T, d), e, n, _tag(dtype, "flat tail"))


@pytest.mark.parametrize("dtype,fmt", [(BF16, "same"), (BF16, "int8"), (F32, "e4m3")])
def test_tree_decode_peaked_rows_and_a_scale(sala, dtype, fmt):
    q, cache, tree = _tree_inputs(32, 2, 128, dtype, fmt, 4, [600, 90], seed=1, mul=3.0)
    out = _tree_run(sala, q, cache, [600, 90], tree, scale=0.11)
    sala.check_status()
    _close(out, *_tree_ref(q, cache, [600, 90], tree, 0.11), 700, _tag(dtype, "peaked tree"))


@pytest.mark.parametrize("dtype,fmt", [(BF16, "same"), (BF16, "int8"), (BF16, "e4m3"), (F32, "same")])
def test_tree_decode_rows_that_see_nothing(sala, dtype, fmt):
    ctx, T = [0, 200], 6
    q, cache, tree = _tree_inputs(32, 2, 128, dtype, fmt, T, ctx, seed=2)
    tree[0] = torch.tensor([0, 2, 0, 0b101000, -64, 0])   # -64: bits at and above T only
    tree[1] = 0
    out = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    assert not out[0, :, [0, 2, 4, 5]].any()
    tree[0, 4] = 0
    _close(out, *_tree_ref(q, cache, ctx, tree), 210, _tag(dtype, "empty rows"))


@pytest.mark.parametrize("dtype,fmt,T", [(BF16, "same", 8), (BF16, "same", 64), (BF16, "int8", 8),
                                         (F32, "same", 8), (F32, "int8", 8)])
def test_tree_decode_hidden_infinities(sala, dtype, fmt, T):
    # a NaN or an infinity in a new token reaches the rows that attend to it and no other
    ctx = [190, 0]
    q, cache, tree = _tree_inputs(32, 2, 128, dtype, fmt, T, ctx, seed=3)
    tree[:] = torch.tensor(sp.signed([1 << t for t in range(T)]))  # every draft sees itself
    tree[:, 5] |= 1 << 2
    tree[:, 7] |= 1 << 4
    o, A, e = _tree_ref(q, cache, ctx, tree)
    for b, c in enumerate(ctx):
        for j, col, val, what in ((2, 3, NAN, "v"), (4, 9, math.inf, "v"), (6, 0, NAN, "k")):
            page, slot = int(cache.table[b, (c + j) // 64]), (c + j) % 64
            if fmt == "same":
                (cache.v if what == "v" else cache.k)[page, :, slot, col] = val
            else:
                (cache.vs if what == "v" else cache.ks)[page, :, slot] = NAN
    out = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    got = out.double().cpu()
    hit = torch.zeros(got.shape, dtype=torch.bool)
    cols = (lambda c: [c]) if fmt == "same" else (lambda c: list(range(128)))
    for t in (2, 5):
        hit[:, :, t, cols(3)] = True
    for t in (4, 7):
        hit[:, :, t, cols(9)] = True
    hit[:, :, 6] = True
    assert bool(((got - o).abs() <= sp.bound(A, e, 200, dtype == BF16))[~hit].all())
    assert not bool(torch.isfinite(got[hit]).any())
    if fmt == "same":
        assert bool(torch.isnan(got[:, :, 2, 3]).all()) and bool((got[:, :, 4, 9] == math.inf).all())


def test_tree_decode_batch_longer_than_a_warp_and_same_bits(sala):
    g = _gen(9)
    ctx = [int(x) for x in torch.randint(0, 400, (70,), generator=g)]
    q, cache, tree = _tree_inputs(32, 2, 128, BF16, "int8", 3, ctx, seed=4)
    a, b = (_tree_run(sala, q, cache, ctx, tree) for _ in range(2))
    sala.check_status()
    assert torch.equal(a, b)
    _close(a, *_tree_ref(q, cache, ctx, tree), 410, "bf16 batch")


@pytest.mark.parametrize("H,Hkv,d,lens", [(8, 2, 64, [70, 1] * 25), (8, 2, 64, [300, 0, 65]), (32, 2, 128, [200, 150]),
                                          (4, 4, 128, [130, 17])])
def test_packed_prefill_fp32_block_sizes(sala, H, Hkv, d, lens):
    # blocks of 32 rows while all of 64 would run at once, else of 64
    q, k, v = _packed_inputs(H, Hkv, d, F32, sum(lens), seed=21)
    out = sala.packed_prefill(q.cuda(), k.cuda(), v.cuda(), sp.offsets(lens).cuda())
    sala.check_status()
    _close(out, *sp.packed64(q, k, v, lens), max(lens), "fp32 blocks")


@pytest.mark.parametrize("fmt", ["same", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d,T,ctx", [(32, 2, 128, 1, [9000]), (32, 2, 128, 2, [700, 0, 64]), (32, 2, 128, 5, [300]),
                                           (8, 2, 64, 4, [20000, 3]), (8, 2, 64, 7, [1000, 100]), (8, 2, 64, 33, [100]),
                                           (4, 4, 128, 1, [200] * 9)])
def test_tree_decode_fp32_block_sizes(sala, H, Hkv, d, T, ctx, fmt):
    # blocks of 16, 32 and 64 rows; one block per SM, and more
    q, cache, tree = _tree_inputs(H, Hkv, d, F32, fmt, T, ctx, seed=22, fill=NAN)
    out = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    _close(out, *_tree_ref(q, cache, ctx, tree), max(ctx) + T, "fp32 blocks")


@pytest.mark.parametrize("fmt,n,top", [("int8", 64, 2500), ("same", 64, 2500), ("same", 10, 2500), ("int8", 64, 4200)])
def test_tree_decode_many_items_of_middle_lengths(sala, fmt, n, top):
    # a block per item, or equal runs of pages over the blocks, by the number of items and their pages
    g = _gen(12)
    ctx = [top, 0, 1, 64] + [int(x) for x in torch.randint(0, 300, (n - 4,), generator=g)]
    q, cache, tree = _tree_inputs(32, 2, 128, BF16, fmt, 1, ctx, seed=11, fill=NAN)
    out = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    _close(out, *_tree_ref(q, cache, ctx, tree), top + 1, "bf16 many items")


@pytest.mark.parametrize("fmt", ["same", "int8"])
@pytest.mark.parametrize("T,n,top", [(2, 3, 400), (2, 3, 700), (8, 40, 900), (8, 40, 1200), (2, 60, 1900), (33, 2, 450),
                                     (33, 2, 600), (64, 16, 2200)])
def test_tree_decode_items_and_runs(sala, fmt, T, n, top):
    # a block per item or equal runs of key tiles, on both sides of the choice
    g = _gen(24)
    ctx = [top, 0, 64][:n] + [int(x) for x in torch.randint(0, 100, (max(n - 3, 0),), generator=g)]
    q, cache, tree = _tree_inputs(32, 2, 128, BF16, fmt, T, ctx, seed=23, fill=NAN)
    a, b = (_tree_run(sala, q, cache, ctx, tree) for _ in range(2))
    sala.check_status()
    assert torch.equal(a, b)
    _close(a, *_tree_ref(q, cache, ctx, tree), top + T, "bf16 items and runs")


@pytest.mark.parametrize("dtype,fmt", [(BF16, "same"), (BF16, "e4m3"), (F32, "same")])
def test_tree_decode_bad_pages_and_contexts_are_flagged(sala, dtype, fmt):
    ctx = [200, 100]
    q, cache, tree = _tree_inputs(32, 2, 128, dtype, fmt, 2, ctx, seed=5)
    good = _tree_run(sala, q, cache, ctx, tree)
    sala.check_status()
    page = int(cache.table[0, 1])
    for bad in (-1, cache.n_pages + 5):
        cache.table[0, 1] = bad
        out = _tree_run(sala, q, cache, ctx, tree)
        with pytest.raises(sala.SalaError) as err:
            sala.check_status()
        assert err.value.code == sala.ERR_BOUNDS
        assert torch.equal(out[1], good[1])            # the other sequence is untouched
        # the page's keys are left out
        cache.table[0, 1] = page
        k, v = ([x] for x in cache.dense64(0, 0, 202))
        keep = torch.ones((2, 202), dtype=torch.bool)
        keep[:, 64:128] = False
        for t in range(2):
            for j in range(2):
                keep[t, 200 + j] = bool((int(tree[0, t]) >> j) & 1)
        for h in (0, 31):
            o, A, e = sp.attention64(q[0, h], k[0][h // 16], v[0][h // 16], keep)
            _close(out[0, h], o, A, e, 202, _tag(dtype, "bad page"))
    c = cache.cuda()
    for lens in ([200, 300], [200, -1]):
        sala.tree_decode_paged(q.cuda(), c.k, c.v, c.table, torch.tensor(lens, dtype=torch.int32).cuda(), 200,
                               tree.cuda(), c.ks, c.vs)
        with pytest.raises(sala.SalaError) as err:
            sala.check_status()
        assert err.value.code == sala.ERR_BOUNDS


def test_tree_decode_pages_shared_by_sequences(sala):
    # two sequences with a common prefix of 128 tokens in the same pages
    q, cache, tree = _tree_inputs(32, 2, 128, BF16, "int8", 2, [200, 180], seed=13)
    cache.table[1, :2] = cache.table[0, :2]
    out = _tree_run(sala, q, cache, [200, 180], tree)
    sala.check_status()
    _close(out, *_tree_ref(q, cache, [200, 180], tree), 202, "bf16 shared pages")


def test_more_sequences_than_the_staged_offsets(sala):
    # 1500 short sequences: the cache calls search the offsets in global memory
    g = _gen(14)
    lens = [int(x) for x in torch.randint(0, 4, (1500,), generator=g)]
    n, Hkv, d = sum(lens), 2, 128
    q, k, v = _packed_inputs(32, Hkv, d, BF16, n, seed=15)
    cu, pos = sp.offsets(lens).cuda(), torch.randint(0, 60, (1500,), generator=g, dtype=torch.int32).cuda()
    o = sala.packed_prefill(q.cuda(), k.cuda(), v.cuda(), cu)
    table = torch.randperm(1500, generator=g).to(torch.int32)[:, None].contiguous().cuda()
    kp, vp = (torch.zeros((1500, Hkv, 64, d), dtype=BF16, device="cuda") for _ in range(2))
    sala.kv_write(k.cuda(), v.cuda(), cu, pos, table, kp, vp)
    rk, rv = sala.kv_read(kp, vp, table, cu, pos, n, BF16)
    sala.check_status()
    assert torch.equal(rk.cpu(), k) and torch.equal(rv.cpu(), v)
    b = torch.searchsorted(cu.cpu().long(), torch.arange(n), right=True) - 1
    at = pos.cpu().long()[b] + torch.arange(n) - cu.cpu().long()[b]
    assert torch.equal(kp.cpu()[table.cpu()[b, 0].long(), :, at].transpose(0, 1), k)
    _close(o, *sp.packed64(q, k, v, lens), 4, "bf16 short sequences")


# ---------------------------------------------------------------------------------------------
# Streams, graphs, a run of them together

@pytest.mark.parametrize("dtype,fmt", [(BF16, "int8"), (BF16, "same"), (F32, "e4m3")])
def test_a_served_run(sala, dtype, fmt):
    """Prompts attended whole, their keys cached, drafts appended and verified, the accepted path
    written over them, one more token decoded; and the prefix read back for block_compress."""
    H, Hkv, d, lens, T = 32, 2, 128, [150, 1, 64], 4
    n, B = sum(lens), len(lens)
    g = _gen(10)
    q, k, v = _rand(g, (H, n, d), dtype), _rand(g, (Hkv, n, d), dtype), _rand(g, (Hkv, n, d), dtype)
    cache = sp.Cache([m + T for m in lens], Hkv, d, dtype, fmt, fill=NAN).cuda()
    pages = cache.table, cache.k, cache.v, cache.ks, cache.vs
    zero, ctx = torch.zeros(B, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    o = sala.packed_prefill(q.cuda(), k.cuda(), v.cuda(), sp.offsets(lens).cuda())
    sala.kv_write(k.cuda(), v.cuda(), sp.offsets(lens).cuda(), zero, *pages)
    kd, vd = _rand(g, (Hkv, B * T, d), dtype), _rand(g, (Hkv, B * T, d), dtype)
    sala.kv_write(kd.cuda(), vd.cuda(), sp.offsets([T] * B).cuda(), ctx, *pages)
    qd = _rand(g, (B, H, T, d), dtype)
    tree = torch.tensor([sp.ancestors([-1, 0, 0, 2])] * B)
    od = sala.tree_decode_paged(qd.cuda(), cache.k, cache.v, cache.table, ctx, max(lens), tree.cuda(),
                                cache.ks, cache.vs)
    sala.check_status()
    _close(o, *sp.packed64(q, k, v, lens), max(lens), _tag(dtype, "prompt"))
    cache.cpu()
    ref = _tree_ref(qd, cache, lens, tree)
    _close(od, *ref, max(lens) + T, _tag(dtype, "drafts"))
    # drafts 0, 2, 3 accepted: their rows again, behind the context
    keep = [0, 2, 3]
    rows = torch.tensor([b * T + i for b in range(B) for i in keep])
    cache.cuda()
    pages = cache.table, cache.k, cache.v, cache.ks, cache.vs
    sala.kv_write(kd[:, rows].cuda(), vd[:, rows].cuda(), sp.offsets([3] * B).cuda(), ctx, *pages)
    q1 = qd[:, :, 3:].contiguous()
    o1 = sala.tree_decode_paged(q1.cuda(), cache.k, cache.v, cache.table, ctx + 2, max(lens) + 2,
                                torch.ones((B, 1), dtype=torch.int64).cuda(), cache.ks, cache.vs)
    full = [m + 3 for m in lens]
    rk, _ = sala.kv_read(cache.k, cache.v, cache.table, sp.offsets(full).cuda(), zero, sum(full), dtype,
                         cache.ks, cache.vs)
    kbar = sala.block_compress(rk[None, :, :full[0]].contiguous())
    sala.check_status()
    # the accepted path's last token sees what draft 3 saw: both are within the bound of that row
    tol = 2 * sp.bound(*ref[1:], max(lens) + T, dtype == BF16)[:, :, 3:]
    cache.cpu()
    kv = [cache.dense64(b, 0, m + 3) for b, m in enumerate(lens)]
    ones = torch.ones((B, 1), dtype=torch.int64)
    _close(o1, *sp.tree64(q1, [x[0] for x in kv], [x[1] for x in kv], [m + 2 for m in lens], ones),
           max(lens) + T, _tag(dtype, "accepted"))
    assert bool(((o1.double().cpu() - od[:, :, 3:].double().cpu()).abs() <= tol).all())
    mean = kv[0][0][:, :128].to(F32).to(dtype).double().reshape(Hkv, 2, 64, d).mean(2)
    torch.testing.assert_close(kbar[0].double().cpu(), mean, rtol=2.0 ** -7, atol=1e-6)


def test_serving_calls_on_another_stream_and_captured(sala):
    H, Hkv, d, lens, T, fmt = 32, 2, 128, [150, 30], 3, "int8"
    n = sum(lens)
    g = _gen(11)
    q, k, v = (_rand(g, (h, n, d), BF16).cuda() for h in (H, Hkv, Hkv))
    qd = _rand(g, (2, H, T, d), BF16).cuda()
    cache = sp.Cache([190, 190], Hkv, d, BF16, fmt).cuda()
    cu, ctx = sp.offsets(lens).cuda(), torch.tensor([m - T for m in lens], dtype=torch.int32).cuda()
    zero = torch.zeros(2, dtype=torch.int32).cuda()
    tree = torch.tensor([sp.ancestors([-1, 0, 0])] * 2).cuda()
    ws = torch.empty(sala.tree_decode_paged_workspace_bytes(2, H, Hkv, T, 180, d), dtype=torch.uint8).cuda()

    def step(**kw):
        o = sala.packed_prefill(q, k, v, cu, **kw)
        sala.kv_write(k, v, cu, zero, cache.table, cache.k, cache.v, cache.ks, cache.vs, **kw)
        od = sala.tree_decode_paged(qd, cache.k, cache.v, cache.table, ctx, 180, tree, cache.ks,
                                    cache.vs, workspace=ws, **kw)
        r = sala.kv_read(cache.k, cache.v, cache.table, cu, zero, n, BF16, cache.ks, cache.vs, **kw)
        return (o, od) + r

    ref = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in (dict(stream=side), dict()):
        with torch.cuda.stream(side) if not kw else torch.cuda.stream(torch.cuda.current_stream()):
            got = step(**kw)
        side.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(2):
        q.mul_(-0.5)
        k.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)
    # other lengths in the same buffers: nothing of them is baked into the graph
    cu.copy_(sp.offsets([31, 149]))
    ctx.copy_(torch.tensor([20, 140], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, step()):
        assert torch.equal(a, b)
    sala.check_status()


def test_two_tree_calls_at_once(sala):
    # two streams, each with its own workspace
    q, cache, tree = _tree_inputs(32, 2, 128, BF16, "e4m3", 2, [500, 100], seed=12)
    ref = _tree_run(sala, q, cache, [500, 100], tree)
    c = cache.cuda()
    qd, td, ctx = q.cuda(), tree.cuda(), torch.tensor([500, 100], dtype=torch.int32).cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s in streams:
            outs.append(sala.tree_decode_paged(qd, c.k, c.v, c.table, ctx, 500, td, c.ks, c.vs, stream=s))
    torch.cuda.synchronize()
    sala.check_status()
    for o in outs:
        assert torch.equal(o, ref)


def test_binding_refuses(sala):
    q, kv = torch.zeros((32, 8, 128), dtype=BF16).cuda(), torch.zeros((2, 8, 128), dtype=BF16).cuda()
    cu = sp.offsets([8]).cuda()
    with pytest.raises(ValueError, match="contiguous"):
        sala.packed_prefill(q.transpose(0, 1).contiguous().transpose(0, 1), kv, kv, cu)
    with pytest.raises(ValueError, match="dtype"):
        sala.packed_prefill(q, kv.float(), kv.float(), cu)
    with pytest.raises(ValueError, match="shape"):
        sala.packed_prefill(q, kv[:, :4].contiguous(), kv[:, :4].contiguous(), cu)
    with pytest.raises(ValueError, match="dtype"):
        sala.packed_prefill(q, kv, kv, cu.long())
    with pytest.raises(TypeError):
        sala.packed_prefill(q.half(), kv.half(), kv.half(), cu)
    kp = torch.zeros((3, 2, 64, 128), dtype=torch.int8).cuda()
    sc = torch.ones((3, 2, 64)).cuda()
    table, pos = torch.zeros((1, 2), dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
    with pytest.raises(ValueError, match="k_scale"):
        sala.kv_write(kv, kv, cu, pos, table, kp, kp)
    with pytest.raises(ValueError, match="shape"):
        sala.kv_write(kv, kv, cu, pos, table, kp, kp, sc, sc[:2].contiguous())
    with pytest.raises(ValueError, match="dtype"):
        sala.kv_write(kv, kv, cu, pos, table, kp.to(torch.uint8), kp.to(torch.uint8), sc, sc)
    tree = torch.ones((1, 2), dtype=torch.int64).cuda()
    qd = torch.zeros((1, 32, 2, 128), dtype=BF16).cuda()
    with pytest.raises(ValueError, match="shape"):
        sala.tree_decode_paged(qd, kp, kp, table, pos, 8, tree[:, :1].contiguous(), sc, sc)
    with pytest.raises(ValueError, match="max_ctx"):
        sala.tree_decode_paged(qd, kp, kp, table, pos, 1 << 32, tree, sc, sc)
    with pytest.raises(sala.SalaError, match="workspace"):
        sala.tree_decode_paged(qd, kp, kp, table, pos, 8, tree, sc, sc,
                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
