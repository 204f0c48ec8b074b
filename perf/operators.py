"""Operators of the dense serving path: packed prompt attention, the quantised paged cache, and
the attention of drafted tokens over it.  Each case is one call (for the cache, a write and the
read that follows it) as a serving program makes it.

Three operators:

* ``packed``: causal softmax attention over whole prompts of different lengths, laid one behind
  the other; q [H, total, d], k and v [Hkv, total, d], ``cu`` [B + 1] row offsets.
* ``cache``: new key and value rows are quantised (8-bit integers, or e4m3 with power-of-two
  scales, one scale per token and head) into pages of 64 tokens, then a span of each sequence is
  read back as dense rows.
* ``tree``: T drafted tokens per sequence attend to their sequence's whole context and, among the
  drafts, to those their mask names (their ancestors in the draft tree and themselves), over the
  paged cache in the inputs' own type or in 8 bits.  T = 1 is the plain decode step.

Where ``own`` is false the operators run as elementary torch operations in 32 bits."""
import math
import random

import torch

own = False

PAGE = 64
INT8, E4M3 = "int8", "e4m3"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FLOOR = 2.0 ** -100  # smallest largest-magnitude a row's scale is made from


# ---------------------------------------------------------------------------------------------
# Cases

def _packed(name, H, Hkv, d, dt, lens):
    return {"name": name, "op": "packed", "H": H, "Hkv": Hkv, "d": d, "dt": dt, "lens": lens}


def _cache(name, Hkv, d, dt, fmt, start, new, back):
    """start: tokens already cached, new: tokens written, back: tokens read (the last ``back``)."""
    return {"name": name, "op": "cache", "Hkv": Hkv, "d": d, "dt": dt, "fmt": fmt, "start": start,
            "new": new, "back": back}


def _tree(name, H, Hkv, d, dt, fmt, T, ctx):
    return {"name": name, "op": "tree", "H": H, "Hkv": Hkv, "d": d, "dt": dt, "fmt": fmt, "T": T,
            "ctx": ctx}


def _join(xs):
    return ",".join(str(x) for x in xs)


def _ints(text):
    return [int(x) for x in text.split(",")]


def listed():
    return [
        # one short question: latency
        _packed("packed one short", 32, 2, 128, "bf16", "37"),
        # a server's batch of waiting prompts, ragged, one of them empty and one a single token
        _packed("packed ragged batch", 32, 2, 128, "bf16",
                "517,1,2048,0,129,64,1411,333,4096,15,700,128,77,1000,250,2501"),
        # one long document
        _packed("packed long", 32, 2, 128, "bf16", "32768"),
        # the fp32 form at the small head size, eight query heads over two key heads
        _packed("packed fp32", 8, 2, 64, "f32", "700,1,0,513,835"),
        # a decode step of 64 conversations: one token each appended, the block it falls into read
        # back for its mean
        _cache("cache decode step", 2, 128, "bf16", INT8,
               _join((i * 977 + 63) % 8192 for i in range(64)), _join([1] * 64),
               _join(((i * 977 + 63) % 8192) % 64 + 1 for i in range(64))),
        # prompts taken in pieces: four pieces written, the whole prefixes read back dense
        _cache("cache prompt pieces", 2, 128, "bf16", E4M3, "8192,0,4100,12345",
               "2048,2048,1500,2048", "10240,2048,5600,14393"),
        # a long document written whole and read whole
        _cache("cache long prompt", 2, 128, "bf16", INT8, "0", "262144", "262144"),
        # fp32 rows of the small head size
        _cache("cache fp32", 2, 64, "f32", E4M3, "100,0,63", "1000,1,65", "1000,1,128"),
        # one conversation, one token, short context: latency
        _tree("tree one token", 32, 2, 128, "bf16", "bf16", 1, "1000"),
        # a server's decode step over long quantised caches
        _tree("tree tokens long", 32, 2, 128, "bf16", INT8, 1, "262144,100001,196608,231072"),
        # sixteen conversations, a draft tree of eight tokens each
        _tree("tree batch", 32, 2, 128, "bf16", E4M3, 8,
              "8000,0,1,63,4096,777,12000,64,2500,16000,9999,130,5,32000,7001,1023"),
        # the widest draft tree over one long context in the inputs' own type
        _tree("tree wide", 32, 2, 128, "bf16", "bf16", 64, "131072"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, total, n):
    """n lengths, zeros among them, that sum to total."""
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


HEADS = [(32, 2, 128)] * 4 + [(16, 1, 128), (8, 2, 64), (4, 4, 128), (6, 2, 64), (12, 4, 128)]


def draw(rng):
    op = rng.choice(["packed", "cache", "tree"])
    H, Hkv, d = rng.choice(HEADS)
    dt = "f32" if rng.random() < 0.2 else "bf16"
    if op == "packed":
        total = _log(rng, 1, 3000 if dt == "f32" else 28000)
        B = min(_log(rng, 1, 64), total)
        c = _packed("", H, Hkv, d, dt, _join(_split(rng, total, B)))
    elif op == "cache":
        B = _log(rng, 1, 64)
        # at most the bytes of the longest listed document
        new = _split(rng, _log(rng, 1, 200000 * 512 // (Hkv * d * (4 if dt == "f32" else 2))), B)
        if rng.random() < 0.3:
            new = [1] * B
        start = [rng.randint(0, _log(rng, 1, 2000)) for _ in range(B)]
        back = [min(n + rng.randint(0, 100), n + s) for n, s in zip(new, start)]
        c = _cache("", Hkv, d, dt, rng.choice([INT8, E4M3]), _join(start), _join(new), _join(back))
    else:
        T = rng.choice([1, 1, 2, 5, 8, 16, 33, 64])
        B = _log(rng, 1, 32)
        most = _log(rng, 64, 100000 if dt == "bf16" else 8000)
        ctx = [rng.randint(0, max(1, most // B)) if rng.random() < 0.9 else 0 for _ in range(B)]
        c = _tree("", H, Hkv, d, dt, rng.choice([dt, INT8, E4M3]), T, _join(ctx))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------
# Inputs

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, shape, dtype, dev):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)


def _keys(g, Hkv, n, d, dtype, dev):
    """Keys with a shared direction per head: one row in fifty leans towards it, so some logits
    stand out as they do in a trained model."""
    u = torch.randn((Hkv, 1, d), generator=g, device=dev)
    lean = (torch.rand((Hkv, n, 1), generator=g, device=dev) < 0.02).float() * 0.5
    return (torch.randn((Hkv, n, d), generator=g, device=dev) + lean * u).to(dtype), u


def _queries(g, u, H, n, d, dtype, dev):
    return (torch.randn((H, n, d), generator=g, device=dev)
            + u.repeat_interleave(H // u.shape[0], dim=0)).to(dtype)


def _offsets(lens, dev):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=dev)


def _pages_of(lens, g, dev):
    """A page table [B, most pages] over a shuffled pool that holds a few pages no one owns."""
    need = [-(-n // PAGE) for n in lens]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, n_pages


def _empty_cache(n_pages, Hkv, d, dt, fmt, dev):
    kind = {INT8: torch.int8, E4M3: torch.float8_e4m3fn}.get(fmt, TYPES[dt])
    kp = torch.zeros((n_pages, Hkv, PAGE, d), dtype=kind, device=dev)
    if fmt == dt:
        return kp, torch.zeros_like(kp), None, None
    sc = torch.ones((n_pages, Hkv, PAGE), dtype=torch.float32, device=dev)
    return kp, torch.zeros_like(kp), sc, sc.clone()


def _draft_trees(seed, B, T, dev):
    """Bit rows [B, T]: bit j of row i says that draft i attends to draft j.  Drafts come in an
    order in which parents stand before their children."""
    rng = random.Random(seed)
    rows = []
    for _ in range(B):
        anc = []
        for i in range(T):
            parent = rng.randint(-1, i - 1)
            anc.append((anc[parent] if parent >= 0 else 0) | (1 << i))
        rows.append([a - (1 << 64) if a >> 63 else a for a in anc])
    return torch.tensor(rows, dtype=torch.int64, device=dev)


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype, d, Hkv = TYPES[case["dt"]], case["d"], case["Hkv"]
    s = dict(case)
    if case["op"] == "packed":
        s["lens"] = _ints(case["lens"])
        n = sum(s["lens"])
        s["k"], u = _keys(g, Hkv, n, d, dtype, dev)
        s["v"] = _normal(g, (Hkv, n, d), dtype, dev)
        s["q"] = _queries(g, u, case["H"], n, d, dtype, dev)
        s["cu"] = _offsets(s["lens"], dev)
        return s
    if case["op"] == "cache":
        start, new, back = _ints(case["start"]), _ints(case["new"]), _ints(case["back"])
        end = [a + b for a, b in zip(start, new)]
        s["table"], n_pages = _pages_of(end, g, dev)
        s["kp"], s["vp"], s["ks"], s["vs"] = _empty_cache(n_pages, Hkv, d, case["dt"], case["fmt"], dev)
        # what stands in the cache already
        old, old_v = (_normal(g, (Hkv, sum(start), d), dtype, dev) for _ in range(2))
        if sum(start):
            _write(s, old, old_v, _offsets(start, dev), torch.zeros(len(start), dtype=torch.int32, device=dev))
        s["k"], _ = _keys(g, Hkv, sum(new), d, dtype, dev)
        s["v"] = _normal(g, (Hkv, sum(new), d), dtype, dev)
        s["cu"], s["pos"] = _offsets(new, dev), torch.tensor(start, dtype=torch.int32, device=dev)
        s["cu_back"] = _offsets(back, dev)
        s["pos_back"] = torch.tensor([e - n for e, n in zip(end, back)], dtype=torch.int32, device=dev)
        s["n_back"] = sum(back)
        return s
    ctx, T = _ints(case["ctx"]), case["T"]
    B = len(ctx)
    total = [c + T for c in ctx]
    s["table"], n_pages = _pages_of(total, g, dev)
    s["kp"], s["vp"], s["ks"], s["vs"] = _empty_cache(n_pages, Hkv, d, case["dt"], case["fmt"], dev)
    k, u = _keys(g, Hkv, sum(total), d, dtype, dev)
    v = _normal(g, (Hkv, sum(total), d), dtype, dev)
    _write(s, k, v, _offsets(total, dev), torch.zeros(B, dtype=torch.int32, device=dev))
    q = _queries(g, u, case["H"], B * T, d, dtype, dev)
    s["q"] = q.reshape(case["H"], B, T, d).transpose(0, 1).contiguous()
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    s["max_ctx"] = max(ctx)
    s["lens"] = ctx
    s["tree"] = _draft_trees(seed, B, T, dev)
    return s


# ---------------------------------------------------------------------------------------------
# Plain forms

def _quantise(x, fmt):
    """Rows of x (last axis) as codes and one fp32 scale each; a row with an infinity or a NaN
    gets the scale NaN and codes 0.  int8: scale = amax / 127, code = the integer nearest to
    x * (127 / amax), each factor a 32-bit number, the product exact.  e4m3: scale = the smallest
    power of two that keeps amax / scale within 448, so the quotient is exact."""
    x = x.float()
    amax = x.abs().amax(-1)
    good = torch.isfinite(x).all(-1)
    a = torch.where(good, amax, torch.ones_like(amax)).clamp_min(FLOOR)
    x = torch.where(good[..., None], x, torch.zeros_like(x))
    if fmt == INT8:
        scale = a / 127
        codes = (x.double() * (127 / a).double()[..., None]).round().to(torch.int8)
    else:
        m, e = torch.frexp(a)
        e = e - 9 + (m > 0.875).to(e.dtype)
        scale = torch.ldexp(torch.ones_like(a), e)
        codes = (x / scale[..., None]).to(torch.float8_e4m3fn)
    return codes, torch.where(good, scale, torch.full_like(scale, float("nan")))


def _places(cu, pos, table, n):
    """Page and slot of each of n packed rows: row r of sequence b stands at pos[b] + r - cu[b]."""
    r = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu.long(), r, right=True) - 1
    p = pos.long()[b] + r - cu.long()[b]
    return table.long()[b, p // PAGE], p % PAGE


def _raw(pages):
    return pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages


def _write(s, k, v, cu, pos):
    page, slot = _places(cu, pos, s["table"], k.shape[1])
    for x, pages, scales in ((k, s["kp"], s["ks"]), (v, s["vp"], s["vs"])):
        if scales is None:
            pages[page, :, slot] = x.transpose(0, 1)
            continue
        codes, sc = _quantise(x, s["fmt"])
        _raw(pages)[page, :, slot] = _raw(codes).transpose(0, 1)
        scales[page, :, slot] = sc.t()


def _value(pages, scales, page, slot):
    """fp32 rows [n, Hkv, d] (slot a tensor) or whole pages (slot a slice)."""
    x = _raw(pages)[page, :, slot]
    x = (x.view(torch.float8_e4m3fn) if pages.dtype == torch.float8_e4m3fn else x).float()
    return x if scales is None else x * scales[page, :, slot][..., None]


def _softmax_av(q, k, v, seen):
    """q [Hkv, rows, d], k and v [Hkv, keys, d] in fp32, seen broadcastable to [Hkv, rows, keys]."""
    x = torch.where(seen, q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1]), float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return (p / p.sum(-1, keepdim=True)) @ v


def _plain_packed(s):
    H, Hkv, d = s["H"], s["Hkv"], s["d"]
    G = H // Hkv
    out, at = torch.empty_like(s["q"]), 0
    for n in s["lens"]:
        k, v = s["k"][:, at:at + n].float(), s["v"][:, at:at + n].float()
        step = max(64, (1 << 28) // (H * max(n, 1)))  # query rows whose logits take about 1 GB
        for i in range(0, n, step):
            m = min(step, n - i)
            q = s["q"][:, at + i:at + i + m].float().reshape(Hkv, G * m, d)
            seen = (torch.arange(i + m, device=q.device)
                    <= torch.arange(i, i + m, device=q.device)[:, None]).repeat(G, 1)
            o = _softmax_av(q, k[:, :i + m], v[:, :i + m], seen)
            out[:, at + i:at + i + m] = o.reshape(H, m, d).to(out.dtype)
        at += n
    return out


def _plain_cache(s):
    _write(s, s["k"], s["v"], s["cu"], s["pos"])
    page, slot = _places(s["cu_back"], s["pos_back"], s["table"], s["n_back"])
    return tuple(_value(p, sc, page, slot).transpose(0, 1).contiguous().to(s["k"].dtype)
                 for p, sc in ((s["kp"], s["ks"]), (s["vp"], s["vs"])))


def _plain_tree(s):
    q, T, Hkv, d = s["q"], s["T"], s["Hkv"], s["d"]
    out = torch.empty_like(q)
    bits = (s["tree"][..., None] >> torch.arange(T, device=q.device)) & 1  # [B, T, T]
    for b, c in enumerate(s["lens"]):
        n = c + T
        page = s["table"][b, :-(-n // PAGE)].long()
        k, v = (_value(p, sc, page, slice(None)).transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
                for p, sc in ((s["kp"], s["ks"]), (s["vp"], s["vs"])))
        seen = torch.ones((T, n), dtype=torch.bool, device=q.device)
        seen[:, c:] = bits[b].bool()
        G = q.shape[1] // Hkv
        o = _softmax_av(q[b].float().reshape(Hkv, G * T, d), k, v, seen.repeat(G, 1))
        out[b] = o.reshape(-1, T, d).to(out.dtype)
    return out


def run(state):
    s = state
    if not own:
        return {"packed": _plain_packed, "cache": _plain_cache, "tree": _plain_tree}[s["op"]](s)
    from hybrid_sparse_linear_b200 import sala
    if s["op"] == "packed":
        return sala.packed_prefill(s["q"], s["k"], s["v"], s["cu"])
    if s["op"] == "cache":
        sala.kv_write(s["k"], s["v"], s["cu"], s["pos"], s["table"], s["kp"], s["vp"],
                      k_scale=s["ks"], v_scale=s["vs"])
        return sala.kv_read(s["kp"], s["vp"], s["table"], s["cu_back"], s["pos_back"], s["n_back"],
                            s["k"].dtype, k_scale=s["ks"], v_scale=s["vs"])
    if "ws" not in s:  # a server keeps one workspace for its steps
        s["ws"] = torch.empty(max(16, sala.tree_decode_paged_workspace_bytes(
            len(s["lens"]), s["H"], s["Hkv"], s["T"], s["max_ctx"], s["d"])),
            dtype=torch.uint8, device=s["q"].device)
    return sala.tree_decode_paged(s["q"], s["kp"], s["vp"], s["table"], s["ctx"], s["max_ctx"],
                                  s["tree"], k_scale=s["ks"], v_scale=s["vs"], workspace=s["ws"])


# ---------------------------------------------------------------------------------------------
# Work

def work(case):
    es, d, Hkv = 2 if case["dt"] == "bf16" else 4, case["d"], case["Hkv"]
    if case["op"] == "packed":
        lens, H = _ints(case["lens"]), case["H"]
        n = sum(lens)
        return {"bytes": 2 * (H + Hkv) * n * d * es + 4 * (len(lens) + 1),
                "flops": sum(4 * d * H * n * (n + 1) // 2 for n in lens)}
    if case["op"] == "cache":
        new, back = _ints(case["new"]), _ints(case["back"])
        # dense rows in, codes and scales out; codes and scales in, dense rows out
        return {"bytes": 2 * Hkv * (sum(new) + sum(back)) * (d * es + d + 4),
                "flops": 2 * Hkv * d * (3 * sum(new) + sum(back))}
    ctx, T, H = _ints(case["ctx"]), case["T"], case["H"]
    row = d * es if case["fmt"] == case["dt"] else d + 4
    keys = sum(c + T for c in ctx)
    return {"bytes": 2 * Hkv * keys * row + 2 * len(ctx) * H * T * d * es + 8 * len(ctx) * T,
            "flops": 4 * d * H * T * keys}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits

def _row_softmax64(q, k, v, hidden):
    """One key head: q [rows, d], k and v [keys, d], hidden [rows, keys] (True: not attended)."""
    x = torch.einsum("rd,kd->rk", q, k) * q.shape[1] ** -0.5
    x.masked_fill_(hidden, -math.inf)
    x = torch.softmax(x, 1)
    return torch.einsum("rk,kd->rd", x, v)


def _codes64(x, fmt):
    """The values that the quantised rows x [.., d] stand for."""
    x = x.double()
    top = x.abs().max(-1, keepdim=True).values.clamp(min=FLOOR)
    if fmt == INT8:  # the scale and its reciprocal are 32-bit numbers
        scale, per = (top / 127).float().double(), (127 / top).float().double()
        return torch.round(x * per) * scale
    scale = torch.exp2(torch.ceil(torch.log2(top / 448)))
    y = x / scale
    # e4m3 near y: steps of 2^(floor(log2 |y|) - 3), of 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * scale


def exact(case, seed):
    s = prepare(case, seed)
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] == "packed":
        H, G = case["H"], case["H"] // Hkv
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        at = 0
        for n in _ints(case["lens"]):
            for h in range(H if n else 0):
                k, v = (s[x][h // G, at:at + n].double() for x in "kv")
                for i in range(0, n, 8192):
                    m = min(n, i + 8192)
                    hidden = torch.ones((m - i, m), dtype=torch.bool, device=k.device).triu(i + 1)
                    out[h, at + i:at + m] = _row_softmax64(s["q"][h, at + i:at + m].double(),
                                                           k[:m], v[:m], hidden)
            at += n
        return out
    table = s["table"].tolist()
    if case["op"] == "cache":
        new, start, back = (_ints(case[x]) for x in ("new", "start", "back"))
        got = []
        for x, pages, scales in ((s["k"], s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
            fresh, at = _codes64(x, case["fmt"]), 0
            parts = []
            for b, (a, n, m) in enumerate(zip(start, new, back)):
                if m > n:  # rows that stood there before the write
                    p = torch.arange(a + n - m, a, device=x.device)
                    own_pages = torch.tensor(table[b], device=x.device)[p // PAGE]
                    c = _raw(pages)[own_pages, :, p % PAGE]
                    c = c.view(pages.dtype).to(torch.float64)
                    parts.append((c * scales[own_pages, :, p % PAGE].double()[..., None]).transpose(0, 1))
                parts.append(fresh[:, at + n - min(n, m):at + n])
                at += n
            got.append(torch.cat(parts, 1))
        return tuple(got)
    T, G = case["T"], case["H"] // Hkv
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b, c in enumerate(_ints(case["ctx"])):
        n = c + T
        ids = table[b][:-(-n // PAGE)]
        hidden = torch.zeros((T, n), dtype=torch.bool, device=out.device)
        for i, row in enumerate(s["tree"][b].tolist()):
            hidden[i, c:] = torch.tensor([not (row >> j) & 1 for j in range(T)])
        for g in range(Hkv):
            kv = []
            for pages, scales in ((s["kp"], s["ks"]), (s["vp"], s["vs"])):
                x = _raw(pages)[ids, g].view(pages.dtype).double()
                kv.append((x if scales is None else x * scales[ids, g].double()[..., None]).reshape(-1, d)[:n])
            rows = s["q"][b, g * G:(g + 1) * G].double().reshape(G * T, d)
            out[b, g * G:(g + 1) * G] = _row_softmax64(rows, *kv, hidden.repeat(G, 1)).reshape(G, T, d)
    return out
