"""Plain 64-bit forms of the dense serving path, and the error bounds of its kernels (test
infrastructure, not collected).  torch on the CPU, one sequence and one head at a time.

Bounds.  With p the softmax weights and A = sum_j p_j |v_j| (so |o| <= A), a kernel's output is off
by at most

* bf16: 2^-8 A for the weights rounded to bf16 before the product with V, 2^-8 |o| for the rounded
  output, and for the weights themselves: 1e-4 A (the exponential's polynomial is 7.5e-5 off) plus
  twice the error of a logit (a weight's relative error is its logit's absolute error, and the
  normaliser has it once more).
* fp32: the same without the bf16 terms, with 2^-22 for the exponential and (n + 8) 2^-24 A for
  sums over n keys.
* A logit scale * q.k is a sum of d products in 32 bits: (d + 4) 2^-24 scale sum_c |q_c k_c| off,
  the maximum over the keys taken for all.
"""
from __future__ import annotations

import math

import torch

PAGE = 64
FLOOR = 2.0 ** -100


def attention64(q, k, v, seen, scale=0.0):
    """q [rows, d], k and v [keys, d] (any type), seen [rows, keys] bool.  Returns (o, bound inputs):
    o [rows, d] fp64, zeros where a row sees nothing; A as above; the logit error term per row.
    Hidden keys and values take no part, whatever they hold."""
    q, k, v = q.double(), k.double(), v.double()
    scale = scale or 1.0 / math.sqrt(q.shape[1])
    o, A = torch.zeros_like(q), torch.zeros_like(q)
    e = torch.zeros(q.shape[0], dtype=torch.float64)
    if len(q) and len(k) and bool(torch.isfinite(k).all()) and bool(torch.isfinite(v).all()):  # all rows at once
        some = seen.any(1)
        x = (q @ k.T * scale).masked_fill(~seen, -math.inf)[some]
        w = torch.exp(x - x.amax(1, keepdim=True))
        w = w / w.sum(1, keepdim=True)
        o[some], A[some] = w @ v, w @ v.abs()
        e[some] = ((q.abs() @ k.abs().T) * seen).amax(1)[some] * scale * (q.shape[1] + 4) * 2.0 ** -24
        return o, A, e
    groups = {}
    for i in range(q.shape[0]):
        groups.setdefault(seen[i].numpy().tobytes(), []).append(i)
    for rows in groups.values():
        at = seen[rows[0]].nonzero()[:, 0]
        if not len(at):
            continue
        x = q[rows] @ k[at].T * scale
        w = torch.exp(x - x.amax(1, keepdim=True))
        w = w / w.sum(1, keepdim=True)
        o[rows], A[rows] = w @ v[at], w @ v[at].abs()
        e[rows] = (q[rows].abs() @ k[at].abs().T).amax(1) * scale * (q.shape[1] + 4) * 2.0 ** -24
    return o, A, e


def bound(A, e, n_keys, bf16):
    rel = 2 * e[..., None] + (2 * 2.0 ** -8 + 1e-4 if bf16 else 2.0 ** -22 + (n_keys + 8) * 2.0 ** -24)
    return A * rel + 1e-30


def packed64(q, k, v, lens, scale=0.0):
    """q [H, total, d], k and v [Hkv, total, d].  Returns o, A, e over the rows of the sequences."""
    H, G = q.shape[0], q.shape[0] // k.shape[0]
    n = sum(lens)
    o = torch.zeros((H, n, q.shape[2]), dtype=torch.float64)
    A, e = torch.zeros_like(o), torch.zeros((H, n), dtype=torch.float64)
    at = 0
    for m in lens:
        seen = torch.ones((m, m), dtype=torch.bool).tril()
        for h in range(H):
            r = slice(at, at + m)
            o[h, r], A[h, r], e[h, r] = attention64(q[h, r], k[h // G, r], v[h // G, r], seen, scale)
        at += m
    return o, A, e


def tree64(q, k, v, ctx, tree, scale=0.0):
    """q [B, H, T, d]; k, v: lists of [Hkv, ctx_b + T, d]; tree [B, T] int64 bits."""
    B, H, T, _ = q.shape
    o = torch.zeros(q.shape, dtype=torch.float64)
    A, e = torch.zeros_like(o), torch.zeros(q.shape[:3], dtype=torch.float64)
    for b in range(B):
        c, G = ctx[b], H // k[b].shape[0]
        seen = torch.ones((T, c + T), dtype=torch.bool)
        for t in range(T):
            for j in range(T):
                seen[t, c + j] = bool((int(tree[b, t]) >> j) & 1)
        for h in range(H):
            o[b, h], A[b, h], e[b, h] = attention64(q[b, h], k[b][h // G], v[b][h // G], seen, scale)
    return o, A, e


def quantise64(x, fmt):
    """Codes' values (before the scale) and scales of the rows of x [..., d], exactly."""
    x = x.double()
    good = torch.isfinite(x).all(-1)
    x = torch.where(good[..., None], x, torch.zeros_like(x))
    a = x.abs().amax(-1).clamp_min(FLOOR)
    if fmt == "int8":
        scale, mul = (a / 127).float().double(), (127 / a).float().double()
        code = torch.round(x * mul[..., None])
    else:
        scale = torch.exp2(torch.ceil(torch.log2(a / 448)))
        y = x / scale[..., None]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        code = torch.round(y / step) * step
    return code, torch.where(good, scale, torch.full_like(scale, math.nan))


KIND = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


class Cache:
    """A page pool filled on the host: sequences' pages scattered over it, unused pages between."""

    def __init__(self, lens, Hkv, d, dtype, fmt, seed=0, spare=3, fill=0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // PAGE) for n in lens]
        self.n_pages = sum(need) + spare
        perm = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.fmt, self.Hkv, self.d, self.dtype = fmt, Hkv, d, dtype
        shape = (self.n_pages, Hkv, PAGE, d)
        if fmt == "same":
            self.k = torch.full(shape, fill, dtype=dtype)
            self.ks = self.vs = None
        else:
            self.k = torch.full(shape, 0, dtype=torch.uint8).view(KIND[fmt])
            self.ks = torch.full(shape[:3], fill, dtype=torch.float32)
            self.vs = self.ks.clone()
        self.v = self.k.clone()

    def put(self, b, pos, k, v):
        """Tokens pos.. of sequence b from dense rows [Hkv, n, d]."""
        for i in range(k.shape[1]):
            page, slot = int(self.table[b, (pos + i) // PAGE]), (pos + i) % PAGE
            for x, pages, sc in ((k, self.k, self.ks), (v, self.v, self.vs)):
                if self.fmt == "same":
                    pages[page, :, slot] = x[:, i]
                else:
                    code, scale = quantise64(x[:, i], self.fmt)
                    pages.view(torch.uint8)[page, :, slot] = code.float().to(KIND[self.fmt]).view(torch.uint8)
                    sc[page, :, slot] = scale.float()

    def dense64(self, b, pos, n):
        """The values that tokens pos .. pos + n - 1 stand for: (k, v) [Hkv, n, d] fp64."""
        p = torch.arange(pos, pos + n)
        page, slot = self.table[b][p // PAGE].long(), p % PAGE
        out = []
        for pages, sc in ((self.k, self.ks), (self.v, self.vs)):
            raw = pages.view(torch.uint8) if self.fmt == "e4m3" else pages
            x = raw[page, :, slot].view(pages.dtype).double()
            if sc is not None:
                x = x * sc[page, :, slot].double()[..., None]
            out.append(x.transpose(0, 1).contiguous())
        return out

    def cuda(self):
        for n in ("k", "v", "ks", "vs", "table"):
            x = getattr(self, n)
            if x is not None:
                setattr(self, n, x.cuda())
        return self

    def cpu(self):
        for n in ("k", "v", "ks", "vs", "table"):
            x = getattr(self, n)
            if x is not None:
                setattr(self, n, x.cpu())
        return self


def ancestors(parents):
    """Mask bits of a draft tree given each draft's parent (-1: hangs on the context)."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
    return bits


def signed(bits):
    return [b - (1 << 64) if b >> 63 else b for b in bits]


def offsets(lens):
    return torch.tensor([0] + torch.tensor(lens, dtype=torch.int64).cumsum(0).tolist(), dtype=torch.int32)
