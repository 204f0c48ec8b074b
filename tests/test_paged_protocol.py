"""A model of the roles and barriers of the kernel for drafted tokens over a paged cache (more than 16 rows
per KV head), in its wide and narrow form, over bf16 pages and 8-bit codes, run as the packed kernel's is.
No GPU."""
import random

import pytest

from test_packed_protocol import Barrier

CONV = 2  # converting warps in the model (eight in the kernel)


class Kernel:
    """items: per item its key tiles, each (drafts, page held): drafts in the last one or two."""

    def __init__(self, items, wide, codes, rng, ring=4, raw=3):
        self.items, self.wide, self.codes, self.rng, self.R, self.raw_n = items, wide, codes, rng, ring, raw
        many = lambda n, c: [Barrier(c) for _ in range(n)]  # noqa: E731
        rings = 1 if wide else 2
        self.full = [many(ring, CONV if codes else 1) for _ in range(rings)]
        self.empty = [many(ring, (2 if wide else 1) * (5 if codes else 1)) for _ in range(rings)]
        self.raw_full, self.raw_empty = many(raw, 1), many(raw, CONV)
        self.q_full, self.q_empty = many(2, 1), Barrier(2)
        self.s_full, self.p_full, self.pv_done = ([many(2, c) for _ in range(2)] for c in (1, 4, 1))
        self.v_landed, self.look_free, self.v_seen = many(2, 1), many(2, 1), many(2, 1)
        self.both_done, self.merged = Barrier(8), Barrier(8)
        self.item_full, self.item_empty = many(2, 1), many(2, 10 + (CONV if codes else 0))
        self.item, self.lk = [None, None], [None, None]
        self.slot = [[None] * ring for _ in range(rings)]  # (item, kind, tile, who still needs it)
        self.raws = [None] * raw
        self.q = [None, None]
        self.s = [[None, None], [None, None]]
        self.o, self.readers, self.noted = [None, None], [set(), set()], -1
        self.pipe, self.loads = [[], []], []
        self.roles = {"load": self.load()}
        if codes:
            for w in range(CONV):
                self.roles[f"conv{w}"] = self.conv(w)
        else:
            self.roles["look"] = self.look()
        for x in range(2):
            self.roles[f"issue{x}"] = self.issue(x)
            for w in range(4):
                self.roles[f"soft{x}{w}"] = self.soft(x, w)

    def ring_of(self, x):
        return 0 if self.wide else x

    def mine(self, n, x):
        return n if self.wide else (n + 1 - x) // 2

    def nth(self, k, x):
        return k if self.wide else 2 * k + x

    def take(self, it):
        yield ("wait", self.item_full[it & 1], (it >> 1) & 1)

    def users(self):
        return {0, 1} if self.wide else {0}

    def load(self):
        rc, rr, kq, looks, it = [0, 0], 0, 0, 0, 0
        while True:
            if it >= 2:
                yield ("wait", self.item_empty[it & 1], ((it - 2) >> 1) & 1)
            tiles = self.items[it] if it < len(self.items) else None
            self.item[it & 1] = tiles
            self.item_full[it & 1].arrive()
            if tiles is None:
                break
            if kq >= 1:
                yield ("wait", self.q_empty, (kq - 1) & 1)
            for x in range(2 if self.wide else 1):
                def land(x=x, it=it):
                    self.q[x] = it
                    self.q_full[x].arrive()
                self.loads.append(land)
            kq += 1
            for i, (drafts, have) in enumerate(tiles):
                for j in range(2):
                    if self.codes:
                        q = rr % self.raw_n
                        if rr >= self.raw_n:
                            yield ("wait", self.raw_empty[q], ((rr - self.raw_n) // self.raw_n) & 1)
                        rr += 1

                        def land(q=q, i=i, j=j, it=it):
                            self.raws[q] = (it, "KV"[j], i)
                            self.raw_full[q].arrive()
                        self.loads.append(land)
                        continue
                    x = 0 if self.wide else i & 1
                    e = rc[x]
                    q = e % self.R
                    if e >= self.R:
                        yield ("wait", self.empty[x][q], ((e - self.R) // self.R) & 1)
                    look = j == 1 and (drafts or not have)
                    if look and looks >= 2:
                        yield ("wait", self.look_free[looks & 1], ((looks - 2) >> 1) & 1)
                    if look:
                        assert self.lk[looks & 1] is None, "a look was overwritten"
                        self.lk[looks & 1] = (x, q, it, drafts and i == len(tiles) - 1)
                    bar = self.v_landed[looks & 1] if look else self.full[x][q]

                    def land(x=x, q=q, i=i, j=j, it=it, bar=bar):
                        self.put(x, q, it, "KV"[j], i)
                        bar.arrive()
                    self.loads.append(land)
                    looks += look
                    rc[x] += 1
            it += 1
        if not self.codes:
            if looks >= 2:
                yield ("wait", self.look_free[looks & 1], ((looks - 2) >> 1) & 1)
            self.lk[looks & 1] = (0, 0, -1, False)
            self.v_landed[looks & 1].arrive()

    def put(self, x, q, it, kind, i):
        assert self.slot[x][q] is None or not self.slot[x][q][3], "a tile in use was overwritten"
        need = {("mma", y) for y in self.users()}
        if self.codes:
            need |= {(y, w) for y in self.users() for w in range(4)}
        self.slot[x][q] = (it, kind, i, need)

    def conv(self, w):
        rc, rr, it = [0, 0], 0, 0
        while True:
            yield from self.take(it)
            tiles = self.item[it & 1]
            if tiles is None:
                return
            for i in range(2 * len(tiles)):
                x = 0 if self.wide else (i >> 1) & 1
                e, rc[x] = rc[x], rc[x] + 1
                q, r = e % self.R, rr % self.raw_n
                yield ("wait", self.raw_full[r], (rr // self.raw_n) & 1)
                if e >= self.R:
                    yield ("wait", self.empty[x][q], ((e - self.R) // self.R) & 1)
                assert self.raws[r] == (it, "KV"[i & 1], i >> 1)
                if self.slot[x][q] is None or self.slot[x][q][:3] != (it, "KV"[i & 1], i >> 1):  # the first to write
                    self.put(x, q, it, "KV"[i & 1], i >> 1)
                yield ("step",)
                self.full[x][q].arrive()
                self.raw_empty[r].arrive()
                rr += 1
            self.item_empty[it & 1].arrive()
            it += 1

    def look(self):
        n = 0
        while True:
            yield ("wait", self.v_landed[n & 1], (n >> 1) & 1)
            x, q, it, last = self.lk[n & 1]
            if it < 0:
                return
            if self.rng.random() < 0.5 and self.noted != it:
                if it >= 1:
                    yield ("wait", self.item_empty[(it - 1) & 1], ((it - 1) >> 1) & 1)
                self.noted = it
            yield ("step",)
            self.lk[n & 1] = None
            self.full[x][q].arrive()
            if last:
                self.v_seen[it & 1].arrive()
            self.look_free[n & 1].arrive()
            n += 1

    def use(self, x, e, it, kind, i):
        t = self.slot[self.ring_of(x)][e % self.R]
        assert t[:3] == (it, kind, i), "another tile stands in the ring"
        t[3].discard(("mma", x if self.wide else 0))

    def issue(self, x):
        rc, a, it = 0, 0, 0
        while True:
            yield from self.take(it)
            tiles = self.item[it & 1]
            if tiles is None:
                return
            nx, g = self.mine(len(tiles), x), self.ring_of(x)

            def issue_s(k):
                e, j = rc + 2 * k, (a + k) & 1
                yield ("wait", self.full[g][e % self.R], (e // self.R) & 1)

                def run(e=e, j=j, k=k, it=it):
                    self.use(x, e, it, "K", self.nth(k, x))
                    assert self.q[x if self.wide else 0] == it
                    old = self.s[x][j]
                    assert old is None or len(old[2]) == 4, "logits that a warp has not read were overwritten"
                    self.s[x][j] = [it, k, set(), set()]
                self.pipe[x] += [run, self.s_full[x][j].arrive, self.empty[g][e % self.R].arrive]
                yield ("step",)
            yield ("wait", self.q_full[x if self.wide else 0], it & 1)
            for k in range(min(2, nx)):
                yield from issue_s(k)
            for k in range(nx):
                e, j = rc + 2 * k + 1, (a + k) & 1
                yield ("wait", self.p_full[x][j], ((a + k) // 2) & 1)
                yield ("wait", self.full[g][e % self.R], (e // self.R) & 1)

                def run(e=e, j=j, k=k, it=it):
                    self.use(x, e, it, "V", self.nth(k, x))
                    assert self.s[x][j][:2] == [it, k] and len(self.s[x][j][3]) == 4, "weights of another round"
                    if k == 0 and self.o[x] is not None:
                        assert len(self.readers[x]) == (4 if self.wide else 8), "an output was overwritten"
                    if k == 0:
                        self.readers[x] = set()
                    self.o[x] = [it, k]
                self.pipe[x] += [run, self.pv_done[x][j].arrive, self.empty[g][e % self.R].arrive]
                if k + 2 < nx:
                    yield from issue_s(k + 2)
            rc, a = rc + 2 * nx, a + nx
            self.pipe[x].append(self.q_empty.arrive)
            self.item_empty[it & 1].arrive()
            yield ("step",)
            it += 1

    def soft(self, x, w):
        rc, a, it, nseen, g = 0, 0, 0, [0, 0], self.ring_of(x)
        while True:
            yield from self.take(it)
            tiles = self.item[it & 1]
            if tiles is None:
                return
            n = len(tiles)
            nx = self.mine(n, x)

            def give(e):
                if self.codes:
                    self.slot[g][e % self.R][3].discard((x if self.wide else 0, w))
                    self.empty[g][e % self.R].arrive()

            def scales(e, kind, k):
                yield ("wait", self.full[g][e % self.R], (e // self.R) & 1)
                assert self.slot[g][e % self.R][:3] == (it, kind, self.nth(k, x)), "scales of another tile"
            for k in range(nx):
                e, j = rc + 2 * k, (a + k) & 1
                yield ("wait", self.s_full[x][j], ((a + k) // 2) & 1)
                if self.codes:
                    yield from scales(e, "K", k)
                s = self.s[x][j]
                assert s[:2] == [it, k], "logits of another round"
                s[2].add(w)
                give(e)
                if self.codes:
                    yield from scales(e + 1, "V", k)
                give(e + 1)
                yield ("step",)
                if not self.wide and k == 0 and it > 0:
                    yield ("wait", self.merged, (it - 1) & 1)
                if k > 0 and self.rng.random() < 0.3:
                    b = a + k - 1
                    yield ("wait", self.pv_done[x][b & 1], (b // 2) & 1)
                    assert self.o[x] == [it, k - 1], "the output is scaled while it is added to"
                s[3].add(w)
                self.p_full[x][j].arrive()
                yield ("step",)
            if not self.codes and tiles[-1][0]:
                yield ("wait", self.v_seen[it & 1], nseen[it & 1] & 1)
                nseen[it & 1] += 1
                assert self.noted <= it, "notes of a later item"
            rc, a = rc + 2 * nx, a + nx
            if nx > 0:
                yield ("wait", self.pv_done[x][(a - 1) & 1], ((a - 1) // 2) & 1)
            if not self.wide:
                if nx == 0 and it > 0:
                    yield ("wait", self.merged, (it - 1) & 1)
                self.both_done.arrive()
                yield ("wait", self.both_done, it & 1)
            for y in [x] if self.wide else [0, 1]:
                if self.mine(n, y) > 0:
                    assert self.o[y] == [it, self.mine(n, y) - 1], "an output of another item"
                    self.readers[y].add((x, w))
            yield ("step",)
            if not self.wide:
                self.merged.arrive()
            self.item_empty[it & 1].arrive()
            it += 1

    def run(self, slow=()):
        at = {name: next(g) for name, g in self.roles.items()}
        while True:
            todo = [n for n, y in at.items() if y[0] == "step" or y[1].ready(y[2])]
            todo += [("pipe", x) for x in range(2) if self.pipe[x]] + [("load", i) for i in range(len(self.loads))]
            if not todo:
                return not at
            name = self.rng.choice([n for n in todo if n not in slow] or todo)
            if isinstance(name, tuple):
                (self.pipe[name[1]].pop(0) if name[0] == "pipe" else self.loads.pop(name[1]))()
                continue
            try:
                at[name] = next(self.roles[name])
            except StopIteration:
                del at[name]


def _items(rng, n):
    out = []
    for _ in range(n):
        m, drafts = rng.choice([1, 1, 2, 3, 5, 8]), rng.choice([0, 1, 2])  # 0: the run ends before the drafts
        out.append([(i >= m - drafts, rng.random() < 0.9) for i in range(m)])
    return out


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_every_wait_ends_whichever_role_is_late(wide, codes):
    names = list(Kernel([], wide, codes, random.Random(0)).roles)
    late = [()] + [(n,) for n in names] + [tuple(n for n in names if n.startswith(p)) for p in ("soft0", "soft1", "conv")]
    for slow in late:
        for seed in range(25):
            rng = random.Random(seed)
            assert Kernel(_items(rng, 6), wide, codes, rng).run(slow), f"{slow}, schedule {seed}: roles wait for good"
