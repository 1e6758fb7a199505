"""Pages of a cache on the GPU against a model of their rules in plain Python: whole numbers, so equal in every bit."""
import random

import pytest
import torch

import quant_packed_gemv_gb300 as q

pytestmark = pytest.mark.gpu


class Model:
    """The rules, on host lists."""

    def __init__(self, pages, seqs, width, ps):
        self.table, self.lens, self.refs = [[-1] * width for _ in range(seqs)], [0] * seqs, [0] * pages
        self.data, self.ps, self.status = list(range(pages)), ps, 0   # data: a tag per page

    def fresh(self, n):
        return [p for p, r in enumerate(self.refs) if r == 0][:n]

    def reserve(self, seqs, add, most):
        ps, need = self.ps, []
        for s, a in zip(seqs, add):
            ok = 0 <= s < len(self.lens) and 0 <= a <= most and -(-(self.lens[s] + a) // ps) <= len(self.table[0])
            need.append(-(-(self.lens[s] + a) // ps) - -(-self.lens[s] // ps) if ok else None)
            self.status |= 0 if ok else q.PLM_KV_BAD_ITEM
        pages = self.fresh(sum(n or 0 for n in need))
        slots = [[-1] * most for _ in seqs]
        if len(pages) < sum(n or 0 for n in need):
            self.status |= q.PLM_KV_OUT_OF_PAGES
            return slots
        for i, (s, a) in enumerate(zip(seqs, add)):
            if need[i] is None:
                continue
            have = -(-self.lens[s] // ps)
            for k in range(need[i]):
                self.table[s][have + k] = pages.pop(0)
                self.refs[self.table[s][have + k]] = 1
            for j in range(a):
                pos = self.lens[s] + j
                slots[i][j] = self.table[s][pos // ps] * ps + pos % ps
            self.lens[s] += a
        return slots

    def fork(self, parents, children, keep=None):
        ps, items = self.ps, []
        for i, (p, c) in enumerate(zip(parents, children)):
            ok = 0 <= p < len(self.lens) and 0 <= c < len(self.lens) and p != c and self.lens[c] == 0 and (keep is None or keep[i] >= 0)
            self.status |= 0 if ok else q.PLM_KV_BAD_ITEM
            items.append((p, c, min(self.lens[p], keep[i]) if keep is not None else self.lens[p]) if ok else None)
        want = sum(1 for it in items if it and it[2] % ps)
        pages = self.fresh(want)
        if len(pages) < want:
            self.status |= q.PLM_KV_OUT_OF_PAGES
            return
        for it in items:
            if it is None:
                continue
            p, c, n = it
            full = n // ps
            self.table[c] = self.table[p][:full] + [-1] * (len(self.table[p]) - full)
            for x in self.table[c][:full]:
                self.refs[x] += 1
            if n % ps:
                new = pages.pop(0)
                self.table[c][full], self.refs[new], self.data[new] = new, 1, self.data[self.table[p][full]]
            self.lens[c] = n

    def free(self, seqs):
        for s in seqs:
            if not 0 <= s < len(self.lens):
                self.status |= q.PLM_KV_BAD_ITEM
                continue
            for p in self.table[s]:
                if p >= 0:
                    self.refs[p] -= 1
            self.table[s], self.lens[s] = [-1] * len(self.table[s]), 0

    def compact(self):
        used = [p for p, r in enumerate(self.refs) if r]
        live = len(used)
        holes = [p for p in range(live) if not self.refs[p]]
        move = {p: h for p, h in zip([p for p in used if p >= live], holes)}
        for p, h in move.items():
            self.refs[h], self.refs[p], self.data[h] = self.refs[p], 0, self.data[p]
        self.table = [[move.get(p, p) for p in row] for row in self.table]
        return live


class Gpu:
    def __init__(self, m, words):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.words = words
        self.base = torch.randint(-2 ** 31, 2 ** 31 - 1, (len(m.refs), words), **i32)
        self.pool = self.base.clone()
        self.table, self.lens, self.refs = (torch.tensor(v, **i32) for v in (m.table, m.lens, m.refs))
        self.status = torch.zeros(1, **i32)
        self.kv = q.plm_kv_state(self.pool, self.table, self.lens, self.refs, m.ps, self.status)
        self.ws = torch.empty(q.plm_kv_workspace_size(len(m.refs), 4096), dtype=torch.uint8, device="cuda")

    def same(self, m):
        assert self.table.tolist() == m.table and self.lens.tolist() == m.lens and self.refs.tolist() == m.refs
        assert int(self.status) == m.status
        assert torch.equal(self.pool, self.base[torch.tensor(m.data, device="cuda")])


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("pages,seqs,width,ps,words", [(40, 6, 12, 4, 4), (300, 40, 20, 16, 1028), (5000, 200, 33, 16, 8),
                                                       (9001, 64, 200, 7, 4), (64, 5, 9, 1, 3000)])
@pytest.mark.parametrize("seed", range(3))
def test_random_histories(pages, seqs, width, ps, words, seed):
    r = random.Random(seed)
    m = Model(pages, seqs, width, ps)
    g = Gpu(m, words)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(24):
        op = r.choice(("reserve", "reserve", "fork", "free", "compact"))
        used, unused = [s for s in range(seqs) if m.lens[s]], [s for s in range(seqs) if not m.lens[s]]
        if op == "reserve":
            most = r.choice((1, 3, 4 * ps))
            items = r.sample(range(seqs), r.randrange(1, seqs + 1))
            add = [r.randrange(0, most + 1) for _ in items]
            if step % 5 == 4:   # an item that cannot be done
                items[0], add[-1] = r.choice((-1, seqs, 10 ** 9)), r.choice((-3, most + 1))
            slots = torch.full((len(items), most), 77, dtype=torch.int64, device="cuda")
            q.plm_kv_reserve(g.kv, ints(items), ints(add), slots, g.ws)
            assert slots.tolist() == m.reserve(items, add, most)
        elif op == "fork" and used and unused:
            n = r.randrange(1, min(len(unused), 30) + 1)
            parents, children = [r.choice(used) for _ in range(n)], r.sample(unused, n)
            keep = None if r.random() < 0.5 else [r.randrange(0, m.lens[p] + 5) for p in parents]
            if step % 4 == 3:
                children[0] = r.choice([-1, seqs, used[0]])
            q.plm_kv_fork(g.kv, ints(parents), ints(children), g.ws, keep=None if keep is None else ints(keep))
            m.fork(parents, children, keep)
        elif op == "free":
            items = r.sample(range(seqs), r.randrange(1, seqs // 2 + 1)) + ([seqs + 1] if step % 3 == 0 else [])
            q.plm_kv_free(g.kv, ints(items))
            m.free(items)
        else:
            q.plm_kv_compact(g.kv, live, g.ws)
            assert int(live) == m.compact()
        g.same(m)


def test_out_of_pages_changes_nothing():
    m = Model(10, 4, 8, 4)
    g = Gpu(m, 4)
    slots = torch.empty(3, 20, dtype=torch.int64, device="cuda")
    for items, add in (([0, 1], [14, 13]), ([2, 0, 3], [1, 18, 9]), ([2, 3], [4, 4])):   # 8 pages; 7 more: too many; 2
        q.plm_kv_reserve(g.kv, ints(items), ints(add), slots[:len(items)], g.ws)
        assert slots[:len(items)].tolist() == m.reserve(items, add, 20)
        g.same(m)
    assert m.status == q.PLM_KV_OUT_OF_PAGES and m.lens == [14, 13, 4, 4]


@pytest.mark.parametrize("n", [1024, 2048])
def test_wishes_that_pass_32_bits_together_change_nothing(n):
    # 2^21 pages for each of n sequences: 2^31 of them for 1024, 2^32 for 2048, and the pool has 64
    width, pages = 1 << 21, 64
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens, refs, status = torch.empty(n, width, **i32), torch.zeros(n, **i32), torch.zeros(pages, **i32), torch.zeros(1, **i32)
    kv = q.plm_kv_state(torch.zeros(pages, 4, **i32), table, lens, refs, 1, status)
    ws, table[:, 0] = torch.empty(q.plm_kv_workspace_size(pages, n), dtype=torch.uint8, device="cuda"), -1
    q.plm_kv_reserve(kv, torch.arange(n, **i32), torch.full((n,), width, **i32), None, ws)
    assert int(status) == q.PLM_KV_OUT_OF_PAGES
    assert not lens.any() and not refs.any() and bool((table[:, 0] == -1).all())


def test_tokens_are_taken_back_by_fork_and_free():
    # drafts that were not accepted: whole pages past the kept tokens become free, the page they end in is copied
    m = Model(40, 8, 10, 4)
    g = Gpu(m, 8)
    steps = [("reserve", [0, 1, 2], [9, 16, 6]), ("reserve", [0, 1, 2], [7, 7, 7])]
    for _, seqs, add in steps:
        q.plm_kv_reserve(g.kv, ints(seqs), ints(add), None, g.ws)
        m.reserve(seqs, add, 99)
    used = sum(r > 0 for r in m.refs)
    old, new, keep = [0, 1, 2], [5, 6, 7], [10, 16, 13]   # 1, 0 and all of the 7 drafts stay
    q.plm_kv_fork(g.kv, ints(old), ints(new), g.ws, keep=ints(keep))
    q.plm_kv_free(g.kv, ints(old))
    m.fork(old, new, keep)
    m.free(old)
    g.same(m)
    assert m.status == 0 and m.lens == [0, 0, 0, 0, 0, 10, 16, 13]
    assert sum(r > 0 for r in m.refs) == 3 + 4 + 4 < used and sum(m.refs) == 3 + 4 + 4


def test_fork_without_room_changes_nothing():
    m = Model(9, 4, 8, 4)
    g = Gpu(m, 4)
    m.reserve([0, 1], [14, 13], 20)
    q.plm_kv_reserve(g.kv, ints([0, 1]), ints([14, 13]), None, g.ws)
    q.plm_kv_fork(g.kv, ints([0, 1]), ints([2, 3]), g.ws)   # two partial pages, one free
    m.fork([0, 1], [2, 3])
    assert m.status == q.PLM_KV_OUT_OF_PAGES
    g.same(m)
    q.plm_kv_fork(g.kv, ints([0, 1]), ints([2, 3]), g.ws, keep=ints([8, 3]))
    m.fork([0, 1], [2, 3], [8, 3])
    g.same(m)


def test_many_items_and_a_sequence_listed_twice_in_free():
    n, ps = 4096, 16
    m = Model(n * 3, n, 4, ps)
    g = Gpu(m, 4)
    r = random.Random(5)
    items, add = r.sample(range(n), n), [r.randrange(0, 41) for _ in range(n)]
    slots = torch.empty(n, 40, dtype=torch.int64, device="cuda")
    q.plm_kv_reserve(g.kv, ints(items), ints(add), slots, g.ws)     # the form with a launch of its own for the items
    assert slots.tolist() == m.reserve(items, add, 40)
    g.same(m)
    q.plm_kv_free(g.kv, ints([7, 8, 7, 7]))
    m.free([7, 8])
    g.same(m)


@pytest.mark.parametrize("n,form", [(2, "one launch"), (40, "one launch"), (40, "two launches")])
def test_a_sequence_listed_twice_in_reserve_stays_inside_its_row(n, form):
    # its state is then undefined, but nothing else: each item alone fills the last row, and what lies behind the
    # table, the other rows and the counts of pages that were in use stay as they are
    seqs, width, ps, pages = 3, 4, 16, 400
    i32 = dict(dtype=torch.int32, device="cuda")
    behind = torch.full((seqs * width + 4096,), 77, **i32)
    table = behind[:seqs * width].view(seqs, width)
    table[:] = -1
    lens, refs = torch.zeros(seqs, **i32), torch.zeros(pages, **i32)
    table[0, 0], lens[0], refs[0] = 0, 5, 1
    kv, ws = q.plm_kv_state(torch.zeros(pages, 4, **i32), table, lens, refs, ps), torch.empty(q.plm_kv_workspace_size(pages, n), dtype=torch.uint8, device="cuda")
    slots = torch.empty(n, 64 if form == "one launch" else 4096, dtype=torch.int64, device="cuda")
    q.plm_kv_reserve(kv, ints([seqs - 1] * n), ints([64] * n), slots, ws)
    assert bool((behind[seqs * width:] == 77).all())
    assert table[:2].tolist() == [[0, -1, -1, -1], [-1] * 4] and lens.tolist() == [5, 0, 64]
    row = table[2].tolist()
    assert all(1 <= p <= 4 * n for p in row) and refs[:4 * n + 1].tolist() == [1] * (4 * n + 1)
    got = slots[:, :64]     # every item's slots lie in pages that it was given, or that a later one put in the row
    assert bool(((got >= ps) & (got < (4 * n + 1) * ps)).all()) and bool((slots[:, 64:] == -1).all())


def test_calls_without_items():
    m = Model(20, 4, 8, 4)
    g = Gpu(m, 4)
    none = ints([])
    m.reserve([1], [9], 9)
    q.plm_kv_reserve(g.kv, ints([1]), ints([9]), None, g.ws)
    q.plm_kv_reserve(g.kv, none, none, None, g.ws)
    q.plm_kv_reserve(g.kv, none, none, torch.empty(0, 3, dtype=torch.int64, device="cuda"), g.ws)
    q.plm_kv_fork(g.kv, none, none, g.ws)
    q.plm_kv_fork(g.kv, none, none, g.ws, keep=none)
    q.plm_kv_free(g.kv, none)
    q.plm_kv_copy_pages(g.kv, none, none)
    g.same(m)


def test_copy_pages():
    for words in (4, 1024, 1028, 70000):
        pool = torch.randint(-9, 9, (50, words), dtype=torch.int32, device="cuda")
        meta = torch.zeros(50, dtype=torch.int32, device="cuda")
        kv = q.plm_kv_state(pool, meta.view(50, 1), meta, meta, 16)
        want = pool.clone()
        src, dst = [3, 3, 49, -1, 5, 60, 7], [10, 11, 0, 12, 50, 13, 14]
        for a, b in zip(src, dst):
            if 0 <= a < 50 and 0 <= b < 50:
                want[b] = want[a]
        q.plm_kv_copy_pages(kv, ints(src), ints(dst))
        assert torch.equal(pool, want)


def test_pool_past_32_bits():
    words, pages = 1 << 20, 1300    # 5.4 GB
    pool = torch.empty(pages, words, dtype=torch.int32, device="cuda")
    pool[1299], pool[1200] = 7, 8
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens, refs = torch.tensor([[1299, 1200], [-1, -1]], **i32), torch.tensor([20, 0], **i32), torch.zeros(pages, **i32)
    refs[1299] = refs[1200] = 1
    kv, live = q.plm_kv_state(pool, table, lens, refs, 16), torch.zeros(1, **i32)
    ws = torch.empty(q.plm_kv_workspace_size(pages, 1), dtype=torch.uint8, device="cuda")
    q.plm_kv_fork(kv, ints([0]), ints([1]), ws)
    assert table.tolist() == [[1299, 1200], [1299, 0]] and bool((pool[0] == 8).all())
    q.plm_kv_compact(kv, live, ws)
    assert int(live) == 3 and table.tolist() == [[2, 1], [2, 0]] and refs[:3].tolist() == [1, 1, 2] and int(refs.sum()) == 4
    assert bool((pool[2] == 7).all()) and bool((pool[1] == 8).all())


def test_binding_refuses():
    i32 = dict(dtype=torch.int32, device="cuda")
    pool, table, lens, refs = torch.zeros(8, 16, **i32), torch.zeros(2, 4, **i32), torch.zeros(2, **i32), torch.zeros(8, **i32)
    kv, ws = q.plm_kv_state(pool, table, lens, refs, 16), torch.empty(4096, dtype=torch.uint8, device="cuda")
    for bad in (lambda: q.plm_kv_state(pool, table.long(), lens, refs, 16), lambda: q.plm_kv_state(pool, table, lens[:1], refs, 16),
                lambda: q.plm_kv_state(pool, table, lens, refs[:5], 16), lambda: q.plm_kv_state(pool[:, :3], table, lens, refs, 16),
                lambda: q.plm_kv_reserve(kv, lens.long(), lens, None, ws), lambda: q.plm_kv_reserve(kv, lens, lens[:1], None, ws),
                lambda: q.plm_kv_fork(kv, lens, lens[:1], ws), lambda: q.plm_kv_copy_pages(kv, lens, lens[:1])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(q.PlmError):
        q.plm_kv_compact(kv, None, ws[:256])
