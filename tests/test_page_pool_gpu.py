"""Page pools on the GPU: llm_pages_update and llm_pages_compact against plain loops over the
rules of include/llm.h.  Everything is whole numbers and copies: compared for equality."""
import numpy as np
import pytest
import torch

from test_batch_ops_gpu import lib  # noqa: F401

pytestmark = pytest.mark.gpu


class Pool:
    """Sequences with pages of their own, scattered, and some free ones; pages of two layers with bits of their own."""

    def __init__(self, lib, lens, page, n_pages, width, layers=2, kind="f16", seed=0):
        r = np.random.RandomState(seed)
        self.page, self.n_pages, self.lens = page, n_pages, np.array(lens, np.int32)
        self.table = np.full((len(lens), width), -1, np.int32)
        order, at = r.permutation(n_pages), 0
        for s, n in enumerate(lens):
            k = -(-n // page)
            self.table[s, :k] = order[at:at + k]
            at += k
        self.refs = np.zeros(n_pages, np.int32)
        self.refs[order[:at]] = 1
        shape = (n_pages, page, 2, 16) if kind == "f16" else (n_pages, 16 * 3)
        shape = ((layers,) if layers else ()) + shape
        self.k, self.v = (r.randint(0, 120, shape).astype(np.uint8 if kind == "q4" else np.int16) for _ in range(2))
        self.kind, self.layers = kind, layers
        self.upload(lib)

    def upload(self, lib):
        up = lambda x: torch.from_numpy(x.copy()).cuda()  # noqa: E731
        self.dev = {n: up(getattr(self, n)) for n in ("table", "lens", "refs", "k", "v")}
        k, v = (self.dev[n].view(torch.float16) if self.kind == "f16" else self.dev[n] for n in "kv")
        self.pool = lib.PagePool(k, v, self.dev["table"], self.dev["lens"], self.dev["refs"], page_size=self.page)

    def planes(self, t):
        return t if self.layers else t[None]

    def check(self):
        torch.cuda.synchronize()
        for n in ("lens", "refs", "table", "k", "v"):
            got, want = self.dev[n].cpu().numpy(), getattr(self, n)
            assert np.array_equal(got, want), (n, np.argwhere(got != want)[:4], got[got != want][:4], want[got != want][:4])

    def held(self, s):
        return -(-int(self.lens[s]) // self.page)

    def update(self, parents, rows):
        """The rules, sequence by sequence; returns the error bits (then nothing is changed)."""
        ps, n = self.page, len(self.lens)
        parents = np.arange(n) if parents is None else parents
        room = self.table.shape[1] * ps
        new, keeps, part = np.full_like(self.table, -1), [], []
        err = 0
        for s in range(n):
            had = int(self.lens[parents[s]]) if 0 <= parents[s] < n else 0
            now = had if rows is None else int(rows[s])
            err |= (16 if not -1 <= parents[s] < n else 0) | (2 if not 0 <= now <= room or not 0 <= self.lens[s] <= room else 0)
            keeps.append((min(had, now), now))
        if err:
            return err
        refs = self.refs.copy()
        for s in range(n):
            old = self.table[s, :self.held(s)]
            if ((old < 0) | (old >= self.n_pages)).any():
                return 1
            for j in old:
                refs[j] -= 1
        if (refs < 0).any():
            return 1
        for s, (keep, _) in enumerate(keeps):
            for i in range(keep // ps):
                new[s, i] = self.table[parents[s], i]
                refs[new[s, i]] += 1
        whole, copies = refs.copy(), []
        for s, (keep, _) in enumerate(keeps):
            part.append(-1)
            if keep % ps:
                j = self.table[parents[s], keep // ps]
                if whole[j] == 0 and refs[j] == 0:
                    new[s, keep // ps], refs[j] = j, 1
                else:
                    part[s] = j
        free = [j for j in range(self.n_pages) if refs[j] == 0]
        for s, (keep, now) in enumerate(keeps):
            first = keep // ps + (1 if keep % ps and part[s] < 0 else 0)
            for i in range(first, -(-now // ps)):
                if not free:
                    return 8
                new[s, i] = free.pop(0)
                refs[new[s, i]] = 1
            if part[s] >= 0:
                copies.append((part[s], new[s, keep // ps], keep % ps))
        before = [self.k.copy(), self.v.copy()]
        for src, dst, m in copies:
            for t, o in zip((self.k, self.v), before):
                m = m if self.kind == "f16" else t.shape[-1]
                self.planes(t)[:, dst, :m] = self.planes(o)[:, src, :m]
        for s in range(n):
            used, was = -(-keeps[s][1] // ps), self.held(s)
            self.table[s, :max(used, was)] = new[s, :max(used, was)]
        self.lens = np.array([now for _, now in keeps], np.int32)
        self.refs = refs
        return 0


def dev(x):
    return None if x is None else torch.from_numpy(np.array(x, np.int32)).cuda()


def run(lib, p, parents, rows, want=0):
    assert p.update(parents, rows) == want
    lib.PagesUpdate(p.pool, dev(parents), dev(rows))()
    p.check()
    assert p.pool.errors() == want


@pytest.mark.parametrize("kind,layers", [("f16", 2), ("f16", 0), ("q4", 3), ("q4", 0)])
@pytest.mark.parametrize("page", [1, 8, 16])
def test_update_steps(lib, page, kind, layers):  # noqa: F811
    """Many updates in a row: forks, orders, cuts, room for more, ends, new sequences."""
    p = Pool(lib, [5, 40, 0, 17, 16, 1, 33, 8], page, 8 * (96 // page) + 5, 96 // page, layers, kind)
    r = np.random.RandomState(page)
    for step in range(25):
        parents = np.arange(8)
        if step % 3 == 0:
            parents = r.randint(-1, 8, 8)
        elif step % 3 == 1:
            parents = r.permutation(8)
        had = np.where(parents < 0, 0, p.lens[parents])
        rows = np.clip(had + r.randint(-20, 21, 8), 0, 96 // page * page)
        run(lib, p, parents, None if step % 7 == 6 else rows)
    run(lib, p, None, None)
    run(lib, p, [-1] * 8, None)
    assert not p.refs.any() and not p.lens.any()


def test_update_keeps_what_others_hold(lib):  # noqa: F811
    """A page that one sequence cuts and another one keeps whole is copied, and so is one with a holder of the caller's."""
    p = Pool(lib, [32, 10], 16, 9, 4)
    run(lib, p, [0, 0], [32, 20])                     # the second keeps 4 rows of a page that the first keeps whole
    assert p.table[0, 1] != p.table[1, 1] and p.table[0, 0] == p.table[1, 0] and p.refs[p.table[0, 0]] == 2
    run(lib, p, [0, 1], [40, 21])
    j = p.table[1, 1]
    p.refs[j] += 1                                    # held by the caller
    p.dev["refs"][int(j)] += 1
    run(lib, p, None, [40, 22])
    assert p.table[1, 1] != j and p.refs[j] == 1
    run(lib, p, [1, 1], [22, 22])                     # the first in order keeps the page, whoever it was
    assert p.table[0, 1] != p.table[1, 1]
    run(lib, p, [-1, 0], [0, 22])
    assert p.refs[j] == 1 and p.refs.sum() == 3


def test_update_refusals_change_nothing(lib):  # noqa: F811
    p = Pool(lib, [20, 30, 5], 8, 10, 6)
    run(lib, p, None, [20, 30, 40], want=8)           # four pages more than the one that is free
    p.pool.err.zero_()
    run(lib, p, [0, 3, 1], None, want=16)
    p.pool.err.zero_()
    run(lib, p, [0, -2, 1], [20, -1, 30], want=18)
    p.pool.err.zero_()
    run(lib, p, None, [20, 30, 49], want=2)
    p.pool.err.zero_()
    run(lib, p, [2, 1, 0], [20, 30, 5])               # and still goes on
    run(lib, p, None, [2 ** 31 - 1, 30, 5], want=2)
    q = Pool(lib, [20, 30, 5], 8, 12, 6)
    q.table[1, 2] = 12
    q.dev["table"][1, 2] = 12
    run(lib, q, None, [20, 23, 5], want=1)            # also where the entry is given up
    q = Pool(lib, [20, 30, 5], 8, 12, 6)
    q.refs[q.table[0, 1]] = 0
    q.dev["refs"][int(q.table[0, 1])] = 0
    run(lib, q, [-1, 1, 2], None, want=1)             # fewer counted holders than there are


def test_update_wants_more_pages_than_32_bits(lib):  # noqa: F811
    """4096 sequences of 2^24 pages each: 2^36 pages, of which the lower 32 bits are zero."""
    lens, refs = torch.zeros(4096, dtype=torch.int32, device="cuda"), torch.zeros(100, dtype=torch.int32, device="cuda")
    s = lib.binding.llm_pool(n_seqs=4096, page_size=1, n_pages=100, max_pages=1 << 24, page_table=refs.data_ptr(), lens=lens.data_ptr(),
                             refs=refs.data_ptr())
    # (no table or workspace of that size is touched: the call stops before)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    s.err = err.data_ptr()
    rows = torch.full((4096,), 1 << 24, dtype=torch.int32, device="cuda")
    need = lib.binding._lib.llm_pages_update_workspace(lib.binding.ctypes.byref(s))
    assert need > 4096 << 24
    assert lib.binding._lib.llm_pages_update(lib.binding.ctypes.byref(s), None, rows.data_ptr(), ws.data_ptr(), need, None) == 0
    torch.cuda.synchronize()
    assert int(err) == lib.LLM_PAGES_FULL and not lens.any() and not refs.any()


@pytest.mark.parametrize("n_seqs,n_pages", [(1, 40), (300, 5000), (4096, 70000)])
def test_update_sizes(lib, n_seqs, n_pages):  # noqa: F811
    r = np.random.RandomState(n_seqs)
    p = Pool(lib, r.randint(0, 81, n_seqs), 8, n_pages, 12, layers=0)
    run(lib, p, r.randint(-1, n_seqs, n_seqs), r.randint(0, 97, n_seqs))
    run(lib, p, r.randint(0, n_seqs, n_seqs), None)
    run(lib, p, None, np.minimum(96, p.lens + 1))


def test_update_without_pages(lib):  # noqa: F811
    """Tables alone, and no pages or entries at all."""
    z = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, refs = z(3, 4) - 1, z(3), z(7)
    pool = lib.PagePool(None, None, table, lens, refs, page_size=4)
    lib.PagesUpdate(pool, rows=dev([5, 0, 9]))()
    assert table.tolist() == [[0, 1, -1, -1], [-1] * 4, [2, 3, 4, -1]] and refs.tolist() == [1] * 5 + [0, 0]
    lib.PagesUpdate(pool, parents=dev([2, 2, 2]), rows=dev([9, 8, 9]))()
    assert table.tolist() == [[2, 3, 4, -1], [2, 3, -1, -1], [2, 3, 0, -1]] and refs.tolist() == [1, 0, 3, 3, 1, 0, 0]
    assert lens.tolist() == [9, 8, 9] and pool.errors() == 0
    none = lib.PagePool(None, None, z(3, 0), z(3), z(0), page_size=4)
    lib.PagesUpdate(none, rows=dev([0, 0, 0]))()
    assert none.errors() == 0
    lib.PagesUpdate(none, rows=dev([0, 1, 0]))()
    assert none.errors() == lib.LLM_PAGES_BAD_LEN
    c = lib.PagesCompact(none)
    c()
    assert int(c.n_live) == 0
    lib.PagesUpdate(lib.PagePool(None, None, z(0, 3), z(0), z(2), page_size=4))()


# ------------------------------------------------------------- compaction --
def compacted(p):
    live = [j for j in range(p.n_pages) if p.refs[j] > 0]
    n = len(live)
    holes, movers = [j for j in range(n) if p.refs[j] <= 0], [j for j in live if j >= n]
    moved = np.full(p.n_pages, -1, np.int32)
    for j in live:
        moved[j] = j
    refs = np.where(np.arange(p.n_pages) < n, p.refs, 0).astype(np.int32)
    k, v = p.k.copy(), p.v.copy()
    for h, m in zip(holes, movers):
        moved[m], refs[h] = h, p.refs[m]
        for t in (k, v):
            p.planes(t)[:, h] = p.planes(t)[:, m]
    table = p.table.copy()
    for s in range(len(p.lens)):
        table[s, :p.held(s)] = moved[table[s, :p.held(s)]]
    return table, refs, moved, n, k, v


@pytest.mark.parametrize("kind,layers", [("f16", 2), ("q4", 0)])
@pytest.mark.parametrize("n_seqs,n_pages", [(1, 12), (3, 40), (60, 700), (500, 33000)])
def test_compact(lib, n_seqs, n_pages, kind, layers):  # noqa: F811
    r = np.random.RandomState(n_pages)
    p = Pool(lib, r.randint(0, 81, n_seqs), 8, n_pages, 11, layers, kind)
    run(lib, p, r.randint(0, n_seqs, n_seqs), None)               # some pages shared
    # apart, what was there is left as it was
    table, refs, moved, n, k, v = compacted(p)
    c = lib.PagesCompact(p.pool, table_out=torch.full_like(p.dev["table"], -9), refs_out=torch.empty_like(p.dev["refs"]))
    c()
    want = np.full_like(p.table, -9)
    for s in range(n_seqs):
        want[s, :p.held(s)] = table[s, :p.held(s)]
    assert np.array_equal(c.table_out.cpu().numpy(), want) and np.array_equal(c.refs_out.cpu().numpy(), refs)
    assert np.array_equal(c.moved.cpu().numpy(), moved) and int(c.n_live) == n
    p.k, p.v = k, v
    p.check()
    # in place (the data are where they belong already)
    c = lib.PagesCompact(p.pool)
    c()
    p.table, p.refs = table, refs
    p.check()
    assert np.array_equal(c.moved.cpu().numpy(), moved)
    c()                                                            # nothing is left to move
    p.check()
    assert int(c.n_live) == n and (p.refs[:n] > 0).all() and not p.refs[n:].any()
    run(lib, p, None, np.minimum(88, p.lens + 9))                  # and the pool goes on


@pytest.mark.parametrize("full", [True, False])
def test_compact_full_and_empty_pools(lib, full):  # noqa: F811
    p = Pool(lib, [64] * 8 if full else [0] * 8, 8, 64, 8)
    c = lib.PagesCompact(p.pool)
    c()
    p.check()
    assert int(c.n_live) == (64 if full else 0)


def test_compact_flags_bad_entries(lib):  # noqa: F811
    p = Pool(lib, [20, 30, 5], 8, 20, 6)
    p.dev["table"][0, 1] = 20
    c = lib.PagesCompact(p.pool)
    c()
    assert p.pool.errors() == lib.LLM_PAGES_BAD_PAGE and int(p.dev["table"][0, 1]) == 20
    p.pool.err.zero_()
    p.dev["table"][0, 1] = 0
    p.dev["table"][0, 3:] = 0
    p.dev["lens"][0] = 50                                          # behind the six pages
    c()
    assert p.pool.errors() & lib.LLM_PAGES_BAD_LEN


def test_pools_behind_32_bits(lib):  # noqa: F811
    """Copies between pages whose offsets pass 2^32 bytes, in several layers."""
    n_pages, one = 300000, 16 * 1024
    k, v = (torch.zeros(2, n_pages, one, dtype=torch.uint8, device="cuda") for _ in range(2))
    z = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, refs = z(2, 2), dev([9, 0]), z(n_pages)
    refs[:] = 1
    far = [n_pages - 1, n_pages - 3]
    table[0], refs[n_pages - 2] = dev(far), 0
    for t, x in ((k, 3), (v, 5)):
        t[0, far[1]], t[1, far[1]] = x, x + 1
    pool = lib.PagePool(k, v, table, lens, refs, page_size=8)
    lib.PagesUpdate(pool, parents=dev([0, 0]))()
    assert table.tolist() == [far, [far[0], n_pages - 2]] and refs[-4:].tolist() == [1, 1, 1, 2]
    assert [int(t[i, n_pages - 2].float().mean()) for t in (k, v) for i in (0, 1)] == [3, 4, 5, 6]
    refs[7] = 0
    k[:, n_pages - 1], v[:, n_pages - 1] = 9, 11
    c = lib.PagesCompact(pool)
    c()
    assert int(c.n_live) == n_pages - 1 and table.tolist() == [[7, far[1]], [7, n_pages - 2]]
    assert int(k[1, 7].float().mean()) == 9 and int(v[0, 7].float().mean()) == 11 and pool.errors() == 0


def test_pools_of_as_many_pages_as_31_bits_count(lib):  # noqa: F811
    """Tables alone over the largest pool: its last pages are counted, given out and moved as the others."""
    n = 2 ** 31 - 65
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough memory for the counts of 2^31 pages")
    z = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    refs, table, lens = torch.ones(n, dtype=torch.int32, device="cuda"), z(2, 4) - 1, z(2)
    refs[[5, 2 ** 30, n - 3, n - 1]] = 0
    pool = lib.PagePool(None, None, table, lens, refs, page_size=1)
    rows = dev([3, 1])
    op = lib.PagesUpdate(pool, None, rows)
    op()
    assert pool.errors() == 0 and table.tolist() == [[5, 2 ** 30, n - 3, -1], [n - 1, -1, -1, -1]] and lens.tolist() == [3, 1]
    assert int(refs.min()) == 1 and int(refs.max()) == 1
    rows[1] = 2
    op()                                                           # nothing is free
    assert pool.errors() == lib.LLM_PAGES_FULL and lens.tolist() == [3, 1] and int(refs.min()) == 1
    pool.err.zero_()
    rows[:] = dev([0, 1])
    op()
    assert pool.errors() == 0 and lens.tolist() == [0, 1] and (refs == 0).nonzero().flatten().tolist() == [5, 2 ** 30, n - 3]
    del op
    refs[n - 2], refs[n - 1] = 7, 9
    c = lib.PagesCompact(pool)
    c()
    assert pool.errors() == 0 and int(c.n_live) == n - 3 and table[1].tolist() == [2 ** 30, -1, -1, -1]
    assert [int(refs[j]) for j in (5, 2 ** 30, n - 4, n - 3, n - 2, n - 1)] == [7, 9, 1, 0, 0, 0]
    assert [int(c.moved[j]) for j in (0, 5, 2 ** 30, n - 4, n - 3, n - 2, n - 1)] == [0, -1, -1, n - 4, -1, 5, 2 ** 30]


def test_sequences_of_as_many_pages_as_31_bits_count(lib):  # noqa: F811
    """The last entries of a table of 2^31 - 2 pages of one row are given up and taken again (the others all name
    page 0)."""
    n = 2 ** 31 - 2
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("not enough memory for a table of 2^31 entries")
    table, refs = torch.zeros(1, n, dtype=torch.int32, device="cuda"), torch.zeros(20, dtype=torch.int32, device="cuda")
    refs[0], lens, rows = n, dev([n]), dev([n - 8])
    pool = lib.PagePool(None, None, table, lens, refs, page_size=1)
    op = lib.PagesUpdate(pool, None, rows)
    op()
    assert pool.errors() == 0 and lens.tolist() == [n - 8] and refs.tolist() == [n - 8] + [0] * 19
    assert table[0, -12:].tolist() == [0] * 4 + [-1] * 8 and not table[0, :-8].any()
    rows[0] = n - 1
    op()
    assert pool.errors() == 0 and lens.tolist() == [n - 1] and refs.tolist() == [n - 8] + [1] * 7 + [0] * 12
    assert table[0, -12:].tolist() == [0] * 4 + [1, 2, 3, 4, 5, 6, 7, -1] and not table[0, :-8].any()


def test_update_wants_as_many_pages_as_32_bits_count(lib):  # noqa: F811
    """4096 sequences of as many pages as the pool has, 2^32 together.  The table, the workspace and what a place of
    32 bits could reach around the workspace are there: a sum cut to 32 bits would go on, within these."""
    n = 1 << 20
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("not enough memory for a table of 2^32 entries")
    refs, lens = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (n, 4096))
    table = torch.full((4096, n), -1, dtype=torch.int32, device="cuda")
    pool = lib.PagePool(None, None, table, lens, refs, page_size=1)
    rows = torch.full((4096,), n, dtype=torch.int32, device="cuda")
    need = lib.binding._lib.llm_pages_update_workspace(lib.binding.ctypes.byref(pool.struct))
    before, behind = 9 << 30, 2 << 30
    ws = torch.empty(before + need + behind, dtype=torch.uint8, device="cuda")
    assert ws.data_ptr() % 256 == 0 and need > table.numel() * 4
    torch.cuda.synchronize()
    call = lambda: lib.binding._lib.llm_pages_update(lib.binding.ctypes.byref(pool.struct), None, rows.data_ptr(), ws.data_ptr() + before, need, None)  # noqa: E731
    assert call() == 0
    torch.cuda.synchronize()
    assert pool.errors() == lib.LLM_PAGES_FULL and not lens.any() and not refs.any() and int(table.max()) == -1
    pool.err.zero_()
    rows[1:] = 0
    torch.cuda.synchronize()
    assert call() == 0                                              # all of them for the first
    torch.cuda.synchronize()
    assert pool.errors() == 0 and torch.equal(table[0], torch.arange(n, dtype=torch.int32, device="cuda")) and int(table[1:].max()) == -1
    assert int(lens[0]) == n and not lens[1:].any() and int(refs.min()) == 1 and int(refs.max()) == 1


# A plan runs as a cluster of blocks where n_seqs > 1024, n_pages > 16384 or there are more than 65536 entries.
@pytest.mark.parametrize("n_seqs,n_pages", [(4096, 70000), (40, 70000)])
def test_update_refusals_of_large_pools_change_nothing(lib, n_seqs, n_pages):  # noqa: F811
    """The refusals of test_update_refusals_change_nothing where another block than the first finds the reason."""
    p = Pool(lib, np.random.RandomState(n_seqs).randint(9, 81, n_seqs), 8, n_pages, 12, layers=0)
    last, mid, held = n_seqs - 1, n_seqs // 2, p.lens.copy()

    def refused(want, parents=None, rows=None):
        run(lib, p, parents, rows, want=want)                      # (compares the whole state with what it was)
        p.pool.err.zero_()

    def with_one(x, at, v):
        y = np.array(x, np.int32)
        y[at] = v
        return y

    order = np.arange(n_seqs)
    for at in (last, mid):
        refused(16, with_one(order, at, n_seqs))
        refused(16, with_one(order, at, -2), held)
        refused(2, None, with_one(held, at, 97))
        refused(2, None, with_one(held, at, -1))
        refused(18, with_one(order, 0, n_seqs), with_one(held, at, -1))
    # more pages than the five that the caller has left free
    kept = np.flatnonzero(p.refs == 0)[:-5]
    p.refs[kept], p.dev["refs"][torch.from_numpy(kept).cuda()] = 1, 1
    for at in (last, mid):
        refused(8, None, with_one(held, np.arange(at - 2, at + 1), 96))
    run(lib, p, None, with_one(held, last, held[last] // 8 * 8 + 9))
    held = p.lens.copy()
    p.refs[kept], p.dev["refs"][torch.from_numpy(kept).cuda()] = 0, 0
    # entries that name no page: given up, taken over whole and in part
    for at in (last, mid):
        for bad in (n_pages, -5):
            good = int(p.table[at, 0])
            p.table[at, 0] = bad
            p.dev["table"][at, 0] = bad
            refused(1, None, with_one(held, at, 0))
            refused(1, with_one(order, 0, at), None)
            p.table[at, 0] = good
            p.dev["table"][at, 0] = good
        i = (int(held[at]) - 1) // 8
        if held[at] % 8:
            good = int(p.table[at, i])
            p.table[at, i] = n_pages + 3
            p.dev["table"][at, i] = n_pages + 3
            refused(1, with_one(order, 0, at), None)
            p.table[at, i] = good
            p.dev["table"][at, i] = good
    # fewer counted holders than there are, of the highest page that is given up
    at = int(max(range(n_seqs), key=lambda s: p.table[s, 0]))
    j = int(p.table[at, 0])
    p.refs[j], p.dev["refs"][j] = 0, 0
    refused(1, None, with_one(held, at, 0))
    p.refs[j], p.dev["refs"][j] = 1, 1
    run(lib, p, order[::-1].copy(), None)                          # and it goes on
    run(lib, p, None, np.minimum(96, p.lens + 3))


@pytest.mark.parametrize("n_seqs,n_pages,width", [(1024, 5000, 12), (1025, 5000, 12), (30, 16384, 12), (30, 16385, 12), (512, 4000, 128), (512, 4000, 129)])
def test_updates_and_copies_around_the_largest_plan_of_one_block(lib, n_seqs, n_pages, width):  # noqa: F811
    """Both plans, with pages: copies from and to every block's share."""
    r = np.random.RandomState(n_pages + n_seqs + width)
    p = Pool(lib, r.randint(0, min(25, n_pages * 4 // n_seqs), n_seqs), 8, n_pages, width, layers=1)
    for parents in (r.randint(-1, n_seqs, n_seqs), r.randint(0, n_seqs, n_seqs), np.arange(n_seqs)):
        had = np.where(parents < 0, 0, p.lens[parents])
        run(lib, p, parents, np.clip(had + r.randint(-8, 4, n_seqs), 0, 24))
    assert (p.refs > 1).any() or n_seqs < 100
    c = lib.PagesCompact(p.pool)
    table, refs, moved, n, p.k, p.v = compacted(p)
    c()
    p.table, p.refs = table, refs
    p.check()
    assert np.array_equal(c.moved.cpu().numpy(), moved) and int(c.n_live) == n
