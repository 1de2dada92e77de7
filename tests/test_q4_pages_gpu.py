"""Pages of 4-bit values on the GPU: the append against the format's rules, element by
element, the read back, and attention against its formula in 64 bits on the values that
the pages stand for.

Tolerances: attention's is test_batch_ops_gpu.attend_bound (the products are those of F16
pages).  The append's numbers follow from F32 operations that numpy rounds alike, so they are
compared bit for bit; the bound of what 4 bits lose is written beside its test."""
import math

import numpy as np
import pytest
import torch

from test_batch_ops_gpu import F16, F32, H16, H32, TYPES, check_attend, lib, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def page_bytes(page, n_kv, hd):
    return -(-page * n_kv * (hd // 2 + 4 * -(-hd // 32)) // 16) * 16


def values(n, d, m):
    """The F16 nearest to d n + m: the product and the sum are exact in 64 bits (11 + 4 bits, and FP16's
    whole range spans 40 bits), and numpy rounds them once."""
    hd = n.shape[-1]
    d, m = (np.repeat(t.astype(np.float64), 32, -1)[..., :hd] for t in (d, m))
    with np.errstate(all="ignore"):
        return (d * n + m).astype(np.float16)


def decode(pages, page, n_kv, hd):
    """Numbers [n_pages, page, n_kv, hd] and pairs [n_pages, page, n_kv, groups] of uint8 pages."""
    t, g, a = pages.cpu().numpy(), -(-hd // 32), page * n_kv * hd // 2
    b = t[:, :a].reshape(-1, n_kv, page, hd // 2)
    n = np.stack([b & 15, b >> 4], -1).reshape(-1, n_kv, page, hd).transpose(0, 2, 1, 3)
    s = np.ascontiguousarray(t[:, a:a + page * n_kv * g * 4]).view(np.float16).reshape(-1, n_kv, page, g, 2).transpose(0, 2, 1, 3, 4)
    return n, s[..., 0], s[..., 1]


class BatchQ4:
    """A batch over 4-bit pages; unused pages and rows behind each sequence's last one hold NaN pairs.
    k, v: the values that the pages stand for, as test_batch_ops_gpu.check_attend takes them."""

    def __init__(self, lib, lens, n_new, prefix, page, n_kv, hd, seed=0, extra=3):
        self.lens, self.n_new, self.prefix, self.page, self.n_kv, self.hd = lens, n_new, prefix, page, n_kv, hd
        need = [-(-max(n, 0) // page) for n in lens]
        self.n_pages, width = sum(need) + extra, max(need + [1])
        r = np.random.RandomState(seed)
        order = r.permutation(self.n_pages)
        table, at = np.full((len(lens), width), -7, np.int32), 0
        live = np.zeros((self.n_pages, page), bool)
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n]
            at += n
            for e in range(max(lens[s], 0)):
                live[table[s, e // page], e % page] = True
        self.table = torch.from_numpy(table).cuda()
        a, g = page * n_kv * hd // 2, -(-hd // 32)
        self.bytes = []
        for _ in range(2):
            t = r.randint(0, 256, (self.n_pages, page_bytes(page, n_kv, hd))).astype(np.uint8)
            d = np.abs(r.randn(self.n_pages, n_kv, page, g)) * 0.2
            s = np.stack([d, -7.5 * d + 0.3 * r.randn(*d.shape)], -1).astype(np.float16)
            s.transpose(0, 2, 1, 3, 4)[~live] = np.nan
            t[:, a:a + page * n_kv * g * 4] = s.reshape(self.n_pages, -1).view(np.uint8)
            self.bytes.append(torch.from_numpy(t).cuda())
        self.lens_dev = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.pages = lib.PagedBatchQ4(*self.bytes, self.table, self.lens_dev, page, n_kv, hd, n_new=n_new, prefix_len=prefix)
        self.read()

    def read(self):
        self.k, self.v = (torch.from_numpy(values(*decode(t, self.page, self.n_kv, self.hd))).cuda() for t in self.bytes)

    def rows(self):
        for s, n in enumerate(self.lens):
            for i in range(self.n_new):
                if n - self.n_new + i >= 0:
                    yield s * self.n_new + i, s, n - self.n_new + i

    def slot(self, s, e):
        return int(self.table[s, e // self.page]), e % self.page

    def gather(self, t, s, n):
        if n == 0:
            return t.new_zeros(0, *t.shape[2:]).double()
        return t[self.table[s, :-(-n // self.page)].long()].flatten(0, 1)[:n].double()


# ------------------------------------------------------------------ append --
def rotated32(x, cs, neox):
    """RoPE of heads [heads, hd] with every product and sum rounded to F32, as llm_kv_append rotates."""
    y, half = x.copy(), cs.shape[0]
    a = np.arange(half) if neox else 2 * np.arange(half)
    b = a + half if neox else a + 1
    c, s = cs[:, 0], cs[:, 1]
    y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, a] * s + x[:, b] * c
    return y


def quantized(x):
    """The format's rules in F32 for heads [heads, hd]."""
    g = -(-x.shape[1] // 32)
    n, d, m = np.zeros(x.shape, np.uint8), np.zeros((len(x), g), np.float16), np.zeros((len(x), g), np.float16)
    with np.errstate(all="ignore"):
        for h in range(len(x)):
            for i in range(g):
                t = x[h, 32 * i:32 * i + 32]
                low, high = t.min(), t.max()
                dd, mm = ((high - low) / np.float32(15)).astype(np.float16), low.astype(np.float16)
                if not np.isfinite(t).all() or not np.isfinite(dd) or not np.isfinite(mm):
                    dd = mm = np.float16(np.nan)
                elif dd > 0:
                    n[h, 32 * i:32 * i + 32] = np.clip(np.rint((t - mm.astype(np.float32)) / dd.astype(np.float32)), 0, 15)
                d[h, i], m[h, i] = dd, mm
    return n, d, m


def same(a, b):
    return np.array_equal(a, b, equal_nan=a.dtype.kind == "f")


def check_append(b, before, q, k, v, q_out, cs, neox):
    cs = cs.cpu().numpy()
    want = [decode(t, b.page, b.n_kv, b.hd) for t in before]
    want = [[np.array(y) for y in w] for w in want]
    half = cs.shape[1]
    for row, s, e in b.rows():
        p, r = b.slot(s, e)
        for w, x, turn in ((want[0], k, True), (want[1], v, False)):
            x = x[row].float().cpu().numpy()
            for y, z in zip(w, quantized(rotated32(x, cs[b.prefix + e], neox) if turn and half else x)):
                y[p, r] = z
        if q is not None:
            x = rotated32(q[row].float().cpu().numpy(), cs[b.prefix + e], neox) if half else q[row].float().cpu().numpy()
            assert same(q_out[row].cpu().numpy(), x.astype(np.float16 if q_out.dtype == F16 else np.float32))
    for t, w, old in zip(b.bytes, want, before):
        assert all(same(x, y) for x, y in zip(decode(t, b.page, b.n_kv, b.hd), w))
        used = b.page * b.n_kv * (b.hd // 2 + 4 * -(-b.hd // 32))
        assert torch.equal(t[:, used:], old[:, used:])             # bytes behind a page's last pair


HEADS = [((8, 2, 32), 32, False), ((6, 6, 48), 48, True), ((4, 2, 64), 64, True), ((4, 2, 64), 64, False), ((4, 2, 64), 20, False), ((4, 2, 64), 20, True),
         ((3, 3, 128), 128, False), ((3, 1, 128), 96, True), ((2, 1, 16), 8, True), ((2, 3, 16), 16, False), ((0, 2, 64), 64, False),
         ((4, 2, 64), 0, True), ((4, 1, 80), 80, True), ((2, 1, 96), 96, False), ((2, 1, 112), 10, True)]


@pytest.mark.parametrize("heads,rope,neox", HEADS)
@pytest.mark.parametrize("dtype,out", TYPES)
def test_append(lib, heads, rope, neox, dtype, out):  # noqa: F811
    n_heads, n_kv, hd = heads
    b = BatchQ4(lib, [1, 17, 40, 0, 3, 64], 3, 21, 16, n_kv, hd)          # padding rows in sequences 0 and 3
    n = 6 * 3
    qkv = rand(5, n, n_heads + 2 * n_kv, hd, dtype=dtype)
    q, k, v = qkv[:, :n_heads], qkv[:, n_heads:n_heads + n_kv], qkv[:, n_heads + n_kv:]
    q = q if n_heads else None
    cs = rand(6, 21 + 64, rope // 2, 2)
    q_out = torch.full((n, n_heads, hd), 7.0, dtype=out, device="cuda")
    before = [t.clone() for t in b.bytes]
    lib.KvAppend(b.pages, q, k, v, cs, q_out=q_out, rope_neox=neox)()
    check_append(b, before, q, k, v, q_out, cs, neox)
    live = {r for r, _, _ in b.rows()}
    assert all((q_out[r] == 7.0).all() for r in range(n) if r not in live)
    # the rows read back are the values that the pages stand for, and the others stay
    b.read()
    for t in (F32, F16):
        wide = torch.full((n, 2 * n_kv + 1, hd), 9.0, dtype=t, device="cuda")
        ko, vo = wide[:, :n_kv], wide[:, n_kv + 1:]
        lib.KvRead(b.pages, ko, vo)()
        for row, s, e in b.rows():
            p, r = b.slot(s, e)
            assert torch.equal(ko[row], b.k[p, r].to(t)) and torch.equal(vo[row], b.v[p, r].to(t))
        assert (wide[:, n_kv] == 9.0).all() and all((wide[r] == 9.0).all() for r in range(n) if r not in live)
    assert b.pages.errors() == 0


@pytest.mark.parametrize("page", [8, 32, 256])
def test_append_page_sizes(lib, page):  # noqa: F811
    b = BatchQ4(lib, [5, 300], 5, 0, page, 2, 32)
    q, k, v, cs = rand(0, 10, 4, 32), rand(1, 10, 2, 32), rand(2, 10, 2, 32), rand(3, 300, 16, 2)
    before, q_out = [t.clone() for t in b.bytes], torch.zeros(10, 4, 32, device="cuda")
    lib.KvAppend(b.pages, q, k, v, cs, q_out=q_out)()
    check_append(b, before, q, k, v, q_out, cs, False)
    lib.KvAppend(b.pages, q, k, v, cs, q_out=q)()                          # q in place
    assert torch.equal(q, q_out)


@pytest.mark.parametrize("size", [1e-30, 1e-7, 3e-5, 1.0, 1e3, 3e4, 6e4, 1e38])
def test_append_magnitudes(lib, size):  # noqa: F811
    """Differences below FP16's smallest d, and values beyond its range."""
    b = BatchQ4(lib, [9], 4, 0, 16, 2, 64)
    k, v, cs = rand(1, 4, 2, 64, std=size), rand(2, 4, 2, 64, std=size), torch.zeros(16, 0, 2, device="cuda")
    k[1], v[2] = 3.0, size                                                  # constant groups
    before = [t.clone() for t in b.bytes]
    lib.KvAppend(b.pages, None, k, v, cs)()
    check_append(b, before, None, k, v, None, cs, False)


@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan])
def test_append_values_that_are_not_finite(lib, what):  # noqa: F811
    """One makes its group NaN, and no other."""
    b = BatchQ4(lib, [9], 4, 0, 16, 2, 64)
    k, v, cs = rand(1, 4, 2, 64), rand(2, 4, 2, 64), torch.zeros(16, 0, 2, device="cuda")
    k[1, 0, 33], v[3, 1, 31] = what, what
    before = [t.clone() for t in b.bytes]
    lib.KvAppend(b.pages, None, k, v, cs)()
    check_append(b, before, None, k, v, None, cs, False)
    b.read()
    (p, r), (o, q) = b.slot(0, 6), b.slot(0, 8)
    assert b.k[p, r, 0, 32:].isnan().all() and b.k[p, r, 0, :32].isfinite().all() and b.k[p, r, 1].isfinite().all()
    assert b.v[o, q, 1, :32].isnan().all() and b.v[o, q, 1, 32:].isfinite().all()


def test_what_four_bits_lose(lib):  # noqa: F811
    """A value is at most half of d off, and what d, m, the value and the F32 operations are rounded by:
    n reaches 15 d, so d's rounding counts 15 times (of d itself at most (max - min) / 15)."""
    b = BatchQ4(lib, [64] * 20, 64, 0, 16, 4, 64)
    k, v, cs = rand(1, 1280, 4, 64), rand(2, 1280, 4, 64, std=3.0), torch.zeros(64, 0, 2, device="cuda")
    lib.KvAppend(b.pages, None, k, v, cs)()
    ko, vo = (torch.empty(1280, 4, 64, device="cuda") for _ in range(2))
    lib.KvRead(b.pages, ko, vo)()
    for x, y in ((k, ko), (v, vo)):
        t = x.double().view(1280, 4, 2, 32)
        span, big = (t.amax(-1) - t.amin(-1))[..., None], t.abs().amax(-1)[..., None]
        tol = span / 30 * (1 + 2 * H16) + H16 * (span + 2 * big) + 40 * H32 * (span + big)
        assert ((t - y.double().view_as(t)).abs() <= tol).all()


def test_bad_places_are_flagged_and_skipped(lib):  # noqa: F811
    b = BatchQ4(lib, [16, 20, 33, 4], 2, 0, 16, 1, 32)
    b.table[0, 0], b.table[1, 1] = b.n_pages, -1
    k, v, cs = rand(1, 8, 1, 32, dtype=F16), rand(2, 8, 1, 32, dtype=F16), rand(3, 33, 16, 2)
    before = [t.clone() for t in b.bytes]
    lib.KvAppend(b.pages, None, k, v, cs)()
    assert b.pages.errors() == lib.LLM_PAGES_BAD_PAGE
    b.lens, b.table[0, 0] = [0, 0, 33, 4], 0
    check_append(b, before, None, k, v, None, cs, False)
    b.table[0, 0] = b.n_pages
    out = torch.full((8, 1, 32), 5.0, device="cuda")
    b.pages.err.zero_()
    lib.KvRead(b.pages, out, out.clone())()
    assert b.pages.errors() == lib.LLM_PAGES_BAD_PAGE
    assert (out[:4] == 5.0).all() and not (out[4:] == 5.0).any()
    c = BatchQ4(lib, [32], 2, 0, 16, 1, 32)
    c.lens_dev[0] = 34                                                     # both rows behind the two pages
    before = [t.clone() for t in c.bytes]
    lib.KvAppend(c.pages, None, k[:2], v[:2], rand(3, 40, 16, 2))()
    assert c.pages.errors() == lib.LLM_PAGES_BAD_LEN and all(torch.equal(x, y) for x, y in zip(before, c.bytes))


@pytest.mark.parametrize("dtype", [F32, F16])
def test_read_of_f16_pages(lib, dtype):  # noqa: F811
    """Also a whole sequence as a prefix, by as many new tokens as it has rows."""
    from test_batch_ops_gpu import Batch
    b = Batch(lib, [40, 0, 17], 40, 0, 8, 2, 40)
    ko, vo = (torch.full((120, 2, 40), 9.0, dtype=dtype, device="cuda") for _ in range(2))
    lib.KvRead(b.pages, ko, vo)()
    for row, s, e in b.rows():
        p, r = b.slot(s, e)
        assert torch.equal(ko[row], b.k[p, r].to(dtype)) and torch.equal(vo[row], b.v[p, r].to(dtype))
    assert torch.equal(ko[:40].double(), b.gather(b.k, 0, 40))
    assert (ko[40:80] == 9.0).all() and (vo[80:103] == 9.0).all()
    assert b.pages.errors() == 0


# --------------------------------------------------------------- attention --
def run_attend(lib, heads, lens, n_new, prefix, page, q_dtype, out_dtype, seed=0, std=1.0, scale=0.0):  # noqa: F811
    n_heads, n_kv, hd = heads
    b = BatchQ4(lib, lens, n_new, prefix, page, n_kv, hd, seed)
    n = len(lens) * n_new
    q = rand(seed + 11, n, n_heads, hd, dtype=q_dtype, std=std)
    pk, pv = (rand(seed + i, prefix + 2, n_kv, hd, dtype=F16) for i in (12, 13))
    for t in (pk, pv):
        t[prefix:] = math.nan
    out = torch.full((n, n_heads, hd), 9.0, dtype=out_dtype, device="cuda")
    lib.AttendBatch(b.pages, q, out, pk, pv, scale=scale)()
    check_attend(b, q, out, pk, pv, scale or None)
    live = {r for r, _, _ in b.rows()}
    assert all((out[r] == 9.0).all() for r in range(n) if r not in live)
    assert b.pages.errors() == 0
    return b, q, pk, pv, out


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("heads", [(8, 2, 32), (6, 6, 48), (8, 2, 64), (3, 3, 128), (10, 2, 128), (7, 1, 80), (4, 2, 16), (16, 1, 64),
                                   (20, 1, 96), (24, 2, 112)])
def test_attend_heads(lib, heads, types):  # noqa: F811
    run_attend(lib, heads, [1, 16, 17, 0, 100, 33, 250], 1, 300, 16, *types)


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
@pytest.mark.parametrize("prefix", [0, 1, 64, 129])
@pytest.mark.parametrize("page", [8, 16, 32, 512])
def test_attend_page_sizes_and_prefixes(lib, page, prefix, types):  # noqa: F811
    run_attend(lib, (4, 2, 64), [1, 2, 7, 8, 9, 31, 32, 33, 127, 129, 700], 1, prefix, page, *types)


@pytest.mark.parametrize("n_new,lens", [(2, [2, 1, 0, 50]), (5, [5, 3, 77, 130]), (9, [9, 200]), (40, [41, 12, 300]), (130, [130, 400])])
@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_attend_several_new_tokens(lib, n_new, lens, types):  # noqa: F811
    run_attend(lib, (8, 2, 64), lens, n_new, 70, 16, *types)
    run_attend(lib, (3, 3, 128), lens, n_new, 0, 8, *types)


@pytest.mark.parametrize("n_seqs", [1, 31, 33, 100, 257])
def test_attend_batch_sizes(lib, n_seqs):  # noqa: F811
    lens = [1 + (37 * s) % 90 for s in range(n_seqs)]
    run_attend(lib, (4, 1, 64), lens, 1, 520, 16, F16, F16)
    run_attend(lib, (2, 2, 32), lens, 1, 0, 16, F32, F32)


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_attend_long(lib, types):  # noqa: F811
    run_attend(lib, (4, 1, 64), [20000, 7, 1], 1, 0, 32, *types)
    run_attend(lib, (2, 2, 128), [9000, 7], 2, 500, 32, *types)


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_attend_peaked_and_flat_scores(lib, types):  # noqa: F811
    run_attend(lib, (4, 2, 64), [60, 200], 1, 90, 16, *types, std=30.0)
    run_attend(lib, (4, 2, 64), [60, 200], 1, 0, 16, *types, std=0.0)
    run_attend(lib, (4, 2, 64), [60, 200], 1, 90, 16, *types, scale=0.37)


def poke(b, which, s, e, g, group, d, m):
    """Another pair for one group of a row."""
    p, r = b.slot(s, e)
    n_groups = -(-b.hd // 32)
    at = b.page * b.n_kv * b.hd // 2 + ((g * b.page + r) * n_groups + group) * 4
    b.bytes[which][p, at:at + 4] = torch.tensor([d, m], dtype=F16, device="cuda").view(torch.uint8)
    b.read()


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_attend_rising_scores(lib, types):  # noqa: F811
    """Every key's score is above the one before."""
    b = BatchQ4(lib, [300], 1, 0, 16, 1, 64)
    p, n_groups, a = b.table[0].tolist(), 2, 16 * 32
    s = torch.zeros(b.n_pages, 1, 16, n_groups, 2, dtype=F16)
    for e in range(300):
        s[p[e // 16], 0, e % 16, :, 1] = e / 4
    b.bytes[0][:, a:] = s.view(b.n_pages, -1).view(torch.uint8).cuda()
    b.read()
    q, out = torch.ones(1, 2, 64, dtype=types[0], device="cuda"), torch.empty(1, 2, 64, dtype=types[1], device="cuda")
    lib.AttendBatch(b.pages, q, out)()
    check_attend(b, q, out, None, None)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("what", [(math.inf, 0.0), (math.nan, math.nan), (0.0, -math.inf), (60000.0, 60000.0)])
@pytest.mark.parametrize("heads", [(4, 2, 64), (4, 2, 128), (16, 2, 64)])
def test_attend_wild_values_of_later_tokens(lib, heads, types, what):  # noqa: F811
    """K or V of a new token that is not finite reaches that token and the ones behind it, none before it."""
    n_heads, n_kv, hd = heads
    h = n_heads // 2
    b = BatchQ4(lib, [37, 4], 4, 40, 16, n_kv, hd)
    q, pk, pv = rand(1, 8, n_heads, hd, dtype=types[0]), rand(2, 40, n_kv, hd, dtype=F16), rand(3, 40, n_kv, hd, dtype=F16)
    poke(b, 1, 0, 35, 0, 1, *what)
    poke(b, 0, 1, 1, 1, 0, math.nan, math.nan)
    poke(b, 1, 1, 1, 1, 0, *what)
    out = torch.empty(8, n_heads, hd, dtype=types[1], device="cuda")
    op = lib.AttendBatch(b.pages, q, out, pk, pv)
    op()
    p, r = b.slot(0, 35)
    bad = ~b.v[p, r, 0].isfinite()
    assert bad[32:64].any() and not bad[:32].any()
    assert out[:2].isfinite().all() and out[4].isfinite().all()
    assert not out[2:4, :h, bad].isfinite().any() and out[2:4, :h, ~bad].isfinite().all() and out[2:4, h:].isfinite().all()
    assert not out[5:, h:].isfinite().any() and out[5:, :h].isfinite().all()
    wild = out.clone()
    poke(b, 1, 0, 35, 0, 1, 0.1, -0.5)
    poke(b, 0, 1, 1, 1, 0, 0.1, -0.5)
    poke(b, 1, 1, 1, 1, 0, 0.1, -0.5)
    op()
    check_attend(b, q, out, pk, pv)
    assert torch.equal(out[:2], wild[:2]) and torch.equal(out[4], wild[4])


def test_attend_bad_pages(lib):  # noqa: F811
    b = BatchQ4(lib, [40, 10, 20], 1, 0, 16, 2, 64)
    b.table[0, 1], b.table[1, 0] = b.n_pages + 5, -1
    q, out = rand(1, 3, 4, 64), torch.full((3, 4, 64), 9.0, device="cuda")
    lib.AttendBatch(b.pages, q, out)()
    assert b.pages.errors() == lib.LLM_PAGES_BAD_PAGE
    assert (out[1] == 0).all()
    part = BatchQ4.__new__(BatchQ4)
    part.__dict__.update(b.__dict__, lens=[24], table=b.table[:1, [0, 2]])          # sequence 0 without its bad page
    check_attend(part, q[:1], out[:1], None, None)
    b.lens = [0, 0, 20]
    check_attend(b, q, out, None, None)
    c = BatchQ4(lib, [32], 1, 0, 16, 2, 64)
    c.lens_dev[0] = 50
    lib.AttendBatch(c.pages, q[:1], out[:1])()
    assert c.pages.errors() == lib.LLM_PAGES_BAD_LEN
    check_attend(c, q[:1], out, None, None)


def test_attend_strides_and_same_bits_every_run(lib):  # noqa: F811
    b = BatchQ4(lib, [200, 1, 77, 500], 2, 100, 16, 2, 64)
    wide, fused, outs = rand(1, 8, 9, 64), rand(2, 100, 4, 64, dtype=F16), torch.full((8, 6, 64), 3.0, device="cuda")
    q, out, pk, pv = wide[:, 2:6], outs[:, 1:5], fused[:, :2], fused[:, 2:]
    op = lib.AttendBatch(b.pages, q, out, pk, pv)
    op()
    check_attend(b, q, out, pk, pv)
    first = outs.clone()
    for _ in range(4):
        op.workspace.fill_(0xFF)
        op()
        assert torch.equal(outs, first)


def test_attend_is_that_of_the_values(lib):  # noqa: F811
    """F16 pages with the values that 4-bit pages stand for give the same attention within both bounds'
    roundings: the same products, summed in another order."""
    b = BatchQ4(lib, [300, 5, 64], 1, 0, 16, 2, 128)
    q = rand(1, 3, 8, 128, dtype=F16)
    out, other = (torch.empty(3, 8, 128, device="cuda") for _ in range(2))
    lib.AttendBatch(b.pages, q, out)()
    lib.AttendBatch(lib.PagedBatch(b.k, b.v, b.table, b.lens_dev), q, other)()
    check_attend(b, q, out, None, None)
    check_attend(b, q, other, None, None)


def test_pool_behind_32_bits(lib):  # noqa: F811
    """Pages whose offset passes 2^32 bytes."""
    n_pages, one = 6500000, page_bytes(16, 1, 64)
    k, v = (torch.zeros(n_pages, one, dtype=torch.uint8, device="cuda") for _ in range(2))
    b = BatchQ4(lib, [60], 1, 0, 16, 1, 64)
    ids = [n_pages - 1, 5, n_pages - 2, 6300000]
    for t, o in zip((k, v), b.bytes):
        for j, p in zip(ids, b.table[0].tolist()):
            t[j] = o[p]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    pages = lib.PagedBatchQ4(k, v, table, b.lens_dev, 16, 1, 64)
    q, out = rand(3, 1, 2, 64), torch.empty(1, 2, 64, device="cuda")
    new_k, new_v, cs = rand(7, 1, 1, 64), rand(8, 1, 1, 64), rand(9, 60, 32, 2)
    for p in (pages, b.pages):
        lib.KvAppend(p, None, new_k, new_v, cs)()
    for j, o in zip(ids, b.table[0].tolist()):
        assert torch.equal(k[j], b.bytes[0][o]) and torch.equal(v[j], b.bytes[1][o])
    b.read()
    lib.AttendBatch(pages, q, out)()
    check_attend(b, q, out, None, None)
    ko, vo = (torch.empty(1, 1, 64, device="cuda") for _ in range(2))
    lib.KvRead(pages, ko, vo)()
    p, r = b.slot(0, 59)
    assert torch.equal(ko[0], b.k[p, r].float()) and torch.equal(vo[0], b.v[p, r].float())


@pytest.mark.parametrize("prefix", [0, 70])
def test_attend_most_sequences(lib, prefix):  # noqa: F811
    run_attend(lib, (2, 1, 16), [1 + s % 21 for s in range(4096)], 1, prefix, 8, F16, F16)


@pytest.mark.parametrize("heads", [(8, 2, 64), (4, 4, 128), (8, 8, 48), (20, 4, 96)])
@pytest.mark.parametrize("n_new", [1, 3])
def test_attend_units_behind_one_another(lib, heads, n_new):  # noqa: F811
    """Many short sequences: warps walk through several units, whole ones and parts."""
    lens = [max(n_new, 1 + (53 * s) % 67) for s in range(300)]
    run_attend(lib, heads, lens, n_new, 0, 32, F16, F32, seed=n_new)


def test_rows_behind_the_last_do_not_matter(lib):  # noqa: F811
    """Other numbers in the rows behind each sequence's last one, and NaN pairs or others: the same bits."""
    b = BatchQ4(lib, [5, 13, 30, 41, 100], 1, 0, 16, 2, 64)
    q, out = rand(1, 5, 8, 64), torch.empty(5, 8, 64, device="cuda")
    op = lib.AttendBatch(b.pages, q, out)
    op()
    first = out.clone()
    for s, n in enumerate(b.lens):
        for e in range(n, -(-n // 16) * 16):
            for g in range(2):
                for which in (0, 1):
                    p, r = int(b.table[s, e // 16]), e % 16
                    b.bytes[which][p, (g * 16 + r) * 32:(g * 16 + r) * 32 + 32] = 0x5A
                    at = 16 * 2 * 32 + ((g * 16 + r) * 2) * 4
                    b.bytes[which][p, at:at + 8] = torch.tensor([1e3, -7.0, math.inf, -math.inf], dtype=F16, device="cuda").view(torch.uint8)
    op()
    assert torch.equal(out, first) and out.isfinite().all()


@pytest.mark.parametrize("kind", ["q4", "f16"])
@pytest.mark.parametrize("n_new", [1, 5])
@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_attend_rows_up_to_the_last_that_31_bits_count(lib, kind, n_new, types):  # noqa: F811
    """Sequences of up to 2^31 - 8 rows whose table names one page again and again, with keys so far below the last four
    pages' that they count for nothing (scores differ by more than 80: 2^31 e^-80 is 4e-26): what those four alone give."""
    from test_batch_ops_gpu import Batch
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("not enough memory for a table of 2^28 entries")
    low, far = 6, [1, 4, 0, 3]                                      # pages
    b = BatchQ4(lib, [32], n_new, 0, 8, 1, 16) if kind == "q4" else Batch(lib, [32], n_new, 0, 8, 1, 16, poison=False)
    if kind == "q4":
        for t, x in zip(b.bytes, (-60.0, 5.0)):
            pairs = t[:, 64:].view(F16).view(b.n_pages, 8, 2)
            pairs[:] = torch.where(pairs.isnan(), torch.tensor([0.1, -0.75], dtype=F16, device="cuda"), pairs)
            pairs[low, :, 0], pairs[low, :, 1] = 0.0, x
        b.read()
    else:
        b.k[low], b.v[low] = -60.0, 5.0
    table = torch.full((1, (1 << 28) - 1), low, dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    pages = (lib.PagedBatchQ4(*b.bytes, table, lens, 8, 1, 16, n_new=n_new) if kind == "q4"
             else lib.PagedBatch(b.k, b.v, table, lens, n_new=n_new))
    q, out = rand(3, n_new, 4, 16).abs().add_(0.3).to(types[0]), torch.empty(n_new, 4, 16, dtype=types[1], device="cuda")
    op = lib.AttendBatch(pages, q, out)
    ko, vo = (torch.empty(n_new, 1, 16, device="cuda") for _ in range(2))
    read = lib.KvRead(pages, ko, vo)
    b.table = torch.tensor([far], dtype=torch.int32, device="cuda")
    for n in (2 ** 31 - 8, 2 ** 31 - 9, 2 ** 31 - 15, 2 ** 31 - 16, 2 ** 31 - 17, 2 ** 31 - 23, 2 ** 31 - 32, 2 ** 31 - 41, 2 ** 30 + 3):
        last = (n - 1) // 8
        table[0, last - 3:last + 1] = b.table[0]
        lens[0], b.lens = n, [n - 8 * (last - 3)]
        op()
        read()
        check_attend(b, q, out, None, None, what=f"{n} rows,")
        for row, s, e in b.rows():
            p, r = b.slot(s, e)
            assert torch.equal(ko[row], b.k[p, r].float()) and torch.equal(vo[row], b.v[p, r].float())
        assert pages.errors() == 0
        table[0, last - 3:last + 1] = low


@pytest.mark.parametrize("offset", [0.3, 1000.24, -1000.24, 60000.0, -60000.0, 65503.0])
@pytest.mark.parametrize("spread", [1e-6, 1e-4, 1e-2, 0.7, 40.0])
def test_append_small_spreads_about_large_values(lib, offset, spread):  # noqa: F811
    """m is off by up to half an FP16 step of the values, many times d: quotients far beyond 15, or far below 0."""
    b = BatchQ4(lib, [9], 8, 0, 16, 2, 64)
    k, v = (offset + spread * torch.rand(8, 2, 64, generator=torch.Generator().manual_seed(i)).cuda() for i in (1, 2))
    k[3, 0, 5], v[4, 1, 40] = k[3, 0, 5] + 15 * spread, v[4, 1, 40] - 15 * spread
    before = [t.clone() for t in b.bytes]
    lib.KvAppend(b.pages, None, k, v, torch.zeros(16, 0, 2, device="cuda"))()
    check_append(b, before, None, k, v, None, torch.zeros(16, 0, 2), False)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("heads,n_new", [((20, 1, 48), 1), ((24, 1, 32), 1), ((36, 2, 16), 1), ((8, 2, 32), 5), ((6, 2, 48), 7), ((4, 1, 16), 6)])
def test_attend_24_query_rows_of_short_heads(lib, heads, n_new, types):  # noqa: F811
    run_attend(lib, heads, [max(n_new, n) for n in (1, 16, 17, 33, 250)] + [2], n_new, 70, 16, *types)
    run_attend(lib, heads, [max(n_new, n) for n in (8, 31, 32, 65)], n_new, 0, 8, *types)


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
@pytest.mark.parametrize("heads,n_new", [((25, 1, 32), 1), ((40, 1, 48), 1), ((8, 2, 32), 10), ((4, 1, 16), 33)])
def test_attend_many_query_rows_of_short_heads(lib, heads, n_new, types):  # noqa: F811
    run_attend(lib, heads, [max(n_new, n) for n in (1, 17, 100, 250)] + [3], n_new, 70, 16, *types)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("what", [(math.inf, 0.0), (math.nan, math.nan), (60000.0, 60000.0)])
@pytest.mark.parametrize("heads,n_new", [((4, 1, 64), 6), ((8, 2, 64), 5), ((6, 2, 48), 7), ((8, 2, 32), 5)])
def test_attend_wild_values_of_later_tokens_in_24_query_rows(lib, heads, n_new, types, what):  # noqa: F811
    """As test_attend_wild_values_of_later_tokens: they reach their token and the ones behind it, none before it."""
    n_heads, n_kv, hd = heads
    h, group = n_heads // n_kv, min(1, -(-hd // 32) - 1)
    b = BatchQ4(lib, [37, 100], n_new, 40, 16, n_kv, hd)
    n = 2 * n_new
    q, pk, pv = rand(1, n, n_heads, hd, dtype=types[0]), rand(2, 40, n_kv, hd, dtype=F16), rand(3, 40, n_kv, hd, dtype=F16)
    poke(b, 1, 0, 35, 0, group, *what)                              # V of the last token but one
    poke(b, 0, 1, 98, 0, 0, math.nan, math.nan)                     # K of the last but one
    out = torch.empty(n, n_heads, hd, dtype=types[1], device="cuda")
    op = lib.AttendBatch(b.pages, q, out, pk, pv)
    op()
    p, r = b.slot(0, 35)
    bad = ~b.v[p, r, 0].isfinite()
    assert bad.any()
    first, second = out[:n_new], out[n_new:]
    assert first[:-2].isfinite().all() and second[:-2].isfinite().all()
    assert not first[-2:, :h, bad].isfinite().any() and first[-2:, :h, ~bad].isfinite().all() and first[-2:, h:].isfinite().all()
    assert second[-2:, :h].isnan().all() and second[-2:, h:].isfinite().all()
    wild = out.clone()
    poke(b, 1, 0, 35, 0, group, 0.1, -0.5)
    poke(b, 0, 1, 98, 0, 0, 0.1, -0.5)
    op()
    check_attend(b, q, out, pk, pv)
    assert torch.equal(out[:n_new - 2], wild[:n_new - 2]) and torch.equal(out[n_new:n - 2], wild[n_new:n - 2])


@pytest.mark.parametrize("q_dtype,std", [(F32, 0.05), (F16, 0.05), (F32, 0.0), (F16, 0.0)])
@pytest.mark.parametrize("heads", [(1, 1, 64), (8, 1, 64), (20, 1, 64), (4, 1, 128), (12, 1, 128), (7, 1, 48)])
def test_attend_sums_of_many_rows_do_not_fall_short(lib, heads, q_dtype, std):  # noqa: F811
    """2^26 rows (of 4096 pages) that count much alike, with values of one sign.

    A share's sum takes N additions, one for each of its pieces of 16 rows, and the join one for each of at most W
    parts.  Each is rounded to nearest, by at most H32 of the sum so far; over pieces in no order these are
    independent, of deviation at most H32 / sqrt(3): six deviations of an element's sum, and of the mean error over the hd
    elements, are allowed.  What may lean to one side: a piece's own sum, whose products the matrix instruction cuts off
    (four cuts of at most a step, 2 H32), a probability as two F16 parts (2^-22), and the scores (attend_bound's ds,
    which moves the mean of the values by at most twice that of their mean distance from it).  A sum that is itself cut
    off at every piece falls short by half a step of a sum half as large on the average: 2e-5 and more here.
    With std 0 (every row counts alike) a thread's sum of probabilities takes N / 2 additions, one a step of 32 rows, of equal
    numbers, whose roundings are not independent: H32 of the sum so far each, half the sum on the average, H32 N / 4."""
    n_heads, n_kv, hd = heads
    n, page, n_pages = 1 << 26, 16, 4096
    b = BatchQ4(lib, [n_pages * page], 1, 0, page, n_kv, hd)
    g = -(-hd // 32)
    pairs = b.bytes[1][:, page * n_kv * hd // 2:][:, :page * n_kv * g * 4].view(F16).view(b.n_pages, -1, 2)
    r = torch.Generator().manual_seed(3)
    pairs[..., 0] = (0.02 + 0.2 * torch.rand(pairs.shape[:2], generator=r)).half().cuda()
    pairs[..., 1] = (0.5 + torch.rand(pairs.shape[:2], generator=r)).half().cuda()
    b.read()
    which = torch.randint(0, n_pages, (n // page,), generator=r)
    pages = lib.PagedBatchQ4(*b.bytes, b.table[0][which.cuda()][None].contiguous(), torch.tensor([n], dtype=torch.int32, device="cuda"), page, n_kv, hd)
    q, out = rand(4, 1, n_heads, hd, dtype=q_dtype, std=std), torch.empty(1, n_heads, hd, device="cuda")
    lib.AttendBatch(pages, q, out)()
    k, v = (b.gather(t, 0, n_pages * page)[:, 0] for t in (b.k, b.v))                 # [rows, hd]
    count = torch.bincount(which, minlength=n_pages).double().cuda().repeat_interleave(page)
    s = q[0].double() @ k.T * hd ** -0.5
    w = count * (s - s.amax(-1, keepdim=True)).exp()
    w /= w.sum(-1, keepdim=True)
    want = w @ v
    mag = float((q[0].double().abs() @ k.abs().T).max()) * hd ** -0.5
    ds = mag * ((hd + 4) * 2 * H32 + 2.0 ** -22) + 3 * (mag + 2 * float(s.abs().max())) * H32 + 2.0 ** -22
    apart = max(float((w[h] @ (v - want[h]).abs() / want[h]).max()) for h in range(n_heads))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    workers = 4 * 2 * sms                                           # at least: two blocks of four warps an SM (at most four)
    deviation = H32 * math.sqrt((n / 16 / workers + 2 * workers) / 3)
    lean = 4 * 2 * H32 + 2.0 ** -22 + 2 * ds * apart + (H32 * n / 16 / workers / 4 if std == 0 else 0)
    e = out[0].double() / want - 1
    assert e.abs().max() <= lean + 6 * deviation, (float(e.abs().max()), lean, deviation)
    assert e.mean(-1).abs().max() <= lean + 6 * deviation / math.sqrt(hd), (e.mean(-1).tolist(), lean, deviation)
    assert pages.errors() == 0
