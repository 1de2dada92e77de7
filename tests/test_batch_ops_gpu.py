"""The operators of batched decoding on the GPU against their formulas in 64
bits: the paged K/V append with RoPE, attention over a shared prefix and the
sequences' own pages, and log probabilities.

Tolerances are error bounds, counted in roundings (half a step: F16 2^-11, F32
2^-24) before the first run:
- append: two products and a sum in F32, then one rounding to the output type;
- attention: see attend_bound;
- log probabilities: see logprob_bound."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, F16 = torch.float32, torch.float16
H16 = 2.0 ** -11        # half a step of F16
H32 = 2.0 ** -24        # half a step of F32


@pytest.fixture(scope="module")
def lib():
    import llama_decode_forward_gb300 as L
    return L


def rand(seed, *shape, dtype=F32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


class Batch:
    """A paged batch with scattered pages; everything that no row may touch is
    NaN: unused pages, rows behind each sequence's last one."""

    def __init__(self, lib, lens, n_new, prefix, page, n_kv, hd, seed=0, extra=3, poison=True):
        self.lens, self.n_new, self.prefix, self.page = lens, n_new, prefix, page
        need = [-(-max(n, 0) // page) for n in lens]
        self.n_pages, width = sum(need) + extra, max(need + [1])
        order = np.random.RandomState(seed).permutation(self.n_pages)
        table = np.full((len(lens), width), -7, np.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        self.k, self.v = (rand(seed + i, self.n_pages, page, n_kv, hd, dtype=F16) for i in (1, 2))
        if poison:
            live = torch.zeros(self.n_pages, page, dtype=torch.bool)
            for s, n in enumerate(lens):
                for e in range(max(n, 0)):
                    live[table[s, e // page], e % page] = True
            for t in (self.k, self.v):
                t[~live.cuda()] = math.nan
        self.lens_dev = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.pages = lib.PagedBatch(self.k, self.v, self.table, self.lens_dev, n_new=n_new, prefix_len=prefix)

    def rows(self):
        """(row, sequence, suffix index) of every new token that is no padding."""
        for s, n in enumerate(self.lens):
            for i in range(self.n_new):
                if n - self.n_new + i >= 0:
                    yield s * self.n_new + i, s, n - self.n_new + i

    def slot(self, s, e):
        return int(self.table[s, e // self.page]), e % self.page

    def gather(self, t, s, n):
        """Rows 0..n-1 of sequence s in 64 bits."""
        if n == 0:
            return t.new_zeros(0, *t.shape[2:]).double()
        return t[self.table[s, :-(-n // self.page)].long()].flatten(0, 1)[:n].double()


# ------------------------------------------------------------------ append --
def rotated(x, cs, neox):
    """RoPE of one row's heads [heads, hd] in 64 bits, and the bound's scale:
    the sum of the two products' magnitudes."""
    y, mag = x.clone(), x.abs()
    half = cs.shape[0]
    a = torch.arange(half) if neox else 2 * torch.arange(half)
    b = a + half if neox else a + 1
    c, s = cs[:, 0], cs[:, 1]
    y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, a] * s + x[:, b] * c
    mag[:, a] = (x[:, a] * c).abs() + (x[:, b] * s).abs()
    mag[:, b] = (x[:, a] * s).abs() + (x[:, b] * c).abs()
    return y, mag


def check_append(b, before, q, k, v, q_out, cs, neox, rope_dims):
    got_k, got_v, got_q = b.k.cpu(), b.v.cpu(), None if q is None else q_out.double().cpu()
    want_k, want_v = before[0].cpu(), before[1].cpu()
    q, k, v = (None if t is None else t.double().cpu() for t in (q, k, v))
    cs = cs.double().cpu()
    half = rope_dims // 2
    h_out = H16 if q is not None and q_out.dtype == F16 else 0.0
    for row, s, e in b.rows():
        p, r = b.slot(s, e)
        y, mag = rotated(k[row], cs[b.prefix + e], neox)
        near = torch.zeros_like(mag, dtype=torch.bool)
        err = (got_k[p, r].double() - y).abs()
        near = err <= 3 * H32 * mag * (1 + H16) + H16 * y.abs() + 2.0 ** -25
        assert near.all(), (row, float(err.max()))
        assert torch.equal(got_k[p, r][:, 2 * half:], k[row][:, 2 * half:].to(F16))       # dims that are not rotated
        assert torch.equal(got_v[p, r], v[row].to(F16))
        want_k[p, r], want_v[p, r] = got_k[p, r], got_v[p, r]
        if q is not None:
            y, mag = rotated(q[row], cs[b.prefix + e], neox)
            assert ((got_q[row] - y).abs() <= 3 * H32 * mag * (1 + h_out) + h_out * y.abs() + (2.0 ** -25 if h_out else 0)).all(), row
    # every other slot keeps its bits
    assert torch.equal(got_k.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(got_v.view(torch.int16), want_v.view(torch.int16))


@pytest.mark.parametrize("heads,rope,neox", [
    ((8, 2, 32), 32, False), ((6, 6, 48), 48, True), ((4, 2, 64), 64, True), ((4, 2, 64), 20, False),
    ((4, 1, 40), 10, True), ((3, 3, 128), 128, False), ((2, 1, 8), 8, True), ((2, 1, 24), 2, True), ((0, 2, 64), 64, False),
    ((4, 2, 64), 0, True), ((4, 2, 128), 96, True),
])
@pytest.mark.parametrize("dtype,out", [(F32, F32), (F32, F16), (F16, F16), (F16, F32)])
def test_append(lib, heads, rope, neox, dtype, out):
    n_heads, n_kv, hd = heads
    b = Batch(lib, [1, 17, 40, 0, 3, 64], 3, 21, 16, n_kv, hd)          # padding rows in sequences 0 and 3
    n = 6 * 3
    qkv = rand(5, n, n_heads + 2 * n_kv, hd, dtype=dtype)
    q, k, v = qkv[:, :n_heads], qkv[:, n_heads:n_heads + n_kv], qkv[:, n_heads + n_kv:]
    cs = rand(6, 21 + 64, rope // 2, 2)
    q_out = torch.full((n, n_heads, hd), 7.0, dtype=out, device="cuda")
    before = b.k.clone(), b.v.clone()
    lib.KvAppend(b.pages, q if n_heads else None, k, v, cs, q_out=q_out, rope_neox=neox)()
    check_append(b, before, q if n_heads else None, k, v, q_out, cs, neox, rope)
    live = {r for r, _, _ in b.rows()}
    for r in range(n):
        if r not in live:
            assert (q_out[r] == 7.0).all()                              # padding rows are left as they were
    assert b.pages.errors() == 0


@pytest.mark.parametrize("page", [1, 2, 8, 64, 256])
def test_append_page_sizes_and_strides(lib, page):
    b = Batch(lib, [5, 130], 5, 0, page, 2, 32)
    wide = rand(1, 10, 11, 32)
    q, k, v = wide[:, :4], wide[:, 5:7], wide[:, 8:10]
    cs = rand(2, 130, 16, 2)
    q_out = torch.zeros(10, 8, 32, device="cuda")[:, 2:6]
    before = b.k.clone(), b.v.clone()
    lib.KvAppend(b.pages, q, k, v, cs, q_out=q_out)()
    check_append(b, before, q, k, v, q_out, cs, False, 32)
    # q rotated in place: the same bits
    again = lib.KvAppend(b.pages, q, k, v, cs, q_out=q)
    again()
    assert torch.equal(q, q_out)


def test_append_without_rotation_needs_no_table(lib):
    b = Batch(lib, [5, 17], 2, 1000, 16, 2, 64)
    k, v = rand(1, 4, 2, 64), rand(2, 4, 2, 64)
    before = b.k.clone(), b.v.clone()
    op = lib.KvAppend(b.pages, None, k, v, torch.zeros(0, 0, 2, device="cuda"))
    op()
    check_append(b, before, None, k, v, None, torch.zeros(1017, 0, 2), False, 0)
    assert b.pages.errors() == 0


@pytest.mark.parametrize("n", [-1, -(1 << 31), 1 - (1 << 31)])
def test_lengths_below_zero_are_padding(lib, n):
    b = Batch(lib, [4, 0, 2], 2, 0, 16, 2, 64, poison=False)
    b.lens_dev[1] = n
    before = b.k.clone()
    q, k, v = rand(3, 6, 4, 64), rand(1, 6, 2, 64), rand(2, 6, 2, 64)
    lib.KvAppend(b.pages, None, k, v, rand(4, 8, 32, 2))()
    changed = {(int(p), int(r)) for p, r in (b.k != before).any(-1).any(-1).nonzero()}
    assert changed == {tuple(map(int, b.slot(s, e))) for s, e in ((0, 2), (0, 3), (2, 0), (2, 1))}
    out = torch.full_like(q, 7.0)
    lib.AttendBatch(b.pages, q, out)()
    assert (out[2:4] == 7.0).all() and not (out[[0, 1, 4, 5]] == 7.0).any()
    assert b.pages.errors() == 0


def test_append_bad_places_are_flagged_and_skipped(lib):
    b = Batch(lib, [16, 20, 33, 4], 2, 0, 16, 1, 32, poison=False)
    b.table[0, 0] = b.n_pages                # a page behind the pool
    b.table[1, 1] = -1                       # a page before it
    k, v, cs = rand(1, 8, 1, 32, dtype=F16), rand(2, 8, 1, 32, dtype=F16), rand(3, 33, 16, 2)
    q_out = torch.full((8, 2, 32), 5.0, device="cuda")
    q = rand(4, 8, 2, 32, dtype=F16)
    before = b.k.clone()
    lib.KvAppend(b.pages, q, k, v, cs, q_out=q_out)()
    assert b.pages.errors() == lib.LLM_PAGES_BAD_PAGE
    b.lens, b.table[0, 0] = [0, 0, 33, 4], 0           # the rows that were written
    want = before.clone()
    for row, s, e in b.rows():
        p, r = b.slot(s, e)
        want[p, r] = b.k[p, r]
        assert not torch.equal(before[p, r], b.k[p, r])
    assert torch.equal(b.k.view(torch.int16), want.view(torch.int16))
    assert not (q_out == 5.0).any()                    # q does not need the pages
    # rows behind a sequence's capacity, and behind the angle table
    c = Batch(lib, [32, 20], 2, 0, 16, 1, 32, poison=False)
    c.lens_dev[0] = 40
    before = c.k.clone()
    q_out.fill_(5.0)
    lib.KvAppend(c.pages, q[:4], k[:4], v[:4], cs[:20].contiguous(), q_out=q_out[:4])()
    assert c.pages.errors() == lib.LLM_PAGES_BAD_LEN
    assert (q_out[:2] == 5.0).all() and not (q_out[2:4] == 5.0).any()
    for p in c.table[0].tolist():
        assert torch.equal(c.k[p], before[p])
    d = Batch(lib, [32], 2, 0, 16, 1, 32, poison=False)
    d.lens_dev[0] = 34                                 # both rows behind the two pages, within the table
    before = d.k.clone()
    lib.KvAppend(d.pages, q[:2], k[:2], v[:2], rand(3, 40, 16, 2), q_out=q_out[:2])()
    assert d.pages.errors() == lib.LLM_PAGES_BAD_LEN and torch.equal(d.k, before)


def test_append_matches_the_decode_step_bit_for_bit(lib):
    """K and V rows that the decode step stores, from its own q, k and v
    (llm_debug_tensor) through llm_rope_table and llm_kv_append."""
    import synth
    for neox in (0, 1):
        cfg = synth.ModelConfig("append", n_layers=2, dim=256, n_heads=8, n_kv_heads=2, head_dim=32, ffn_dim=512,
                                vocab=500, max_seq=64, eps=1e-5, rope_base=500000.0, rope_neox=neox, wtype=synth.F16,
                                tied=True, bias=True, number=31)
        dec = lib.Decoder(cfg, synth.make_weights(cfg))
        cs = lib.rope_table(64, 32, cfg.rope_base)
        for pos in (0, 1, 63):
            lib.llm_decode_step(dec.h, 3 + pos, pos)
            for layer in range(2):
                k, v = (torch.from_numpy(lib.llm_debug_tensor(dec.h, layer, w)).cuda().view(1, 2, 32)
                        for w in (lib.LLM_DEBUG_K, lib.LLM_DEBUG_V))
                b = Batch(lib, [pos + 1], 1, 0, 16, 2, 32, poison=False)
                lib.KvAppend(b.pages, None, k, v, cs, rope_neox=bool(neox))()
                p, r = b.slot(0, pos)
                kc, vc = dec.kv_tensors(layer)
                assert torch.equal(b.k[p, r].view(torch.int16).flatten(), kc[pos])
                assert torch.equal(b.v[p, r].view(torch.int16).flatten(), vc[pos])
        dec.close()


def test_rope_table_far_positions_and_factors(lib):
    f = torch.linspace(1.0, 8.0, 16).cuda()
    a, b = lib.rope_table(40, 32, 10000.0, rope_freqs=f), lib.rope_table(8, 32, 10000.0, rope_freqs=f, pos0=32)
    assert torch.equal(a[32:], b)
    # the float angle chain, restated
    theta = np.arange(40, dtype=np.float32)
    step = np.float32(10000.0 ** (-2.0 / 32))
    for j in range(16):
        ang = (theta / f[j].cpu().numpy()).astype(np.float64)
        # sin and cos in 64 bits, rounded once to 32 (half a step), with a last-bit difference of the 64-bit functions
        assert np.abs(a[:, j, 0].cpu().numpy() - np.cos(ang)).max() <= H32 * (1 + 1e-6)
        assert np.abs(a[:, j, 1].cpu().numpy() - np.sin(ang)).max() <= H32 * (1 + 1e-6)
        theta = (theta * step).astype(np.float32)


# --------------------------------------------------------------- attention --
def attend_exact(q, scale, keys, values, n_kv):
    """One row in 64 bits: q [n_heads, hd], keys/values [t, n_kv, hd]; the
    output and, for the bound, sum p|v| and the largest sum |q_i k_i| scale."""
    n_heads, hd = q.shape
    if keys.shape[0] == 0:
        z = torch.zeros_like(q)
        return z, z, z[:, :1], z[:, :1]
    qg = q.view(n_kv, n_heads // n_kv, hd)
    s = torch.einsum("ghd,tgd->ght", qg, keys) * scale
    mag = torch.einsum("ghd,tgd->ght", qg.abs(), keys.abs()) * scale
    p = torch.softmax(s, -1)
    o = torch.einsum("ght,tgd->ghd", p, values)
    w = torch.einsum("ght,tgd->ghd", p, values.abs())
    far = (s.amax(-1, keepdim=True) - s)                          # how far below the maximum
    return (o.reshape(n_heads, hd), w.reshape(n_heads, hd), mag.amax(-1).reshape(n_heads, 1),
            far.amax(-1).reshape(n_heads, 1))


def attend_bound(o, w, mag, far, vmax, t, hd, q_dtype, out_dtype):
    """|error| of an output element, from
    - the scores: hd products summed in F32 (each of the at most hd + 4 sums,
      rounded towards zero at worst, a full step 2 H32 of the magnitudes), and
      an F32 q cut to two F16 parts (2^-22); scaled and shifted (3 roundings of
      at most mag + far);
    - exp2 of the fastest kind, 2^-22 relative;
    - a probability as one F16 (H16) for F16 outputs, as two (2^-22) for F32,
      never finer than 2^-33 of the largest (subnormal F16 parts);
    - the weighted sum: at most t / 8 + 8 additions of partial sums, each a full
      step at worst, joined over at most 64 parts;
    - the sum of the probabilities: t / 32 + 64 additions in F32;
    - one rounding to the output type."""
    ds = mag * ((hd + 4) * 2 * H32 + 2.0 ** -22) + 3 * (mag + far) * H32 + 2.0 ** -22
    dp = ds + (H16 if out_dtype == F16 else 2.0 ** -22)
    sums = (t / 8 + 8 + 64 + t / 32 + 64) * 2 * H32
    tol = w * (2 * dp + ds + sums) + t * 2.0 ** -33 * vmax
    return tol + ((H16 * (o.abs() + tol) + 2.0 ** -25) if out_dtype == F16 else 2 * H32 * o.abs())


def check_attend(b, q, out, pk, pv, scale=None, what=""):
    hd, n_kv = q.shape[2], b.k.shape[2]
    scale = hd ** -0.5 if scale is None else scale
    pk, pv = (torch.zeros(0, n_kv, hd, dtype=torch.float64, device="cuda") if t is None else t[:b.prefix].double() for t in (pk, pv))
    for row, s, e in b.rows():
        keys, values = torch.cat([pk, b.gather(b.k, s, e + 1)]), torch.cat([pv, b.gather(b.v, s, e + 1)])
        o, w, mag, far = attend_exact(q[row].double(), scale, keys, values, n_kv)
        tol = attend_bound(o, w, mag, far, values.abs().max(), keys.shape[0], hd, q.dtype, out.dtype)
        err = (out[row].double() - o).abs()
        assert (err <= tol).all(), f"{what} row {row}: error {err.max():.3g}, bound there {tol.flatten()[err.argmax()]:.3g}"


def run_attend(lib, heads, lens, n_new, prefix, page, q_dtype, out_dtype, seed=0, std=1.0, scale=0.0):
    n_heads, n_kv, hd = heads
    b = Batch(lib, lens, n_new, prefix, page, n_kv, hd, seed)
    n = len(lens) * n_new
    q = rand(seed + 11, n, n_heads, hd, dtype=q_dtype, std=std)
    # two rows more than the prefix has, which nothing may read
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


TYPES = [(F32, F32), (F32, F16), (F16, F16), (F16, F32)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("heads", [(8, 2, 32), (6, 6, 48), (8, 2, 64), (3, 3, 128), (10, 2, 128), (7, 1, 72), (4, 2, 8),
                                   (16, 1, 64), (20, 1, 96)])
def test_attend_heads(lib, heads, types):
    run_attend(lib, heads, [1, 16, 17, 0, 100, 33, 250], 1, 300, 16, *types)


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
@pytest.mark.parametrize("prefix", [0, 1, 2, 63, 64, 65, 127, 128, 129, 1000, 4097])
def test_attend_prefix_lengths(lib, prefix, types):
    run_attend(lib, (8, 2, 64), [1, 5, 64, 65], 1, prefix, 16, *types)


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
@pytest.mark.parametrize("page", [1, 4, 8, 32, 128, 512])
def test_attend_page_sizes(lib, page, types):
    run_attend(lib, (4, 2, 64), [1, 31, 32, 33, 127, 129, 700], 1, 50, page, *types)


@pytest.mark.parametrize("n_new,lens", [(2, [2, 1, 0, 50]), (5, [5, 3, 77, 130]), (9, [9, 200]), (40, [41, 12, 300]),
                                        (130, [130, 400])])
@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_attend_several_new_tokens(lib, n_new, lens, types):
    run_attend(lib, (8, 2, 64), lens, n_new, 70, 16, *types)
    run_attend(lib, (3, 3, 128), lens, n_new, 0, 8, *types)


@pytest.mark.parametrize("n_seqs", [1, 31, 32, 33, 100, 257])
def test_attend_batch_sizes(lib, n_seqs):
    lens = [1 + (37 * s) % 90 for s in range(n_seqs)]
    run_attend(lib, (4, 1, 64), lens, 1, 520, 16, F16, F16)
    run_attend(lib, (2, 2, 32), lens, 1, 20, 16, F32, F32)


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_attend_long(lib, types):
    """A long prefix with a few sequences, and a long sequence among short ones."""
    run_attend(lib, (4, 1, 64), [3, 40], 1, 33001, 16, *types)
    run_attend(lib, (4, 1, 64), [20000, 7, 1], 1, 0, 32, *types)
    run_attend(lib, (2, 2, 128), [9000, 7], 2, 5000, 32, *types)


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_attend_peaked_and_flat_scores(lib, types):
    """Scores far apart (one key takes all) and all equal, and another scale."""
    run_attend(lib, (4, 2, 64), [60, 200], 1, 900, 16, *types, std=30.0)
    run_attend(lib, (4, 2, 64), [60, 200], 1, 900, 16, *types, std=0.0)
    run_attend(lib, (4, 2, 64), [60, 200], 1, 900, 16, *types, scale=0.37)


@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_attend_rising_scores(lib, types):
    """Every key's score is above the one before: the running maximum moves all
    the way, far enough that a sum kept at an old maximum would overflow."""
    b = Batch(lib, [300], 1, 700, 16, 1, 64)
    q = torch.ones(1, 2, 64, dtype=types[0], device="cuda")
    pk, pv = rand(1, 700, 1, 64, dtype=F16), rand(2, 700, 1, 64, dtype=F16)
    pk[:] = (torch.arange(700.) / 8).cuda()[:, None, None]
    rise = (87.5 + torch.arange(300.) / 8).cuda()
    for e in range(300):
        p, r = b.slot(0, e)
        b.k[p, r] = rise[e]
    out = torch.empty(1, 2, 64, dtype=types[1], device="cuda")
    lib.AttendBatch(b.pages, q, out, pk, pv)()
    check_attend(b, q, out, pk, pv)


def test_attend_strides(lib):
    """q and out as parts of wider rows, the prefix as one half of a fused cache."""
    b = Batch(lib, [20, 33], 2, 100, 16, 2, 64)
    wide, fused = rand(1, 4, 9, 64), rand(2, 100, 4, 64, dtype=F16)
    outs = torch.full((4, 6, 64), 3.0, device="cuda")
    q, out, pk, pv = wide[:, 2:6], outs[:, 1:5], fused[:, :2], fused[:, 2:]
    lib.AttendBatch(b.pages, q, out, pk, pv)()
    check_attend(b, q, out, pk, pv)
    assert (outs[:, 0] == 3.0).all() and (outs[:, 5] == 3.0).all()


def test_attend_bad_pages(lib):
    """A bad page's rows are left out and flagged; a row without any key is
    zero; a length behind the capacity reads the rows that exist."""
    b = Batch(lib, [40, 10, 20], 1, 0, 16, 2, 64)
    b.table[0, 1] = b.n_pages + 5
    b.table[1, 0] = -1
    q, out = rand(1, 3, 4, 64), torch.full((3, 4, 64), 9.0, device="cuda")
    lib.AttendBatch(b.pages, q, out)()
    assert b.pages.errors() == lib.LLM_PAGES_BAD_PAGE
    assert (out[1] == 0).all()
    rows = lambda t: torch.cat([t[b.table[0, 0]], t[b.table[0, 2], :8]]).double()  # noqa: E731
    o, w, mag, far = attend_exact(q[0].double(), 0.125, rows(b.k), rows(b.v), 2)
    assert ((out[0].double() - o).abs() <= attend_bound(o, w, mag, far, rows(b.v).abs().max(), 24, 64, F32, F32)).all()
    b.lens = [0, 0, 20]
    check_attend(b, q, out, None, None)
    c = Batch(lib, [32], 1, 0, 16, 2, 64)
    c.lens_dev[0] = 50
    out = torch.empty(1, 4, 64, device="cuda")
    lib.AttendBatch(c.pages, q[:1], out)()
    assert c.pages.errors() == lib.LLM_PAGES_BAD_LEN
    c.lens = [32]
    check_attend(c, q[:1], out, None, None)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("what", [math.inf, math.nan])
def test_attend_wild_values_of_later_tokens(lib, types, what):
    """K or V of a new token that is not finite reaches that token and the ones
    behind it, none before it."""
    b = Batch(lib, [37, 4], 4, 40, 16, 2, 64)
    q, pk, pv = rand(1, 8, 4, 64, dtype=types[0]), rand(2, 40, 2, 64, dtype=F16), rand(3, 40, 2, 64, dtype=F16)
    p, r = b.slot(0, 35)
    b.v[p, r, 0, 5] = what
    p, r = b.slot(1, 1)
    b.k[p, r, 1, 9] = math.nan
    b.v[p, r, 1, :] = what
    out = torch.empty(8, 4, 64, dtype=types[1], device="cuda")
    lib.AttendBatch(b.pages, q, out, pk, pv)()
    assert out[:2].isfinite().all() and out[4].isfinite().all()
    assert not out[2:4, :2, 5].isfinite().any() and out[2:4, 2:].isfinite().all()
    assert not out[5:, 2:].isfinite().any() and out[5:, :2].isfinite().all()
    wild = out.clone()
    for s, e in ((0, 35), (1, 1)):
        p, r = b.slot(s, e)
        b.k[p, r] = b.v[p, r] = 0.5
    lib.AttendBatch(b.pages, q, out, pk, pv)()
    check_attend(b, q, out, pk, pv)
    assert torch.equal(out[:2], wild[:2]) and torch.equal(out[4], wild[4])


def test_attend_same_bits_every_run(lib):
    b, q, pk, pv, out = run_attend(lib, (8, 2, 64), [200, 1, 77, 500, 350], 2, 3000, 16, F32, F32)
    first = out.clone()
    op = lib.AttendBatch(b.pages, q, out, pk, pv)
    for _ in range(5):
        op.workspace.fill_(0xFF)                      # the workspace's contents do not matter
        out.zero_()
        op()
        live = [r for r, _, _ in b.rows()]
        assert torch.equal(out[live], first[live])


def test_attend_pool_behind_32_bits(lib):
    """Pages whose offset passes 2^31 elements (and 2^32 bytes)."""
    n_pages = 2200000
    k = torch.empty(n_pages, 16, 1, 64, dtype=F16, device="cuda")
    v = torch.empty_like(k)
    ids = [n_pages - 1, 5, n_pages - 2, 2100000]
    for i, p in enumerate(ids):
        k[p], v[p] = rand(i, 16, 1, 64, dtype=F16), rand(50 + i, 16, 1, 64, dtype=F16)
    b = Batch.__new__(Batch)
    b.lens, b.n_new, b.prefix, b.page, b.k, b.v, b.n_pages = [60], 1, 0, 16, k, v, n_pages
    b.table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    lens = torch.tensor([60], dtype=torch.int32, device="cuda")
    pages = lib.PagedBatch(k, v, b.table, lens)
    new_k, new_v, cs = rand(7, 1, 1, 64), rand(8, 1, 1, 64), rand(9, 60, 32, 2)
    lib.KvAppend(pages, None, new_k, new_v, cs)()
    assert torch.equal(v[2100000, 11], new_v[0].to(F16))
    q, out = rand(3, 1, 2, 64), torch.empty(1, 2, 64, device="cuda")
    lib.AttendBatch(pages, q, out)()
    check_attend(b, q, out, None, None)


def test_attend_prefix_behind_32_bits(lib):
    """A strided prefix whose last rows lie behind 2^31 elements."""
    stride, n = 1 << 20, 2100
    big = torch.empty(n, stride, dtype=F16, device="cuda")
    pk, pv = (big[:, at:at + 64].unsqueeze(1) for at in (0, 128))
    pk.copy_(rand(1, n, 1, 64, dtype=F16))
    pv.copy_(rand(2, n, 1, 64, dtype=F16))
    b = Batch(lib, [3, 9], 1, n, 16, 1, 64)
    q, out = rand(3, 2, 2, 64), torch.empty(2, 2, 64, device="cuda")
    lib.AttendBatch(b.pages, q, out, pk, pv)()
    check_attend(b, q, out, pk, pv)


# ------------------------------------------------------- log probabilities --
def logprob_bound(x, logp, vocab):
    """|error| of ln p = (x - m) - ln S: the sum S of at most vocab terms, kept
    by at least 256 partial sums (vocab / 256 + 64 additions of H32 each, and the
    running maximum's rescalings among them), exp2 2^-22, its argument's
    rounding at the most probable tokens (2 H32 of at most 40), then two
    roundings of at most |x - m| + ln S each."""
    s = (vocab / 256 + 64) * H32 + 2.0 ** -22 + 80 * H32
    return s, s + 4 * H32 * (logp.abs() + math.log(vocab) + 1)


def check_logprobs(lib, x, targets=None, top=0):
    n, vocab = x.shape
    op = lib.LogProbs(x, targets, top=top)
    op()
    d = x.double().cpu()
    logp = torch.log_softmax(d, -1)
    p = logp.exp()
    ds, tol = logprob_bound(d, torch.where(logp.isinf(), 0.0, logp), vocab)
    mean = (p * torch.where(p > 0, logp, 0.0).abs()).sum(-1)
    ent = -torch.special.xlogy(p, p).sum(-1)
    # H = ln S - T / S: S and T = sum e (x - m) carry ds each, T's terms a rounding more
    err = (op.entropy.double().cpu() - ent).abs()
    assert (err <= 4 * ds * (mean + math.log(vocab) + 1)).all(), float(err.max())
    if targets is not None:
        want, bound = logp.gather(1, targets.long().cpu()), tol.gather(1, targets.long().cpu())
        got = op.logprob.double().cpu()
        assert torch.equal(got.isinf(), want.isinf())
        assert ((got - want).abs()[~want.isinf()] <= bound[~want.isinf()]).all()
    if top:
        order = (d + 0.0).sort(dim=-1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(op.top_id.long().cpu(), order)
        want, bound, got = logp.gather(1, order), tol.gather(1, order), op.top_logprob.double().cpu()
        assert torch.equal(got.isinf(), want.isinf())
        assert ((got - want).abs()[~want.isinf()] <= bound[~want.isinf()]).all()
    return op


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 255, 1000, 4099, 32000, 128256, 151936])
def test_logprobs_vocabularies(lib, vocab, dtype):
    for n, top in ((1, 1), (3, 20), (5, 32)):
        x = rand(vocab + n, n, vocab, dtype=dtype, std=3.0)
        t = torch.randint(0, vocab, (n, 3), dtype=torch.int32, generator=torch.Generator().manual_seed(n)).cuda()
        check_logprobs(lib, x, t, min(top, vocab))


@pytest.mark.parametrize("n", [1, 2, 7, 40, 151, 200, 700])
def test_logprobs_row_counts(lib, n):
    x = rand(n, n, 9001, std=2.0)
    check_logprobs(lib, x, torch.arange(n, dtype=torch.int32, device="cuda")[:, None], 7)
    check_logprobs(lib, x, None, 0)
    check_logprobs(lib, x, None, 3)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("offset,stride", [(1, 5003), (3, 5001), (2, 5005), (7, 5999), (0, 5000)])
def test_logprobs_any_alignment(lib, dtype, offset, stride):
    flat = torch.full((6 * stride + offset,), math.nan, dtype=dtype, device="cuda")
    x = flat[offset:].as_strided((6, 5000), (stride, 1))
    x.copy_(rand(1, 6, 5000, dtype=dtype))
    check_logprobs(lib, x, torch.tensor([[0, 4999]] * 6, dtype=torch.int32, device="cuda"), 5)


def test_logprobs_ties(lib):
    x = torch.zeros(3, 5000, device="cuda")
    x[0, 4000:] = 1.0
    x[1, ::2] = -0.0                                  # equal to the zeros between them
    x[2, [7, 4999, 2500]] = 2.0
    check_logprobs(lib, x, None, 32)
    check_logprobs(lib, (rand(5, 4, 20000) * 4).round().half(), None, 20)
    check_logprobs(lib, torch.arange(30000., device="cuda").view(1, -1) / 1000, None, 32)      # rising: every token is a new best
    check_logprobs(lib, -torch.arange(30000., device="cuda").view(1, -1) / 1000, None, 32)


@pytest.mark.parametrize("vocab", [3, 40, 6000, 128256])
def test_logprobs_masks(lib, vocab):
    """-infinity takes a token out; the type's lowest value is a number."""
    x = rand(3, 5, vocab, std=2.0)
    x[0, 1:] = -math.inf                              # one token left
    x[1, ::2] = -math.inf
    x[2, 0] = torch.finfo(F32).min
    x[3] = torch.finfo(F32).min                       # all equal: uniform
    x[4, :vocab - 2] = torch.finfo(F32).min
    t = torch.tensor([[0, 1, 2]] * 5, dtype=torch.int32, device="cuda")
    op = check_logprobs(lib, x, t, 3)
    assert float(op.entropy[0]) == 0.0 and float(op.logprob[0, 0]) == 0.0
    h = x.half()                                      # the lowest F32 becomes -infinity
    h[3] = torch.finfo(F16).min
    check_logprobs(lib, h, t, 3)
    # nothing left at all
    x[:] = -math.inf
    op = lib.LogProbs(x, t, top=2)
    op()
    assert (op.logprob == -math.inf).all() and (op.top_logprob == -math.inf).all() and (op.entropy == 0).all()
    assert op.top_id.tolist() == [[0, 1]] * 5


def test_logprobs_not_numbers(lib):
    x = rand(4, 4, 10000)
    x[0, 77] = math.nan
    x[1, 9999] = math.inf
    x[2, :] = math.nan
    x[2, 5] = 1.0
    x[3, :5000] = -math.inf
    x[3, 100] = math.nan
    t = torch.tensor([[0], [1], [5], [6000]], dtype=torch.int32, device="cuda")
    op = lib.LogProbs(x, t, top=4)
    op()
    assert op.logprob.isnan().all() and op.entropy.isnan().all() and op.top_logprob.isnan().all()
    assert op.top_id[1, 0] == 9999 and op.top_id[2].tolist() == [5, -1, -1, -1]
    z = x.clone()
    z[0, 77] = -100.0
    assert op.top_id[0].tolist() == z[0].topk(4).indices.tolist()


def test_logprobs_targets(lib):
    x = rand(5, 2, 100)
    t = torch.tensor([[-1, 0, 99, 100], [-2, 5, -1, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    op = lib.LogProbs(x, t)
    op()
    got = op.logprob.cpu()
    assert got[0, 0] == 0 and got[1, 2] == 0 and got[0, 3].isnan() and got[1, 0].isnan() and got[1, 3].isnan()
    want = torch.log_softmax(x.double().cpu(), -1)
    assert abs(got[0, 2] - want[0, 99]) < 1e-5 and abs(got[1, 1] - want[1, 5]) < 1e-5
    many = torch.randint(0, 100, (2, 1500), dtype=torch.int32, device="cuda")
    check_logprobs(lib, x, many, 0)


def test_logprobs_rows_behind_32_bits(lib):
    stride = 1 << 26
    flat = torch.empty(33 * stride + 4096, dtype=F16, device="cuda")
    x = flat.as_strided((34, 4096), (stride, 1))
    x.copy_(rand(6, 34, 4096, dtype=F16))
    check_logprobs(lib, x, torch.arange(34, dtype=torch.int32, device="cuda")[:, None], 4)


# ------------------------------------------------------------------- together --
class Chain:
    """The three operators as a decoding step uses them: rotate and append,
    attend, then log probabilities of logits made from the attention's output."""

    def __init__(self, lib, lens, capacity, n_new=1, prefix=200, heads=(8, 2, 64), vocab=3001, seed=0):
        n_heads, n_kv, hd = heads
        self.lens, n = lens, len(lens) * n_new
        self.b = Batch(lib, [capacity] * len(lens), n_new, prefix, 16, n_kv, hd, seed, poison=False)
        self.b.lens_dev.copy_(torch.tensor(lens, dtype=torch.int32))
        self.qkv = rand(seed + 1, n, n_heads + 2 * n_kv, hd)
        self.q = torch.zeros(n, n_heads, hd, device="cuda")
        self.out = torch.zeros(n, n_heads, hd, device="cuda")
        self.pk, self.pv = (rand(seed + i, prefix, n_kv, hd, dtype=F16) for i in (2, 3))
        self.proj = rand(seed + 4, n_heads * hd, vocab, std=0.1)
        self.logits = torch.zeros(n, vocab, device="cuda")
        self.cs = lib.rope_table(prefix + capacity, hd, 10000.0)
        p = self.b.pages
        self.ops = [lib.KvAppend(p, self.qkv[:, :n_heads], self.qkv[:, n_heads:n_heads + n_kv], self.qkv[:, n_heads + n_kv:],
                                 self.cs, q_out=self.q),
                    lib.AttendBatch(p, self.q, self.out, self.pk, self.pv)]
        self.lp = lib.LogProbs(self.logits, top=5)

    def step(self):
        for op in self.ops:
            op()
        torch.matmul(self.out.view(len(self.out), -1), self.proj, out=self.logits)
        self.lp()

    def check(self):
        b = self.b
        b.lens = b.lens_dev.tolist()
        check_attend(b, self.q, self.out, self.pk, self.pv)
        for row, s, e in b.rows():
            y, mag = rotated(self.qkv[row, self.q.shape[1]:-b.k.shape[2]].double().cpu(), self.cs[b.prefix + e].double().cpu(), False)
            p, r = b.slot(s, e)
            assert ((b.k[p, r].double().cpu() - y).abs() <= 3 * H32 * mag * (1 + H16) + H16 * y.abs() + 2.0 ** -25).all()
        want = self.logits.double().log_softmax(-1).topk(5).values
        assert ((self.lp.top_logprob.double() - want).abs() <= 1e-5).all()      # ln 3001 = 8.0: 4 H32 * 20, ds = 2e-5 / 4
        assert b.pages.errors() == 0


def test_chain_over_steps(lib):
    c = Chain(lib, [1, 7, 0, 30], 48)
    for step in range(5):
        c.step()
        c.check()
        c.qkv.copy_(rand(100 + step, *c.qkv.shape))
        c.b.lens_dev.add_(1)


def test_chain_captured_and_replayed(lib):
    """One capture serves every later step: the lengths live on the device.
    Two graphs with their own workspaces replayed side by side on two streams."""
    chains = [Chain(lib, [1, 20, 3], 64, seed=10), Chain(lib, [5, 1, 40, 2, 2], 64, seed=20, prefix=900)]
    graphs, streams = [], []
    for c in chains:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            c.step()                                  # warm up (the matmul's own workspace)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            c.step()
        graphs.append(g)
        streams.append(st)
    for step in range(6):
        torch.cuda.synchronize()
        for c in chains:
            c.qkv.copy_(rand(200 + step, *c.qkv.shape))
            c.b.lens_dev.add_(1)
            c.out.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for c in chains:
            c.check()


def test_operators_run_on_the_stream_they_are_given(lib):
    """Work queued on the given stream is seen, whatever the current stream is."""
    c = Chain(lib, [9, 17], 32)
    st = torch.cuda.Stream()
    src = rand(9, *c.qkv.shape)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20000000)
        c.qkv.copy_(src)
    for op in c.ops:
        op(stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(c.qkv, src)
    b = c.b
    b.lens = b.lens_dev.tolist()
    check_attend(b, c.q, c.out, c.pk, c.pv)
    y, _ = rotated(src[0, :8].double().cpu(), c.cs[b.prefix + 8].double().cpu(), False)
    assert (c.q[0].double().cpu() - y).abs().max() < 1e-5


def test_empty_batches(lib):
    k = torch.zeros(2, 16, 2, 64, dtype=F16, device="cuda")
    pages = lib.PagedBatch(k, k.clone(), torch.zeros(0, 1, dtype=torch.int32, device="cuda"),
                           torch.zeros(0, dtype=torch.int32, device="cuda"))
    z = torch.zeros(0, 4, 64, device="cuda")
    lib.AttendBatch(pages, z, z.clone())()
    lib.KvAppend(pages, None, z[:, :2].contiguous(), z[:, :2].contiguous(), torch.zeros(4, 32, 2, device="cuda"))()
    lib.LogProbs(torch.zeros(0, 50, device="cuda"), top=3)()
    torch.cuda.synchronize()
    assert pages.errors() == 0


def test_calls_at_the_same_time(lib):
    """Two streams run attention (a prefix each, a workspace each) and log probabilities
    side by side; every run gives the bits of a run alone."""
    def make(seed):
        b = Batch(lib, [int(n) for n in np.random.RandomState(seed).randint(1, 200, 24)], 1, 3000, 16, 8, 64, seed=seed)
        pk, pv = (rand(seed + i, 3000, 8, 64, dtype=F16) for i in (3, 4))
        q, out = rand(seed + 5, 24, 32, 64), torch.zeros(24, 32, 64, device="cuda")
        return lib.AttendBatch(b.pages, q, out, pk, pv), out, lib.LogProbs(rand(seed + 6, 40, 30000), None, top=4)
    sides = [make(100), make(200)]
    alone = []
    for attend, out, lp in sides:
        attend()
        lp()
        alone.append([t.clone() for t in (out, lp.top_id, lp.top_logprob, lp.entropy)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sides]
    for _ in range(10):
        for s, (attend, out, lp) in zip(streams, sides):
            with torch.cuda.stream(s):
                out.zero_()
                attend()
                lp()
        torch.cuda.synchronize()
        for (attend, out, lp), want in zip(sides, alone):
            assert all(torch.equal(x, y) for x, y in zip((out, lp.top_id, lp.top_logprob, lp.entropy), want))


@pytest.mark.parametrize("top", [1, 8, 32])
def test_logprobs_long_rows_that_rise(lib, top):
    """Rows of many steps whose largest logits come last, first, or all over: the floor of
    a block rises at every rank, or never again.  Few rows take a cluster of blocks each,
    many one block: the same tokens, and values that are each within their bound."""
    n = 90000
    base = torch.linspace(-5, 5, n)
    shuffled = base[torch.randperm(n, generator=torch.Generator().manual_seed(1))]
    x = torch.stack([base, base.flip(0), shuffled, torch.zeros(n), base.round()]).cuda()
    few = check_logprobs(lib, x, None, top)
    many = lib.LogProbs(x.repeat(120, 1), None, top=top)
    many()
    assert torch.equal(many.top_id, few.top_id.repeat(120, 1))
    d = x.double().cpu()
    logp = torch.log_softmax(d, -1)
    bound = logprob_bound(d, logp, n)[1].gather(1, few.top_id.long().cpu()).repeat(120, 1)
    assert ((many.top_logprob - few.top_logprob.repeat(120, 1)).abs().double().cpu() <= 2 * bound).all()


@pytest.mark.parametrize("rows,vocab,dtype", [(3, 1000003, F32), (2, 1500001, F16), (160, 50021, F32), (300, 20011, F16)])
def test_logprobs_blocks_of_several_steps(lib, rows, vocab, dtype):
    """A cluster whose blocks walk several steps each, rows that start anywhere in a
    16-byte word, some tokens at -infinity, values that occur many times (F16)."""
    x = rand(21, rows, vocab, dtype=dtype, std=3.0)
    x[:, ::97] = -math.inf
    t = torch.randint(0, vocab, (rows, 2), generator=torch.Generator().manual_seed(5)).int().cuda()
    for top in (5, 32):
        check_logprobs(lib, x, t, top)


@pytest.mark.parametrize("prefix", [0, 70])
def test_attend_most_sequences(lib, prefix):
    run_attend(lib, (2, 1, 32), [s % 23 for s in range(4096)], 1, prefix, 8, F16, F32)


@pytest.mark.parametrize("q_dtype", [F32, F16])
@pytest.mark.parametrize("heads", [(8, 2, 64), (4, 4, 128), (8, 2, 32)])
@pytest.mark.parametrize("prefix,lens", [(5, [1, 1, 1]), (0, [2, 7, 12]), (3, [4, 9, 1]), (70, [1, 33, 18])])
def test_attend_f16_output_is_rounded_once(lib, prefix, lens, heads, q_dtype):
    """An F16 output is the F32 one's value rounded once: the probabilities keep 22 bits
    whatever the output's type, so its bound is the F32 output's and half a step of F16
    (with few keys one F16 per probability, 2^-11 of each term, would be far outside)."""
    n_heads, n_kv, hd = heads
    b = Batch(lib, lens, 1, prefix, 16, n_kv, hd, seed=prefix)
    q = rand(1, 3, n_heads, hd, dtype=q_dtype)
    pk, pv = rand(2, max(prefix, 1), n_kv, hd, dtype=F16), rand(3, max(prefix, 1), n_kv, hd, dtype=F16)
    out = torch.zeros(3, n_heads, hd, dtype=F16, device="cuda")
    lib.AttendBatch(b.pages, q, out, pk, pv)()
    for s, n in enumerate(lens):
        keys, values = torch.cat([pk[:prefix].double(), b.gather(b.k, s, n)]), torch.cat([pv[:prefix].double(), b.gather(b.v, s, n)])
        o, w, mag, far = attend_exact(q[s].double(), hd ** -0.5, keys, values, n_kv)
        tol = attend_bound(o, w, mag, far, values.abs().max(), keys.shape[0], hd, q_dtype, F32)
        err = (out[s].double() - o).abs()
        assert (err <= tol + H16 * (o.abs() + tol) + 2.0 ** -25).all(), (s, float((err / (tol + H16 * o.abs())).max()))


@pytest.mark.parametrize("rows,vocab", [(210, 60001), (3, 1000003), (600, 20000)])
def test_logprobs_masks_of_long_rows(lib, rows, vocab):
    """Tokens masked with a very low number, in rows of which every thread walks several
    steps: its first logits may all be masked ones, the later ones not."""
    low = torch.finfo(F32).min
    x = rand(31, rows, vocab, std=2.0)
    g = torch.Generator().manual_seed(32)
    for r in range(rows):
        kind = r % 6
        if kind == 0:
            x[r, :vocab - 200] = low
        elif kind == 1:
            x[r, :vocab * 9 // 10] = low
        elif kind == 2:
            x[r, (torch.rand(vocab, generator=g) < 0.98).cuda()] = low
        elif kind == 3:
            x[r, :vocab // 2] = -1e38
        elif kind == 4:
            x[r, 200:] = low
        else:
            x[r, :vocab - 1] = low
    check_logprobs(lib, x, torch.full((rows, 1), vocab - 1, dtype=torch.int32, device="cuda"), 3)
    # far from zero both ways: one token takes all
    x[:] = low
    x[:, vocab - 5] = 3e38
    op = lib.LogProbs(x, torch.full((rows, 1), vocab - 5, dtype=torch.int32, device="cuda"), top=1)
    op()
    assert (op.entropy == 0).all() and (op.logprob == 0).all() and (op.top_id == vocab - 5).all()


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("vocab", [64, 500, 1000, 20000])
@pytest.mark.parametrize("top", [8, 25, 32])
def test_logprobs_alternatives_among_nans(lib, top, vocab, dtype):
    """top_id counts the logits that are numbers, wherever the NaNs lie: -1 only where there
    are fewer than `top` of them."""
    x = rand(vocab + top, 24, vocab, dtype=dtype, std=3.0)
    g = torch.Generator().manual_seed(top)
    for r in range(24):
        x[r, (torch.rand(vocab, generator=g) < (r % 8 + 1) / 10).cuda()] = math.nan
    x[22] = math.nan
    x[22, :20:2] = rand(5, 10, dtype=dtype)
    # a lane's 16 logits of a step: one large, NaNs behind it, then small ones
    x[23] = -5.0
    x[23, :vocab // 2:4], x[23, 1:vocab // 2:4] = 10.0, math.nan
    op = lib.LogProbs(x, None, top=top)
    op()
    assert op.entropy.isnan().all() and op.top_logprob.isnan().all()
    for r, row in enumerate(x.double().cpu()):
        order = torch.where(row.isnan(), -math.inf, row).sort(descending=True, stable=True).indices[:top]
        want = [int(i) if not row[i].isnan() else -1 for i in order]
        assert op.top_id[r].tolist() == want, r


@pytest.mark.parametrize("by_number", [False, True])
def test_operator_dropped_while_its_run_is_queued(lib, by_number):
    """An operator made on one stream, run on another and dropped before the run has begun:
    its workspace is not given to the first stream's next tensors meanwhile."""
    b = Batch(lib, [40, 7, 90], 1, 300, 16, 2, 64)
    q, pk, pv = rand(1, 3, 8, 64), rand(2, 300, 2, 64, dtype=F16), rand(3, 300, 2, 64, dtype=F16)
    out = torch.zeros(3, 8, 64, device="cuda")
    side, queued = torch.cuda.Stream(), 0
    lib.AttendBatch(b.pages, q, out, pk, pv)()         # (the first call loads the kernels)
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        op = lib.AttendBatch(b.pages, q, out, pk, pv)
        size, at = op.workspace.numel(), op.workspace.data_ptr()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100000000)
            if not by_number:
                op()
        if by_number:
            op(stream=side.cuda_stream)
        done = side.record_event()
        del op
        junk = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
        if not done.query():
            queued += 1
            assert all(t.data_ptr() != at for t in junk)
        side.synchronize()
        check_attend(b, q, out, pk, pv)
    assert queued > 0


@pytest.mark.parametrize("prefix", [1, 64, 65, 130])
@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_attend_many_short_units(lib, prefix, types):
    """Blocks of the prefix kernel that walk several (row tile, kv head) units of one, two
    or three 64-key tiles each; every run gives the same bits."""
    b = Batch(lib, [1 + s % 3 for s in range(2500)], 1, prefix, 16, 32, 64, poison=False)
    q = rand(1, 2500, 32, 64, dtype=types[0])
    pk, pv = rand(2, prefix, 32, 64, dtype=F16), rand(3, prefix, 32, 64, dtype=F16)
    out = torch.zeros(2500, 32, 64, dtype=types[1], device="cuda")
    op = lib.AttendBatch(b.pages, q, out, pk, pv)
    op()
    first = out.clone()
    b.lens = [n if s % 97 < 2 else 0 for s, n in enumerate(b.lens)]           # rows that are looked at
    check_attend(b, q, out, pk, pv)
    for _ in range(20):
        out.zero_()
        op()
        assert torch.equal(out, first)
    assert b.pages.errors() == 0


@pytest.mark.parametrize("out_dtype", [F32, F16])
@pytest.mark.parametrize("heads,lens,n_new", [((8, 2, 64), [40, 7, 1], 1), ((12, 2, 64), [40, 7, 5], 5), ((4, 4, 128), [3, 70], 2)])
@pytest.mark.parametrize("size", [1e7, 1e30, 3e38 / 256, 1e-9, 1e-36])
def test_attend_f32_queries_of_any_magnitude(lib, size, heads, lens, n_new, out_dtype):
    """F32 queries far above F16's largest number and far below its smallest, rows of
    different magnitudes in one tile: the bound is the one of queries near 1."""
    n_heads, n_kv, hd = heads
    b = Batch(lib, lens, n_new, 130, 16, n_kv, hd)
    q = rand(1, len(lens) * n_new, n_heads, hd) * size
    q[:, 1::2] *= 2.0 ** -20                          # flat scores next to pointed ones
    q[:, 0, ::3] *= 2.0 ** -12                        # small elements beside large ones
    pk, pv = rand(2, 130, n_kv, hd, dtype=F16), rand(3, 130, n_kv, hd, dtype=F16)
    out = torch.zeros(*q.shape, dtype=out_dtype, device="cuda")
    scale = float(np.float32(hd ** -0.5 / size))
    lib.AttendBatch(b.pages, q, out, pk, pv, scale=scale)()
    check_attend(b, q, out, pk, pv, scale)
    assert b.pages.errors() == 0


def test_attend_f32_queries_not_finite(lib):
    """A query that is not finite gives NaN in its own row and head, nowhere else; one of
    zeros the mean of the values."""
    b = Batch(lib, [20, 5], 1, 70, 16, 2, 64)
    q = rand(1, 2, 4, 64)
    q[0, 1, 3], q[1, 2, 63] = math.inf, math.nan
    q[1, 3] = 0.0
    pk, pv = rand(2, 70, 2, 64, dtype=F16), rand(3, 70, 2, 64, dtype=F16)
    out = torch.zeros(2, 4, 64, device="cuda")
    lib.AttendBatch(b.pages, q, out, pk, pv)()
    assert out[0, 1].isnan().all() and out[1, 2].isnan().all()
    q[0, 1] = q[1, 2] = 1.0
    again = torch.zeros_like(out)
    lib.AttendBatch(b.pages, q, again, pk, pv)()
    check_attend(b, q, again, pk, pv)
    for row, h in ((0, 0), (0, 2), (0, 3), (1, 0), (1, 1), (1, 3)):
        assert torch.equal(out[row, h], again[row, h])


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("q_dtype,q_size,k_size", [(F32, 1e30, 1), (F32, 1e9, 1), (F16, 30000, 4000), (F32, 2e3, 4000)])
@pytest.mark.parametrize("prefix,lens", [(90, [1]), (0, [70]), (700, [40])])
def test_attend_scores_far_from_zero(lib, prefix, lens, q_dtype, q_size, k_size, sign):
    """Scores of 10^8 to 10^32, all on one side of zero: the largest takes all."""
    b = Batch(lib, lens, 1, prefix, 16, 1, 64)
    q = torch.full((1, 2, 64), float(q_size), dtype=q_dtype, device="cuda")
    pk, pv = (rand(2, max(prefix, 1), 1, 64).abs() + 0.1).mul(sign * k_size).half(), rand(3, max(prefix, 1), 1, 64, dtype=F16)
    b.k.copy_((b.k.abs() + 0.1) * sign * k_size)
    out = torch.zeros(1, 2, 64, device="cuda")
    lib.AttendBatch(b.pages, q, out, pk, pv)()
    keys, values = torch.cat([pk[:prefix].double(), b.gather(b.k, 0, lens[0])]), torch.cat([pv[:prefix].double(), b.gather(b.v, 0, lens[0])])
    total = keys[:, 0].sum(-1)
    best = total.argmax()
    # the second best is far behind, whatever 64 additions of F32 leave of the scores (2^-17)
    assert total.sort().values[-2] < total[best] - total[best].abs() * 2.0 ** -16
    # one probability of 1 as two F16 parts, one division: 2^-22 and a few roundings
    assert ((out[0].double() - values[best, 0]).abs() <= 2.0 ** -20 * values[best, 0].abs()).all()


def test_calls_of_several_threads(lib):
    """Host threads that make their first calls together, each on a stream of its own:
    every one gets its own results."""
    import threading
    def make(seed):
        b = Batch(lib, [40, 3, 100], 1, 130, 16, 2, 64, seed=seed)
        return b, rand(seed + 5, 3, 4, 64), rand(seed + 6, 130, 2, 64, dtype=F16), rand(seed + 7, 130, 2, 64, dtype=F16), torch.zeros(3, 4, 64, device="cuda")
    sides, errors = [make(10 * i) for i in range(6)], []
    gate = threading.Barrier(6)
    torch.cuda.synchronize()

    def work(side):
        try:
            b, q, pk, pv, out = side
            with torch.cuda.stream(torch.cuda.Stream()):
                op = lib.AttendBatch(b.pages, q, out, pk, pv)
                lp = lib.LogProbs(q.view(3, 256), top=3)
                gate.wait()
                for _ in range(20):
                    op()
                    lp()
                torch.cuda.current_stream().synchronize()
                assert torch.equal(lp.top_id.long(), q.view(3, 256).topk(3).indices)
        except Exception as e:                         # (an exception of a thread would otherwise be lost)
            errors.append(e)
            gate.abort()
    threads = [threading.Thread(target=work, args=(s,)) for s in sides]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for b, q, pk, pv, out in sides:
        check_attend(b, q, out, pk, pv)


@pytest.mark.parametrize("heads,n_seqs,prefix", [((16, 16, 128), 700, 150), ((16, 16, 128), 700, 200), ((32, 8, 64), 600, 330), ((8, 8, 64), 2000, 190)])
@pytest.mark.parametrize("q_dtype", [F16, F32])
def test_attend_units_behind_one_another(lib, heads, n_seqs, prefix, q_dtype):
    """Blocks of the prefix kernel that go from unit to unit, with even and odd numbers of
    tiles: the queries of the next unit must not take their place before both groups' last
    scores have read the present ones.  Every run gives the same bits, and the right ones."""
    n_heads, n_kv, hd = heads
    b = Batch(lib, [1] * n_seqs, 1, prefix, 16, n_kv, hd, poison=False)
    q = rand(1, n_seqs, n_heads, hd, dtype=q_dtype)
    pk, pv = rand(2, prefix, n_kv, hd, dtype=F16), rand(3, prefix, n_kv, hd, dtype=F16)
    out = torch.zeros(n_seqs, n_heads, hd, dtype=F16, device="cuda")
    op = lib.AttendBatch(b.pages, q, out, pk, pv)
    op()
    first = out.clone()
    # all rows against 64 bits, one key of its own each
    own_k, own_v = (t[b.table[:, 0].long(), 0].double() for t in (b.k, b.v))
    qd = q.double().view(n_seqs, n_kv, n_heads // n_kv, hd)
    s = torch.cat([torch.einsum("nghd,tgd->nght", qd, pk.double()), (qd * own_k[:, :, None]).sum(-1, keepdim=True)], -1) * hd ** -0.5
    p = s.softmax(-1)
    o = torch.einsum("nght,tgd->nghd", p[..., :-1], pv.double()) + p[..., -1:] * own_v[:, :, None]
    o = o.reshape(n_seqs, n_heads, hd)
    values = torch.cat([pv.double().flatten(), own_v.flatten()]).abs().max()
    w = torch.einsum("nght,tgd->nghd", p[..., :-1], pv.double().abs()) + p[..., -1:] * own_v[:, :, None].abs()
    mag = torch.cat([torch.einsum("nghd,tgd->nght", qd.abs(), pk.double().abs()), (qd * own_k[:, :, None]).abs().sum(-1, keepdim=True)], -1).amax(-1) * hd ** -0.5
    far = s.amax(-1) - s.amin(-1)
    tol = attend_bound(o, w.reshape(o.shape), mag.reshape(n_seqs, n_heads, 1), far.reshape(n_seqs, n_heads, 1), values, prefix + 1, hd, q_dtype, F16)
    assert ((out.double() - o).abs() <= tol).all()
    for _ in range(100):
        op()
        assert torch.equal(out, first)


@pytest.mark.parametrize("by_number", [False, True])
def test_operator_made_on_a_busy_stream(lib, by_number):
    """An operator's own tensors lie where tensors of its stream's queued work lay; its first
    run on another stream waits for that work.  (Its inputs are ready: the user saw to them.)"""
    b = Batch(lib, [40, 7, 90], 1, 300, 16, 2, 64)
    q, pk, pv = rand(1, 3, 8, 64), rand(2, 300, 2, 64, dtype=F16), rand(3, 300, 2, 64, dtype=F16)
    logits = rand(4, 40, 5000)
    out = torch.zeros(3, 8, 64, device="cuda")
    size = lib.AttendBatch(b.pages, q, out, pk, pv).workspace.numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(20000000)
        for n in (size, 40 * 3 * 4, 40 * 4):           # queued: what will have written where the operators' tensors lie
            junk = torch.empty(n, dtype=torch.uint8, device="cuda")
            junk.fill_(0x7F)
            del junk
        pages = lib.PagedBatch(b.k, b.v, b.table, b.lens_dev, prefix_len=300)
        op, lp = lib.AttendBatch(pages, q, out, pk, pv), lib.LogProbs(logits, top=3)
        if by_number:
            op(stream=side.cuda_stream)
            lp(stream=side.cuda_stream)
        else:
            with torch.cuda.stream(side):
                op()
                lp()
        side.synchronize()
        torch.cuda.synchronize()
        check_attend(b, q, out, pk, pv)
        assert torch.equal(lp.top_id.long(), logits.topk(3).indices) and pages.errors() == 0


def test_errors_wait_for_every_stream(lib):
    """A bad page met on a stream that is not the current one is seen."""
    b = Batch(lib, [20], 1, 0, 16, 1, 64, poison=False)
    b.table[0, 1] = -1
    q, out = rand(1, 1, 2, 64), torch.zeros(1, 2, 64, device="cuda")
    op = lib.AttendBatch(b.pages, q, out)
    op()
    assert b.pages.errors() == lib.LLM_PAGES_BAD_PAGE
    b.pages.err.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100000000)
        op()
    assert b.pages.errors() == lib.LLM_PAGES_BAD_PAGE
