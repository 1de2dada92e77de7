"""llm_logits_adjust on the GPU against its formula in 64 bits.

Tolerance, in F32 roundings (H32 each, counted before the first run): the quotient or product of the
repetition penalty one, of |y / rho|; frequency times count one, plus presence one more, of |f c + p|
together two; the difference one of the result; the bias one of its result; then one rounding to the output
type (H16, or 2^-25 where that is subnormal)."""
import math

import numpy as np
import pytest
import torch

from test_batch_ops_gpu import F16, F32, H16, H32, lib, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def make(rows, vocab, dtype, history=0, biases=0, masks=0, seed=0, allowed=0.3):
    r = np.random.RandomState(seed)
    x = {"logits": rand(seed + 1, rows, vocab, dtype=dtype, std=3.0)}
    if history:
        few = r.randint(0, vocab, max(1, history // 3))
        x["history"] = few[r.randint(0, len(few), (rows, history))].astype(np.int32)
        x["history"][r.rand(rows, history) < 0.05] = -1
        x["history"][r.rand(rows, history) < 0.05] = vocab                      # no tokens
        x["history_lens"] = r.randint(0, history + 1, rows).astype(np.int32)
        x["history_lens"][0] = history
        for name, a, b in (("repetition", 0.8, 1.6), ("frequency", -0.2, 0.5), ("presence", 0.0, 0.9)):
            x[name] = r.uniform(a, b, rows).astype(np.float32)
    if biases:
        x["bias_ids"] = r.randint(-1, vocab + 1, (rows, biases)).astype(np.int32)
        x["bias_ids"][:, -1] = x["bias_ids"][:, 0]                              # the same token twice
        x["bias"] = (4 * r.randn(rows, biases)).astype(np.float32)
    if masks:
        x["masks"] = np.packbits(r.rand(masks, -(-vocab // 32) * 32) < allowed, axis=1, bitorder="little").view(np.int32)
        x["mask_of"] = r.randint(-1, masks + 1, rows).astype(np.int32)
    return {k: torch.from_numpy(t).cuda() if isinstance(t, np.ndarray) else t for k, t in x.items()}


def exact(x, window):
    """The adjusted logits in 64 bits, and the bound before the last rounding."""
    a = {k: t.cpu().numpy() for k, t in x.items()}
    y = a["logits"].astype(np.float64)
    tol, (rows, vocab) = np.zeros_like(y), y.shape
    for r in range(rows):
        if "history" in a:
            n = min(max(int(a["history_lens"][r]), 0), a["history"].shape[1])
            t = a["history"][r, max(0, n - window) if window else 0:n]
            ids, c = np.unique(t[(t >= 0) & (t < vocab)], return_counts=True)
            rho, f, p = (float(a[k][r]) if k in a else z for k, z in (("repetition", 1.0), ("frequency", 0.0), ("presence", 0.0)))
            z = np.where(y[r, ids] > 0, y[r, ids] / rho, y[r, ids] * rho)
            y[r, ids] = z - (f * c + p)
            tol[r, ids] = H32 * (np.abs(z) + 2 * (np.abs(f * c) + abs(p)) + np.abs(y[r, ids])) * 1.001
        if "bias_ids" in a:
            last = {int(t): float(b) for t, b in zip(a["bias_ids"][r], a["bias"][r]) if 0 <= t < vocab}
            for t, b in last.items():
                y[r, t] += b
                tol[r, t] += H32 * (abs(y[r, t]) + tol[r, t])
        if "masks" in a:
            k = int(a["mask_of"][r]) if "mask_of" in a else r
            if 0 <= k < len(a["masks"]):
                bits = np.unpackbits(np.ascontiguousarray(a["masks"][k]).view(np.uint8), bitorder="little")[:vocab]
                y[r, bits == 0], tol[r, bits == 0] = -math.inf, 0
    return y, tol


def check(out, want, tol):
    got = out.double().cpu().numpy()
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    e = np.abs(got[~inf] - want[~inf])
    t = tol[~inf]
    t = t + (H16 * (np.abs(want[~inf]) + t) + 2.0 ** -25 if out.dtype == F16 else 0)
    assert (e <= t).all(), (e.max(), int((e > t).sum()))


def run(lib, x, out_dtype, window=0):  # noqa: F811
    want, tol = exact(x, window)
    out = torch.full(x["logits"].shape, 7.0, dtype=out_dtype, device="cuda")
    lib.AdjustLogits(**{**x, "out": out}, window=window)()
    check(out, want, tol)
    # in place: the same values
    if x["logits"].dtype == out_dtype:
        y = x["logits"].clone()
        lib.AdjustLogits(**{**x, "logits": y}, window=window)()
        assert torch.equal(y, out)
    return out


TYPES = [(F32, F32), (F32, F16), (F16, F16), (F16, F32)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 31, 32, 33, 127, 128, 129, 1000, 4099, 32000, 151936])
def test_vocabularies(lib, vocab, types):  # noqa: F811
    run(lib, make(3, vocab, types[0], 200, 20, 2, seed=vocab), types[1])


@pytest.mark.parametrize("what", [dict(history=50), dict(biases=7), dict(masks=3), dict(history=50, biases=7), dict(history=9, masks=1),
                                  dict(biases=1, masks=2), dict()])
@pytest.mark.parametrize("types", TYPES)
def test_parts(lib, what, types):  # noqa: F811
    run(lib, make(5, 5003, types[0], **what), types[1])


@pytest.mark.parametrize("rows", [1, 2, 9, 40, 151, 160, 400])
def test_row_counts(lib, rows):  # noqa: F811
    run(lib, make(rows, 20011, F32, 300, 30, 4, seed=rows), F32)
    run(lib, make(rows, 20016, F16, 300, 30, 4, seed=rows), F16)


@pytest.mark.parametrize("window", [1, 5, 64, 299, 300, 301, 10 ** 6])
def test_windows(lib, window):  # noqa: F811
    run(lib, make(6, 500, F32, 300), F32, window)


def test_lengths_beyond_the_history(lib):  # noqa: F811
    x = make(5, 300, F32, 40)
    x["history_lens"][:] = torch.tensor([-3, 0, 1, 40, 400], dtype=torch.int32)
    run(lib, x, F32)
    run(lib, x, F32, 7)


def test_long_history_of_one_token(lib):  # noqa: F811
    """A count beyond 16 bits, and penalties left out."""
    x = make(2, 40000, F32, 150000)
    x["history"][1] = 39999
    x["history_lens"][1] = 150000
    run(lib, x, F32)
    for name in ("repetition", "presence", "frequency"):
        del x[name]
        run(lib, x, F32, 100)


@pytest.mark.parametrize("vocab", [300007, 1000003])
def test_vocabularies_of_several_tiles(lib, vocab):  # noqa: F811
    run(lib, make(2, vocab, F32, 3000, 500, 1), F32)
    run(lib, make(2, vocab, F16, 3000), F16)


@pytest.mark.parametrize("offset,stride", [(1, 5003), (2, 5001), (3, 5999), (0, 5002), (4, 5008)])
@pytest.mark.parametrize("types", TYPES)
def test_any_alignment(lib, offset, stride, types):  # noqa: F811
    """Rows within wider ones: nothing behind or before them is touched."""
    x = make(4, 5000, types[0], 60, 9, 2)
    a = torch.full((4 * stride + 16,), 5.0, dtype=types[0], device="cuda")
    b = torch.full((4 * 5011 + 16,), 5.0, dtype=types[1], device="cuda")
    inner = a[offset:offset + 4 * stride].view(4, stride)[:, :5000]
    out = b[3:3 + 4 * 5011].view(4, 5011)[:, :5000]
    inner.copy_(x["logits"])
    want, tol = exact(x, 0)
    lib.AdjustLogits(**{**x, "logits": inner, "out": out})()
    check(out, want, tol)
    assert torch.equal(inner, x["logits"])
    rest = torch.ones_like(b, dtype=torch.bool)
    rest[3:3 + 4 * 5011].view(4, 5011)[:, :5000] = False
    assert (b[rest] == 5.0).all()
    lib.AdjustLogits(**{**x, "logits": inner})()
    assert torch.equal(inner.double(), out.double()) or types[0] != types[1]
    rest = torch.ones_like(a, dtype=torch.bool)
    rest[offset:offset + 4 * stride].view(4, stride)[:, :5000] = False
    assert (a[rest] == 5.0).all()


def test_values_that_are_not_finite(lib):  # noqa: F811
    x = make(1, 64, F32, 0)
    x["logits"][0, :6] = torch.tensor([math.inf, -math.inf, math.nan, 1.0, -1.0, 0.0])
    x["history"] = torch.tensor([[0, 1, 2, 3, 4, 5, 5]], dtype=torch.int32, device="cuda")
    x["history_lens"] = torch.tensor([7], dtype=torch.int32, device="cuda")
    for name, v in (("repetition", 2.0), ("frequency", 0.25), ("presence", 1.0)):
        x[name] = torch.tensor([v], device="cuda")
    out = torch.empty(1, 64, device="cuda")
    lib.AdjustLogits(**{**x, "out": out})()
    assert out[0, 0] == math.inf and out[0, 1] == -math.inf and out[0, 2].isnan()
    assert out[0, 3:6].tolist() == [0.5 - 1.25, -2.0 - 1.25, -1.5]
    assert torch.equal(out[0, 6:], x["logits"][0, 6:])
    x["masks"] = torch.tensor([[~7, -1]], dtype=torch.int32, device="cuda")        # bits 0 to 2 banned, NaN too
    lib.AdjustLogits(**{**x, "out": out})()
    assert (out[0, :3] == -math.inf).all() and out[0, 3] == -0.75
    # a row that the mask leaves nothing of; its log probabilities
    x["masks"][:] = 0
    lib.AdjustLogits(**{**x, "out": out})()
    assert (out == -math.inf).all()


def test_masks_by_row_and_by_number(lib):  # noqa: F811
    x = make(4, 700, F32, 0, 0, 4)
    del x["mask_of"]
    run(lib, x, F32)
    wide = torch.zeros(4, 40, dtype=torch.int32, device="cuda")
    wide[:, 3:3 + x["masks"].shape[1]] = x["masks"]
    out, again = torch.empty(4, 700, device="cuda"), torch.empty(4, 700, device="cuda")
    lib.AdjustLogits(x["logits"], out, masks=x["masks"])()
    lib.AdjustLogits(x["logits"], again, masks=wide[:, 3:3 + x["masks"].shape[1]])()
    assert torch.equal(out, again)


def test_rows_behind_32_bits(lib):  # noqa: F811
    n, vocab = 17000, 151936                                   # 2.58e9 elements
    x = torch.empty(n, vocab, dtype=F16, device="cuda")
    x[-1], x[0] = rand(1, vocab, dtype=F16), 1.0
    ids = torch.full((n, 1), 7, dtype=torch.int32, device="cuda")
    before = x[-1].clone()
    lib.AdjustLogits(x, bias_ids=ids, bias=torch.full((n, 1), 2.0, device="cuda"))()
    before[7] += 2.0
    assert torch.equal(x[-1], before) and x[0, 7] == 3.0 and x[0, 8] == 1.0


def test_binding_refuses_what_does_not_belong_together(lib):  # noqa: F811
    x = make(2, 100, F32, 10, 2, 1)
    for drop in (("history",), ("history_lens",), ("bias",), ("bias_ids",), ("masks",)):
        with pytest.raises((ValueError, TypeError)):
            lib.AdjustLogits(**{k: t for k, t in x.items() if k not in drop})
    with pytest.raises(ValueError, match="words"):
        lib.AdjustLogits(x["logits"], masks=x["masks"][:, :3].contiguous(), mask_of=x["mask_of"])
    with pytest.raises(ValueError, match="masks for"):
        lib.AdjustLogits(x["logits"], masks=x["masks"])
    with pytest.raises(lib.LlmError):
        lib.AdjustLogits(x["logits"], window=-1)()
    with pytest.raises(lib.LlmError):                          # the same memory as another type
        lib.AdjustLogits(x["logits"], x["logits"].view(F16)[:, :100])()


@pytest.mark.parametrize("biases,window", [(4094, 0), (4096, 0), (6000, 7)])
@pytest.mark.parametrize("types", [(F32, F32), (F16, F16)])
def test_many_biases_beside_a_history(lib, biases, window, types):  # noqa: F811
    """An entry and a count share a word up to 4095 entries; tokens of both lists, of one, and entries given twice."""
    x = make(3, 9001, types[0], 700, biases, 1, seed=biases)
    x["bias_ids"][:, ::3] = x["bias_ids"][:, 1::3][:, :x["bias_ids"][:, ::3].shape[1]] if biases % 3 == 0 else x["bias_ids"][:, ::3]
    x["history"][:, ::5] = 17                                  # counted, and biased by the entries set here
    x["bias_ids"][:, 5], x["bias_ids"][:, 9] = 17, 17
    run(lib, x, types[1], window)


def test_counts_that_fill_their_bits(lib):  # noqa: F811
    """More than 2^20 tokens counted, with biases."""
    n = (1 << 20) + 5
    x = make(1, 5000, F32, 8, 30)
    x["history"] = torch.full((1, n), 4, dtype=torch.int32, device="cuda")
    x["history"][0, :100] = torch.arange(100, dtype=torch.int32, device="cuda")
    x["history_lens"] = torch.tensor([n], dtype=torch.int32, device="cuda")
    x["bias_ids"][0, 3], x["bias_ids"][0, 4] = 4, 50
    run(lib, x, F32)


def test_lists_of_as_many_entries_as_31_bits_count(lib):  # noqa: F811
    """Entries up to the last places that an int32 names, among others that are no tokens: what the same tokens give in
    short lists."""
    n = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory for lists of 2^31 entries")
    places = [0, 1, 511, 512, 2047, 2048, n - 4096, n - 2049, n - 2048, n - 513, n - 512, n - 2, n - 1]
    tokens = torch.tensor([[17, 4, 17, 4999, 0, 17, 4, 250, 17, 9, 4, 250, 17]], dtype=torch.int32, device="cuda")
    x = make(1, 5000, F32, 1)
    x["history"], x["history_lens"] = tokens, torch.tensor([len(places)], dtype=torch.int32, device="cuda")
    many = torch.full((1, n), -1, dtype=torch.int32, device="cuda")
    many[0, places] = tokens[0]
    y = {**x, "history": many, "history_lens": torch.tensor([n], dtype=torch.int32, device="cuda")}
    out = torch.empty(1, 5000, device="cuda")
    lib.AdjustLogits(**{**y, "out": out})()
    check(out, *exact(x, 0))
    lib.AdjustLogits(**{**y, "out": out}, window=n - 2)()                           # without the first two
    x["history"], x["history_lens"] = tokens[:, 2:], x["history_lens"] - 2
    check(out, *exact(x, 0))
    # biases (the last entry of a token counts), alone and beside that history
    values = torch.zeros(1, n, device="cuda")
    b = rand(5, 1, len(places))
    values[0, places] = b[0]
    short, long = {"bias_ids": tokens, "bias": b}, {"bias_ids": many, "bias": values}
    lib.AdjustLogits(x["logits"], out, **long)()
    check(out, *exact({"logits": x["logits"], **short}, 0))
    lib.AdjustLogits(**{**y, **long, "out": out}, window=n - 2)()
    check(out, *exact({**x, **short}, 0))
