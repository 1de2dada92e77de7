"""llm_decode_batch_q4: whole steps on pages of 4-bit values against a forward pass in 64 bits
("What a Llama model computes, and why" §2) that takes K and V from the pages as they stand, the
values that the numbers stand for: a number that lies on either side of a border is then
the same on both sides.  That the pages hold what they should is checked apart, within half a
step of the numbers.  Logits are held to the batched step's tolerance."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from harness import TOL, check_logits
from test_decode_batch_gpu import config, lib, put, scatter, token  # noqa: F401
from test_q4_pages_gpu import H16, decode, page_bytes, values

pytestmark = pytest.mark.gpu


def matrix(cfg, w, rows, cols):
    """A weight matrix in 64 bits from its GGUF layout."""
    if cfg.wtype == synth.F16:
        return np.ascontiguousarray(w).view(np.float16).reshape(rows, cols).astype(np.float64)
    b = np.ascontiguousarray(w).view(np.uint8).reshape(rows, cols // 32, 34)
    d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(np.float64)
    return (d * b[..., 2:].view(np.int8)).reshape(rows, cols)


class Model:
    def __init__(self, cfg, W):
        self.cfg, q, kv = cfg, cfg.q_dim, cfg.kv_dim
        shapes = {"wq": (q, cfg.dim), "wk": (kv, cfg.dim), "wv": (kv, cfg.dim), "wo": (cfg.dim, q), "w_gate": (cfg.ffn_dim, cfg.dim),
                  "w_up": (cfg.ffn_dim, cfg.dim), "w_down": (cfg.dim, cfg.ffn_dim)}
        self.embd = matrix(cfg, W.tok_embd, cfg.vocab, cfg.dim)
        self.out = self.embd if W.output is None else matrix(cfg, W.output, cfg.vocab, cfg.dim)
        self.out_norm = W.output_norm.astype(np.float64)
        self.layers = [{**{k: matrix(cfg, L[k], *s) for k, s in shapes.items()},
                        **{k: None if L.get(k) is None else L[k].astype(np.float64) for k in ("attn_norm", "ffn_norm", "bq", "bk", "bv")}}
                       for L in W.layers]

    def norm(self, x, g):
        return x / np.sqrt((x * x).mean() + self.cfg.eps) * g

    def rope(self, x, pos):
        c, half = self.cfg, self.cfg.head_dim // 2
        a = pos * c.rope_base ** (-2.0 * np.arange(half) / c.head_dim)
        x, y = x.reshape(-1, c.head_dim), np.empty((x.size // c.head_dim, c.head_dim))
        i, j = (np.arange(half), np.arange(half) + half) if c.rope_neox else (2 * np.arange(half), 2 * np.arange(half) + 1)
        y[:, i], y[:, j] = x[:, i] * np.cos(a) - x[:, j] * np.sin(a), x[:, i] * np.sin(a) + x[:, j] * np.cos(a)
        return y

    def row(self, tok, pos, kv):
        """Logits of one row and every layer's own k and v; kv(layer): keys and values [rows seen, n_kv, hd], the row's own the last."""
        c, own = self.cfg, []
        x = self.embd[tok].copy()
        for l, L in enumerate(self.layers):
            h = self.norm(x, L["attn_norm"])
            q, k, v = (L[w] @ h + (0 if L[b] is None else L[b]) for w, b in (("wq", "bq"), ("wk", "bk"), ("wv", "bv")))
            q, own_k = self.rope(q, pos).reshape(c.n_kv_heads, -1, c.head_dim), self.rope(k, pos)
            own.append((own_k, v.reshape(-1, c.head_dim)))
            keys, vals = kv(l)
            s = np.einsum("ghd,tgd->ght", q, keys) / np.sqrt(c.head_dim)
            p = np.exp(s - s.max(-1, keepdims=True))
            o = np.einsum("ght,tgd->ghd", p / p.sum(-1, keepdims=True), vals)
            x = x + L["wo"] @ o.reshape(-1)
            h = self.norm(x, L["ffn_norm"])
            z = L["w_gate"] @ h
            x = x + L["w_down"] @ (z / (1 + np.exp(-z)) * (L["w_up"] @ h))
        return self.out @ self.norm(x, self.out_norm), own


def layer_pages(bd, cfg, l):
    """Numbers, pairs and values of layer l's K and V pages."""
    n, page = bd.struct.n_pages, bd.struct.page_size
    flat = bd.pages.view(cfg.n_layers, 2, n, page_bytes(page, cfg.n_kv_heads, cfg.head_dim))
    return [(nd, values(*nd)) for nd in (decode(flat[l, i], page, cfg.n_kv_heads, cfg.head_dim) for i in (0, 1))]


def check_steps(lib, cfg, prefix, n_new, steps, page=16):  # noqa: F811
    W = synth.make_weights(cfg)
    model, dec = Model(cfg, W), lib.Decoder(cfg, W)
    shared = [(np.zeros((0, cfg.n_kv_heads, cfg.head_dim)),) * 2] * cfg.n_layers
    if prefix:
        lib.llm_prefill(dec.h, synth.prompt(cfg, prefix), 0)
        shared = [tuple(t[:prefix].cpu().numpy().view(np.float16).astype(np.float64).reshape(prefix, cfg.n_kv_heads, cfg.head_dim)
                        for t in dec.kv_tensors(l)) for l in range(cfg.n_layers)]
    n_seqs = len(steps[0])
    bd = lib.BatchDecoder(dec, n_seqs, max(max(s) for s in steps), prefix, n_new, page, q4=True)
    scatter(bd, 5)
    table = bd.page_table.cpu().numpy()
    for lens in steps:
        put(bd, cfg, lens)
        bd.step()
        lib.llm_sync(dec.h)
        got, pages = bd.logits.cpu().numpy(), [layer_pages(bd, cfg, l) for l in range(cfg.n_layers)]
        for s, n in enumerate(lens):
            for i in range(n_new):
                e = n - n_new + i
                if e < 0:
                    continue
                at = [(table[s, j // page], j % page) for j in range(e + 1)]
                rows = lambda l, which: np.concatenate([shared[l][which], np.stack([pages[l][which][1][p, r] for p, r in at]).astype(np.float64)])  # noqa: E731
                ref, own = model.row(token(cfg, s, e), prefix + e, lambda l: (rows(l, 0), rows(l, 1)))
                check_logits(got[s, i], ref.astype(np.float32), cfg.wtype, f"sequence {s} of {n}, row {i}")
                # what the row's numbers stand for: half a step of them off, what its top loses by d's rounding (15 2^-11 d), its own rounding, and
                # what k and v were off before (the operands' F16 rounding: the logits' tolerance)
                for l in range(cfg.n_layers):
                    for which in (0, 1):
                        (_, d, _), v = pages[l][which]
                        d = np.repeat(d[at[-1]].astype(np.float64), 32, -1)[:, :cfg.head_dim]
                        off = np.abs(v[at[-1]].astype(np.float64) - own[l][which])
                        assert (off <= d * (0.5 + 0.01) + H16 * np.abs(v[at[-1]]) + TOL[cfg.wtype]).all(), (l, which, off.max())
    assert bd.errors() == 0
    dec.close()


@pytest.mark.parametrize("kw", [dict(), dict(wtype=synth.Q8_0, rope_neox=0, tied=False, bias=False, number=82),
                                dict(dim=256, n_heads=4, n_kv_heads=4, head_dim=64, number=83), dict(dim=256, n_heads=2, n_kv_heads=1, head_dim=128, number=84)])
def test_steps(lib, kw):  # noqa: F811
    check_steps(lib, config(**kw), 20, 1, [[1, 1, 0], [2, 2, 1], [3, 3, 2]])
    check_steps(lib, config(**kw), 0, 3, [[3, 2, 1], [6, 5, 4]], page=8)


def test_steps_of_both_kinds_in_turn(lib):  # noqa: F811
    """A handle's steps on FP16 and on 4-bit pages do not touch each other."""
    cfg = config()
    W = synth.make_weights(cfg)
    alone, both = [], []
    for other in (False, True):
        dec = lib.Decoder(cfg, W)
        a = lib.BatchDecoder(dec, 2, 20, 0, q4=True)
        b = lib.BatchDecoder(dec, 3, 20, 0)
        for n in range(1, 8):
            put(a, cfg, [n, n])
            a.step()
            if other:
                put(b, cfg, [n, n, n])
                b.step()
            (both if other else alone).append(a.logits.clone())
        dec.close()
    assert all(torch.equal(x, y) for x, y in zip(alone, both))


def test_captured_and_replayed(lib):  # noqa: F811
    cfg = config()
    runs = []
    for captured in (False, True):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            dec = lib.Decoder(cfg, synth.make_weights(cfg), stream=s.cuda_stream)
            bd = lib.BatchDecoder(dec, 3, 40, 0, q4=True)
            put(bd, cfg, [1, 1, 1])
            bd.step()
            if captured:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=s):
                    bd.step()
            got = []
            for n in range(2, 30):
                put(bd, cfg, [n, n, n])
                g.replay() if captured else bd.step()
                got.append(bd.logits.clone())
            s.synchronize()
            lib.llm_sync(dec.h)
            if captured:
                del g
            dec.close()
        runs.append(got)
    assert all(torch.equal(x, y) for x, y in zip(*runs))


def test_refusals(lib):  # noqa: F811
    cfg = config(dim=320, n_heads=8, n_kv_heads=2, head_dim=40, number=85)
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    with pytest.raises(lib.LlmError):
        lib.BatchDecoder(dec, 2, 20, 0, q4=True)               # head_dim 40
    b = lib.binding.llm_batch(n_seqs=1, n_new=1, page_size=16, n_pages=2, max_pages=2, pages=0x10000, page_table=0x10000, lens=0x10000, tokens=0x10000,
                              logits=0x10000)
    assert lib.binding._lib.llm_decode_batch_q4(dec.h, ctypes.addressof(b)) == lib.LLM_ERR_UNSUPPORTED
    dec.close()
    dec = lib.Decoder(config(), synth.make_weights(config()))
    with pytest.raises(lib.LlmError):
        lib.BatchDecoder(dec, 2, 20, 0, page_size=4, q4=True)
    b.page_size = 4
    assert lib.binding._lib.llm_decode_batch_q4(dec.h, ctypes.addressof(b)) == lib.LLM_ERR_UNSUPPORTED
    assert lib.llm_last_error(dec.h)
    dec.close()


def test_forks(lib):  # noqa: F811
    """Sequences that fork through a pool over 4-bit pages go on as their parent would."""
    cfg = config()
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    runs = []
    for forked in (False, True):
        bd = lib.BatchDecoder(dec, 3, 40, 0, page_size=8, q4=True)
        bd.page_table.fill_(-1)
        refs = torch.zeros(15, dtype=torch.int32, device="cuda")
        pool = bd.pool(refs)
        rows, parents, got = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda"), []
        up = lib.PagesUpdate(pool, parents, rows)
        for step in range(20):
            which = torch.arange(3)
            if forked and step >= 11:
                which[:] = 1
                parents.copy_(torch.tensor([1, 1, 1] if step == 11 else [0, 1, 2], dtype=torch.int32))
            rows.add_(1)
            up()
            bd.tokens.copy_(((step * 7 + which * 31) % 499)[:, None].int())
            bd.step()
            got.append(bd.logits.clone())
        assert bd.errors() == 0 and pool.errors() == 0
        runs.append(got)
    for step, (x, y) in enumerate(zip(*runs)):
        assert torch.equal(x[1], y[1])
        if step >= 11:
            assert (y[0] - x[1]).abs().max() <= TOL[cfg.wtype] and (y[2] - x[1]).abs().max() <= TOL[cfg.wtype]
    dec.close()


@pytest.mark.parametrize("kw,page", [(dict(dim=320, n_heads=8, n_kv_heads=2, head_dim=40, number=85), 16), (dict(), 4)])
def test_refusals_with_tensors_of_a_step_on_f16_pages(lib, kw, page):  # noqa: F811
    """Every pointer is a real one (pages in FP16 are larger than those of 4-bit values), and nothing is written."""
    cfg = config(**kw)
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    bd = lib.BatchDecoder(dec, 2, 20, 0, page_size=page)
    put(bd, cfg, [1, 1])
    bd.logits.fill_(7.0)
    bd.pages.fill_(3.0)
    torch.cuda.synchronize()
    assert lib.binding._lib.llm_decode_batch_q4(dec.h, ctypes.addressof(bd.struct)) == lib.LLM_ERR_UNSUPPORTED
    assert lib.llm_last_error(dec.h)
    torch.cuda.synchronize()
    assert (bd.logits == 7.0).all() and (bd.pages == 3.0).all() and bd.errors() == 0
    bd.step()                                                       # the handle goes on
    lib.llm_sync(dec.h)
    assert bd.logits.isfinite().all() and not (bd.logits == 7.0).any() and bd.errors() == 0
    dec.close()
