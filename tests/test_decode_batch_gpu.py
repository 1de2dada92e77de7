"""llm_decode_batch: steps of several continuations of one prompt against the
oracle, and against the decode step run sequence by sequence ("What a Llama
model computes, and why" §2 and §4).  The projections' operands are rounded to
F16 as in the batched prefill, so logits are held to its tolerance; the prompt's
rows are the handle's cache, the sequences' own rows are pages."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import synth
from harness import TOL, check_logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import llama_decode_forward_gb300 as L
    return L


def config(**kw):
    base = dict(n_layers=2, dim=256, n_heads=8, n_kv_heads=2, head_dim=32, ffn_dim=576, vocab=1000, max_seq=300,
                eps=1e-5, rope_base=1e6, rope_neox=1, wtype=synth.F16, tied=True, bias=True, number=81)
    base.update(kw)
    return synth.ModelConfig("decode_batch", **base)


def token(cfg, s, e):
    return (7919 * (s + 1) + 104729 * (e + 1)) % cfg.vocab


def put(bd, cfg, lens):
    """The step's lens, and the tokens of its rows; padding rows hold no token."""
    n_new = bd.tokens.shape[1]
    tok = [[token(cfg, s, n - n_new + e) if n - n_new + e >= 0 else -5 for e in range(n_new)] for s, n in enumerate(lens)]
    bd.tokens.copy_(torch.tensor(tok, dtype=torch.int32))
    bd.lens.copy_(torch.tensor(lens, dtype=torch.int32))


def scatter(bd, seed):
    """Pages in an order that is not the sequences'."""
    flat = bd.page_table.flatten()
    order = torch.from_numpy(np.random.RandomState(seed).permutation(flat.numel())).cuda()
    bd.page_table.copy_(flat[order].view_as(bd.page_table))


def check_steps(lib, cfg, prefix, n_new, steps, page=16, copy=False):
    """steps: each step's lens.  Every step's logits, against an oracle that runs
    the sequences one after another from the prompt's rows."""
    W = synth.make_weights(cfg)
    ora, dec = oracle.OracleModel(cfg, W), lib.Decoder(cfg, W)
    if copy:
        lib.llm_prefill_f16_copy(dec.h)
    if prefix:
        toks = synth.prompt(cfg, prefix)
        ora.prefill(toks, 0)
        lib.llm_prefill(dec.h, toks, 0)
    n_seqs = len(steps[0])
    bd = lib.BatchDecoder(dec, n_seqs, max(max(s) for s in steps), prefix, n_new, page)
    scatter(bd, 5)
    ref = [[ora.forward(token(cfg, s, e), prefix + e) for e in range(max(st[s] for st in steps))] for s in range(n_seqs)]
    launches = lib.llm_launch_count(dec.h)
    for lens in steps:
        put(bd, cfg, lens)
        bd.step()
        lib.llm_sync(dec.h)
        got = bd.logits.cpu().numpy()
        for s, n in enumerate(lens):
            for e in range(n_new):
                if n - n_new + e >= 0:
                    check_logits(got[s, e], ref[s][n - n_new + e], cfg.wtype, f"sequence {s} of {n}, row {e}")
    assert bd.errors() == 0
    assert lib.llm_launch_count(dec.h) > launches
    dec.close()


@pytest.mark.parametrize("kw", [{}, dict(rope_neox=0, bias=False, tied=False, number=82),
                                dict(wtype=synth.Q8_0, rope_neox=0, bias=False, number=83),
                                dict(wtype=synth.Q8_0, tied=False, rope_freqs=True, number=84),
                                dict(n_heads=4, n_kv_heads=4, head_dim=64, bias=False, number=85),
                                dict(dim=512, n_heads=4, n_kv_heads=1, head_dim=128, vocab=1003, number=86),
                                dict(wtype=synth.Q8_0, n_heads=16, n_kv_heads=4, head_dim=16, vocab=999, bias=False, number=87)])
def test_steps_match_the_oracle(lib, kw):
    check_steps(lib, config(**kw), 150, 1, [[1, 1, 1, 1, 1], [2, 2, 2, 2, 2], [3, 3, 3, 3, 3]])


@pytest.mark.parametrize("prefix", [0, 1, 127, 129])
def test_prefix_lengths(lib, prefix):
    check_steps(lib, config(), prefix, 1, [[n] * 3 for n in range(1, 6)], page=4)


def test_several_rows_and_padding(lib):
    # sequences that start with 5, 3, 1 rows and none, then two that stand still
    # behind ones that go on (their rows are written again)
    check_steps(lib, config(), 40, 5, [[5, 3, 1, 0], [10, 8, 4, 5], [15, 8, 5, 5]], page=8)


def test_one_sequence_and_many(lib):
    check_steps(lib, config(), 33, 1, [[1], [2]])
    check_steps(lib, config(), 33, 2, [[2] * 100, [4] * 100], page=2)
    check_steps(lib, config(wtype=synth.Q8_0, bias=False, number=83), 33, 1, [[1] * 40], copy=True)


@pytest.mark.parametrize("n_seqs,n_new", [(1, 512), (512, 1), (4, 128)])
def test_the_most_rows(lib, n_seqs, n_new):
    check_steps(lib, config(max_seq=600), 30, n_new, [[n_new] * n_seqs], page=32)


def test_two_batches_on_one_prompt(lib):
    """Two batches take turns on one handle, one of them sharing a full page between its
    sequences; each goes on as if it were alone."""
    cfg = config()
    W = synth.make_weights(cfg)
    ora, dec = oracle.OracleModel(cfg, W), lib.Decoder(cfg, W)
    toks = synth.prompt(cfg, 25)
    ora.prefill(toks, 0)
    lib.llm_prefill(dec.h, toks, 0)
    a, b = lib.BatchDecoder(dec, 2, 12, 25, page_size=4), lib.BatchDecoder(dec, 3, 8, 25, n_new=2)
    common = [3, 1, 4, 1]                               # four rows that both sequences of a share
    a.page_table[1, 0] = a.page_table[0, 0]
    for e, t in enumerate(common):
        a.tokens.fill_(t)
        a.lens.copy_(torch.tensor([e + 1, 0], dtype=torch.int32))          # written once, by sequence 0
        a.step()
    for n in range(4):
        a.tokens.copy_(torch.tensor([[token(cfg, s, 4 + n)] for s in range(2)], dtype=torch.int32))
        a.lens.fill_(5 + n)
        a.step()
        put(b, cfg, [2 * n + 2] * 3)
        b.step()
    lib.llm_sync(dec.h)
    for s in range(2):
        for e, t in enumerate(common + [token(cfg, s, 4 + n) for n in range(4)]):
            ref = ora.forward(t, 25 + e)
        check_logits(a.logits[s, 0].cpu().numpy(), ref, cfg.wtype, f"batch a, sequence {s}")
    for s in range(3):
        for e in range(8):
            ref = ora.forward(token(cfg, s, e), 25 + e)
        check_logits(b.logits[s, 1].cpu().numpy(), ref, cfg.wtype, f"batch b, sequence {s}")
    assert a.errors() == 0 and b.errors() == 0
    dec.close()


@pytest.mark.parametrize("base", [synth.QWEN2_F16, synth.LLAMA1B_Q8], ids=["qwen2-1b-f16", "llama-3.2-1b-q8_0"])
def test_full_width_equals_sequence_by_sequence(lib, base):
    """Two layers of the full-width models: 24 continuations of a 200-token
    prompt, against the decode step of the same handle, one sequence at a time."""
    import dataclasses
    cfg = dataclasses.replace(base, n_layers=2, max_seq=256)
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    prefix, n_seqs, n = 200, 24, 3
    lib.llm_prefill(dec.h, synth.prompt(cfg, prefix), 0)
    bd = lib.BatchDecoder(dec, n_seqs, 16, prefix)
    got = []
    for i in range(n):
        put(bd, cfg, [i + 1] * n_seqs)
        bd.step()
        lib.llm_sync(dec.h)
        got.append(bd.logits[:, 0].cpu().numpy())
    ref = np.empty(cfg.vocab, np.float32)
    for s in range(n_seqs):
        for i in range(n):
            lib.llm_decode_step(dec.h, token(cfg, s, i), prefix + i, ref)
            check_logits(got[i][s], ref, cfg.wtype, f"sequence {s}, step {i}")
    assert bd.errors() == 0
    dec.close()


def test_captured_steps_feed_on_their_own_tokens(lib):
    """Greedy steps as a user runs them: the step, the best token's log
    probability (llm_logprobs), that token as the next step's, the lengths one
    further; captured once, replayed, against the same steps without a graph."""
    cfg = config()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        dec = lib.Decoder(cfg, synth.make_weights(cfg))
        lib.llm_prefill(dec.h, synth.prompt(cfg, 60), 0)
        runs = []
        for graph in (False, True):
            bd = lib.BatchDecoder(dec, 6, 32, 60)
            lp = lib.LogProbs(bd.logits.view(6, cfg.vocab), None, top=2)

            def step():
                bd.step()
                lp()
                bd.tokens.copy_(lp.top_id[:, :1])
                bd.lens.add_(1)

            put(bd, cfg, [1] * 6)
            if graph:
                bd.step()                       # allocates before the capture; writes what the first replay writes
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=stream):
                    step()
            out = []
            for _ in range(8):
                g.replay() if graph else step()
                out.append((lp.top_id.clone(), lp.top_logprob.clone(), lp.entropy.clone()))
            lib.llm_sync(dec.h)
            assert bd.errors() == 0 and bd.lens.tolist() == [9] * 6
            runs.append(out)
        for a, b in zip(*runs):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        torch.cuda.synchronize()
        dec.close()


def test_the_handle_goes_on(lib):
    """A batch's steps leave the handle's cache, logits and next steps as they were."""
    cfg = config()
    W = synth.make_weights(cfg)
    a, b = lib.Decoder(cfg, W), lib.Decoder(cfg, W)
    for d in (a, b):
        lib.llm_prefill(d.h, synth.prompt(cfg, 50), 0)
        lib.llm_decode_step(d.h, 3, 50)
    before = [t.clone() for layer in range(2) for t in a.kv_tensors(layer)] + [a.logits_tensor().clone()]
    bd = lib.BatchDecoder(a, 4, 20, 51)
    for n in range(1, 4):
        put(bd, cfg, [n] * 4)
        bd.step()
    lib.llm_sync(a.h)
    after = [t for layer in range(2) for t in a.kv_tensors(layer)] + [a.logits_tensor()]
    assert all(torch.equal(x, y) for x, y in zip(before, after))
    x, y = np.empty(cfg.vocab, np.float32), np.empty(cfg.vocab, np.float32)
    for run in (lambda d, o: lib.llm_decode_step(d.h, 9, 51, o), lambda d, o: lib.llm_prefill(d.h, synth.prompt(cfg, 70), 0, o)):
        run(a, x)
        run(b, y)
        assert np.array_equal(x.view(np.uint32), y.view(np.uint32))
    a.close()
    b.close()


def test_rows_are_independent_of_the_rest(lib):
    """A sequence's logits do not depend on the others: the same sequence in
    every place of the batch, and twice on the same pages."""
    cfg = config()
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    lib.llm_prefill(dec.h, synth.prompt(cfg, 20), 0)
    bd = lib.BatchDecoder(dec, 5, 16, 20)
    bd.tokens.fill_(17)
    bd.lens.fill_(1)
    bd.page_table[4] = bd.page_table[3]                 # the same rows, written twice alike
    bd.step()
    lib.llm_sync(dec.h)
    assert all(torch.equal(bd.logits[0], bd.logits[s]) for s in range(1, 5))
    dec.close()


def test_tokens_and_pages_out_of_range(lib):
    cfg = config()
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    lib.llm_prefill(dec.h, synth.prompt(cfg, 20), 0)
    bd = lib.BatchDecoder(dec, 3, 16, 20)
    put(bd, cfg, [1, 1, 1])
    bd.step()
    lib.llm_sync(dec.h)
    want = bd.logits.clone()
    bd.page_table[1, 0] = bd.struct.n_pages             # a page that is not there: one sequence's, reported
    bd.step()
    lib.llm_sync(dec.h)
    assert bd.errors() == lib.LLM_PAGES_BAD_PAGE
    assert torch.equal(bd.logits[0], want[0]) and torch.equal(bd.logits[2], want[2])
    bd.page_table[1, 0] = 1
    bd.err.zero_()
    bd.lens[2] = 17                                     # behind the table
    bd.step()
    lib.llm_sync(dec.h)
    assert bd.errors() == lib.LLM_PAGES_BAD_LEN
    assert torch.equal(bd.logits[:2], want[:2])
    bd.lens[2] = 1
    for bad in (-1, cfg.vocab):
        bd.tokens[1, 0] = bad
        bd.step()
        with pytest.raises(lib.LlmError) as e:
            lib.llm_sync(dec.h)
        assert e.value.status == lib.LLM_ERR_OUT_OF_RANGE
        with pytest.raises(lib.LlmError) as e:
            bd.step()
        assert e.value.status == lib.LLM_ERR_STATE
        lib.llm_reset(dec.h)
    bd.err.zero_()
    lib.llm_prefill(dec.h, synth.prompt(cfg, 20), 0)
    put(bd, cfg, [1, 1, 1])
    bd.step()
    lib.llm_sync(dec.h)
    assert torch.equal(bd.logits, want) and bd.errors() == 0
    dec.close()


def test_refusals(lib):
    cfg = config()
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    bd = lib.BatchDecoder(dec, 3, 16, 20)
    logits = bd.logits.fill_(7).clone()
    R, U, I = lib.LLM_ERR_OUT_OF_RANGE, lib.LLM_ERR_UNSUPPORTED, lib.LLM_ERR_INVALID_ARG
    for field, value, code in [("n_seqs", -1, R), ("n_seqs", 513, R), ("n_new", 0, R), ("n_new", 171, R), ("prefix_len", -1, R),
                               ("prefix_len", 301, R), ("max_pages", -1, R), ("max_pages", 1 << 22, R), ("page_size", 0, R),
                               ("page_size", 24, I), ("n_pages", -1, I), ("pages", 0, I), ("pages", bd.pages.data_ptr() + 2, I),
                               ("page_table", 0, I), ("page_table", bd.page_table.data_ptr() + 1, I), ("lens", 0, I),
                               ("lens", bd.lens.data_ptr() + 2, I), ("tokens", 0, I), ("tokens", bd.tokens.data_ptr() + 2, I),
                               ("logits", 0, I), ("logits", bd.logits.data_ptr() + 4, I), ("err", bd.err.data_ptr() + 2, I)]:
        keep = getattr(bd.struct, field)
        setattr(bd.struct, field, value)
        with pytest.raises(lib.LlmError) as e:
            bd.step()
        assert e.value.status == code, (field, value)
        setattr(bd.struct, field, keep)
    assert lib.binding._lib.llm_decode_batch(dec.h, None) == I
    assert lib.binding._lib.llm_batch_pages_bytes(dec.h, 3, 24) == I
    assert lib.binding._lib.llm_batch_pages_bytes(dec.h, -1, 16) == I
    assert lib.llm_batch_pages_bytes(dec.h, 3, 16) == 2 * 2 * 3 * 16 * 64 * 2
    empty = lib.llm_batch(n_seqs=0, n_new=1, prefix_len=5, page_size=16)
    lib.llm_decode_batch(dec.h, empty)                  # nothing to do
    lib.llm_sync(dec.h)
    assert torch.equal(bd.logits, logits)
    dec.close()
    for kw, code in ((dict(wtype=synth.F32, bias=False, number=88), U), (dict(dim=512, n_heads=2, n_kv_heads=1, head_dim=256, number=89), U)):
        cfg = config(**kw)
        dec = lib.Decoder(cfg, synth.make_weights(cfg))
        bd = lib.BatchDecoder(dec, 3, 16, 20)
        with pytest.raises(lib.LlmError) as e:
            bd.step()
        assert e.value.status == code
        dec.close()


def test_allocation_failure_leaves_the_handle_usable(lib):
    cfg = config()
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    lib.llm_prefill(dec.h, synth.prompt(cfg, 20), 0)
    bd = lib.BatchDecoder(dec, 3, 16, 20)
    put(bd, cfg, [1, 1, 1])
    for n in (1, 2):                                  # the attention's workspace, then the angle table
        lib.llm_test_fail_alloc(n)
        with pytest.raises(lib.LlmError) as e:
            bd.step()
        assert e.value.status == lib.LLM_ERR_NO_MEMORY
        lib.llm_test_fail_alloc(0)
    bd.step()
    lib.llm_sync(dec.h)
    assert bool(torch.isfinite(bd.logits).all()) and bd.errors() == 0
    dec.close()


@pytest.mark.parametrize("copy", [False, True])
def test_captured_step_outlives_larger_batches(lib, copy):
    """A step captured on a handle keeps its memory when a larger batch on the same handle
    replaces the workspace and the angle table, and when the F16 copy that it reads is given
    up: the replay gives the same bits.  Within a capture a call that would allocate is
    refused, and the capture goes on."""
    cfg = config(wtype=synth.Q8_0, bias=False, number=83)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        dec = lib.Decoder(cfg, synth.make_weights(cfg))
        if copy:
            lib.llm_prefill_f16_copy(dec.h)
        lib.llm_prefill(dec.h, synth.prompt(cfg, 20), 0)
        small, large = lib.BatchDecoder(dec, 2, 16, 20), lib.BatchDecoder(dec, 64, 600, 20)
        put(small, cfg, [3, 1])
        put(large, cfg, [1] * 64)
        small.step()
        torch.cuda.synchronize()
        want = small.logits.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            with pytest.raises(lib.LlmError) as e:
                large.step()
            small.step()
        assert e.value.status == lib.LLM_ERR_STATE
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(small.logits, want)
        large.step()
        if copy:
            lib.llm_prefill_f16_copy(dec.h, False)
        torch.cuda.synchronize()
        junk = [torch.full((1 << 19,), float("nan"), device="cuda") for _ in range(64)]     # whatever was freed is in use again
        small.logits.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(small.logits, want)
        assert all(bool(t.isnan().all()) for t in junk) and small.errors() == 0
        lib.llm_sync(dec.h)
        del graph
        dec.close()


@pytest.mark.parametrize("outer", [False, True])
def test_decoder_on_its_own_stream(lib, outer):
    """The decoder's stream is not the current one, and the current one is busy when the
    batch is made, its tensors are written and its results are read (outer: it is a side
    stream too): each step sees the values written before it and nothing lands later."""
    cfg = config()
    W = synth.make_weights(cfg)
    prompt, steps = synth.prompt(cfg, 40), [[1, 1, 1], [2, 2, 2], [3, 3, 3]]
    want = []
    dec = lib.Decoder(cfg, W)
    lib.llm_prefill(dec.h, prompt, 0)
    bd = lib.BatchDecoder(dec, 3, 16, 40)
    for lens in steps:
        put(bd, cfg, lens)
        bd.step()
        lib.llm_sync(dec.h)
        want.append(bd.logits.clone())
    dec.close()
    own = torch.cuda.Stream()
    dec = lib.Decoder(cfg, W, stream=own.cuda_stream)
    lib.llm_prefill(dec.h, prompt, 0)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream() if outer else torch.cuda.current_stream()):
        host = [[torch.tensor(v, dtype=torch.int32).pin_memory() for v in
                 ([[token(cfg, s, n - 1)] for s, n in enumerate(lens)], lens)] for lens in steps]
        got = []
        torch.cuda._sleep(20000000)
        bd = lib.BatchDecoder(dec, 3, 16, 40)
        for tokens, lens in host:
            bd.tokens.copy_(tokens, non_blocking=True)
            bd.lens.copy_(lens, non_blocking=True)
            torch.cuda._sleep(2000000)
            bd.step()
            got.append(bd.logits.clone())
        bd.pages.fill_(0)                              # behind the last step, whose logits are already there
        del bd                                         # memory given back while the steps are still queued
        junk = [torch.full((1 << 16,), float("nan"), device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(junk) == 8
    lib.llm_sync(dec.h)
    dec.close()


@pytest.mark.parametrize("kw", [{}, dict(wtype=synth.Q8_0, bias=False, number=83),
                                dict(dim=512, n_heads=4, n_kv_heads=1, head_dim=128, vocab=1003, number=86)])
def test_wait_that_gives_up_reaches_the_handle(lib, kw):
    """A wait of the prefix attention that runs out (nothing is copied, its limit is short)
    is the handle's device error, with the batch's own error word and without one."""
    cfg = config(**kw)
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    lib.llm_prefill(dec.h, synth.prompt(cfg, 150), 0)
    bd = lib.BatchDecoder(dec, 3, 16, 150)
    put(bd, cfg, [1, 1, 1])
    bd.step()
    lib.llm_sync(dec.h)
    want = bd.logits.clone()
    err = bd.struct.err
    for word in (None, err):
        bd.struct.err = word
        lib.llm_test_batch_wait(dec.h, 20)
        bd.step()
        lib.llm_test_batch_wait(dec.h, 0)
        with pytest.raises(lib.LlmError) as e:
            lib.llm_sync(dec.h)
        assert e.value.status == lib.LLM_ERR_DEVICE_TIMEOUT
        assert bd.errors() == (lib.LLM_PAGES_TIMEOUT if word else 0)
        with pytest.raises(lib.LlmError) as e:
            bd.step()
        assert e.value.status == lib.LLM_ERR_STATE
        lib.llm_reset(dec.h)
        lib.llm_prefill(dec.h, synth.prompt(cfg, 150), 0)
        bd.err.zero_()
        bd.step()
        lib.llm_sync(dec.h)
        assert torch.equal(bd.logits, want) and bd.errors() == 0
    for bad in (-1, 1001):
        with pytest.raises(lib.LlmError) as e:
            lib.llm_test_batch_wait(dec.h, bad)
        assert e.value.status == lib.LLM_ERR_OUT_OF_RANGE
    dec.close()


def test_guard_bands_of_the_batch(lib):
    """Steps of the smallest and of larger batches, with padding and a growing workspace,
    leave every guard byte as written; a byte changed next to either end of the step's own
    buffers is reported."""
    cfg = config()
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    lib.llm_prefill(dec.h, synth.prompt(cfg, 150), 0)
    for n_seqs, n_new, prefix, lens in ((1, 1, 150, [16]), (3, 5, 0, [5, 2, 40]), (64, 8, 129, [8] * 63 + [300])):
        bd = lib.BatchDecoder(dec, n_seqs, max(lens), prefix, n_new)
        put(bd, cfg, lens)
        bd.pages.fill_(0.25)
        bd.step()
        lib.llm_sync(dec.h)
        assert bd.errors() == 0 and lib.llm_test_guards(dec.h) == 0
    for band in range(10):                    # cache, activations, prefill workspace, the batch's workspace and angles
        lib.llm_test_poke_guard(dec.h, band)
        assert lib.llm_test_guards(dec.h) == band + 1
    with pytest.raises(lib.LlmError) as e:
        lib.llm_test_poke_guard(dec.h, 10)
    assert e.value.status == lib.LLM_ERR_OUT_OF_RANGE
    dec.close()


def test_host_allocation_failure_is_a_status(lib):
    """The tables that a prefill and a batch step make on the host: their allocation
    failing is NO_MEMORY with a reason, and the next call works."""
    cfg = config()
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    toks, logits = synth.prompt(cfg, 20), np.empty(cfg.vocab, np.float32)
    lib.llm_prefill(dec.h, toks, 0, logits)
    bd = lib.BatchDecoder(dec, 3, 16, 20)
    put(bd, cfg, [1, 1, 1])
    bd.step()
    lib.llm_sync(dec.h)
    want = bd.logits.clone()
    again = np.empty(cfg.vocab, np.float32)
    for call in (bd.step, lambda: lib.llm_prefill(dec.h, toks, 0, again)):
        lib.llm_test_fail_alloc(1)                    # (the device memory is there: the table is the first)
        with pytest.raises(lib.LlmError) as e:
            call()
        lib.llm_test_fail_alloc(0)
        assert e.value.status == lib.LLM_ERR_NO_MEMORY and "tensor maps" in str(e.value)
        call()
    bd.step()
    lib.llm_sync(dec.h)
    assert torch.equal(bd.logits, want) and np.array_equal(again.view(np.uint32), logits.view(np.uint32))
    dec.close()


def test_copy_that_no_graph_reads_is_freed(lib):
    """After a captured step's copy was kept, a new copy that no captured step reads is
    given back at once."""
    cfg = config(wtype=synth.Q8_0, bias=False, number=83, dim=512, n_heads=16, ffn_dim=4096, n_layers=4)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        dec = lib.Decoder(cfg, synth.make_weights(cfg))
        lib.llm_prefill_f16_copy(dec.h)
        bd = lib.BatchDecoder(dec, 2, 16, 0)
        put(bd, cfg, [1, 1])
        bd.step()
        torch.cuda.synchronize()
        want = bd.logits.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            bd.step()
        lib.llm_prefill_f16_copy(dec.h, False)         # kept for the graph
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        for _ in range(3):
            lib.llm_prefill_f16_copy(dec.h)
            bd.step()
            lib.llm_prefill_f16_copy(dec.h, False)
        torch.cuda.synchronize()
        assert torch.cuda.mem_get_info()[0] == free
        bd.logits.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bd.logits, want)
        del graph
        dec.close()
