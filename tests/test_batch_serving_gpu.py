"""The operators around a batch's pages run together, as a decoding loop runs them: room for the
next rows (PagesUpdate), append and attention on 4-bit pages, adjusted logits and their log
probabilities, sequences that fork and end, and pools that are compacted; captured into a graph and
replayed; on other streams."""
import numpy as np
import pytest
import torch

from test_batch_ops_gpu import F16, F32, check_attend, lib, rand  # noqa: F401
from test_q4_pages_gpu import decode, values

pytestmark = pytest.mark.gpu

N_SEQS, HEADS, N_KV, HD, PAGE, MAX_PAGES, N_PAGES, VOCAB = 5, 4, 2, 64, 8, 12, 50, 1000


class Loop:
    """A decoding loop of one layer whose logits are a fixed matrix times the attention's output."""

    def __init__(self, lib, seed=0):
        z = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.k, self.v = lib.q4_pages(N_PAGES, PAGE, N_KV, HD), lib.q4_pages(N_PAGES, PAGE, N_KV, HD)
        self.table, self.lens, self.refs = z(N_SEQS, MAX_PAGES) - 1, z(N_SEQS), z(N_PAGES)
        self.parents, self.rows = torch.arange(N_SEQS, dtype=torch.int32, device="cuda"), z(N_SEQS)
        self.pages = lib.PagedBatchQ4(self.k, self.v, self.table, self.lens, PAGE, N_KV, HD)
        self.pool = lib.PagePool(self.k, self.v, self.table, self.lens, self.refs, page_size=PAGE, err=self.pages.err)
        self.qkv = rand(seed, N_SEQS, HEADS + 2 * N_KV, HD)
        q, k, v = self.qkv[:, :HEADS], self.qkv[:, HEADS:HEADS + N_KV], self.qkv[:, HEADS + N_KV:]
        self.q, self.out = torch.empty(N_SEQS, HEADS, HD, device="cuda"), torch.zeros(N_SEQS, HEADS, HD, device="cuda")
        self.matrix, self.logits = rand(7, HEADS * HD, VOCAB), torch.empty(N_SEQS, VOCAB, device="cuda")
        self.history, self.counts = z(N_SEQS, 64), z(N_SEQS)
        ones = torch.ones(N_SEQS, device="cuda")
        self.update = lib.PagesUpdate(self.pool, self.parents, self.rows)
        self.ops = [self.update, lib.KvAppend(self.pages, q, k, v, lib.rope_table(96, HD, 1e4), q_out=self.q),
                    lib.AttendBatch(self.pages, self.q, self.out)]
        self.adjust = lib.AdjustLogits(self.logits, history=self.history, history_lens=self.counts, repetition=ones * 1.3, presence=ones * 0.5)
        self.logprobs = lib.LogProbs(self.logits, top=3)
        self.compact = lib.PagesCompact(self.pool)

    def step(self):
        for op in self.ops:
            op()
        torch.matmul(self.out.view(N_SEQS, -1), self.matrix, out=self.logits)
        self.adjust()
        self.logprobs()
        # the most likely token is next: into the history, and the next step's input
        self.history.scatter_(1, self.counts.long()[:, None], self.logprobs.top_id[:, :1])
        self.counts += 1
        self.qkv.mul_(0.9).add_(self.logprobs.top_logprob[:, :1, None], alpha=0.01)

    def choose(self, step):
        """Parents and rows of the next step, by its number alone."""
        r = np.random.RandomState(step)
        parents = np.arange(N_SEQS)
        if step % 4 == 3:
            parents = r.randint(0, N_SEQS, N_SEQS)
            if step % 8 == 7:
                parents[r.randint(N_SEQS)] = -1
        return torch.from_numpy(parents.astype(np.int32)).cuda()

    def go_on(self, step):
        parents = self.choose(step)
        self.parents.copy_(parents)
        at = parents.long().clamp(min=0)
        new = parents < 0
        self.rows.copy_(torch.where(new, 0, self.lens[at]) + 1)
        self.history.copy_(self.history[at])
        self.counts.copy_(torch.where(new, 0, self.counts[at]))

    def state(self):
        held = torch.arange(MAX_PAGES, device="cuda") < -(-self.lens[:, None] // PAGE)
        return [self.lens.clone(), (self.table * held).clone(), self.refs.clone(), self.out.clone(), self.logits.clone(), self.logprobs.top_id.clone(),
                self.history.clone()]


def test_steps(lib):  # noqa: F811
    """Every step's attention against the rows that each sequence was given, kept on the host through forks and ends."""
    c, rows = Loop(lib), [[] for _ in range(N_SEQS)]
    for step in range(30):
        c.go_on(step)
        parents = c.parents.tolist()
        c.step()
        assert c.pages.errors() == 0
        if step % 6 == 5:
            # (the data are moved behind the step: its own results are checked below all the same)
            c.compact()
            assert (c.refs[:int(c.compact.n_live)] > 0).all() and not c.refs[int(c.compact.n_live):].any()
        kv = [values(*decode(t, PAGE, N_KV, HD)) for t in (c.k, c.v)]
        rows = [list(rows[p]) if p >= 0 else [] for p in parents]
        table, lens = c.table.cpu().numpy(), c.lens.tolist()
        assert lens == [len(r) + 1 for r in rows]
        for s in range(N_SEQS):
            mine = [tuple(t[table[s, e // PAGE], e % PAGE].tobytes() for t in kv) for e in range(lens[s])]
            assert mine[:-1] == rows[s], (step, s)          # what the sequence held before, bit for bit
            rows[s] = mine
        b = type("B", (), dict(lens=lens, n_new=1, prefix=0, k=torch.from_numpy(kv[0]).cuda(), v=torch.from_numpy(kv[1]).cuda()))
        b.rows = lambda: ((s, s, n - 1) for s, n in enumerate(lens))
        b.gather = lambda t, s, n: t[c.table[s, :-(-n // PAGE)].long()].flatten(0, 1)[:n].double()
        check_attend(b, c.q, c.out, None, None)
        held = [table[s, i] for s in range(N_SEQS) for i in range(-(-lens[s] // PAGE))]
        assert np.array_equal(np.bincount(held, minlength=N_PAGES), c.refs.cpu().numpy())


def test_captured_and_replayed(lib):  # noqa: F811
    a, b = Loop(lib), Loop(lib)
    a.go_on(0)
    a.step()
    a.compact()
    b.go_on(0)
    b.step()
    b.compact()
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step()
    with torch.cuda.graph(h):
        b.compact()
    for step in range(1, 16):
        a.go_on(step)
        a.step()
        a.compact()
        b.go_on(step)
        g.replay()
        h.replay()
        assert all(torch.equal(x, y) for x, y in zip(a.state(), b.state())), step
    assert a.pages.errors() == b.pages.errors() == 0


def test_two_loops_on_two_streams(lib):  # noqa: F811
    one, streams, loops = Loop(lib), [torch.cuda.Stream() for _ in range(2)], [Loop(lib) for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for step in range(12):
        one.go_on(step)
        one.step()
        one.compact()
        for s, c in zip(streams, loops):
            with torch.cuda.stream(s):
                c.go_on(step)
                c.step()
                c.compact()
    torch.cuda.synchronize()
    for c in loops:
        assert all(torch.equal(x, y) for x, y in zip(one.state(), c.state()))


def test_f16_pages_of_a_batch_decoder_fork(lib):  # noqa: F811
    """A BatchDecoder's sequences fork through a pool over its pages: each then goes on as its parent would."""
    import synth
    cfg = synth.ModelConfig("fork", n_layers=2, dim=256, n_heads=8, n_kv_heads=2, head_dim=32, ffn_dim=512, vocab=500, max_seq=64, eps=1e-5,
                            rope_base=500000.0, rope_neox=0, wtype=synth.F16, tied=True, number=41)
    dec = lib.Decoder(cfg, synth.make_weights(cfg))
    prompt = np.arange(20, dtype=np.int32) + 3
    lib.llm_prefill(dec.h, prompt, 0)
    runs = []
    for forked in (False, True):
        bd = lib.BatchDecoder(dec, 3, 40, 20, page_size=8)
        refs = torch.zeros(15, dtype=torch.int32, device="cuda")
        bd.page_table.fill_(-1)
        pool = bd.pool(refs)
        rows, parents = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
        up, got = lib.PagesUpdate(pool, parents, rows), []
        for step in range(24):
            if forked and step == 11:
                parents.copy_(torch.tensor([1, 1, 1], dtype=torch.int32))
            rows.add_(1)
            up()
            parents.copy_(torch.arange(3, dtype=torch.int32))
            # after the fork every sequence is given what sequence 1 is given
            which = torch.arange(3) if not forked or step < 11 else torch.ones(3, dtype=torch.long)
            bd.tokens.copy_(((step * 7 + which * 31) % 499)[:, None].int())
            bd.step()
            got.append(bd.logits.clone())
        assert bd.errors() == 0 and pool.errors() == 0
        runs.append(got)
    for step, (x, y) in enumerate(zip(*runs)):
        assert torch.equal(x[1], y[1])
        if step >= 11:
            # (the sequences' pages are dealt to other warps, so their sums are ordered otherwise: the decode step's own tolerance)
            assert (y[0] - x[1]).abs().max() <= 2e-2 and (y[2] - x[1]).abs().max() <= 2e-2
    dec.close()
