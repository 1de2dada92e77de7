"""Batched decoding of several continuations of one prompt: the operators that
are measured, with their plain forms.

append    rotate the new tokens' q and k and store K and V in the pages of a cache
attend    attention of every new token over a prefix that all sequences share and
          over its own sequence's pages
logprobs  log probabilities of given tokens, the entropy and the top alternatives

Rows: n_seqs sequences of n_new new tokens each; lens[s] counts the rows of
sequence s behind the prefix, the new ones among them, so that new token i of s
is row lens[s] - n_new + i of its pages (negative: a padding row, left as it
was) at position prefix_len + that.  Plain forms compute in 32 bits, whatever
the inputs' type, and round once at the end.
"""
import math

import numpy as np
import torch

own = False

# Head layouts and vocabularies of the repository's own model shapes.
HEADS = {"tiny": (8, 2, 32), "stories": (6, 6, 48), "1b": (32, 8, 64), "7b": (32, 32, 128)}
VOCABS = (32000, 128256, 151936)
TYPES = {"f32": torch.float32, "f16": torch.float16}


def _append(name, heads, n_seqs, n_new, max_len, prefix, page, dtype, q_out, neox):
    return {"op": "append", "name": name, "heads": heads, "n_seqs": n_seqs, "n_new": n_new, "max_len": max_len,
            "prefix": prefix, "page": page, "dtype": dtype, "q_out": q_out, "neox": neox}


def _attend(name, heads, n_seqs, n_new, max_len, prefix, page, q, out):
    return {"op": "attend", "name": name, "heads": heads, "n_seqs": n_seqs, "n_new": n_new, "max_len": max_len,
            "prefix": prefix, "page": page, "q": q, "out": out}


def _logprobs(name, rows, vocab, targets, top, dtype, banned):
    return {"op": "logprobs", "name": name, "rows": rows, "vocab": vocab, "targets": targets, "top": top,
            "dtype": dtype, "banned": banned}


def listed():
    return [
        # one token of one sequence: pure latency
        _append("append-one", "1b", 1, 1, 300, 511, 16, "f32", "f32", False),
        # a decode step of 64 sequences, multi-head layout, NEOX pairs, q handed on in F16
        _append("append-step-7b", "7b", 64, 1, 512, 2000, 32, "f32", "f16", True),
        # 16 prompts' chunks of 500 tokens each
        _append("append-chunks", "1b", 16, 500, 900, 100, 16, "f16", "f16", False),
        # a few short continuations on the smallest model
        _attend("attend-tiny", "tiny", 3, 1, 20, 93, 16, "f32", "f32"),
        # best of 16 behind a 4k prompt
        _attend("attend-16", "1b", 16, 1, 130, 4095, 16, "f16", "f16"),
        # drafts of five tokens, verified in one step
        _attend("attend-drafts", "1b", 12, 5, 700, 2000, 16, "f32", "f32"),
        # multi-head attention, head size 128
        _attend("attend-7b", "7b", 48, 1, 512, 4000, 32, "f16", "f16"),
        # 64 continuations of a prompt near the context's end, queries in F32
        _attend("attend-long", "1b", 64, 1, 768, 32000, 64, "f32", "f16"),
        # 256 samples of one long prompt
        _attend("attend-256", "1b", 256, 1, 500, 16000, 16, "f16", "f16"),
        # one step's logits of one sequence
        _logprobs("logprobs-one", 1, 128256, 1, 20, "f32", 0),
        # four choices scored at each of 64 rows, half-precision logits
        _logprobs("logprobs-choices", 64, 32000, 4, 5, "f16", 0),
        # a prompt of 512 tokens scored, some tokens banned
        _logprobs("logprobs-prompt", 512, 151936, 1, 8, "f32", 1000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "logprobs"])
    top = max(work(c)["flops"] for c in listed() if c["op"] == op), max(work(c)["bytes"] for c in listed() if c["op"] == op)
    while True:
        if op == "logprobs":
            c = _logprobs("", _log_int(rng, 1, 512), rng.choice(VOCABS + (_log_int(rng, 1000, 160000),)), rng.choice([1, 1, 2, 4, 7]),
                          rng.choice([0, 1, 5, 8, 20, 32]), rng.choice(["f32", "f32", "f16"]), rng.choice([0, 0, 17, 500]))
        elif op == "append":
            n_new = rng.choice([1, 1, 2, 5, _log_int(rng, 3, 500)])
            c = _append("", rng.choice(list(HEADS)), _log_int(rng, 1, 256), n_new, n_new + _log_int(rng, 1, 900), rng.choice([0, _log_int(rng, 10, 30000)]),
                        rng.choice([8, 16, 32, 64]), rng.choice(["f32", "f16"]), rng.choice(["f32", "f16"]), rng.random() < 0.4)
        else:
            n_new = rng.choice([1, 1, 1, 2, 5, 8])
            c = _attend("", rng.choice(list(HEADS)), _log_int(rng, 1, 256), n_new, n_new + _log_int(rng, 1, 900), _log_int(rng, 50, 32000),
                        rng.choice([8, 16, 32, 64]), rng.choice(["f32", "f16"]), rng.choice(["f32", "f16"]))
        del c["name"]
        w = work(c)
        if w["flops"] <= top[0] and w["bytes"] <= top[1]:
            return c


def _lens(case, seed):
    """Rows behind the prefix of each sequence, ragged; the first sequence is the longest."""
    r = np.random.RandomState(seed % 2**31)
    lens = r.randint(case["n_new"], case["max_len"] + 1, case["n_seqs"])
    lens[0] = case["max_len"]
    return lens


def _pages(case, seed, gen):
    """A pool of pages in F16 with room for every sequence at its longest, and each sequence's table: scattered
    pages, -1 behind a sequence's last one."""
    _, n_kv, hd = HEADS[case["heads"]]
    ps, lens = case["page"], _lens(case, seed)
    need = -(-lens // ps)
    n_pages = case["n_seqs"] * int(need.max()) + 3
    order = np.random.RandomState(seed % 2**31 + 1).permutation(n_pages)
    table = np.full((case["n_seqs"], int(need.max())), -1, np.int32)
    at = np.arange(table.shape[1])[None, :] < need[:, None]
    table[at] = order[:int(need.sum())]
    kv = [torch.randn(n_pages, ps, n_kv, hd, device="cuda", dtype=torch.float16, generator=gen) for _ in range(2)]
    return {"k_pages": kv[0], "v_pages": kv[1], "table": torch.from_numpy(table).cuda(), "lens": torch.from_numpy(lens.astype(np.int32)).cuda()}


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "logprobs":
        n, v = case["rows"], case["vocab"]
        x = torch.randn(n, v, device="cuda", generator=gen).mul_(2.5)
        if case["banned"]:
            x[:, torch.randperm(v, device="cuda", generator=gen)[:case["banned"]]] = -math.inf
        s["logits"] = x.to(TYPES[case["dtype"]])
        s["targets"] = torch.randint(0, v, (n, case["targets"]), device="cuda", generator=gen, dtype=torch.int32)
        if own:
            import llama_decode_forward_gb300 as L
            s["plan"] = L.LogProbs(s["logits"], s["targets"], top=case["top"])
        return s
    n_heads, n_kv, hd = HEADS[case["heads"]]
    rows = case["n_seqs"] * case["n_new"]
    s.update(_pages(case, seed, gen))
    if case["op"] == "append":
        # q, k and v of a row lie behind one another, as the projection leaves them
        qkv = torch.randn(rows, n_heads + 2 * n_kv, hd, device="cuda", generator=gen).to(TYPES[case["dtype"]])
        s["q"], s["k"], s["v"] = qkv[:, :n_heads], qkv[:, n_heads:n_heads + n_kv], qkv[:, n_heads + n_kv:]
        pos = torch.arange(case["prefix"] + case["max_len"], device="cuda", dtype=torch.float64)
        theta = pos[:, None] * 500000.0 ** (-2.0 * torch.arange(hd // 2, device="cuda", dtype=torch.float64) / hd)
        s["cos_sin"] = torch.stack([theta.cos(), theta.sin()], -1).float()
        s["q_out"] = torch.empty(rows, n_heads, hd, device="cuda", dtype=TYPES[case["q_out"]])
    else:
        s["q"] = torch.randn(rows, n_heads, hd, device="cuda", generator=gen).to(TYPES[case["q"]])
        s["prefix_k"], s["prefix_v"] = (torch.randn(case["prefix"], n_kv, hd, device="cuda", dtype=torch.float16, generator=gen) for _ in range(2))
        s["out"] = torch.zeros(rows, n_heads, hd, device="cuda", dtype=TYPES[case["out"]])
    if own:
        import llama_decode_forward_gb300 as L
        pages = L.PagedBatch(s["k_pages"], s["v_pages"], s["table"], s["lens"], n_new=case["n_new"], prefix_len=case["prefix"])
        if case["op"] == "append":
            s["plan"] = L.KvAppend(pages, s["q"], s["k"], s["v"], s["cos_sin"], q_out=s["q_out"], rope_neox=case["neox"])
        else:
            s["plan"] = L.AttendBatch(pages, s["q"], s["out"], prefix_k=s["prefix_k"], prefix_v=s["prefix_v"])
    return s


def run(state):
    op = state["case"]["op"]
    if op == "append":
        if own:
            state["plan"]()
            return state["q_out"], state["k_pages"], state["v_pages"]
        return _plain_append(state)
    if op == "attend":
        if own:
            state["plan"]()
            return state["out"]
        return _plain_attend(state)
    if own:
        p = state["plan"]
        p()
        return p.logprob, p.entropy, p.top_id, p.top_logprob
    return _plain_logprobs(state)


def _index(s):
    """[n_seqs, n_new]: the row of its sequence's pages that each new token is."""
    n_new = s["case"]["n_new"]
    return s["lens"].long()[:, None] - n_new + torch.arange(n_new, device="cuda")


def _rotate(x, cs, neox):
    """The pairs of each head rotated; x: [rows, heads, hd] in 32 bits, cs: [rows, 1, hd / 2, 2]."""
    c, s = cs[..., 0], cs[..., 1]
    if neox:
        a, b = x.chunk(2, -1)
        return torch.cat([a * c - b * s, a * s + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _plain_append(s):
    case, e = s["case"], _index(s)
    cs = s["cos_sin"][(e + case["prefix"]).flatten()][:, None]
    slot = (s["table"].long().gather(1, e // case["page"]) * case["page"] + e % case["page"]).flatten()
    n_kv, hd = s["k"].shape[1:]
    s["k_pages"].view(-1, n_kv, hd)[slot] = _rotate(s["k"].float(), cs, case["neox"]).half()
    s["v_pages"].view(-1, n_kv, hd)[slot] = s["v"].half()
    s["q_out"].copy_(_rotate(s["q"].float(), cs, case["neox"]))
    return s["q_out"], s["k_pages"], s["v_pages"]


def _plain_attend(s):
    case = s["case"]
    n_heads, n_kv, hd = HEADS[case["heads"]]
    S, N, P, G = case["n_seqs"], case["n_new"], case["prefix"], n_heads // n_kv
    e = _index(s)
    # [n_kv, sequence, new token and head of the group, hd]
    q = (s["q"].float() * hd ** -0.5).view(S, N, n_kv, G, hd).permute(2, 0, 1, 3, 4).reshape(n_kv, S, N * G, hd)
    pk, pv = (t.float().permute(1, 0, 2) for t in (s["prefix_k"], s["prefix_v"]))
    at = s["table"].long().clamp(min=0)
    k, v = (t[at].float().view(S, -1, n_kv, hd).permute(2, 0, 1, 3) for t in (s["k_pages"], s["v_pages"]))
    seen = torch.arange(k.shape[2], device="cuda") <= e.repeat_interleave(G, 1)[:, :, None]
    own_scores = (q @ k.transpose(-1, -2)).masked_fill(~seen, -math.inf)
    prefix_scores = (q.reshape(n_kv, -1, hd) @ pk.transpose(-1, -2)).view(n_kv, S, N * G, P)
    m = torch.maximum(own_scores.amax(-1, keepdim=True), prefix_scores.amax(-1, keepdim=True))
    a, b = (own_scores - m).exp_(), (prefix_scores - m).exp_()
    o = a @ v + (b.view(n_kv, -1, P) @ pv).view(n_kv, S, N * G, hd)
    o = o / (a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True))
    return o.view(n_kv, S, N, G, hd).permute(1, 2, 0, 3, 4).reshape(S * N, n_heads, hd).to(s["out"].dtype)


def _plain_logprobs(s):
    x, k = s["logits"].float(), s["case"]["top"]
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    lse = m + total.log()
    logprob = x.gather(1, s["targets"].long()) - lse
    entropy = total[:, 0].log() - torch.where(e > 0, e * (x - m), 0.0).sum(-1) / total[:, 0]
    value, at = x.sort(stable=True, dim=-1, descending=True)
    return logprob, entropy, at[:, :k].int(), value[:, :k] - lse


def work(case):
    size = {"f32": 4, "f16": 2}
    if case["op"] == "logprobs":
        n, v = case["rows"], case["vocab"]
        return {"bytes": n * v * size[case["dtype"]] + n * (8 * case["targets"] + 4 + 8 * case["top"]), "flops": 6 * n * v}
    n_heads, n_kv, hd = HEADS[case["heads"]]
    rows = case["n_seqs"] * case["n_new"]
    if case["op"] == "append":
        row = (n_heads + 2 * n_kv) * hd * size[case["dtype"]] + n_heads * hd * size[case["q_out"]] + 2 * n_kv * hd * 2 + hd * 4
        return {"bytes": rows * row, "flops": rows * 3 * (n_heads + n_kv) * hd}
    # the lengths are spread evenly between n_new and max_len; a new token sees half of the new ones
    mean = (case["n_new"] + case["max_len"]) / 2
    keys = case["prefix"] + mean - (case["n_new"] - 1) / 2
    return {"bytes": (case["prefix"] + case["n_seqs"] * mean) * n_kv * hd * 4 + rows * n_heads * hd * (size[case["q"]] + size[case["out"]]),
            "flops": 4 * rows * n_heads * hd * keys}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        x = s["logits"].double()
        p = torch.softmax(x, -1)
        logp = torch.log_softmax(x, -1)
        entropy = -torch.special.xlogy(p, p).sum(-1)
        # whole numbers are held to be equal elsewhere; only computed values are given here
        top = logp.topk(case["top"], -1).values
        return logp.gather(1, s["targets"].long()), entropy, None, top
    n_heads, n_kv, hd = HEADS[case["heads"]]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    ps, n_new = case["page"], case["n_new"]
    if case["op"] == "append":
        def turn(x, pos):                                       # a complex number for each pair, times e^(i theta)
            z = torch.view_as_complex(s["cos_sin"].double()[pos])[:, None]
            x = x.double()
            pair = torch.stack([x[..., :hd // 2], x[..., hd // 2:]], -1) if case["neox"] else x.unflatten(-1, (-1, 2))
            y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            return torch.cat([y[..., 0], y[..., 1]], -1) if case["neox"] else y.flatten(-2)

        q, k, v = torch.empty_like(s["q"], dtype=torch.float64), s["k_pages"].double(), s["v_pages"].double()
        for i, n in enumerate(lens):
            e = torch.arange(n - n_new, n)
            page = torch.tensor(table[i])[e // ps].cuda()
            e, rows = e.cuda(), slice(i * n_new, (i + 1) * n_new)
            q[rows] = turn(s["q"][rows], e + case["prefix"])
            k[page, e % ps] = turn(s["k"][rows], e + case["prefix"])
            v[page, e % ps] = s["v"][rows].double()
        return q, k, v
    out = torch.empty(case["n_seqs"], n_new, n_heads, hd, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(case["n_seqs"], n_new, n_heads, hd)
    pk, pv = s["prefix_k"].double(), s["prefix_v"].double()
    for i, n in enumerate(lens):
        at = torch.tensor(table[i][:-(-n // ps)], device="cuda")
        k, v = (torch.cat([p, t[at].double().flatten(0, 1)[:n]]) for p, t in ((pk, s["k_pages"]), (pv, s["v_pages"])))
        last = len(k) - n_new + torch.arange(n_new, device="cuda")
        hidden = torch.arange(len(k), device="cuda") > last[:, None, None, None]
        x = torch.einsum("nghd,tgd->nght", q[i].unflatten(1, (n_kv, -1)), k) / math.sqrt(hd)
        w = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
        out[i] = torch.einsum("nght,tgd->nghd", w, v).flatten(1, 2)
    return out.flatten(0, 1)
