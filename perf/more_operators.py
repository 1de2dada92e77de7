"""What a batch of continuations needs around its pages: the operators that are
measured, with their plain forms.

append    rotate the new tokens' q and k, store K and V in pages of 4-bit values,
          and read the new rows back as the values that they stand for
attend    attention of every new token over a shared prefix (F16) and over its own
          sequence's pages of 4-bit values
adjust    penalties for repeated tokens, biases and masks on logits
update    sequences forked, reordered, cut and extended: page tables, counts of
          holders, and copies of the pages that two sequences would write into
compact   the pages in use moved to the front of their pool

A group of up to 32 elements of a row's head is held as sixteenths: d and m in F16 and a
number n of 4 bits for each element, which stands for the F16 nearest to d n + m.  Plain
forms compute in 32 bits, whatever the inputs' type, and round once at the end.
"""
import math

import numpy as np
import torch

own = False

# Head layouts, vocabularies and depths of the repository's own model shapes.
HEADS = {"tiny": (8, 2, 32), "stories": (6, 6, 48), "1b": (32, 8, 64), "7b": (32, 32, 128)}
LAYERS = {"tiny": 4, "stories": 6, "1b": 16, "7b": 32}
VOCABS = (32000, 128256, 151936)
TYPES = {"f32": torch.float32, "f16": torch.float16}
SIZE = {"f32": 4, "f16": 2}


def _append(name, heads, n_seqs, n_new, max_len, prefix, page, dtype, q_out, neox):
    return {"op": "append", "name": name, "heads": heads, "n_seqs": n_seqs, "n_new": n_new, "max_len": max_len,
            "prefix": prefix, "page": page, "dtype": dtype, "q_out": q_out, "neox": neox}


def _attend(name, heads, n_seqs, n_new, max_len, prefix, page, q, out):
    return {"op": "attend", "name": name, "heads": heads, "n_seqs": n_seqs, "n_new": n_new, "max_len": max_len,
            "prefix": prefix, "page": page, "q": q, "out": out}


def _adjust(name, rows, vocab, dtype, out, history, window, biases, masks, allowed):
    return {"op": "adjust", "name": name, "rows": rows, "vocab": vocab, "dtype": dtype, "out": out, "history": history,
            "window": window, "biases": biases, "masks": masks, "allowed": allowed}


def _update(name, heads, layers, n_seqs, max_len, page, kind):
    return {"op": "update", "name": name, "heads": heads, "layers": layers, "n_seqs": n_seqs, "max_len": max_len,
            "page": page, "kind": kind}


def _compact(name, heads, layers, n_seqs, max_len, page, spare):
    return {"op": "compact", "name": name, "heads": heads, "layers": layers, "n_seqs": n_seqs, "max_len": max_len,
            "page": page, "spare": spare}


def listed():
    return [
        # a decode step of 64 sequences, multi-head layout, NEOX pairs, q handed on in F16
        _append("append4-step-7b", "7b", 64, 1, 512, 2000, 32, "f32", "f16", True),
        # 16 prompts' chunks of 500 tokens each
        _append("append4-chunks", "1b", 16, 500, 900, 100, 16, "f16", "f16", False),
        # a few short continuations on the smallest model
        _attend("attend4-tiny", "tiny", 3, 1, 40, 93, 16, "f32", "f32"),
        # drafts of five tokens, verified in one step behind a prompt
        _attend("attend4-drafts", "1b", 12, 5, 3100, 2000, 16, "f32", "f32"),
        # 64 conversations of their own, nothing shared
        _attend("attend4-long", "1b", 64, 1, 8192, 0, 16, "f16", "f16"),
        # multi-head attention, head size 128: the largest cache
        _attend("attend4-7b", "7b", 32, 1, 4096, 500, 32, "f16", "f16"),
        # one sequence's next token, 300 tokens behind it
        _adjust("adjust-one", 1, 128256, "f32", "f32", 300, 0, 10, 0, 0.0),
        # answers that must follow one of eight grammars, long histories
        _adjust("adjust-batch", 256, 151936, "f32", "f32", 4000, 1024, 50, 8, 0.05),
        # four beams on the smallest model: the two best go on twice
        _update("update-beams", "tiny", 4, 4, 60, 16, "beams"),
        # 64 samples: the weak ones give way to copies of the strong ones
        _update("update-samples", "1b", 16, 64, 600, 64, "samples"),
        # a pool of a few sequences after some have ended
        _compact("compact-tiny", "tiny", 4, 8, 100, 16, 0.3),
        # a large pool to be given back in part
        _compact("compact-1b", "1b", 16, 48, 700, 16, 0.2),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "adjust", "update", "compact"])
    mine = [work(c) for c in listed() if c["op"] == op]
    top = {k: max(w[k] for w in mine) for k in ("bytes", "flops")}
    while True:
        heads, page = rng.choice(list(HEADS)), rng.choice([8, 16, 32, 64])
        if op == "append":
            n_new = rng.choice([1, 1, 2, 5, _log_int(rng, 3, 500)])
            c = _append("", heads, _log_int(rng, 1, 256), n_new, n_new + _log_int(rng, 1, 900), rng.choice([0, _log_int(rng, 10, 30000)]),
                        page, rng.choice(["f32", "f16"]), rng.choice(["f32", "f16"]), rng.random() < 0.4)
        elif op == "attend":
            n_new = rng.choice([1, 1, 1, 2, 5, 8])
            c = _attend("", heads, _log_int(rng, 1, 256), n_new, n_new + _log_int(rng, 1, 16000), rng.choice([0, 0, _log_int(rng, 50, 16000)]),
                        page, rng.choice(["f32", "f16"]), rng.choice(["f32", "f16"]))
        elif op == "adjust":
            c = _adjust("", _log_int(rng, 1, 512), rng.choice(VOCABS + (_log_int(rng, 1000, 160000),)), rng.choice(["f32", "f32", "f16"]),
                        rng.choice(["f32", "f16"]), rng.choice([0, _log_int(rng, 1, 8000)]), rng.choice([0, 0, 64, 1000]),
                        rng.choice([0, 0, 1, 30, 300]), rng.choice([0, 0, 1, 5, 20]), rng.choice([0.01, 0.3, 0.98]))
        elif op == "update":
            c = _update("", heads, rng.randint(1, LAYERS[heads]), _log_int(rng, 1, 256), _log_int(rng, 1, 2000), page,
                        rng.choice(["beams", "samples", "drafts"]))
        else:
            c = _compact("", heads, rng.randint(1, LAYERS[heads]), _log_int(rng, 1, 256), _log_int(rng, 1, 2000), page, rng.choice([0.1, 0.3, 0.7]))
        del c["name"]
        w = work(c)
        if w["flops"] <= top["flops"] and w["bytes"] <= top["bytes"] and _state_bytes(c) <= 3e9:
            return c


def _pool_pages(case):
    """Pages of a pool: every sequence at its longest has room, and something is spare."""
    return int(case["n_seqs"] * -(-(case["max_len"] + 8) // case["page"]) * (1 + case.get("spare", 0))) + 2


def _state_bytes(case):
    """What a state's pool takes."""
    if case["op"] not in ("update", "compact"):
        return 0
    _, n_kv, hd = HEADS[case["heads"]]
    return _pool_pages(case) * case["page"] * n_kv * hd * 4 * case["layers"]


def _lens(case, seed):
    """Rows behind the prefix of each sequence, ragged; the first sequence is the longest."""
    r = np.random.RandomState(seed % 2**31)
    lens = r.randint(case.get("n_new", 1), case["max_len"] + 1, case["n_seqs"])
    lens[0] = case["max_len"]
    return lens


def _table(need, seed, n_pages):
    """A table of scattered pages, -1 behind a sequence's last one."""
    order = np.random.RandomState(seed % 2**31 + 1).permutation(n_pages)
    table = np.full((len(need), int(need.max()) + 2), -1, np.int32)
    at = np.arange(table.shape[1])[None, :] < need[:, None]
    table[at] = order[:int(need.sum())]
    return torch.from_numpy(table).cuda()


def _groups(hd):
    return -(-hd // 32)


def _page_bytes(page, n_kv, hd):
    """A page of 4-bit values: [n_kv][page][hd / 2] bytes, the lower half of one first, then [n_kv][page][groups] d and m."""
    return -(-page * n_kv * (hd // 2 + 4 * _groups(hd)) // 16) * 16


def _scales(pages, page, n_kv, hd):
    """d and m in the pages: float16 [n_pages, n_kv, page, groups, 2]."""
    a, g = page * n_kv * hd // 2, _groups(hd)
    return pages[:, a:a + page * n_kv * g * 4].contiguous().view(torch.float16).view(-1, n_kv, page, g, 2)


def _pages(case, seed, gen):
    """Pages of 4-bit values as rows of normal values leave them."""
    _, n_kv, hd = HEADS[case["heads"]]
    lens, ps = _lens(case, seed), case["page"]
    need = -(-lens // ps)
    n_pages = int(need.sum()) + 3
    table = _table(need, seed, n_pages)
    kv = []
    for _ in range(2):
        t = torch.randint(0, 256, (n_pages, _page_bytes(ps, n_kv, hd)), device="cuda", dtype=torch.uint8, generator=gen)
        spread = 4.1 + 0.6 * torch.randn(n_pages, n_kv, ps, _groups(hd), device="cuda", generator=gen)
        low = -spread * (0.5 + 0.05 * torch.randn(spread.shape, device="cuda", generator=gen))
        s = torch.stack([spread.abs() / 15, low], -1).half()
        a = ps * n_kv * hd // 2
        t[:, a:a + s[0].numel() * 2] = s.view(n_pages, -1).view(torch.uint8)
        kv.append(t)
    return {"k_pages": kv[0], "v_pages": kv[1], "table": table, "lens": torch.from_numpy(lens.astype(np.int32)).cuda()}


def _pool(case, seed, gen):
    """Pages in F16 of every layer, with some pages more than the sequences hold."""
    _, n_kv, hd = HEADS[case["heads"]]
    lens, ps = _lens(case, seed), case["page"]
    need = -(-lens // ps)
    # every sequence at its longest fits
    n_pages = _pool_pages(case)
    table = _table(need, seed, n_pages)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    kv = [torch.empty(case["layers"], n_pages, ps, n_kv, hd, device="cuda", dtype=torch.float16) for _ in range(2)]
    for t in kv:
        for layer in t:
            layer.normal_(generator=gen)
    s = {"k_pages": kv[0], "v_pages": kv[1], "table": table, "refs": refs, "lens": torch.from_numpy(lens.astype(np.int32)).cuda()}
    s["k_bits"], s["v_bits"] = (t.view(torch.int16) for t in kv)
    return s


def _choice(case, seed):
    """Which sequence each one goes on from, and how many rows it then has."""
    r, n, lens = np.random.RandomState(seed % 2**31 + 2), case["n_seqs"], _lens(case, seed)
    parents = np.arange(n)
    if case["kind"] == "beams":              # the better half goes on twice, in a new order
        parents = r.permutation(np.repeat(r.permutation(n)[:(n + 1) // 2], 2)[:n])
        rows = np.minimum(lens[parents] + 1, case["max_len"] + 1)
    elif case["kind"] == "samples":          # a third gives way to copies of others; a few end
        weak = r.rand(n) < 0.33
        parents[weak] = r.randint(0, n, int(weak.sum()))
        parents[r.rand(n) < 0.05] = -1
        rows = np.where(parents < 0, 0, lens[parents] + 1)
    else:                                    # drafts refused: rows cut off, and room for the next ones
        rows = np.maximum(1, lens - r.randint(0, 9, n)) + r.randint(0, 9, n)
    return parents.astype(np.int32), rows.astype(np.int32)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "adjust":
        return _prepare_adjust(s, case, seed, gen)
    if case["op"] in ("update", "compact"):
        s.update(_pool(case, seed, gen))
        if case["op"] == "update":
            s["parents"], s["rows"] = (torch.from_numpy(t).cuda() for t in _choice(case, seed))
        else:
            s["table_out"], s["refs_out"], s["moved"] = torch.full_like(s["table"], -1), torch.empty_like(s["refs"]), torch.empty_like(s["refs"])
            s["n_live"] = torch.empty(1, dtype=torch.int32, device="cuda")
        if own:
            import llama_decode_forward_gb300 as L
            pool = L.PagePool(s["k_pages"], s["v_pages"], s["table"], s["lens"], s["refs"])
            if case["op"] == "update":
                s["plan"] = L.PagesUpdate(pool, parents=s["parents"], rows=s["rows"])
            else:
                s["plan"] = L.PagesCompact(pool, table_out=s["table_out"], refs_out=s["refs_out"], moved=s["moved"], n_live=s["n_live"])
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
        s["k_rows"], s["v_rows"] = (torch.empty(rows, n_kv, hd, device="cuda", dtype=torch.float16) for _ in range(2))
    else:
        s["q"] = torch.randn(rows, n_heads, hd, device="cuda", generator=gen).to(TYPES[case["q"]])
        s["prefix_k"], s["prefix_v"] = (torch.randn(case["prefix"], n_kv, hd, device="cuda", dtype=torch.float16, generator=gen) for _ in range(2))
        s["out"] = torch.zeros(rows, n_heads, hd, device="cuda", dtype=TYPES[case["out"]])
    if own:
        import llama_decode_forward_gb300 as L
        pages = L.PagedBatchQ4(s["k_pages"], s["v_pages"], s["table"], s["lens"], case["page"], n_kv, hd, n_new=case["n_new"],
                               prefix_len=case["prefix"])
        if case["op"] == "append":
            s["plan"] = L.KvAppend(pages, s["q"], s["k"], s["v"], s["cos_sin"], q_out=s["q_out"], rope_neox=case["neox"])
            s["back"] = L.KvRead(pages, s["k_rows"], s["v_rows"])
        else:
            s["plan"] = L.AttendBatch(pages, s["q"], s["out"], prefix_k=s["prefix_k"], prefix_v=s["prefix_v"])
    return s


def _prepare_adjust(s, case, seed, gen):
    n, v, h = case["rows"], case["vocab"], case["history"]
    r = np.random.RandomState(seed % 2**31)
    s["logits"] = torch.randn(n, v, device="cuda", generator=gen).mul_(2.5).to(TYPES[case["dtype"]])
    s["out"] = torch.empty(n, v, device="cuda", dtype=TYPES[case["out"]])
    if h:
        # text repeats itself: few tokens often, many once
        u = torch.rand(n, h, device="cuda", generator=gen, dtype=torch.float64)
        s["history"] = (v ** u - 1).int().clamp_(0, v - 1)
        s["history_lens"] = torch.from_numpy(r.randint(0, h + 1, n).astype(np.int32)).cuda()
        s["history_lens"][0] = h
        s["repetition"], s["frequency"], s["presence"] = (torch.from_numpy(r.uniform(a, b, n).astype(np.float32)).cuda()
                                                          for a, b in ((1.0, 1.5), (0.0, 0.4), (0.0, 0.8)))
    if case["biases"]:
        s["bias_ids"] = torch.randint(0, v, (n, case["biases"]), device="cuda", generator=gen, dtype=torch.int32)
        s["bias_ids"][:, -1] = torch.where(torch.rand(n, device="cuda", generator=gen) < 0.5, -1, s["bias_ids"][:, 0])
        s["bias"] = torch.randn(n, case["biases"], device="cuda", generator=gen).mul_(4)
    if case["masks"]:
        words = -(-v // 32)
        bits = torch.rand(case["masks"], words, 32, device="cuda", generator=gen) < case["allowed"]
        s["masks"] = (bits.long() << torch.arange(32, device="cuda")).sum(-1).to(torch.int32)
        s["mask_of"] = torch.from_numpy(r.randint(-1, case["masks"], n).astype(np.int32)).cuda()
    if own:
        import llama_decode_forward_gb300 as L
        names = ("history", "history_lens", "repetition", "frequency", "presence", "bias_ids", "bias", "masks", "mask_of")
        s["plan"] = L.AdjustLogits(s["logits"], s["out"], window=case["window"], **{k: s[k] for k in names if k in s})
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        state["plan"]()
        if op == "append":
            state["back"]()
            return state["q_out"], state["k_rows"], state["v_rows"]
        if op in ("attend", "adjust"):
            return state["out"]
        if op == "update":
            return tuple(state[k] for k in ("table", "lens", "refs", "k_bits", "v_bits"))
        return tuple(state[k] for k in ("table_out", "refs_out", "moved", "n_live", "k_bits", "v_bits"))
    return {"append": _plain_append, "attend": _plain_attend, "adjust": _plain_adjust, "update": _plain_update, "compact": _plain_compact}[op](state)


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


def _quantize(x):
    """n, d and m of rows [..., hd] in 32 bits: groups of 32 elements, the last one padded with its own first element."""
    hd = x.shape[-1]
    g = _groups(hd)
    pad = x[..., 32 * (g - 1):32 * (g - 1) + 1].expand(*x.shape[:-1], 32 * g - hd)
    x = torch.cat([x, pad], -1).unflatten(-1, (g, 32))
    low, high = x.amin(-1), x.amax(-1)
    d, m = ((high - low) / torch.full_like(low, 15.0)).half(), low.half()
    n = ((x - m.float()[..., None]) / d.float()[..., None]).round().clamp(0, 15)
    return torch.where(d[..., None] == 0, torch.zeros_like(n), n).flatten(-2)[..., :hd].to(torch.uint8), d, m


def _values(n, d, m):
    """The F16 values that numbers [..., hd] with d and m [..., groups] stand for."""
    hd = n.shape[-1]
    d, m = (t.float().repeat_interleave(32, -1)[..., :hd] for t in (d, m))
    return (n.float() * d + m).half()


def _plain_append(s):
    case, e = s["case"], _index(s)
    n_kv, hd = s["k"].shape[1:]
    ps, g = case["page"], _groups(hd)
    cs = s["cos_sin"][(e + case["prefix"]).flatten()][:, None]
    page, row = s["table"].long().gather(1, e // ps).flatten(), (e % ps).flatten()
    page, row, head = page[:, None, None], row[:, None, None], torch.arange(n_kv, device="cuda")[:, None]
    at = (head * ps + row) * (hd // 2) + torch.arange(hd // 2, device="cuda")
    at_scale = ps * n_kv * hd // 2 + (head * ps + row) * g * 4 + torch.arange(g * 4, device="cuda")
    back = []
    for x, pages in ((_rotate(s["k"].float(), cs, case["neox"]), s["k_pages"]), (s["v"].float(), s["v_pages"])):
        n, d, m = _quantize(x)
        pages[page, at] = n[..., 0::2] | (n[..., 1::2] << 4)
        pages[page, at_scale] = torch.stack([d, m], -1).flatten(-2).view(torch.uint8)
        back.append(_values(n, d, m))
    s["q_out"].copy_(_rotate(s["q"].float(), cs, case["neox"]))
    return s["q_out"], back[0], back[1]


def _plain_attend(s):
    case = s["case"]
    n_heads, n_kv, hd = HEADS[case["heads"]]
    S, N, P, G, ps = case["n_seqs"], case["n_new"], case["prefix"], n_heads // n_kv, case["page"]
    e = _index(s)
    # [n_kv, sequence, new token and head of the group, hd]
    q = (s["q"].float() * hd ** -0.5).view(S, N, n_kv, G, hd).permute(2, 0, 1, 3, 4).reshape(n_kv, S, N * G, hd)
    pk, pv = (t.float().permute(1, 0, 2) for t in (s["prefix_k"], s["prefix_v"]))
    at = s["table"].long().clamp(min=0)

    def rows(pages):
        b = pages[:, :ps * n_kv * hd // 2].unflatten(1, (n_kv, ps, hd // 2))
        scales = _scales(pages, ps, n_kv, hd)
        x = _values(torch.stack([b & 15, b >> 4], -1).flatten(-2), scales[..., 0], scales[..., 1])
        return x[at].permute(2, 0, 1, 3, 4).flatten(2, 3).float()                  # [n_kv, S, rows, hd]

    k, v = rows(s["k_pages"]), rows(s["v_pages"])
    seen = torch.arange(k.shape[2], device="cuda") <= e.repeat_interleave(G, 1)[:, :, None]
    a = (q @ k.transpose(-1, -2)).masked_fill_(~seen, -math.inf)
    b = (q.reshape(n_kv, S * N * G, hd) @ pk.transpose(-1, -2)).view(n_kv, S, N * G, P)
    m = a.amax(-1, keepdim=True)
    if P:
        m = torch.maximum(m, b.amax(-1, keepdim=True))
    a, b = (a - m).exp_(), (b - m).exp_()
    o = a @ v + (b.view(n_kv, S * N * G, P) @ pv).view(n_kv, S, N * G, hd)
    o = o / (a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True))
    return o.view(n_kv, S, N, G, hd).permute(1, 2, 0, 3, 4).reshape(S * N, n_heads, hd).to(s["out"].dtype)


def _plain_adjust(s):
    x, case = s["logits"].float(), s["case"]
    n, v = x.shape
    if "history" in s:
        at, lens = torch.arange(case["history"], device="cuda"), s["history_lens"][:, None]
        counted = (at < lens) & (at >= (lens - case["window"] if case["window"] else 0))
        c = torch.zeros(n, v, device="cuda").scatter_add_(1, s["history"].long(), counted.float())
        rho, f, p = (s[k][:, None] for k in ("repetition", "frequency", "presence"))
        x = torch.where(c > 0, torch.where(x > 0, x / rho, x * rho) - (f * c + p), x)
    if "bias_ids" in s:
        # of a token's entries the last one counts
        entry = torch.arange(1, case["biases"] + 1, device="cuda").expand(n, -1).where(s["bias_ids"] >= 0, 0)
        last = torch.zeros(n, v, dtype=torch.long, device="cuda").scatter_reduce_(1, s["bias_ids"].long().clamp(min=0), entry, "amax")
        x = torch.where(last > 0, x + s["bias"].gather(1, (last - 1).clamp(min=0)), x)
    if "masks" in s:
        words, at = s["masks"][s["mask_of"].long().clamp(min=0)], torch.arange(v, device="cuda")
        allowed = (words[:, at // 32] >> (at % 32)) & 1
        x = x.masked_fill((allowed == 0) & (s["mask_of"] >= 0)[:, None], -math.inf)
    return x.to(s["out"].dtype)


def _plain_update(s):
    ps, table, lens, refs = s["case"]["page"], s["table"].long(), s["lens"].long(), s["refs"].long()
    n_seqs, width = table.shape
    me, i = torch.arange(n_seqs, device="cuda"), torch.arange(width, device="cuda")[None, :]
    parent, rows = s["parents"].long(), s["rows"].long()
    keep = torch.minimum(torch.where(parent >= 0, lens[parent.clamp(min=0)], 0), rows)
    full, tail, total = keep // ps, keep % ps, -(-rows // ps)
    source = table[parent.clamp(min=0)]
    held, shared = i < -(-lens // ps)[:, None], i < full[:, None]
    refs = refs - torch.bincount(table[held], minlength=len(refs)) + torch.bincount(source[shared], minlength=len(refs))
    # a page that is kept in part stays with the first of its sequences, unless another holds all of it
    part = source.gather(1, full.clamp(max=width - 1)[:, None])[:, 0].where(tail > 0, 0)
    first = torch.full_like(refs, n_seqs).scatter_reduce_(0, part, me.where(tail > 0, n_seqs), "amin")
    stays = (tail > 0) & (refs[part] == 0) & (first[part] == me)
    refs = refs.index_add(0, part, stays.long())
    fresh = (i >= (full + stays)[:, None]) & (i < total[:, None])
    pages = (refs == 0).nonzero()[:, 0][:int(fresh.sum())]
    new = source.where(shared | ((i == full[:, None]) & stays[:, None]), table.where(~held, -1))
    new[fresh] = pages
    refs[pages] = 1
    copied = ((tail > 0) & ~stays).nonzero()[:, 0]
    to, rows_of = new[copied, full[copied]], (torch.arange(ps, device="cuda") < tail[copied][:, None])[..., None, None]
    for t in (s["k_pages"], s["v_pages"]):
        t[:, to] = torch.where(rows_of, t[:, part[copied]], t[:, to])
    s["table"].copy_(new)
    s["lens"].copy_(rows)
    s["refs"].copy_(refs)
    return tuple(s[k] for k in ("table", "lens", "refs", "k_bits", "v_bits"))


def _plain_compact(s):
    refs, at = s["refs"], torch.arange(len(s["refs"]), device="cuda")
    live = refs > 0
    n_live = live.sum()
    holes, movers = (~live & (at < n_live)).nonzero()[:, 0], (live & (at >= n_live)).nonzero()[:, 0]
    moved = at.where(live, -1)
    moved[movers] = holes
    held = torch.arange(s["table"].shape[1], device="cuda") < -(-s["lens"].long() // s["case"]["page"])[:, None]
    s["table_out"].copy_(moved[s["table"].long().clamp(min=0)].where(held, s["table_out"].long()))
    s["refs_out"].copy_(refs.where(at < n_live, 0))
    s["refs_out"][holes] = refs[movers]
    s["moved"].copy_(moved)
    s["n_live"].copy_(n_live)
    for t in (s["k_pages"], s["v_pages"]):
        t[:, holes] = t[:, movers]
    return tuple(s[k] for k in ("table_out", "refs_out", "moved", "n_live", "k_bits", "v_bits"))


def work(case):
    op = case["op"]
    if op == "adjust":
        n, v = case["rows"], case["vocab"]
        most = min(case["history"], case["window"] or case["history"])
        read = n * most * 2 + n * case["biases"] * 8 + case["masks"] * v / 8
        return {"bytes": n * v * (SIZE[case["dtype"]] + SIZE[case["out"]]) + read, "flops": 4 * n * v}
    n_heads, n_kv, hd = HEADS[case["heads"]]
    mean, ps = (case.get("n_new", 1) + case["max_len"]) / 2, case["page"]
    if op in ("update", "compact"):
        row, held = n_kv * hd * 4 * case["layers"], case["n_seqs"] * (mean / ps + 0.5)
        if op == "compact":
            # a hole for each page that lies behind the last place, which is as good as any other
            return {"bytes": held * (1 - held / _pool_pages(case)) * ps * row * 2 + held * 8, "flops": held}
        copies = {"beams": 0.5, "samples": 0.33, "drafts": 0.0}[case["kind"]] * case["n_seqs"]
        return {"bytes": copies * ps / 2 * row * 2 + held * 8, "flops": held}
    rows, own_row = case["n_seqs"] * case["n_new"], n_kv * (hd / 2 + 4 * _groups(hd)) * 2
    if op == "append":
        row = (n_heads + 2 * n_kv) * hd * SIZE[case["dtype"]] + n_heads * hd * SIZE[case["q_out"]] + 2 * own_row + 2 * n_kv * hd * 2 + hd * 4
        return {"bytes": rows * row, "flops": rows * (3 * n_heads + 12 * n_kv) * hd}
    # the lengths are spread evenly between n_new and max_len; a new token sees half of the new ones
    keys = case["prefix"] + mean - (case["n_new"] - 1) / 2
    return {"bytes": case["prefix"] * n_kv * hd * 4 + case["n_seqs"] * mean * own_row + rows * n_heads * hd * (SIZE[case["q"]] + SIZE[case["out"]]),
            "flops": 4 * rows * n_heads * hd * keys}


def exact(case, seed):
    if case["op"] in ("update", "compact"):
        return None                                             # whole numbers, and values that are moved
    s = prepare(case, seed)
    if case["op"] == "adjust":
        y = s["logits"].double()
        n, v = y.shape
        if "history" in s:
            lens = s["history_lens"].tolist()
            lists = [s["history"][r, max(0, k - case["window"]) if case["window"] else 0:k].long() for r, k in enumerate(lens)]
            times = torch.stack([torch.bincount(t, minlength=v) for t in lists]).double()
            rho, f, p = (s[k].double()[:, None] for k in ("repetition", "frequency", "presence"))
            y = torch.where(times == 0, y, torch.maximum(y, y * 0) / rho + torch.minimum(y, y * 0) * rho - f * times - p)
        for j in range(case["biases"]):                         # the entries behind j do not name its token again
            ids = s["bias_ids"][:, j].long()
            last = (ids >= 0) & ~(s["bias_ids"][:, j + 1:] == ids[:, None]).any(1)
            y.scatter_add_(1, ids.clamp(min=0)[:, None], (s["bias"][:, j].double() * last)[:, None])
        if "masks" in s:
            bits = torch.stack([(s["masks"] >> b) & 1 for b in range(32)], -1).flatten(1)[:, :v].bool()
            for r, k in enumerate(s["mask_of"].tolist()):
                if k >= 0:
                    y[r, ~bits[k]] = -math.inf
        return y
    n_heads, n_kv, hd = HEADS[case["heads"]]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    ps, n_new, g = case["page"], case["n_new"], _groups(hd)
    if case["op"] == "append":
        def turn(x, pos):                                       # a complex number for each pair, times e^(i theta)
            z = torch.view_as_complex(s["cos_sin"].double()[pos])[:, None]
            x = x.double()
            pair = torch.stack([x[..., :hd // 2], x[..., hd // 2:]], -1) if case["neox"] else x.unflatten(-1, (-1, 2))
            y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            return torch.cat([y[..., 0], y[..., 1]], -1) if case["neox"] else y.flatten(-2)

        def held(x):                                            # group by group
            for a in range(0, hd, 32):
                t = x[..., a:a + 32]
                m = t.min(-1, keepdim=True).values.half().double()
                d = ((t.max(-1, keepdim=True).values - t.min(-1, keepdim=True).values) / 15).half().double()
                x[..., a:a + 32] = m + d * torch.where(d > 0, (t - m) / d, 0.0).round().clamp(0, 15)
            return x

        pos = torch.tensor([n - n_new + i + case["prefix"] for n in lens for i in range(n_new)], device="cuda")
        return turn(s["q"], pos), held(turn(s["k"], pos)), held(s["v"].double())

    def rows(pages, at, n):                                     # a sequence's rows, [n, n_kv, hd]
        p = pages[at]
        b, sc = p[:, :ps * n_kv * hd // 2].long(), _scales(p, ps, n_kv, hd).double()
        x = torch.empty(len(at), n_kv, ps, hd, dtype=torch.float64, device="cuda")
        x[..., 0::2], x[..., 1::2] = ((t.view(len(at), n_kv, ps, hd // 2)) for t in (b % 16, b // 16))
        for k in range(g):
            x[..., 32 * k:32 * k + 32] = (x[..., 32 * k:32 * k + 32] * sc[..., k, :1] + sc[..., k, 1:]).half().double()
        return x.transpose(1, 2).flatten(0, 1)[:n]

    out = torch.empty(case["n_seqs"], n_new, n_heads, hd, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(case["n_seqs"], n_new, n_heads, hd)
    for i, n in enumerate(lens):
        at = torch.tensor(table[i][:-(-n // ps)], device="cuda")
        k, v = (torch.cat([p.double(), rows(t, at, n)]) for p, t in ((s["prefix_k"], s["k_pages"]), (s["prefix_v"], s["v_pages"])))
        last = len(k) - n_new + torch.arange(n_new, device="cuda")
        hidden = torch.arange(len(k), device="cuda") > last[:, None, None, None]
        x = torch.einsum("nghd,tgd->nght", q[i].unflatten(1, (n_kv, -1)), k) / math.sqrt(hd)
        w = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
        out[i] = torch.einsum("nght,tgd->nghd", w, v).flatten(1, 2)
    return out.flatten(0, 1)
