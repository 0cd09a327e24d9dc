"""The operators on the target's side of a draft-and-verify step, as cases that can be timed and compared:
the page pool of a paged cache, rotary positions with the cache append, attention of new tokens over the
paged cache, and log probabilities of given tokens.

With `own` false, run() computes an operator in elementary torch operations; with `own` true it makes the
calls a user makes of the library. Lengths follow from the case alone, values from the seed."""
import math
import random

import torch

own = False

PAGE = 64
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a single chat at the Qwen3-8B-shaped target, 2K of context: latency
        attend_case("attend: 1 x 2048, one token", 1, 1, 2048, 2048, 32, 8, 128, "fp16"),
        # one decoding step of a ragged serving batch (the batched workload's lengths)
        attend_case("attend: 32 ragged, one token", 32, 1, 512, 8192, 32, 8, 128, "fp16"),
        # verification of 16-token blocks at long context (the Llama-3.1-8B-shaped workload)
        attend_case("attend: 4 x 32768, block 16", 4, 16, 32768, 32768, 32, 8, 128, "bf16"),
        # a small target with 64-wide heads, short odd lengths and short blocks
        attend_case("attend: 7 short, block 5, d 64", 7, 5, 3, 517, 12, 4, 64, "bf16"),
        # the new row of one sequence: latency of the append alone
        append_case("append: one row", 1, 1, 2000, 32, 8, 128, "bf16", "fp16", 128, False),
        # the blocks of a serving batch
        append_case("append: 32 blocks of 16", 32, 16, 4352, 32, 8, 128, "bf16", "fp16", 128, False),
        # a prompt's rows, interleaved pairs on half of each head
        append_case("append: prompt of 8191", 1, 8191, 0, 32, 8, 128, "bf16", "bf16", 64, True),
        # room for the blocks of a serving batch, and back
        pages_case("pages: 32 blocks of 16", 32, 16, 512, 8192, False),
        # prompts admitted to the pool and dropped again
        pages_case("pages: 256 prompts", 256, 2048, 17, 2048, True),
        # the block that was just verified, with 20 alternatives a token
        logprobs_case("logprobs: block of 16, top 20", 16, 151936, "fp32", 20, False),
        # a serving batch's blocks, rows behind the accepted prefix left out
        logprobs_case("logprobs: 32 blocks, top 5", 512, 151936, "fp32", 5, True),
        # scoring a prompt from half-precision logits, without alternatives; an odd vocabulary
        logprobs_case("logprobs: prompt of 1000", 1000, 50257, "bf16", 0, False),
    ]


def attend_case(name, seqs, new, lo, hi, heads, kv_heads, dim, dtype):
    return dict(name=name, op="attend", seqs=seqs, new=new, lo=lo, hi=hi, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype)


def append_case(name, seqs, new, hi, heads, kv_heads, dim, x, dtype, rope, interleaved):
    return dict(name=name, op="append", seqs=seqs, new=new, lo=hi // 2, hi=hi, heads=heads, kv_heads=kv_heads, dim=dim, x=x,
                dtype=dtype, rope=rope, interleaved=interleaved)


def pages_case(name, seqs, new, lo, hi, admit):
    return dict(name=name, op="pages", seqs=seqs, new=new, lo=lo, hi=hi, admit=admit)


def logprobs_case(name, rows, vocab, dtype, top, committed):
    return dict(name=name, op="logprobs", rows=rows, vocab=vocab, dtype=dtype, top=top, committed=committed, temperature=1.0)


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "append", "pages", "logprobs"])
    kv, group, dim = rng.choice([1, 2, 4, 8]), rng.randint(1, 8), rng.choice([64, 128])
    kv = max(kv, 128 // dim)
    if op == "attend":
        hi = _log_int(rng, 1, 32768)
        seqs = _log_int(rng, 1, max(1, min(64, 4 * 32768 // hi)))
        c = attend_case("", seqs, rng.choice([1, 1, 2, 3, 4, 6, 8, 11, 16]), _log_int(rng, 1, hi), hi, kv * group, kv, dim,
                        rng.choice(["fp16", "bf16"]))
    elif op == "append":
        new = _log_int(rng, 1, 4096)
        c = append_case("", _log_int(rng, 1, max(1, 8191 // new)), new, _log_int(rng, 1, 16384), kv * min(group, 4), kv, dim,
                        rng.choice(["fp16", "bf16"]), rng.choice(["fp16", "bf16"]), 16 * rng.randint(0, dim // 16),
                        rng.random() < 0.5)
    elif op == "pages":
        admit = rng.random() < 0.5
        hi = _log_int(rng, 1, 2048 if admit else 8192)
        c = pages_case("", _log_int(rng, 1, 256), hi if admit else rng.randint(1, 16), _log_int(rng, 1, hi), hi, admit)
    else:
        vocab = _log_int(rng, 1000, 151936)
        c = logprobs_case("", _log_int(rng, 1, 512), vocab, rng.choice(["fp32", "bf16", "fp16"]), rng.choice([0, 1, 5, 20, 32]),
                          rng.random() < 0.5)
        c["temperature"] = rng.choice([1.0, 0.7, 1.3])
    del c["name"]
    return c


def _lengths(case):
    """The lengths of the case's sequences before the new rows, and how many of those each one has."""
    r = random.Random("%(op)s %(seqs)d %(new)d %(lo)d %(hi)d" % case)
    n = case["seqs"]
    if case["op"] == "pages" and case["admit"]:
        return [0] * n, [r.randint(case["lo"], case["hi"]) for _ in range(n)]
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(n)]
    lens[0] = case["hi"]
    new = [case["new"] if i == 0 or r.random() < 0.75 else r.randint(1, case["new"]) for i in range(n)]
    return lens, new


def _pages(n):
    return -(-n // PAGE)


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "logprobs":
        size = 4 if case["dtype"] == "fp32" else 2
        rows = sum(t >= 0 for t in _committed(case))
        return {"bytes": float(rows * case["vocab"] * size + case["rows"] * (12 + 8 * case["top"])), "flops": 6.0 * rows * case["vocab"]}
    lens, new = _lengths(case)
    rows = sum(new)
    if op == "pages":
        held = 0 if case["admit"] else sum(map(_pages, lens))
        moved = sum(_pages(a + b) for a, b in zip(lens, new)) - held
        # slots and table entries written, list entries read; entries and list written back; per-sequence state
        return {"bytes": float(4 * case["seqs"] * case["new"] + 4 * 4 * moved + 4 * 7 * case["seqs"]), "flops": 0.0}
    nq, nkv, d = case["heads"], case["kv_heads"], case["dim"]
    if op == "append":
        return {"bytes": float(rows * ((nq + 2 * nkv) * d * 4 + 4 + 4 * case["rope"])), "flops": float(rows * (nq + nkv) * case["rope"] * 3)}
    keys = sum(a + b for a, b in zip(lens, new))
    pairs = sum(sum(a + r + 1 for r in range(b)) for a, b in zip(lens, new))
    return {"bytes": float(keys * nkv * d * 4 + rows * nq * d * 4 + 4 * _pages(keys)), "flops": 4.0 * pairs * nq * d}


# ---------------------------------------------------------------- states
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"attend": _prepare_attend, "append": _prepare_append, "pages": _prepare_pages, "logprobs": _prepare_logprobs}[case["op"]](case, g)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _randn(g, dtype, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _paged(case, g):
    """Lengths, a page table with the pages in random order, and the slots of the new rows."""
    lens, new = _lengths(case)
    need = [_pages(a + b) for a, b in zip(lens, new)]
    cols, n_pages = max(need), sum(need) + 3
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    held = torch.tensor(need, device="cuda")
    j = torch.arange(cols, device="cuda")
    table = torch.where(j < held[:, None], ids[((held.cumsum(0) - held)[:, None] + j).clamp(max=n_pages - 1)], -1).to(torch.int32)
    ln, nn = _ints(lens), _ints(new)
    r = torch.arange(case["new"], device="cuda")
    pos = (ln[:, None] + r).long()
    rows = table.gather(1, (pos // PAGE).clamp(max=cols - 1)) * PAGE + pos % PAGE
    slots = torch.where(r < nn[:, None], rows, -1).to(torch.int32).reshape(-1).contiguous()
    return ln, nn, table.contiguous(), slots, n_pages


def _cache(case, st, rope=None):
    """What a user's program keeps: the library's page pool and cache over the state's own buffers."""
    from block_diffusion_drafter_kv_gb300 import binding as B
    pool = B.PagePool(st["n_pages"], st["table"].shape[1], case["seqs"])
    pool.page_table.copy_(st["table"])
    kw = {} if rope is None else dict(rope_cos=rope[0], rope_sin=rope[1], rope_interleaved=case["interleaved"])
    return B.PagedCache(1, case["heads"], case["kv_heads"], case["dim"], pool, st["len"], dtype=DTYPES[case["dtype"]],
                        k_pool=st["k"], v_pool=st["v"], **kw)


def _prepare_attend(case, g):
    st = {"case": case}
    st["len"], st["new"], st["table"], _, st["n_pages"] = _paged(case, g)
    t = DTYPES[case["dtype"]]
    rows = case["seqs"] * case["new"]
    # query and key norms as after a trained projection: scores of a few units, so that the softmax is neither flat nor one key
    st["k"] = _randn(g, t, 1, st["n_pages"] * PAGE, case["kv_heads"], case["dim"])
    st["v"] = _randn(g, t, 1, st["n_pages"] * PAGE, case["kv_heads"], case["dim"])
    st["q"] = (1.5 * _randn(g, torch.float32, rows, case["heads"], case["dim"])).to(t)
    st["out"] = torch.zeros_like(st["q"])
    if own:
        st["cache"] = _cache(case, st)
    return st


def _angles(case, n):
    inv = 1e6 ** (-torch.arange(case["rope"] // 2, dtype=torch.float64, device="cuda") * 2 / max(1, case["rope"]))
    return torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv


def _prepare_append(case, g):
    st = {"case": case}
    st["len"], st["new"], st["table"], st["slots"], st["n_pages"] = _paged(case, g)
    nq, nkv, d, rows = case["heads"], case["kv_heads"], case["dim"], case["seqs"] * case["new"]
    t = DTYPES[case["dtype"]]
    st["qkv"] = _randn(g, DTYPES[case["x"]], rows, (nq + 2 * nkv) * d)
    st["k"] = torch.zeros(1, st["n_pages"] * PAGE, nkv, d, dtype=t, device="cuda")
    st["v"] = torch.zeros_like(st["k"])
    st["q"] = torch.zeros(rows, nq, d, dtype=t, device="cuda")
    # the first row of a page that no sequence uses
    used = torch.zeros(st["n_pages"] + 1, dtype=torch.int32, device="cuda")
    used[st["table"].where(st["table"] >= 0, st["n_pages"]).long().reshape(-1)] = 1
    st["spare"] = (used.argmin() * PAGE).to(torch.int32)
    a = _angles(case, st["table"].shape[1] * PAGE)
    st["cos"], st["sin"] = a.cos().float().contiguous(), a.sin().float().contiguous()
    if own:
        st["cache"] = _cache(case, st, (st["cos"], st["sin"]) if case["rope"] else None)
    return st


def _prepare_pages(case, g):
    lens, new = _lengths(case)
    held = [0] * len(lens) if case["admit"] else list(map(_pages, lens))
    cols = max(_pages(a + b) for a, b in zip(lens, new))
    n_pages = sum(_pages(a + b) for a, b in zip(lens, new)) + 5
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    h, j = torch.tensor(held, device="cuda"), torch.arange(cols, device="cuda")
    n_free = n_pages - sum(held)
    table = torch.where(j < h[:, None], ids[(n_free + (h.cumsum(0) - h)[:, None] + j).clamp(max=n_pages - 1)], -1).to(torch.int32)
    st = {"case": case, "len": _ints(lens), "new": _ints(new), "slots": torch.full((case["seqs"] * case["new"],), -1, dtype=torch.int32, device="cuda")}
    st["table"], st["held"], st["free"], st["n_free"] = table.contiguous(), h.to(torch.int32), ids, _ints([n_free])
    if own:
        from block_diffusion_drafter_kv_gb300 import binding as B
        p = st["pool"] = B.PagePool(n_pages, cols, case["seqs"])
        p.page_table.copy_(st["table"])
        p.held.copy_(st["held"])
        p.free_list.copy_(st["free"])
        p.n_free.copy_(st["n_free"])
    return st


def _committed(case):
    """Which rows have a token: all of them, or an accepted prefix of each block of 16."""
    r = random.Random("%(rows)d %(vocab)d" % case)
    n, kept = case["rows"], []
    while len(kept) < n:
        tau = r.randint(1, 16) if case["committed"] else 16
        kept += [0] * tau + [-1] * (16 - tau)
    return kept[:n]


def _prepare_logprobs(case, g):
    rows, vocab, t = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    # a wide bulk with a few raised tokens in each row, as a language model's output has
    z = 2.0 * torch.randn(rows, vocab, generator=g, device="cuda")
    z.scatter_add_(1, torch.randint(0, vocab, (rows, 24), generator=g, device="cuda"), 8.0 + 3.0 * torch.randn(rows, 24, generator=g, device="cuda"))
    tokens = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.8, z.argmax(1), torch.randint(0, vocab, (rows,), generator=g, device="cuda"))
    kept = _ints(_committed(case))
    st = {"case": case, "logits": z.to(t), "tokens": torch.where(kept < 0, -1, tokens).to(torch.int32)}
    st["lp"], st["entropy"] = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    st["ids"] = torch.zeros(rows, case["top"], dtype=torch.int32, device="cuda")
    st["top"] = torch.zeros(rows, case["top"], device="cuda")
    if own:
        st["drafter"] = _drafter(vocab)
    return st


def _drafter(vocab):
    """The drafter that a user's program has bound; a small one, since only its vocabulary counts here."""
    from dataclasses import replace
    from types import SimpleNamespace

    from block_diffusion_drafter_kv_gb300 import binding as B
    from synth import TINY
    s = replace(TINY, vocab=vocab)
    z = lambda *n: torch.zeros(*n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    layer = lambda: SimpleNamespace(  # noqa: E731
        wq=z(s.n_heads * s.head_dim, s.hidden), wk=z(s.n_kv_heads * s.head_dim, s.hidden), wv=z(s.n_kv_heads * s.head_dim, s.hidden),
        wo=z(s.hidden, s.n_heads * s.head_dim), w_gate=z(s.intermediate, s.hidden), w_up=z(s.intermediate, s.hidden),
        w_down=z(s.hidden, s.intermediate), g_attn=z(s.hidden), g_mlp=z(s.hidden))
    w = SimpleNamespace(w_fc=z(s.hidden, s.n_taps * s.target_hidden), g_ctx=z(s.hidden), embed=z(vocab, s.hidden), mask_emb=z(s.hidden),
                        g_final=z(s.hidden), lm_head=z(vocab, s.hidden), layers=[layer() for _ in range(s.n_layers)])
    return B.Drafter(s, w, max_block=16, max_batch=1, kv_capacity=64)


# ---------------------------------------------------------------- one pass
def run(st):
    return {"attend": _run_attend, "append": _run_append, "pages": _run_pages, "logprobs": _run_logprobs}[st["case"]["op"]](st)


def _run_attend(st):
    c = st["case"]
    if own:
        st["cache"].attend(0, st["q"], st["new"], c["seqs"], c["new"], st["out"])
        return st["out"]
    n, b, nkv, d = c["seqs"], c["new"], c["kv_heads"], c["dim"]
    grp = c["heads"] // nkv
    rows = (st["table"].clamp(min=0).long()[:, :, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(n, -1)
    k = st["k"][0][rows].float().permute(0, 2, 3, 1)
    q = st["q"].float().reshape(n, b, nkv, grp, d).permute(0, 2, 1, 3, 4).reshape(n, nkv, b * grp, d)
    s = (q @ k) / math.sqrt(d)
    r = torch.arange(b, device="cuda")
    seen = torch.arange(rows.shape[1], device="cuda") <= st["len"][:, None, None] + r[:, None]
    s = s.masked_fill(~seen.repeat_interleave(grp, 1)[:, None], -math.inf)
    e = torch.exp(s - s.max(-1, keepdim=True).values)
    o = (e @ st["v"][0][rows].float().permute(0, 2, 1, 3)) / e.sum(-1, keepdim=True)
    o = o.reshape(n, nkv, b, grp, d).permute(0, 2, 1, 3, 4).reshape(n * b, c["heads"], d)
    there = (r < st["new"][:, None]).reshape(-1, 1, 1)
    st["out"].copy_(torch.where(there, o.to(st["out"].dtype), st["out"]))
    return st["out"]


def _rotate(x, cos, sin, rope, interleaved):
    a, b = (x[..., 0:rope:2], x[..., 1:rope:2]) if interleaved else (x[..., : rope // 2], x[..., rope // 2: rope])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([y, x[..., rope:]], -1)


def _split(c, x):
    nq, nkv, d = c["heads"], c["kv_heads"], c["dim"]
    return [t.unflatten(1, (-1, d)) for t in (x[:, : nq * d], x[:, nq * d: (nq + nkv) * d], x[:, (nq + nkv) * d:])]


def _run_append(st):
    c = st["case"]
    q, k, v = _split(c, st["qkv"])
    if own:
        st["cache"].append(0, q, k, v, st["slots"], c["seqs"], c["new"], st["q"])
        return {"q": st["q"], "k": st["k"], "v": st["v"]}
    pos = (st["len"][:, None] + torch.arange(c["new"], device="cuda")).reshape(-1).clamp(max=st["cos"].shape[0] - 1)
    cos, sin = st["cos"][pos][:, None], st["sin"][pos][:, None]
    there = (st["slots"] >= 0)[:, None, None]
    qr = _rotate(q.float(), cos, sin, c["rope"], c["interleaved"]).to(st["q"].dtype)
    st["q"].copy_(torch.where(there, qr, st["q"]))
    kr = _rotate(k.float(), cos, sin, c["rope"], c["interleaved"]).to(st["k"].dtype)
    # a row without a slot writes the zero that the spare row holds
    to = torch.where(st["slots"] >= 0, st["slots"], st["spare"]).long()
    st["k"][0].index_copy_(0, to, torch.where(there, kr, 0))
    st["v"][0].index_copy_(0, to, torch.where(there, v.float().to(st["v"].dtype), 0))
    return {"q": st["q"], "k": st["k"], "v": st["v"]}


def _run_pages(st):
    c = st["case"]
    if own:
        p = st["pool"]
        p.reserve(st["len"], st["new"], c["new"], c["seqs"], st["slots"])
        p.release(st["len"], c["seqs"])
        return {"slots": st["slots"], "table": p.page_table, "held": p.held, "free": p.free_list, "n_free": p.n_free}
    ln, nn, table, held, free, n_free = st["len"], st["new"], st["table"], st["held"], st["free"], st["n_free"]
    cols, j = table.shape[1], torch.arange(table.shape[1], device="cuda")
    need = (ln + nn + PAGE - 1) // PAGE
    bad = (need > cols) | (nn > c["new"])
    add = torch.where(bad, 0, (need - held).clamp(min=0))
    upto = add.cumsum(0)
    ok = ~bad & ((upto <= n_free) | (add == 0))
    rank = (upto - add - held)[:, None] + j
    fresh = ok[:, None] & (j >= held[:, None]) & (j < need[:, None])
    table.copy_(torch.where(fresh, free[(n_free - 1 - rank).clamp(0, free.numel() - 1).long()], table))
    n_free.sub_(torch.where(ok, add, 0).sum())
    held.copy_(torch.where(ok, torch.maximum(held, need), held))
    r = torch.arange(c["new"], device="cuda")
    pos = ln[:, None] + r
    at = table.gather(1, (pos // PAGE).clamp(max=cols - 1).long()) * PAGE + pos % PAGE
    st["slots"].copy_(torch.where(ok[:, None] & (r < nn[:, None]), at, -1).reshape(-1))
    # and back: pages past the length, the last one first
    keep = (ln + PAGE - 1) // PAGE
    drop = (held - keep).clamp(min=0)
    total = drop.sum()
    rank = (drop.cumsum(0) - drop - keep)[:, None] + j
    back = (j >= keep[:, None]) & (j < held[:, None])
    more = torch.cat([free, free[:1]])
    more[torch.where(back, n_free + total - 1 - rank, free.numel()).long().reshape(-1)] = table.reshape(-1)
    free.copy_(more[:-1])
    table.copy_(torch.where(back, -1, table))
    n_free.add_(total)
    held.copy_(torch.minimum(held, keep))
    return {"slots": st["slots"], "table": table, "held": held, "free": free, "n_free": n_free}


def _run_logprobs(st):
    c = st["case"]
    if own:
        top = (st["ids"], st["top"]) if c["top"] else (None, None)
        st["drafter"].logprobs(st["logits"], st["tokens"], st["lp"], st["entropy"], *top, temperature=c["temperature"])
        return {"lp": st["lp"], "entropy": st["entropy"], "ids": st["ids"], "top": st["top"]}
    z = st["logits"].float() / c["temperature"]
    m = z.max(1, keepdim=True).values
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + total.log()
    there = st["tokens"] >= 0
    lp = z.gather(1, st["tokens"].clamp(min=0).long()[:, None]) - lse
    h = total.log()[:, 0] - (e * (z - m)).sum(1) / total[:, 0]
    st["lp"].copy_(torch.where(there, lp[:, 0], 0))
    st["entropy"].copy_(torch.where(there, h, 0))
    if c["top"]:
        v, i = torch.sort(st["logits"], dim=1, descending=True, stable=True)
        st["ids"].copy_(torch.where(there[:, None], i[:, : c["top"]], -1))
        st["top"].copy_(torch.where(there[:, None], v[:, : c["top"]].float() / c["temperature"] - lse, 0))
    return {"lp": st["lp"], "entropy": st["entropy"], "ids": st["ids"], "top": st["top"]}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "pages": _exact_pages, "logprobs": _exact_logprobs}[case["op"]](case, st)


def _exact_attend(c, st):
    out = torch.zeros(c["seqs"] * c["new"], c["heads"], c["dim"], dtype=torch.float64, device="cuda")
    lens, new = _lengths(c)
    grp = c["heads"] // c["kv_heads"]
    for s in range(c["seqs"]):
        n = lens[s] + new[s]
        p = torch.arange(n, device="cuda")
        at = st["table"][s].long()[p // PAGE] * PAGE + p % PAGE
        k, v = (st[w][0][at].double().transpose(0, 1) for w in "kv")          # [kv head][position][dim]
        for r in range(new[s]):
            q = st["q"][s * c["new"] + r].double().reshape(c["kv_heads"], grp, c["dim"])
            m = lens[s] + r + 1
            w = torch.softmax(torch.einsum("hgd,hnd->hgn", q, k[:, :m]) * c["dim"] ** -0.5, -1)
            out[s * c["new"] + r] = torch.einsum("hgn,hnd->hgd", w, v[:, :m]).reshape(c["heads"], c["dim"])
    return out


def _exact_append(c, st):
    lens, new = _lengths(c)
    rows = torch.tensor([s * c["new"] + r for s in range(c["seqs"]) for r in range(new[s])], device="cuda")
    pos = torch.tensor([lens[s] + r for s in range(c["seqs"]) for r in range(new[s])], device="cuda", dtype=torch.float64)
    seq = rows // c["new"]
    at = st["table"].long()[seq, (pos // PAGE).long()] * PAGE + (pos % PAGE).long()
    q, k, v = (t[rows].double() for t in _split(c, st["qkv"]))
    half = c["rope"] // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       pos[:, None] * 1e6 ** (-2.0 * torch.arange(half, device="cuda", dtype=torch.float64) / max(1, c["rope"])))[:, None]

    def turned(x):
        first, second = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if c["interleaved"] else (x[..., :half], x[..., half:2 * half])
        z = torch.complex(first, second) * turn
        y = x.clone()
        if c["interleaved"]:
            y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
        else:
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        return y

    out = {"q": torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"), "k": torch.zeros(st["k"].shape, dtype=torch.float64, device="cuda")}
    out["v"] = torch.zeros_like(out["k"])
    out["q"][rows], out["k"][0, at], out["v"][0, at] = turned(q), turned(k), v
    return out


def _exact_pages(c, st):
    lens, new = _lengths(c)
    table, held, free = st["table"].tolist(), st["held"].tolist(), st["free"].tolist()
    stack, slots, top = free[: int(st["n_free"])], [], int(st["n_free"])
    for s, row in enumerate(table):
        while held[s] < _pages(lens[s] + new[s]):
            row[held[s]] = stack.pop()
            held[s] += 1
        slots += [row[p // PAGE] * PAGE + p % PAGE for p in range(lens[s], lens[s] + new[s])] + [-1] * (c["new"] - new[s])
    gone = []
    for s, row in enumerate(table):
        keep = _pages(lens[s])
        gone += row[keep: held[s]]
        row[keep: held[s]] = [-1] * (held[s] - keep)
        held[s] = keep
    stack += gone[::-1]
    assert len(stack) == top
    as_int = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"slots": as_int(slots), "table": as_int(table), "held": as_int(held), "free": as_int(stack + free[top:]), "n_free": as_int([top])}


def _exact_logprobs(c, st):
    z = st["logits"].double() / c["temperature"]
    lsm = torch.log_softmax(z, 1)
    there = st["tokens"] >= 0
    lp = torch.where(there, lsm.gather(1, st["tokens"].clamp(min=0).long()[:, None])[:, 0], 0.0)
    h = torch.where(there, -(lsm.exp() * lsm).sum(1), 0.0)
    v = torch.topk(lsm, c["top"], 1).values if c["top"] else lsm[:, :0]
    return {"lp": lp, "entropy": h, "ids": None, "top": torch.where(there[:, None], v, 0.0)}
