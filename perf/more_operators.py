"""More operators on the target's side of a draft-and-verify step, as cases that can be timed and compared: a paged
cache held in 8 bits (rotary append that quantises as it writes, attention of new tokens over it, reading it back),
and attention of a batch whose sequences share a prefix, which is read and multiplied once for all of them.

With `own` false, run() computes an operator in elementary torch operations; with `own` true it makes the
calls a user makes of the library. Lengths follow from the case alone, values from the seed.

8 bits: a row of K or V (one position, one KV head) is e4m3 values times 2^e, e the least whole number with
max |x| <= 448 * 2^e, at least -40; its byte in `scales` is e + 127."""
import math
import random

import torch

own = False

PAGE = 64
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the new row of one sequence: latency of the append alone
        append_case("append 8: one row", 1, 1, 2000, 32, 8, 128, "bf16", 128, False, 0),
        # the blocks of a serving batch, behind a system prompt that all its sequences share
        append_case("append 8: 32 blocks of 16", 32, 16, 4352, 32, 8, 128, "bf16", 128, False, 1000),
        # a prompt's rows, interleaved pairs on half of each head
        append_case("append 8: prompt of 8191", 1, 8191, 0, 32, 8, 128, "fp16", 64, True, 0),
        # the last window of one sequence, for a prompt chunk's attention in the caller's own code
        read_case("read: 1 x 700 of 16 bits", 1, 700, 2048, 8, 128, "fp16", 16),
        # whole ragged caches back in 16 bits, to leave the card
        read_case("read: 8 ragged of 8 bits", 8, 8192, 8192, 8, 128, "bf16", 8),
        # one decoding step of a single chat at the Qwen3-8B-shaped target, 2K of context: latency
        attend_case("attend 8: 1 x 2048, one token", 1, 1, 2048, 2048, 32, 8, 128, "bf16"),
        # one decoding step of a ragged serving batch (the batched workload's lengths)
        attend_case("attend 8: 32 ragged, one token", 32, 1, 512, 8192, 32, 8, 128, "fp16"),
        # verification of 16-token blocks at long context (the Llama-3.1-8B-shaped workload)
        attend_case("attend 8: 4 x 32768, block 16", 4, 16, 32768, 32768, 32, 8, 128, "bf16"),
        # a small target with 64-wide heads, short odd lengths and short blocks
        attend_case("attend 8: 7 short, block 5, d 64", 7, 5, 3, 517, 12, 4, 64, "bf16"),
        # one decoding step of 32 chats behind one system prompt
        shared_case("shared: 32 x 4096 + own, one token", 32, 1, 4096, 1, 700, 32, 8, 128, "bf16", 16),
        # samples of one long document, verified in blocks
        shared_case("shared: 16 x 8190 + own, block 16", 16, 16, 8190, 1, 512, 32, 8, 128, "fp16", 16),
        # the same on the 8-bit cache, with 64-wide heads and an odd group
        shared_case("shared: 9 x 2500 + own, block 5, d 64, 8 bits", 9, 5, 2500, 1, 300, 12, 4, 64, "bf16", 8),
    ]


def append_case(name, seqs, new, hi, heads, kv_heads, dim, dtype, rope, interleaved, prefix):
    return dict(name=name, op="append", seqs=seqs, new=new, lo=hi // 2, hi=hi, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                bits=8, rope=rope, interleaved=interleaved, prefix=prefix)


def read_case(name, seqs, new, hi, kv_heads, dim, dtype, bits):
    return dict(name=name, op="read", seqs=seqs, new=new, lo=hi // 2, hi=hi, heads=kv_heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                bits=bits, prefix=0)


def attend_case(name, seqs, new, lo, hi, heads, kv_heads, dim, dtype):
    return dict(name=name, op="attend", seqs=seqs, new=new, lo=lo, hi=hi, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, bits=8,
                prefix=0)


def shared_case(name, seqs, new, prefix, lo, hi, heads, kv_heads, dim, dtype, bits):
    return dict(name=name, op="shared", seqs=seqs, new=new, lo=lo, hi=hi, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, bits=bits,
                prefix=prefix)


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "shared", "shared"])
    kv, group, dim, dtype = rng.choice([1, 2, 4, 8]), rng.randint(1, 8), rng.choice([64, 128]), rng.choice(["fp16", "bf16"])
    kv = max(kv, 128 // dim)
    block = rng.choice([1, 1, 2, 3, 4, 6, 8, 11, 16])
    if op == "append":
        new = _log_int(rng, 1, 4096)
        c = append_case("", _log_int(rng, 1, max(1, 8191 // new)), new, _log_int(rng, 1, 16384), kv * min(group, 4), kv, dim, dtype,
                        16 * rng.randint(0, dim // 16), rng.random() < 0.5, rng.choice([0, _log_int(rng, 1, 4096)]))
    elif op == "read":
        hi = _log_int(rng, 1, 8192)
        c = read_case("", _log_int(rng, 1, max(1, min(64, 65536 // hi))), _log_int(rng, 1, hi), hi, kv, dim, dtype, rng.choice([8, 8, 16]))
    elif op == "attend":
        hi = _log_int(rng, 1, 32768)
        c = attend_case("", _log_int(rng, 1, max(1, min(64, 4 * 32768 // hi))), block, _log_int(rng, 1, hi), hi, kv * group, kv, dim, dtype)
    else:
        hi = _log_int(rng, 1, 1024)
        c = shared_case("", _log_int(rng, 1, 64 if block == 1 else 16), block, _log_int(rng, 1, 8192), 1, hi, kv * min(group, 4), kv, dim,
                        dtype, rng.choice([8, 16]))
    del c["name"]
    return c


def _lengths(case):
    """The lengths of the case's sequences before the new rows, and how many of those each one has."""
    r = random.Random("%(op)s %(seqs)d %(new)d %(lo)d %(hi)d" % case)
    n = case["seqs"]
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(n)]
    lens[0] = case["hi"]
    new = [case["new"] if i == 0 or r.random() < 0.75 else r.randint(1, case["new"]) for i in range(n)]
    if case["op"] == "read":  # the last positions of each cache
        new = [min(a, b) for a, b in zip(lens, new)]
    return lens, new


def _pages(n):
    return -(-n // PAGE)


# ---------------------------------------------------------------- work
def work(case):
    lens, new = _lengths(case)
    rows, nq, nkv, d, op = sum(new), case["heads"], case["kv_heads"], case["dim"], case["op"]
    row = 2 * nkv * (d + 1 if case["bits"] == 8 else 2 * d)  # of K and V in the cache, with its scales
    if op == "append":
        return {"bytes": float(rows * ((nq + 2 * nkv) * d * 2 + nq * d * 2 + row + 4 + 4 * case["rope"])),
                "flops": float(rows * ((nq + nkv) * case["rope"] * 3 + 4 * nkv * d))}
    if op == "read":
        return {"bytes": float(rows * (row + 4 * nkv * d) + 4 * sum(_pages(a) for a in lens)), "flops": float(rows * 2 * nkv * d)}
    keys = sum(a + b for a, b in zip(lens, new)) + case["prefix"]
    pairs = sum(sum(a + r + 1 + case["prefix"] for r in range(b)) for a, b in zip(lens, new))
    return {"bytes": float(keys * row + rows * nq * d * 4 + 4 * _pages(keys)), "flops": 4.0 * pairs * nq * d}


# ---------------------------------------------------------------- states
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _exponents(x):
    """The exponents of the rows x[..., d] in 8 bits."""
    m, e = torch.frexp(x.abs().amax(-1))
    # |x| <= 448 * 2^e for m * 2^e' with m in [0.5, 1): 448 is 0.875 * 2^9
    e = e - 9 + (m > 0.875)
    return torch.where(m == 0, -40, e).clamp(min=-40).to(torch.int32)


def _quantised(x):
    e = _exponents(x)
    return torch.ldexp(x, -e[..., None]).to(F8), (e + 127).to(torch.uint8)


def _paged(case, g):
    """Lengths, a page table with the pages in random order (the prefix's pages in its last row), and the slots of the new rows."""
    lens, new = _lengths(case)
    held = lens if case["op"] == "read" else [a + b for a, b in zip(lens, new)]
    need = [_pages(a) for a in held + [case["prefix"]]]
    cols, n_pages = max(need), sum(need) + 3
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    h = torch.tensor(need, device="cuda")
    j = torch.arange(cols, device="cuda")
    table = torch.where(j < h[:, None], ids[((h.cumsum(0) - h)[:, None] + j).clamp(max=n_pages - 1)], -1).to(torch.int32)
    st = {"case": case, "len": _ints(lens + [case["prefix"]]), "new": _ints(new), "table": table.contiguous(), "n_pages": n_pages}
    r = torch.arange(case["new"], device="cuda")
    first = st["len"][:-1] - (st["new"] if case["op"] == "read" else 0)
    pos = (first[:, None] + r).long()
    rows = table[:-1].gather(1, (pos // PAGE).clamp(max=cols - 1)) * PAGE + pos % PAGE
    st["slots"] = torch.where(r < st["new"][:, None], rows, -1).to(torch.int32).reshape(-1).contiguous()
    st["first"] = first.contiguous()
    return st


def _fill(case, g, st):
    """K and V of all pages: a spread of row norms, scores of a few units."""
    n, nkv, d = st["n_pages"], case["kv_heads"], case["dim"]
    for w in "kv":
        x = _randn(g, n * PAGE, nkv, d) * torch.exp2(0.3 * _randn(g, n * PAGE, nkv, 1) - (0 if w == "k" else 1.0))
        x = x.to(DTYPES[case["dtype"]])
        if case["bits"] == 8:
            x, s = _quantised(x.float())
            st["scales"][0, :, :, "kv".index(w)] = s.view(n, PAGE, nkv).transpose(1, 2)
        st[w] = x[None].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = _paged(case, g)
    op, nq, nkv, d, t = case["op"], case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    rows, pool = case["seqs"] * case["new"], (1, st["n_pages"] * PAGE, nkv, d)
    if case["bits"] == 8:
        st["scales"] = torch.zeros(1, st["n_pages"], nkv, 2, PAGE, dtype=torch.uint8, device="cuda")
    if op == "append":
        st["qkv"] = _randn(g, rows, (nq + 2 * nkv) * d).to(t)
        st["k"], st["v"] = torch.zeros(pool, device="cuda").to(F8), torch.zeros(pool, device="cuda").to(F8)
        st["q"] = torch.zeros(rows, nq, d, dtype=t, device="cuda")
        # the first row of a page that no sequence uses
        used = torch.zeros(st["n_pages"] + 1, dtype=torch.int32, device="cuda")
        used[st["table"].where(st["table"] >= 0, st["n_pages"]).long().reshape(-1)] = 1
        st["spare"] = (used.argmin() * PAGE).to(torch.int32)
        inv = 1e6 ** (-torch.arange(case["rope"] // 2, dtype=torch.float64, device="cuda") * 2 / max(1, case["rope"]))
        a = torch.arange(case["prefix"] + case["hi"] + case["new"], dtype=torch.float64, device="cuda")[:, None] * inv
        st["cos"], st["sin"] = a.cos().float().contiguous(), a.sin().float().contiguous()
    else:
        _fill(case, g, st)
        if op == "read":
            st["k_out"], st["v_out"] = (torch.zeros(rows, nkv, d, dtype=t, device="cuda") for _ in "kv")
        else:
            # query and key norms as after a trained projection: the softmax is neither flat nor one key
            st["q"] = (1.5 * _randn(g, rows, nq, d)).to(t)
            st["out"] = torch.zeros_like(st["q"])
    if own:
        st["cache"] = _cache(case, st)
    return st


def _cache(case, st):
    """What a user's program keeps: the library's page pool and cache over the state's own buffers."""
    from block_diffusion_drafter_kv_gb300 import binding as B
    pool = B.PagePool(st["n_pages"], st["table"].shape[1], case["seqs"] + 1)
    pool.page_table.copy_(st["table"])
    kw = {} if not case.get("rope") else dict(rope_cos=st["cos"], rope_sin=st["sin"], rope_interleaved=case["interleaved"])
    if case["bits"] == 8:
        kw |= dict(bits=8, scales=st["scales"])
    if case["op"] == "shared":
        kw["shared_rows"] = case["seqs"] * case["new"]
    return B.PagedCache(1, case["heads"], case["kv_heads"], case["dim"], pool, st["len"], dtype=DTYPES[case["dtype"]],
                        k_pool=st["k"], v_pool=st["v"], **kw)


# ---------------------------------------------------------------- one pass
def run(st):
    return {"append": _run_append, "read": _run_read, "attend": _run_attend, "shared": _run_attend}[st["case"]["op"]](st)


def _rotate(x, cos, sin, rope, interleaved):
    a, b = (x[..., 0:rope:2], x[..., 1:rope:2]) if interleaved else (x[..., : rope // 2], x[..., rope // 2: rope])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([y, x[..., rope:]], -1)


def _split(c, x):
    nq, nkv, d = c["heads"], c["kv_heads"], c["dim"]
    return [t.unflatten(1, (-1, d)) for t in (x[:, : nq * d], x[:, nq * d: (nq + nkv) * d], x[:, (nq + nkv) * d:])]


def _run_append(st):
    """The cache's values as e4m3 numbers, with the exponents that they are multiplied by."""
    c = st["case"]
    q, k, v = _split(c, st["qkv"])
    if own:
        st["cache"].append(0, q, k, v, st["slots"], c["seqs"], c["new"], st["q"], prefix=c["seqs"] if c["prefix"] else None)
        return {"q": st["q"], "k": st["k"], "v": st["v"], "scales": st["scales"]}
    pos = (st["len"][:-1, None] + torch.arange(c["new"], device="cuda")).reshape(-1) + c["prefix"]
    pos = pos.clamp(max=st["cos"].shape[0] - 1)
    cos, sin = st["cos"][pos][:, None], st["sin"][pos][:, None]
    there = (st["slots"] >= 0)[:, None, None]
    qr = _rotate(q.float(), cos, sin, c["rope"], c["interleaved"]).to(st["q"].dtype)
    st["q"].copy_(torch.where(there, qr, st["q"]))
    # a row without a slot writes the zeros that the spare row holds
    to = torch.where(st["slots"] >= 0, st["slots"], st["spare"]).long()
    for i, (w, x) in enumerate((("k", _rotate(k.float(), cos, sin, c["rope"], c["interleaved"])), ("v", v.float()))):
        y, e = _quantised(x)
        y = torch.where(there, y.view(torch.uint8), 0)
        st[w].view(torch.uint8)[0].index_copy_(0, to, y)
        st["scales"][0, to // PAGE, :, i, to % PAGE] = torch.where(there[:, 0], e, 0)
    return {"q": st["q"], "k": st["k"], "v": st["v"], "scales": st["scales"]}


def _held(st, w, rows):
    """Rows of K or V (any shape of indices) as the fp32 values they stand for: [...][kv head][dim]."""
    x = st[w][0].view(torch.uint8)[rows].view(F8).float() if st["case"]["bits"] == 8 else st[w][0][rows].float()
    if st["case"]["bits"] == 8:
        s = st["scales"][0, :, :, "kv".index(w)]
        x = torch.ldexp(x, s[rows // PAGE, :, rows % PAGE].to(torch.int32)[..., None] - 127)
    return x


def _run_read(st):
    c = st["case"]
    if own:
        st["cache"].read(0, st["first"], st["new"], c["seqs"], c["new"], st["k_out"], st["v_out"])
    else:
        there = (st["slots"] >= 0)[:, None, None]
        at = st["slots"].clamp(min=0).long()
        for w in "kv":
            o = st[w + "_out"]
            o.copy_(torch.where(there, _held(st, w, at).to(o.dtype), o))
    return {"k": st["k_out"], "v": st["v_out"]}


def _run_attend(st):
    c = st["case"]
    if own:
        st["cache"].attend(0, st["q"], st["new"], c["seqs"], c["new"], st["out"], prefix=c["seqs"] if c["prefix"] else None)
        return st["out"]
    n, b, nkv, d = c["seqs"], c["new"], c["kv_heads"], c["dim"]
    grp = c["heads"] // nkv
    q = st["q"].float().reshape(n, b, nkv, grp, d).permute(0, 2, 1, 3, 4).reshape(n, nkv, b * grp, d) / math.sqrt(d)
    cols = _pages(c["hi"] + b)
    rows = (st["table"][:-1, :cols].clamp(min=0).long()[:, :, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(n, -1)
    r = torch.arange(b, device="cuda")
    s = q @ _held(st, "k", rows).permute(0, 2, 3, 1)
    seen = torch.arange(rows.shape[1], device="cuda") <= st["len"][:-1, None, None] + r[:, None]
    s = s.masked_fill(~seen.repeat_interleave(grp, 1)[:, None], -math.inf)
    m = s.max(-1, keepdim=True).values
    if c["prefix"]:
        p = torch.arange(c["prefix"], device="cuda")
        rows_p = st["table"][-1].long()[p // PAGE] * PAGE + p % PAGE
        sp = q @ _held(st, "k", rows_p).permute(1, 2, 0)
        m = torch.maximum(m, sp.max(-1, keepdim=True).values)
    e = torch.exp(s - m)
    o, total = e @ _held(st, "v", rows).permute(0, 2, 1, 3), e.sum(-1, keepdim=True)
    if c["prefix"]:
        e = torch.exp(sp - m)
        o, total = o + e @ _held(st, "v", rows_p).permute(1, 0, 2), total + e.sum(-1, keepdim=True)
    o = (o / total).reshape(n, nkv, b, grp, d).permute(0, 2, 1, 3, 4).reshape(n * b, c["heads"], d)
    there = (r < st["new"][:, None]).reshape(-1, 1, 1)
    st["out"].copy_(torch.where(there, o.to(st["out"].dtype), st["out"]))
    return st["out"]


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attend": _exact_attend, "shared": _exact_attend}[case["op"]](case, st)


def _places(c, st):
    """Of every new (or read) row: its number, its sequence, its position there, its row in the cache."""
    lens, new = _lengths(c)
    at0 = [a - b if c["op"] == "read" else a for a, b in zip(lens, new)]
    table = st["table"].tolist()
    at = [(s * c["new"] + r, s, at0[s] + r) for s in range(c["seqs"]) for r in range(new[s])]
    return at, torch.tensor([table[s][p // PAGE] * PAGE + p % PAGE for _, s, p in at], device="cuda")


def _exact_append(c, st):
    at, to = _places(c, st)
    rows = torch.tensor([a[0] for a in at], device="cuda")
    pos = torch.tensor([a[2] + c["prefix"] for a in at], device="cuda", dtype=torch.float64)
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

    def e4m3(x, e):
        """x / 2^e rounded to 3 bits behind the leading one, ties to even; steps of 2^-9 below 2^-6."""
        y = x * torch.exp2(-e.double())[..., None]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(y / step) * step

    out = {"q": torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"),
           "scales": torch.zeros(st["scales"].shape, dtype=torch.uint8, device="cuda")}
    out["q"][rows] = turned(q)
    for i, (w, x) in enumerate((("k", turned(k)), ("v", v))):
        e = torch.ceil(torch.log2(x.abs().amax(-1).clamp(min=1e-300) / 448)).clamp(min=-40)
        out[w] = torch.zeros(st[w].shape, dtype=torch.float64, device="cuda")
        out[w][0, to] = e4m3(x, e)
        out["scales"][0, to // PAGE, :, i, to % PAGE] = (e + 127).to(torch.uint8)
    return out


def _values(c, st, w, at):
    x = st[w][0].double()[at] if c["bits"] == 16 else st[w][0].float()[at].double()
    if c["bits"] == 8:
        x = x * 2.0 ** (st["scales"][0, at // PAGE, :, "kv".index(w), at % PAGE].double() - 127)[..., None]
    return x


def _exact_read(c, st):
    at, to = _places(c, st)
    out = {}
    for w in "kv":
        out[w] = torch.zeros(st[w + "_out"].shape, dtype=torch.float64, device="cuda")
        out[w][torch.tensor([a[0] for a in at], device="cuda")] = _values(c, st, w, to)
    return out


def _exact_attend(c, st):
    out = torch.zeros(c["seqs"] * c["new"], c["heads"], c["dim"], dtype=torch.float64, device="cuda")
    lens, new = _lengths(c)
    grp = c["heads"] // c["kv_heads"]

    def held(s, n):
        p = torch.arange(n, device="cuda")
        at = st["table"][s].long()[p // PAGE] * PAGE + p % PAGE
        return [_values(c, st, w, at).transpose(0, 1) for w in "kv"]          # [kv head][position][dim]

    before = held(c["seqs"], c["prefix"])
    for s in range(c["seqs"]):
        k, v = (torch.cat(x, 1) for x in zip(before, held(s, lens[s] + new[s])))
        for r in range(new[s]):
            q = st["q"][s * c["new"] + r].double().reshape(c["kv_heads"], grp, c["dim"])
            m = c["prefix"] + lens[s] + r + 1
            w = torch.softmax(torch.einsum("hgd,hnd->hgn", q, k[:, :m]) * c["dim"] ** -0.5, -1)
            out[s * c["new"] + r] = torch.einsum("hgn,hnd->hgd", w, v[:, :m]).reshape(c["heads"], c["dim"])
    return out
