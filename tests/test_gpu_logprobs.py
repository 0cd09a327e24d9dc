"""Log probabilities, entropies and top alternatives against float64.

Tolerances, with c = 1 / T, d_v = c (z_v - max z), p = softmax, and a summation depth D of 16
values of a thread's batch, one add per batch (V / 4096 at most), 13 joins of threads and
warps, and up to 256 chunks: D = 300 + V / 4096 roundings of 2^-24 relative to the sum:
  log S     D 2^-24, plus the exponentials': 2^-22 each and 2^-23 |d| from their arguments,
            in the mean over p: 2^-22 + 2^-23 E|d|
  logprob   that, plus the roundings of c (z - max) and of the result: 2^-22 (|d| + |logprob| + 1)
  entropy   twice log S's (1 + E|d|), since W / S has terms p |d|"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
TOKEN = 4


@pytest.fixture(scope="module")
def make():
    from dataclasses import replace
    from block_diffusion_drafter_kv_gb300 import binding as B
    from block_diffusion_drafter_kv_gb300.build import build
    from synth import TINY
    from synth import inputs as I
    build()
    kept = {}

    def get(vocab):
        if vocab not in kept:
            s = replace(TINY, vocab=vocab)
            kept[vocab] = B.Drafter(s, I.make_weights(s, 1).to("cuda"), max_block=4, max_batch=2, kv_capacity=64)
        return kept[vocab]
    get.B = B
    return get


def call(dr, z, tokens, n, temperature=1.0, **kw):
    rows = z.shape[0]
    lp, h = torch.full((rows,), 9.0, device="cuda"), torch.full((rows,), 9.0, device="cuda")
    ids = torch.full((rows, n), -9, dtype=torch.int32, device="cuda") if n else None
    top = torch.full((rows, n), 9.0, device="cuda") if n else None
    dr.logprobs(z, tokens, None if tokens is None else lp, h, ids, top, temperature=temperature, **kw)
    return lp, h, ids, top


def reference_top(z, n):
    """The n largest, ties and -0 / +0 by the lowest index, NaN first."""
    key = torch.where(z.isnan(), torch.full_like(z, INF), z).double()
    key = key + 0.0
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    # NaN before a true +inf
    rank = torch.gather(z.isnan().int(), 1, order)
    order = torch.gather(order, 1, torch.sort(rank, dim=1, descending=True, stable=True).indices)
    return order[:, :n]


def check(z, tokens, got, n, temperature=1.0):
    lp, h, ids, top = got
    V = z.shape[1]
    d = (z.double() - z.double().amax(1, keepdim=True)) / temperature
    p = torch.softmax(d, 1)
    ln = torch.log_softmax(d, 1)
    ed = (p * torch.where(p > 0, d, 0.0).abs()).sum(1)
    depth = (300 + V / 4096) * 2.0 ** -24
    ls = depth + 2.0 ** -22 + 2.0 ** -23 * ed
    there = torch.ones(z.shape[0], dtype=torch.bool, device="cuda") if tokens is None else (tokens >= 0) & (tokens < V)
    want_h = -(p * torch.where(p > 0, ln, 0.0)).sum(1)
    assert bool(((h.double() - want_h).abs() <= 2 * ls * (1 + ed) + 2.0 ** -22 * (1 + want_h))[there].all())
    assert bool((h[~there] == 0).all())
    if tokens is not None:
        at = tokens.clamp(0, V - 1).long()[:, None]
        want, dt = ln.gather(1, at)[:, 0], d.gather(1, at)[:, 0].abs()
        ok = (lp.double() - want).abs() <= ls + 2.0 ** -22 * (dt + want.abs() + 1)
        ok |= (lp.double() == want)     # -inf
        assert bool(ok[there].all())
        assert bool((lp[~there] == 0).all())
    if n:
        order = reference_top(z, n)
        assert torch.equal(ids[there].long(), order[there])
        want, dt = ln.gather(1, order), d.gather(1, order).abs()
        ok = (top.double() - want).abs() <= ls[:, None] + 2.0 ** -22 * (dt + want.abs() + 1)
        ok |= top.double() == want
        assert bool(ok[there].all())
        assert bool((ids[~there] == -1).all()) and bool((top[~there] == 0).all())


def logits(rows, V, dtype, seed=0, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = spread * torch.randn(rows, V, generator=g, device="cuda")
    z.scatter_add_(1, torch.randint(0, V, (rows, 9), generator=g, device="cuda"), 6 + 3 * torch.randn(rows, 9, generator=g, device="cuda"))
    t = torch.where(torch.arange(rows, device="cuda") % 2 == 0, z.argmax(1), torch.randint(0, V, (rows,), generator=g, device="cuda"))
    return z.to(dtype), t.to(torch.int32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,V,n", [(1, 2, 2), (1, 1024, 32), (3, 1000, 5), (2, 4099, 20), (16, 32001, 1), (5, 151936, 20),
                                      (700, 1023, 8), (1, 151936, 32), (4097, 70, 3)])
def test_sizes_and_types(make, dtype, rows, V, n):
    z, t = logits(rows, V, dtype, seed=rows + V)
    check(z, t, call(make(V), z, t, n), n)
    assert make(V).device_error() == 0


@pytest.mark.parametrize("temperature", [0.05, 0.7, 30.0])
def test_temperature(make, temperature):
    z, t = logits(6, 5000, torch.float32, seed=3)
    check(z, t, call(make(5000), z, t, 4, temperature), 4, temperature)


def test_no_tokens_and_no_alternatives(make):
    z, t = logits(7, 5001, torch.bfloat16)
    check(z, None, call(make(5001), z, None, 6), 6)
    check(z, t, call(make(5001), z, t, 0), 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_without_a_token(make, dtype):
    """-1 skips a row, which may then hold anything; other ids outside the vocabulary set the flag."""
    V = 40000
    for rows in (9, 5000):
        z, t = logits(rows, V if rows == 9 else 128, dtype)
        dr = make(z.shape[1])
        t[1::3] = -1
        z[1::3] = NAN
        check(torch.nan_to_num(z), t, call(dr, z, t, 3), 3)
        assert dr.device_error() == 0
        for bad in (z.shape[1], -2, 2 ** 31 - 1, -2 ** 31):
            t[4] = bad
            check(torch.nan_to_num(z), t, call(dr, z, t, 3), 3)
            assert dr.device_error() == TOKEN
    check(torch.nan_to_num(z), torch.full_like(t, -1), call(dr, z, torch.full_like(t, -1), 3), 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_strides_and_alignment(make, dtype):
    """Rows of a wider buffer, from any element on."""
    V = 3001
    for off, stride in ((0, 3001), (1, 3005), (3, 3010), (5, 3008), (7, 4000)):
        buf = torch.full((6 * stride + 16,), NAN, dtype=dtype, device="cuda")
        z = torch.as_strided(buf, (6, V), (stride, 1), off)
        src, t = logits(6, V, dtype, seed=off)
        z.copy_(src)
        check(src, t, call(make(V), z, t, 5), 5)


def test_ties_go_to_the_lowest_index(make):
    V = 9000
    g = torch.Generator(device="cuda").manual_seed(1)
    cases = [torch.zeros(4, V, device="cuda"), torch.randint(0, 3, (4, V), generator=g, device="cuda").float(),
             torch.where(torch.rand(4, V, generator=g, device="cuda") < 0.5, 0.0, -0.0),
             torch.randint(-40, 40, (4, V), generator=g, device="cuda").float()]
    t = torch.tensor([0, V - 1, 17, 4000], dtype=torch.int32, device="cuda")
    for z in cases:
        for n in (1, 7, 32):
            check(z, t, call(make(V), z, t, n), n)
            check(z.bfloat16(), t, call(make(V), z.bfloat16(), t, n), n)


@pytest.mark.parametrize("V,rows", [(30000, 2), (30000, 1300)])
def test_sorted_logits(make, V, rows):
    """Ascending and descending rows, where every value is, or none is, a new best."""
    up = torch.linspace(-30, 10, V, device="cuda").expand(rows, V).contiguous()
    up[1::2] = up[1::2].flip(1)
    t = torch.full((rows,), V // 2, dtype=torch.int32, device="cuda")
    for n in (1, 20, 32):
        check(up, t, call(make(V), up, t, n), n)


@pytest.mark.parametrize("n", [8, 32])
def test_a_row_whose_late_values_count_before_a_higher_row(make, n):
    """Rows of one CTA, high after low: a low row's n-th largest stands in its last stage, where a
    warp without candidates is already at the high row."""
    V, rows = 32768, 1000
    e = torch.arange(V, device="cuda")
    owner = e // 128 % 8                       # the warp that reads it
    low = -1.0 - e.float() / V
    per = n // 8
    for w in range(1, 8):                      # all warps but 0 have their share of the largest early
        low[(owner == w).nonzero()[:per, 0]] = 10.0 + torch.arange(per, device="cuda") + 0.1 * w
    low[-700:] = torch.where(owner[-700:] > 0, 5.0 + e[-700:] % 50 / 10, low[-700:])   # the rest of them late
    z = low.expand(rows, V).contiguous()
    z[1::2] += 100.0
    t = torch.full((rows,), V - 1, dtype=torch.int32, device="cuda")
    for _ in range(5):
        check(z, t, call(make(V), z, t, n), n)


def test_one_certain_token_and_extreme_temperatures(make):
    """An entropy is not negative; the smallest and largest temperatures give the limits."""
    V = 20000
    z, t = logits(64, V, torch.float32, seed=5)
    z[torch.arange(64, device="cuda"), t.long()] = 60 + torch.arange(64, device="cuda") * 0.37
    lp, h, ids, top = call(make(V), z, t, 2)
    assert bool((h >= 0).all()) and bool((h < 1e-6).all()) and torch.equal(ids[:, 0], t)
    lp, h, ids, top = call(make(V), z, t, 2, 2.0 ** -126)
    assert bool((lp == 0).all()) and bool((h == 0).all()) and bool((top[:, 0] == 0).all()) and bool((top[:, 1] < -1e30).all())
    lp, h, ids, top = call(make(V), z, t, 2, 3e38)
    for x, want in ((lp, -math.log(V)), (h, math.log(V))):
        assert bool(((x - want).abs() < 1e-4).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_masked_logits_at_high_temperatures(make, dtype):
    """-inf stays out of a distribution that is nearly uniform."""
    V = 5000
    z, t = logits(8, V, dtype, seed=7)
    keep = torch.rand(8, V, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda") < 0.3
    keep[torch.arange(8, device="cuda"), t.long()] = True
    z = torch.where(keep, z, torch.tensor(-INF, dtype=dtype, device="cuda"))
    for temperature in (300.0, 600.0, 20000.0, 1e20, 1e30):
        check(z, t, call(make(V), z, t, 4, temperature), 4, temperature)


def test_masked_logits(make):
    """-inf masks, masks of the type's lowest value, rows with one token left, and rows with none."""
    V = 20000
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        for mask in (-INF, torch.finfo(dtype).min):
            z, t = logits(6, V, dtype, seed=2)
            keep = torch.rand(6, V, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") < 0.001
            keep[0] = False
            keep[0, 777] = True
            keep[torch.arange(6, device="cuda"), t.long()] = True
            z = torch.where(keep, z, torch.tensor(mask, dtype=dtype, device="cuda"))
            t[5] = int((~keep[5]).nonzero()[5])      # a masked token
            got = call(make(V), z, t, 8)
            check(z, t, got, 8)
            if mask == -INF:
                assert got[0][5].item() == -INF
    z, t = torch.full((2, V), -INF, device="cuda"), torch.tensor([5, 0], dtype=torch.int32, device="cuda")
    lp, h, ids, top = call(make(V), z, t, 3)
    assert lp.tolist() == [-INF] * 2 and h.tolist() == [0.0] * 2
    assert ids.tolist() == [[0, 1, 2]] * 2 and top.tolist() == [[-INF] * 3] * 2
    z = torch.full((2, V), torch.finfo(torch.float32).min, device="cuda")   # nothing but the lowest value: uniform
    lp, h, ids, top = call(make(V), z, t, 3)
    for x in (lp[0], -h[1], top[0, 2]):
        assert abs(x.item() + math.log(V)) < 1e-4
    assert ids.tolist() == [[0, 1, 2]] * 2


def test_nan_and_infinite_logits(make):
    """They show: NaN in the row's numbers, the NaN itself first among the alternatives."""
    V = 12000
    for bad in (NAN, -NAN, INF):
        z, t = logits(3, V, torch.float32)
        z[1, 9000] = bad
        lp, h, ids, top = call(make(V), z, t, 4)
        assert math.isnan(lp[1]) and math.isnan(h[1]) and bool(top[1].isnan().all())
        assert ids[1].tolist() == reference_top(z, 4)[1].tolist() and ids[1, 0] == 9000
        keep = torch.tensor([0, 2], device="cuda")
        check(z[keep], t[keep], (lp[keep], h[keep], ids[keep], top[keep]), 4)


def test_captured_replayed_and_repeated(make):
    """The same results every time, from a graph too, with the counters left at zero."""
    V = 151936
    dr = make(V)
    z, t = logits(4, V, torch.float32, seed=9)
    out = call(dr, z, t, 20)
    first = [x.clone() for x in out]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dr.logprobs(z, t, out[0], out[1], out[2], out[3])
    for _ in range(20):
        for x in out:
            x.zero_()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, out))
    z2, t2 = logits(4, V, torch.float32, seed=10)
    z.copy_(z2)
    t.copy_(t2)
    g.replay()
    check(z, t, out, 20)
    assert dr.last_launch_count() == 1


def test_two_handles_on_two_streams_at_once(make):
    """Each with its own workspace, one replaying a graph while the other is called."""
    V = (60000, 60001)
    sets = []
    for i in range(2):
        z, t = logits(40 + i, V[i], torch.float32, seed=20 + i)
        out = call(make(V[i]), z, t, 6)
        sets.append((make(V[i]), z, t, out, [x.clone() for x in out], torch.cuda.Stream()))
    torch.cuda.synchronize()
    dr, z, t, out, _, _ = sets[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dr.logprobs(z, t, *out)
    for _ in range(30):
        with torch.cuda.stream(sets[0][5]):
            for x in out:
                x.zero_()
            g.replay()
        dr1, z1, t1, out1, _, s1 = sets[1]
        with torch.cuda.stream(s1):
            for x in out1:
                x.zero_()
            dr1.logprobs(z1, t1, *out1, stream=s1)
    torch.cuda.synchronize()
    for dr, z, t, out, want, _ in sets:
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and dr.device_error() == 0


def test_bad_arguments_are_refused_before_a_launch(make):
    dr, B = make(1000), make.B
    z, t = logits(2, 1000, torch.float32)
    o = torch.zeros(2, 32, device="cuda")
    f, p = dr.L.dflash_logprobs, o.data_ptr()
    def c(logits=z.data_ptr(), dtype=B.F32, stride=1000, tokens=t.data_ptr(), rows=2, temp=1.0, n=2, lp=p, h=p, ids=p, top=p):
        return f(dr.h, logits, dtype, stride, tokens, rows, temp, n, lp, h, ids, top, None)
    for bad in (dict(logits=None), dict(logits=z.data_ptr() + 2), dict(dtype=3), dict(dtype=-1), dict(stride=999), dict(tokens=None),
                dict(lp=None), dict(h=None), dict(rows=0), dict(temp=0.0), dict(temp=-1.0), dict(temp=NAN), dict(temp=INF), dict(n=-1),
                dict(n=33), dict(ids=None), dict(top=None), dict(tokens=t.data_ptr() + 1), dict(ids=p + 2), dict(h=p + 1)):
        assert c(**bad) == -1, bad
    assert bool((o == 0).all())
    for bad in (1e-39, 2.0 ** -149):           # 1 / T overflows
        assert c(temp=bad) == -1
    tiny = make(2)
    assert tiny.L.dflash_logprobs(tiny.h, z.data_ptr(), B.F32, 2, t.data_ptr(), 2, 1.0, 3, p, p, p, p, None) == -1
