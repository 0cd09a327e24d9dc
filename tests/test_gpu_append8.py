"""Rotary append into an 8-bit cache, and reading caches back, against their definitions in 64 bits.

A stored value stands for y + error, y the rotated one: three fp32 roundings of terms of at most |a| + |b|
(2^-22 of them), then half a step of e4m3: 2^-4 |y|, and 2^-10 2^e below its normal range. A scale is
that of the 64-bit maximum unless this lies within 2^-21 of a border between two scales."""
import pytest
import torch

from cache_cases import CAP, F8, HALF, INF, NAN, Case as AttendCase, ints, quantised
from test_gpu_append import rotated

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


class Case:
    def __init__(self, B, nq, nkv, d, x, y, rope, interleaved, lens, news, rows, prefix=None, seed=0, pad=0, layers=1, layer=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dims, self.rows, self.batch, self.layer, self.prefix = (nq, nkv, d), rows, len(lens), layer, prefix
        cols = max(-(-(a + rows) // 64) for a in list(lens) + [prefix or 0])
        self.pool = B.PagePool(cols * (self.batch + 1) + 2, cols, self.batch + 1)
        self.len, self.new = ints(list(lens) + [prefix or 0]), ints(news)
        self.slots = torch.empty(self.batch * rows, dtype=torch.int32, device="cuda")
        self.pool.reserve(self.len, self.new, rows, self.batch, self.slots)
        self.cos, self.sin = B.rope_tables(2 * cols * 64, rope, 1e4) if rope else (None, None)
        self.interleaved = interleaved
        self.cache = B.PagedCache(layers, nq, nkv, d, self.pool, self.len, dtype=y, rope_cos=self.cos, rope_sin=self.sin,
                                  rope_interleaved=interleaved, bits=8)
        self.cache.k_pool.view(torch.uint8).fill_(7)
        self.cache.v_pool.view(torch.uint8).fill_(9)
        self.cache.scales.fill_(11)
        n = self.batch * rows
        self.qkv = (torch.randn(n, (nq + 2 * nkv) * d + pad, generator=g, device="cuda")
                    * torch.exp2(2 * torch.randn(n, 1, generator=g, device="cuda"))).to(x)
        self.q_out = torch.full((n, nq, d), 3.0, dtype=y, device="cuda")

    def parts(self):
        nq, nkv, d = self.dims
        return self.qkv[:, : nq * d], self.qkv[:, nq * d: (nq + nkv) * d], self.qkv[:, (nq + nkv) * d: (nq + 2 * nkv) * d]

    def append(self, **kw):
        q, k, v = self.parts()
        self.cache.append(self.layer, q, k, v, self.slots, self.batch, self.rows, self.q_out,
                          prefix=None if self.prefix is None else self.batch, **kw)

    def check(self):
        nq, nkv, d = self.dims
        there = (self.slots >= 0).nonzero()[:, 0]
        at = self.slots[there].long()
        pos = ((self.prefix or 0) + self.len[: self.batch].long()[:, None] + torch.arange(self.rows, device="cuda")).reshape(-1)[there]
        q, k, v = (t.reshape(t.shape[0], -1, d)[there].double() for t in self.parts())
        cos, sin = (self.cos[pos], self.sin[pos]) if self.cos is not None else [torch.zeros(len(there), 0, device="cuda")] * 2
        y, size = rotated(q, cos, sin, self.interleaved)
        got = self.q_out[there].double()
        assert bool(((got - y).abs() <= 2.0 ** -22 * size + HALF[self.q_out.dtype] * y.abs() + 2.0 ** -25).all())
        assert bool((self.q_out[(self.slots < 0)] == 3).all())
        for i, (pool, (y, size)) in enumerate(((self.cache.k_pool, rotated(k, cos, sin, self.interleaved)), (self.cache.v_pool, (v, v.abs())))):
            raw = pool.view(torch.uint8)[self.layer]
            b = self.cache.scales[self.layer, at // 64, :, i, at % 64].double()
            top = y.abs().amax(-1)
            want = [torch.ceil(torch.log2((top * f).clamp(min=1e-300) / 448)).clamp(min=-40) + 127 for f in (1 - 2.0 ** -21, 1 + 2.0 ** -21)]
            assert bool(((b >= want[0]) & (b <= want[1])).all())
            f = torch.exp2(b - 127)[..., None]
            got = raw[at].view(F8).float().double() * f
            assert bool(((got - y).abs() <= 2.0 ** -22 * size + 2.0 ** -4 * y.abs() + 2.0 ** -10 * f).all())
            rest = torch.ones(raw.shape[0], dtype=torch.bool, device="cuda")
            rest[at] = False
            assert bool((raw[rest] == (7, 9)[i]).all())
            assert bool((self.cache.scales[self.layer].permute(0, 3, 1, 2).reshape(-1, nkv, 2)[rest][..., i] == 11).all())


@pytest.mark.parametrize("x", TYPES)
@pytest.mark.parametrize("y", TYPES)
@pytest.mark.parametrize("nq,nkv,d,rope,interleaved", [(8, 2, 128, 128, False), (8, 2, 128, 64, True), (3, 3, 128, 32, False), (12, 4, 64, 64, False),
                                                       (4, 2, 64, 16, True), (2, 1, 128, 0, False), (5, 1, 64, 48, False), (32, 8, 128, 128, True)])
def test_types_heads_and_rotations(B, x, y, nq, nkv, d, rope, interleaved):
    c = Case(B, nq, nkv, d, x, y, rope, interleaved, [0, 63, 64, 200], [5, 5, 0, 3], 5, seed=nq + d + rope, pad=8)
    c.append()
    c.check()
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("lens,rows", [([0], 1), ([70], 1), ([0], 3000), ([n for n in range(300)], 4)])
def test_one_row_a_prompt_and_many(B, lens, rows):
    c = Case(B, 4, 2, 128, torch.bfloat16, torch.bfloat16, 128, False, lens, [rows] * len(lens), rows, seed=rows, layers=2, layer=1)
    c.append()
    c.check()


@pytest.mark.parametrize("prefix", [0, 1, 64, 1000])
def test_positions_behind_a_prefix(B, prefix):
    c = Case(B, 4, 2, 64, torch.float16, torch.bfloat16, 64, False, [0, 9, 100], [3, 2, 3], 3, prefix=prefix, seed=prefix)
    c.append()
    c.check()
    assert c.cache.device_error() == 0


def test_sixteen_bits_behind_a_prefix(B):
    """The 16-bit append with the same offset: equal to a plain one at lengths that include the prefix."""
    from test_gpu_append import Case as Plain
    outs = []
    for lens, prefix in (([100, 140], None), ([0, 40], 100)):
        c = Plain(B, 4, 2, 64, torch.bfloat16, torch.float16, 64, False, lens, [3, 3], 3, seed=4)
        if prefix:
            length = ints(lens + [prefix])
            cos, sin = B.rope_tables(256, 64, 1e4)
            pool = B.PagePool(8, 4, 3)
            pool.reserve(length, c.new, 3, 2, c.slots)
            c.cache = B.PagedCache(1, 4, 2, 64, pool, length, rope_cos=cos, rope_sin=sin)
        q, k, v = c.parts()
        c.cache.append(0, q, k, v, c.slots, 2, 3, c.q_out, prefix=2 if prefix else None)
        outs.append((c.q_out, c.cache.k_pool[0][c.slots.long()], c.cache.v_pool[0][c.slots.long()]))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_cannot_be_held_are_nan(B, d):
    """Infinities and NaN anywhere in a row, and magnitudes past 448 * 2^40: scale 255, values 0; the neighbours
    are as ever. Zeros and the smallest values: scale -40."""
    c = Case(B, 2, 2, d, torch.bfloat16, torch.bfloat16, 0, False, [60], [10], 10, seed=1)
    for i, x in enumerate((INF, -INF, NAN, 448 * 2.0 ** 40 * 1.01, 448.0 * 2.0 ** 40)):
        c.qkv[i, 2 * d: 4 * d] = 1.0
        c.qkv[i, 2 * d + (37 * i) % d] = x
    c.qkv[5, 2 * d: 3 * d] = 0
    c.qkv[6, 2 * d: 3 * d] = 1e-38
    c.qkv[7, 2 * d: 3 * d] = 2.0 ** -42
    c.append()
    at = c.slots.long()
    b = c.cache.scales[0, at // 64, :, :, at % 64].cpu()      # [10][2 heads][k, v]
    raw = c.cache.k_pool.view(torch.uint8)[0, at].cpu()
    assert b[:4, 0, 0].tolist() == [255] * 4 and bool((raw[:4, 0] == 0).all())
    assert b[:5, 1, 0].tolist() == [127 - 8] * 5              # 1.0 = 256 * 2^-8
    assert int(b[4, 0, 0]) == 167 and b[5:8, 0, 0].tolist() == [87] * 3
    assert bool((raw[5:7, 0] == 0).all()) and bool((raw[7, 0].view(F8).float() == 0.25).all())
    assert c.cache.device_error() == 0


def test_refused_slots_and_positions(B):
    c = Case(B, 2, 1, 64, torch.float16, torch.float16, 64, False, [0, 9], [4, 4], 4, seed=2)
    keep = c.slots.clone()
    for bad in (-2, c.pool.n_pages * 64, 1 << 30):
        c.slots.copy_(keep)
        c.slots[3] = bad
        c.append()
        assert c.cache.device_error() == CAP
        c.slots[3] = -1
        c.check()
    c.slots.copy_(keep)
    before = [t.clone() for t in (c.q_out, c.cache.k_pool.view(torch.uint8), c.cache.scales)]
    c.prefix = 0
    for n in (-1, 1 << 30):     # a prefix's length out of range
        c.len[2] = n
        c.append()
        assert c.cache.device_error() == CAP
        assert all(torch.equal(a, b) for a, b in zip(before, (c.q_out, c.cache.k_pool.view(torch.uint8), c.cache.scales)))


def test_keys_alone_and_captured(B):
    c = Case(B, 2, 1, 64, torch.float16, torch.float16, 64, False, [0, 9], [4, 4], 4, seed=2)
    _, k, v = c.parts()
    c.cache.append(0, None, k, v, c.slots, 2, 4, None)
    c.q_out.fill_(3.0)
    first = c.cache.k_pool.view(torch.uint8).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append()
    c.cache.k_pool.view(torch.uint8).fill_(7)
    g.replay()
    c.check()
    assert torch.equal(first, c.cache.k_pool.view(torch.uint8))


# ---------------------------------------------------------------- reading back
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("nkv,d", [(1, 64), (3, 64), (2, 128), (8, 128)])
def test_read(B, dtype, out, bits, nkv, d):
    """Windows that begin and end anywhere in pages, empty ones, whole sequences; rows behind them left alone."""
    lens = [1, 64, 65, 300, 129]
    c = AttendCase(B, nkv, nkv, d, dtype, lens, [0] * 5, 1, bits=bits, seed=nkv + d, layers=2, layer=1)
    first, count, rows = [0, 63, 3, 17, 129], [1, 1, 62, 200, 0], 200
    k, v = (torch.full((5 * rows, nkv, d), 3.0, dtype=out, device="cuda") for _ in "kv")
    c.cache.read(1, ints(first), ints(count), 5, rows, k, v)
    for w, o in zip("kv", (k, v)):
        o = o.reshape(5, rows, nkv, d)
        for s in range(5):
            want = c.values(w, c.at(s)[first[s]: first[s] + count[s]])[0].transpose(0, 1).to(out)
            assert torch.equal(o[s, : count[s]], want) and bool((o[s, count[s]:] == 3).all())
    assert c.cache.device_error() == 0


def test_read_refuses_what_is_out_of_range(B):
    c = AttendCase(B, 2, 2, 64, torch.float16, [100] * 6, [0] * 6, 1, seed=1)
    cols = c.pool.pages_per_seq
    first, count = [-1, 0, 64 * cols - 1, 0, 0, 1 << 30], [1, -1, 2, 5, 100, 1]
    c.pool.page_table[4, 1] = -1
    k, v = (torch.full((6 * 100, 2, 64), 3.0, dtype=torch.float16, device="cuda") for _ in "kv")
    c.cache.read(0, ints(first), ints(count), 6, 100, k, v)
    assert c.cache.device_error() == CAP
    k = k.reshape(6, 100, 2, 64)
    for s in (0, 1, 2, 5):
        assert bool((k[s] == 3).all())
    want = c.values("k", c.at(3)[:5])[0].transpose(0, 1).to(torch.float16)
    assert torch.equal(k[3, :5], want) and bool((k[3, 5:] == 3).all())
    want = c.values("k", c.at(4)[:64])[0].transpose(0, 1).to(torch.float16)
    assert torch.equal(k[4, :64], want) and bool((k[4, 64:] == 3).all())
    c.cache.read(0, ints(first), ints([1, 0, 0, 5, 5, 0]), 6, 4, k.reshape(-1, 2, 64)[: 24].clone(), v[: 24].clone())
    assert c.cache.device_error() == CAP     # more than rows_per_seq


def test_read_of_nan_rows(B):
    c = AttendCase(B, 1, 1, 64, torch.bfloat16, [10], [0], 1, seed=1)
    at = c.at(0)
    c.set_scales("k", at[3:4], torch.full((1, 1), 255, dtype=torch.uint8, device="cuda"))
    k, v = (torch.zeros(10, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    c.cache.read(0, ints([0]), ints([10]), 1, 10, k, v)
    assert bool(torch.isnan(k[3].float()).all()) and bool(torch.isfinite(k[4:].float()).all()) and bool(torch.isfinite(v.float()).all())


def test_what_is_appended_is_read(B):
    """append, then read, then the same rows appended from what was read: the cache does not change."""
    c = Case(B, 2, 2, 128, torch.bfloat16, torch.bfloat16, 0, False, [0, 40], [50, 70], 70, seed=3)
    c.append()
    k, v = (torch.zeros(2 * 70, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    c.cache.read(0, c.len, c.new, 2, 70, k, v)
    before = [t.view(torch.uint8).clone() for t in (c.cache.k_pool, c.cache.v_pool, c.cache.scales)]
    c.cache.append(0, None, k, v, c.slots, 2, 70, None)
    after = [t.view(torch.uint8) for t in (c.cache.k_pool, c.cache.v_pool, c.cache.scales)]
    at = c.slots[c.slots >= 0].long()
    k8, b8 = quantised(c.parts()[1].reshape(140, 2, 128)[c.slots >= 0].float())
    assert torch.equal(before[0][0, at], k8.view(torch.uint8)) and torch.equal(before[2][0, at // 64, :, 0, at % 64], b8)
    # a maximum just above 448 * 2^(e - 1) that was rounded down to it has the next lower scale now: the same values come back
    f = lambda p, s: p.view(F8).float().reshape(-1, 2, 128) * torch.exp2(s.float() - 127)  # noqa: E731
    for i in range(2):
        sc = [t[2].reshape(1, -1, 2, 2, 64)[0, :, :, i].transpose(1, 2).reshape(-1, 2, 1) for t in (before, after)]
        assert torch.equal(f(before[i], sc[0])[at], f(after[i], sc[1])[at])
