"""Rotary append against the rotation in 64 bits: types, pair layouts, rotated widths, strided
rows of a fused projection, rows without a slot, and slots that are refused.

Tolerance of a rotated value y = a cos -+ b sin: three fp32 roundings of terms of at most
|a| + |b|, then half a step of the result's type: 2^-22 (|a| + |b|) + u |y|, and half the
spacing of fp16's subnormals (2^-25)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
CAP = 2


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rotated(x, cos, sin, interleaved):
    """x [rows][heads][d] float64, cos / sin [rows][rope / 2]; also |a| + |b| of every value."""
    half = cos.shape[1]
    y, size = x.clone(), x.abs()
    c, s = cos[:, None].double(), sin[:, None].double()
    i0 = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    i1 = i0 + (1 if interleaved else half)
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    size[..., i0] = size[..., i1] = a.abs() + b.abs()
    return y, size


def close(got, want, size):
    u = HALF[got.dtype]
    tol = 2.0 ** -22 * size + u * want.abs() + 2.0 ** -25
    assert bool(((got.double() - want).abs() <= tol).all())


class Case:
    def __init__(self, B, nq, nkv, d, x, y, rope, interleaved, lens, news, rows, layers=1, layer=0, seed=0, pad=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.dims, self.rows, self.batch, self.layer = B, (nq, nkv, d), rows, len(lens), layer
        cols = max(-(-(a + rows) // 64) for a in lens)
        self.pool = B.PagePool(cols * self.batch + 2, cols, self.batch)
        self.len, self.new = ints(lens), ints(news)
        self.slots = torch.empty(self.batch * rows, dtype=torch.int32, device="cuda")
        self.pool.reserve(self.len, self.new, rows, self.batch, self.slots)
        self.cos, self.sin = B.rope_tables(cols * 64, rope, 1e4) if rope else (None, None)
        self.interleaved = interleaved
        self.cache = B.PagedCache(layers, nq, nkv, d, self.pool, self.len, dtype=y, rope_cos=self.cos, rope_sin=self.sin,
                                  rope_interleaved=interleaved)
        self.cache.k_pool.fill_(7.0)
        self.cache.v_pool.fill_(-7.0)
        n = self.batch * rows
        self.qkv = torch.randn(n, (nq + 2 * nkv) * d + pad, generator=g, device="cuda").to(x)
        self.q_out = torch.full((n, nq, d), 3.0, dtype=y, device="cuda")

    def parts(self):
        nq, nkv, d = self.dims
        return self.qkv[:, : nq * d], self.qkv[:, nq * d: (nq + nkv) * d], self.qkv[:, (nq + nkv) * d: (nq + 2 * nkv) * d]

    def append(self):
        q, k, v = self.parts()
        self.cache.append(self.layer, q, k, v, self.slots, self.batch, self.rows, self.q_out)

    def check(self, slots=None):
        nq, nkv, d = self.dims
        slots = self.slots if slots is None else slots
        there = (slots >= 0).nonzero()[:, 0]
        at = slots[there].long()
        pos = (self.len.long()[:, None] + torch.arange(self.rows, device="cuda")).reshape(-1)[there]
        q, k, v = (t.reshape(t.shape[0], -1, d)[there].double() for t in self.parts())
        cos, sin = (self.cos[pos], self.sin[pos]) if self.cos is not None else [torch.zeros(len(there), 0, device="cuda")] * 2
        close(self.q_out[there], *rotated(q, cos, sin, self.interleaved))
        close(self.cache.k_pool[self.layer][at], *rotated(k, cos, sin, self.interleaved))
        assert torch.equal(self.cache.v_pool[self.layer][at], v.to(self.cache.dtype))
        # everything else is as it was
        rest = torch.ones(self.q_out.shape[0], dtype=torch.bool, device="cuda")
        rest[there] = False
        assert bool((self.q_out[rest] == 3).all())
        free = torch.ones(self.cache.k_pool.shape[:2], dtype=torch.bool, device="cuda")
        free[self.layer, at] = False
        assert bool((self.cache.k_pool[free] == 7).all()) and bool((self.cache.v_pool[free] == -7).all())


@pytest.mark.parametrize("x", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("y", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,rope", [(64, 64), (128, 128), (128, 48), (64, 16), (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_and_layouts(B, x, y, d, rope, interleaved):
    c = Case(B, 6, 2, d, x, y, rope, interleaved, [0, 61, 200], [5, 9, 0], 9)
    c.append()
    c.check()
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("nq,nkv,lens,rows,pad,layers", [(1, 1, [0], 1, 0, 1), (32, 8, [1000], 1, 8, 2), (5, 5, [63, 64, 127], 2, 24, 3),
                                                         (40, 8, [0], 777, 0, 1), (8, 1, list(range(0, 330, 11)), 16, 16, 1), (2, 1, [n % 300 for n in range(8192)], 1, 0, 1)])
def test_sizes_and_strides(B, nq, nkv, lens, rows, pad, layers):
    c = Case(B, nq, nkv, 128, torch.bfloat16, torch.float16, 128, False, lens, [rows] * len(lens), rows, layers, layers - 1, pad=pad)
    c.append()
    c.check()
    assert c.cache.device_error() == 0


def test_keys_and_values_alone_and_separate_tensors(B):
    c = Case(B, 4, 2, 64, torch.bfloat16, torch.bfloat16, 64, True, [10, 20], [3, 3], 3)
    q, k, v = (t.contiguous().reshape(6, -1, 64) for t in c.parts())
    c.cache.append(0, None, k, v, c.slots, 2, 3, None)
    assert bool((c.q_out == 3).all())
    want = c.cache.k_pool.clone(), c.cache.v_pool.clone()
    c.append()
    assert torch.equal(want[0], c.cache.k_pool) and torch.equal(want[1], c.cache.v_pool)
    c.check()


def test_refused_slots_leave_everything_and_set_the_flag(B):
    c = Case(B, 4, 2, 128, torch.float16, torch.float16, 64, False, [0, 5], [4, 4], 4)
    good = c.slots.clone()
    rows = c.cache.k_pool.shape[1]
    for bad in (rows, 2 ** 31 - 1, -2, -2 ** 31):
        c.slots.copy_(good)
        c.slots[5] = bad
        c.cache.k_pool.fill_(7.0)
        c.cache.v_pool.fill_(-7.0)
        c.q_out.fill_(3.0)
        c.append()
        seen = c.slots.clone()
        seen[5] = -1
        c.check(seen)
        assert c.cache.device_error() == CAP and c.cache.device_error() == 0


def test_positions_past_the_tables_are_refused(B):
    c = Case(B, 2, 2, 64, torch.float16, torch.float16, 64, False, [60], [6], 6)
    short = B.PagedCache(1, 2, 2, 64, c.pool, c.len, rope_cos=c.cos[:63].contiguous(), rope_sin=c.sin[:63].contiguous(),
                         k_pool=c.cache.k_pool, v_pool=c.cache.v_pool)
    c.cache = short
    c.append()
    seen = c.slots.clone()
    seen[3:] = -1
    c.check(seen)
    assert short.device_error() == CAP
    c.len.fill_(-1)          # row 0 is position -1
    c.slots[1:] = -1
    short.k_pool.fill_(7.0)
    c.append()
    assert short.device_error() == CAP and bool((short.k_pool == 7).all())


def test_special_values_pass_through(B):
    """Infinities and NaN stay themselves in the values; a bf16 beyond fp16's range becomes infinite."""
    c = Case(B, 2, 2, 64, torch.bfloat16, torch.float16, 0, False, [0], [2], 2)
    v = c.parts()[2]
    v[0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1e30], dtype=torch.bfloat16)
    c.append()
    got = c.cache.v_pool[0][int(c.slots[0])].reshape(-1)[:4].tolist()
    assert got[0] == float("inf") and got[1] == float("-inf") and got[2] != got[2] and got[3] == float("inf")


def test_bad_arguments_are_refused_before_a_launch(B):
    c = Case(B, 4, 2, 64, torch.float16, torch.float16, 64, False, [0], [1], 1)
    q, k, v = c.parts()
    f, h = c.cache.L.dflash_cache_append, c.cache.c
    def call(layer=0, q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), x=B.F16, qs=512, ks=512, vs=512, slots=c.slots.data_ptr(),
             batch=1, rows=1, out=c.q_out.data_ptr()):
        return f(h, layer, q, k, v, x, qs, ks, vs, slots, batch, rows, out, None)
    assert call(layer=1) == call(layer=-1) == call(k=None) == call(v=None) == call(slots=None) == -1
    assert call(out=None) == call(q=None) == call(x=B.F32) == call(x=7) == -1
    assert call(k=k.data_ptr() + 2) == call(out=c.q_out.data_ptr() + 8) == call(slots=c.slots.data_ptr() + 1) == -1
    assert call(qs=248) == call(qs=260) == call(ks=120) == call(vs=129) == call(batch=0) == call(rows=0) == -1
    assert call(batch=2) == -3
    e = B.c_void_p()
    B.check(c.cache.L.dflash_cache_create(B.ctypes.byref(c.cache.cfg), B.ctypes.byref(e)), "create")
    assert f(e, 0, q.data_ptr(), k.data_ptr(), v.data_ptr(), B.F16, 512, 512, 512, c.slots.data_ptr(), 1, 1, c.q_out.data_ptr(), None) == -5
    assert c.cache.L.dflash_cache_attend(e, 0, c.q_out.data_ptr(), c.len.data_ptr(), 1, 1, c.q_out.data_ptr(), None) == -5
    ws, n, p = c.cache.workspace, c.cache.workspace.numel(), (c.cache.workspace.data_ptr() + 255) // 256 * 256
    kp, vp, pt, ln, cs = c.cache.k_pool.data_ptr(), c.cache.v_pool.data_ptr(), c.pool.page_table.data_ptr(), c.len.data_ptr(), c.cos.data_ptr()
    bind = c.cache.L.dflash_cache_bind
    assert bind(e, None, vp, pt, ln, cs, cs, p, n) == bind(e, kp + 8, vp, pt, ln, cs, cs, p, n) == -1
    assert bind(e, kp, vp, pt, ln, None, cs, p, n) == bind(e, kp, vp, pt, ln, cs, cs, p + 16, n) == -1
    assert bind(e, kp, vp, pt, ln, cs, cs, p, 4096) == -3
    assert c.cache.L.dflash_cache_destroy(e) == 0
