"""Set-up of the tests of 8-bit caches and shared prefixes: a pool in random order, a cache of either width
whose unwritten positions are NaN, and attention in 64 bits over the values that the cache holds.

Tolerance of a row of attention, with w = sum p |V| / sum p, n keys, u half a step of the output's type:
  scores   16 bits: fp32 sums of d products and the scale, (d + 8) 2^-24 max_j scale sum |q K_j|, and 2^-20 for the
           exponential. 8 bits: q goes in as two (bf16) or three (fp16) e4m3 numbers, which is exact but for
           what lies 2^-17 below the row's largest |q|; up to 3 d products of at most 1.1 |q K|, each addition to
           within a whole step of fp32: (3 d + 8) 2^-23 1.1 max_j scale sum |q K_j| + 2^-17 max |q| max_j scale sum |K_j|.
           At most 2 e w in the output
  weights  16 bits: u w, and in fp16 2^-25 absolute. 8 bits: two e4m3 numbers (bf16), 2^-4 of 2^-4: 2^-8 w;
           rounded to fp16 and then three of them (fp16): (2^-11 + 2^-12) w; absolute, of a weight times its V row's scale
           against the largest such product: 2^-18 (bf16), 2^-22 (fp16), times values of at most 448
  sums     n + 64 fp32 additions, twice (output and normaliser): 2 (n + 64) 2^-24 w; 8 bits: up to 3 n, to a whole step
  result   rounded once: u |out|, and half of fp16's smallest step"""
import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
F8 = torch.float8_e4m3fn
CAP = 2
INF, NAN = float("inf"), float("nan")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def quantised(x):
    """Rows x[..., d] (fp32 or fp64, finite) as e4m3 values and scale bytes, by the definition, in 64 bits."""
    x = x.double()
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(min=-40)
    y = x * torch.exp2(-e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).float().to(F8), (e + 127).to(torch.uint8)


class Case:
    def __init__(self, B, nq, nkv, d, dtype, lens, news, rows, bits=8, prefix=None, seed=0, spread=1.0, layers=1, layer=0, scale=0.0,
                 v_spread=0.3):
        """prefix: positions of a prefix that all sequences share, or None; it is sequence batch + 1 of the pool."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dims, self.rows, self.batch, self.layer, self.dtype, self.bits = (nq, nkv, d), rows, len(lens), layer, dtype, bits
        self.lens, self.news, self.prefix = list(lens), list(news), prefix
        self.slot = None if prefix is None else self.batch + 1
        held = [a + n for a, n in zip(lens, news)] + ([] if prefix is None else [0, prefix])
        cols = max(1, max(-(-a // 64) for a in held))
        self.pool = B.PagePool(sum(-(-a // 64) for a in held) + 3, cols, len(held))
        self.pool.free_list.copy_(torch.randperm(self.pool.n_pages, generator=g, device="cuda"))
        self.len, self.new = ints(list(lens) + ([] if prefix is None else [0, prefix])), ints(news)
        all_new = ints(list(news) + ([] if prefix is None else [0, 0]))
        self.pool.reserve(self.len, all_new, max(rows, max(news)), len(held))
        assert self.pool.device_error() == 0
        kw = {} if prefix is None else dict(shared_rows=self.batch * rows)
        self.cache = B.PagedCache(layers, nq, nkv, d, self.pool, self.len, dtype=dtype, scale=scale, bits=bits, **kw)
        self.scale = scale or d ** -0.5
        # what no sequence has written is NaN
        for p in (self.cache.k_pool, self.cache.v_pool):
            p.view(torch.uint8).fill_(0x7f) if bits == 8 else p.fill_(NAN)
        if bits == 8:
            self.cache.scales.fill_(255)
        for s in range(len(held)):
            if not held[s]:
                continue
            at = self.at(s)
            for w in "kv":
                x = torch.randn(len(at), nkv, d, generator=g, device="cuda")
                if w == "v" and bits == 8:
                    x = x * torch.exp2(v_spread * torch.randn(len(at), nkv, 1, generator=g, device="cuda"))
                self.put(w, at, x)
        self.q = (spread * torch.randn(self.batch * rows, nq, d, generator=g, device="cuda")).to(dtype)
        self.out = torch.full_like(self.q, 3.0)

    def held(self, s):
        return self.lens[s] + self.news[s] if s < self.batch else self.prefix if s == self.slot else 0

    def at(self, s):
        p = torch.arange(self.held(s), device="cuda")
        return self.pool.page_table[s].long()[p // 64] * 64 + p % 64

    def put(self, w, at, x):
        """Rows x [n][nkv][d] into the cache at rows `at`."""
        pool = self.cache.k_pool if w == "k" else self.cache.v_pool
        if self.bits == 16:
            pool[self.layer, at] = x.to(self.dtype)
            return
        y, s = quantised(x)
        pool.view(torch.uint8)[self.layer, at] = y.view(torch.uint8)
        self.set_scales(w, at, s)

    def set_scales(self, w, at, s):
        self.cache.scales[self.layer, at // 64, :, "kv".index(w), at % 64] = s

    def values(self, w, at):
        """[nkv][n][d] in 64 bits, and the rows' scales [nkv][n]."""
        pool = self.cache.k_pool if w == "k" else self.cache.v_pool
        if self.bits == 16:
            x = pool[self.layer][at].double()
            return x.transpose(0, 1), torch.zeros(x.shape[1], x.shape[0], dtype=torch.float64, device="cuda")
        b = self.cache.scales[self.layer, at // 64, :, "kv".index(w), at % 64].double()
        f = torch.where(b == 255, NAN, torch.exp2(b - 127))
        return (pool.view(torch.uint8)[self.layer, at].view(F8).float().double() * f[..., None]).transpose(0, 1), f.t()

    def attend(self, **kw):
        self.cache.attend(self.layer, self.q, self.new, self.batch, self.rows, self.out, prefix=self.slot, **kw)

    def check(self, seqs=None, rows=None, skip=None):
        """skip(s, position in own sequence or -1 - position in the prefix) -> whether the key's page was dropped."""
        nq, nkv, d = self.dims
        u, grp = HALF[self.dtype], nq // nkv
        half = self.dtype == torch.float16
        pre = None if not self.prefix else [self.values(w, self.at(self.slot)) for w in "kv"]
        for s in range(self.batch) if seqs is None else seqs:
            at = self.at(s)
            parts = [self.values(w, at) for w in "kv"]
            before = self.prefix or 0
            place = torch.arange(len(at), device="cuda")
            if pre is not None:
                parts = [[torch.cat([a, b], 1) for a, b in zip(p, o)] for p, o in zip(pre, parts)]
                place = torch.cat([-1 - torch.arange(before, device="cuda"), place])
            (k, _), (v, vs) = parts
            kept = torch.tensor([not skip(s, int(p)) for p in place.tolist()], device="cuda") if skip else None
            for r in range(self.rows):
                got = self.out[s * self.rows + r]
                if r >= self.news[s]:
                    assert bool((got == 3).all())     # left as it was
                    continue
                if rows is not None and r not in rows:
                    continue
                n = before + self.lens[s] + r + 1
                kk, vv, vf = k[:, :n], v[:, :n], vs[:, :n]
                if kept is not None:
                    kk, vv, vf = kk[:, kept[:n]], vv[:, kept[:n]], vf[:, kept[:n]]
                    if kk.shape[1] == 0:
                        assert bool((got == 0).all())
                        continue
                q = self.q[s * self.rows + r].double().reshape(nkv, grp, d)
                sc = torch.einsum("hgd,hnd->hgn", q, kk) * self.scale
                mag = torch.einsum("hgd,hnd->hgn", q.abs(), kk.abs()).amax(-1, keepdim=True) * self.scale
                e = torch.exp(sc - sc.amax(-1, keepdim=True))
                tot = e.sum(-1, keepdim=True)
                want = torch.einsum("hgn,hnd->hgd", e / tot, vv)
                w = torch.einsum("hgn,hnd->hgd", e / tot, vv.abs())
                if self.bits == 8:
                    far = q.abs().amax(-1, keepdim=True) * kk.abs().sum(-1).amax(-1)[:, None, None] * self.scale * 2.0 ** -17
                    err = (3 * d + 8) * 2.0 ** -23 * 1.1 * mag + far + 2.0 ** -20
                    tol = (2 * err + (2.0 ** -11 + 2.0 ** -12 if half else 2.0 ** -8) + 2 * (3 * n + 64) * 2.0 ** -23) * w
                    tol = tol + n * (2.0 ** -22 if half else 2.0 ** -18) * 448 * (e * vf[:, None]).amax(-1, keepdim=True) / tot
                else:
                    tol = (2 * ((d + 8) * 2.0 ** -24 * mag + 2.0 ** -20) + u + 2 * (n + 64) * 2.0 ** -24) * w
                    tol = tol + n * 2.0 ** -25 * vv.abs().amax() / tot
                tol = tol + u * want.abs() + (2.0 ** -25 if half else 0.0)
                off = (got.double().reshape(nkv, grp, d) - want).abs() - tol
                assert bool((off <= 0).all()), (s, r, off.max().item())
