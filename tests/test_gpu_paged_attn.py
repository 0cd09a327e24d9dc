"""Attention over the paged cache against softmax attention in 64 bits.

Tolerance of a row, with u half a step of the cache's type, w = sum p |V| / sum p and n keys:
  scores   fp32 sums of d products and the scale: e = (d + 8) 2^-24 max_j scale sum |q K_j| + 2^-20
           in the exponent (2^-20 for the exponential itself), at most 2 e w in the output
  weights  rounded to the cache's type: u w; in fp16 those below 2^-14 by 2^-25 absolute,
           n 2^-25 max |V| / sum_j exp(s_j - max) (a weight is taken against a maximum that is no larger)
  sums     n + 64 fp32 additions: (n + 64) 2^-24 w, twice (output and normaliser)
  result   rounded once: u |out|"""
import pytest
import torch

pytestmark = pytest.mark.gpu
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
CAP = 2
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, B, nq, nkv, d, dtype, lens, news, rows, seed=0, spread=1.0, layers=1, layer=0, scale=0.0, spare_cols=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dims, self.rows, self.batch, self.layer, self.dtype = (nq, nkv, d), rows, len(lens), layer, dtype
        self.lens, self.news = list(lens), list(news)
        cols = max(1, max(-(-(a + n) // 64) for a, n in zip(lens, news))) + spare_cols
        self.pool = B.PagePool(sum(-(-(a + n) // 64) for a, n in zip(lens, news)) + 3, cols, self.batch)
        # the free list in random order, so that a sequence's pages lie anywhere
        self.pool.free_list.copy_(torch.randperm(self.pool.n_pages, generator=g, device="cuda"))
        self.len, self.new = ints(lens), ints(news)
        self.pool.reserve(self.len, self.new, max(rows, max(news)), self.batch)
        assert self.pool.device_error() == 0
        self.cache = B.PagedCache(layers, nq, nkv, d, self.pool, self.len, dtype=dtype, scale=scale)
        self.scale = scale or d ** -0.5
        # what no sequence has written is NaN
        self.cache.k_pool.fill_(NAN)
        self.cache.v_pool.fill_(NAN)
        for s in range(self.batch):
            at = self.at(s)
            self.cache.k_pool[layer, at] = torch.randn(len(at), nkv, d, generator=g, device="cuda").to(dtype)
            self.cache.v_pool[layer, at] = torch.randn(len(at), nkv, d, generator=g, device="cuda").to(dtype)
        self.q = (spread * torch.randn(self.batch * rows, nq, d, generator=g, device="cuda")).to(dtype)
        self.out = torch.full_like(self.q, 3.0)

    def at(self, s):
        p = torch.arange(self.lens[s] + self.news[s], device="cuda")
        return self.pool.page_table[s].long()[p // 64] * 64 + p % 64

    def attend(self):
        self.cache.attend(self.layer, self.q, self.new, self.batch, self.rows, self.out)

    def check(self, seqs=None, drop=lambda s, j: False):
        nq, nkv, d = self.dims
        u, grp = HALF[self.dtype], nq // nkv
        for s in range(self.batch) if seqs is None else seqs:
            at = self.at(s)
            k, v = (t[self.layer][at].double().transpose(0, 1) for t in (self.cache.k_pool, self.cache.v_pool))
            for r in range(self.rows):
                got = self.out[s * self.rows + r]
                if r >= self.news[s]:
                    assert bool((got == 3).all())     # left as it was
                    continue
                n = self.lens[s] + r + 1
                q = self.q[s * self.rows + r].double().reshape(nkv, grp, d)
                sc = torch.einsum("hgd,hnd->hgn", q, k[:, :n]) * self.scale
                mag = torch.einsum("hgd,hnd->hgn", q.abs(), k[:, :n].abs()).amax(-1, keepdim=True) * self.scale
                e = torch.exp(sc - sc.amax(-1, keepdim=True))
                tot = e.sum(-1, keepdim=True)
                want = torch.einsum("hgn,hnd->hgd", e / tot, v[:, :n])
                w = torch.einsum("hgn,hnd->hgd", e / tot, v[:, :n].abs())
                tol = (2 * ((d + 8) * 2.0 ** -24 * mag + 2.0 ** -20) + u + 2 * (n + 64) * 2.0 ** -24) * w + u * want.abs()
                tol = tol + n * 2.0 ** -25 * v[:, :n].abs().amax() / tot
                off = (got.double().reshape(nkv, grp, d) - want).abs() - tol
                assert bool((off <= 0).all()), (s, r, off.max().item())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv,rows", [(2, 2, 1), (8, 2, 1), (14, 2, 1), (16, 1, 1), (8, 2, 5), (12, 4, 9), (8, 2, 16),
                                         (6, 1, 16), (8, 1, 16), (32, 1, 4), (128, 1, 1)])
def test_heads_rows_and_types(B, dtype, d, nq, nkv, rows):
    """Every row variant (16, 32, 64 and 128), at lengths around a tile's and a slice's end."""
    lens = [0, 1, 15, 16, 63, 64, 100, 447]
    news = [rows, 1, rows, max(1, rows - 1), rows, 0, rows, rows]
    c = Case(B, nq, nkv, d, dtype, lens, news, rows, seed=nq + rows + d)
    c.attend()
    c.check()
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("rows", [1, 3, 16])
def test_tile_edges(B, rows):
    """New rows that begin or end at, before and behind a page's edge."""
    lens = [x for e in (64, 128) for x in range(e - rows - 1, e + 2)]
    c = Case(B, 4, 1, 128, torch.float16, lens, [rows] * len(lens), rows, seed=rows)
    c.attend()
    c.check()


@pytest.mark.parametrize("nq,nkv,rows,lens", [(8, 2, 1, [40000]), (8, 8, 1, [9000, 1, 3000]), (32, 8, 16, [5000, 64, 0, 777]),
                                              (32, 8, 1, [n * 997 % 8000 for n in range(32)]), (12, 4, 5, [n * 641 % 6000 for n in range(40)]),
                                              (4, 2, 1, [n * 37 % 900 for n in range(400)]), (8, 4, 2, list(range(1024))),
                                              (2, 1, 1, [n % 70 for n in range(2500)])])
def test_long_ragged_and_many(B, nq, nkv, rows, lens):
    """Long caches split over every CTA, ragged batches whose CTAs walk many tiles and segments, and
    as many sequences as a call takes."""
    c = Case(B, nq, nkv, 128, torch.bfloat16, lens, [rows] * len(lens), rows, seed=len(lens))
    c.attend()
    c.check(seqs=range(len(lens)) if len(lens) < 20 else range(0, len(lens), max(7, len(lens) // 10)))
    assert c.cache.device_error() == 0


def test_same_result_every_time(B):
    c = Case(B, 8, 2, 128, torch.float16, [5000, 33, 700], [4, 4, 4], 4)
    c.attend()
    first = c.out.clone()
    for _ in range(5):
        c.out.fill_(3.0)
        c.attend()
        assert torch.equal(first, c.out)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("nq,rows", [(4, 8), (8, 4), (1, 16), (5, 9), (8, 8), (6, 16), (8, 16)])
def test_keys_hidden_from_a_row_may_be_anything(B, dtype, nq, rows):
    """An infinite or NaN value (or key) in a new row's position reaches only the rows that see it."""
    for what, pool in ((INF, "v_pool"), (NAN, "v_pool"), (-INF, "v_pool"), (NAN, "k_pool"), (INF, "k_pool")):
        c = Case(B, nq, 1, 128, dtype, [5, 60, 125], [rows] * 3, rows, seed=rows)
        c.attend()
        want = c.out.clone()
        bad = rows // 2
        for s in range(3):
            getattr(c.cache, pool)[0, c.at(s)[c.lens[s] + bad], 0, 7] = what
        c.out.fill_(3.0)
        c.attend()
        got, want = (t.reshape(3, rows, nq, 128) for t in (c.out, want))
        # the rows before it: the same up to how the products are taken
        u = HALF[dtype]
        assert bool((got[:, :bad].double() - want[:, :bad].double()).abs().max() <= 8 * u * 6)
        assert bool(torch.isfinite(got[:, :bad]).all())
        spoilt = ~torch.isfinite(got[:, bad:].float()).all(-1)
        # an infinite key's score is inf times the sign of q's value there: -inf drops the key, +inf spoils the row
        assert torch.equal(spoilt, c.q.reshape(3, rows, nq, 128)[:, bad:, :, 7] >= 0 if pool == "k_pool" and what == INF else torch.ones_like(spoilt))
        if pool == "v_pool":   # only the dim that holds it
            rest = got[:, bad:].float()
            assert bool(torch.isfinite(rest[..., :7]).all()) and bool(torch.isfinite(rest[..., 8:]).all())


@pytest.mark.parametrize("nq,rows", [(4, 4), (4, 8), (8, 16)])
def test_new_rows_on_two_pages_with_an_infinite_value_on_the_first(B, nq, rows):
    """Each page in a CTA of its own: the rows that do not see the value get their result."""
    full = Case(B, nq, 1, 128, torch.bfloat16, [0] * 200, [rows] * 200, rows)
    full.cache.v_pool.fill_(NAN)               # every CTA meets NaN among its new values
    full.attend()
    c = Case(B, nq, 1, 128, torch.bfloat16, [62, 62], [rows] * 2, rows, seed=1)
    c.attend()
    want = c.out.clone()
    c.cache.v_pool[0, c.at(0)[63], 0, 9] = INF
    c.out.fill_(3.0)
    c.attend()
    got = c.out.reshape(2, rows, nq, 128)
    assert torch.equal(got[1], want.reshape(2, rows, nq, 128)[1])
    off = (got[0, 0].double() - want.reshape(2, rows, nq, 128)[0, 0].double()).abs()
    assert bool((off <= 8 * HALF[torch.bfloat16] * 6).all())
    rest = got[0, 1:].float()
    assert not bool(torch.isfinite(rest[..., 9]).any())
    assert bool(torch.isfinite(rest[..., :9]).all()) and bool(torch.isfinite(rest[..., 10:]).all())


def test_nothing_but_nan_is_nan(B):
    """A sequence whose every key is NaN, in one CTA and split over several."""
    c = Case(B, 4, 2, 128, torch.float16, [0, 3000, 5], [1, 1, 1], 1)
    c.cache.k_pool[0, c.at(0)] = NAN
    c.cache.k_pool[0, c.at(1)] = NAN
    c.attend()
    assert bool(c.out[:2].isnan().all())
    c.check(seqs=[2])


def test_large_and_equal_scores(B):
    """Scores of hundreds (one key takes all), and all-zero queries (the mean of the values)."""
    c = Case(B, 8, 2, 128, torch.bfloat16, [700, 3], [3, 3], 3, spread=100.0)
    c.attend()
    c.check()
    c.q.zero_()
    c.attend()
    c.check()
    c = Case(B, 8, 2, 64, torch.float16, [700, 3], [1, 1], 1, scale=0.03)
    c.attend()
    c.check()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("nq,rows", [(4, 1), (4, 8), (8, 16)])
def test_scores_of_billions(B, dtype, nq, rows):
    """One key takes all where its score is 2^30 and more and the next a millionth less."""
    c = Case(B, nq, 1, 128, dtype, [300, 7], [rows] * 2, rows, seed=rows)
    c.q.copy_(torch.where(c.q > 0, 59648.0, 58880.0).to(dtype))     # 233 and 230 times 256: exact in both types
    for s in range(2):
        at = c.at(s)
        c.cache.k_pool[0, at] = (torch.arange(len(at), device="cuda") * 37 % len(at) * 0.25 + 40000.0).to(dtype)[:, None, None].expand(-1, 1, 128)
        c.cache.k_pool[0, at[3]] = 50176.0
    c.attend()
    for s in range(2):
        want = c.cache.v_pool[0, c.at(s)[3], 0]
        assert torch.equal(c.out[s * rows:(s + 1) * rows], want.expand(rows, nq, 128))


def test_layers_and_spare_columns(B):
    c = Case(B, 8, 2, 128, torch.float16, [100, 300], [2, 2], 2, layers=3, layer=2, spare_cols=5)
    c.attend()
    c.check()
    assert c.cache.device_error() == 0


def test_a_page_id_out_of_range_drops_its_positions(B):
    for bad in (-1, 10 ** 6, -2 ** 31):
        c = Case(B, 4, 2, 64, torch.float16, [200, 30, 70], [1, 1, 1], 1, seed=4)
        c.attend()
        want = c.out.clone()
        c.pool.page_table[0, 1] = bad      # positions 64..127 of sequence 0
        c.pool.page_table[1, 0] = bad      # all of sequence 1
        c.out.fill_(3.0)
        c.attend()
        assert c.cache.device_error() == CAP and c.cache.device_error() == 0
        assert bool((c.out[1] == 0).all()) and torch.equal(c.out[2], want[2])
        p = torch.tensor([j for j in range(201) if j // 64 != 1], device="cuda")
        at = c.pool.page_table[0].long()[p // 64] * 64 + p % 64
        k, v = c.cache.k_pool[0, at].double(), c.cache.v_pool[0, at].double()
        q = c.q[0].double().reshape(2, 2, 64)
        w = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) / 8, -1)
        ref = torch.einsum("hgn,nhd->hgd", w, v).reshape(4, 64)
        assert bool(((c.out[0].double() - ref).abs() <= 2.0 ** -10 * (ref.abs() + 4)).all())


def test_lengths_out_of_range_leave_a_sequence_out(B):
    c = Case(B, 4, 2, 64, torch.float16, [100, 50, 20], [2, 2, 2], 2)
    c.attend()
    want = c.out.clone()
    most = c.pool.page_table.shape[1] * 64
    for length, new in ((-1, 2), (most - 1, 2), (50, 3), (50, -1), (2 ** 31 - 1, 2)):
        c.len[1], c.new[1] = length, new
        c.out.fill_(3.0)
        c.attend()
        assert c.cache.device_error() == CAP
        assert torch.equal(c.out[:2], want[:2]) and torch.equal(c.out[4:], want[4:]) and bool((c.out[2:4] == 3).all())
    c.new.zero_()
    c.out.fill_(3.0)
    c.attend()                                # nothing to do at all
    assert c.cache.device_error() == CAP and bool((c.out == 3).all())


def test_captured_and_replayed_with_other_lengths(B):
    """One graph serves growing sequences; two handles run on two streams at once."""
    cases = [Case(B, 8, 2, 128, torch.float16, [900, 30], [4, 4], 4, seed=s) for s in (1, 2)]
    graphs = []
    for c in cases:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            c.attend()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.attend()
        graphs.append((g, st))
    for lens, news in (([800, 3], [4, 1]), ([64, 0], [0, 4]), ([0, 33], [3, 1])):
        for c in cases:
            c.lens, c.news = lens, news
            c.len.copy_(ints(lens))
            c.new.copy_(ints(news))
            c.out.fill_(3.0)
        torch.cuda.synchronize()
        for g, st in graphs:
            with torch.cuda.stream(st):
                for _ in range(4):
                    g.replay()
        torch.cuda.synchronize()
        for c in cases:
            c.check()


def test_bad_arguments_are_refused_before_a_launch(B):
    c = Case(B, 4, 2, 64, torch.float16, [5], [1], 1)
    f, q, n, o = c.cache.L.dflash_cache_attend, c.q.data_ptr(), c.new.data_ptr(), c.out.data_ptr()
    assert f(c.cache.c, -1, q, n, 1, 1, o, None) == f(c.cache.c, 1, q, n, 1, 1, o, None) == -1
    assert f(c.cache.c, 0, None, n, 1, 1, o, None) == f(c.cache.c, 0, q, None, 1, 1, o, None) == f(c.cache.c, 0, q, n, 1, 1, None, None) == -1
    assert f(c.cache.c, 0, q + 2, n, 1, 1, o, None) == f(c.cache.c, 0, q, n, 1, 1, o + 8, None) == f(c.cache.c, 0, q, n + 2, 1, 1, o, None) == -1
    assert f(c.cache.c, 0, q, n, 0, 1, o, None) == f(c.cache.c, 0, q, n, 1, 0, o, None) == -1
    assert f(c.cache.c, 0, q, n, 2, 1, o, None) == f(c.cache.c, 0, q, n, 1, 17, o, None) == -3
    assert bool((c.out == 3).all())
