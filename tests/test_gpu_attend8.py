"""Attention over the 8-bit paged cache against softmax attention in 64 bits over the values that the
cache holds (tolerances: cache_cases.py)."""
import pytest
import torch

from cache_cases import CAP, F8, INF, NAN, Case, ints

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv,rows", [(2, 2, 1), (8, 2, 1), (14, 2, 1), (16, 1, 1), (8, 2, 5), (12, 4, 9), (8, 2, 16), (6, 1, 16),
                                         (8, 1, 16), (32, 1, 4), (128, 1, 1)])
def test_heads_rows_and_types(B, dtype, d, nq, nkv, rows):
    """From one row a KV head to 128, at lengths around the ends of pages and of pairs of pages."""
    lens = [0, 1, 15, 16, 63, 64, 100, 127, 447]
    news = [rows, 1, rows, max(1, rows - 1), rows, 0, rows, rows, rows]
    c = Case(B, nq, nkv, d, dtype, lens, news, rows, seed=nq + rows + d)
    c.attend()
    c.check()
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("rows", [1, 3, 16])
def test_page_edges(B, rows):
    """New rows that begin or end at, before and behind a page's edge."""
    lens = [x for e in (64, 128, 192) for x in range(e - rows - 1, e + 2)]
    c = Case(B, 4, 1, 128, torch.float16, lens, [rows] * len(lens), rows, seed=rows)
    c.attend()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nq,nkv,rows,lens", [(8, 2, 1, [40000]), (8, 8, 1, [9000, 1, 3000]), (32, 8, 16, [5000, 64, 0, 777]),
                                              (32, 8, 1, [n * 997 % 8000 for n in range(32)]), (12, 4, 5, [n * 641 % 6000 for n in range(40)]),
                                              (4, 2, 1, [n * 37 % 900 for n in range(400)]), (16, 2, 16, [3000, 20011, 64, 1]),
                                              (2, 1, 1, [n % 70 for n in range(2500)])])
def test_long_ragged_and_many(B, dtype, nq, nkv, rows, lens):
    """Long caches split over every CTA, ragged batches whose CTAs walk many tiles and segments, and
    more sequences than a launch takes."""
    c = Case(B, nq, nkv, 128, dtype, lens, [rows] * len(lens), rows, seed=len(lens), spread=1.5)
    c.attend()
    c.check(seqs=range(len(lens)) if len(lens) < 20 else range(0, len(lens), max(7, len(lens) // 10)))
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 7])
def test_value_rows_of_very_different_size(B, dtype, rows):
    """A first key that takes most of the weight with values 2^-12 of the others', rows of zeros, and scales
    at both ends of their range in keys and values."""
    c = Case(B, 4, 1, 128, dtype, [5000, 900, 70], [rows] * 3, rows, seed=rows, v_spread=3.0)
    at = c.at(0)
    c.put("k", at[:1], 4 * c.q[:1, :1].float())
    c.put("v", at[:1], torch.randn(1, 1, 128, device="cuda") * 2.0 ** -12)
    at = c.at(1)
    c.put("v", at[10:500], torch.zeros(490, 1, 128, device="cuda"))
    c.put("k", at[20:30], torch.zeros(10, 1, 128, device="cuda"))
    c.put("v", at[600:610], torch.full((10, 1, 128), 1e-14, device="cuda"))
    at = c.at(2)
    c.put("v", at[:64], torch.randn(64, 1, 128, device="cuda") * 1e-13)   # e = -40 in all
    c.put("v", at[64:], torch.randn(len(at) - 64, 1, 128, device="cuda") * 1e-13)
    c.attend()
    c.check()


@pytest.mark.parametrize("dtype", TYPES)
def test_values_at_the_largest_scale(B, dtype):
    """e = 40: finite in the weighted sums, past fp16 in the result."""
    c = Case(B, 2, 1, 64, dtype, [100], [1], 1, seed=3)
    at = c.at(0)
    c.put("v", at, torch.randn(len(at), 1, 64, device="cuda") * 2.0 ** 46)
    c.attend()
    if dtype == torch.bfloat16:
        c.check()
    else:
        assert bool(torch.isinf(c.out).all())


@pytest.mark.parametrize("nq,rows", [(4, 1), (4, 5), (8, 16)])
def test_scores_of_billions(B, nq, rows):
    """The key with the largest score takes all: the row is that key's value."""
    c = Case(B, nq, 1, 128, torch.bfloat16, [300, 7], [rows] * 2, rows, seed=rows)
    c.q.copy_(58880 + 256 * ((c.q.float() * 10).abs().int() % 8))
    for s in range(2):
        at = c.at(s)
        c.put("k", at, (torch.arange(len(at), device="cuda") % 7 + 1.0)[:, None, None].expand(-1, 1, 128) * 64)
        c.put("k", at[c.lens[s]: c.lens[s] + 1], torch.full((1, 1, 128), 40000.0, device="cuda"))
    c.attend()
    got = c.out.reshape(2, rows, nq, 128)
    for s in range(2):
        want = c.values("v", c.at(s)[c.lens[s]: c.lens[s] + 1])[0][0, 0].to(torch.bfloat16)
        off = (got[s].float() - want.float()).abs()
        assert bool((off <= 2.0 ** -7 * want.float().abs()).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,rows", [(2, 3), (4, 16), (8, 16)])
def test_nan_rows_are_seen_by_those_that_see_them(B, nq, rows, d):
    """A NaN scale, or a NaN among the values, of a new key's K or V spoils the rows from that key on and no
    others; of a key before the new rows, all of them."""
    for what in ("k scale", "v scale", "k value", "v value"):
        for new in range(0, rows, 2):
            for pos in (700 + new, 3):
                c = Case(B, nq, 1, d, torch.float16, [700, 50], [rows] * 2, rows, seed=rows + new)
                at = c.at(0)[pos: pos + 1]
                w = what[0]
                if what.endswith("scale"):
                    c.set_scales(w, at, torch.full((1, 1), 255, dtype=torch.uint8, device="cuda"))
                else:
                    (c.cache.k_pool if w == "k" else c.cache.v_pool).view(torch.uint8)[0, at, 0, d // 2] = 0xff
                c.attend()
                first = new if pos >= 700 else 0
                got = c.out.reshape(2, rows, nq, d)
                assert bool(torch.isnan(got[0, first:].float()).any(-1).all()), (what, new, pos)
                c.check(seqs=[1])
                if first:
                    c.check(seqs=[0], rows=range(first))


def test_what_lies_behind_is_never_used(B):
    """Positions behind the new rows, other sequences' and free pages: NaN bytes and NaN scales (cache_cases
    fills them so), for every row variant."""
    for nq, rows in ((1, 1), (4, 2), (4, 16), (8, 16)):
        c = Case(B, nq, 1, 128, torch.bfloat16, [5, 64, 65, 130, 257], [rows] * 5, rows, seed=nq)
        c.attend()
        c.check()


def test_queries_that_are_not_finite(B):
    c = Case(B, 4, 1, 128, torch.float16, [100, 200], [3, 3], 3, seed=5)
    c.q[1, 2, 7] = INF
    c.q[4, 0, 0] = NAN
    keep = c.q.clone()
    c.attend()
    got = c.out.float()
    assert bool(torch.isnan(got[1, 2]).all()) and bool(torch.isnan(got[4, 0]).all())
    got[1, 2] = got[4, 0] = 0
    assert bool(torch.isfinite(got).all())
    c.q[1, 2] = c.q[4, 0] = 0
    good = c.out.clone()
    c.attend()
    same = torch.ones(6, 4, dtype=torch.bool, device="cuda")
    same[1, 2] = same[4, 0] = False
    assert torch.equal(good[same], c.out[same])     # rows do not depend on one another
    c.check()
    del keep


def test_tiny_and_zero_queries(B):
    c = Case(B, 4, 2, 64, torch.bfloat16, [100, 200], [2, 2], 2, seed=6)
    c.q[0] = 0
    c.q[1] *= 1e-30
    c.q[2, 0] = 1e-38
    c.attend()
    c.check()


def test_lengths_and_pages_that_are_refused(B):
    """Sequences with lengths out of range are left out, pages outside the pool dropped; both are flagged."""
    c = Case(B, 4, 1, 128, torch.float16, [100, 200, 300, 130], [2, 2, 2, 2], 2, seed=8)
    c.len[0] = -1
    c.new[2] = 3
    c.pool.page_table[1, 1] = c.pool.n_pages
    c.pool.page_table[3, 0] = -5
    c.pool.page_table[3, 1] = -5
    c.pool.page_table[3, 2] = 1 << 30
    before = c.out.clone()
    table = c.pool.page_table.clone()
    c.attend()
    assert c.cache.device_error() == CAP
    got = c.out.reshape(4, 2, 4, 128)
    assert torch.equal(got[0], before.reshape(4, 2, 4, 128)[0]) and torch.equal(got[2], before.reshape(4, 2, 4, 128)[2])
    assert bool((got[3] == 0).all())
    c.pool.page_table[1, 1] = 0
    c.check(seqs=[1], skip=lambda s, p: 64 <= p < 128)
    c.pool.page_table.copy_(table)
    c.len[0] = 64 * c.pool.pages_per_seq - 1
    c.attend()
    assert c.cache.device_error() == CAP and c.cache.device_error() == 0


def test_layers_scale_and_a_small_step_of_lengths(B):
    for scale in (0.0, 0.02, 1.0):
        c = Case(B, 4, 2, 64, torch.float16, [70, 3], [1, 1], 1, seed=9, layers=3, layer=2, scale=scale)
        c.attend()
        c.check()


@pytest.mark.parametrize("nq,rows", [(4, 1), (4, 16), (8, 16)])
def test_captured_replayed_and_on_two_streams(B, nq, rows):
    """Two handles on two streams, one replaying a graph while the other is called; new lengths between replays;
    the same bits every time."""
    sets = []
    for i, lens in enumerate(([9000, 30, 64], [5000, 2000])):
        c = Case(B, nq, 1, 128, torch.bfloat16, lens, [rows] * len(lens), rows, seed=7 + i)
        c.attend()
        c.check()
        sets.append((c, c.out.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    c = sets[0][0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend()
    for _ in range(30):
        for i, (c, _, st) in enumerate(sets):
            with torch.cuda.stream(st):
                c.out.fill_(3.0)
                g.replay() if i == 0 else c.attend()
    torch.cuda.synchronize()
    for c, want, _ in sets:
        assert torch.equal(c.out, want) and c.cache.device_error() == 0
    c = sets[0][0]
    c.len[0] -= 1000
    c.lens[0] -= 1000
    g.replay()
    c.check()
    with torch.cuda.stream(sets[1][2]):     # an explicit stream, not the current one
        pass
    c.out.fill_(3.0)
    c.cache.attend(0, c.q, c.new, c.batch, c.rows, c.out, stream=sets[1][2])
    sets[1][2].synchronize()
    c.check()


@pytest.mark.parametrize("nq,nkv,rows", [(8, 2, 1), (8, 2, 5), (32, 8, 16), (16, 2, 16)])
def test_again_and_again(B, nq, nkv, rows):
    """Sequences with fewer new rows than others (softmax groups without rows beside groups with some), many
    calls in a row: the same bits every time."""
    lens = [n * 997 % 6000 for n in range(24)]
    news = [1 + n * 7 % rows for n in range(24)]
    c = Case(B, nq, nkv, 128, torch.bfloat16, lens, news, rows, seed=rows)
    c.attend()
    c.check(seqs=range(0, 24, 5))
    want = c.out.clone()
    for _ in range(100):
        c.out.fill_(3.0)
        c.attend()
        assert torch.equal(c.out, want)
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("nq,nkv,rows", [(2, 1, 2), (4, 1, 8)])
def test_as_many_sequences_as_a_handle_takes(B, nq, nkv, rows):
    lens = [(n * 37) % 200 for n in range(8192)]
    news = [rows if n % 5 else n % rows for n in range(8192)]
    c = Case(B, nq, nkv, 64, torch.float16, lens, news, rows, seed=rows)
    c.attend()
    c.check(seqs=sorted({min(8191, max(0, 1024 * k + i)) for k in range(9) for i in (-2, -1, 0, 1)} | set(range(5, 8192, 700))))
    assert c.cache.device_error() == 0


def test_pools_past_two_to_the_31_bytes(B):
    """Rows whose offsets pass 32 bits: the last pages of a pool of 3 GB a tensor."""
    n_pages = 49152     # 64 x 8 x 128 bytes each: 3.2 GB
    pool = B.PagePool(n_pages, 8, 1)
    pool.free_list.copy_(torch.arange(n_pages, device="cuda"))     # the last page is handed out first
    length, new = ints([200]), ints([1])
    pool.reserve(length, new, 1, 1)
    cache = B.PagedCache(1, 8, 8, 128, pool, length, dtype=torch.bfloat16, bits=8)
    at = pool.page_table[0].long()[torch.arange(201, device="cuda") // 64] * 64 + torch.arange(201, device="cuda") % 64
    assert int(at.min()) * 1024 > 1 << 31
    v = torch.randn(201, 8, 128, device="cuda")
    cache.v_pool.view(torch.uint8)[0, at] = v.to(F8).view(torch.uint8)
    cache.scales[0, at // 64, :, :, at % 64] = 127
    q, out = torch.zeros(1, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 8, 128, dtype=torch.bfloat16, device="cuda")
    cache.attend(0, q, new, 1, 1, out)
    want = v.to(F8).double().mean(0)     # equal weights: K is zero
    assert bool(((out[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -8 * v.abs().mean(0)).all())
    k_out, v_out = torch.zeros(201, 8, 128, dtype=torch.float16, device="cuda"), torch.zeros(201, 8, 128, dtype=torch.float16, device="cuda")
    cache.read(0, ints([0]), ints([201]), 1, 201, k_out, v_out)
    assert torch.equal(v_out.float(), v.to(F8).float()) and cache.device_error() == 0
