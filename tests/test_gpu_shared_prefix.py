"""Attention with a prefix that all sequences of a batch share, over caches of 16 and 8 bits, against softmax
attention in 64 bits over prefix and own positions together (tolerances: cache_cases.py)."""
import pytest
import torch

from cache_cases import CAP, NAN, Case

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nq,nkv,d,rows", [(2, 2, 64, 1), (8, 2, 128, 1), (14, 2, 128, 1), (8, 2, 64, 5), (12, 4, 128, 9), (8, 2, 128, 16), (8, 1, 64, 16),
                                           (8, 1, 128, 16), (128, 1, 128, 1), (3, 1, 64, 16), (18, 1, 128, 7)])
def test_heads_rows_and_types(B, bits, dtype, nq, nkv, d, rows):
    lens = [0, 1, 15, 63, 64, 100, 127, 447]
    news = [rows, 1, max(1, rows - 1), rows, 0, rows, rows, rows]
    c = Case(B, nq, nkv, d, dtype, lens, news, rows, bits=bits, prefix=333, seed=nq + rows + d)
    c.attend()
    c.check()
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 127, 128, 129, 1000])
@pytest.mark.parametrize("rows", [1, 6])
def test_lengths_of_the_prefix(B, bits, prefix, rows):
    c = Case(B, 8, 2, 128, torch.float16, [0, 70, 300], [rows] * 3, rows, bits=bits, prefix=prefix, seed=prefix)
    c.attend()
    c.check()


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("seqs,rows,prefix,own", [(1, 1, 30000, 5), (40, 16, 2500, 400), (64, 1, 8192, 700), (33, 3, 777, 2000), (5, 16, 5000, 5000)])
def test_long_and_many(B, bits, seqs, rows, prefix, own):
    lens = [(n * 641 + 17) % own for n in range(seqs)]
    news = [rows if n % 3 else max(1, n % (rows + 1)) for n in range(seqs)]
    c = Case(B, 16, 4, 128, torch.bfloat16, lens, news, rows, bits=bits, prefix=prefix, seed=seqs, spread=1.5)
    c.attend()
    c.check(seqs=range(0, seqs, max(1, seqs // 8)))
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("rows", [1, 4])
def test_more_sequences_than_a_launch_takes(B, bits, rows):
    lens = [(n * 37) % 200 for n in range(1300)]
    news = [rows if n % 5 else n % (rows + 1) for n in range(1300)]
    c = Case(B, 4, 2, 64, torch.float16, lens, news, rows, bits=bits, prefix=200, seed=rows)
    c.attend()
    c.check(seqs=sorted({min(1299, max(0, 256 * k + i)) for k in range(6) for i in (-2, -1, 0, 1)} | set(range(5, 1300, 150))))
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("rows", [1, 16])
def test_a_prefix_that_takes_all_or_none_of_the_weight(B, bits, rows):
    """Scores of the prefix far above, and far below, those of the own positions."""
    for factor in (30.0, -30.0):
        c = Case(B, 4, 1, 128, torch.bfloat16, [200, 0, 31], [rows] * 3, rows, bits=bits, prefix=500, seed=rows)
        c.q.abs_()
        at = c.at(c.slot)
        c.put("k", at, factor * torch.rand(len(at), 1, 128, device="cuda"))
        c.attend()
        c.check()


@pytest.mark.parametrize("bits", [16, 8])
def test_refusals_on_the_device(B, bits):
    """A prefix's length out of range leaves the whole batch out; its bad pages are dropped; sequences with bad
    lengths are left out; all are flagged."""
    c = Case(B, 4, 1, 128, torch.float16, [100, 200, 3], [2, 2, 2], 2, bits=bits, prefix=300, seed=8)
    for n in (-1, 64 * c.pool.pages_per_seq + 1, 1 << 30):
        c.len[c.slot] = n
        c.attend()
        assert c.cache.device_error() == CAP and bool((c.out == 3).all())
    c.len[c.slot] = 300
    c.len[0] = -7
    kept = c.pool.page_table[c.slot, 2].clone()
    c.pool.page_table[c.slot, 2] = -1
    c.attend()
    assert c.cache.device_error() == CAP
    assert bool((c.out[:2] == 3).all())
    c.pool.page_table[c.slot, 2] = kept
    c.check(seqs=[1, 2], skip=lambda s, p: p < 0 and 128 <= -1 - p < 192)
    # nothing left at all: every page of the prefix and of a sequence
    c.pool.page_table[c.slot] = -1
    c.pool.page_table[2] = c.pool.n_pages
    c.attend()
    assert c.cache.device_error() == CAP and bool((c.out[4:] == 0).all())


@pytest.mark.parametrize("bits", [16, 8])
def test_what_lies_behind_the_prefix_is_never_used(B, bits):
    """NaN behind its last position and behind the sequences' (cache_cases fills them so), and in the new keys of a row."""
    c = Case(B, 4, 1, 128, torch.float16, [9, 64], [5, 5], 5, bits=bits, prefix=70, seed=2)
    at = c.at(0)[9 + 3: 9 + 4]
    if bits == 8:
        c.set_scales("v", at, 255)
    else:
        c.cache.v_pool[0, at] = NAN
    c.attend()
    got = c.out.reshape(2, 5, 4, 128).float()
    assert bool(torch.isnan(got[0, 3:]).all())
    c.check(seqs=[0], rows=range(3))
    c.check(seqs=[1])
    # a NaN in the prefix is seen by every row
    at = c.at(c.slot)[69:70]
    if bits == 8:
        c.set_scales("v", at, 255)
    else:
        c.cache.v_pool[0, at] = NAN
    c.attend()
    assert bool(torch.isnan(c.out.float()).all())


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv,rows,seqs", [(8, 1, 16, 3), (8, 2, 16, 5), (4, 1, 5, 40)])
@pytest.mark.parametrize("odd", [7, 1, 0])
def test_new_keys_that_are_not_finite(B, bits, d, nq, nkv, rows, seqs, odd):
    """A new key whose values are NaN, before and behind a page's end: the rows before it are as they were, in the other
    sequences too, those from it on are NaN."""
    odd = min(odd, rows - 1)
    lens = [60 if n % 2 else 64 * (n % 7) + 63 for n in range(seqs)]
    c = Case(B, nq, nkv, d, torch.bfloat16, lens, [rows] * seqs, rows, bits=bits, prefix=130, seed=odd)
    for s in (0, seqs - 2):
        at = c.at(s)[lens[s] + odd: lens[s] + odd + 1]
        if bits == 8:
            c.set_scales("v", at, 255)
        else:
            c.cache.v_pool[0, at] = NAN
    c.attend()
    got = c.out.reshape(seqs, rows, nq, d).float()
    for s in (0, seqs - 2):
        assert bool(torch.isnan(got[s, odd:]).all())
        c.check(seqs=[s], rows=range(odd))
    c.check(seqs=[s for s in range(0, seqs, 1 + seqs // 8) if s not in (0, seqs - 2)])
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("rows", [1, 16])
def test_captured_replayed_and_on_two_streams(B, bits, rows):
    sets = []
    for i, lens in enumerate(([900, 30, 64], [500, 2000])):
        c = Case(B, 8, 2, 128, torch.bfloat16, lens, [rows] * len(lens), rows, bits=bits, prefix=3000, seed=7 + i)
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
    c = sets[0][0]     # another prefix in the same graph
    c.len[c.slot] -= 1234
    c.prefix -= 1234
    g.replay()
    c.check()


def test_a_prefix_of_some_sequences_and_a_plain_call(B):
    """Calls of smaller batches and blocks on one handle, and the plain attention of the prefix's own last position."""
    c = Case(B, 8, 2, 128, torch.bfloat16, [100, 30, 64, 5], [4] * 4, 4, bits=16, prefix=700, seed=3)
    for batch, rows in ((1, 4), (4, 1), (2, 3), (4, 4)):
        c.batch, c.rows, c.news = batch, rows, [rows] * batch
        c.new[:] = rows
        q = c.q[: batch * rows].contiguous()
        out = torch.full_like(q, 3.0)
        c.cache.attend(0, q, c.new, batch, rows, out, prefix=c.slot)
        kept, c.q, c.out = (c.q, c.out), q, out
        c.check()
        c.q, c.out = kept
