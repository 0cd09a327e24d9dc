"""Attention with page tables of 2^24 pages a sequence: a launch takes as many sequences as its list of tiles can count in 31 bits
(tolerances: cache_cases.py)."""
import pytest
import torch

from cache_cases import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


@pytest.mark.parametrize("bits,prefix,rows", [(8, 130, 3), (16, 130, 3), (8, None, 16)])
def test_more_sequences_than_a_list_counts(B, bits, prefix, rows):
    seqs, cols = 100, 1 << 24
    lens = [n * 37 % 150 for n in range(seqs)]
    news = [rows if n % 5 else n % (rows + 1) for n in range(seqs)]
    c = Case(B, 4, 1, 64, torch.bfloat16, lens, news, rows, bits=bits, prefix=prefix, seed=rows)
    table = c.pool.page_table
    wide = torch.full((table.shape[0], cols), -1, dtype=torch.int32, device="cuda")
    wide[:, : table.shape[1]] = table
    pool = B.PagePool(c.pool.n_pages, 8, table.shape[0])
    pool.page_table, pool.pages_per_seq = wide, cols
    kw = {} if prefix is None else dict(shared_rows=seqs * rows)
    if bits == 8:
        kw.update(bits=8, scales=c.cache.scales)
    c.cache = B.PagedCache(1, 4, 1, 64, pool, c.len, dtype=torch.bfloat16, k_pool=c.cache.k_pool, v_pool=c.cache.v_pool, **kw)
    c.attend()
    c.check(seqs=[0, 1, 61, 62, 63, 64, 65, 99])
    assert c.cache.device_error() == 0
    # the longest position that such a table has room for, in a sequence that then has no page there
    c.len[0], c.new[0] = 64 * cols - 1, 2
    before = c.out.clone()
    c.attend()
    assert c.cache.device_error() != 0 and torch.equal(c.out[:rows], before[:rows])
