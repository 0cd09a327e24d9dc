"""Attention over the 8-bit cache where pages are missing in the middle of a sequence: their steps have values to clear, but
no new keys to look through (tolerances: cache_cases.py)."""
import pytest
import torch

from cache_cases import CAP, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("nq,rows", [(4, 1), (2, 12), (4, 16), (8, 16)])
@pytest.mark.parametrize("dropped", [(0,), (3,), (4, 5), (2, 7, 8, 9), (1, 3, 5, 7)])
def test_pages_missing_in_the_middle(B, dtype, nq, rows, dropped):
    """Single tiles and whole steps of two, for one, two and four strands a CTA; lengths whose new keys begin at a page's
    last place, at a page, and inside one. What the stages held before is NaN now and then."""
    lens = [700, 64 * 11, 64 * 10 - 1, 64 * 12 - 1, 1280]
    c = Case(B, nq, 1, 128, dtype, lens, [rows] * 5, rows, seed=nq + rows)
    table = c.pool.page_table.clone()
    want = None
    for _ in range(3):
        c.pool.page_table.copy_(table)
        for s in (0, 2, 4):
            c.pool.page_table[s, list(dropped)] = c.pool.n_pages if s else -1
        c.out.fill_(3.0)
        c.attend()
        assert c.cache.device_error() == CAP
        assert want is None or torch.equal(c.out, want)
        want = c.out.clone()
        c.pool.page_table.copy_(table)
        c.check(skip=lambda s, p: s in (0, 2, 4) and p // 64 in dropped)
        # a call between that leaves NaN behind in shared memory
        keep = c.cache.v_pool.view(torch.uint8).clone()
        c.cache.v_pool.view(torch.uint8).fill_(0x7f)
        c.attend()
        c.cache.v_pool.view(torch.uint8).copy_(keep)
    assert c.cache.device_error() == 0
