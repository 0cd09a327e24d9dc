"""Rows of one attention call that share products: what one row's result may depend on (tolerances: cache_cases.py)."""
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


@pytest.mark.parametrize("nq,rows", [(4, 5), (4, 16), (8, 16)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_other_rows_change_no_bit_in_16_bits(B, dtype, nq, rows):
    """Rows with scores of up to millions beside others, whose own rounding is as without them."""
    c = Case(B, nq, 1, 128, dtype, [700, 40], [rows] * 2, rows, bits=16, seed=nq + rows, spread=2.0)
    c.attend()
    c.check()
    want = c.out.clone().view(-1, 128)
    q = c.q.clone()
    for change in (0.0, 30.0, -3000.0) + ((1e7, 1e30) if dtype == torch.bfloat16 else ()):
        for keep in (0, nq - 1, nq * rows // 2, nq * rows - 1, nq * rows + 1, 2 * nq * rows - 1):
            c.q.copy_(q * change)
            c.q.view(-1, 128)[keep] = q.view(-1, 128)[keep]
            c.attend()
            assert torch.equal(c.out.view(-1, 128)[keep], want[keep]), (change, keep)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("nq,nkv,rows", [(4, 1, 1), (8, 2, 5), (4, 1, 16), (8, 1, 16), (8, 1, 3)])
def test_rows_of_other_sequences_behind_a_prefix(B, bits, nq, nkv, rows):
    """Behind a prefix products take rows of several sequences together. What lies in rows that are none of this call's changes
    no bit of the others, and in 16 bits other sequences' queries do not either; in 8 bits these change roundings alone."""
    lens, news = [300, 0, 70, 500, 9, 31, 64], [rows, 1, max(1, rows - 1), 0, rows, max(1, rows // 2), rows]
    c = Case(B, nq, nkv, 128, torch.bfloat16, lens, news, rows, bits=bits, prefix=1500, seed=nq + rows, spread=2.0)
    c.attend()
    c.check(seqs=[1, 5])
    want = c.out.clone()
    q = c.q.clone()
    there = torch.tensor([r < n for n in news for r in range(rows)], device="cuda")
    for change in (0.0, 30.0, -100.0, 3000.0, 1e30, float("nan")):
        c.q.copy_(q)
        c.q[~there] *= change
        c.out.fill_(3.0)
        c.attend()
        assert torch.equal(c.out, want), change
        if change != change or change > 3000 and bits == 8:
            continue
        for s in (0, 4, 6):     # one sequence as it was
            c.q.copy_(q * change)
            mine = slice(s * rows, (s + 1) * rows)
            c.q[mine] = q[mine]
            c.out.fill_(3.0)
            c.attend()
            if bits == 16:
                assert torch.equal(c.out[mine], want[mine]), (change, s)
            else:
                c.check(seqs=[s])
    assert c.cache.device_error() == 0
