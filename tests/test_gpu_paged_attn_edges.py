"""Attention over the paged cache where two edges meet: scores so large that a product's rounding
is worth powers of two, in a step whose new keys hold an infinite value."""
import pytest
import torch

from test_gpu_paged_attn import INF, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("nq,rows", [(4, 4), (4, 8), (8, 16)])
def test_scores_of_billions_beside_an_infinite_new_value(B, dtype, nq, rows):
    """The first new key takes all, at a score of 2^30 and more; the last one's value is infinite in one
    dim. Weight and sum of a key are the same number, so every row is that key's value exactly: the rows
    before the last in all dims, the last in all but the one."""
    for seed in range(4):
        c = Case(B, nq, 1, 128, dtype, [300, 7], [rows] * 2, rows, seed=rows + 100 * seed)
        # whole multiples of 256 between 58880 and 60672: exact in both types, other scores in every row
        c.q.copy_((58880 + 256 * ((c.q.float() * 10).abs().int() % 8)).to(dtype))
        for s in range(2):
            at = c.at(s)
            c.cache.k_pool[0, at] = (torch.arange(len(at), device="cuda") * 37 % len(at) * 0.25 + 40000.0).to(dtype)[:, None, None].expand(-1, 1, 128)
            c.cache.k_pool[0, at[c.lens[s]]] = 50176.0
            c.cache.v_pool[0, at[-1], 0, 9] = INF
        c.attend()
        got = c.out.reshape(2, rows, nq, 128)
        for s in range(2):
            want = c.cache.v_pool[0, c.at(s)[c.lens[s]], 0]
            assert torch.equal(got[s, :-1], want.expand(rows - 1, nq, 128)), (seed, s)
            rest = torch.arange(128, device="cuda") != 9
            assert torch.equal(got[s, -1][:, rest], want[rest].expand(nq, 127))
            assert not bool(torch.isfinite(got[s, -1, :, 9].float()).any())
