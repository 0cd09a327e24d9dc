"""Rows of the cache read back straight behind the calls that wrote what it reads: page table, scales, values. The kernels
of such a chain start before the ones in front of them have ended."""
import pytest
import torch

from cache_cases import F8, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


def stored(x):
    """What an 8-bit cache holds for rows x: exponents from frexp, since a logarithm may miss a magnitude of 448 * 2^e by a bit."""
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    e = (e - 9 + (m > 0.875)).clamp(min=-40)     # 448 is 0.875 * 2^9
    return torch.ldexp(torch.ldexp(x, -e).to(F8).float(), e)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("seqs,rows,nkv,d", [(1, 1, 1, 64), (5, 70, 2, 128), (40, 200, 8, 128)])
def test_reserve_append_read(B, bits, seqs, rows, nkv, d):
    """One graph of release, reserve, append and read, replayed with other rows and lengths: pages change hands between replays, so
    that a table entry, a scale or a value of the replay before would show."""
    pool = B.PagePool(seqs * -(-rows // 64) + 7, -(-rows // 64), seqs)
    length, new, none = ints([0] * seqs), ints([rows] * seqs), ints([0] * seqs)
    cache = B.PagedCache(1, nkv, nkv, d, pool, length, dtype=torch.bfloat16, bits=bits)
    k, v = (torch.zeros(seqs * rows, nkv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    slots = ints([-1] * (seqs * rows))
    k_out, v_out = torch.zeros_like(k), torch.zeros_like(v)

    def chain():
        pool.release(none, seqs)
        pool.reserve(length, new, rows, seqs, slots)
        cache.append(0, None, k, v, slots, seqs, rows, None)
        cache.read(0, none, new, seqs, rows, k_out, v_out)

    chain()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    gen = torch.Generator(device="cuda").manual_seed(rows)
    for turn in range(40):
        k.copy_(torch.randn(k.shape, generator=gen, device="cuda") * 2.0 ** (turn % 7))
        v.copy_(torch.randn(v.shape, generator=gen, device="cuda") * 2.0 ** -(turn % 5))
        new.copy_(torch.randint(0, rows + 1, (seqs,), generator=gen, device="cuda"))
        k_out.fill_(3.0), v_out.fill_(3.0)
        pool.release(none, seqs)
        pool.free_list.copy_(pool.free_list.roll(turn + 1))        # (all pages are in it)
        g.replay()
        there = (torch.arange(rows, device="cuda") < new[:, None]).reshape(-1)
        for x, got in ((k, k_out), (v, v_out)):
            if bits == 8:
                x = stored(x.float()).to(torch.bfloat16)
            assert torch.equal(got[there], x[there]) and bool((got[~there] == 3).all()), turn
        assert pool.device_error() == 0 and cache.device_error() == 0
