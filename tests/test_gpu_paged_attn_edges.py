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


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,nkv,rows", [(8, 2, 1), (8, 2, 4), (12, 4, 7), (16, 4, 16), (16, 2, 16)])
def test_long_caches_in_both_types_and_widths(B, dtype, d, nq, nkv, rows):
    """Small weights in fp16 and sums over tens of thousands of keys, for every kernel (16, 64 and 128 rows)."""
    lens = [20011, 700, 8192 - rows, 64, 3333]
    c = Case(B, nq, nkv, d, dtype, lens, [rows, max(1, rows - 1), rows, rows, 1], rows, seed=d + rows, spread=1.5)
    c.attend()
    c.check()
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("nq,nkv,rows", [(2, 1, 2), (4, 1, 8)])
def test_as_many_sequences_as_a_handle_takes(B, nq, nkv, rows):
    """8192 sequences, 1024 to a launch: those on both sides of every launch's end, and some between."""
    lens = [(n * 37) % 200 for n in range(8192)]
    news = [rows if n % 5 else n % rows for n in range(8192)]
    c = Case(B, nq, nkv, 64, torch.float16, lens, news, rows, seed=rows)
    c.attend()
    c.check(seqs=sorted({min(8191, max(0, 1024 * k + i)) for k in range(9) for i in (-2, -1, 0, 1)} | set(range(5, 8192, 700))))
    assert c.cache.device_error() == 0


@pytest.mark.parametrize("nq,rows", [(8, 8), (8, 16)])
def test_tcgen05_twice_at_once(B, nq, rows):
    """Two handles on two streams, one replaying a graph while the other is called, each with tensor memory
    and a workspace of its own."""
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
    for _ in range(50):
        for i, (c, _, st) in enumerate(sets):
            with torch.cuda.stream(st):
                c.out.fill_(3.0)
                g.replay() if i == 0 else c.attend()
    torch.cuda.synchronize()
    for c, want, _ in sets:
        assert torch.equal(c.out, want) and c.cache.device_error() == 0
