"""Attention with a prefix on one cache by several streams and graphs at once, each with a workspace of its own."""
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


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("rows", [1, 16])
def test_one_cache_on_three_streams(B, bits, rows):
    """Two graphs and an eager call at a time, with queries of their own: the bits of the same calls one after another. The cuts of
    their lists leave parts of every row in the workspaces, long enough for the calls to overlap."""
    c = Case(B, 8, 2, 128, torch.bfloat16, [900, 30, 64], [rows] * 3, rows, bits=bits, prefix=20000, seed=rows)
    gen = torch.Generator(device="cuda").manual_seed(1)
    calls = []
    for i in range(3):
        q = torch.randn(c.q.shape, generator=gen, device="cuda").to(c.q.dtype)
        out = torch.full_like(q, 3.0)
        ws = c.cache.shared_workspace(3 * rows)
        c.cache.attend(0, q, c.new, 3, rows, out, prefix=c.slot, workspace=ws)
        kept, c.q, c.out = (c.q, c.out), q, out
        c.check()
        c.q, c.out = kept
        calls.append([q, out, ws, out.clone(), torch.cuda.Stream(), None])
    # the cache's own workspace gives the same
    out = torch.full_like(calls[0][1], 3.0)
    c.cache.attend(0, calls[0][0], c.new, 3, rows, out, prefix=c.slot)
    assert torch.equal(out, calls[0][3])
    torch.cuda.synchronize()
    for call in calls[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                c.cache.attend(0, call[0], c.new, 3, rows, call[1], prefix=c.slot, workspace=call[2])
        call[5] = g
    for turn in range(30):
        for q, out, ws, _, st, g in calls:
            with torch.cuda.stream(st):
                out.fill_(3.0)
                if g is not None:
                    g.replay()
                else:
                    for _ in range(4):
                        c.cache.attend(0, q, c.new, 3, rows, out, prefix=c.slot, workspace=ws)
        torch.cuda.synchronize()
        for _, out, _, want, _, _ in calls:
            assert torch.equal(out, want), turn
    assert c.cache.device_error() == 0


def test_too_small(B):
    c = Case(B, 8, 2, 64, torch.float16, [9, 30], [4, 4], 4, prefix=70, seed=1)
    for rows, status in ((7, -3), (8, 0)):
        ws = c.cache.shared_workspace(rows)
        if status == 0:
            c.attend(workspace=ws)
            c.check()
            continue
        with pytest.raises(B.DFlashError) as e:
            c.attend(workspace=ws)
        assert e.value.status == status and bool((c.out == 3).all())
    for n in (0, 1, 255, 4096):
        with pytest.raises(B.DFlashError) as e:
            c.attend(workspace=torch.zeros(n, dtype=torch.uint8, device="cuda"))
        assert e.value.status in (-1, -3)
