"""Generation over a page pool that runs out: shorter blocks to the last position, then an error, with
the target's own greedy tokens until then."""
import pytest
import torch

from synth import TINY
from synth import inputs as I

pytestmark = pytest.mark.gpu
CAP = 2


@pytest.mark.parametrize("n_pages,cols", [(2, 12), (12, 2), (1, 1)])
def test_a_pool_or_table_that_runs_out(n_pages, cols):
    from block_diffusion_drafter_kv_gb300 import binding as B
    from block_diffusion_drafter_kv_gb300.build import build
    from block_diffusion_drafter_kv_gb300.generate import spec_generate
    from synthetic_target import TinyTarget, greedy_reference
    build()
    w = I.make_weights(TINY, 21)
    for lw in w.layers:
        lw.wo.zero_()
        lw.w_down.zero_()
    pages = B.PagePool(n_pages, cols, 1)
    dr = B.Drafter(TINY, w.to("cuda"), max_block=16, max_batch=1, kv_capacity=64 * cols, pages=pages)
    tgt = lambda: TinyTarget(TINY.vocab, TINY.target_hidden, seed=3, bias_token=77, bias=4.8, device="cuda")  # noqa: E731
    room = 64 * min(n_pages, cols)
    ids = torch.randint(0, TINY.vocab, (33,), generator=torch.Generator().manual_seed(1)).cuda()
    most = room - 33 + 1
    ref = greedy_reference(tgt(), ids, most)
    for _ in range(2):
        out, st = spec_generate(dr, tgt(), ids, most, logprobs=2)
        assert out == ref and len(st.token_logprobs) == most and int(dr.len[0]) == room
        assert all(top[0][0] == tok for top, tok in zip(st.top_logprobs, ref))
        assert dr.device_error() == 0 and pages.device_error() == CAP      # a block was refused, none went wrong
        with pytest.raises(B.DFlashError) as e:
            spec_generate(dr, tgt(), ids, most + 1)
        assert e.value.status == B.DFLASH_E_CAPACITY and dr.device_error() == 0 and pages.device_error() == CAP
    with pytest.raises(B.DFlashError) as e:
        spec_generate(dr, tgt(), torch.zeros(room + 1, dtype=torch.int64, device="cuda"), 5)
    assert e.value.status == B.DFLASH_E_CAPACITY and dr.device_error() == 0 and pages.device_error() == CAP
