"""Generation on a stream of the caller's, behind work that both streams have queued: the same tokens,
log probabilities and pages as on the current stream."""
import pytest
import torch

from synth import TINY
from synth import inputs as I

pytestmark = pytest.mark.gpu


def busy(ms):
    """About so many milliseconds of real work on the current stream (a 4096 product takes some 0.1 ms)."""
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    for _ in range(10 * ms):
        a = a @ a * 1e-2
    return a


@pytest.mark.parametrize("temperature", [0.0, 0.8])
def test_generation_on_a_side_stream(temperature):
    from block_diffusion_drafter_kv_gb300 import binding as B
    from block_diffusion_drafter_kv_gb300.build import build
    from block_diffusion_drafter_kv_gb300.generate import spec_generate
    from synthetic_target import TinyTarget
    build()
    w = I.make_weights(TINY, 21)
    for lw in w.layers:
        lw.wo.zero_()
        lw.w_down.zero_()
    w = w.to("cuda")
    side, results = torch.cuda.Stream(), []
    for stream in (None, side, side):
        pages = B.PagePool(12, 12, 1)
        dr = B.Drafter(TINY, w, max_block=16, max_batch=1, kv_capacity=12 * 64, pages=pages)
        t = TinyTarget(TINY.vocab, TINY.target_hidden, seed=3, bias_token=77, bias=4.8, device="cuda")
        gen = torch.Generator(device="cuda").manual_seed(5)
        for prompt in (90, 40):                    # the second takes the slot over, and its pages
            ids = torch.zeros(prompt, dtype=torch.int64, device="cuda")
            if stream is not None:
                with torch.cuda.stream(side):
                    busy(20)
                busy(20)
            ids.copy_(torch.randint(0, TINY.vocab, (prompt,), generator=torch.Generator().manual_seed(prompt)))
            out, st = spec_generate(dr, t, ids, 100, temperature=temperature, generator=gen, stream=stream, logprobs=3)
            tail = pages.held.clone(), pages.page_table.clone(), dr.len.clone()   # on the current stream again
            results.append((stream is None, prompt, out, st, [x.tolist() for x in tail]))
        assert dr.device_error() == 0 and pages.device_error() == 0
    for own, prompt, out, st, tail in results[2:]:
        _, _, out0, st0, tail0 = results[0 if prompt == 90 else 1]
        assert out == out0 and st.accept_lens == st0.accept_lens and tail == tail0
        assert st.token_logprobs == st0.token_logprobs and st.token_entropies == st0.token_entropies and st.top_logprobs == st0.top_logprobs
