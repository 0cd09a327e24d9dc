"""Generation that also collects log probabilities, on the CPU with a stand-in drafter: the tokens
stay the target's, every token gets the log probability, entropy and alternatives of its own
row, and lists end with the tokens. A drafter with a page pool asks it for room in step."""
from types import SimpleNamespace

import torch

from block_diffusion_drafter_kv_gb300.generate import spec_generate
from synthetic_target import TinyTarget, greedy_reference
from test_generate_host import FakeDrafter


class Scoring(FakeDrafter):
    def logprobs(self, logits, tokens, logprob, entropy, top_ids=None, top_logprobs=None, temperature=1.0, stream=None):
        assert logits.dtype == torch.float32 and tokens.dtype == torch.int32 and logits.shape[0] == tokens.numel()
        ln = torch.log_softmax(logits.double(), 1)
        logprob.copy_(torch.where(tokens >= 0, ln.gather(1, tokens.clamp(min=0).long()[:, None])[:, 0], 0.0))
        entropy.copy_(-(ln.exp() * ln).sum(1))
        if top_ids is not None:
            v, i = torch.topk(ln, top_ids.numel() // len(tokens), 1)
            top_ids.copy_(i.reshape(-1))
            top_logprobs.copy_(v.reshape(-1))


def target():
    return TinyTarget(1024, 256, seed=3, bias_token=77, bias=4.8, device="cpu")


IDS = torch.randint(0, 1024, (24,), generator=torch.Generator().manual_seed(1))


def test_scores_belong_to_the_tokens():
    ref = greedy_reference(target(), IDS, 60)
    out, st = spec_generate(Scoring(1024, 8, 77), target(), IDS, 60, logprobs=3)
    assert out == ref
    assert len(st.token_logprobs) == len(st.token_entropies) == len(st.top_logprobs) == 60
    # the target alone, one token after another
    t = target()
    _, z = t.prefill(IDS)
    for k, tok in enumerate(ref):
        ln = torch.log_softmax(z.reshape(-1).double(), 0)
        assert abs(st.token_logprobs[k] - ln[tok].item()) < 1e-4
        assert abs(st.token_entropies[k] + (ln.exp() * ln).sum().item()) < 1e-4
        assert [i for i, _ in st.top_logprobs[k]] == torch.topk(ln, 3).indices.tolist()
        assert st.top_logprobs[k][0][0] == tok and abs(st.top_logprobs[k][0][1] - st.token_logprobs[k]) < 1e-6
        _, z = t.forward_block(torch.tensor([tok]))


def test_lists_end_with_the_tokens_and_zero_alternatives():
    for n in (1, 7):
        out, st = spec_generate(Scoring(1024, 8, 77), target(), IDS, n, logprobs=0)
        assert len(out) == len(st.token_logprobs) == n and st.top_logprobs == [[]] * n
    out, st = spec_generate(Scoring(1024, 8, 77), target(), IDS, 5)
    assert st.token_logprobs == [] and st.top_logprobs == []


def test_a_page_pool_is_asked_for_room_before_every_write():
    calls = []
    d = Scoring(1024, 8, 77)
    d.pages = SimpleNamespace(
        reserve=lambda length, n, rows, batch, slots=None, stream=None: calls.append(("reserve", int(length[0]), int(n[0]))),
        release=lambda length, batch, stream=None: calls.append(("release", int(length[0]))))
    out, st = spec_generate(d, target(), IDS, 40)
    assert out == greedy_reference(target(), IDS, 40)
    assert calls[:2] == [("release", 0), ("reserve", 0, 24)]
    n = 24
    for call, tau in zip(calls[2:], st.accept_lens):
        assert call == ("reserve", n, 8)
        n += tau
    assert len(calls) == 2 + st.steps
