"""Generation in slot 0 of a drafter of several sequences, on the CPU with a stand-in: the other slots
stay as they are."""
import torch

from block_diffusion_drafter_kv_gb300.generate import spec_generate
from synthetic_target import greedy_reference
from test_generate_logprobs_host import IDS, Scoring, target


def test_other_sequences_keep_their_lengths():
    d = Scoring(1024, 8, 77)
    d.len = torch.tensor([99, 33, 7], dtype=torch.int32)
    d.last_token = torch.tensor([1, 2, 3], dtype=torch.int32)
    out, st = spec_generate(d, target(), IDS, 20)
    assert out == greedy_reference(target(), IDS, 20)
    assert d.len.tolist() == [24 + sum(st.accept_lens), 33, 7] and d.last_token.tolist()[1:] == [2, 3]
