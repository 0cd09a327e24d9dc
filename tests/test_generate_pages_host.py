"""Generation over a page pool that runs out, on the CPU with stand-ins: blocks shrink to what is left of
the last page, and where nothing is left it ends with an error before drafter and target go on."""
from types import SimpleNamespace

import pytest
import torch

from block_diffusion_drafter_kv_gb300 import binding as B
from block_diffusion_drafter_kv_gb300.generate import spec_generate
from synthetic_target import greedy_reference
from test_generate_logprobs_host import IDS, Scoring, target


class Pooled(Scoring):
    """A drafter over a pool of one sequence and so many pages, which refuses as the library's does; it
    fails if it is asked to work on positions that were refused."""

    def __init__(self, pages_left):
        super().__init__(1024, 8, 77)
        self.blocks = []
        self.room = 64 * pages_left

        def reserve(length, n_new, rows, batch, slots=None, stream=None):
            have = int(length[0]) + int(n_new[0]) <= self.room
            for r in range(rows if slots is not None else 0):
                slots[r] = int(length[0]) + r if have and r < int(n_new[0]) else -1
        self.pages = SimpleNamespace(reserve=reserve, release=lambda length, batch, stream=None: None)

    def inject(self, hidden, rows_per_seq, n_new, batch, stream=None):
        super().inject(hidden, rows_per_seq, n_new, batch)
        assert int(self.len[0]) <= self.room

    def draft(self, batch, block, drafted, logits=None, x_trace=None, stream=None):
        assert int(self.len[0]) + block <= self.room
        self.blocks.append(block)
        super().draft(batch, block, drafted)

    def verify(self, logits, drafted, batch, block, acc, com, stream=None):
        assert logits.shape[1] == block
        part = torch.zeros(1, block, dtype=torch.int32)
        super().verify(logits, drafted, batch, block, acc, part)
        com[:, :block] = part


def test_no_pages_for_the_prompt():
    d, t = Pooled(0), target()
    with pytest.raises(B.DFlashError) as e:
        spec_generate(d, t, IDS, 30)
    assert e.value.status == B.DFLASH_E_CAPACITY and int(d.len[0]) == 0 and t.n == 0


@pytest.mark.parametrize("pages", [1, 2])
def test_blocks_shrink_until_the_last_position_is_taken(pages):
    """Every position of the pages is used: the last token to come out is the one that has none."""
    d, t = Pooled(pages), target()
    most = 64 * pages - len(IDS) + 1
    out, st = spec_generate(d, t, IDS, most, logprobs=2)
    assert out == greedy_reference(target(), IDS, most) and len(st.token_logprobs) == len(st.top_logprobs) == most
    assert 1 <= min(d.blocks) < 8 == max(d.blocks) and int(d.len[0]) == t.n == 64 * pages
    d = Pooled(pages)
    with pytest.raises(B.DFlashError) as e:
        spec_generate(d, target(), IDS, most + 1)
    assert e.value.status == B.DFLASH_E_CAPACITY and int(d.len[0]) == 64 * pages


def test_pages_enough_change_nothing():
    out, st = spec_generate(Pooled(4), target(), IDS, 100)
    assert out == greedy_reference(target(), IDS, 100)
