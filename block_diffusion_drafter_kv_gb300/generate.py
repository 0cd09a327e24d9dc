"""End-to-end speculative generation with the DFlash drafter (the user-level loop the pages
show as spec_generate(input_ids, max_new_tokens, temperature, target, stop_token_ids):
7minutos.es, "Ejecutando DFlash").

Every step of the draft-and-verify path runs in the library's kernels through the C ABI;
this module only sequences the calls around the caller's target model:

  prefill   the target reads the prompt; the hidden states of its tapped layers at every
            prompt position are injected into the drafter's KV cache, and the target's own
            next token becomes slot 0 of the first block
  repeat    draft a block of B slots (slot 0 = last committed token, slots 1..B-1 drafted)
            -> the target runs once over those B tokens -> verification keeps the longest
            valid prefix plus one token of the target's own (greedy, or speculative
            sampling at temperature > 0) -> the target drops the rejected positions -> the
            hidden states of the tau kept positions are injected -> the last committed
            token becomes the next slot 0

Greedy generation is lossless: the committed tokens are exactly the target's own greedy
continuation (theaistack.guide, "DFlash").

The target is any object with three methods:
  prefill(input_ids int64 [P]) -> (tapped bf16 [k, P, Ht], logits fp32 [V] after the last token)
  forward_block(tokens int64 [B]) -> (tapped bf16 [k, B, Ht], logits fp32 [B, V]); row i
      predicts the token after tokens[i]; the B positions are appended to its cache
  truncate(length) keeps the first `length` positions of its cache
"""
from __future__ import annotations

from dataclasses import dataclass, field
from typing import List, Optional, Sequence, Tuple

import torch

from .binding import DFLASH_E_CAPACITY, PAGE_POSITIONS, DFlashError


@dataclass
class GenerationStats:
    steps: int = 0                       # draft-and-verify steps
    accept_lens: List[int] = field(default_factory=list)
    # with logprobs=n, one entry per new token, under the target's distribution at temperature 1:
    token_logprobs: List[float] = field(default_factory=list)
    token_entropies: List[float] = field(default_factory=list)
    top_logprobs: List[List[Tuple[int, float]]] = field(default_factory=list)  # n (token, log probability), best first

    @property
    def mean_tau(self) -> float:
        return sum(self.accept_lens) / max(1, len(self.accept_lens))


def spec_generate(drafter, target, input_ids, max_new_tokens: int, temperature: float = 0.0,
                  stop_token_ids: Sequence[int] = (), block: Optional[int] = None,
                  generator: Optional[torch.Generator] = None, stream=None, logprobs: Optional[int] = None):
    """Generate up to max_new_tokens tokens after input_ids (a 1-D token sequence) with the
    drafter (a binding.Drafter bound with max_batch >= 1; sequence slot 0 is used and reset)
    and the caller's target. Generation stops after the first token in stop_token_ids.
    temperature > 0 verifies by speculative sampling with uniforms drawn from `generator`.
    logprobs=n (0..32) also collects every new token's log probability, the entropy of its
    distribution and the n most likely tokens at its place in the stats. A drafter bound with
    `pages` gets its pages as the sequence grows. Where the pool or the table has no further page for
    it, blocks shrink to what is left of its last one; where nothing is left, or the prompt has no
    room, DFlashError (capacity exceeded) is raised before drafter and target go on. The pool's flag
    is set in either case. With a `stream` (torch.cuda.Stream) all of it, the
    target's calls included, runs on that stream, after what the current one has queued and before
    what it queues next. Returns (new tokens as a list of ints, GenerationStats)."""
    if stream is None:
        return _generate(drafter, target, input_ids, max_new_tokens, temperature, stop_token_ids, block, generator, logprobs)
    caller = torch.cuda.current_stream(stream.device)
    stream.wait_stream(caller)
    try:
        # the library's calls take the current stream, so that they, torch's and the target's are in one order
        with torch.cuda.stream(stream):
            return _generate(drafter, target, input_ids, max_new_tokens, temperature, stop_token_ids, block, generator, logprobs)
    finally:
        caller.wait_stream(stream)


def _generate(drafter, target, input_ids, max_new_tokens, temperature, stop_token_ids, block, generator, logprobs):
    """spec_generate on the current stream."""
    dev = drafter.last_token.device
    B = block or drafter.cfg.max_block
    V = drafter.shape.vocab
    stops = set(int(t) for t in stop_token_ids)
    out: List[int] = []
    stats = GenerationStats()
    if max_new_tokens <= 0:
        return out, stats

    def pick(logits_row):
        if temperature > 0:
            p = torch.softmax(logits_row.double() / temperature, dim=-1)
            u = torch.rand((), generator=generator, device=logits_row.device, dtype=torch.float64)
            return int(min(int(torch.searchsorted(torch.cumsum(p, 0), u, right=True)), V - 1))
        return int(torch.argmax(logits_row))

    def score(rows, tokens):
        """(log probability, entropy, alternatives) of each token >= 0 from its row of logits."""
        n = rows.shape[0]
        lp, ent, tv = (torch.empty(k, dtype=torch.float32, device=dev) for k in (n, n, n * logprobs))
        ti = torch.empty(n * logprobs, dtype=torch.int32, device=dev)
        drafter.logprobs(rows, tokens, lp, ent, ti if logprobs else None, tv if logprobs else None)
        alts = [list(zip(i, v)) for i, v in zip(ti.reshape(n, logprobs).tolist(), tv.reshape(n, logprobs).tolist())]
        return list(zip(lp.tolist(), ent.tolist(), alts))

    def emit(tokens, scores) -> bool:
        for k, t in enumerate(tokens):
            out.append(int(t))
            if scores is not None:
                for to, x in zip((stats.token_logprobs, stats.token_entropies, stats.top_logprobs), scores[k]):
                    to.append(x)
            if int(t) in stops or len(out) >= max_new_tokens:
                return True
        return False

    pages = getattr(drafter, "pages", None)
    n_cached = 0

    def make_room(n: int) -> int:
        """Pages for the next n positions; returns how many of them there is room for. A refused sequence
        has -1 in its slots (the pool's flag would also tell of other sequences than this one)."""
        n_new, slots = torch.full((1,), n, dtype=torch.int32, device=dev), torch.zeros(n, dtype=torch.int32, device=dev)
        pages.reserve(drafter.len, n_new, n, 1, slots)
        return n if int(slots[0]) >= 0 else min(n, -n_cached % PAGE_POSITIONS)

    ids = torch.as_tensor(input_ids, dtype=torch.int64, device=dev).reshape(-1)
    P = ids.numel()
    drafter.len[:1].zero_()
    if pages is not None:
        pages.release(drafter.len, 1)   # what an earlier sequence in the slot still holds
        if make_room(P) < P:
            raise DFlashError(DFLASH_E_CAPACITY, f"no pages for a prompt of {P} positions")
    tapped, logits = target.prefill(ids)
    drafter.inject(tapped.contiguous(), P, torch.tensor([P], dtype=torch.int32, device=dev), 1)
    first = pick(logits.reshape(-1))
    drafter.last_token[0] = first
    scores = None
    if logprobs is not None:
        scores = score(logits.to(torch.float32).reshape(1, V), drafter.last_token[:1])
    if emit([first], scores):
        return out, stats
    drafted = torch.zeros(1, max(B - 1, 1), dtype=torch.int32, device=dev)
    acc = torch.zeros(1, dtype=torch.int32, device=dev)
    com = torch.zeros(1, B, dtype=torch.int32, device=dev)
    n_cached = P
    n = B   # slots of the block
    while True:
        if pages is not None:
            n = make_room(B)
            if n == 0:
                raise DFlashError(DFLASH_E_CAPACITY, f"no pages for a block after {len(out)} new tokens")
        drafter.draft(1, n, drafted)
        block_tokens = torch.cat([drafter.last_token[:1].to(torch.int64), drafted[0, : n - 1].to(torch.int64)])
        tapped, logits = target.forward_block(block_tokens)
        logits = logits.to(torch.float32).reshape(1, n, V).contiguous()
        if temperature > 0:
            u = torch.rand(1, n, generator=generator, device=dev, dtype=torch.float32)
            drafter.verify_sampling(logits, drafted, u, temperature, 1, n, acc, com)
        else:
            drafter.verify(logits, drafted, 1, n, acc, com)
        tau = int(acc[0])
        stats.steps += 1
        stats.accept_lens.append(tau)
        target.truncate(n_cached + tau)   # keep slot 0 and the accepted drafts
        rows = torch.zeros(tapped.shape[0], n, tapped.shape[2], dtype=torch.bfloat16, device=dev)
        rows[:, :tau] = tapped[:, :tau]
        drafter.inject(rows, n, acc, 1)
        n_cached += tau
        if logprobs is not None:
            scores = score(logits[0], com[0, :n])
        if emit(com[0, :tau].tolist(), scores):
            return out, stats
