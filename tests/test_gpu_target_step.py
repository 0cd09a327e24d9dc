"""The target-side operators together, as a step uses them: a small causal target whose cache,
rotary positions and attention run in the library, verified against the same target in float64
without a cache; and generation with log probabilities over a drafter whose pages a pool keeps."""
import numpy as np
import pytest
import torch

from synth import TINY, W_TINY
from synth import inputs as I

pytestmark = pytest.mark.gpu
LAYERS, NQ, NKV, D, H, V = 2, 6, 2, 64, 384, TINY.vocab


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


class Target:
    """Pre-norm attention layers and a head; projections in float64 on both sides, so that only
    the operators differ."""

    def __init__(self, B, seqs, dtype=torch.float16):
        g = torch.Generator(device="cuda").manual_seed(11)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
        self.B, self.seqs, self.dtype = B, seqs, dtype
        self.embed, self.head = rnd(V, H), rnd(H, V) * 3 / H ** 0.5
        self.wqkv = [rnd(H, (NQ + 2 * NKV) * D) / H ** 0.5 for _ in range(LAYERS)]
        self.wo = [rnd(NQ * D, H) / (NQ * D) ** 0.5 for _ in range(LAYERS)]
        self.cos, self.sin = B.rope_tables(8 * 64, 48, 1e4)
        self.pages = B.PagePool(8 * seqs, 8, seqs)
        self.len = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.cache = B.PagedCache(LAYERS, NQ, NKV, D, self.pages, self.len, dtype=dtype, rope_cos=self.cos, rope_sin=self.sin)

    def norm(self, x):
        return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()

    def step(self, tokens, n_new):
        """tokens [seqs][rows]; logits fp32 [seqs * rows][V] of every row, from the paged cache."""
        rows = tokens.shape[1]
        x = self.embed[tokens.reshape(-1).long()]
        slots = torch.empty(self.seqs * rows, dtype=torch.int32, device="cuda")
        self.pages.reserve(self.len, n_new, rows, self.seqs, slots)
        q_out = torch.zeros(self.seqs * rows, NQ, D, dtype=self.dtype, device="cuda")
        out = torch.zeros_like(q_out)
        for l in range(LAYERS):
            qkv = (self.norm(x) @ self.wqkv[l]).to(torch.float16)
            q, k, v = qkv.split([NQ * D, NKV * D, NKV * D], 1)
            self.cache.append(l, q, k, v, slots, self.seqs, rows, q_out)
            if rows <= 16:
                self.cache.attend(l, q_out, n_new, self.seqs, rows, out)
            else:   # a prompt, sixteen rows at a time: the later rows' keys are there already and hidden
                whole, base = q_out.reshape(self.seqs, rows, NQ, D), self.len.clone()
                for r in range(0, rows, 16):
                    part = whole[:, r: r + 16].contiguous()
                    o = torch.zeros_like(part)
                    self.cache.attend(l, part.reshape(-1, NQ, D), (n_new - r).clamp(0, part.shape[1]).to(torch.int32), self.seqs, part.shape[1], o)
                    out.reshape(self.seqs, rows, NQ, D)[:, r: r + 16] = o
                    self.len += (n_new - r).clamp(0, part.shape[1]).to(torch.int32)
                self.len.copy_(base)
            x = x + out.reshape(-1, NQ * D).double() @ self.wo[l]
        return (self.norm(x) @ self.head).float()

    def whole(self, seq):
        """Logits of every position of one sequence, without cache, pages or library."""
        n = len(seq)
        x = self.embed[torch.tensor(seq, device="cuda")]
        cos, sin = self.cos[:n, None].double(), self.sin[:n, None].double()
        causal = torch.ones(n, n, device="cuda").tril().bool()
        for l in range(LAYERS):
            q, k, v = (self.norm(x) @ self.wqkv[l]).split([NQ * D, NKV * D, NKV * D], 1)
            turned = []
            for t in (q.reshape(n, NQ, D), k.reshape(n, NKV, D)):
                a, b = t[..., :24], t[..., 24:48]
                turned.append(torch.cat([a * cos - b * sin, b * cos + a * sin, t[..., 48:]], -1))
            kk, vv = (t.repeat_interleave(NQ // NKV, 1) for t in (turned[1], v.reshape(n, NKV, D)))
            s = torch.einsum("ihd,jhd->hij", turned[0], kk) / 8
            p = torch.softmax(s.masked_fill(~causal, float("-inf")), -1)
            x = x + torch.einsum("hij,jhd->ihd", p, vv).reshape(n, -1) @ self.wo[l]
        return self.norm(x) @ self.head


def test_prompt_decode_and_blocks_equal_the_target_without_a_cache(B):
    """Prompts, single tokens, blocks with a rejected tail, a sequence that ends and is replaced.

    Tolerance: q, k, v, the weights and the outputs are each rounded to fp16 (2^-11 relative) in two
    layers whose residual stream they enter; logits of standard deviation 3 that are 10 such
    roundings deep stay within 10 x 2^-11 x max |logit| (about 13): 0.07."""
    t = Target(B, 3)
    dr = B.Drafter(TINY, I.make_weights(TINY, 2).to("cuda"), max_block=16, max_batch=3, kv_capacity=64)
    g = torch.Generator().manual_seed(5)
    seqs = [[], [], []]
    free0 = int(t.pages.n_free)

    def run(rows, n_new, keep):
        toks = torch.randint(0, V, (3, rows), generator=g)
        z = t.step(toks.cuda(), torch.tensor(n_new, dtype=torch.int32, device="cuda")).reshape(3, rows, V)
        nxt = torch.full((3, rows), -1, dtype=torch.int32)
        for s in range(3):
            full = t.whole(seqs[s] + toks[s, : n_new[s]].tolist())[len(seqs[s]):] if n_new[s] else None
            if full is not None:
                assert (z[s, : n_new[s]].double() - full).abs().max().item() <= 0.07
                nxt[s, : keep[s]] = full.argmax(1)[: keep[s]].int().cpu()
            seqs[s] += toks[s, : keep[s]].tolist()
        # the kept rows' log probabilities, straight from the step's logits
        lp, h = torch.zeros(3 * rows, device="cuda"), torch.zeros(3 * rows, device="cuda")
        ids, top = torch.zeros(3 * rows, 4, dtype=torch.int32, device="cuda"), torch.zeros(3 * rows, 4, device="cuda")
        dr.logprobs(z.reshape(-1, V), nxt.reshape(-1).cuda(), lp, h, ids, top)
        ln = torch.log_softmax(z.reshape(-1, V).double(), 1)
        m = (nxt.reshape(-1) >= 0).cuda()
        want = ln.gather(1, nxt.reshape(-1).clamp(min=0).long().cuda()[:, None])[:, 0]
        assert (lp[m].double() - want[m]).abs().max() < 1e-4 and bool((lp[~m] == 0).all())
        assert (h[m].double() + (ln.exp() * ln).sum(1)[m]).abs().max() < 1e-4
        assert torch.equal(ids[m].long(), torch.topk(ln, 4, 1).indices[m])
        t.len += torch.tensor(keep, dtype=torch.int32, device="cuda")
        t.pages.release(t.len, 3)
        assert t.len.tolist() == [len(s) for s in seqs]
        assert t.pages.held.tolist() == [-(-len(s) // 64) for s in seqs]

    run(70, [70, 33, 0], [70, 33, 0])      # two prompts
    for _ in range(3):
        run(1, [1, 1, 0], [1, 1, 0])       # token by token
    run(16, [16, 5, 16], [3, 5, 16])       # blocks, some of it rejected; the third sequence starts
    run(16, [16, 16, 1], [16, 1, 1])
    seqs[1] = []                           # the second ends and another takes its place
    t.len[1] = 0
    t.pages.release(t.len, 3)
    run(40, [1, 40, 7], [1, 40, 7])
    run(16, [16, 16, 16], [9, 16, 2])
    assert t.cache.device_error() == 0 and t.pages.device_error() == 0 and dr.device_error() == 0
    t.len.zero_()
    t.pages.release(t.len, 3)
    assert int(t.pages.n_free) == free0


def test_a_whole_step_captured_in_one_graph(B):
    """Reserve, append, attend, log probabilities and release replay as one graph with other lengths."""
    t = Target(B, 3)
    dr = B.Drafter(TINY, I.make_weights(TINY, 2).to("cuda"), max_block=16, max_batch=3, kv_capacity=64)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = 4
    qkv = torch.randn(3 * rows, (NQ + 2 * NKV) * D, generator=gen, device="cuda").half()
    z = torch.randn(3 * rows, V, generator=gen, device="cuda")
    tok, n_new = torch.zeros(3 * rows, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    slots = torch.zeros(3 * rows, dtype=torch.int32, device="cuda")
    q_out, out = (torch.zeros(3 * rows, NQ, D, dtype=torch.float16, device="cuda") for _ in range(2))
    lp, h = torch.zeros(3 * rows, device="cuda"), torch.zeros(3 * rows, device="cuda")

    def step():
        t.pages.reserve(t.len, n_new, rows, 3, slots)
        q, k, v = qkv.split([NQ * D, NKV * D, NKV * D], 1)
        t.cache.append(0, q, k, v, slots, 3, rows, q_out)
        t.cache.attend(0, q_out, n_new, 3, rows, out)
        dr.logprobs(z, tok, lp, h)
        t.len.add_(n_new)
        t.pages.release(t.len, 3)

    order = t.pages.free_list.clone()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    results = []
    for replay in (False, True):
        t.len.zero_()
        t.pages.release(t.len, 3)
        t.pages.free_list.copy_(order)     # both times the same pages in the same order
        t.cache.k_pool.zero_()
        t.cache.v_pool.zero_()
        seen = []
        for i in range(40):
            n_new.copy_(torch.tensor([i % 5, 4 - i % 5, 4], dtype=torch.int32).clamp(max=4))
            qkv.copy_(torch.randn(qkv.shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda"))
            out.zero_()
            graph.replay() if replay else step()
            seen.append([x.clone() for x in (slots, out, lp, h, t.len, t.pages.page_table)])
        results.append(seen)
    for a, b in zip(*results):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert t.cache.device_error() == 0 and t.pages.device_error() == 0


def test_generation_with_log_probabilities_over_a_page_pool(B):
    """spec_generate over a drafter whose pages grow with the sequence: the target's own greedy
    continuation, with every token's log probability from the target's logits."""
    from block_diffusion_drafter_kv_gb300.generate import spec_generate
    from synthetic_target import TinyTarget, greedy_reference
    w = I.make_weights(TINY, 21)
    for lw in w.layers:
        lw.wo.zero_()
        lw.w_down.zero_()
    pages = B.PagePool(12, 12, 1)
    dr = B.Drafter(TINY, w.to("cuda"), max_block=16, max_batch=1, kv_capacity=12 * 64, pages=pages)
    tgt = lambda: TinyTarget(TINY.vocab, TINY.target_hidden, seed=3, bias_token=77, bias=4.8, device="cuda")  # noqa: E731
    ids = torch.randint(0, TINY.vocab, (50,), generator=torch.Generator().manual_seed(1)).cuda()
    ref = greedy_reference(tgt(), ids, 120)
    for _ in range(2):                     # the second run takes the slot over
        out, st = spec_generate(dr, tgt(), ids, 120, logprobs=5)
        assert out == ref
        assert int(pages.held[0]) >= -(-int(dr.len[0]) // 64) and pages.device_error() == 0 and dr.device_error() == 0
    t = tgt()
    _, z = t.prefill(ids)
    for k, tok in enumerate(ref):
        ln = torch.log_softmax(z.reshape(-1).double(), 0)
        assert abs(st.token_logprobs[k] - ln[tok].item()) < 1e-3
        assert abs(st.token_entropies[k] + (ln.exp() * ln).sum().item()) < 1e-3
        assert st.top_logprobs[k][0][0] == tok and len(st.top_logprobs[k]) == 5
        assert np.allclose([v for _, v in st.top_logprobs[k]], torch.topk(ln, 5).values.tolist(), atol=1e-3)
        _, z = t.forward_block(torch.tensor([tok], device="cuda"))
