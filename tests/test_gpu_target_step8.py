"""The 8-bit cache, the shared prefix and reading back together, as a serving step uses them: a system prompt read
once and moved to a place of its own, chats that decode behind it, blocks with rejected tails, and a cache that
leaves the card and comes back. And what the calls refuse."""
import ctypes

import pytest
import torch

from cache_cases import CAP, ints
from test_gpu_target_step import D, LAYERS, NKV, NQ, Target

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


class Shared(Target):
    """The target of the 16-bit tests over a cache of either width, its sequences behind sequence `seqs`."""

    def __init__(self, B, seqs, bits):
        super().__init__(B, seqs)
        self.pages = B.PagePool(8 * (seqs + 1), 8, seqs + 1)
        self.len = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
        self.cache = B.PagedCache(LAYERS, NQ, NKV, D, self.pages, self.len, dtype=self.dtype, rope_cos=self.cos, rope_sin=self.sin,
                                  bits=bits, shared_rows=seqs * 16)

    def step(self, tokens, n_new, batch, prefix=None):
        """Hidden states (before the head) of up to 16 rows a sequence."""
        rows = tokens.shape[1]
        x = self.embed[tokens.reshape(-1).long()]
        slots = torch.empty(batch * rows, dtype=torch.int32, device="cuda")
        self.pages.reserve(self.len, n_new, rows, batch, slots)
        q_out = torch.zeros(batch * rows, NQ, D, dtype=self.dtype, device="cuda")
        out = torch.zeros_like(q_out)
        for l in range(LAYERS):
            q, k, v = (self.norm(x) @ self.wqkv[l]).to(torch.float16).split([NQ * D, NKV * D, NKV * D], 1)
            self.cache.append(l, q, k, v, slots, batch, rows, q_out, prefix=prefix)
            self.cache.attend(l, q_out, n_new, batch, rows, out, prefix=prefix)
            x = x + out.reshape(-1, NQ * D).double() @ self.wo[l]
        return (self.norm(x) @ self.head).float()


@pytest.mark.parametrize("bits", [16, 8])
def test_chats_behind_a_system_prompt(B, bits):
    """Against the same target in float64 without a cache, over prompt and chat together.

    Tolerance: as for the 16-bit step, 0.07 for logits of standard deviation 3 and at most 13; in 8 bits K and
    V are rounded to 2^-4 of each value (uniformly, 2^-4 / sqrt 3 in the mean) instead of 2^-11: scores of a unit move by
    2^-4 / sqrt(3 D) of |q| |k| and outputs by 2^-4 / sqrt 3 of one value, so by at most a twelfth of the
    attention's part of the residual a layer; two layers, logits of deviation 3: 0.5 in the mean square, and 2.5 for
    the largest of some thousand."""
    seqs = 4
    t = Shared(B, seqs, bits)
    g = torch.Generator().manual_seed(5)
    prompt = torch.randint(0, t.embed.shape[0], (150,), generator=g).tolist()
    for i in range(0, 150, 16):                                          # the prompt, as sequence 0
        part = prompt[i: i + 16]
        toks = torch.tensor([part + [0] * (16 - len(part))], device="cuda")
        t.step(toks, ints([len(part)]), 1)
        t.len[0] += len(part)
    free = int(t.pages.n_free)
    t.pages.move(0, seqs, t.len)
    assert t.len.tolist() == [0] * seqs + [150] and t.pages.held.tolist() == [0] * seqs + [3] and int(t.pages.n_free) == free
    chats = [[] for _ in range(seqs)]
    worst, squares = 0.0, []
    for rows, news, keep in ((5, [5, 1, 3, 2], [5, 1, 3, 2]), (1, [1] * 4, [1, 1, 1, 1]), (16, [16, 16, 9, 0], [3, 16, 1, 0]),
                             (1, [1] * 4, [1] * 4), (16, [16] * 4, [16, 2, 7, 16]), (7, [7, 1, 7, 7], [7, 1, 7, 7])):
        toks = torch.randint(0, t.embed.shape[0], (seqs, rows), generator=g)
        z = t.step(toks.cuda(), ints(news), seqs, prefix=seqs).reshape(seqs, rows, -1)
        for s in range(seqs):
            if news[s]:
                full = t.whole(prompt + chats[s] + toks[s, : news[s]].tolist())[150 + len(chats[s]):]
                off = (z[s, : news[s]].double() - full).abs()
                worst = max(worst, off.max().item())
                squares.append(off.square().mean().item())
            chats[s] += toks[s, : keep[s]].tolist()
        t.len[:seqs] += ints(keep)
        t.pages.release(t.len, seqs)
        assert t.pages.device_error() == 0 and t.cache.device_error() == 0
    assert worst <= (0.07 if bits == 16 else 2.5)
    assert (sum(squares) / len(squares)) ** 0.5 <= (0.07 if bits == 16 else 0.5)
    # a chat leaves the card and comes back in other pages: the same values
    n = int(t.len[0])
    before, k, v = [], [], []
    for l in range(LAYERS):
        k.append(torch.zeros(n, NKV, D, dtype=t.dtype, device="cuda"))
        v.append(torch.zeros_like(k[l]))
        t.cache.read(l, ints([0]), ints([n]), 1, n, k[l], v[l])
    t.len[0] = 0
    t.pages.release(t.len, 1)
    hold = ints([64])
    t.pages.reserve(torch.zeros(seqs, dtype=torch.int32, device="cuda"), ints([0, 0, 0, 64]), 64, seqs)   # pages move on
    del hold
    slots = torch.empty(n, dtype=torch.int32, device="cuda")
    t.pages.reserve(t.len, ints([n]), n, 1, slots)
    plain = B.PagedCache(LAYERS, NQ, NKV, D, t.pages, t.len, dtype=t.dtype, bits=bits, k_pool=t.cache.k_pool, v_pool=t.cache.v_pool,
                         scales=t.cache.scales)                           # (no rotation: the rows have theirs)
    for l in range(LAYERS):
        plain.append(l, None, k[l], v[l], slots, 1, n, None)
        k2, v2 = torch.zeros_like(k[l]), torch.zeros_like(v[l])
        t.cache.read(l, ints([0]), ints([n]), 1, n, k2, v2)
        assert torch.equal(k[l], k2) and torch.equal(v[l], v2)
    del before


def test_pages_that_move(B):
    p = B.PagePool(20, 6, 5)
    length = ints([100, 0, 300, 7, 0])
    p.reserve(torch.zeros(5, dtype=torch.int32, device="cuda"), length, 300, 5)
    table, held = p.page_table.clone(), p.held.tolist()
    p.move(2, 4, length)
    assert p.device_error() == 0 and length.tolist() == [100, 0, 0, 7, 300] and p.held.tolist() == [held[0], 0, 0, held[3], held[2]]
    assert torch.equal(p.page_table[4], table[2]) and bool((p.page_table[2] == -1).all())
    assert torch.equal(p.page_table[0], table[0]) and torch.equal(p.page_table[3], table[3])
    p.move(0, 4)                      # sequence 4 holds pages
    assert p.device_error() == CAP and p.held.tolist() == [held[0], 0, 0, held[3], held[2]]
    p.move(1, 2)                      # nothing to move
    assert p.device_error() == 0
    for a, b, status in ((1, 1, -1), (-1, 2, -1), (0, -1, -1), (5, 0, -3), (0, 5, -3)):
        with pytest.raises(B.DFlashError) as e:
            p.move(a, b)
        assert e.value.status == status
    p.release(torch.zeros(5, dtype=torch.int32, device="cuda"), 5)
    assert int(p.n_free) == 20


def test_refusals(B):
    """What the host can see is refused before anything runs."""
    pool = B.PagePool(8, 4, 4)
    length = ints([10, 10, 10, 10])
    q = torch.zeros(8, 8, 64, dtype=torch.float16, device="cuda")
    kv = torch.zeros(8, 2, 64, dtype=torch.float16, device="cuda")
    slots, n = ints([-1] * 8), ints([1] * 4)
    for bits in (16, 8):
        c = B.PagedCache(2, 8, 2, 64, pool, length, bits=bits, shared_rows=4)
        L, ws, size = c.L, (c._shared.data_ptr() + 255) // 256 * 256, c._shared_bytes
        args = (q.data_ptr(), n.data_ptr())
        for prefix in (-1, 0, 1, 4, 100):
            with pytest.raises(B.DFlashError) as e:
                c.attend(0, q[:2], n, 2, 1, q[2:4].clone(), prefix=prefix)
            assert e.value.status == -1, prefix
            with pytest.raises(B.DFlashError) as e:
                c.append(0, q[:2], kv[:2], kv[:2], slots[:2], 2, 1, q[2:4].clone(), prefix=prefix)
            assert e.value.status == -1, prefix
        with pytest.raises(B.DFlashError) as e:       # more rows than the workspace was asked for
            c.attend(0, q, n, 2, 4, q.clone(), prefix=3)
        assert e.value.status == -3
        f = L.dflash_cache_attend_shared
        assert f(c.c, 0, *args, 1, 1, 2, q.data_ptr(), None, size, None) == -1
        assert f(c.c, 0, *args, 1, 1, 2, q.data_ptr(), ws + 16, size, None) == -1
        assert f(c.c, 0, *args, 1, 1, 2, q.data_ptr(), ws, 1000, None) == -3
        assert f(c.c, 2, *args, 1, 1, 2, q.data_ptr(), ws, size, None) == -1
        assert f(c.c, 0, *args, 0, 1, 2, q.data_ptr(), ws, size, None) == -1
        assert f(c.c, 0, q.data_ptr() + 2, n.data_ptr(), 1, 1, 2, q.data_ptr(), ws, size, None) == -1
        for a in ((-1, ints([0]), ints([1]), 1, 1), (2, ints([0]), ints([1]), 1, 1)):
            with pytest.raises(B.DFlashError):
                c.read(*a, kv[:1], kv[1:2].clone())
        with pytest.raises(B.DFlashError) as e:
            c.read(0, ints([0] * 8), ints([0] * 8), 8, 1, kv, kv.clone())
        assert e.value.status == -3
        with pytest.raises(B.DFlashError):
            c.read(0, ints([0]), ints([1]), 1, 1, kv[:1].float(), kv[:1].float())
        h = ctypes.c_void_p()
        assert L.dflash_cache_create(ctypes.byref(c.cfg), ctypes.byref(h)) == 0
        assert f(h, 0, *args, 1, 1, 2, q.data_ptr(), ws, size, None) == -5
        assert L.dflash_cache_read(h, 0, n.data_ptr(), n.data_ptr(), 1, 1, B.F16, kv.data_ptr(), kv.data_ptr(), None) == -5
        ptrs = (c.k_pool.data_ptr(), c.v_pool.data_ptr())
        rest = (pool.page_table.data_ptr(), length.data_ptr(), None, None, (c.workspace.data_ptr() + 255) // 256 * 256)
        nbytes = L.dflash_cache_workspace_size(ctypes.byref(c.cfg))
        if bits == 8:                                 # without scales, or with misaligned ones
            assert L.dflash_cache_bind(h, *ptrs, *rest, nbytes) == -1
            assert L.dflash_cache_bind_8bit(h, *ptrs, c.scales.data_ptr() + 4, *rest, nbytes) == -1
            assert L.dflash_cache_bind_8bit(h, *ptrs, None, *rest, nbytes) == -1
            assert L.dflash_cache_bind_8bit(h, *ptrs, c.scales.data_ptr(), *rest, nbytes - 1) == -3
        else:                                         # scales for a 16-bit cache
            assert L.dflash_cache_bind_8bit(h, *ptrs, q.data_ptr(), *rest, nbytes) == -1
        assert L.dflash_cache_destroy(h) == 0
        assert c.device_error() == 0
