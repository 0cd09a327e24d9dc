"""The page pool against a list of pages kept in Python: reserve and release in any order, pools
that run out, lengths out of range, more sequences than threads, and replayed graphs."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
CAP = 2   # DFLASH_DEV_CAPACITY


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


class Model:
    def __init__(self, n_pages, pages_per_seq, max_batch):
        self.cols = pages_per_seq
        self.free = list(range(n_pages))[::-1]
        self.held = [[] for _ in range(max_batch)]
        self.flags = 0

    def reserve(self, lens, news, rows):
        want, slots = [], []
        for s, (a, n) in enumerate(zip(lens, news)):
            need = -(-(a + n) // 64)
            bad = a < 0 or n < 0 or n > rows or need > self.cols
            want.append(-1 if bad else max(0, need - len(self.held[s])))
        total, left = 0, len(self.free)
        for s, w in enumerate(want):
            total += max(w, 0)
            if w > 0 and total > left:
                want[s] = -1
        for s, w in enumerate(want):
            self.flags |= CAP * (w < 0)
            for _ in range(max(w, 0)):
                self.held[s].append(self.free.pop())
            for r in range(rows):
                p = lens[s] + r
                slots.append(self.held[s][p // 64] * 64 + p % 64 if w >= 0 and r < news[s] else -1)
        return slots

    def release(self, lens):
        gone = []
        for s, a in enumerate(lens):
            if a < 0:
                self.flags |= CAP
                continue
            keep = -(-a // 64)
            gone += self.held[s][keep:]
            del self.held[s][keep:]
        self.free += gone[::-1]

    def check(self, p):
        n = int(p.n_free)
        assert p.free_list[:n].tolist() == self.free
        assert p.held.tolist() == [len(h) for h in self.held]
        assert p.page_table.tolist() == [h + [-1] * (self.cols - len(h)) for h in self.held]
        assert p.device_error() == self.flags
        assert p.state[1:].tolist() == [0, 0, 0]
        self.flags = 0


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n_pages,cols,batch", [(1, 1, 1), (40, 3, 7), (700, 40, 33), (5000, 17, 300), (9000, 5, 4096), (9000, 5, 8192)])
def test_random_steps(B, n_pages, cols, batch):
    rng = random.Random(n_pages * 7 + batch)
    p, m = B.PagePool(n_pages, cols, batch), Model(n_pages, cols, batch)
    m.check(p)
    lens = [0] * batch
    for step in range(12):
        rows = rng.choice([1, 16, 70, 200])
        n = batch if step % 3 else rng.randint(1, batch)   # the sequences behind stay as they are
        news = [rng.choice([0, 1, rows, rng.randint(0, rows)]) for _ in range(n)]
        bad = rng.random() < 0.4
        if bad:
            news[rng.randrange(n)] = rng.choice([-1, rows + 1])
        use = lens[:n]
        if bad and rng.random() < 0.5:
            use[rng.randrange(n)] = rng.choice([-5, 64 * cols, 2 ** 31 - 1])
        slots = torch.full((n * rows + 3,), -7, dtype=torch.int32, device="cuda")
        p.reserve(ints(use), ints(news), rows, n, slots[: n * rows])
        want = m.reserve(use, news, rows)
        assert slots.tolist() == want + [-7] * 3
        m.check(p)
        for s in range(n):   # some of the new positions stay, some sequences end, one length is out of range
            if want[s * rows] >= 0:
                lens[s] = 0 if rng.random() < 0.2 else lens[s] + rng.randint(0, max(0, news[s]))
        back = list(lens[:n])
        if bad:
            back[rng.randrange(n)] = -1
        p.release(ints(back), n)
        m.release(back)
        m.check(p)


def test_release_of_a_reserve_restores_the_list(B):
    p = B.PagePool(100, 10, 8)
    lens, news = ints([5, 64, 0, 130, 63, 0, 1, 64]), ints([60, 1, 0, 200, 1, 300, 63, 0])
    p.reserve(lens, ints([0] * 8), 1, 8)   # pages for what is there: lengths alone
    before = [t.clone() for t in (p.page_table, p.held, p.free_list, p.state)]
    p.reserve(lens, news, 300, 8)          # no slots wanted
    assert int(p.n_free) < int(before[3][0])
    p.release(lens, 8)
    for a, b in zip(before, (p.page_table, p.held, p.free_list, p.state)):
        assert torch.equal(a, b)
    p.release(ints([0] * 8), 8)
    assert int(p.n_free) == 100 and sorted(p.free_list.tolist()) == list(range(100))


def test_inconsistent_state_is_refused_and_flagged(B):
    p = B.PagePool(8, 4, 2)
    p.held.copy_(ints([4, 4]))             # all eight pages held, and all eight free
    p.release(ints([0, 0]), 2)
    assert p.device_error() == CAP and int(p.n_free) == 8 and p.held.tolist() == [4, 4]
    p.held.copy_(ints([-1, 5]))
    slots = ints([9, 9])
    p.reserve(ints([0, 0]), ints([1, 1]), 1, 2, slots)
    assert p.device_error() == CAP and slots.tolist() == [-1, -1] and int(p.n_free) == 8


def test_captured_steps_replay(B):
    p, m = B.PagePool(200, 20, 5), Model(200, 20, 5)
    lens, news, slots = ints([0] * 5), ints([0] * 5), ints([0] * 5 * 40)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        p.reserve(lens, news, 40, 5, slots)
        p.release(lens, 5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.reserve(lens, news, 40, 5, slots)
    rng = random.Random(2)
    cur = [0] * 5
    for _ in range(6):
        n = [rng.randint(0, 40) for _ in range(5)]
        lens.copy_(ints(cur))
        news.copy_(ints(n))
        g.replay()
        assert slots.tolist() == m.reserve(cur, n, 40)
        m.check(p)
        cur = [a + b for a, b in zip(cur, n)]


def test_a_drafter_over_a_pool_equals_the_sequence_major_cache(B):
    """Injection and drafts of a paged drafter whose pages the pool hands out as it goes, step by step."""
    from synth import TINY
    from synth import inputs as I
    w = I.make_weights(TINY, 5).to("cuda")
    cap, batch, blk = 256, 3, 8
    pages = B.PagePool(3 * batch + 1, 4, batch)
    a = B.Drafter(TINY, w, max_block=blk, max_batch=batch, kv_capacity=cap)
    b = B.Drafter(TINY, w, max_block=blk, max_batch=batch, kv_capacity=cap, pages=pages)
    hid = I.make_hidden(TINY, 60 * batch, 3).cuda().contiguous()
    for step in range(3):
        n = ints([[60, 17, 1], [3, 60, 60], [1, 2, 60]][step])
        pages.reserve(b.len, n, 60, batch)
        out = []
        for d in (a, b):
            d.inject(hid, 60, n, batch)
            d.last_token.fill_(step + 1)
            if d is b:
                pages.reserve(b.len, ints([blk] * batch), blk, batch)
            drafted, logits = torch.zeros(batch, blk - 1, dtype=torch.int32, device="cuda"), torch.zeros(batch, blk - 1, TINY.vocab, device="cuda")
            d.draft(batch, blk, drafted, logits)
            out.append((drafted, logits, d.device_error()))
        pages.release(b.len, batch)
        assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1]) and out[0][2] == out[1][2] == 0
    assert pages.device_error() == 0
    with pytest.raises(B.DFlashError):
        B.Drafter(TINY, w, max_block=blk, max_batch=batch + 1, kv_capacity=cap, pages=pages)
