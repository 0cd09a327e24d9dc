"""Independent page pools at sizes that need more shared memory than a launch gets unasked: used by host
threads of their own, and captured into one graph, the larger pool's call first."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
SIZES = (8192, 2500)


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


class Set:
    def __init__(self, B, batch):
        self.batch, self.pool = batch, B.PagePool(2 * batch, 2, batch)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.news = torch.full((batch,), 70, dtype=torch.int32, device="cuda")
        self.slots = torch.zeros(70 * batch, dtype=torch.int32, device="cuda")

    def reserve(self, slots=None):
        self.pool.reserve(self.lens, self.news, 70, self.batch, slots)

    def release(self):
        self.pool.release(self.lens, self.batch)

    def check(self):
        """All pages handed out in order, two to a sequence."""
        want = 128 * torch.arange(self.batch, device="cuda")[:, None] + torch.arange(70, device="cuda")
        assert torch.equal(self.slots.reshape(self.batch, 70).long(), want)
        assert self.pool.held.tolist() == [2] * self.batch and int(self.pool.n_free) == 0 and self.pool.device_error() == 0


def test_threads_with_pools_of_different_sizes(B):
    """The bare library call in a tight loop (a call with the wrapper's checks around it is too seldom in the
    library for two of them to meet there)."""
    errors = []
    start = threading.Barrier(6)

    def work(batch):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                s = Set(B, batch)
                f, lens = s.pool.L.dflash_pages_reserve, s.lens.data_ptr()
                args = (s.pool._ref, lens, lens, batch, 70, None, stream.cuda_stream)
                start.wait()
                refused = sum(f(*args) != 0 for _ in range(20000))
                assert refused == 0
                s.reserve(s.slots)
                s.check()
        except BaseException as e:  # noqa: BLE001  (shown by the test)
            errors.append((batch, repr(e)))
            start.abort()

    threads = [threading.Thread(target=work, args=(SIZES[i % 2],)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert errors == []


def test_two_sizes_in_one_graph(B):
    sets = [Set(B, n) for n in SIZES]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for s in sets:
            s.reserve(s.slots)
    g.replay()
    for s in sets:
        s.check()
    sets[1].release()
    sets[1].reserve()
    sets[0].release()
    sets[1].release()
    g.replay()                                     # after calls of the smaller one
    for s in sets:
        s.check()
