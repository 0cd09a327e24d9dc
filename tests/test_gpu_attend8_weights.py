"""What the 8-bit cache's attention keeps of small weights (cache_cases.py has the other tolerances).

A weight is pieces of e4m3, each 32 times the rest of the one before, that end at 2^-10 / 32 = 2^-15 (bf16) or 2^-10 / 32^2 =
2^-20 (fp16): that much of each may be lost, times values of at most 448. It is measured against a row's reference, which
makes a step's largest product of a weight and its V row's scale 16, and is looked at in one step (128 keys) of 8: 2 points for a
largest product of 8 or more, -1 for a smaller one; from 4 points at most down to -1 it is set anew. With m good looks there are
at most 5 + 3 m of 1024 keys each until then (or 4 + 3 m and a last, shorter one with up to 3 steps that are not looked at),
whose steps' largest products sum to 16 + 8 m or more: (5.4 + 3 m) / (16 + 8 m) <= 3 / 8. So the loss is at most
3 / 8 x 1024 x 2^-15 (2^-20) x 448 of the sum of the steps' largest products, which the sum over tiles of 64 keys of theirs is
not below, and does not grow with the keys. Behind a key that is 2^12 or more above all before it the points are none, and
the next look is at most 8 steps away: where what follows is even, 1024 / 16 of those 2^-15 (2^-20)."""
import pytest
import torch

from cache_cases import F8, HALF, ints, quantised

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def B():
    from block_diffusion_drafter_kv_gb300 import binding
    from block_diffusion_drafter_kv_gb300.build import build
    build()
    return binding


def check(got, q, k, v, vf, scale, lost=384):
    """got, q [h][d] of one KV head against its keys' values k, v [n][d] and V's scales vf [n], in 64 bits.
    lost: weights of the last piece's least that are, of each tile's largest product."""
    n, d = k.shape
    half = q.dtype == torch.float16
    q = q.double()
    sc = q @ k.t() * scale
    mag = (q.abs() @ k.abs().t()).amax(-1, keepdim=True) * scale
    far = q.abs().amax(-1, keepdim=True) * k.abs().sum(-1).amax() * scale * 2.0 ** -17
    err = (3 * d + 8) * 2.0 ** -23 * 1.1 * mag + far + 2.0 ** -20
    e = torch.exp(sc - sc.amax(-1, keepdim=True))
    tot = e.sum(-1, keepdim=True)
    want, w = e @ v / tot, e @ v.abs() / tot
    tol = (2 * err + (2.0 ** -11 + 2.0 ** -12 if half else 2.0 ** -8) + 2 * (3 * n + 64) * 2.0 ** -23) * w
    most = torch.nn.functional.pad(e * vf, (0, -n % 64)).unflatten(-1, (-1, 64)).amax(-1).sum(-1, keepdim=True)
    tol = tol + lost * (2.0 ** -20 if half else 2.0 ** -15) * 448 * most / tot
    tol = tol + HALF[torch.float16 if half else torch.bfloat16] * want.abs() + (2.0 ** -25 if half else 0.0)
    off = (got.double() - want).abs() - tol
    assert bool((off <= 0).all()), (off.max().item(), ((got.double() - want).abs() / w).max().item())


class OneCache:
    """As many sequences as the card has ranges, all over the same pages, so that a range is a whole sequence of n keys:
    one KV head, nq query heads, one new row."""

    def __init__(self, B, nq, d, dtype, n, k, v, scale):
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        self.seqs = sms * (4 if nq <= 16 else 2 if nq <= 32 else 1)
        pages = -(-n // 64)
        self.pool = B.PagePool(pages, pages, self.seqs)
        self.pool.page_table.copy_(torch.arange(pages, device="cuda").expand(self.seqs, -1))
        self.len, self.new = ints([n - 1] * self.seqs), ints([1] * self.seqs)
        self.cache = B.PagedCache(1, nq, 1, d, self.pool, self.len, dtype=dtype, bits=8, scale=scale)
        self.values = []
        at = torch.arange(n, device="cuda")
        for which, (x, p) in enumerate(((k, self.cache.k_pool), (v, self.cache.v_pool))):
            y, s = quantised(x)
            p.view(torch.uint8)[0, at, 0] = y.view(torch.uint8)
            self.cache.scales[0, at // 64, 0, which, at % 64] = s
            self.values.append(y.view(F8).double() * torch.exp2(s.double() - 127)[:, None])
        self.vf = torch.exp2(s.double() - 127)

    def attend(self, q):
        qs = q.expand(self.seqs, -1, -1).contiguous()
        out = torch.full_like(qs, 3.0)
        self.cache.attend(0, qs, self.new, self.seqs, 1, out)
        assert self.cache.device_error() == 0
        return out


@pytest.mark.parametrize("dtype,nats", [(torch.bfloat16, x) for x in (11.0, 12.0, 12.5, 13.0)] + [(torch.float16, x) for x in (14.0, 15.0, 16.0)])
@pytest.mark.parametrize("nq,d", [(4, 128), (4, 64), (20, 128), (64, 128), (128, 128)])
def test_one_key_far_above_many(B, dtype, nats, nq, d):
    """One key whose weight is e^11 to e^16 times each of 30000 others', which have up to a third of the sum together:
    as where the first position of a context draws most of the weight."""
    n = 30000
    g = torch.Generator(device="cuda").manual_seed(nq + d)
    q = (1 + 0.05 * torch.randn(nq, d, generator=g, device="cuda")).to(dtype)
    for place in (0, n // 2 + 77):
        k = -0.5 * (1 + 0.02 * torch.randn(n, d, generator=g, device="cuda"))
        v = 1 + 0.5 * torch.randn(n, d, generator=g, device="cuda")
        k[place], v[place] = 0.5, -v[place]
        c = OneCache(B, nq, d, dtype, n, k, v, scale=nats / d)
        out = c.attend(q)
        assert bool((out == out[:1]).all())     # every range had the same to do
        check(out[0], q, *c.values, c.vf, nats / d, lost=64)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nq,d", [(1, 64), (16, 128), (32, 128), (64, 64), (128, 128)])
def test_scores_that_rise_and_fall(B, dtype, nq, d):
    """Levels of the scores that change by up to 40 nats every 100 to 700 keys, other heads with other slopes; rows of zeros
    and rows of large values among them."""
    n = 9000
    g = torch.Generator(device="cuda").manual_seed(nq + d)
    q = (1 + 0.3 * torch.randn(nq, d, generator=g, device="cuda")).to(dtype)
    k, v = torch.empty(n, d, device="cuda"), torch.randn(n, d, generator=g, device="cuda")
    at, step = 0, 100
    for level in [0.2, -0.6, -0.1, 0.5, -1.0, -0.9, 0.4, -0.3, 1.0, 0.0, -0.8, 0.3, 0.7, -0.2, 0.1, -1.0, 0.9] * 3:
        end = min(n, at + step)
        k[at:end] = level + 0.1 * torch.randn(end - at, d, generator=g, device="cuda")
        at, step = end, 100 + (step * 7 + 13) % 600
    k[at:] = -1.0
    v[2000:2400] = 0
    v[3000:3100] *= 1000
    c = OneCache(B, nq, d, dtype, n, k, v, scale=20 / d)
    out = c.attend(q)
    assert bool((out == out[:1]).all())
    check(out[0], q, *c.values, c.vf, 20 / d)
