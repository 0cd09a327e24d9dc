"""Log probabilities of so many rows that products of their number pass 31 bits."""
import pytest
import torch

from test_gpu_logprobs import check, make  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_tokens", [False, True])
def test_more_than_two_to_the_28_rows(make, with_tokens):  # noqa: F811
    rows, step = 2 ** 28 + 3, 2 ** 24
    g = torch.Generator(device="cuda").manual_seed(3)
    dr = make(2)
    z = torch.empty(rows, 2, dtype=torch.float16, device="cuda")
    z.copy_(torch.randn(step, 2, generator=g, device="cuda")[torch.arange(rows, device="cuda") % step])
    t = torch.randint(-1, 2, (rows,), generator=g, device="cuda", dtype=torch.int32) if with_tokens else None
    lp = torch.full((rows,), 9.0, device="cuda") if with_tokens else None
    h = torch.full((rows,), 9.0, device="cuda")
    dr.logprobs(z, t, lp, h)
    assert dr.device_error() == 0
    for a in range(0, rows, step):
        b = min(rows, a + step)
        part = [None if x is None else x[a:b] for x in (t, lp, h)]
        check(z[a:b], part[0], (part[1], part[2], None, None), 0)
