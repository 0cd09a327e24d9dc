"""Refusals of the binding's wrappers that need neither GPU nor library: objects on other devices, and
sizes that do not fit the library's 32-bit arguments."""
from types import SimpleNamespace

import pytest
import torch

from block_diffusion_drafter_kv_gb300 import binding as B

META = torch.device("meta")


def test_a_drafter_refuses_a_pool_of_another_device():
    """The kernels follow the table's pointer on the weights' device."""
    pool = object.__new__(B.PagePool)
    pool.max_batch, pool.n_pages, pool.page_table, pool.device = 4, 8, torch.zeros(4, 2, dtype=torch.int32), torch.device("cpu")
    w = SimpleNamespace(w_fc=torch.zeros(1, device=META))
    with pytest.raises(B.DFlashError) as e:
        B.Drafter(None, w, max_block=4, max_batch=2, kv_capacity=64, pages=pool)
    assert e.value.status == B.DFLASH_E_INVAL and "meta" in str(e.value)


def test_sizes_past_31_bits_are_refused_not_wrapped():
    """2^32 + 4 rows are not 4 rows."""
    d = object.__new__(B.Drafter)
    d.cfg, d.last_token, d.L = SimpleNamespace(vocab=8), torch.zeros(1, device=META), None
    p = object.__new__(B.PagePool)
    p.device, p.L = META, None
    lens = torch.zeros(4, dtype=torch.int32, device=META)
    for n in (2 ** 31, 2 ** 32 + 4):
        z, f = torch.zeros(n, 8, dtype=torch.float16, device=META), torch.zeros(n, device=META)
        for call in (lambda: d.logprobs(z, None, None, f), lambda: p.reserve(lens, lens, n, 4),
                     lambda: B.PagePool(n, 1, 1, device=META), lambda: B.PagePool(1, n, 1, device=META),
                     lambda: B.PagePool(1, 1, n, device=META)):
            with pytest.raises(B.DFlashError) as e:
                call()
            assert e.value.status == B.DFLASH_E_CAPACITY
