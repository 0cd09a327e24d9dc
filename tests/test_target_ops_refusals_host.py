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
