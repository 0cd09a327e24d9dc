"""Refusals of an attend's own workspace, without a GPU."""
import pytest
import torch

from block_diffusion_drafter_kv_gb300 import binding as B
from block_diffusion_drafter_kv_gb300.build import build


@pytest.fixture(scope="module")
def cache():
    build()
    meta = torch.device("meta")
    c = object.__new__(B.PagedCache)
    c.L, c.c = B.lib(), None
    c.cfg = B.DflashCacheConfig(2, 8, 2, 128, B.E4M3_F16, 32, 8, 4, 16, 128, 0, 512, 0.0)
    c.device, c.dtype, c._q_row, c._kv_row, c._shared = meta, torch.float16, 1024, 256, None
    return c


def test_sizes(cache):
    w = cache.shared_workspace(40)
    assert w.dtype == torch.uint8 and w.device == cache.device
    assert w.numel() == 256 + cache.L.dflash_cache_shared_workspace_size(B.ctypes.byref(cache.cfg), 40)
    for rows, status in ((0, B.DFLASH_E_INVAL), (-3, B.DFLASH_E_INVAL), (1 << 31, B.DFLASH_E_CAPACITY)):
        with pytest.raises(B.DFlashError) as e:
            cache.shared_workspace(rows)
        assert e.value.status == status


def test_what_attend_refuses(cache):
    h, n = torch.zeros(4, 1024, dtype=torch.float16, device="meta"), torch.zeros(4, dtype=torch.int32, device="meta")
    good = cache.shared_workspace(4)
    for kw in (dict(workspace=good),                                       # without a prefix
               dict(prefix=3),                                             # neither the cache's nor one of its own
               dict(prefix=3, workspace=good.view(torch.int8)),
               dict(prefix=3, workspace=good[::2]),
               dict(prefix=3, workspace=torch.zeros(1 << 16, dtype=torch.uint8))):   # another device
        with pytest.raises(B.DFlashError) as e:
            cache.attend(0, h, n, 4, 1, h, **kw)
        assert e.value.status == B.DFLASH_E_INVAL, kw
