"""Refusals of the 8-bit cache, of attention with a shared prefix and of reading back, without a GPU."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from block_diffusion_drafter_kv_gb300 import binding as B
from block_diffusion_drafter_kv_gb300.build import build

P4, P16 = 1 << 21, 1 << 20   # never dereferenced: every call below fails its checks first


@pytest.fixture(scope="module")
def L():
    build()
    return B.lib()


def cfg(**kw):
    c = B.DflashCacheConfig(2, 8, 2, 128, B.E4M3_F16, 32, 8, 4, 16, 128, 0, 512, 0.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def test_config_check(L):
    for kw in (dict(), dict(dtype=B.E4M3_BF16), dict(head_dim=64, rope_dim=64), dict(n_heads=16)):
        assert L.dflash_cache_config_check(cfg(**kw)) == 0
        assert 0 < L.dflash_cache_workspace_size(cfg(**kw)) < 1 << 28
    for kw in (dict(dtype=5), dict(dtype=-1), dict(head_dim=96), dict(n_heads=34)):
        assert L.dflash_cache_config_check(cfg(**kw)) == -2


def test_shared_workspace_size(L):
    f = L.dflash_cache_shared_workspace_size
    assert f(cfg(), 0) == f(cfg(), -1) == f(None, 1) == f(cfg(dtype=5), 1) == 0
    assert f(cfg(), 10) >= 2 * 10 * 8 * 130 * 4 and f(cfg(), 2 ** 31 - 1) > 2 ** 31


def test_calls_need_a_handle(L):
    assert L.dflash_cache_bind_8bit(None, P16, P16, P16, P4, P4, P16, P16, P16, 1 << 30) == -1
    assert L.dflash_cache_append_shared(None, 0, P16, P16, P16, B.F16, 8, 8, 8, P4, 1, 1, 2, P16, None) == -1
    assert L.dflash_cache_attend_shared(None, 0, P16, P4, 1, 1, 2, P16, P16, 1 << 30, None) == -1
    assert L.dflash_cache_read(None, 0, P4, P4, 1, 1, B.F16, P16, P16, None) == -1
    assert L.dflash_pages_move(None, 0, 1, None, None) == -1


def test_wrappers_refuse_what_the_library_would_misread():
    meta = torch.device("meta")
    i32 = torch.zeros(4, dtype=torch.int32, device=meta)
    c = object.__new__(B.PagedCache)
    c.device, c.dtype, c._q_row, c._kv_row, c._shared = meta, torch.float16, 256, 128, None
    h, kv = torch.zeros(4, 256, dtype=torch.float16, device=meta), torch.zeros(4, 128, dtype=torch.float16, device=meta)
    calls = [
        lambda: c.attend(0, h, i32, 4, 1, h, prefix=4),                  # no workspace was asked for
        lambda: c.attend(0, h.bfloat16(), i32, 4, 1, h, prefix=4),
        lambda: c.read(0, i32.long(), i32, 4, 1, kv, kv),
        lambda: c.read(0, i32, i32[:3], 4, 1, kv, kv),
        lambda: c.read(0, i32, i32, 4, 1, kv, kv[:3]),
        lambda: c.read(0, i32, i32, 4, 1, kv, kv.bfloat16()),            # two types
        lambda: c.read(0, i32, i32, 4, 1, torch.zeros(4, 256, dtype=torch.float16, device=meta)[:, ::2], kv),
        lambda: c.read(0, i32, i32, 4, 1, torch.zeros(4, 128, dtype=torch.float16), kv),   # another device
    ]
    for n, call in enumerate(calls):
        with pytest.raises(B.DFlashError) as e:
            call()
        assert e.value.status == B.DFLASH_E_INVAL, n
    pool = SimpleNamespace(device=meta, max_batch=4, n_pages=2, pages_per_seq=2)
    for kw in (dict(bits=4), dict(bits=16, scales=i32), dict(bits=8, dtype=torch.float32),
               dict(bits=8, k_pool=torch.zeros(128, 2, 128, dtype=torch.float16, device=meta)),
               dict(bits=8, scales=torch.zeros(2, 2, 2, 64, dtype=torch.int8, device=meta)),
               dict(bits=8, scales=torch.zeros(2, 2, 2, 63, dtype=torch.uint8, device=meta))):
        with pytest.raises(B.DFlashError):
            B.PagedCache(1, 4, 2, 128, pool, i32, **kw)
    with pytest.raises(B.DFlashError) as e:
        B.PagedCache(1, 4, 2, 128, pool, i32, shared_rows=1 << 31)
    assert e.value.status == B.DFLASH_E_CAPACITY
