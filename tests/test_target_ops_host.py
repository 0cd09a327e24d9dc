"""The target-side operators without a GPU: every refusal that comes before a launch, struct
layouts, and the rotary tables against their formulas."""
import ctypes
import math

import pytest
import torch

from block_diffusion_drafter_kv_gb300 import binding as B
from block_diffusion_drafter_kv_gb300.build import build

P4, P16 = 1 << 21, 1 << 20   # never dereferenced: every call below fails its checks first


@pytest.fixture(scope="module")
def L():
    build()
    return B.lib()


def pool(**kw):
    p = B.DflashPagePool(16, 4, 8, 0, P4, P4, P4, P4)
    for k, v in kw.items():
        setattr(p, k, v)
    return ctypes.byref(p)


def test_struct_layouts():
    assert ctypes.sizeof(B.DflashPagePool) == 4 * 4 + 4 * 8
    assert ctypes.sizeof(B.DflashCacheConfig) == 13 * 4


@pytest.mark.parametrize("bad", [dict(n_pages=0), dict(n_pages=1 << 25), dict(pages_per_seq=0), dict(pages_per_seq=1 << 25),
                                 dict(max_batch=0), dict(max_batch=8193), dict(page_table=None), dict(held=None),
                                 dict(free_list=None), dict(state=None), dict(state=P4 + 2), dict(held=P4 + 1)])
def test_page_pool_refuses_a_bad_pool(L, bad):
    assert L.dflash_pages_init(pool(**bad), None) == -1
    assert L.dflash_pages_reserve(pool(**bad), P4, P4, 1, 1, P4, None) == -1
    assert L.dflash_pages_release(pool(**bad), P4, 1, None) == -1


def test_page_pool_refuses_bad_arguments(L):
    f = L.dflash_pages_reserve
    assert L.dflash_pages_init(None, None) == -1
    assert f(None, P4, P4, 1, 1, P4, None) == -1
    assert f(pool(), None, P4, 1, 1, P4, None) == -1
    assert f(pool(), P4, None, 1, 1, P4, None) == -1
    assert f(pool(), P4 + 2, P4, 1, 1, P4, None) == -1
    assert f(pool(), P4, P4, 1, 1, P4 + 1, None) == -1
    assert f(pool(), P4, P4, 0, 1, P4, None) == -1
    assert f(pool(), P4, P4, 1, 0, P4, None) == -1
    assert f(pool(), P4, P4, 9, 1, P4, None) == -3
    assert f(pool(), P4, P4, 8, 1 << 28, P4, None) == -3
    assert L.dflash_pages_release(pool(), None, 1, None) == -1
    assert L.dflash_pages_release(pool(), P4, 0, None) == -1
    assert L.dflash_pages_release(pool(), P4, 9, None) == -3


def cfg(**kw):
    c = B.DflashCacheConfig(2, 8, 2, 128, B.F16, 32, 8, 4, 16, 128, 0, 512, 0.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


@pytest.mark.parametrize("bad", [dict(n_layers=0), dict(n_kv_heads=0), dict(n_heads=9), dict(n_heads=0), dict(n_heads=34),
                                 dict(head_dim=96), dict(dtype=B.F32), dict(dtype=-1), dict(n_pages=0), dict(n_pages=1 << 25),
                                 dict(pages_per_seq=0), dict(max_batch=0), dict(max_batch=8193), dict(max_block=0),
                                 dict(max_block=17), dict(rope_dim=24), dict(rope_dim=144), dict(rope_dim=-16),
                                 dict(rope_interleaved=2), dict(rope_positions=0), dict(scale=-1.0), dict(scale=float("nan")),
                                 dict(scale=float("inf"))])
def test_cache_config_check_rejects(L, bad):
    assert L.dflash_cache_config_check(cfg(**bad)) == -2
    assert L.dflash_cache_workspace_size(cfg(**bad)) == 0
    h = ctypes.c_void_p()
    assert L.dflash_cache_create(cfg(**bad), ctypes.byref(h)) == -2


def test_cache_config_check_rejects_a_scale_that_overflows(L):
    assert L.dflash_cache_config_check(cfg(scale=2e38)) == -2 and L.dflash_cache_config_check(cfg(scale=1e38)) == 0


def test_cache_config_check_accepts(L):
    for kw in (dict(), dict(head_dim=64, rope_dim=64, dtype=B.BF16), dict(n_heads=16, max_block=16), dict(n_heads=256, max_block=1),
               dict(rope_dim=0, rope_positions=0), dict(rope_dim=32, rope_interleaved=1), dict(scale=0.25), dict(max_batch=8192)):
        assert L.dflash_cache_config_check(cfg(**kw)) == 0, kw
        assert 0 < L.dflash_cache_workspace_size(cfg(**kw)) < 1 << 28


def test_cache_calls_need_a_handle(L):
    f = ctypes.c_int32(0)
    assert L.dflash_cache_config_check(None) == -1
    assert L.dflash_cache_workspace_size(None) == 0
    assert L.dflash_cache_create(None, None) == -1
    assert L.dflash_cache_create(cfg(), None) == -1
    assert L.dflash_cache_destroy(None) == -1
    assert L.dflash_cache_bind(None, P16, P16, P4, P4, P16, P16, P16, 1 << 30) == -1
    assert L.dflash_cache_append(None, 0, P16, P16, P16, B.F16, 8, 8, 8, P4, 1, 1, P16, None) == -1
    assert L.dflash_cache_attend(None, 0, P16, P4, 1, 1, P16, None) == -1
    assert L.dflash_cache_read_error(None, ctypes.byref(f), 0, None) == -1
    assert L.dflash_logprobs(None, P16, B.F32, 8, P4, 1, 1.0, 0, P4, P4, None, None, None) == -1


def test_wrappers_refuse_tensors_the_library_would_misread():
    """The binding checks type, device, size and layout before any library call: objects that were
    never bound are enough to see each refusal."""
    from types import SimpleNamespace
    meta = torch.device("meta")
    i32 = torch.zeros(4, dtype=torch.int32, device=meta)
    d = object.__new__(B.Drafter)
    d.cfg, d.last_token = SimpleNamespace(vocab=8), i32
    z, f = torch.zeros(4, 8, device=meta), torch.zeros(4, device=meta)
    ids, top = torch.zeros(4, 3, dtype=torch.int32, device=meta), torch.zeros(4, 3, device=meta)
    p = object.__new__(B.PagePool)
    p.device = meta
    c = object.__new__(B.PagedCache)
    c.device, c.dtype, c._q_row, c._kv_row = meta, torch.float16, 256, 128
    h = torch.zeros(4, 256, dtype=torch.float16, device=meta)
    calls = [
        lambda: d.logprobs(z.double(), i32, f, f),                       # fp64 logits
        lambda: d.logprobs(z[:, :7], i32, f, f),                         # another vocabulary
        lambda: d.logprobs(torch.zeros(8, 4, device=meta).t(), i32, f, f),   # logits column by column
        lambda: d.logprobs(torch.zeros(4, 8), i32, f, f),                # another device
        lambda: d.logprobs(z, i32.long(), f, f),
        lambda: d.logprobs(z, i32[:3], f, f),
        lambda: d.logprobs(z, i32, f[:3], f),
        lambda: d.logprobs(z, i32, f, None),
        lambda: d.logprobs(z, i32, f, f, ids),                           # ids without values
        lambda: d.logprobs(z, i32, f, f, ids, top[:, :2].contiguous()),
        lambda: d.logprobs(z, i32, f, f, ids.t(), top),
        lambda: p.reserve(i32.long(), i32, 1, 4),
        lambda: p.reserve(i32, i32, 1, 5),
        lambda: p.reserve(i32, i32, 2, 4, i32),                          # slots too short
        lambda: p.release(torch.zeros(8, dtype=torch.int32, device=meta)[::2], 4),
        lambda: c.attend(0, h.float(), i32, 4, 1, h),
        lambda: c.attend(0, h, i32, 4, 1, h[:, ::2]),
        lambda: c.attend(0, h, i32, 2, 1, h),
        lambda: c.attend(0, h, i32.long(), 4, 1, h),
        lambda: c.append(0, h, h[:, :128], h[:, 128:].bfloat16(), i32, 4, 1, h),   # types differ
        lambda: c.append(0, h, h[:, ::2], h[:, :128], i32, 4, 1, h),               # rows not dense
        lambda: c.append(0, h, h[:3, :128], h[:3, :128], i32, 4, 1, h),
        lambda: c.append(0, h, h[:, :128], h[:, :128], i32[:3], 4, 1, h),
        lambda: c.append(0, h, h[:, :128], h[:, :128], i32, 4, 1, h.bfloat16()),
    ]
    for n, call in enumerate(calls):
        with pytest.raises(B.DFlashError) as ei:
            call()
        assert ei.value.status == B.DFLASH_E_INVAL, n


def test_rope_tables():
    cos, sin = B.rope_tables(70000, 64, 1e6, device="cpu")
    assert cos.shape == sin.shape == (70000, 32) and cos.dtype == torch.float32
    for p, j in ((0, 0), (1, 0), (69999, 3), (12345, 31)):
        a = p * 1e6 ** (-2 * j / 64)
        assert abs(cos[p, j].item() - math.cos(a)) <= 2 ** -24 and abs(sin[p, j].item() - math.sin(a)) <= 2 ** -24
    c2, s2 = B.rope_tables(64, 16, 1e4, linear=4.0, attention_factor=1.25, device="cpu")
    assert abs(c2[63, 0].item() - 1.25 * math.cos(63 / 4)) <= 2 ** -23
    # banded: the fast pairs as they are, the slow ones divided, in between a mixture
    factor, low, high, trained = 8.0, 1.0, 4.0, 8192
    c3, _ = B.rope_tables(2, 128, 5e5, bands=(factor, low, high, trained), device="cpu")
    for j in range(64):
        inv = 5e5 ** (-2 * j / 128)
        turns = trained * inv / (2 * math.pi)
        k = min(1.0, max(0.0, (turns - low) / (high - low)))
        assert abs(c3[1, j].item() - math.cos(inv * k + inv / factor * (1 - k))) <= 2 ** -23
