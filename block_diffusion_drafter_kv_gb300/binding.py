"""ctypes binding of libdflash.so (include/dflash.h): argument marshalling only.

Every step of the draft-and-verify path runs in the library's CUDA kernels. PyTorch
supplies device memory and the current stream. If the shared library is missing the
import of `lib()` raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_float, c_int32, c_size_t, c_void_p
from typing import Optional

from .build import LIB_PATH

DFLASH_OK = 0
DFLASH_E_INVAL = -1
DFLASH_E_CAPACITY = -3
STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported drafter shape", -3: "capacity exceeded",
          -4: "CUDA error", -5: "state not bound"}
DEV_TIMEOUT, DEV_CAPACITY, DEV_TOKEN = 1, 2, 4
OPT_WAIT_LIMIT_NS, OPT_CHAIN_MAX, OPT_GEMV_VARIANT, OPT_ATTN_SPLIT, OPT_ATTN_KEY_GROUPS = 1, 2, 3, 4, 5
OPT_INJECT_PASS_ROWS = 6
OPT_ATTN_MODE = 7
F32, F16, BF16, E4M3_F16, E4M3_BF16 = 0, 1, 2, 3, 4
PAGE_POSITIONS = 64


class DflashConfig(ctypes.Structure):
    _fields_ = [("hidden", c_int32), ("n_heads", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32),
                ("n_layers", c_int32), ("intermediate", c_int32), ("vocab", c_int32), ("n_taps", c_int32),
                ("target_hidden", c_int32), ("rope_theta", c_float), ("rms_eps", c_float),
                ("max_block", c_int32), ("max_batch", c_int32), ("kv_capacity", c_int32)]


class DflashLayerWeights(ctypes.Structure):
    _fields_ = [(n, c_void_p) for n in ("wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down", "g_attn", "g_mlp")]


class DflashWeights(ctypes.Structure):
    _fields_ = [("w_fc", c_void_p), ("g_ctx", c_void_p), ("embed", c_void_p), ("mask_emb", c_void_p),
                ("g_final", c_void_p), ("lm_head", c_void_p), ("layers", POINTER(DflashLayerWeights))]


class DflashPagePool(ctypes.Structure):
    _fields_ = [("n_pages", c_int32), ("pages_per_seq", c_int32), ("max_batch", c_int32), ("reserved", c_int32),
                ("page_table", c_void_p), ("held", c_void_p), ("free_list", c_void_p), ("state", c_void_p)]


class DflashCacheConfig(ctypes.Structure):
    _fields_ = [("n_layers", c_int32), ("n_heads", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32),
                ("dtype", c_int32), ("n_pages", c_int32), ("pages_per_seq", c_int32), ("max_batch", c_int32),
                ("max_block", c_int32), ("rope_dim", c_int32), ("rope_interleaved", c_int32),
                ("rope_positions", c_int32), ("scale", c_float)]


# name -> (restype, argtypes); mirrors include/dflash.h
SIGNATURES = {
    "dflash_config_check": (c_int32, [POINTER(DflashConfig)]),
    "dflash_workspace_size": (c_size_t, [POINTER(DflashConfig)]),
    "dflash_create": (c_int32, [POINTER(DflashConfig), POINTER(DflashWeights), POINTER(c_void_p)]),
    "dflash_destroy": (c_int32, [c_void_p]),
    "dflash_bind_state": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_size_t]),
    "dflash_bind_state_paged": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_void_p,
                                          c_void_p, c_void_p, c_size_t]),
    "dflash_inject_ctx": (c_int32, [c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_void_p]),
    "dflash_draft_block": (c_int32, [c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p]),
    "dflash_verify_greedy": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_void_p,
                                       c_void_p]),
    "dflash_verify_sampling": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_float, c_int32, c_int32, c_void_p,
                                         c_void_p, c_void_p]),
    "dflash_verify_greedy_hidden": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                              c_void_p, c_void_p, c_void_p]),
    "dflash_logprobs": (c_int32, [c_void_p, c_void_p, c_int32, ctypes.c_int64, c_void_p, c_int32, c_float, c_int32,
                                  c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "dflash_pages_init": (c_int32, [POINTER(DflashPagePool), c_void_p]),
    "dflash_pages_reserve": (c_int32, [POINTER(DflashPagePool), c_void_p, c_void_p, c_int32, c_int32, c_void_p,
                                       c_void_p]),
    "dflash_pages_release": (c_int32, [POINTER(DflashPagePool), c_void_p, c_int32, c_void_p]),
    "dflash_pages_move": (c_int32, [POINTER(DflashPagePool), c_int32, c_int32, c_void_p, c_void_p]),
    "dflash_cache_config_check": (c_int32, [POINTER(DflashCacheConfig)]),
    "dflash_cache_workspace_size": (c_size_t, [POINTER(DflashCacheConfig)]),
    "dflash_cache_create": (c_int32, [POINTER(DflashCacheConfig), POINTER(c_void_p)]),
    "dflash_cache_destroy": (c_int32, [c_void_p]),
    "dflash_cache_bind": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                    c_size_t]),
    "dflash_cache_bind_8bit": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_size_t]),
    "dflash_cache_append": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_int32, ctypes.c_int64,
                                      ctypes.c_int64, ctypes.c_int64, c_void_p, c_int32, c_int32, c_void_p, c_void_p]),
    "dflash_cache_attend": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_void_p]),
    "dflash_cache_append_shared": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_int32, ctypes.c_int64,
                                             ctypes.c_int64, ctypes.c_int64, c_void_p, c_int32, c_int32, c_int32, c_void_p,
                                             c_void_p]),
    "dflash_cache_shared_workspace_size": (c_size_t, [POINTER(DflashCacheConfig), c_int32]),
    "dflash_cache_attend_shared": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p,
                                             c_void_p, c_size_t, c_void_p]),
    "dflash_cache_read": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p,
                                    c_void_p]),
    "dflash_cache_read_error": (c_int32, [c_void_p, POINTER(c_int32), c_int32, c_void_p]),
    "dflash_linear_bf16": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_int32, c_void_p,
                                     c_void_p]),
    "dflash_read_device_error": (c_int32, [c_void_p, POINTER(c_int32), c_int32, c_void_p]),
    "dflash_set_option": (c_int32, [c_void_p, c_int32, ctypes.c_int64]),
    "dflash_get_option": (c_int32, [c_void_p, c_int32, POINTER(ctypes.c_int64)]),
    "dflash_selftest_timeout": (c_int32, [c_void_p, c_void_p]),
    "dflash_last_launch_count": (c_int32, [c_void_p]),
    "dflash_trace_events": (c_int32, [c_void_p, POINTER(c_void_p), c_int32]),
    "dflash_timeline": (c_int32, [c_void_p, c_void_p, ctypes.c_int64]),
    "dflash_timeline_used": (ctypes.c_int64, [c_void_p]),
    "dflash_status_string": (ctypes.c_char_p, [c_int32]),
    "dflash_verify_greedy_noalloc": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p,
                                               c_void_p, c_void_p]),
    "dflash_synth_plant": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_int32, c_int32, c_int32,
                                     c_float, c_void_p, c_void_p]),
    "dflash_synth_unplant": (c_int32, [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p]),
}

_LIB = None


def lib(path: Optional[str] = None):
    """Load libdflash.so (built by `build.build()`); raises if it is absent."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libdflash.so not found at {p}: run block_diffusion_drafter_kv_gb300.build.build()")
    L = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    if path is None:
        _LIB = L
    return L


class DFlashError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status})")
        self.status = status


def check(status: int, what: str) -> None:
    if status != DFLASH_OK:
        raise DFlashError(status, what)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def make_config(shape, max_block: int, max_batch: int, kv_capacity: int) -> DflashConfig:
    return DflashConfig(shape.hidden, shape.n_heads, shape.n_kv_heads, shape.head_dim, shape.n_layers,
                        shape.intermediate, shape.vocab, shape.n_taps, shape.target_hidden,
                        float(shape.rope_theta), float(shape.rms_eps), max_block, max_batch, kv_capacity)


class Drafter:
    """One registered drafter plus its caller-owned state (KV caches, lengths, workspace).

    `weights` has the attributes of the input generator's `Weights` (bf16 CUDA tensors)."""

    def __init__(self, shape, weights, max_block: int, max_batch: int, kv_capacity: int, n_pages: int = 0,
                 page_table=None, pages: "Optional[PagePool]" = None):
        """n_pages > 0 binds a paged KV cache: a pool of n_pages pages of 64 positions
        (k_cache / v_cache [L][n_pages * 64][nkv][d]) and `page_table`, an int32 CUDA tensor
        [max_batch][pages_per_seq] of page ids that the caller fills (and may change between
        calls). `pages` binds one whose table a PagePool keeps instead: reserve room for
        [len, len + B) before a draft and for the new positions before an injection."""
        import torch
        if pages is not None:
            if n_pages or page_table is not None or pages.max_batch < max_batch:
                raise DFlashError(DFLASH_E_INVAL, "pages: a pool of at least max_batch sequences, without n_pages or page_table")
            if pages.device != weights.w_fc.device:
                raise DFlashError(DFLASH_E_INVAL, f"pages on {pages.device}, the weights on {weights.w_fc.device}")
            n_pages, page_table = pages.n_pages, pages.page_table
        self.pages = pages
        self.L = lib()
        self.shape = shape
        self.cfg = make_config(shape, max_block, max_batch, kv_capacity)
        self.weights = weights  # keep the tensors alive
        lw = (DflashLayerWeights * shape.n_layers)()
        for i, w in enumerate(weights.layers):
            lw[i] = DflashLayerWeights(*[getattr(w, n).data_ptr() for n in
                                         ("wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down", "g_attn", "g_mlp")])
        self._lw = lw
        W = DflashWeights(weights.w_fc.data_ptr(), weights.g_ctx.data_ptr(), weights.embed.data_ptr(),
                          weights.mask_emb.data_ptr(), weights.g_final.data_ptr(), weights.lm_head.data_ptr(),
                          ctypes.cast(lw, POINTER(DflashLayerWeights)))
        h = c_void_p()
        check(self.L.dflash_create(ctypes.byref(self.cfg), ctypes.byref(W), ctypes.byref(h)), "dflash_create")
        self.h = h
        dev = weights.w_fc.device
        s = shape
        rows = (n_pages * 64,) if n_pages else (max_batch, kv_capacity)
        self.k_cache = torch.zeros(s.n_layers, *rows, s.n_kv_heads, s.head_dim, dtype=torch.float16, device=dev)
        self.v_cache = torch.zeros(s.n_layers, *rows, s.n_kv_heads, s.head_dim, dtype=torch.float16, device=dev)
        self.page_table = page_table
        self.len = torch.zeros(max_batch, dtype=torch.int32, device=dev)
        self.last_token = torch.zeros(max_batch, dtype=torch.int32, device=dev)
        nbytes = self.L.dflash_workspace_size(ctypes.byref(self.cfg))
        if nbytes == 0:
            raise DFlashError(-2, "dflash_workspace_size")
        self.workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device=dev)
        base = self.workspace.data_ptr()
        self._ws_ptr = (base + 255) // 256 * 256
        if n_pages:
            assert page_table is not None and page_table.dtype == torch.int32 and page_table.is_cuda
            check(self.L.dflash_bind_state_paged(self.h, self.k_cache.data_ptr(), self.v_cache.data_ptr(), n_pages,
                                                 page_table.data_ptr(), page_table.shape[1], self.len.data_ptr(),
                                                 self.last_token.data_ptr(), self._ws_ptr, nbytes),
                  "dflash_bind_state_paged")
        else:
            check(self.L.dflash_bind_state(self.h, self.k_cache.data_ptr(), self.v_cache.data_ptr(),
                                           self.len.data_ptr(), self.last_token.data_ptr(), self._ws_ptr, nbytes),
                  "dflash_bind_state")

    # -- the three calls of the step ---------------------------------------------------
    def inject(self, hidden, rows_per_seq: int, n_new, batch: int, stream=None):
        import torch
        _require(hidden, torch.bfloat16, "hidden")
        _require(n_new, torch.int32, "n_new")
        check(self.L.dflash_inject_ctx(self.h, hidden.data_ptr(), rows_per_seq, n_new.data_ptr(), batch,
                                       _stream(stream)), "dflash_inject_ctx")

    def draft(self, batch: int, block: int, drafted, logits=None, x_trace=None, stream=None):
        import torch
        _require_opt(drafted, torch.int32, "drafted")
        _require_opt(logits, torch.float32, "logits")
        _require_opt(x_trace, torch.float32, "x_trace")
        check(self.L.dflash_draft_block(self.h, batch, block, _ptr(drafted), _ptr(logits), _ptr(x_trace),
                                        _stream(stream)), "dflash_draft_block")

    def verify(self, target_logits, drafted, batch: int, block: int, accept_len, committed, stream=None):
        import torch
        _require(target_logits, torch.float32, "target_logits")
        _require_opt(drafted, torch.int32, "drafted")
        _require(accept_len, torch.int32, "accept_len")
        _require(committed, torch.int32, "committed")
        check(self.L.dflash_verify_greedy(self.h, target_logits.data_ptr(), _ptr(drafted), batch, block,
                                          accept_len.data_ptr(), committed.data_ptr(), _stream(stream)),
              "dflash_verify_greedy")

    def verify_sampling(self, target_logits, drafted, uniforms, temperature: float, batch: int, block: int,
                        accept_len, committed, stream=None):
        """Speculative-sampling verification at `temperature` with caller-drawn uniforms
        (fp32 [batch][B]: accept tests, then the sampling draw)."""
        import torch
        _require(target_logits, torch.float32, "target_logits")
        _require_opt(drafted, torch.int32, "drafted")
        _require(uniforms, torch.float32, "uniforms")
        _require(accept_len, torch.int32, "accept_len")
        _require(committed, torch.int32, "committed")
        check(self.L.dflash_verify_sampling(self.h, target_logits.data_ptr(), _ptr(drafted), uniforms.data_ptr(),
                                            float(temperature), batch, block, accept_len.data_ptr(),
                                            committed.data_ptr(), _stream(stream)), "dflash_verify_sampling")

    def verify_hidden(self, target_hidden, target_gain, target_lm_head, drafted, batch: int, block: int, accept_len,
                      committed, stream=None):
        """Greedy verification from the target's last hidden states (bf16 [batch*B][Ht]), its
        final-norm gain (bf16 [Ht]) and LM head (bf16 [V][Ht])."""
        import torch
        for t, n in ((target_hidden, "target_hidden"), (target_gain, "target_gain"), (target_lm_head, "target_lm_head")):
            _require(t, torch.bfloat16, n)
        _require_opt(drafted, torch.int32, "drafted")
        _require(accept_len, torch.int32, "accept_len")
        _require(committed, torch.int32, "committed")
        check(self.L.dflash_verify_greedy_hidden(self.h, target_hidden.data_ptr(), target_gain.data_ptr(),
                                                 target_lm_head.data_ptr(), _ptr(drafted), batch, block,
                                                 accept_len.data_ptr(), committed.data_ptr(), _stream(stream)),
              "dflash_verify_greedy_hidden")

    def logprobs(self, logits, tokens, logprob, entropy, top_ids=None, top_logprobs=None, temperature: float = 1.0,
                 stream=None):
        """Log probabilities of `tokens` (int32 [rows]; -1: a row without one, left out; None
        with logprob None) under softmax(logits / temperature), the rows' entropies and, with
        top_ids (int32 [rows][n]) and top_logprobs (fp32 [rows][n]), the n most likely tokens.
        logits: fp32, fp16 or bf16 [rows][vocab], rows a stride apart."""
        import torch
        rows, vocab = logits.shape if logits.dim() == 2 else (0, 0)
        dtype = _DTYPES.get(str(logits.dtype), -1)
        if dtype < 0 or vocab != self.cfg.vocab or logits.stride(1) != 1 or logits.device != self.last_token.device:
            raise DFlashError(DFLASH_E_INVAL, "logits must be fp32, fp16 or bf16 [rows][vocab] on the drafter's device")
        _require_31_bits(rows, "rows")
        n = 0 if top_ids is None else top_ids.numel() // max(rows, 1)
        for t, dt, size, name in ((tokens, torch.int32, rows, "tokens"), (logprob, torch.float32, rows, "logprob"),
                                  (entropy, torch.float32, rows, "entropy"), (top_ids, torch.int32, rows * n, "top_ids"),
                                  (top_logprobs, torch.float32, rows * n, "top_logprobs")):
            _require_on(t, dt, size, name, logits.device)
        if entropy is None or (n > 0) != (top_logprobs is not None and top_logprobs.numel() > 0):
            raise DFlashError(DFLASH_E_INVAL, "entropy, and top_ids with top_logprobs, are needed")
        check(self.L.dflash_logprobs(self.h, logits.data_ptr(), dtype, logits.stride(0) if rows > 1 else vocab,
                                     _ptr(tokens), rows, float(temperature), n, _ptr(logprob), entropy.data_ptr(),
                                     _ptr(top_ids) if n else None, _ptr(top_logprobs) if n else None,
                                     _stream_on(stream, logits.device)), "dflash_logprobs")

    # -- helpers -------------------------------------------------------------------------
    def linear(self, W, X, Y, stream=None):
        import torch
        _require(W, torch.bfloat16, "W")
        _require(X, torch.bfloat16, "X")
        _require(Y, torch.float32, "Y")
        check(self.L.dflash_linear_bf16(self.h, W.data_ptr(), W.shape[0], W.shape[1], X.data_ptr(), X.shape[0],
                                        Y.data_ptr(), _stream(stream)), "dflash_linear_bf16")

    def device_error(self, clear: bool = True, stream=None) -> int:
        """The device error flag once the work queued on `stream` (default: the current
        stream) has finished; with `clear`, the flag and the kernels' counters are reset."""
        f = c_int32(0)
        check(self.L.dflash_read_device_error(self.h, ctypes.byref(f), 1 if clear else 0, _stream(stream)),
              "dflash_read_device_error")
        return f.value

    def set_option(self, option: int, value: int) -> None:
        check(self.L.dflash_set_option(self.h, option, int(value)), "dflash_set_option")

    def get_option(self, option: int) -> int:
        v = ctypes.c_int64(0)
        check(self.L.dflash_get_option(self.h, option, ctypes.byref(v)), "dflash_get_option")
        return v.value

    def selftest_timeout(self, stream=None) -> None:
        check(self.L.dflash_selftest_timeout(self.h, _stream(stream)), "dflash_selftest_timeout")

    def last_launch_count(self) -> int:
        return self.L.dflash_last_launch_count(self.h)

    def timeline(self, records=None) -> None:
        """Per-CTA timeline into `records` (int64 CUDA tensor [n, 21]); None turns it off."""
        n = 0 if records is None else records.shape[0]
        self._tl_keep = records
        check(self.L.dflash_timeline(self.h, None if records is None else records.data_ptr(), n), "dflash_timeline")

    def timeline_used(self) -> int:
        return self.L.dflash_timeline_used(self.h)

    def trace_events(self, events) -> None:
        """Record torch.cuda.Event objects around each launch of later calls ([] turns it off)."""
        arr = (c_void_p * max(1, len(events)))(*[e.cuda_event for e in events])
        self._trace_keep = (arr, list(events))
        check(self.L.dflash_trace_events(self.h, arr, len(events)), "dflash_trace_events")

    def close(self):
        if getattr(self, "h", None):
            self.L.dflash_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _require(t, dtype, name):
    import torch
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise DFlashError(DFLASH_E_INVAL, f"{name} must be a contiguous {dtype} CUDA tensor "
                                          f"(got {t.dtype}, cuda={t.is_cuda}, contiguous={t.is_contiguous()})")


def _require_opt(t, dtype, name):
    if t is not None:
        _require(t, dtype, name)


def _require_on(t, dtype, numel, name, device):
    if t is not None and (t.dtype != dtype or t.device != device or not t.is_contiguous() or t.numel() != numel):
        raise DFlashError(DFLASH_E_INVAL, f"{name} must be a contiguous {dtype} tensor of {numel} values on {device} "
                                          f"(got {t.dtype}, {t.numel()} values on {t.device}, contiguous={t.is_contiguous()})")


def _stream_on(stream, device) -> int:
    return _torch_calls()[0](device.index) if stream is None else stream.cuda_stream


_calls = None


def _torch_calls():
    """(raw handle of a device's current stream, index of the current device, int32, uint8), looked up once:
    the small calls below take a few microseconds in all."""
    global _calls
    if _calls is None:
        import torch
        _calls = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice, torch.int32, torch.uint8
    return _calls


_DTYPES = {"torch.float32": F32, "torch.float16": F16, "torch.bfloat16": BF16}


class PagePool:
    """Cache pages handed out on the GPU from sequence lengths: the page table of a paged
    cache, the pages each sequence holds and the free list, all int32 CUDA tensors."""

    def __init__(self, n_pages: int, pages_per_seq: int, max_batch: int, device="cuda"):
        import torch
        self.L = lib()
        self.n_pages, self.pages_per_seq, self.max_batch = n_pages, pages_per_seq, max_batch
        if min(n_pages, pages_per_seq, max_batch) < 1:
            raise DFlashError(DFLASH_E_INVAL, "PagePool")
        _require_31_bits(max(n_pages, pages_per_seq, max_batch), "the pool's sizes")
        with torch.cuda.device(device):
            self.page_table = torch.empty(max_batch, pages_per_seq, dtype=torch.int32, device="cuda")
            self.held = torch.empty(max_batch, dtype=torch.int32, device="cuda")
            self.free_list = torch.empty(n_pages, dtype=torch.int32, device="cuda")
            self.state = torch.empty(4, dtype=torch.int32, device="cuda")
            self.device = self.state.device
            self._pool = DflashPagePool(n_pages, pages_per_seq, max_batch, 0, self.page_table.data_ptr(),
                                        self.held.data_ptr(), self.free_list.data_ptr(), self.state.data_ptr())
            self._ref = ctypes.byref(self._pool)
            check(self.L.dflash_pages_init(self._ref, _stream_on(None, self.device)), "dflash_pages_init")
        self.n_free = self.state[:1]

    def reserve(self, length, n_new, rows_per_seq: int, batch: int, slots=None, stream=None):
        """Pages for positions [length[s], length[s] + n_new[s]) of every sequence; `slots` (int32
        [batch * rows_per_seq]) gets their cache rows, -1 for rows past n_new[s] and for
        sequences that the pool has no pages for."""
        i32 = _torch_calls()[2]
        _require_min(length, i32, batch, "length", self.device)
        _require_min(n_new, i32, batch, "n_new", self.device)
        if slots is not None:
            _require_on(slots, i32, batch * rows_per_seq, "slots", self.device)
        _require_31_bits(rows_per_seq, "rows_per_seq")
        self._call(self.L.dflash_pages_reserve, "dflash_pages_reserve", stream, length.data_ptr(), n_new.data_ptr(), batch,
                   rows_per_seq, _ptr(slots))

    def release(self, length, batch: int, stream=None):
        """Gives back every page past the first length[s] positions of each sequence (0: all)."""
        _require_min(length, _torch_calls()[2], batch, "length", self.device)
        self._call(self.L.dflash_pages_release, "dflash_pages_release", stream, length.data_ptr(), batch)

    def move(self, src: int, dst: int, length=None, stream=None):
        """The pages of sequence src, and with `length` (int32 [max_batch]) its length, become those of sequence
        dst, which holds none: a prompt read as sequence 0 becomes a prefix that others share."""
        if length is not None:
            _require_min(length, _torch_calls()[2], max(src, dst) + 1, "length", self.device)
        self._call(self.L.dflash_pages_move, "dflash_pages_move", stream, src, dst, _ptr(length))

    def device_error(self, clear: bool = True) -> int:
        """The device error flags of the calls so far (waits for the current stream)."""
        v = int(self.state[2])
        if clear and v:
            self.state[2:3].zero_()
        return v

    def _call(self, f, what, stream, *args):
        if _torch_calls()[1]() == self.device.index:
            check(f(self._ref, *args, _stream_on(stream, self.device)), what)
        else:
            import torch
            with torch.cuda.device(self.device):
                check(f(self._ref, *args, _stream_on(stream, self.device)), what)


class PagedCache:
    """The paged K/V cache of a causal target model: rotary append and attention of new rows.

    `pages` keeps the page table; `length` (int32 CUDA [max_batch]) holds every sequence's
    positions before the new rows and stays the caller's to advance. k_pool / v_pool:
    [n_layers][n_pages * 64][n_kv_heads][head_dim] of `dtype` (fp16 or bf16), allocated here
    unless given. rope_cos / rope_sin: fp32 [positions][rope_dim / 2] (see rope_tables).

    bits=8: the pools hold e4m3 values (torch.float8_e4m3fn), each row of one position and KV head with a
    power of two in `scales` (uint8 [n_layers][n_pages][n_kv_heads][2][64]: exponent + 127 of K, of V);
    q and out stay of `dtype`.

    Sequences that share a prefix: append and attend take `prefix`, the number of the sequence whose
    positions come before those of every sequence of the call (one of the page table's that is not in the
    batch: read as sequence 0, then PagePool.move). shared_rows: the most rows (batch * rows_per_seq) of such an attend;
    its workspace is kept here.

    Calls on one cache are ordered on one stream, and so are replays of graphs that hold them: attend leaves its parts in a
    workspace of the cache's. An attend with a prefix may run beside others where it is given a workspace of its own
    (shared_workspace)."""

    def __init__(self, n_layers: int, n_heads: int, n_kv_heads: int, head_dim: int, pages: PagePool, length, dtype=None,
                 max_block: int = 0, rope_cos=None, rope_sin=None, rope_interleaved: bool = False, scale: float = 0.0,
                 k_pool=None, v_pool=None, bits: int = 16, scales=None, shared_rows: int = 0):
        import torch
        self.L = lib()
        dtype = torch.float16 if dtype is None else dtype
        if bits not in (8, 16) or (bits == 16 and scales is not None):
            raise DFlashError(DFLASH_E_INVAL, "bits: 16, or 8 with scales")
        _require_31_bits(shared_rows, "shared_rows")
        self.dtype, self.device, self.pages, self.length = dtype, pages.device, pages, length
        batch = min(length.numel(), pages.max_batch)
        _require_min(length, torch.int32, 1, "length", self.device)
        positions, rope_dim = (0, 0) if rope_cos is None else (rope_cos.shape[0], 2 * rope_cos.shape[1])
        for t, n in ((rope_cos, "rope_cos"), (rope_sin, "rope_sin")):
            if (t is None) != (rope_cos is None):
                raise DFlashError(DFLASH_E_INVAL, "rope_cos and rope_sin go together")
            _require_on(t, torch.float32, positions * rope_dim // 2, n, self.device)
        if not max_block:  # as many rows as a call can take
            max_block = max(1, min(16, 128 // max(1, n_heads // max(1, n_kv_heads))))
        code = _DTYPES.get(str(dtype), -1)
        if bits == 8:
            code = {F16: E4M3_F16, BF16: E4M3_BF16}.get(code, -1)
        self.cfg = DflashCacheConfig(n_layers, n_heads, n_kv_heads, head_dim, code, pages.n_pages, pages.pages_per_seq, batch,
                                     max_block, rope_dim, int(rope_interleaved), positions, float(scale))
        check(self.L.dflash_cache_config_check(ctypes.byref(self.cfg)), "dflash_cache_config_check")
        shape = (n_layers, pages.n_pages * PAGE_POSITIONS, n_kv_heads, head_dim)
        numel = shape[0] * shape[1] * shape[2] * shape[3]
        pool_dtype = torch.float8_e4m3fn if bits == 8 else dtype
        _require_on(k_pool, pool_dtype, numel, "k_pool", self.device)
        _require_on(v_pool, pool_dtype, numel, "v_pool", self.device)
        self.k_pool = torch.zeros(shape, dtype=pool_dtype, device=self.device) if k_pool is None else k_pool
        self.v_pool = torch.zeros(shape, dtype=pool_dtype, device=self.device) if v_pool is None else v_pool
        self.bits, self.scales = bits, scales
        if bits == 8:
            shape = (n_layers, pages.n_pages, n_kv_heads, 2, PAGE_POSITIONS)
            _require_on(scales, torch.uint8, 2 * numel // head_dim, "scales", self.device)
            if scales is None:
                self.scales = torch.zeros(shape, dtype=torch.uint8, device=self.device)
        self.rope_cos, self.rope_sin = rope_cos, rope_sin
        nbytes = self.L.dflash_cache_workspace_size(ctypes.byref(self.cfg))
        with torch.cuda.device(self.device):
            self.workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device="cuda")
            h = c_void_p()
            check(self.L.dflash_cache_create(ctypes.byref(self.cfg), ctypes.byref(h)), "dflash_cache_create")
            self.c = h
            args = (pages.page_table.data_ptr(), length.data_ptr(), _ptr(rope_cos), _ptr(rope_sin),
                    (self.workspace.data_ptr() + 255) // 256 * 256, nbytes)
            if bits == 8:
                check(self.L.dflash_cache_bind_8bit(h, self.k_pool.data_ptr(), self.v_pool.data_ptr(), self.scales.data_ptr(),
                                                    *args), "dflash_cache_bind_8bit")
            else:
                check(self.L.dflash_cache_bind(h, self.k_pool.data_ptr(), self.v_pool.data_ptr(), *args), "dflash_cache_bind")
            self._shared = None
            if shared_rows:
                self._shared = self.shared_workspace(shared_rows)
                self._shared_bytes = self._shared.numel() - 256
        self._q_row, self._kv_row = n_heads * head_dim, n_kv_heads * head_dim

    def shared_workspace(self, rows: int):
        """A workspace for attend with a prefix, of up to `rows` rows (batch * rows_per_seq), on the cache's device."""
        import torch
        _require_31_bits(rows, "rows")
        nbytes = self.L.dflash_cache_shared_workspace_size(ctypes.byref(self.cfg), rows)
        if not nbytes:
            raise DFlashError(DFLASH_E_INVAL, "rows: 1 or more")
        return torch.empty(nbytes + 256, dtype=torch.uint8, device=self.device)

    def append(self, layer: int, q, k, v, slots, batch: int, rows_per_seq: int, q_out, stream=None, prefix: Optional[int] = None):
        """Rotary positions on q and k, k and v into the cache at `slots` (from
        PagePool.reserve), the rotated q to q_out. q, k, v: fp16 or bf16 [batch * rows_per_seq]
        rows of heads x dims, rows a stride apart (slices of one fused projection are fine);
        q and q_out may be None. With `prefix`, row r of a sequence is position
        length[prefix] + length[s] + r."""
        rows, dev, dt = batch * rows_per_seq, self.device, k.dtype
        q_stride = 0 if q is None else _row_stride(q, dt, rows, self._q_row, "q", dev)
        k_stride = _row_stride(k, dt, rows, self._kv_row, "k", dev)
        v_stride = _row_stride(v, dt, rows, self._kv_row, "v", dev)
        _require_on(slots, _torch_calls()[2], rows, "slots", dev)
        _require_on(q_out, self.dtype, rows * self._q_row, "q_out", dev)
        args = (self.c, layer, _ptr(q), k.data_ptr(), v.data_ptr(), _DTYPES.get(str(dt), -1), q_stride, k_stride, v_stride,
                slots.data_ptr(), batch, rows_per_seq)
        if prefix is None:
            check(self.L.dflash_cache_append(*args, _ptr(q_out), _stream_on(stream, dev)), "dflash_cache_append")
        else:
            check(self.L.dflash_cache_append_shared(*args, prefix, _ptr(q_out), _stream_on(stream, dev)), "dflash_cache_append_shared")

    def attend(self, layer: int, q, n_new, batch: int, rows_per_seq: int, out, stream=None, prefix: Optional[int] = None,
               workspace=None):
        """Causal attention of row r of every sequence (position length[s] + r, r < n_new[s]) over
        the cache; q and out: contiguous [batch * rows_per_seq][n_heads][head_dim] of the
        cache's dtype. Rows past n_new[s] of out are left as they were. With `prefix`, every row sees
        all length[prefix] positions of that sequence first; they are read once for the sequences that fill 128 rows of
        q for a KV head (64 in 8 bits where a sequence has no more), not once a sequence. `workspace`: one from
        shared_workspace in place of the cache's own, for a call that others may overlap; it is the call's until that has run."""
        numel = batch * rows_per_seq * self._q_row
        _require_on(q, self.dtype, numel, "q", self.device)
        _require_on(out, self.dtype, numel, "out", self.device)
        _require_min(n_new, _torch_calls()[2], batch, "n_new", self.device)
        if prefix is None:
            if workspace is not None:
                raise DFlashError(DFLASH_E_INVAL, "workspace: of an attend with a prefix")
            check(self.L.dflash_cache_attend(self.c, layer, q.data_ptr(), n_new.data_ptr(), batch, rows_per_seq, out.data_ptr(),
                                             _stream_on(stream, self.device)), "dflash_cache_attend")
            return
        if workspace is None:
            if self._shared is None:
                raise DFlashError(DFLASH_E_INVAL, "attention with a prefix needs a cache with shared_rows, or a workspace")
            workspace, nbytes = self._shared, self._shared_bytes
        else:
            _require_on(workspace, _torch_calls()[3], workspace.numel(), "workspace", self.device)
            nbytes = max(0, workspace.numel() - 256)
        check(self.L.dflash_cache_attend_shared(self.c, layer, q.data_ptr(), n_new.data_ptr(), batch, rows_per_seq, prefix,
                                                out.data_ptr(), (workspace.data_ptr() + 255) // 256 * 256, nbytes,
                                                _stream_on(stream, self.device)), "dflash_cache_attend_shared")

    def read(self, layer: int, first, count, batch: int, rows_per_seq: int, k_out, v_out, stream=None):
        """K and V of positions [first[s], first[s] + count[s]) of every sequence, dense: row
        s * rows_per_seq + r of k_out and v_out (fp16 or bf16 [batch * rows_per_seq][n_kv_heads][head_dim])
        is position first[s] + r. Rows past count[s] are left as they were."""
        i32 = _torch_calls()[2]
        numel = batch * rows_per_seq * self._kv_row
        _require_min(first, i32, batch, "first", self.device)
        _require_min(count, i32, batch, "count", self.device)
        _require_on(k_out, k_out.dtype, numel, "k_out", self.device)
        _require_on(v_out, k_out.dtype, numel, "v_out", self.device)
        check(self.L.dflash_cache_read(self.c, layer, first.data_ptr(), count.data_ptr(), batch, rows_per_seq,
                                       _DTYPES.get(str(k_out.dtype), -1), k_out.data_ptr(), v_out.data_ptr(),
                                       _stream_on(stream, self.device)), "dflash_cache_read")

    def device_error(self, clear: bool = True, stream=None) -> int:
        """The device error flags once the work queued on `stream` has finished."""
        f = c_int32(0)
        check(self.L.dflash_cache_read_error(self.c, ctypes.byref(f), 1 if clear else 0, _stream_on(stream, self.device)),
              "dflash_cache_read_error")
        return f.value

    def close(self):
        if getattr(self, "c", None):
            self.L.dflash_cache_destroy(self.c)
            self.c = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _require_31_bits(n: int, name) -> None:
    """The library's arguments are int32, and ctypes would drop the bits above."""
    if n >= 1 << 31:
        raise DFlashError(DFLASH_E_CAPACITY, f"{name} ({n}) must be less than 2^31")


def _require_min(t, dtype, numel, name, device):
    if t.dtype != dtype or t.device != device or not t.is_contiguous() or t.numel() < numel:
        raise DFlashError(DFLASH_E_INVAL, f"{name} must be a contiguous {dtype} tensor of at least {numel} values on {device}")


def _row_stride(t, dtype, rows: int, row: int, name, device) -> int:
    """Elements from one row of a [rows][row] or [rows][heads][dims] tensor to the next; each row
    has to be dense."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        n, heads, dims = shape
        step, per_head, one = stride
        dense = heads * dims == row and one == 1 and (heads == 1 or per_head == dims)
    else:
        n, step = shape[0] if shape else 0, stride[0] if stride else 0
        dense = len(shape) == 2 and shape[1] == row and stride[1] == 1
    if not dense or n != rows or t.dtype != dtype or t.device != device:
        raise DFlashError(DFLASH_E_INVAL, f"{name} must be {rows} dense rows of {row} values of one type on {device}")
    return step if rows > 1 else max(row, step // 8 * 8)   # a single row's stride means nothing


def rope_tables(n_positions: int, rope_dim: int, theta: float, linear: float = 1.0, bands=None, attention_factor: float = 1.0,
                device="cuda"):
    """cos and sin (fp32 [n_positions][rope_dim / 2], angles in float64) of rotary positions for
    PagedCache. Pair j turns by position * theta^(-2j / rope_dim). For contexts past the trained
    length: `linear` divides every angle; `bands` = (factor, low, high, trained) divides by `factor`
    the pairs that make fewer than `low` turns within `trained` positions, keeps those that make
    more than `high`, and goes linearly (in the number of turns) from one to the other between them.
    attention_factor scales cos and sin."""
    import math
    import torch
    inv = theta ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64) / max(1, rope_dim)) / linear
    if bands is not None:
        factor, low, high, trained = bands
        turns = trained * inv / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        inv = inv / factor * (1 - keep) + inv * keep
    angle = torch.arange(n_positions, dtype=torch.float64)[:, None] * inv
    return [(attention_factor * f(angle)).float().contiguous().to(device) for f in (torch.cos, torch.sin)]


def verify_greedy_noalloc(target_logits, drafted, batch: int, block: int, accept_len, committed, last_token,
                          stream=None):
    """Greedy verification with no handle and no allocation (scratch is a fixed array in the library)."""
    import torch
    _require(target_logits, torch.float32, "target_logits")
    for t, n in ((accept_len, "accept_len"), (committed, "committed"), (last_token, "last_token")):
        _require(t, torch.int32, n)
    if drafted is not None:
        _require(drafted, torch.int32, "drafted")
    check(lib().dflash_verify_greedy_noalloc(target_logits.data_ptr(), _ptr(drafted), batch, block,
                                             target_logits.shape[-1], accept_len.data_ptr(), committed.data_ptr(),
                                             last_token.data_ptr(), _stream(stream)), "dflash_verify_greedy_noalloc")


def synth_plant(logits, drafted, masks, n_steps: int, step_counter, batch: int, block: int, bump: float, saved,
                stream=None):
    check(lib().dflash_synth_plant(logits.data_ptr(), _ptr(drafted), masks.data_ptr(), n_steps,
                                   step_counter.data_ptr(), batch, block, logits.shape[-1], bump, saved.data_ptr(),
                                   _stream(stream)), "dflash_synth_plant")


def synth_unplant(logits, step_counter, n_steps: int, batch: int, block: int, saved, stream=None):
    check(lib().dflash_synth_unplant(logits.data_ptr(), step_counter.data_ptr(), n_steps, batch, block,
                                     saved.data_ptr(), _stream(stream)), "dflash_synth_unplant")
