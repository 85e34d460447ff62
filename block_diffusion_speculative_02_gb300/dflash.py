"""Thin ctypes binding of ``libdflash.so`` (the C ABI in include/dflash.h).

Argument marshalling only: every function takes torch tensors that already
live on the GPU, passes their device pointers and the current CUDA stream to
the library, and raises :class:`DFlashError` on a negative return code.  All
arithmetic happens in the CUDA kernels; there is no CPU fallback, and the
module refuses to load when the library has not been built.
"""
from __future__ import annotations

import ctypes
import operator
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# DFLASH_LIBRARY may name another build of the same library (e.g. one compiled
# with different tile parameters); the default is the in-tree build.
LIB_PATH = os.environ.get("DFLASH_LIBRARY") or os.path.join(_PKG, "libdflash.so")

DFLASH_OK = 0
STATUS_BITS = {
    "crop_grow": 1 << 0,
    "out_overflow": 1 << 1,
    "page_missing": 1 << 2,
    "pool_empty": 1 << 3,
    "bad_token": 1 << 4,
    "capacity": 1 << 5,
    "timeout": 1 << 6,
    "bad_value": 1 << 7,
}

EXPORTED = ["dflash_workspace_bytes", "dflash_workspace_init", "dflash_ctx_project",
            "dflash_block_attention", "dflash_verify_accept", "dflash_kv_crop",
            "dflash_read_status", "dflash_status_string", "dflash_version",
            "dflash_verify_accept_noalloc", "dflash_cycle_sm_split",
            "dflash_draft_workspace_bytes", "dflash_draft_qkv", "dflash_draft_mlp",
            "dflash_draft_tokens", "dflash_verify_attention", "dflash_gdn_replay",
            "dflash_prefill_workspace_bytes", "dflash_ctx_prefill", "dflash_selftest_wait",
            "dflash_prefill_attention", "dflash_prefill_staged",
            "dflash_kv4_workspace_bytes", "dflash_kv_reserve", "dflash_qk_norm_rope",
            "dflash_kv4_append", "dflash_kv4_gather", "dflash_kv4_attention",
            "dflash_fp8_norm_rows", "dflash_fp8_silu_mul", "dflash_fp8_weight",
            "dflash_fp8_linear", "dflash_fp8_grouped", "dflash_fp8_plan"]


class DFlashError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("block", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("n_ctx_layers", ctypes.c_int32),
                ("max_ctx", ctypes.c_int32), ("rope_theta", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("sm_budget", ctypes.c_int32)]


class KVViewC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("seq_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("free_list", ctypes.c_void_p), ("free_count", ctypes.c_void_p),
                ("capacity", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("n_pages", ctypes.c_int32)]


class KV4Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_tokens", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class KV4ViewC(ctypes.Structure):
    _fields_ = [("kv", KVViewC), ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    lib.dflash_workspace_bytes.restype = sz
    lib.dflash_workspace_bytes.argtypes = [ctypes.POINTER(Dims)]
    lib.dflash_workspace_init.restype = ctypes.c_int
    lib.dflash_workspace_init.argtypes = [vp, sz, vp]
    lib.dflash_ctx_project.restype = ctypes.c_int
    lib.dflash_ctx_project.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(vp), vp, vp, vp, vp,
                                       vp, vp, ctypes.POINTER(KVViewC), vp, sz, vp]
    lib.dflash_block_attention.restype = ctypes.c_int
    lib.dflash_block_attention.argtypes = [ctypes.POINTER(Dims), vp, vp, vp,
                                           ctypes.POINTER(KVViewC), ctypes.c_float, vp, vp, sz,
                                           vp]
    lib.dflash_verify_attention.restype = ctypes.c_int
    lib.dflash_verify_attention.argtypes = [ctypes.POINTER(Dims), vp, vp, vp,
                                            ctypes.POINTER(KVViewC), ctypes.c_float, vp, vp, sz,
                                            vp]
    lib.dflash_selftest_wait.restype = ctypes.c_int
    lib.dflash_selftest_wait.argtypes = [ctypes.c_int, vp, sz, vp]
    lib.dflash_prefill_workspace_bytes.restype = sz
    lib.dflash_prefill_workspace_bytes.argtypes = [ctypes.POINTER(Dims), i32]
    lib.dflash_ctx_prefill.restype = ctypes.c_int
    lib.dflash_ctx_prefill.argtypes = [ctypes.POINTER(Dims), i32, ctypes.POINTER(vp), vp, vp, vp,
                                       vp, vp, vp, ctypes.POINTER(KVViewC), vp, sz, vp]
    lib.dflash_prefill_attention.restype = ctypes.c_int
    lib.dflash_prefill_attention.argtypes = [ctypes.POINTER(Dims), i32, vp, vp, vp,
                                             ctypes.POINTER(KVViewC), ctypes.c_float, vp, vp, sz,
                                             vp]
    lib.dflash_prefill_staged.restype = ctypes.c_int
    lib.dflash_prefill_staged.argtypes = [ctypes.POINTER(Dims), vp, ctypes.c_int64, vp, vp, vp,
                                          sz, vp]
    lib.dflash_gdn_replay.restype = ctypes.c_int
    lib.dflash_gdn_replay.argtypes = [i32, i32, i32, i32] + [vp] * 6 + [vp, sz, vp]
    lib.dflash_verify_accept.restype = ctypes.c_int
    lib.dflash_verify_accept.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, vp, vp, vp, vp, vp,
                                         vp, i32, vp, sz, vp]
    lib.dflash_verify_accept_noalloc.restype = ctypes.c_int
    lib.dflash_verify_accept_noalloc.argtypes = [ctypes.POINTER(Dims), vp, vp, vp, vp, vp, vp, vp,
                                                 vp, vp, i32, vp]
    lib.dflash_kv_crop.restype = ctypes.c_int
    lib.dflash_kv_crop.argtypes = [ctypes.POINTER(KVViewC), i32, vp, i32, vp, sz, vp]
    lib.dflash_read_status.restype = ctypes.c_int
    lib.dflash_read_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int, vp]
    lib.dflash_status_string.restype = ctypes.c_char_p
    lib.dflash_status_string.argtypes = [ctypes.c_int]
    lib.dflash_version.restype = ctypes.c_int
    lib.dflash_version.argtypes = []
    lib.dflash_draft_workspace_bytes.restype = sz
    lib.dflash_draft_workspace_bytes.argtypes = [ctypes.POINTER(Dims), i32]
    lib.dflash_draft_qkv.restype = ctypes.c_int
    lib.dflash_draft_qkv.argtypes = [ctypes.POINTER(Dims)] + [vp] * 10 + [vp, sz, vp]
    lib.dflash_draft_mlp.restype = ctypes.c_int
    lib.dflash_draft_mlp.argtypes = [ctypes.POINTER(Dims), i32] + [vp] * 8 + [vp, sz, vp]
    lib.dflash_draft_tokens.restype = ctypes.c_int
    lib.dflash_draft_tokens.argtypes = [ctypes.POINTER(Dims)] + [vp] * 6 + [vp, sz, vp]
    dims4, view4, i64, f32 = (ctypes.POINTER(KV4Dims), ctypes.POINTER(KV4ViewC), ctypes.c_int64,
                              ctypes.c_float)
    lib.dflash_kv4_workspace_bytes.restype = sz
    lib.dflash_kv4_workspace_bytes.argtypes = [dims4]
    lib.dflash_kv_reserve.restype = ctypes.c_int
    lib.dflash_kv_reserve.argtypes = [dims4, ctypes.POINTER(KVViewC)] + [vp] * 6 + [sz, vp]
    lib.dflash_qk_norm_rope.restype = ctypes.c_int
    lib.dflash_qk_norm_rope.argtypes = [dims4, vp, i64, vp, i64, vp, vp, vp, f32, f32, vp, i64, vp,
                                        i64, vp]
    lib.dflash_kv4_append.restype = ctypes.c_int
    lib.dflash_kv4_append.argtypes = [dims4, vp, i64, vp, i64, vp, view4, vp, sz, vp]
    lib.dflash_kv4_gather.restype = ctypes.c_int
    lib.dflash_kv4_gather.argtypes = [dims4, vp, view4, vp, vp, vp, sz, vp]
    lib.dflash_kv4_attention.restype = ctypes.c_int
    lib.dflash_kv4_attention.argtypes = [dims4, vp, vp, view4, f32, ctypes.c_int, vp, vp, sz, vp]
    lib.dflash_fp8_norm_rows.restype = ctypes.c_int
    lib.dflash_fp8_norm_rows.argtypes = [i32, i32, vp, i64, vp, i64, vp, f32, vp, i64, vp, vp, vp]
    lib.dflash_fp8_silu_mul.restype = ctypes.c_int
    lib.dflash_fp8_silu_mul.argtypes = [i32, i32, vp, i64, vp, vp, vp]
    lib.dflash_fp8_weight.restype = ctypes.c_int
    lib.dflash_fp8_weight.argtypes = [i32, i32, i32, vp, vp, vp, vp]
    lib.dflash_fp8_linear.restype = ctypes.c_int
    lib.dflash_fp8_linear.argtypes = [i32] * 3 + [vp] * 5 + [i64, vp, sz, vp]
    lib.dflash_fp8_grouped.restype = ctypes.c_int
    lib.dflash_fp8_grouped.argtypes = [i32] * 5 + [vp] * 7 + [i64, vp, sz, vp]
    lib.dflash_fp8_plan.restype = ctypes.c_int
    lib.dflash_fp8_plan.argtypes = [i32] * 4 + [ctypes.c_int, i32] + [ctypes.POINTER(i32)] * 3
    lib.dflash_cycle_sm_split.restype = ctypes.c_int
    lib.dflash_cycle_sm_split.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(i32),
                                          ctypes.POINTER(i32)]
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().dflash_status_string(int(code)).decode()


def _check(rc: int, where: str):
    if rc != DFLASH_OK:
        raise DFlashError(rc, where)


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t: Optional[torch.Tensor], dtype=None, name="tensor") -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def make_dims(batch, hidden, n_q_heads, n_kv_heads, head_dim, vocab, n_ctx_layers, max_ctx,
              rope_theta=1.0e6, rms_eps=1.0e-6, block=16, sm_budget=0) -> Dims:
    return Dims(batch, block, hidden, n_q_heads, n_kv_heads, head_dim, vocab, n_ctx_layers,
                max_ctx, rope_theta, rms_eps, sm_budget)


def with_sm_budget(dims: Dims, sm_budget: int) -> Dims:
    """A copy of ``dims`` whose LM-head / projection grids use at most ``sm_budget`` SMs."""
    d = Dims.from_buffer_copy(dims)
    d.sm_budget = int(sm_budget)
    return d


def dflash_cycle_sm_split(dims: Dims):
    """(verify_sms, project_sms): SM budgets for running verify and the projection concurrently."""
    v, p = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(load_library().dflash_cycle_sm_split(ctypes.byref(dims), ctypes.byref(v),
                                                ctypes.byref(p)), "dflash_cycle_sm_split")
    return int(v.value), int(p.value)


class _View:
    """A view's fields, and the C structs that _view_struct keeps on it: these hold addresses, so
    they stay out of copies and pickles, and go when a field that they are made of is set."""

    _KEPT = ("_struct", "_pages")

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k not in self._KEPT}

    def _drop(self, name):
        d = self.__dict__
        d.pop("_struct", None)
        if name not in ("cells", "k_exp", "v_exp"):
            d.pop("_pages", None)

    def __setattr__(self, name, value):
        self._drop(name)
        super().__setattr__(name, value)

    def __delattr__(self, name):
        self._drop(name)
        super().__delattr__(name)


@dataclass
class KVView(_View):
    """A KV cache held in torch tensors (see dflash_kv_view in include/dflash.h)."""
    k: Optional[torch.Tensor]
    v: Optional[torch.Tensor]
    seq_len: torch.Tensor                      # int32 [B]
    capacity: int
    page_table: Optional[torch.Tensor] = None  # int32 [B, max_pages]
    free_list: Optional[torch.Tensor] = None   # int32 [n_pages]
    free_count: Optional[torch.Tensor] = None  # int32 [1]
    page_size: int = 16

    def c(self) -> KVViewC:
        paged = self.page_table is not None
        return KVViewC(
            _dev(self.k, torch.bfloat16, "k"), _dev(self.v, torch.bfloat16, "v"),
            _dev(self.seq_len, torch.int32, "seq_len"),
            _dev(self.page_table, torch.int32, "page_table"),
            _dev(self.free_list, torch.int32, "free_list"),
            _dev(self.free_count, torch.int32, "free_count"),
            int(self.capacity), int(self.page_size if paged else 0),
            int(self.page_table.shape[1]) if paged else 0,
            int(self.free_list.shape[0]) if paged else 0)


def dflash_workspace_bytes(dims: Dims) -> int:
    n = load_library().dflash_workspace_bytes(ctypes.byref(dims))
    if n == 0:
        raise DFlashError(-3, "dflash_workspace_bytes")
    return int(n)


def alloc_workspace(dims: Dims, device="cuda") -> torch.Tensor:
    """A zeroed workspace tensor of the size the library asks for."""
    return torch.zeros(dflash_workspace_bytes(dims), dtype=torch.uint8, device=device)


def dflash_workspace_init(ws: torch.Tensor, stream=None):
    _check(load_library().dflash_workspace_init(_dev(ws, name="ws"), ws.numel(), _stream(stream)),
           "dflash_workspace_init")


def dflash_ctx_project(dims: Dims, layer_hidden: Sequence[torch.Tensor], w_fc, hidden_norm_w,
                       w_k, w_v, k_norm_w, write_pos, cache: KVView, ws, stream=None):
    ptrs = (ctypes.c_void_p * len(layer_hidden))(
        *[_dev(h, torch.bfloat16, "layer_hidden") for h in layer_hidden])
    view = cache.c()
    _check(load_library().dflash_ctx_project(
        ctypes.byref(dims), ptrs, _dev(w_fc, torch.bfloat16, "w_fc"),
        _dev(hidden_norm_w, torch.bfloat16, "hidden_norm_w"), _dev(w_k, torch.bfloat16, "w_k"),
        _dev(w_v, torch.bfloat16, "w_v"), _dev(k_norm_w, torch.bfloat16, "k_norm_w"),
        _dev(write_pos, torch.int32, "write_pos"), ctypes.byref(view), _dev(ws, name="ws"),
        ws.numel(), _stream(stream)), "dflash_ctx_project")


def dflash_selftest_wait(arrive: bool, ws, stream=None):
    """The bounded waits: completed at once (arrive) or timed out after ~1 s (status bit)."""
    _check(load_library().dflash_selftest_wait(1 if arrive else 0, _dev(ws, name="ws"),
                                               ws.numel(), _stream(stream)),
           "dflash_selftest_wait")


def dflash_prefill_workspace_bytes(dims: Dims, tokens_per_seq: int) -> int:
    n = load_library().dflash_prefill_workspace_bytes(ctypes.byref(dims), int(tokens_per_seq))
    if n == 0:
        raise DFlashError(-3, "dflash_prefill_workspace_bytes")
    return int(n)


def alloc_prefill_workspace(dims: Dims, tokens_per_seq: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for dflash_ctx_prefill with this many tokens per sequence."""
    return torch.zeros(dflash_prefill_workspace_bytes(dims, tokens_per_seq), dtype=torch.uint8,
                       device=device)


def dflash_ctx_prefill(dims: Dims, tokens_per_seq: int, layer_hidden: Sequence[torch.Tensor],
                       w_fc, hidden_norm_w, w_k, w_v, k_norm_w, write_pos, cache: KVView, ws,
                       stream=None):
    """Whole-prompt context projection: tokens_per_seq rows per sequence appended at write_pos."""
    ptrs = (ctypes.c_void_p * len(layer_hidden))(
        *[_dev(h, torch.bfloat16, "layer_hidden") for h in layer_hidden])
    view = cache.c()
    _check(load_library().dflash_ctx_prefill(
        ctypes.byref(dims), int(tokens_per_seq), ptrs, _dev(w_fc, torch.bfloat16, "w_fc"),
        _dev(hidden_norm_w, torch.bfloat16, "hidden_norm_w"), _dev(w_k, torch.bfloat16, "w_k"),
        _dev(w_v, torch.bfloat16, "w_v"), _dev(k_norm_w, torch.bfloat16, "k_norm_w"),
        _dev(write_pos, torch.int32, "write_pos"), ctypes.byref(view), _dev(ws, name="ws"),
        ws.numel(), _stream(stream)), "dflash_ctx_prefill")


def dflash_prefill_attention(dims: Dims, tokens_per_seq: int, q, k, v, cache: KVView,
                             scale: float, out, ws, stream=None):
    """The target's attention over a prompt chunk of tokens_per_seq rows per
    sequence (causal), the chunk's K/V appended to ``cache``."""
    view = cache.c()
    _check(load_library().dflash_prefill_attention(
        ctypes.byref(dims), int(tokens_per_seq), _dev(q, torch.bfloat16, "q"),
        _dev(k, torch.bfloat16, "k"), _dev(v, torch.bfloat16, "v"), ctypes.byref(view),
        float(scale), _dev(out, torch.bfloat16, "out"), _dev(ws, name="ws"), ws.numel(),
        _stream(stream)), "dflash_prefill_attention")


def dflash_prefill_staged(dims: Dims, last_hidden, w_lm, staged, ws, stream=None):
    """The first staged token per sequence: argmax of the LM head at the last
    prompt row.  ``last_hidden``: bf16 [B, H] whose rows may be strided (e.g.
    ``h[:, -1]`` of a [B, T, H] tensor); its row stride is passed on."""
    if not isinstance(last_hidden, torch.Tensor) or not last_hidden.is_cuda:
        raise ValueError("last_hidden must be a CUDA tensor")
    if last_hidden.dtype != torch.bfloat16 or last_hidden.dim() != 2 or last_hidden.stride(1) != 1:
        raise ValueError("last_hidden must be bf16 [B, H] with unit column stride")
    _check(load_library().dflash_prefill_staged(
        ctypes.byref(dims), last_hidden.data_ptr(), int(last_hidden.stride(0)),
        _dev(w_lm, torch.bfloat16, "w_lm"), _dev(staged, torch.int32, "staged"),
        _dev(ws, name="ws"), ws.numel(), _stream(stream)), "dflash_prefill_staged")


def dflash_block_attention(dims: Dims, q_blk, k_blk, v_blk, cache: KVView, scale: float, out,
                           ws, stream=None):
    view = cache.c()
    _check(load_library().dflash_block_attention(
        ctypes.byref(dims), _dev(q_blk, torch.bfloat16, "q_blk"),
        _dev(k_blk, torch.bfloat16, "k_blk"), _dev(v_blk, torch.bfloat16, "v_blk"),
        ctypes.byref(view), float(scale), _dev(out, torch.bfloat16, "out"), _dev(ws, name="ws"),
        ws.numel(), _stream(stream)), "dflash_block_attention")


def dflash_verify_attention(dims: Dims, q_blk, k_blk, v_blk, cache: KVView, scale: float, out,
                            ws, stream=None):
    """The target's verify attention: causal inside the block, block K/V appended to ``cache``."""
    view = cache.c()
    _check(load_library().dflash_verify_attention(
        ctypes.byref(dims), _dev(q_blk, torch.bfloat16, "q_blk"),
        _dev(k_blk, torch.bfloat16, "k_blk"), _dev(v_blk, torch.bfloat16, "v_blk"),
        ctypes.byref(view), float(scale), _dev(out, torch.bfloat16, "out"), _dev(ws, name="ws"),
        ws.numel(), _stream(stream)), "dflash_verify_attention")


def dflash_verify_accept(dims: Dims, hidden, w_lm, block_ids, len_before, posterior, accept_len,
                         next_staged, commit_len, out_tokens, ws, stream=None):
    _check(load_library().dflash_verify_accept(
        ctypes.byref(dims), _dev(hidden, torch.bfloat16, "hidden"),
        _dev(w_lm, torch.bfloat16, "w_lm"), _dev(block_ids, torch.int32, "block_ids"),
        _dev(len_before, torch.int32, "len_before"), _dev(posterior, torch.int32, "posterior"),
        _dev(accept_len, torch.int32, "accept_len"),
        _dev(next_staged, torch.int32, "next_staged"),
        _dev(commit_len, torch.int32, "commit_len"), _dev(out_tokens, torch.int32, "out_tokens"),
        int(out_tokens.shape[-1]), _dev(ws, name="ws"), ws.numel(), _stream(stream)),
        "dflash_verify_accept")


def dflash_verify_accept_noalloc(dims: Dims, hidden, w_lm, block_ids, len_before, posterior,
                                 accept_len, next_staged, commit_len, out_tokens, stream=None):
    """dflash_verify_accept without a workspace (library-owned static scratch)."""
    _check(load_library().dflash_verify_accept_noalloc(
        ctypes.byref(dims), _dev(hidden, torch.bfloat16, "hidden"),
        _dev(w_lm, torch.bfloat16, "w_lm"), _dev(block_ids, torch.int32, "block_ids"),
        _dev(len_before, torch.int32, "len_before"), _dev(posterior, torch.int32, "posterior"),
        _dev(accept_len, torch.int32, "accept_len"),
        _dev(next_staged, torch.int32, "next_staged"),
        _dev(commit_len, torch.int32, "commit_len"), _dev(out_tokens, torch.int32, "out_tokens"),
        int(out_tokens.shape[-1]), _stream(stream)), "dflash_verify_accept_noalloc")


def dflash_kv_crop(views: Sequence[KVView], new_len, batch: int, ws, stream=None):
    arr = (KVViewC * len(views))(*[v.c() for v in views])
    _check(load_library().dflash_kv_crop(arr, len(views), _dev(new_len, torch.int32, "new_len"),
                                         int(batch), _dev(ws, name="ws"), ws.numel(),
                                         _stream(stream)), "dflash_kv_crop")


def dflash_read_status(ws, clear: bool = True, stream=None) -> int:
    out = ctypes.c_uint32(0)
    _check(load_library().dflash_read_status(_dev(ws, name="ws"), ctypes.byref(out),
                                             1 if clear else 0, _stream(stream)),
           "dflash_read_status")
    return int(out.value)


def dflash_version() -> int:
    return int(load_library().dflash_version())


# ---------------------------------------------------------------------------
# the rest of one drafter layer and the drafter's tokens
# ---------------------------------------------------------------------------
def dflash_draft_workspace_bytes(dims: Dims, ffn: int) -> int:
    n = load_library().dflash_draft_workspace_bytes(ctypes.byref(dims), int(ffn))
    if n == 0:
        raise DFlashError(-3, "dflash_draft_workspace_bytes")
    return int(n)


def alloc_draft_workspace(dims: Dims, ffn: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for the dflash_draft_* calls."""
    return torch.zeros(dflash_draft_workspace_bytes(dims, ffn), dtype=torch.uint8, device=device)


def dflash_draft_qkv(dims: Dims, x, ln1_w, w_q, w_k, w_v, q_norm_w, k_norm_w, q_out, k_out, v_out,
                     ws, stream=None):
    bf = torch.bfloat16
    _check(load_library().dflash_draft_qkv(
        ctypes.byref(dims), _dev(x, bf, "x"), _dev(ln1_w, bf, "ln1_w"), _dev(w_q, bf, "w_q"),
        _dev(w_k, bf, "w_k"), _dev(w_v, bf, "w_v"), _dev(q_norm_w, bf, "q_norm_w"),
        _dev(k_norm_w, bf, "k_norm_w"), _dev(q_out, bf, "q_out"), _dev(k_out, bf, "k_out"),
        _dev(v_out, bf, "v_out"), _dev(ws, name="ws"), ws.numel(), _stream(stream)),
        "dflash_draft_qkv")


def dflash_draft_mlp(dims: Dims, ffn: int, x, attn_out, w_o, ln2_w, w_gate, w_up, w_down, x_out,
                     ws, stream=None):
    bf = torch.bfloat16
    _check(load_library().dflash_draft_mlp(
        ctypes.byref(dims), int(ffn), _dev(x, bf, "x"), _dev(attn_out, bf, "attn_out"),
        _dev(w_o, bf, "w_o"), _dev(ln2_w, bf, "ln2_w"), _dev(w_gate, bf, "w_gate"),
        _dev(w_up, bf, "w_up"), _dev(w_down, bf, "w_down"), _dev(x_out, bf, "x_out"),
        _dev(ws, name="ws"), ws.numel(), _stream(stream)), "dflash_draft_mlp")


def dflash_draft_tokens(dims: Dims, x, final_norm_w, w_lm, staged, block_ids, posterior, ws,
                        stream=None):
    bf = torch.bfloat16
    _check(load_library().dflash_draft_tokens(
        ctypes.byref(dims), _dev(x, bf, "x"), _dev(final_norm_w, bf, "final_norm_w"),
        _dev(w_lm, bf, "w_lm"), _dev(staged, torch.int32, "staged"),
        _dev(block_ids, torch.int32, "block_ids"), _dev(posterior, torch.int32, "posterior"),
        _dev(ws, name="ws"), ws.numel(), _stream(stream)), "dflash_draft_tokens")


def dflash_gdn_replay(state, tape_k, tape_v, tape_beta, tape_g, accept_len, ws, stream=None):
    """Replay the committed 1 + a steps of the recorded tape onto ``state`` (in place)."""
    B, NH, Dv, Dk = state.shape
    _check(load_library().dflash_gdn_replay(
        int(B), int(NH), int(Dk), int(Dv), _dev(state, torch.float32, "state"),
        _dev(tape_k, torch.bfloat16, "tape_k"), _dev(tape_v, torch.bfloat16, "tape_v"),
        _dev(tape_beta, torch.float32, "tape_beta"), _dev(tape_g, torch.float32, "tape_g"),
        _dev(accept_len, torch.int32, "accept_len"), _dev(ws, name="ws"), ws.numel(),
        _stream(stream)), "dflash_gdn_replay")


# ---------------------------------------------------------------------------
# serving over a KV cache held in 4 bits
# ---------------------------------------------------------------------------
def make_kv4_dims(batch, n_tokens, max_tokens, n_q_heads, n_kv_heads, head_dim) -> KV4Dims:
    return KV4Dims(batch, n_tokens, max_tokens, n_q_heads, n_kv_heads, head_dim)


@dataclass
class KV4View(_View):
    """A KV cache in 4-bit cells (see dflash_kv4_view in include/dflash.h).

    ``cells``: uint8 [n_pages, Hkv, page_size / 16, 18 D] (paged) or
    [B, Hkv, capacity / 16, 18 D].  A paged view has its ``free_list`` in every
    call: its length is n_pages.  ``pages()`` is the view that
    dflash_kv_reserve and dflash_kv_crop take."""
    cells: torch.Tensor
    seq_len: torch.Tensor                      # int32 [B]
    capacity: int
    page_table: Optional[torch.Tensor] = None  # int32 [B, max_pages]
    free_list: Optional[torch.Tensor] = None   # int32 [n_pages]
    free_count: Optional[torch.Tensor] = None  # int32 [1]
    page_size: int = 16
    k_exp: Optional[torch.Tensor] = None       # int32 [Hkv]
    v_exp: Optional[torch.Tensor] = None

    def pages(self) -> KVView:
        return KVView(None, None, self.seq_len, self.capacity, self.page_table, self.free_list,
                      self.free_count, self.page_size)


def alloc_kv4_cells(n_slabs: int, n_kv_heads: int, rows: int, head_dim: int,
                    device="cuda") -> torch.Tensor:
    """Zeroed cells for ``n_slabs`` pages (or sequences) of ``rows`` rows (a multiple of 16)."""
    if rows < 16 or rows % 16 or head_dim not in (64, 128):
        raise ValueError("rows must be a multiple of 16 and head_dim 64 or 128")
    return torch.zeros(n_slabs, n_kv_heads, rows // 16, 18 * head_dim, dtype=torch.uint8,
                       device=device)


def dflash_kv4_workspace_bytes(dims: KV4Dims) -> int:
    n = load_library().dflash_kv4_workspace_bytes(ctypes.byref(dims))
    if n == 0:
        raise DFlashError(-3, "dflash_kv4_workspace_bytes")
    return int(n)


def alloc_kv4_workspace(dims: KV4Dims, device="cuda") -> torch.Tensor:
    """A zeroed workspace for the calls over a 4-bit cache."""
    return torch.zeros(dflash_kv4_workspace_bytes(dims), dtype=torch.uint8, device=device)


def _bad(t, device: int, dtype, numel, name: str):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != device \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{device}")
    raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")


def _on(t, device: int, dtype, numel: int, name: str) -> int:
    """Pointer of a contiguous tensor on this device with this type and size."""
    if getattr(t, "dtype", None) is not dtype or t.get_device() != device \
            or not t.is_contiguous() or t.numel() != numel:
        _bad(t, device, dtype, numel, name)
    return t.data_ptr()


def _opt(t, device: int, dtype, numel: int, name: str) -> Optional[int]:
    return None if t is None else _on(t, device, dtype, numel, name)


def _ws_on(ws, device: int):
    """(pointer, bytes) of a workspace."""
    if getattr(ws, "dtype", None) is not torch.uint8 or ws.get_device() != device \
            or not ws.is_contiguous():
        _bad(ws, device, torch.uint8, None, "ws")
    return ws.data_ptr(), ws.numel()


def _rows_on(t, device: int, rows: int, heads: int, d: int, name: str):
    """(pointer, row pitch) of a bf16 [rows, heads, D] tensor whose rows are contiguous."""
    if getattr(t, "dtype", None) is not torch.bfloat16 or t.get_device() != device:
        raise ValueError(f"{name} must be a bf16 tensor on cuda:{device}")
    if t.shape != (rows, heads, d):
        raise ValueError(f"{name} must be [{rows}, {heads}, {d}], got {tuple(t.shape)}")
    st = t.stride()
    if st[2] != 1 or (st[1] != d and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.data_ptr(), st[0] if rows > 1 else heads * d


_PAGE_TENSORS = operator.attrgetter("seq_len", "page_table", "free_list", "free_count")
_VIEW_TENSORS = operator.attrgetter("seq_len", "page_table", "free_list", "free_count", "cells",
                                    "k_exp", "v_exp")


def _view_struct(v, device: int, batch: int, hkv: int, d: int):
    """The C struct of a view (with hkv 0: of its lengths and pages only), checked.

    The struct is kept on the view until one of its fields is set, and used again as long as the
    tensors lie where they did, have the shapes they had, and are contiguous still.  It holds
    none of them alive."""
    try:
        tensors = (_VIEW_TENSORS if hkv else _PAGE_TENSORS)(v)
        key = [device, batch, hkv, d,
               *[t if t is None else (t.data_ptr(), t.shape, t.is_contiguous()) for t in tensors]]
    except AttributeError:                    # not a view, or not a tensor: see below
        if not isinstance(v, KV4View) and (hkv or not isinstance(v, KVView)):
            raise ValueError("the cache must be a KV4View" + ("" if hkv else " or a KVView")) \
                from None
        key = None
    slot = "_struct" if hkv else "_pages"
    memo = v.__dict__.get(slot)
    if memo is not None and memo[0] == key:
        return memo[1]
    i32 = torch.int32
    seq = _on(v.seq_len, device, i32, batch, "seq_len")
    table, n, k = v.page_table, 0, None
    if table is not None:
        if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[0] != batch:
            raise ValueError(f"page_table must be an int32 tensor [{batch}, max_pages]")
        if not isinstance(v.free_list, torch.Tensor):
            raise ValueError("free_list must be a tensor: its length is the pool's number of pages")
        n = v.free_list.numel()
    if hkv:
        rows, slabs = (v.page_size, n) if table is not None else (v.capacity, batch)
        k = _on(v.cells, device, torch.uint8, slabs * hkv * (rows // 16) * 18 * d, "cells")
    if table is None:
        c = KVViewC(k, None, seq, None, None, None, v.capacity, 0, 0, 0)
    else:
        c = KVViewC(k, None, seq, _on(table, device, i32, table.numel(), "page_table"),
                    _on(v.free_list, device, i32, n, "free_list"),
                    _on(v.free_count, device, i32, 1, "free_count"),
                    v.capacity, v.page_size, table.shape[1], n)
    if hkv:
        c = KV4ViewC(c, _opt(v.k_exp, device, i32, hkv, "k_exp"),
                     _opt(v.v_exp, device, i32, hkv, "v_exp"))
    v.__dict__[slot] = (key, c)
    return c


def _here(stream):
    """(current device, the stream to launch on)."""
    dev = torch._C._cuda_getDevice()
    return dev, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def dflash_kv_reserve(dims: KV4Dims, cache, n_new, start, pos, slot, new_len, ws, stream=None):
    """Pages, positions and slots of the batch's new rows.  ``cache``: a KVView or KV4View."""
    dev, st = _here(stream)
    i32, b, n = torch.int32, dims.batch, dims.n_tokens
    rc = load_library().dflash_kv_reserve(
        dims, _view_struct(cache, dev, b, 0, 0),
        _on(n_new, dev, i32, b, "n_new"), _on(start, dev, i32, b + 1, "start"),
        _on(pos, dev, i32, n, "pos"), _on(slot, dev, i32, n, "slot"),
        _on(new_len, dev, i32, b, "new_len"), *_ws_on(ws, dev), st)
    if rc:
        _check(rc, "dflash_kv_reserve")


def dflash_qk_norm_rope(dims: KV4Dims, q, k, q_norm_w, k_norm_w, pos, rope_theta: float,
                        rms_eps: float, q_out, k_out, stream=None):
    """Per-head norms of q [N, Hq, D] and k [N, Hkv, D], rotated at ``pos``; rows may be strided."""
    dev, st = _here(stream)
    bf, n, d, hq, hkv = torch.bfloat16, dims.n_tokens, dims.head_dim, dims.n_q_heads, \
        dims.n_kv_heads
    rc = load_library().dflash_qk_norm_rope(
        dims, *_rows_on(q, dev, n, hq, d, "q"), *_rows_on(k, dev, n, hkv, d, "k"),
        _opt(q_norm_w, dev, bf, d, "q_norm_w"), _opt(k_norm_w, dev, bf, d, "k_norm_w"),
        _on(pos, dev, torch.int32, n, "pos"), rope_theta, rms_eps,
        *_rows_on(q_out, dev, n, hq, d, "q_out"), *_rows_on(k_out, dev, n, hkv, d, "k_out"), st)
    if rc:
        _check(rc, "dflash_qk_norm_rope")


def dflash_kv4_append(dims: KV4Dims, k, v, slot, cache: KV4View, ws, stream=None):
    """Quantise k, v [N, Hkv, D] (rows may be strided) into the rows ``slot`` of the cache."""
    dev, st = _here(stream)
    n, hkv, d = dims.n_tokens, dims.n_kv_heads, dims.head_dim
    rc = load_library().dflash_kv4_append(
        dims, *_rows_on(k, dev, n, hkv, d, "k"), *_rows_on(v, dev, n, hkv, d, "v"),
        _on(slot, dev, torch.int32, n, "slot"), _view_struct(cache, dev, dims.batch, hkv, d),
        *_ws_on(ws, dev), st)
    if rc:
        _check(rc, "dflash_kv4_append")


def dflash_kv4_gather(dims: KV4Dims, slot, cache: KV4View, k_out, v_out, ws, stream=None):
    """Rows ``slot`` of the cache as bf16 [N, Hkv, D]."""
    dev, st = _here(stream)
    bf, n, hkv, d = torch.bfloat16, dims.n_tokens, dims.n_kv_heads, dims.head_dim
    size = n * hkv * d
    rc = load_library().dflash_kv4_gather(
        dims, _on(slot, dev, torch.int32, n, "slot"), _view_struct(cache, dev, dims.batch, hkv, d),
        _on(k_out, dev, bf, size, "k_out"), _on(v_out, dev, bf, size, "v_out"), *_ws_on(ws, dev),
        st)
    if rc:
        _check(rc, "dflash_kv4_gather")


def dflash_kv4_attention(dims: KV4Dims, q, start, cache: KV4View, scale: float, causal: bool, out,
                         ws, stream=None):
    """Attention of the rows q [N, Hq, D] over the 4-bit cache that holds them already."""
    dev, st = _here(stream)
    bf, b, hkv, d = torch.bfloat16, dims.batch, dims.n_kv_heads, dims.head_dim
    size = dims.n_tokens * dims.n_q_heads * d
    rc = load_library().dflash_kv4_attention(
        dims, _on(q, dev, bf, size, "q"), _on(start, dev, torch.int32, b + 1, "start"),
        _view_struct(cache, dev, b, hkv, d), scale, 1 if causal else 0,
        _on(out, dev, bf, size, "out"), *_ws_on(ws, dev), st)
    if rc:
        _check(rc, "dflash_kv4_attention")


# ---------------------------------------------------------------------------
# linear layers in 8-bit floating point
# ---------------------------------------------------------------------------
F8, _BF, _F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


def _up128(n: int) -> int:
    return -(-n // 128)


def alloc_fp8_workspace(device="cuda") -> torch.Tensor:
    """A zeroed workspace for dflash_fp8_linear and dflash_fp8_grouped (their status word)."""
    return torch.zeros(256, dtype=torch.uint8, device=device)


def alloc_fp8_rows(rows: int, cols: int, device="cuda"):
    """(codes e4m3 [rows, cols], scales fp32 [ceil(cols / 128), rows])."""
    return (torch.empty(rows, cols, dtype=F8, device=device),
            torch.empty(_up128(cols), rows, dtype=torch.float32, device=device))


def alloc_fp8_weight(*shape, device="cuda"):
    """(codes e4m3 [.., N, K], scales fp32 [.., ceil(N / 128), ceil(K / 128)])."""
    *g, n, k = shape
    return (torch.empty(*g, n, k, dtype=F8, device=device),
            torch.empty(*g, _up128(n), _up128(k), dtype=torch.float32, device=device))


def _whole(t, device: int, dtype, shape, name: str) -> int:
    """Pointer of a contiguous tensor of this type and shape (None: any) on this device."""
    if getattr(t, "dtype", None) is not dtype or t.get_device() != device \
            or not t.is_contiguous():
        _bad(t, device, dtype, None, name)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _codes(q, scale, device: int, shape, scales, name: str, scale_name: str):
    """Pointers of e4m3 codes (shape None: the one the call goes by) and their fp32 scales, both
    contiguous.  (Checked in one expression; where it does not hold, one by one, to say what is
    wrong.)"""
    try:
        if q.dtype is F8 and scale.dtype is _F32 and (shape is None or q.shape == shape) \
                and scale.shape == scales and q.is_contiguous() and scale.is_contiguous() \
                and q.get_device() == device and scale.get_device() == device:
            return q.data_ptr(), scale.data_ptr()
    except AttributeError:
        pass
    return _whole(q, device, F8, shape, name), _whole(scale, device, _F32, scales, scale_name)


def _matrix(t, device: int, name: str, shape):
    """(pointer, row pitch) of a bf16 matrix whose rows are contiguous and may lie apart."""
    if getattr(t, "dtype", None) is not _BF or t.get_device() != device:
        raise ValueError(f"{name} must be a bf16 tensor on cuda:{device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    pitch, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the columns of a row must be contiguous")
    return t.data_ptr(), pitch if shape[0] > 1 else shape[1]


def _shape(t, dims: int, name: str):
    """The shape of a tensor of this many dimensions."""
    shape = getattr(t, "shape", None)
    if shape is None or len(shape) != dims:
        raise ValueError(f"{name} must be a tensor of {dims} dimensions")
    return shape


def _past_31_bits(*sizes):
    """The C calls take sizes of 31 bits; ctypes would cut off the rest."""
    raise ValueError(f"sizes {list(sizes)}: none may be past 2^31 - 1")


def dflash_fp8_norm_rows(x, residual, norm_w, rms_eps: float, sum_out, q, scale, stream=None):
    """q, scale = 8-bit rows of RMSNorm(x + residual) * norm_w; sum_out = x + residual.

    ``residual``, ``norm_w`` and ``sum_out`` may be None: nothing added, not normed, not stored."""
    dev, st = _here(stream)
    shape = rows, cols = _shape(x, 2, "x")
    if (rows | cols) >> 31:
        _past_31_bits(rows, cols)
    rc = load_library().dflash_fp8_norm_rows(
        rows, cols, *_matrix(x, dev, "x", shape),
        *((None, 0) if residual is None else _matrix(residual, dev, "residual", shape)),
        None if norm_w is None else _whole(norm_w, dev, _BF, (cols,), "norm_w"), rms_eps,
        *((None, 0) if sum_out is None else _matrix(sum_out, dev, "sum_out", shape)),
        *_codes(q, scale, dev, shape, (-(-cols // 128), rows), "q", "scale"), st)
    if rc:
        _check(rc, "dflash_fp8_norm_rows")


def dflash_fp8_silu_mul(gate_up, q, scale, stream=None):
    """q, scale = 8-bit rows of silu(gate) * up, gate_up [M, 2 F]: gate, then up."""
    dev, st = _here(stream)
    shape = rows, cols = _shape(gate_up, 2, "gate_up")
    if cols % 2:
        raise ValueError("gate_up must have an even number of columns: gate, then up")
    cols //= 2
    if (rows | cols) >> 31:
        _past_31_bits(rows, cols)
    rc = load_library().dflash_fp8_silu_mul(
        rows, cols, *_matrix(gate_up, dev, "gate_up", shape),
        *_codes(q, scale, dev, (rows, cols), (-(-cols // 128), rows), "q", "scale"), st)
    if rc:
        _check(rc, "dflash_fp8_silu_mul")


def dflash_fp8_weight(w, q, scale, stream=None):
    """q, scale = 8-bit weights of w, bf16 [N, K] or, of several experts, [G, N, K]."""
    dev, st = _here(stream)
    shape = getattr(w, "shape", ())
    if len(shape) not in (2, 3):
        raise ValueError("w must be a tensor [N, K] or [G, N, K]")
    *g, n, k = shape
    groups = g[0] if g else 1
    if (groups | n | k) >> 31:
        _past_31_bits(groups, n, k)
    rc = load_library().dflash_fp8_weight(
        groups, n, k, _whole(w, dev, _BF, None, "w"),
        *_codes(q, scale, dev, shape, (*g, -(-n // 128), -(-k // 128)), "q", "scale"), st)
    if rc:
        _check(rc, "dflash_fp8_weight")


def _product(x, x_scale, w, w_scale, out, ws, device: int, xs_shape, ws_shape, out_shape):
    """What a product takes: pointers of x, w and their scales, of out with its row pitch, and of
    the workspace with its size.  (Checked in one expression; where it does not hold, one by one.)"""
    try:
        if x.dtype is F8 and w.dtype is F8 and x_scale.dtype is _F32 and w_scale.dtype is _F32 \
                and out.dtype is _BF and ws.dtype is torch.uint8 \
                and x_scale.shape == xs_shape and w_scale.shape == ws_shape \
                and out.shape == out_shape and x.is_contiguous() and w.is_contiguous() \
                and x_scale.is_contiguous() and w_scale.is_contiguous() and ws.is_contiguous() \
                and device == x.get_device() == w.get_device() == x_scale.get_device() \
                == w_scale.get_device() == out.get_device() == ws.get_device():
            pitch, step = out.stride()
            if step == 1:
                return (x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
                        out.data_ptr(), pitch if out_shape[0] > 1 else out_shape[1],
                        ws.data_ptr(), ws.numel())
    except AttributeError:
        pass
    return (*_codes(x, x_scale, device, None, xs_shape, "x", "x_scale"),
            *_codes(w, w_scale, device, None, ws_shape, "w", "w_scale"),
            *_matrix(out, device, "out", out_shape), *_ws_on(ws, device))


def dflash_fp8_linear(x, x_scale, w, w_scale, out, ws, stream=None):
    """out [M, N] (bf16, rows may be strided) = x w^T of 8-bit rows x [M, K], weights w [N, K]."""
    dev, st = _here(stream)
    m, k = _shape(x, 2, "x")
    n, kw = _shape(w, 2, "w")
    if kw != k:
        raise ValueError(f"x has {k} columns, w {kw}")
    if (m | n | k) >> 31:
        _past_31_bits(m, n, k)
    kb = -(-k // 128)
    rc = load_library().dflash_fp8_linear(
        m, n, k, *_product(x, x_scale, w, w_scale, out, ws, dev, (kb, m), (-(-n // 128), kb),
                           (m, n)), st)
    if rc:
        _check(rc, "dflash_fp8_linear")


def dflash_fp8_grouped(x, x_scale, w, w_scale, start, rows, out, ws, stream=None):
    """Rows start[e] .. start[e + 1] - 1 of out = x w[e]^T, w [E, N, K]; ``rows``: int32 [len(out)],
    the row of x that each row of out is made of, or None: the same row."""
    dev, st = _here(stream)
    src, k = _shape(x, 2, "x")
    e, n, kw = _shape(w, 3, "w")
    if kw != k:
        raise ValueError(f"x has {k} columns, w {kw}")
    m, kb = _shape(out, 2, "out")[0], -(-k // 128)
    if (m | src | e | n | k) >> 31:
        _past_31_bits(m, src, e, n, k)
    if rows is None and m != src:
        raise ValueError(f"out has {m} rows, x {src}: rows must say which")
    xp, xsp, wp, wsp, op, pitch, sp, size = _product(
        x, x_scale, w, w_scale, out, ws, dev, (kb, src), (e, -(-n // 128), kb), (m, n))
    rc = load_library().dflash_fp8_grouped(
        m, src, e, n, k, xp, xsp, wp, wsp, _whole(start, dev, torch.int32, (e + 1,), "start"),
        None if rows is None else _whole(rows, dev, torch.int32, (m,), "rows"), op, pitch, sp,
        size, st)
    if rc:
        _check(rc, "dflash_fp8_grouped")


def dflash_fp8_plan(rows: int, n_out: int, n_in: int, n_groups: int = 0, by_index: bool = False,
                    num_sms: int = 0):
    """(tile rows, tile features, CTAs that share a tile's n_in) of the kernel that a product of these
    sizes goes to: dflash_fp8_linear, or, of n_groups experts, dflash_fp8_grouped."""
    if max(rows, n_out, n_in, n_groups, num_sms) >> 31:
        _past_31_bits(rows, n_out, n_in, n_groups, num_sms)
    got = [ctypes.c_int32() for _ in range(3)]
    _check(load_library().dflash_fp8_plan(rows, n_groups, n_out, n_in, int(by_index), num_sms,
                                          *map(ctypes.byref, got)), "dflash_fp8_plan")
    return tuple(v.value for v in got)
