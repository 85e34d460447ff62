"""DFlash per-cycle hot path on GB300: hand-written sm_103a CUDA kernels behind a C ABI.

``libdflash.so`` holds the four calls of one draft/verify cycle (context
projection, dual-source block attention, verification epilogue, KV-cache
crop) and the calls around it: the rest of the drafter layer and its token
choice (``dflash_draft_qkv``, ``dflash_draft_mlp``, ``dflash_draft_tokens``),
the target's verify attention, the prefill (the target's attention over
prompt chunks, ``dflash_prefill_attention``, its first staged token,
``dflash_prefill_staged``, and the whole-prompt context projection,
``dflash_ctx_prefill``), the GatedDeltaNet tape-replay rollback
(``dflash_gdn_replay``) and the serving calls over a KV cache held in 4 bits
(``dflash_kv_reserve``, ``dflash_qk_norm_rope``, ``dflash_kv4_append``,
``dflash_kv4_gather``, ``dflash_kv4_attention``).  :mod:`.dflash` is the ctypes binding (argument
marshalling only); :mod:`.cycle` composes one cycle (``run_cycle``), captures
it as a CUDA graph (``CycleGraph``) and runs the serving loop with the input
copies overlapped (``PipelinedCycles``).
"""
from . import dflash  # noqa: F401
from .dflash import (DFlashError, Dims, KV4Dims, KV4View, KVView,  # noqa: F401
                     alloc_draft_workspace, alloc_kv4_cells, alloc_kv4_workspace,
                     alloc_prefill_workspace, alloc_workspace, dflash_block_attention,
                     dflash_ctx_prefill, dflash_ctx_project, dflash_cycle_sm_split,
                     dflash_draft_mlp, dflash_draft_qkv, dflash_draft_tokens, dflash_gdn_replay,
                     dflash_kv4_append, dflash_kv4_attention, dflash_kv4_gather,
                     dflash_kv4_workspace_bytes, dflash_kv_crop, dflash_kv_reserve,
                     dflash_prefill_attention, dflash_prefill_staged, dflash_qk_norm_rope,
                     dflash_read_status, dflash_verify_accept,
                     dflash_verify_attention, dflash_workspace_bytes, dflash_workspace_init,
                     load_library, make_dims, make_kv4_dims, with_sm_budget)
