"""MI355X-native chunkwise TTT fast-weight layer (HIP, gfx950) and In-Place TTT update.

The compute lives in ``libttt.so`` (C ABI in ``include/ttt.h``); this package
is its ctypes binding (``binding``), device plumbing (``layer``), seeded
synthetic workloads (``workloads``) and the build script (``build``).
"""
from .binding import (ENTRY_BWD, ENTRY_FWD, EXPORTS, Act, Decay, DType, Loss, Status, TTTDesc,
                      Gate, RecInput, TTTError, TTTLnDesc, TTTMlpDesc, TTTRecDesc, make_ln_desc, make_mlp_desc, make_rec_desc,
                      ttt_layernorm_bwd, ttt_layernorm_fwd, ttt_layernorm_workspace_size, ttt_recurrence_bwd,
                      ttt_recurrence_fwd, ttt_recurrence_saved_size, ttt_recurrence_step, ttt_recurrence_workspace_size, ttt_mlp_bwd_workspace_size, ttt_mlp_chunk_bwd, ttt_mlp_chunk_fwd, ttt_mlp_saved_size,
                      ttt_mlp_workspace_size, inplace_ttt_bwd, inplace_ttt_bwd_workspace_size, inplace_ttt_fwd, inplace_ttt_fwd_guarded,
                      inplace_ttt_guarded_workspace_size,
                      inplace_ttt_workspace_size, lib, make_desc, ttt_chunk_bwd, ttt_chunk_fwd,
                      ttt_last_error, ttt_saved_size, ttt_version, ttt_workspace_size,
                      HeadNorm, RopePairs, TTTDeltaDesc, TTTQkNormDesc, make_delta_desc, make_qknorm_desc, ttt_delta_bwd,
                      ttt_delta_fwd, ttt_delta_saved_size, ttt_delta_step, ttt_delta_workspace_size, ttt_qknorm_bwd,
                      ttt_qknorm_fwd, ttt_qknorm_workspace_size)

__all__ = ["ENTRY_BWD", "ENTRY_FWD", "EXPORTS", "Act", "Decay", "DType", "Loss", "Status", "TTTDesc",
           "Gate", "RecInput", "TTTError", "TTTLnDesc", "TTTMlpDesc", "TTTRecDesc", "make_ln_desc", "make_rec_desc",
           "ttt_layernorm_bwd", "ttt_layernorm_fwd", "ttt_layernorm_workspace_size", "ttt_recurrence_bwd",
           "ttt_recurrence_fwd", "ttt_recurrence_saved_size", "ttt_recurrence_step", "ttt_recurrence_workspace_size",
           "make_mlp_desc", "ttt_mlp_bwd_workspace_size", "ttt_mlp_chunk_bwd",
           "ttt_mlp_chunk_fwd", "ttt_mlp_saved_size", "ttt_mlp_workspace_size",
           "inplace_ttt_bwd", "inplace_ttt_bwd_workspace_size", "inplace_ttt_fwd", "inplace_ttt_fwd_guarded",
           "inplace_ttt_guarded_workspace_size", "inplace_ttt_workspace_size", "lib", "make_desc", "ttt_chunk_bwd", "ttt_chunk_fwd",
           "ttt_last_error", "ttt_saved_size", "ttt_version", "ttt_workspace_size",
           "HeadNorm", "RopePairs", "TTTDeltaDesc", "TTTQkNormDesc", "make_delta_desc", "make_qknorm_desc", "ttt_delta_bwd",
           "ttt_delta_fwd", "ttt_delta_saved_size", "ttt_delta_step", "ttt_delta_workspace_size", "ttt_qknorm_bwd",
           "ttt_qknorm_fwd", "ttt_qknorm_workspace_size"]
