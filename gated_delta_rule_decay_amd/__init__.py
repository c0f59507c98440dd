"""gated_delta_rule_decay_amd: the gated delta rule-2 (GDN-2) token mixer on MI355X.

The compute path is a HIP library for gfx950 (``libgdn2.so``, C ABI declared
in ``include/gdn2.h``): a chunkwise-parallel forward and an O(1)-memory
recurrent decode step, plus the chunkwise backward, both also over packed
sequences.  ``chunk_fwd``, ``chunk_fwd_static`` (no allocation: the
library's static scratch), ``chunk_fwd_varlen``, ``chunk_bwd``,
``chunk_bwd_varlen`` and ``recurrent_step`` below only
marshal torch tensors into that ABI, as do linear attention with a decay
for each head (``linear_chunk_fwd``, ``linear_chunk_bwd``, their packed
forms and ``linear_recurrent_step``), layer norm (``layer_norm_fwd``,
``layer_norm_bwd``), rotary positions and the norms of queries and keys
(``rotary_fwd``, ``qk_norm_rotary_fwd`` and their backward calls) and the
gated scan over channels (``gated_scan_fwd``, ``gated_scan_bwd``, their
packed forms and ``gated_scan_step``); importing this package does not load
the library, calling either function does (and fails loudly if it is not
built).
"""
from .binding import (chunk_fwd, chunk_fwd_static, chunk_fwd_varlen, chunk_bwd, chunk_bwd_varlen, recurrent_step,  # noqa: F401
                      chunk_fwd_workspace, chunk_fwd_varlen_workspace, chunk_bwd_workspace,
                      chunk_bwd_varlen_workspace, library_path, abi_version)
from .linear import (linear_chunk_fwd, linear_chunk_fwd_varlen, linear_chunk_bwd, linear_chunk_bwd_varlen,  # noqa: F401
                     linear_recurrent_step, layer_norm_fwd, layer_norm_bwd, linear_chunk_fwd_workspace,
                     linear_chunk_fwd_varlen_workspace, linear_chunk_bwd_workspace, linear_chunk_bwd_varlen_workspace,
                     layer_norm_bwd_workspace)
from .rotary import (rotary_frequencies, rotary_fwd, rotary_bwd, qk_norm_rotary_fwd, qk_norm_rotary_bwd,  # noqa: F401
                     qk_norm_rotary_bwd_workspace)
from .scan import (gated_scan_fwd, gated_scan_fwd_varlen, gated_scan_bwd, gated_scan_bwd_varlen, gated_scan_step,  # noqa: F401
                   gated_scan_fwd_workspace, gated_scan_fwd_varlen_workspace, gated_scan_bwd_workspace,
                   gated_scan_bwd_varlen_workspace)

__all__ = ["chunk_fwd", "chunk_fwd_static", "chunk_fwd_varlen", "chunk_bwd", "chunk_bwd_varlen", "recurrent_step",
           "chunk_fwd_workspace", "chunk_fwd_varlen_workspace", "chunk_bwd_workspace",
           "chunk_bwd_varlen_workspace", "library_path", "abi_version",
           "linear_chunk_fwd", "linear_chunk_fwd_varlen", "linear_chunk_bwd", "linear_chunk_bwd_varlen",
           "linear_recurrent_step", "layer_norm_fwd", "layer_norm_bwd", "linear_chunk_fwd_workspace",
           "linear_chunk_fwd_varlen_workspace", "linear_chunk_bwd_workspace", "linear_chunk_bwd_varlen_workspace",
           "layer_norm_bwd_workspace",
           "rotary_frequencies", "rotary_fwd", "rotary_bwd", "qk_norm_rotary_fwd", "qk_norm_rotary_bwd",
           "qk_norm_rotary_bwd_workspace",
           "gated_scan_fwd", "gated_scan_fwd_varlen", "gated_scan_bwd", "gated_scan_bwd_varlen", "gated_scan_step",
           "gated_scan_fwd_workspace", "gated_scan_fwd_varlen_workspace", "gated_scan_bwd_workspace",
           "gated_scan_bwd_varlen_workspace"]
