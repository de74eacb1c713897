"""gated_delta_rule_29_gb300 -- GB300-native (sm_103a) chunked Gated DeltaNet forward.

The computation lives in liblinattn.so (C ABI: include/liblinattn.h), built
in-tree from csrc/ by ``_build.build()``.  This package is its thin Python
binding: ``gdn_fwd``, ``gdn_bwd``, ``gdn_summary``, ``gdn_summary_bwd`` and ``gdn_decode`` marshal torch tensors
into the C structs and launch on the current CUDA stream.  Around the recurrence, the
token-mixer operators: ``glr_*`` (gated linear recurrence), ``gn_*`` (per-head group norm with an
activation or gate) and ``sconv_*`` (short causal convolution), with their autograd forms
``gated_linear_recurrence``, ``group_norm`` and ``short_conv``.  There is no CPU fallback.
"""
from .api import (checkpoint_rows, gdn_bwd, gdn_decode, gdn_fwd, gdn_fwd_host, gdn_summary,  # noqa: F401
                  gdn_summary_bwd, read_status, workspace_bytes)
from . import binding  # noqa: F401
from .autograd import gdn_attention  # noqa: F401
from .mixer import (gated_linear_recurrence, glr_bwd, glr_checkpoint_rows, glr_decode, glr_fwd, gn_bwd,  # noqa: F401
                    gn_fwd, group_norm, sconv_bwd, sconv_decode, sconv_fwd, short_conv)

__all__ = ["gdn_fwd", "gdn_fwd_host", "gdn_summary", "gdn_summary_bwd", "gdn_decode", "gdn_bwd", "gdn_attention",
           "read_status", "checkpoint_rows", "workspace_bytes", "binding", "glr_fwd", "glr_bwd", "glr_decode",
           "glr_checkpoint_rows", "gated_linear_recurrence", "gn_fwd", "gn_bwd", "group_norm", "sconv_fwd",
           "sconv_bwd", "sconv_decode", "short_conv"]
