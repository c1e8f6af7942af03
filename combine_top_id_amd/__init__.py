"""MI355X-native balanced expert-parallel hot path: plan -> zero-copy dispatch ->
weighted combine -> replica-gradient reduce, and the expert block's compute around it (the
gated feed-forward experts and the norm in front of them, forward and backward), as HIP
kernels behind a C ABI (include/moonep.h, libmoonep.so), with a thin ctypes binding."""

from .moonep import (moonep_query, moonep_plan, moonep_plan_noalloc, moonep_dispatch,  # noqa: F401
                     moonep_combine,
                     moonep_reduce_grad, moonep_plan_status, moonep_dispatch_bwd,
                     moonep_combine_bwd, moonep_prefetch_weight, moonep_expert_stub,
                     moonep_dispatch_staged, moonep_combine_staged, moonep_expert_ffn,
                     moonep_expert_ffn_bwd_data, moonep_expert_ffn_bwd_weight, moonep_expert_tile, moonep_rmsnorm,
                     moonep_rmsnorm_q8, moonep_q8_row_bytes, moonep_q8_unpack,
                     moonep_rmsnorm_bwd, Plan,
                     Sizes, MoonepError, lib, LIB_PATH, EXPORTS)
