"""libspecverify: batched speculative-decoding verification on MI355X (gfx950).

The HIP library (``libspecverify.so``, C ABI in ``include/specverify.h``) does
all of the work; ``binding`` marshals torch tensors into it: ``verify`` (one
verification step), ``sample`` (draws from processed distributions, e.g. the
draft model's), ``acceptance_rates`` (per-position sum_x min(p, q)),
``round_stats`` and ``DraftLengthMonitor`` (round statistics and the adaptive
draft length, on the device).

``libspecverify_ops.so`` (``include/specverify_ops.h``, bound in ``ops``) holds
the operators around that step: ``verify_probs`` (the verification from given
probabilities), ``hidden_norm`` (the norms before the LM head) and the LM head
on 8-bit floats (``quantize_fp8``, ``pack_fp8_lm_head``, ``fp8_lm_head``,
``verify_fp8_lm_head``).
"""

from .binding import (  # noqa: F401
    TOTAL_FIELDS,
    DraftLengthMonitor,
    acceptance_rates,
    round_stats,
    sample,
    PATH_BONUS,
    PATH_EOS,
    PATH_ERROR,
    PATH_REJECT,
    SpecVerifyError,
    library_path,
    load_library,
    status_string,
    verify,
    workspace_bytes,
)
from .ops import (  # noqa: F401
    PackedFp8LmHead,
    fp8_lm_head,
    hidden_norm,
    load_ops_library,
    ops_library_path,
    pack_fp8_lm_head,
    quantize_fp8,
    verify_fp8_lm_head,
    verify_probs,
)
