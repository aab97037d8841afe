"""Fused chunked KL distillation loss for MI355X (gfx950): HIP kernels behind a C ABI.

``binding`` loads libckl.so on first use and raises if it is missing;
``vocab`` has the operators around the vocabulary table (embedding,
sampling, the head's product with an 8-bit weight);
``workloads`` draws the seeded synthetic inputs.
"""
from .binding import (  # noqa: F401
    CklError,
    bwd,
    debug_rows,
    fused_kl,
    fwd,
    fwd_bwd,
    plan,
    recompute_kl,
    release_workspace,
    timing_enable,
    topk,
    timing_query,
    workspace_bytes_held,
)
from .vocab import (  # noqa: F401
    embed,
    embed_bwd,
    embedding,
    logits_fp8,
    matmul_fp8,
    quantize_fp8,
    sample,
    teacher_topk,
)
