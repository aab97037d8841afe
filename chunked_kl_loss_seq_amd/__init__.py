"""Fused chunked KL distillation loss for MI355X (gfx950): HIP kernels behind a C ABI.

``binding`` loads libckl.so on first use and raises if it is missing;
``vocab`` has the operators around the vocabulary table (embedding,
sampling, the head's product with an 8-bit weight); ``residual`` the end of a
block before it (norms around the residual, dropout); ``logprob`` the
log-probabilities of given tokens, from logits and from hidden states;
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
from .logprob import (  # noqa: F401
    HeadLogProbs,
    LogProbs,
    head_logprobs,
    head_logprobs_bwd,
    head_logprobs_plan,
    head_token_logprobs,
    logprobs,
    logprobs_bwd,
    token_logprobs,
)
from .residual import (  # noqa: F401
    add_norm,
    add_norm_bwd,
    drop,
    dropout,
    residual_norm,
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
