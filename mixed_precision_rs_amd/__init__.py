"""MI355X-native implementation of TIDE's one-GPU hot path: the level-1
bf16 -> fp32 reduce-scatter into padded rank-major shards and the all-gather
placement into parameter storage (C ABI in include/tide.h, HIP kernels for
gfx950 in csrc/), and the training layer beside them: tokens sorted by expert
and back, 8-bit activation checkpoints, and weight gradients from them; at the
step's ends embedding, log probabilities, gradient norm and clipping, and norm
and rotation of queries and keys.
Importing this package loads libtide.so and fails loudly if it has not been
built."""
from ._lib import (  # noqa: F401
    Call,
    ENGINE_KERNEL,
    ENGINE_RUNTIME,
    ENGINE_SDMA,
    ENGINES,
    EXPORTS,
    FLAG_NO_LDS_FENCE,
    FLAG_SCALAR_PATH,
    LAUNCH_BUDGETED,
    LAUNCH_FULL,
    LIB_PATH,
    Launch,
    Plan,
    PointerTable,
    TideError,
    allgather_place,
    allgather_place_stage,
    budgeted,
    counted,
    decode_trace,
    diag_occupy,
    diag_stream,
    dma_engine_count,
    grads_table,
    landing_sum_fp32,
    landing_trace_records,
    latin_square,
    lib,
    params_table,
    plan_create,
    prepare_allgather_place,
    prepare_reduce_scatter_bf16_fp32,
    prepare_stage_grads_bf16,
    rd_schedule,
    reduce_scatter_bf16_fp32,
    reduce_scatter_bf16_fp32_noalloc,
    slot_grads_table,
    stage_grads_bf16,
    trace_buffer,
    traced,
    version,
)
from ._layer import (  # noqa: F401
    checkpoint_pack,
    checkpoint_unpack,
    combine_tokens,
    combine_tokens_grad,
    dispatch_tokens,
    gated_silu,
    gated_silu_grad,
    route_tokens,
    route_workspace_bytes,
    weight_grads_bf16,
    weight_grads_workspace_bytes,
)

from ._step import (  # noqa: F401
    TensorTable,
    clip_grads,
    embed_tokens,
    embed_tokens_grad,
    embed_tokens_grad_workspace_bytes,
    grad_squares,
    grad_squares_workspace_bytes,
    norm_rotate,
    norm_rotate_grad,
    norm_rotate_grad_workspace_bytes,
    sort_ids,
    sort_ids_workspace_bytes,
    token_logprobs,
    token_logprobs_grad,
    token_logprobs_workspace_bytes,
)

lib()  # load now: no silent fallback exists
