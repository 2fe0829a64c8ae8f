"""DP-GRAPE private update step on one AMD MI355X (gfx950).

The compute lives in libdpg.so (C ABI in include/dpg.h, HIP kernels in
csrc/); this package is its thin Python binding.
"""
from .binding import (  # noqa: F401
    DPG_BF16, DPG_FP32, DpgError, EXPORTED, GatedGrads, LayerGrad, LayerHat, LayerParam,
    PackedActivations, PreparedStep, PreparedStreamingStep, adam_workspace_size,
    dpg_adam_backproject, dpg_clip_sum_noise, dpg_distill_loss, dpg_distill_loss_grad,
    dpg_embed, dpg_embed_grad, dpg_embed_norms, dpg_gated, dpg_gated_grad, dpg_pack_act,
    dpg_philox_normals, dpg_private_step, dpg_private_step_static, dpg_project_clip_noise,
    dpg_project_layer, dpg_project_layer_packed, dpg_rc_norms, dpg_unpack_act, dpg_vocab_loss,
    dpg_vocab_loss_grad, library_path, load_library,
    project_workspace_size, static_scratch_bytes, timing_enable, timing_read, version,
)
from .feedforward import GatedFeedForward, gated_feed_forward  # noqa: F401
from .streaming import GrapeOptimizer, ProjectedLinear  # noqa: F401
from .tokens import TokenEmbedding, distill_cross_entropy, vocab_cross_entropy  # noqa: F401
