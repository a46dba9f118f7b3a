"""MI355X-native fused linear cross-entropy (FLCE).

The lm_head projection of hidden states onto the vocabulary, fused with the
cross-entropy loss, the token-accuracy argmax and the backward pass, without
ever materialising the [tokens, vocab] logits (Liger-Kernel "Muse Glimmer" and
"DeepSeek-V3" commit pages, Summary and Memory sections).  All computation runs
in the HIP kernels of ``libflce.so``; this package only marshals arguments and
uses PyTorch for device memory and streams.
"""
from __future__ import annotations

from ._lib import (  # noqa: F401
    EXPORTED,
    FLCE_DTYPE_BF16,
    FLCE_DTYPE_F32,
    FLCE_DTYPE_MX8,
    FLCE_EDEVICE,
    FLCE_EINVAL,
    FLCE_ELABEL,
    FLCE_ESCRATCH,
    FLCE_EUNSUPPORTED,
    FLCE_EWORKSPACE,
    FLCE_OK,
    FLCE_REDUCTION_MEAN,
    FLCE_REDUCTION_NONE,
    FLCE_REDUCTION_SUM,
    KERNEL_KINDS,
    NOALLOC_SCRATCH_BYTES,
    WS_N_VALID_OFFSET,
    FlceError,
    flce_cross_entropy,
    flce_cross_entropy_workspace_size,
    flce_dropout,
    flce_fwd,
    flce_fwd_bwd,
    flce_fwd_bwd_ex,
    flce_fwd_bwd_noalloc,
    flce_fwd_workspace_size,
    flce_layer_norm_bwd,
    flce_layer_norm_bwd_workspace_size,
    flce_layer_norm_fwd,
    flce_logits,
    flce_logits_mx,
    flce_options_t,
    flce_pack_mx,
    flce_profile_enable,
    flce_profile_read,
    flce_plan,
    flce_read_status,
    flce_rms_norm_bwd,
    flce_rms_norm_bwd_workspace_size,
    flce_rms_norm_fwd,
    flce_rms_norm_mx,
    flce_sample,
    flce_sample_params_t,
    flce_sample_workspace_size,
    flce_scale_grads,
    flce_strerror,
    flce_workspace_size,
)
from .head import (  # noqa: F401
    LayerNormForward,
    LayerNormGrads,
    RmsNormForward,
    RmsNormGrads,
    RmsNormMx8,
    SampleOutputs,
    dropout,
    layer_norm,
    layer_norm_bwd,
    layer_norm_fwd,
    lm_head_loss,
    lm_head_sample,
    rms_norm,
    rms_norm_bwd,
    rms_norm_fwd,
    rms_norm_mx8,
    sample,
)
from .mx import Mx4Weight, Mx8Rows, logits_mx4, mx4_pack  # noqa: F401
from .torch_api import (  # noqa: F401
    CrossEntropyOutputs,
    FlceForward,
    FlceOutputs,
    cross_entropy,
    forward,
    fwd_bwd,
    linear_cross_entropy,
    logits,
    read_status,
    scale_grads,
    token_accuracy,
)
