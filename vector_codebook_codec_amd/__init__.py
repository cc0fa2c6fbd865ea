"""QAM-W weight codec on AMD Instinct MI355X (gfx950).

The codec's work runs in hand-written HIP kernels behind the C ABI of
include/qamw.h (libqamw.so, built in-tree by ``_build.build()``).  This
package binds that ABI for torch device tensors; see ``codec`` for the entry
points ``qamw_calibrate``, ``qamw_encode`` and ``qamw_decode``, ``mxfp4`` for
the microscaled 4-bit format, ``cache`` for an attention cache in it, and
``cross_entropy`` for the model's loss.
"""
from .cache import (  # noqa: F401
    qamw_mxfp4_cache_attention,
    qamw_mxfp4_cache_attention_workspace_bytes,
    qamw_mxfp4_cache_new,
    qamw_mxfp4_cache_read,
    qamw_mxfp4_cache_row_bytes,
    qamw_mxfp4_cache_scale_bytes,
    qamw_mxfp4_cache_write,
)
from .codec import (  # noqa: F401
    load_codebook,
    load_polar,
    qamw_build_plan,
    qamw_calibrate,
    qamw_calibrate_encode,
    qamw_calibrate_prepare,
    qamw_calibrate_encode_workspace_bytes,
    qamw_calibrate_workspace_bytes,
    qamw_channel_rms,
    qamw_channel_rms_workspace_bytes,
    qamw_decode,
    qamw_decode_matmul,
    qamw_encode,
    qamw_encode_noalloc,
    qamw_encode_indices,
    qamw_encode_polar,
    qamw_encode_prepare,
    qamw_encode_workspace_bytes,
    qamw_index_bits,
    qamw_learn_codebook,
    qamw_lloyd_update,
    qamw_lloyd_workspace_bytes,
    qamw_output_error,
    qamw_output_error_workspace_bytes,
    qamw_packed_row_words,
    qamw_plan_bytes,
    qamw_rotate_activations,
)
from .cross_entropy import (  # noqa: F401
    qamw_cross_entropy,
    qamw_cross_entropy_grad,
    qamw_cross_entropy_grad_workspace_bytes,
    qamw_cross_entropy_workspace_bytes,
)
from .mxfp4 import (  # noqa: F401
    qamw_mxfp4_adapter_matmul,
    qamw_mxfp4_adapter_matmul_workspace_bytes,
    qamw_mxfp4_dequantize,
    qamw_mxfp4_matmul,
    qamw_mxfp4_matmul_workspace_bytes,
    qamw_mxfp4_quantize,
    qamw_mxfp4_row_bytes,
    qamw_mxfp4_scale_bytes,
)

__version__ = "0.1.0"
