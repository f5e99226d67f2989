"""B200-native binary convolution (XNOR / AND / binaryWeights) behind a C-ABI library.

This package is a thin ctypes binding over ``libbconv.so`` (built in-tree by
``python -m binarized_convolution_b200.build``).  The functions named like the C entry
points (``bconv_create``, ``bconv_forward``, ``bfc_create``, ...) only marshal arguments;
every step of the computation runs in the library's CUDA kernels.  PyTorch supplies device
memory and the current CUDA stream in the convenience classes :class:`BinaryConv2d` and
:class:`BinaryFC`, and for the operators around low-bit layers of a language model:
:class:`QuantFC` (4-bit weights), :func:`block_norm` and :func:`token_logprobs` with their
gradients.

There is no CPU fallback: if the library is missing or no CUDA device is visible, the calls
raise.
"""
from __future__ import annotations

from ._native import (  # noqa: F401
    ALGO_AUTO,
    ALGO_POPC,
    ALGO_SIMT_F32,
    ALGO_TCGEN05,
    CODES_AUTO,
    CODES_BF16X3,
    CODES_FP4,
    CODES_INT8,
    CTA_AUTO,
    CTA_PAIR,
    CTA_SINGLE,
    DTYPE_BF16,
    DTYPE_F16,
    DTYPE_F32,
    STAGING_AUTO,
    STAGING_PER_TAP,
    STAGING_ROWS,
    STAGING_INPUT,
    FLAG_NONE,
    FLAG_USE_BETA_SCALING,
    NEURON_NONE,
    NEURON_RELU,
    TYPE_AND,
    TYPE_BINARY_WEIGHTS,
    TYPE_XNOR,
    BconvError,
    bconv_block_norm_backward,
    bconv_block_norm_desc_t,
    bconv_block_norm_forward,
    bconv_block_norm_sync_status,
    bconv_block_norm_workspace_bytes,
    bconv_create,
    bconv_cta_mode,
    bconv_set_cta_mode,
    bconv_set_tc_codes,
    bconv_tc_codes,
    bconv_set_staging,
    bconv_staging,
    bconv_desc_t,
    bconv_destroy,
    bconv_effective_algo,
    bconv_forward,
    bconv_forward_host,
    bconv_forward_noalloc,
    bconv_forward_io,
    bconv_check_wait_timeout,
    bconv_set_output_terms,
    bconv_io_t,
    bfc_forward_io,
    bfc_set_output_terms,
    NOALLOC_SCRATCH_BYTES,
    bconv_get_output_dims,
    bconv_input_feature_channels,
    bconv_launches_per_forward,
    bconv_measure_peak,
    bconv_output_feature_channels,
    bconv_pack_bits,
    bconv_profile_begin,
    bconv_profile_end,
    bconv_profile_stride,
    bconv_set_algo,
    bconv_status_string,
    bconv_sync_status,
    bconv_token_desc_t,
    bconv_token_logprobs_backward,
    bconv_token_logprobs_forward,
    bconv_version,
    bfc_create,
    bfc_cta_mode,
    bfc_tc_codes,
    bfc_desc_t,
    bfc_destroy,
    bfc_effective_algo,
    bfc_forward,
    bfc_forward_host,
    bfc_input_feature_channels,
    bfc_launches_per_forward,
    bfc_output_feature_channels,
    bfc_profile_begin,
    bfc_profile_end,
    bfc_profile_stride,
    bfc_quant_create,
    bfc_quant_desc_t,
    bfc_quant_destroy,
    bfc_quant_forward,
    bfc_quant_input_feature_channels,
    bfc_quant_output_feature_channels,
    bfc_quant_sync_status,
    bfc_quant_workspace_bytes,
    bfc_set_algo,
    bfc_sync_status,
    exported_symbols,
    library_path,
    load_library,
)
from .layers import BinaryConv2d, BinaryFC  # noqa: F401


_LM_OPS = ("QuantFC", "BlockNorm", "BlockNormGrad", "TokenLogprobs", "block_norm", "block_norm_backward",
           "token_logprobs", "token_logprobs_backward")


def __getattr__(name):
    # (the module of these needs torch at import; the C binding above does not)
    if name in _LM_OPS:
        from . import lm_ops

        for n in _LM_OPS:
            globals()[n] = getattr(lm_ops, n)
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
