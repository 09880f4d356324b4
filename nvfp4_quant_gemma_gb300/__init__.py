"""GB300-native fused Gemma add-RMSNorm + FP8 / NVFP4 input quantization, and
the operators around the NVFP4 linear that follows it.

The compute path is the sm_103a library ``libgemma_nq.so`` (C ABI declared in
``include/gemma_nq.h``); the functions below are its thin Python binding.
Importing the package does not load the library; the first call does, and
raises if the library has not been built."""
from ._binding import (  # noqa: F401
    add_rms_norm_quant,
    alloc_outputs,
    encode_e4m3_e2m1,
    expert_combine,
    expert_dequantize,
    expert_quantize,
    expert_route,
    expert_scale_rows,
    gated_act_quant,
    gemma_add_rms_norm,
    gemma_add_rms_norm_quant,
    gemma_add_rms_norm_quant_parts,
    gemma_sandwich_norm_quant,
    inject_split_timeout,
    inject_wait_timeout,
    library_path,
    nvfp4_dequantize,
    nvfp4_expert_linear,
    nvfp4_linear,
    quantize,
    quantize_fp8_values,
    read_device_error,
    load,
    pdl_consumer,
    query_launch,
    query_linear,
    set_launch_policy,
    set_linear_policy,
    set_constant_weights,
    set_pdl,
    status_string,
)
