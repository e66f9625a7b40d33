"""MI355X (gfx950) NVFP4 block-scaled GEMM: y = x . W^T with E2M1 operands,
E4M3FN scales per 16 elements and fp32 per-tensor global scales; MXFP4 and
FP8 (E4M3, one fp32 scale per 128) variants, grouped products for experts and
the router that orders their tokens.

The computation lives in ``libnvfp4.so`` (HIP kernels + C ABI, declared in
``include/nvfp4.h``); this package only marshals torch tensors into it.
"""
from ._lib import (  # noqa: F401
    EXPORTED, LIB_PATH, NVFP4_BF16, NVFP4_GROUPED_MAX_PROBLEMS, GroupedProblem, NVFP4_ERR_HIP, NVFP4_ERR_INVALID_ARG,
    NVFP4_ERR_UNSUPPORTED, NVFP4_F32, NVFP4_GLOBAL_SCALE_GIVEN, NVFP4_OK, Nvfp4Error,
    Packed, load, nvfp4_gemm, nvfp4_gemm_nvfp4_out, nvfp4_gemm_nvfp4_out_raw, nvfp4_gemm_raw,
    nvfp4_grouped_gemm, nvfp4_grouped_gemm_gather_raw, nvfp4_grouped_gemm_multi,
    nvfp4_grouped_gemm_multi_raw, nvfp4_grouped_gemm_raw, nvfp4_mxfp4_gemm,
    nvfp4_mxfp4_gemm_raw, nvfp4_mxfp4_quantize, nvfp4_mxfp4_quantize_raw,
    nvfp4_quantize, nvfp4_quantize_noalloc_raw, nvfp4_quantize_raw, nvfp4_quantize_workspace_bytes,
    Fp8Packed, MoeRoute, NVFP4_ACCUMULATE, NVFP4_ROUTE_RENORMALIZE, nvfp4_fp8_gemm,
    nvfp4_fp8_gemm_raw, nvfp4_fp8_grouped_columns, nvfp4_fp8_grouped_gemm,
    nvfp4_fp8_grouped_gemm_raw, nvfp4_fp8_grouped_quantize, nvfp4_fp8_grouped_quantize_raw,
    nvfp4_fp8_grouped_wgrad, nvfp4_fp8_grouped_wgrad_raw, nvfp4_fp8_quantize,
    nvfp4_fp8_quantize_raw, nvfp4_moe_route, nvfp4_moe_route_backward,
    nvfp4_moe_route_backward_raw, nvfp4_moe_route_raw, nvfp4_moe_route_workspace_bytes,
)
