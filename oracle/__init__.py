"""CPU oracle for the NVFP4 block-scaled GEMM (test infrastructure only).

Only tests, ``__graft_entry__.smoke()`` and the ``cpu_baseline`` leg of
``bench.py`` may import this package; the HIP library never does.
"""
from .nvfp4_ref import (  # noqa: F401
    E2M1_MAGNITUDES, E2M1_TABLE, E4M3_MAX, GLOBAL_DIVISOR, REL_TOL,
    check_gemm, dequantize_ref, e2m1_decode, e4m3_decode, gemm_ref,
    global_scale_ref, grouped_gemm_ref, pack_nibbles, quantize_ref,
    tolerance, ulp_bf16, unpack_nibbles,
)
from .mxfp4_ref import (  # noqa: F401
    MX_BLOCK, e8m0_decode, mxfp4_dequantize_ref, mxfp4_gemm_ref, mxfp4_quantize_ref,
)
from .fp8_ref import (  # noqa: F401
    E4M3_TABLE, FP8_BLOCK, e4m3_encode, fp8_dequantize_ref, fp8_gemm_ref, fp8_grouped_columns_ref,
    fp8_grouped_quantize_t_ref, fp8_quantize_ref, fp8_quantize_t_ref, fp8_tolerance,
    moe_route_backward_ref, moe_route_ref,
)
from .feed_forward_ref import (  # noqa: F401
    act_error, act_ref, clip_ref, gated_backward_ref, gated_ref, gated_tolerance, int8_gemm_ref,
    int8_quantize_ref, sums_tolerance,
)
