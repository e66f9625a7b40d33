// Host-side launchers shared between the C ABI (api.cpp) and the kernel files.
// Every launcher assumes its arguments were validated by api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stddef.h>

namespace nvfp4 {

// quantize.hip
size_t quantize_workspace_bytes(int64_t rows, int64_t cols);
hipError_t launch_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x,
                           uint8_t* q, uint8_t* s, float* gscale, bool scale_given,
                           void* workspace, hipStream_t stream);
// The library's own quantise workspace (a device array, one per GPU): its
// size in bytes, and its address on the current device (found once per
// device with hipGetSymbolAddress).
size_t quantize_scratch_bytes();
hipError_t quantize_scratch(void** ptr);

// Operand description of one packed NVFP4 matrix [rows, K].
struct PackedOperand {
  const uint8_t* q;  // [rows, K/2]
  const uint8_t* s;  // [rows, K/16]
  const float* g;    // device scalar (or [G] for grouped weights)
};

// NVFP4 output of a dense GEMM (y_dtype 2): y quantised with the given
// global scale *g (device fp32) into q [M, N/2] and s [M, N/16] (row-major,
// contiguous, N % 16 == 0, q 8-byte aligned), from the same fp32 values
// y_dtype 0 would store.
struct QuantOut {
  uint8_t* q;
  uint8_t* s;
  const float* g;
};

// gemm_generic.hip: any M, N, K % 16 == 0.
hipError_t launch_gemm_generic(int64_t M, int64_t N, int64_t K, PackedOperand a,
                               PackedOperand b, void* y, int y_dtype, int64_t ld_y,
                               hipStream_t stream, QuantOut qo = {});

// row_index (nullptr: none): grouped row r reads activation row row_index[r]
// of the a_rows rows of `a`; an index outside [0, a_rows) reads as zeros.
hipError_t launch_gemm_grouped_generic(int32_t G, const int32_t* m_offsets,
                                       const int32_t* row_index, int64_t total_m, int64_t a_rows,
                                       int64_t N, int64_t K, PackedOperand a, PackedOperand b,
                                       void* y, int y_dtype, int64_t ld_y, hipStream_t stream);

// mxfp4.hip: MXFP4 conversion (cols % 32 == 0, 16-byte aligned x rows and
// q) and the general MXFP4 GEMM (any M, N, K % 32 == 0).
hipError_t launch_mx_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x,
                              uint8_t* q, uint8_t* s, hipStream_t stream);
hipError_t launch_mx_gemm_generic(int64_t M, int64_t N, int64_t K, const uint8_t* a_q,
                                  const uint8_t* a_s, const uint8_t* b_q, const uint8_t* b_s,
                                  void* y, int y_dtype, int64_t ld_y, hipStream_t stream);
// gemm_mfma.hip: MXFP4 on the scaled FP4 matrix instruction; K % 128 == 0,
// 16-byte aligned nibble rows, 4-byte aligned scale rows.
hipError_t launch_gemm_mx_mfma(int64_t M, int64_t N, int64_t K, const uint8_t* a_q,
                               const uint8_t* a_s, const uint8_t* b_q, const uint8_t* b_s,
                               void* y, int y_dtype, int64_t ld_y, hipStream_t stream);

// gemm_mfma.hip: K % 128 == 0, 16-byte aligned operand rows.
hipError_t launch_gemm_mfma(int64_t M, int64_t N, int64_t K, PackedOperand a,
                            PackedOperand b, void* y, int y_dtype, int64_t ld_y,
                            hipStream_t stream, QuantOut qo = {});

// gemm_decode_lds.hip: M <= 32, K % 1024 == 0, 16-byte aligned nibble and
// scale bases, both operands' bytes < 4 GiB.
hipError_t launch_gemm_decode_lds(int64_t M, int64_t N, int64_t K, PackedOperand a,
                                  PackedOperand b, void* y, int y_dtype, int64_t ld_y,
                                  hipStream_t stream, QuantOut qo = {});

// gemm_decode_rows.hip: whole-row weight stream for the shapes
// decode_rows_shape (nvfp4_dispatch.h) accepts, fp32 / bf16 output only;
// 16-byte aligned nibble and scale bases, both operands' bytes < 4 GiB.
hipError_t launch_gemm_decode_rows(int64_t M, int64_t N, int64_t K, PackedOperand a,
                                   PackedOperand b, void* y, int y_dtype, int64_t ld_y,
                                   hipStream_t stream);

// gemm_skinny.hip: M <= 128 (decode; 64-row passes), K % 256 == 0, N * K / 2 < 4 GiB.
hipError_t launch_gemm_decode(int64_t M, int64_t N, int64_t K, PackedOperand a,
                              PackedOperand b, void* y, int y_dtype, int64_t ld_y,
                              hipStream_t stream, QuantOut qo = {});

// One grouped GEMM of a launch (row_index as above; a_rows is used only with
// a row_index).
struct GroupedProblem {
  int32_t G;
  const int32_t* m_offsets;
  const int32_t* row_index;
  int64_t total_m, a_rows, N, K;
  PackedOperand a, b;
  void* y;
  int y_dtype;
  int64_t ld_y;
};
constexpr int kGroupedMaxProblems = 4;  // = NVFP4_GROUPED_MAX_PROBLEMS

// gemm_grouped.hip: 1..kGroupedMaxProblems problems in one persistent launch,
// each with K % 512 == 0 and operands < 4 GiB.
hipError_t launch_gemm_grouped_multi(int count, const GroupedProblem* probs, hipStream_t stream);
// The streaming grouped kernel numbers its work units with 32-bit ints:
// true when a problem of this size fits.
bool grouped_units_fit(int64_t G, int64_t total_m, int64_t N);

// gemm_grouped.hip: K % 512 == 0, operands < 4 GiB; row_index as above.
hipError_t launch_gemm_grouped(int32_t G, const int32_t* m_offsets, const int32_t* row_index,
                               int64_t total_m, int64_t a_rows, int64_t N, int64_t K,
                               PackedOperand a, PackedOperand b, void* y, int y_dtype,
                               int64_t ld_y, hipStream_t stream);

// FP8 block-128 operand [rows, K] and output (fp8_gemm.hip).
struct Fp8Operand {
  const uint8_t* q;  // E4M3 bytes [rows, K]
  const float* s;    // [ceil(K / 128), ceil(rows / block_rows)]
};
struct Fp8Out {
  void* y;
  int64_t ld;  // elements
  int dtype;   // 0 fp32, 1 bf16
  bool add;    // fp32 only: y += product
  bool vec;    // rows start on 16-byte borders
};

// Whether a launch's threads fit the 32-bit count of a grid's dimension.  The
// FP8 launchers answer hipErrorNotSupported where they do not, before any
// other call.
inline bool grid_fits(int64_t blocks, int64_t threads) { return blocks <= 0xFFFFFFFFll / threads; }

// Columns of an expert-wise transposed operand: total_m tokens of G experts,
// each expert's starting on a border of 128 (an upper bound known on the
// host; the experts' counts are not).
inline int64_t fp8_padded_tokens(int64_t total_m, int64_t G) {
  const int64_t g = G < total_m ? G : total_m;
  return (total_m + 127 * g) / 128 * 128;
}

// fp8_quantize.hip: rows layout q/s and transposed layout qt/st (either may
// be null).
hipError_t launch_fp8_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols,
                               int64_t ld_x, int block_rows, uint8_t* q, float* s, uint8_t* qt,
                               float* st, hipStream_t stream);
hipError_t launch_fp8_grouped_quantize(const void* x, int dtype, int32_t G,
                                       const int32_t* m_offsets, const int32_t* row_index,
                                       int64_t total_m, int64_t x_rows, int64_t cols, int64_t ld_x,
                                       uint8_t* q, float* s, uint8_t* qt, float* st,
                                       hipStream_t stream);
// fp8_gemm.hip: K % 16 == 0, K <= 2^22, 16-byte aligned q.
hipError_t launch_fp8_gemm(int64_t M, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b,
                           int b_block_rows, Fp8Out y, hipStream_t stream);
// fp8_stream.hip: the same for few rows or few outputs, and which those are.
bool fp8_streams(int64_t M, int64_t N);
hipError_t launch_fp8_stream(int64_t M, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b,
                             int b_block_rows, Fp8Out y, hipStream_t stream);
// row_index != nullptr: a_rows * K < 2^31
bool fp8_grouped_streams(int64_t G, int64_t total_m, int64_t N, int64_t K);
hipError_t launch_fp8_grouped_stream(int32_t G, const int32_t* m_offsets, const int32_t* row_index,
                                     int64_t total_m, int64_t a_rows, int64_t N, int64_t K,
                                     Fp8Operand a, Fp8Operand b, Fp8Out y, hipStream_t stream);
hipError_t launch_fp8_grouped(int32_t G, const int32_t* m_offsets, const int32_t* row_index,
                              int64_t total_m, int64_t a_rows, int64_t N, int64_t K, Fp8Operand a,
                              Fp8Operand b, Fp8Out y, hipStream_t stream);
// P: columns of the transposed operands (fp8_padded_tokens)
hipError_t launch_fp8_wgrad(int32_t G, const int32_t* m_offsets, int64_t total_m, int64_t P,
                            int64_t N, int64_t K, Fp8Operand a, Fp8Operand b, Fp8Out y,
                            hipStream_t stream);

// moe_route.hip
struct RouteOut {
  int32_t* expert_index;  // [T, k]
  float* weights;         // [T, k]
  int32_t* counts;        // [E]
  int32_t* m_offsets;     // [E + 1]
  int32_t* row_index;     // [T * k]
  int32_t* pair_row;      // [T, k]
  int32_t* routed;        // [1]
  float* loss;            // [1]
};
size_t moe_route_workspace_bytes(int64_t T, int64_t E);
hipError_t launch_moe_route(int64_t T, int64_t E, int topk, const void* logits, int dtype,
                            int64_t ld, const uint8_t* mask, bool renorm, RouteOut out,
                            void* workspace, hipStream_t stream);
hipError_t launch_moe_route_backward(int64_t T, int64_t E, int topk, const void* logits, int dtype,
                                     int64_t ld, const uint8_t* mask, bool renorm,
                                     const int32_t* expert_index, const int32_t* counts,
                                     const int32_t* routed, const float* d_weights,
                                     const float* d_loss, void* d_logits, int64_t ld_d,
                                     hipStream_t stream);

}  // namespace nvfp4
