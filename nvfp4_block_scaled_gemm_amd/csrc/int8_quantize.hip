// INT8 quantiser: x (fp32 | bf16) -> 8-bit integers and one fp32 scale per row,
//
//   A   = max(max |x_i|, 2^-100)         (a zero row gets a tiny scale)
//   s   = fl32(A / 127),  r = fl32(127 / A)
//   q_i = fl32(x_i * r) to the nearest integer, ties to even
//
// |q_i| <= 127.  A row that holds a NaN or an infinity gets a NaN scale and
// zero bytes.  Bound by HBM: one read and one write.  A row is held in
// registers between its maximum and its integers, by a wave up to 2048 columns
// and by a workgroup of four or sixteen waves up to 32768; a longer row is read
// twice, the second time mostly from a cache.
#include "fp8_quant_tile.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

using namespace fp8;

struct RowScale {
  float s, r;
  bool finite;
};
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  const bool finite = amax_bits < kInf;
  const float a = finite ? fmaxf(__uint_as_float(amax_bits), kTiny) : 1.0f;
  return {finite ? a / 127.0f : __uint_as_float(0x7FC00000u), 127.0f / a, finite};
}

__device__ __forceinline__ uint32_t pack4(const float* v, float r) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) w |= ((uint32_t)(int)__builtin_rintf(v[e] * r) & 0xFFu) << (8 * e);
  return w;
}

__device__ __forceinline__ void put8(int8_t* q, const float* v, const RowScale& s) {
  const u32x2 w = s.finite ? u32x2{pack4(v, s.r), pack4(v + 4, s.r)} : u32x2{0, 0};
  *reinterpret_cast<u32x2*>(q) = w;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
  m = max16(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  return max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
}

// Largest over a row's WAVES waves (one workgroup if more than one).
template <int WAVES>
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
  m = wave_max(m);
  if constexpr (WAVES > 1) {
    __shared__ uint32_t part[WAVES];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w) m = max(m, part[w]);
  }
  return m;
}

// Rows of up to 512 * WAVES * CHUNKS columns, WAVES waves a row, eight columns a
// lane and chunk; four rows a workgroup of single waves.
template <int DT, int WAVES, int CHUNKS>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void int8_rows_kernel(
    const void* __restrict__ x, int64_t rows, int64_t cols, int64_t ld_x, int8_t* __restrict__ q,
    float* __restrict__ s) {
  const int64_t row = WAVES == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (row >= rows) return;
  const int t = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  float v[CHUNKS][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const int64_t c = (int64_t)(i * 64 * WAVES + t) * 8;
    if (c < cols) {
      load8<DT>(x, row * ld_x + c, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) m = max(m, amax8(v[i]));
  const RowScale sc = row_scale(row_max<WAVES>(m));
  if (t == 0) s[row] = sc.s;
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const int64_t c = (int64_t)(i * 64 * WAVES + t) * 8;
    if (c < cols) put8(q + row * cols + c, v[i], sc);
  }
}

// Longer rows, one workgroup of sixteen waves each, read twice.
template <int DT>
__global__ __launch_bounds__(1024) void int8_long_rows_kernel(const void* __restrict__ x, int64_t cols, int64_t ld_x,
                                                              int8_t* __restrict__ q, float* __restrict__ s) {
  const int64_t row = blockIdx.x;
  float v[8];
  uint32_t m = 0;
  for (int64_t c = threadIdx.x * 8; c < cols; c += 8192) {
    load8<DT>(x, row * ld_x + c, v);
    m = max(m, amax8(v));
  }
  const RowScale sc = row_scale(row_max<16>(m));
  if (threadIdx.x == 0) s[row] = sc.s;
  for (int64_t c = threadIdx.x * 8; c < cols; c += 8192) {
    load8<DT>(x, row * ld_x + c, v);
    put8(q + row * cols + c, v, sc);
  }
}

template <int DT, int WAVES, int CHUNKS>
hipError_t rows_cfg(const void* x, int64_t rows, int64_t cols, int64_t ld_x, int8_t* q, float* s, hipStream_t stream) {
  const int64_t grid = WAVES == 1 ? (rows + 3) / 4 : rows;
  const int threads = WAVES == 1 ? 256 : 64 * WAVES;
  if (!grid_fits(grid, threads)) return hipErrorNotSupported;
  int8_rows_kernel<DT, WAVES, CHUNKS><<<(unsigned)grid, threads, 0, stream>>>(x, rows, cols, ld_x, q, s);
  return hipGetLastError();
}

template <int DT>
hipError_t quantize(const void* x, int64_t rows, int64_t cols, int64_t ld_x, int8_t* q, float* s, hipStream_t stream) {
  if (cols <= 512) return rows_cfg<DT, 1, 1>(x, rows, cols, ld_x, q, s, stream);
  if (cols <= 1024) return rows_cfg<DT, 1, 2>(x, rows, cols, ld_x, q, s, stream);
  if (cols <= 2048) return rows_cfg<DT, 1, 4>(x, rows, cols, ld_x, q, s, stream);
  if (cols <= 4096) return rows_cfg<DT, 4, 2>(x, rows, cols, ld_x, q, s, stream);
  if (cols <= 8192) return rows_cfg<DT, 4, 4>(x, rows, cols, ld_x, q, s, stream);
  if (cols <= 32768) return rows_cfg<DT, 16, 4>(x, rows, cols, ld_x, q, s, stream);
  if (!grid_fits(rows, 1024)) return hipErrorNotSupported;
  int8_long_rows_kernel<DT><<<(unsigned)rows, 1024, 0, stream>>>(x, cols, ld_x, q, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, int8_t* q,
                                float* s, hipStream_t stream) {
  return dtype == 1 ? quantize<1>(x, rows, cols, ld_x, q, s, stream) : quantize<0>(x, rows, cols, ld_x, q, s, stream);
}

}  // namespace nvfp4
