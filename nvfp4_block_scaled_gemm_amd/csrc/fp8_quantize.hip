// FP8 block-128 quantiser: x (fp32 | bf16) -> E4M3 bytes and one fp32 scale
// per block, for a block b of 1 x 128 or 128 x 128 elements
//
//   A   = max(max |x_i|, 2^-100)         (a zero block gets a tiny scale)
//   s_b = fl32(A / 448),  r = fl32(448 / A)
//   q_i = E4M3, nearest even, of fl32(x_i * r)
//
// so both layouts and every tiling give the same bytes.  The product with r
// rounds before the E4M3 rounding (off by at most 2^-24 relative): a second
// division-free step per element keeps the kernels at the memory's rate.  A
// block that holds a NaN or an infinity gets a NaN scale and zero bytes.
//
// Two kernels, both bound by HBM:
//  * rows layout alone: 16 lanes take one 1 x 128 block, 8 elements each;
//    one read, one write, no shared memory;
//  * anything that needs a column's or a 128 x 128 block's maximum, or the
//    transposed bytes: a workgroup holds one 128 x 128 tile in registers,
//    each thread 4 rows x 8 columns, so x is read once for all outputs.
//    Row maxima join 16 lanes, column maxima the workgroup through LDS, and
//    the transposed bytes leave through a 16 KB LDS tile in whole 128-byte
//    rows.
// Measured, bf16: 32768 x 4096 to rows 83 us (403 MB, 4.9 TB/s), to both
// layouts 111 (4.9 TB/s); 16 x 8192 2.5 and 4.6, which is the launch.
#include "fp8_quant_tile.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

using namespace fp8;

// Rows layout, 1 x 128 blocks: workgroup (block of K, run of 16 * ROWS rows).
constexpr int kRowPasses = 4;
template <int DT, int PASSES>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* __restrict__ x, int64_t rows,
                                                            int64_t cols, int64_t ld_x, int kblocks,
                                                            uint8_t* __restrict__ q,
                                                            float* __restrict__ s) {
  const int kb = blockIdx.x % kblocks;
  const int64_t r0 = (int64_t)(blockIdx.x / kblocks) * (16 * PASSES) + (threadIdx.x >> 4);
  const int64_t col = (int64_t)kb * kBlock + (threadIdx.x & 15) * 8;
  float v[PASSES][8];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < rows && col < cols) {
      load8<DT>(x, r * ld_x + col, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int64_t r = r0 + 16 * i;
    const BlockScale b = block_scale(max16(amax8(v[i])));
    if (r < rows) {
      if (col < cols) *reinterpret_cast<u32x2*>(q + r * cols + col) = encode8(v[i], b.r, b.finite);
      if ((threadIdx.x & 15) == 0) s[(int64_t)kb * rows + r] = b.s;
    }
  }
}

// One tile of x: the source rows are t.src_row + r, through `index` if given.
template <int DT, bool BLK>
__device__ __forceinline__ void quantize_tile(
    const void* __restrict__ x, int64_t ld_x, int64_t cols, const int32_t* __restrict__ index,
    int64_t x_rows, const QuantTile& t, int64_t kb, uint8_t* __restrict__ q, float* __restrict__ s,
    int64_t s_ld, int64_t s_row, uint8_t* __restrict__ qt, int64_t ld_t, int64_t t_limit,
    float* __restrict__ st, int64_t st_ld, int64_t st_row) {
  constexpr int R = kTileRows;
  const int tid = threadIdx.x;
  const int r0 = (tid >> 4) * R, cg = tid & 15;  // rows from r0, columns from 8 * cg
  const int64_t col = kb * kBlock + cg * 8;
  const bool col_in = col < cols;
  float v[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + i;
    int64_t src = t.src_row + r;
    bool in = r < t.rows && col_in;
    if (index != nullptr && r < t.rows) {
      src = index[src];
      in = in && src >= 0 && src < x_rows;
    }
    if (in) {
      load8<DT>(x, src * ld_x + col, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
  quantize_held<BLK>(v, cols, t, kb, q, s, s_ld, s_row, qt, ld_t, t_limit, st, st_ld, st_row);
}

// Matrices of one batch, 128 x 128 tiles; transposed rows are `rows` rounded
// up to 16 bytes (t_limit).
template <int DT, bool BLK>
__global__ __launch_bounds__(kTileThreads) void quantize_tile_kernel(
    const void* __restrict__ x, int64_t rows, int64_t cols, int64_t ld_x, int kblocks, int rblocks,
    uint8_t* __restrict__ q, float* __restrict__ s, uint8_t* __restrict__ qt,
    float* __restrict__ st) {
  const int kb = blockIdx.x % kblocks, rest = blockIdx.x / kblocks;
  const int rb = rest % rblocks;
  const int64_t b = rest / rblocks;
  const int64_t rows_t = (rows + 15) / 16 * 16;
  const int64_t s_ld = BLK ? rblocks : rows, st_ld = BLK ? kblocks : cols;
  const int64_t r0 = (int64_t)rb * kBlock;
  const QuantTile t{b * rows + r0, (int)min((int64_t)kBlock, rows - r0), r0, r0};
  quantize_tile<DT, BLK>(x, ld_x, cols, nullptr, 0, t, kb, q == nullptr ? q : q + b * rows * cols,
                         s == nullptr ? s : s + b * kblocks * s_ld, s_ld, BLK ? rb : r0,
                         qt == nullptr ? qt : qt + b * cols * rows_t, rows_t, rows_t,
                         st == nullptr ? st : st + b * rblocks * st_ld, st_ld, rb);
}

// Experts' tokens: tile column b of the padded order belongs to the expert
// whose running block count passes it; blocks behind the last expert are
// zero blocks.
template <int DT>
__global__ __launch_bounds__(kTileThreads) void quantize_grouped_kernel(
    const void* __restrict__ x, int G, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ index, int64_t total_m, int64_t x_rows, int64_t cols, int64_t ld_x,
    int64_t P, int kblocks, uint8_t* __restrict__ q, float* __restrict__ s,
    uint8_t* __restrict__ qt, float* __restrict__ st) {
  const int kb = blockIdx.x % kblocks;
  const int64_t pb = blockIdx.x / kblocks;
  const QuantTile t = grouped_tile(G, offsets, total_m, pb);
  quantize_tile<DT, false>(x, ld_x, cols, index, x_rows, t, kb, q, s, total_m, t.dst_row, qt, P, P,
                           st, cols, pb);
}

}  // namespace

hipError_t launch_fp8_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols,
                               int64_t ld_x, int block_rows, uint8_t* q, float* s, uint8_t* qt,
                               float* st, hipStream_t stream) {
  const int64_t kblocks = (cols + kBlock - 1) / kBlock, rblocks = (rows + kBlock - 1) / kBlock;
  if (block_rows == 1 && qt == nullptr && batch == 1) {
    const int64_t grid = kblocks * ((rows + 16 * kRowPasses - 1) / (16 * kRowPasses));
    if (!grid_fits(grid, 256)) return hipErrorNotSupported;
    auto kern = dtype == 1 ? quantize_rows_kernel<1, kRowPasses> : quantize_rows_kernel<0, kRowPasses>;
    kern<<<(unsigned)grid, 256, 0, stream>>>(x, rows, cols, ld_x, (int)kblocks, q, s);
    return hipGetLastError();
  }
  const int64_t tiles = kblocks * rblocks;  // below 2^47
  if (!grid_fits(tiles, kTileThreads) || !grid_fits(batch * tiles, kTileThreads)) return hipErrorNotSupported;
  const int64_t grid = batch * tiles;
  auto kern = block_rows == 1
                  ? (dtype == 1 ? quantize_tile_kernel<1, false> : quantize_tile_kernel<0, false>)
                  : (dtype == 1 ? quantize_tile_kernel<1, true> : quantize_tile_kernel<0, true>);
  kern<<<(unsigned)grid, kTileThreads, 0, stream>>>(x, rows, cols, ld_x, (int)kblocks, (int)rblocks, q, s, qt, st);
  return hipGetLastError();
}

hipError_t launch_fp8_grouped_quantize(const void* x, int dtype, int32_t G,
                                       const int32_t* m_offsets, const int32_t* row_index,
                                       int64_t total_m, int64_t x_rows, int64_t cols, int64_t ld_x,
                                       uint8_t* q, float* s, uint8_t* qt, float* st,
                                       hipStream_t stream) {
  const int64_t P = fp8_padded_tokens(total_m, G);
  const int64_t kblocks = (cols + kBlock - 1) / kBlock;
  const int64_t grid = kblocks * (P / kBlock);
  if (!grid_fits(grid, kTileThreads)) return hipErrorNotSupported;
  auto kern = dtype == 1 ? quantize_grouped_kernel<1> : quantize_grouped_kernel<0>;
  kern<<<(unsigned)grid, kTileThreads, 0, stream>>>(x, G, m_offsets, row_index, total_m, x_rows, cols, ld_x, P,
                                           (int)kblocks, q, s, qt, st);
  return hipGetLastError();
}

}  // namespace nvfp4
