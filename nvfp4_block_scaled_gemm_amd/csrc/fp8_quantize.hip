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
#include "fp8_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

using namespace fp8;

constexpr float kTiny = 0x1p-100f, kTop = 448.0f;
constexpr uint32_t kInf = 0x7F800000u;

// Scale, reciprocal and finiteness of a block from the bits of its largest
// magnitude (non-negative floats order like their bits; NaN and infinity sit
// at kInf and above).
struct BlockScale {
  float s, r;
  bool finite;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
  const bool finite = amax_bits < kInf;
  const float a = finite ? fmaxf(__uint_as_float(amax_bits), kTiny) : 1.0f;
  return {finite ? a / kTop : __uint_as_float(0x7FC00000u), kTop / a, finite};
}

__device__ __forceinline__ u32x2 encode8(const float* v, float r, bool finite) {
  u32x2 w = {encode4(v[0] * r, v[1] * r, v[2] * r, v[3] * r),
             encode4(v[4] * r, v[5] * r, v[6] * r, v[7] * r)};
  if (!finite) w = u32x2{0, 0};
  return w;
}

template <int DT>
__device__ __forceinline__ void load8(const void* x, int64_t at, float* v) {
  if constexpr (DT == 1) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(x) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const float*>(x) + at);
    const u32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  }
}

__device__ __forceinline__ uint32_t amax8(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// Largest over the 16 lanes of a row group (all lanes receive it): rotations
// inside the group, no LDS.
template <int N>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  m = max(m, ror16<8>(m));
  m = max(m, ror16<4>(m));
  m = max(m, ror16<2>(m));
  return max(m, ror16<1>(m));
}

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

// What a tile kernel's workgroup works on.
struct QuantTile {
  int64_t src_row;   // first row of x (index: first entry of the row list)
  int rows;          // rows of the tile that exist
  int64_t dst_row;   // first row in the rows layout
  int64_t dst_col;   // first column in the transposed layout
};

// One 128 x 128 tile by 512 threads, 4 rows x 8 columns each (8 x 8 by 256
// threads: 155 registers, three waves a SIMD and 152 instead of 127 us for
// 32768 x 4096 bf16 in both layouts).  BLK: one scale for the tile; else 1 x
// 128 blocks along each layout's own axis.
constexpr int kTileThreads = 512, kTileRows = 4, kTileWaves = kTileThreads / 64;

// Byte of row r (a multiple of 4) of column c in the transposed tile: chunks
// of 16 rows move with the column's group of 8, which is the lane, so that a
// wave's writes spread over the banks.
__device__ __forceinline__ int turned_at(int c, int r) {
  return c * kBlock + ((((r >> 4) ^ ((c >> 3) & 7)) << 4) | (r & 15));
}

template <int DT, bool BLK>
__device__ __forceinline__ void quantize_tile(
    const void* __restrict__ x, int64_t ld_x, int64_t cols, const int32_t* __restrict__ index,
    int64_t x_rows, const QuantTile& t, int64_t kb, uint8_t* __restrict__ q, float* __restrict__ s,
    int64_t s_ld, int64_t s_row, uint8_t* __restrict__ qt, int64_t ld_t, int64_t t_limit,
    float* __restrict__ st, int64_t st_ld, int64_t st_row) {
  constexpr int R = kTileRows;
  __shared__ uint32_t part[kTileWaves][kBlock], rowpart[kBlock];
  __shared__ __attribute__((aligned(16))) float mul[2][kBlock];  // reciprocals: rows, columns
  __shared__ __attribute__((aligned(16))) uint8_t turned[kBlock * kBlock];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
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
  // maxima: a block's scale is computed by one thread and read by those that
  // encode (two divisions a block, not a lane)
  uint32_t colmax[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    colmax[j] = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) colmax[j] = max(colmax[j], __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
  }
  if constexpr (BLK) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, colmax[j]);
    m = max16(m);
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    if (lane == 0) part[wave][0] = m;
    __syncthreads();
    m = 0;
#pragma unroll
    for (int w = 0; w < kTileWaves; ++w) m = max(m, part[w][0]);
    const BlockScale b = block_scale(m);
    if (tid == 0) {
      if (q != nullptr) s[kb * s_ld + s_row] = b.s;
      if (qt != nullptr) st[st_row * st_ld + kb] = b.s;
    }
    u32x2 w[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      w[i] = encode8(v[i], b.r, b.finite);
      if (q != nullptr && r0 + i < t.rows && col_in)
        *reinterpret_cast<u32x2*>(q + (t.dst_row + r0 + i) * cols + col) = w[i];
    }
    if (qt == nullptr) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t o = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) o |= ((w[i][j >> 2] >> (8 * (j & 3))) & 0xFFu) << (8 * i);
      *reinterpret_cast<uint32_t*>(turned + turned_at(cg * 8 + j, r0)) = o;
    }
  } else {
    if (q != nullptr) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint32_t m = max16(amax8(v[i]));
        if (cg == 0) rowpart[r0 + i] = m;
      }
    }
    if (qt != nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = colmax[j];
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if (lane < 16) part[wave][cg * 8 + j] = m;
      }
    }
    __syncthreads();
    const int at = tid & (kBlock - 1);
    if (tid < kBlock) {
      if (q != nullptr) {
        const BlockScale b = block_scale(rowpart[at]);
        mul[0][at] = b.finite ? b.r : -1.f;
        if (at < t.rows) s[kb * s_ld + s_row + at] = b.s;
      }
    } else if (tid < 2 * kBlock && qt != nullptr) {
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < kTileWaves; ++w) m = max(m, part[w][at]);
      const BlockScale b = block_scale(m);
      mul[1][at] = b.finite ? b.r : -1.f;
      if (kb * kBlock + at < cols) st[st_row * st_ld + kb * kBlock + at] = b.s;
    }
    __syncthreads();
    if (q != nullptr) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float m = mul[0][r0 + i];
        if (r0 + i < t.rows && col_in)
          *reinterpret_cast<u32x2*>(q + (t.dst_row + r0 + i) * cols + col) = encode8(v[i], m, m >= 0.f);
      }
    }
    if (qt == nullptr) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float m = mul[1][cg * 8 + j];
      const uint32_t o = encode4(v[0][j] * m, v[1][j] * m, v[2][j] * m, v[3][j] * m);
      *reinterpret_cast<uint32_t*>(turned + turned_at(cg * 8 + j, r0)) = m >= 0.f ? o : 0u;
    }
  }
  __syncthreads();
  // transposed rows: 16 bytes per thread, 8 threads a row
#pragma unroll
  for (int p = 0; p < kBlock * 8 / kTileThreads; ++p) {
    const int c = p * (kTileThreads / 8) + (tid >> 3), r = (tid & 7) * 16;
    const int64_t at = t.dst_col + r;
    if (kb * kBlock + c < cols && at < t_limit)
      *reinterpret_cast<u32x4*>(qt + (kb * kBlock + c) * ld_t + at) =
          *reinterpret_cast<const u32x4*>(turned + turned_at(c, r));
  }
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
  const int lane = threadIdx.x & 63;
  QuantTile t{0, 0, 0, pb * kBlock};
  int64_t before = 0;
  for (int e0 = 0; e0 < G; e0 += 64) {
    const Segment sg = e0 + lane < G ? segment(offsets, e0 + lane, total_m) : Segment{0, 0};
    const uint32_t upto = wave_scan((uint32_t)((sg.n + kBlock - 1) / kBlock));
    const uint64_t past = __ballot(before + (int64_t)upto > pb);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      const int64_t start = before + (l == 0 ? 0 : (int64_t)__builtin_amdgcn_readlane(upto, l - 1));
      const int32_t lo = __builtin_amdgcn_readlane(sg.lo, l), n = __builtin_amdgcn_readlane(sg.n, l);
      const int64_t in = (pb - start) * kBlock;
      t.src_row = t.dst_row = lo + in;
      t.rows = (int)min((int64_t)kBlock, n - in);
      break;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
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
