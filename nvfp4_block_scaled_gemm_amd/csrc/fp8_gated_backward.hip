// Backward of h = act(g) * u: from dh [rows, F] and the kept products
// gate_up [rows, 2F] = [g, u]
//
//   dg = dh u act'(g),   du = dh act(g)
//
// written as the FP8 operand [dg, du] [rows, 2F] in either layout (blocks as in
// fp8_quantize.hip), so that the products for dx and dW follow without a
// bf16 gradient in between.  Everything is fp32 up to the E4M3 rounding.
//
// Bound by HBM: 6 bytes read (bf16) and 4 written (both layouts) per element of
// h.  Where F is a multiple of 128 a workgroup turns one 128 x 128 tile of the
// three inputs into the two tiles of dg and du, so the inputs are read once;
// for other F a block of 128 columns straddles the halves and each workgroup
// computes one output tile (its inputs are read twice, the second time mostly
// from a cache).  Both gradients and what they come from take 150 registers: one
// workgroup of eight waves on a CU, where the quantiser's 76 leave room for three.
// The rows layout alone needs no shared memory: 16 lanes take one 1 x 128 block
// (experts' rows go through the tile kernel all the same).  Not timed.
#include "fp8_quant_tile.h"
#include "gated_act.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

using namespace fp8;

struct GatedIn {
  const void* dh;  // [rows, F], row stride ld_dh
  const void* gu;  // [rows, 2F], row stride ld_gu
  int64_t ld_dh, ld_gu, F;
  int act;
};

// Eight elements of dg and du from column c of row r.
template <int DTD, int DTG>
__device__ __forceinline__ void gradients8(const GatedIn& in, int64_t r, int64_t c, float* dg, float* du) {
  float d[8], g[8], u[8];
  load8<DTD>(in.dh, r * in.ld_dh + c, d);
  load8<DTG>(in.gu, r * in.ld_gu + c, g);
  load8<DTG>(in.gu, r * in.ld_gu + in.F + c, u);
  auto all = [&](auto act) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const Sigma a = sigma_of<decltype(act)::value>(g[j]);
      const float v = g[j] * a.sigma;
      dg[j] = d[j] * u[j] * __builtin_fmaf(v, a.turn, a.sigma);
      du[j] = d[j] * v;
    }
  };
  if (in.act == kGelu) all(std::integral_constant<int, kGelu>{});
  else all(std::integral_constant<int, kSilu>{});
}

__device__ __forceinline__ void zero8(float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
}

// Where the two layouts go; null: not wanted.
struct GatedOut {
  uint8_t* q;
  float* s;
  int64_t s_ld;  // rows of the rows layout's scales
  uint8_t* qt;
  float* st;
  int64_t ld_t;  // bytes of a transposed row
};

// Tile t of output columns 128 * kb (PAIR: of dg, and the tile of du F
// columns on).
template <int DTD, int DTG, bool PAIR>
__device__ __forceinline__ void backward_tile(const GatedIn& in, const GatedOut& out, const QuantTile& t,
                                              int64_t kb, int64_t st_row) {
  constexpr int R = kTileRows;
  const int tid = threadIdx.x, r0 = (tid >> 4) * R, cg = tid & 15;
  const int64_t col = kb * kBlock + cg * 8, cols = 2 * in.F;
  const bool up = !PAIR && col >= in.F;
  const int64_t c = up ? col - in.F : col;
  float dg[R][8], du[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (r0 + i < t.rows && col < cols) {
      gradients8<DTD, DTG>(in, t.src_row + r0 + i, c, dg[i], du[i]);
    } else {
      zero8(dg[i]);
      zero8(du[i]);
    }
    if constexpr (!PAIR) {
#pragma unroll
      for (int j = 0; j < 8; ++j) dg[i][j] = up ? du[i][j] : dg[i][j];
    }
  }
  quantize_held<false>(dg, cols, t, kb, out.q, out.s, out.s_ld, t.dst_row, out.qt, out.ld_t, out.ld_t, out.st,
                       cols, st_row);
  if constexpr (PAIR) {
    __syncthreads();  // the first tile's bytes have left the shared memory
    quantize_held<false>(du, cols, t, kb + in.F / kBlock, out.q, out.s, out.s_ld, t.dst_row, out.qt, out.ld_t,
                         out.ld_t, out.st, cols, st_row);
  }
}

template <int DTD, int DTG, bool PAIR>
__global__ __launch_bounds__(kTileThreads) void gated_backward_kernel(GatedIn in, GatedOut out, int64_t rows,
                                                                      int kblocks) {
  const int kb = blockIdx.x % kblocks;
  const int64_t rb = blockIdx.x / kblocks, r0 = rb * kBlock;
  backward_tile<DTD, DTG, PAIR>(in, out, {r0, (int)min((int64_t)kBlock, rows - r0), r0, r0}, kb, rb);
}

template <int DTD, int DTG, bool PAIR>
__global__ __launch_bounds__(kTileThreads) void gated_backward_grouped_kernel(
    GatedIn in, GatedOut out, int G, const int32_t* __restrict__ offsets, int64_t total_m, int kblocks) {
  const int kb = blockIdx.x % kblocks;
  const int64_t pb = blockIdx.x / kblocks;
  backward_tile<DTD, DTG, PAIR>(in, out, grouped_tile(G, offsets, total_m, pb), kb, pb);
}

// Rows layout alone: 16 lanes a block of 128 columns, 16 rows a pass.
constexpr int kRowPasses = 2;
template <int DTD, int DTG, bool PAIR>
__global__ __launch_bounds__(256) void gated_backward_rows_kernel(GatedIn in, uint8_t* __restrict__ q,
                                                                  float* __restrict__ s, int64_t rows,
                                                                  int kblocks) {
  const int kb = blockIdx.x % kblocks;
  const int64_t r0 = (int64_t)(blockIdx.x / kblocks) * (16 * kRowPasses) + (threadIdx.x >> 4);
  const int64_t col = (int64_t)kb * kBlock + (threadIdx.x & 15) * 8, cols = 2 * in.F;
  const bool up = !PAIR && col >= in.F;
  const int64_t c = up ? col - in.F : col;
  auto put = [&](int64_t r, int64_t at, int64_t block, const float* v) {
    const BlockScale b = block_scale(max16(amax8(v)));
    if (r < rows) {
      if (at < cols) *reinterpret_cast<u32x2*>(q + r * cols + at) = encode8(v, b.r, b.finite);
      if ((threadIdx.x & 15) == 0) s[block * rows + r] = b.s;
    }
  };
#pragma unroll
  for (int i = 0; i < kRowPasses; ++i) {
    const int64_t r = r0 + 16 * i;
    float dg[8], du[8];
    if (r < rows && col < cols) {
      gradients8<DTD, DTG>(in, r, c, dg, du);
    } else {
      zero8(dg);
      zero8(du);
    }
    if constexpr (PAIR) {
      put(r, col, kb, dg);
      put(r, col + in.F, kb + in.F / kBlock, du);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) dg[j] = up ? du[j] : dg[j];
      put(r, col, kb, dg);
    }
  }
}

// Calls f with the inputs' types and whether F is whole blocks as constants.
template <typename F>
hipError_t by_kind(int dh_dtype, int gu_dtype, int64_t width, F&& f) {
  auto kept = [&](auto d, auto g) {
    return width % kBlock == 0 ? f(d, g, std::true_type{}) : f(d, g, std::false_type{});
  };
  auto typed = [&](auto d) {
    return gu_dtype == 1 ? kept(d, std::integral_constant<int, 1>{}) : kept(d, std::integral_constant<int, 0>{});
  };
  return dh_dtype == 1 ? typed(std::integral_constant<int, 1>{}) : typed(std::integral_constant<int, 0>{});
}

int64_t column_blocks(int64_t F) { return F % kBlock == 0 ? F / kBlock : (2 * F + kBlock - 1) / kBlock; }

}  // namespace

hipError_t launch_fp8_gated_backward(GatedGradient g, int64_t rows, uint8_t* q, float* s, uint8_t* qt, float* st,
                                     hipStream_t stream) {
  const GatedIn in{g.dh, g.gate_up, g.ld_dh, g.ld_gu, g.F, g.act};
  const int64_t kblocks = column_blocks(g.F);
  const bool tiles = qt != nullptr;
  const int64_t per = tiles ? kBlock : 16 * kRowPasses;
  const int threads = tiles ? kTileThreads : 256;
  const int64_t grid = kblocks * ((rows + per - 1) / per);
  if (!grid_fits(grid, threads)) return hipErrorNotSupported;
  return by_kind(g.dh_dtype, g.gu_dtype, g.F, [&](auto d, auto k, auto pair) {
    constexpr int DTD = decltype(d)::value, DTG = decltype(k)::value;
    constexpr bool PAIR = decltype(pair)::value;
    if (tiles)
      gated_backward_kernel<DTD, DTG, PAIR><<<(unsigned)grid, threads, 0, stream>>>(
          in, {q, s, rows, qt, st, (rows + 15) / 16 * 16}, rows, (int)kblocks);
    else
      gated_backward_rows_kernel<DTD, DTG, PAIR><<<(unsigned)grid, threads, 0, stream>>>(in, q, s, rows, (int)kblocks);
    return hipGetLastError();
  });
}

hipError_t launch_fp8_grouped_gated_backward(GatedGradient g, int32_t G, const int32_t* m_offsets, int64_t total_m,
                                             uint8_t* q, float* s, uint8_t* qt, float* st, hipStream_t stream) {
  const GatedIn in{g.dh, g.gate_up, g.ld_dh, g.ld_gu, g.F, g.act};
  const int64_t kblocks = column_blocks(g.F), P = fp8_padded_tokens(total_m, G);
  const int64_t grid = kblocks * (P / kBlock);
  if (!grid_fits(grid, kTileThreads)) return hipErrorNotSupported;
  return by_kind(g.dh_dtype, g.gu_dtype, g.F, [&](auto d, auto k, auto pair) {
    gated_backward_grouped_kernel<decltype(d)::value, decltype(k)::value, decltype(pair)::value>
        <<<(unsigned)grid, kTileThreads, 0, stream>>>(in, {q, s, total_m, qt, st, P}, G, m_offsets, total_m,
                                                      (int)kblocks);
    return hipGetLastError();
  });
}

}  // namespace nvfp4
