// INT8 product with a scale per row of either operand (tokens and output
// channels):
//
//   y[m, n] = fl(sum_k qa[m, k] qb[n, k]) * sa[m] * sb[n]
//
// The sums are 32-bit integers, exact for K < 2^17 (128 * 128 * K < 2^31), so no
// order of adding changes a result; the sum is rounded to fp32 once and
// multiplied by the two scales.  v_mfma_i32_16x16x64_i8 runs at the 8-bit rate.
//
// Many rows: the tile of the FP8 products (fp8_tile.h) without scales in its
// loop.  Few rows or outputs: the weights are streamed, K split over a
// workgroup's waves, as in fp8_stream.hip.  There the compiler keeps a block's
// loads together; here, where nothing waits for scales, it puts the last of them
// behind the block's first product, so three or four 16-byte loads of a wave are in
// flight (44 to 47 registers) and UNROLL does not add to them.  Not timed.
#include <type_traits>

#include "fp8_launch.h"

namespace nvfp4 {
namespace {

using namespace fp8;

__device__ __forceinline__ TileOut out_of(const Fp8Out& y, int64_t m0, int64_t n0, int m, int n) {
  return {(uint8_t*)y.y + (m0 * y.ld + n0) * (y.dtype == 0 ? 4 : 2), y.ld, m, n, y.dtype, false, y.vec};
}

__device__ __forceinline__ TileOperand rows_of(const Int8Operand& a, int64_t r0, int rows, int64_t K) {
  return {reinterpret_cast<const uint8_t*>(a.q) + r0 * K, a.s + r0, 0, (uint32_t)(rows * K), 0, nullptr, 0, 0};
}

template <int BM, int BN, int WM, int WN, int STAGES, int KG>
__global__ __launch_bounds__(64 * WM * WN * KG, 2) void int8_dense_kernel(int64_t M, int64_t N, int64_t K,
                                                                         Int8Operand a, Int8Operand b, Fp8Out y) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tiles_m = (int)ceil_div(M, BM), tiles_n = (int)ceil_div(N, BN);
  // groups of 8 tile rows, walked column by column
  const int pid = xcd_run(blockIdx.x, gridDim.x);
  const int group = pid / (8 * tiles_n), first = group * 8, gsz = min(tiles_m - first, 8);
  const int in = pid - group * 8 * tiles_n;
  const int64_t m0 = (int64_t)(first + in % gsz) * BM, n0 = (int64_t)(in / gsz) * BN;
  const int rm = (int)min((int64_t)BM, M - m0), rn = (int)min((int64_t)BN, N - n0);
  using T = Tile<BM, BN, WM, WN, STAGES, KG, false, false, false, true>;
  T::template run<false>(rows_of(a, m0, rm, K), rows_of(b, n0, rn, K), (uint32_t)K, (uint32_t)K,
                         out_of(y, m0, n0, rm, rn), smem);
}

__device__ __forceinline__ i32x8 load_fragment(__amdgpu_buffer_rsrc_t r, uint32_t lo, uint32_t hi, uint32_t soff) {
  const auto a = __builtin_amdgcn_raw_buffer_load_b128(r, lo, soff, 0);
  const auto b = __builtin_amdgcn_raw_buffer_load_b128(r, hi, soff, 0);
  return join(__builtin_bit_cast(u32x4, a), __builtin_bit_cast(u32x4, b));
}

// BM x BN outputs, WAVES waves taking blocks of 128 of K in turn.
template <int BM, int BN, int UNROLL, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void int8_stream_kernel(int64_t M, int64_t N, int64_t K, Int8Operand a,
                                                                 Int8Operand b, Fp8Out y) {
  constexpr int FM = BM / 16, FN = BN / 16;
  __shared__ __attribute__((aligned(16))) int part[WAVES][BM][BN];
  const int64_t tiles_n = (N + BN - 1) / BN;
  const int64_t m0 = blockIdx.x / tiles_n * BM, n0 = blockIdx.x % tiles_n * BN;
  const int rm = (int)min((int64_t)BM, M - m0), rn = (int)min((int64_t)BN, N - n0);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const int nk = (int)((K + kBlock - 1) / kBlock);
  const uint32_t ld = (uint32_t)K, end = (uint32_t)K - (uint32_t)(nk - 1) * kBlock;
  const bool lo_past = (uint32_t)lg * 16 >= end, hi_past = (uint32_t)(lg + 4) * 16 >= end;
  const auto ra = make_rsrc(a.q + m0 * K, (uint32_t)rm * ld), rb = make_rsrc(b.q + n0 * K, (uint32_t)rn * ld);
  i32x4 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  for (int k0 = wave; k0 < nk; k0 += WAVES * UNROLL) {
    i32x8 bf[UNROLL][FN], af[UNROLL][FM];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int kb = k0 + u * WAVES;
      const bool none = kb >= nk, cut = kb == nk - 1;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const uint32_t at = (uint32_t)(16 * i + li) * ld + lg * 16;
        bf[u][i] = load_fragment(rb, none || (cut && lo_past) ? kNoRow : at,
                                 none || (cut && hi_past) ? kNoRow : at + 64, (uint32_t)kb * kBlock);
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int kb = k0 + u * WAVES;
      const bool none = kb >= nk, cut = kb == nk - 1;
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        const uint32_t at = (uint32_t)(16 * j + li) * ld + lg * 16;
        af[u][j] = load_fragment(ra, none || (cut && lo_past) ? kNoRow : at,
                                 none || (cut && hi_past) ? kNoRow : at + 64, (uint32_t)kb * kBlock);
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (k0 + u * WAVES >= nk) break;
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          acc[i][j] = mfma_half<0>(bf[u][i], af[u][j], acc[i][j]);
          acc[i][j] = mfma_half<1>(bf[u][i], af[u][j], acc[i][j]);
        }
    }
  }
#pragma unroll
  for (int j = 0; j < FM; ++j)
#pragma unroll
    for (int i = 0; i < FN; ++i) *reinterpret_cast<i32x4*>(&part[wave][16 * j + li][16 * i + 4 * lg]) = acc[i][j];
  __syncthreads();
  const TileOut out = out_of(y, m0, n0, rm, rn);
  for (int t = tid; t < BM * BN / 8; t += 64 * WAVES) {
    const int m = t / (BN / 8), n = t % (BN / 8) * 8;
    if (m >= rm || n >= rn) continue;
    int sum[8];
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += part[w][m][n + e];
    const float sm = a.s[m0 + m];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)sum[e] * sm * b.s[n0 + min(n + e, rn - 1)];
    store8(out, m, n, v);
  }
}

template <typename S>
hipError_t dense(int64_t M, int64_t N, int64_t K, Int8Operand a, Int8Operand b, Fp8Out y, hipStream_t stream) {
  using T = Tile<S::BM, S::BN, S::WM, S::WN, S::S, S::KG, false, false, false, true>;
  auto kern = int8_dense_kernel<S::BM, S::BN, S::WM, S::WN, S::S, S::KG>;
  const int64_t tiles = tiles_of(M, N, S::BM, S::BN);
  if (!grid_fits(tiles, T::kThreads)) return hipErrorNotSupported;
  static std::atomic<uint64_t> done{0};
  const hipError_t err = allow_lds(kern, T::kSmem, done);
  if (err != hipSuccess) return err;
  kern<<<(unsigned)tiles, T::kThreads, T::kSmem, stream>>>(M, N, K, a, b, y);
  return hipGetLastError();
}

template <int BM, int BN, int UNROLL, int WAVES>
hipError_t stream_cfg(int64_t M, int64_t N, int64_t K, Int8Operand a, Int8Operand b, Fp8Out y, hipStream_t stream) {
  const int64_t tiles = tiles_of(M, N, BM, BN);
  if (!grid_fits(tiles, 64 * WAVES)) return hipErrorNotSupported;
  int8_stream_kernel<BM, BN, UNROLL, WAVES><<<(unsigned)tiles, 64 * WAVES, 0, stream>>>(M, N, K, a, b, y);
  return hipGetLastError();
}

}  // namespace

// The FP8 products' borders and times (fp8_stream.hip, fp8_gemm.hip), whose tiles
// these are.  None was measured with integers: those times hold the scaled additions
// that this loop is without.  Every variant gives the same bits.
hipError_t launch_int8_gemm(int64_t M, int64_t N, int64_t K, Int8Operand a, Int8Operand b, Fp8Out y,
                            hipStream_t stream) {
  if (M <= 16 || tiles_of(M, N, 32, 32) <= 256) {
    if (M <= 4 && K >= 48 * kBlock) return stream_cfg<16, 16, 2, 16>(M, N, K, a, b, y, stream);
    if (M <= 8 || tiles_of(M, N, 16, 16) <= 256) return stream_cfg<16, 16, 4, 8>(M, N, K, a, b, y, stream);
    if (M <= 16 || tiles_of(M, N, 16, 32) <= 256) return stream_cfg<16, 32, 2, 8>(M, N, K, a, b, y, stream);
    return stream_cfg<32, 32, 2, 8>(M, N, K, a, b, y, stream);
  }
  const int64_t cost[5] = {shape_cost(M, N, 64, 64, 35, 70), shape_cost(M, N, 128, 64, 46, 91),
                           shape_cost(M, N, 128, 128, 90, 122), shape_cost(M, N, 128, 256, 118, 236),
                           shape_cost(M, N, 256, 256, 170, 340)};
  int best = 0;
  for (int i = 1; i < 5; ++i)
    if (cost[i] < cost[best]) best = i;
  if (best == 4) return dense<S256x256>(M, N, K, a, b, y, stream);
  if (best == 3) return dense<S128x256>(M, N, K, a, b, y, stream);
  if (best == 2) return dense<S128x128>(M, N, K, a, b, y, stream);
  if (best == 1) return dense<S128x64>(M, N, K, a, b, y, stream);
  return dense<S64x64>(M, N, K, a, b, y, stream);
}

}  // namespace nvfp4
