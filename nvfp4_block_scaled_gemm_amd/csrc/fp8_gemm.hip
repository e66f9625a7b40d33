// FP8 block-128 products: dense, per expert, and the experts' weight
// gradients.  The tile itself is in fp8_tile.h; here is which tile a
// workgroup takes.
#include <atomic>

#include "fp8_tile.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

using namespace fp8;

constexpr int kXcds = 8;

__device__ __forceinline__ int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Hardware workgroup ids go round-robin over the XCDs; a bijection that
// gives each XCD a run of neighbouring logical ids (shared rows in its L2).
__device__ __forceinline__ int xcd_run(int pid, int n) {
  const int per = n / kXcds, extra = n % kXcds;
  const int x = pid % kXcds, i = pid / kXcds;
  return x * per + min(x, extra) + i;
}

// Rows [r0, r0 + rows) of a whole operand as a tile operand.
__device__ __forceinline__ TileOperand rows_of(const uint8_t* q, const float* s, int64_t s_ld,
                                               int block_rows, int64_t r0, int rows, int64_t K) {
  const int ns = block_rows == 1 ? rows : (rows + kBlock - 1) / kBlock;
  return {q + r0 * K, s + r0 / block_rows, s_ld, (uint32_t)(rows * K), (uint32_t)ns * 4, nullptr, 0, 0};
}

__device__ __forceinline__ TileOut out_of(const Fp8Out& y, int64_t at, int m, int n) {
  const int es = y.dtype == 0 ? 4 : 2;
  return {(uint8_t*)y.y + at * es, y.ld, m, n, y.dtype, y.add, y.vec};
}

template <int BM, int BN, int WM, int WN, int STAGES, int KG, bool BROWS, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN * KG, 2) void fp8_dense_kernel(int64_t M, int64_t N, int64_t K,
                                                                 Fp8Operand a, Fp8Operand b,
                                                                 Fp8Out y) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int tiles_m = (int)ceil_div(M, BM), tiles_n = (int)ceil_div(N, BN);
  // groups of 8 tile rows, walked column by column
  const int pid = xcd_run(blockIdx.x, gridDim.x);
  const int group = pid / (8 * tiles_n), first = group * 8, gsz = min(tiles_m - first, 8);
  const int in = pid - group * 8 * tiles_n;
  const int64_t m0 = (int64_t)(first + in % gsz) * BM, n0 = (int64_t)(in / gsz) * BN;
  const int rm = (int)min((int64_t)BM, M - m0), rn = (int)min((int64_t)BN, N - n0);
  using T = Tile<BM, BN, WM, WN, STAGES, KG, BROWS, WIDE>;
  T::template run<false>(rows_of(a.q, a.s, M, 1, m0, rm, K),
                         rows_of(b.q, b.s, BROWS ? N : ceil_div(N, kBlock), BROWS ? 1 : kBlock, n0, rn, K),
                         (uint32_t)K, (uint32_t)K, out_of(y, m0 * y.ld + n0, rm, rn), smem);
}

// Experts' products: workgroups walk the list of (expert, tile column, tile
// row) tiles, tile rows fastest so that neighbours share a weight tile.  The
// list is known on the device only: each wave keeps 64 experts' running tile
// counts in its lanes and finds a tile's expert by one ballot.  (In the 256 x
// 256 shape that walk costs three spilled registers, stored once and read again
// before and after each tile's loop over K, never in it; the dense kernel of
// the shape has none.)
template <int BM, int BN, int WM, int WN, int STAGES, bool GATHER, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_grouped_kernel(
    int G, const int32_t* __restrict__ offsets, const int32_t* __restrict__ row_index,
    int64_t total_m, int64_t a_rows, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b, Fp8Out y) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  using T = Tile<BM, BN, WM, WN, STAGES, 1, false, WIDE>;
  const int lane = threadIdx.x & 63;
  const int64_t tiles_n = ceil_div(N, BN), nb = ceil_div(N, kBlock), kb = ceil_div(K, kBlock);
  const int step = gridDim.x;
  int64_t before = 0;            // tile rows of the experts below e0
  int e0 = 0;
  auto load = [&](Segment& sg) {
    sg = e0 + lane < G ? segment(offsets, e0 + lane, total_m) : Segment{0, 0};
    return wave_scan((uint32_t)((sg.n + BM - 1) / BM));
  };
  Segment sg;
  uint32_t upto = load(sg);
  for (int64_t u = xcd_run(blockIdx.x, step);; u += step) {
    uint32_t all = __builtin_amdgcn_readlane(upto, 63);
    while (u >= (before + all) * tiles_n) {
      before += all;
      e0 += 64;
      if (e0 >= G) return;
      upto = load(sg);
      all = __builtin_amdgcn_readlane(upto, 63);
    }
    // first lane whose running count passes the tile
    const int64_t v = u - before * tiles_n;
    const uint64_t past = __ballot((int64_t)upto * tiles_n > v);
    const int l = __builtin_ctzll(past);
    const int64_t start = l == 0 ? 0 : (int64_t)__builtin_amdgcn_readlane(upto, l - 1);
    const int32_t lo = __builtin_amdgcn_readlane(sg.lo, l), n = __builtin_amdgcn_readlane(sg.n, l);
    const int32_t te = (n + BM - 1) / BM;
    const int32_t w = (int32_t)(v - start * tiles_n);
    const int32_t tm = w % te, tn = w / te;
    const int64_t e = e0 + l, m0 = lo + (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int rm = min(BM, n - tm * BM), rn = (int)min((int64_t)BN, N - n0);
    TileOperand A;
    if constexpr (GATHER)
      A = {a.q, a.s, a_rows, (uint32_t)(a_rows * K), (uint32_t)a_rows * 4, row_index + m0, rm, (int32_t)a_rows};
    else
      A = rows_of(a.q, a.s, total_m, 1, m0, rm, K);
    const TileOperand B = rows_of(b.q + e * N * K, b.s + e * kb * nb, nb, kBlock, n0, rn, K);
    T::template run<GATHER>(A, B, (uint32_t)K, (uint32_t)K, out_of(y, m0 * y.ld + n0, rm, rn), smem);
    workgroup_barrier();  // every wave is past its last fragment reads
  }
}

// dW_e = A_e . B_e^T over the expert's own columns of the transposed
// operands; each expert's columns start on a block border.
template <int BM, int BN, int WM, int WN, int STAGES, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN, 2) void fp8_wgrad_kernel(
    int G, const int32_t* __restrict__ offsets, int64_t total_m, int64_t P, int64_t N, int64_t K,
    Fp8Operand a, Fp8Operand b, Fp8Out y) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  using T = Tile<BM, BN, WM, WN, STAGES, 1, true, WIDE>;
  const int tiles_m = (int)ceil_div(N, BM), tiles_n = (int)ceil_div(K, BN);
  // every XCD takes an eighth of each expert's tiles, so that experts of
  // uneven load keep them all busy
  const int tiles = tiles_m * tiles_n, per = (tiles + kXcds - 1) / kXcds;
  const int e = blockIdx.x / kXcds / per, in = blockIdx.x % kXcds * per + blockIdx.x / kXcds % per;
  if (in >= tiles) return;
  // along the rows of dW first: neighbours write neighbouring columns (down
  // the columns first: 1125 instead of 1086 us for 64 x 4096 x 2048 fp32)
  const int64_t m0 = (int64_t)(in / tiles_n) * BM, n0 = (int64_t)(in % tiles_n) * BN;
  const int lane = threadIdx.x & 63;
  uint32_t blocks = 0;  // blocks of the experts before e
  for (int i = lane; i < e; i += 64) blocks += (uint32_t)((segment(offsets, i, total_m).n + kBlock - 1) / kBlock);
  blocks = __builtin_amdgcn_readlane(wave_scan(blocks), 63);
  const int64_t k0 = min((int64_t)blocks * kBlock, P);
  const int32_t cnt = __builtin_amdgcn_readfirstlane(segment(offsets, e, total_m).n);
  const int64_t len = min(ceil_div(cnt, kBlock) * kBlock, P - k0);
  const int rm = (int)min((int64_t)BM, N - m0), rn = (int)min((int64_t)BN, K - n0);
  const int64_t b0 = k0 / kBlock;
  // rows are P bytes apart: the range ends with the tile's last row
  TileOperand A{a.q + m0 * P + k0, a.s + b0 * N + m0, N, (uint32_t)(rm * P - k0), (uint32_t)rm * 4, nullptr, 0, 0};
  TileOperand B{b.q + n0 * P + k0, b.s + b0 * K + n0, K, (uint32_t)(rn * P - k0), (uint32_t)rn * 4, nullptr, 0, 0};
  T::template run<false>(A, B, (uint32_t)len, (uint32_t)P, out_of(y, ((int64_t)e * N + m0) * K + n0, rm, rn), smem);
}

// Allows a kernel its LDS, once per kernel and device.
template <typename Kern>
hipError_t allow_lds(Kern kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
  e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// A tile shape: BM x BN outputs by WM x WN waves with a ring of S stages.
template <int BM_, int BN_, int WM_, int WN_, int S_, int KG_ = 1>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_, KG = KG_;
};
using S256x256 = Shape<256, 256, 2, 4, 2>;
using S128x256 = Shape<128, 256, 2, 4, 3>;
using S128x128 = Shape<128, 128, 2, 2, 2>;
using S128x64 = Shape<128, 64, 2, 2, 3, 2>;
using S64x128 = Shape<64, 128, 2, 2, 3>;
using S64x64 = Shape<64, 64, 2, 2, 3, 2>;

template <typename S, bool BROWS, bool WIDE>
hipError_t dense(int64_t M, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b, Fp8Out y,
                 hipStream_t stream) {
  using T = Tile<S::BM, S::BN, S::WM, S::WN, S::S, S::KG, BROWS, WIDE>;
  auto kern = fp8_dense_kernel<S::BM, S::BN, S::WM, S::WN, S::S, S::KG, BROWS, WIDE>;
  const int64_t tiles = ((M + S::BM - 1) / S::BM) * ((N + S::BN - 1) / S::BN);
  if (!grid_fits(tiles, T::kThreads)) return hipErrorNotSupported;
  static std::atomic<uint64_t> done{0};
  const hipError_t err = allow_lds(kern, T::kSmem, done);
  if (err != hipSuccess) return err;
  kern<<<(unsigned)tiles, T::kThreads, T::kSmem, stream>>>(M, N, K, a, b, y);
  return hipGetLastError();
}

// Time of a shape in units of 0.01 us per block of K, from the tiles that the
// busiest of 256 CUs gets: t1 for one tile alone on a CU, t2 for two (shapes
// of which one fits a CU: twice t1).
int64_t tiles_cost(int64_t tiles, int64_t t1, int64_t t2) {
  const int64_t n = (tiles + 255) / 256;
  return n / 2 * t2 + n % 2 * t1;
}

int64_t tiles_of(int64_t rows, int64_t cols, int64_t bm, int64_t bn) {
  return ((rows + bm - 1) / bm) * ((cols + bn - 1) / bn);
}

int64_t shape_cost(int64_t M, int64_t N, int64_t bm, int64_t bn, int64_t t1, int64_t t2) {
  return tiles_cost(tiles_of(M, N, bm, bn), t1, t2);
}

// The shape with the least expected time.  Measured (us per block of 128,
// one / two tiles on each CU): 8-bit products 256 x 256 1.70 / 3.40, 128 x 256
// 1.18 / 2.36, 128 x 128 0.90 / 1.22, 128 x 64 0.46 / 0.91, 64 x 64
// 0.35 / 0.70; wide ones 128 x 128 1.26 / 2.06, 128 x 64 0.67 / 1.34, 64 x 64
// 0.55 / 1.10 (their larger shapes spill).  So 4096 x 8192 takes 256 x 256
// (230 us at K = 8192; 128 x 256: 290), 1024 x 8192 takes 128 x 256 (75;
// 256 x 256: 99), 512 x 4096 takes 128 x 64 (24.3 at K = 6144; 128 x 128:
// 41.5), 96 x 8192 takes 64 x 64 (22.5 at K = 8192; 128 x 64: 29.2).  The two
// smallest split K over two groups of waves (one group: 64 x 4096, K = 6144
// 15.5 instead of 13.5 us; 203 x 8192, K = 8192 31.8 instead of 29.6).
template <bool BROWS, bool WIDE>
hipError_t dense_any(int64_t M, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b, Fp8Out y,
                     hipStream_t stream) {
  constexpr int kShapes = WIDE ? 3 : 5;
  int64_t cost[kShapes];
  if constexpr (WIDE) {
    cost[0] = shape_cost(M, N, 64, 64, 55, 110);
    cost[1] = shape_cost(M, N, 128, 64, 67, 134);
    cost[2] = shape_cost(M, N, 128, 128, 126, 206);
  } else {
    cost[0] = shape_cost(M, N, 64, 64, 35, 70);
    cost[1] = shape_cost(M, N, 128, 64, 46, 91);
    cost[2] = shape_cost(M, N, 128, 128, 90, 122);
    cost[3] = shape_cost(M, N, 128, 256, 118, 236);
    cost[4] = shape_cost(M, N, 256, 256, 170, 340);
  }
  int best = 0;
  for (int i = 1; i < kShapes; ++i)
    if (cost[i] < cost[best]) best = i;
  if constexpr (!WIDE) {
    if (best == 4) return dense<S256x256, BROWS, WIDE>(M, N, K, a, b, y, stream);
    if (best == 3) return dense<S128x256, BROWS, WIDE>(M, N, K, a, b, y, stream);
  }
  if (best == 2) return dense<S128x128, BROWS, WIDE>(M, N, K, a, b, y, stream);
  if (best == 1) return dense<S128x64, BROWS, WIDE>(M, N, K, a, b, y, stream);
  return dense<S64x64, BROWS, WIDE>(M, N, K, a, b, y, stream);
}

template <typename S, bool GATHER, bool WIDE>
hipError_t grouped(int32_t G, const int32_t* m_offsets, const int32_t* row_index, int64_t total_m,
                   int64_t a_rows, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b, Fp8Out y,
                   hipStream_t stream) {
  using T = Tile<S::BM, S::BN, S::WM, S::WN, S::S, 1, false, WIDE>;
  auto kern = fp8_grouped_kernel<S::BM, S::BN, S::WM, S::WN, S::S, GATHER, WIDE>;
  static std::atomic<uint64_t> done{0};
  const hipError_t err = allow_lds(kern, T::kSmem, done);
  if (err != hipSuccess) return err;
  constexpr unsigned per_cu = T::kSmem > 80 * 1024 ? 1 : 2;
  kern<<<256 * per_cu, T::kThreads, T::kSmem, stream>>>(G, m_offsets, row_index, total_m, a_rows, N,
                                                        K, a, b, y);
  return hipGetLastError();
}

template <bool GATHER, bool WIDE>
hipError_t grouped_any(int32_t G, const int32_t* m_offsets, const int32_t* row_index,
                       int64_t total_m, int64_t a_rows, int64_t N, int64_t K, Fp8Operand a,
                       Fp8Operand b, Fp8Out y, hipStream_t stream) {
  // The counts are on the device.  Expected tile rows: one for every expert
  // that can have rows, or the rows' worth and half a tile more for each; then
  // the least expected time, with the dense figures and 0.60 / 0.97 for
  // 64 x 128, wide 0.90 / 1.40.  Measured in us, 64 x 128 / 128 x 128 /
  // 256 x 256 (K = 2048 but for the second): 256 experts of 16 rows, N = 4096
  // 383 / 422 / 433; 8 of 150, N = K = 4096 50 / 39 / 60; 64 of 64, N = 2048
  // 60 / 53 / 59; 64 of 128 96 / 89 / 78; 128 of 512, N = 4096 1088 / 840 / 686.
  // Wide, the first two shapes: 32 of 19, N = 1024 26 / 32; 8 of 150, N = K =
  // 4096 75 / 62; 64 of 128, N = 2048 121 / 116; 128 of 512 1530 / 1254.
  const int64_t live = G < total_m ? G : total_m;
  auto cost = [&](int64_t bm, int64_t bn, int64_t t1, int64_t t2) {
    const int64_t rows = total_m / bm + live / 2;
    return tiles_cost((rows > live ? rows : live) * ((N + bn - 1) / bn), t1, t2);
  };
  const int64_t small = WIDE ? cost(64, 128, 90, 140) : cost(64, 128, 60, 97);
  const int64_t middle = WIDE ? cost(128, 128, 126, 206) : cost(128, 128, 90, 122);
  if constexpr (!WIDE) {
    const int64_t large = cost(256, 256, 170, 340);
    if (large < small && large < middle)
      return grouped<S256x256, GATHER, WIDE>(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y, stream);
  }
  if (middle < small)
    return grouped<S128x128, GATHER, WIDE>(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y, stream);
  return grouped<S64x128, GATHER, WIDE>(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y, stream);
}

template <typename S, bool WIDE>
hipError_t wgrad(int32_t G, const int32_t* m_offsets, int64_t total_m, int64_t P, int64_t N,
                 int64_t K, Fp8Operand a, Fp8Operand b, Fp8Out y, hipStream_t stream) {
  using T = Tile<S::BM, S::BN, S::WM, S::WN, S::S, 1, true, WIDE>;
  auto kern = fp8_wgrad_kernel<S::BM, S::BN, S::WM, S::WN, S::S, WIDE>;
  const int64_t tiles = ((N + S::BM - 1) / S::BM) * ((K + S::BN - 1) / S::BN);
  const int64_t per_group = (tiles + kXcds - 1) / kXcds * kXcds;
  if (!grid_fits(per_group, T::kThreads) || !grid_fits(G * per_group, T::kThreads)) return hipErrorNotSupported;
  const int64_t grid = G * per_group;
  static std::atomic<uint64_t> done{0};
  const hipError_t err = allow_lds(kern, T::kSmem, done);
  if (err != hipSuccess) return err;
  kern<<<(unsigned)grid, T::kThreads, T::kSmem, stream>>>(G, m_offsets, total_m, P, N, K, a, b, y);
  return hipGetLastError();
}

// Calls f with the output's width as a constant: fp32 outputs take the wide
// products, bf16 ones the 8-bit.
template <typename F>
hipError_t by_width(const Fp8Out& y, F&& f) {
  return y.dtype == 0 ? f(std::true_type{}) : f(std::false_type{});
}

}  // namespace

hipError_t launch_fp8_gemm(int64_t M, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b,
                           int b_block_rows, Fp8Out y, hipStream_t stream) {
  if (fp8_streams(M, N)) return launch_fp8_stream(M, N, K, a, b, b_block_rows, y, stream);
  return by_width(y, [&](auto wide) {
    constexpr bool W = decltype(wide)::value;
    return b_block_rows == 1 ? dense_any<true, W>(M, N, K, a, b, y, stream)
                             : dense_any<false, W>(M, N, K, a, b, y, stream);
  });
}

hipError_t launch_fp8_grouped(int32_t G, const int32_t* m_offsets, const int32_t* row_index,
                              int64_t total_m, int64_t a_rows, int64_t N, int64_t K, Fp8Operand a,
                              Fp8Operand b, Fp8Out y, hipStream_t stream) {
  if (fp8_grouped_streams(G, total_m, N, K))
    return launch_fp8_grouped_stream(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y, stream);
  return by_width(y, [&](auto wide) {
    constexpr bool W = decltype(wide)::value;
    return row_index != nullptr
               ? grouped_any<true, W>(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y, stream)
               : grouped_any<false, W>(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y, stream);
  });
}

hipError_t launch_fp8_wgrad(int32_t G, const int32_t* m_offsets, int64_t total_m, int64_t P,
                            int64_t N, int64_t K, Fp8Operand a, Fp8Operand b, Fp8Out y,
                            hipStream_t stream) {
  if (y.dtype == 0) return wgrad<S128x128, true>(G, m_offsets, total_m, P, N, K, a, b, y, stream);
  // the dense rule's figures: 128 x 128 where 256 x 256 leaves CUs idle (bf16,
  // 32 experts of 256 x 384 11.8 us instead of 16.8, 8 of 1024 x 1024 33
  // instead of 40; 16 of 2048 x 1024 46 instead of 42)
  const int64_t large = tiles_cost(G * tiles_of(N, K, 256, 256), 170, 340);
  const int64_t middle = tiles_cost(G * tiles_of(N, K, 128, 128), 90, 122);
  return middle < large ? wgrad<S128x128, false>(G, m_offsets, total_m, P, N, K, a, b, y, stream)
                        : wgrad<S256x256, false>(G, m_offsets, total_m, P, N, K, a, b, y, stream);
}

}  // namespace nvfp4
