// What the launchers of the tiled 8-bit products share: the order of tiles over
// the XCDs, a kernel's LDS, tile shapes and their expected times (gfx950 only).
#pragma once

#include <atomic>

#include "fp8_tile.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace fp8 {

constexpr int kXcds = 8;

__device__ __forceinline__ int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Hardware workgroup ids go round-robin over the XCDs; a bijection that
// gives each XCD a run of neighbouring logical ids (shared rows in its L2).
__device__ __forceinline__ int xcd_run(int pid, int n) {
  const int per = n / kXcds, extra = n % kXcds;
  const int x = pid % kXcds, i = pid / kXcds;
  return x * per + min(x, extra) + i;
}

// Allows a kernel its LDS, once per kernel and device.
template <typename Kern>
inline hipError_t allow_lds(Kern kern, int bytes, std::atomic<uint64_t>& done) {
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

// Time of a shape in units of 0.01 us per block of K, from the tiles that the
// busiest of 256 CUs gets: t1 for one tile alone on a CU, t2 for two (shapes
// of which one fits a CU: twice t1).
inline int64_t tiles_cost(int64_t tiles, int64_t t1, int64_t t2) {
  const int64_t n = (tiles + 255) / 256;
  return n / 2 * t2 + n % 2 * t1;
}

inline int64_t tiles_of(int64_t rows, int64_t cols, int64_t bm, int64_t bn) {
  return ((rows + bm - 1) / bm) * ((cols + bn - 1) / bn);
}

inline int64_t shape_cost(int64_t M, int64_t N, int64_t bm, int64_t bn, int64_t t1, int64_t t2) {
  return tiles_cost(tiles_of(M, N, bm, bn), t1, t2);
}

}  // namespace fp8
}  // namespace nvfp4
