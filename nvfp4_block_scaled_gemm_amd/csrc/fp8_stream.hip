// FP8 block-128 product for few tokens or few outputs: the weights are
// streamed once, K is split over a workgroup's waves.
//
// With up to 16 rows of A the product does at most 32 operations per weight
// byte, far below what the matrix cores could take, so only the stream of W
// counts; with few outputs the loops over K are too few and too long to fill
// the card.  A workgroup owns BM x BN outputs and its WAVES waves take the
// blocks of K in turn (wave w blocks w, w + WAVES, ..): each wave loads UNROLL
// blocks of both operands straight into fragment registers -- no LDS, no
// barrier in the loop, 16 bytes per lane and 64 contiguous bytes per row and
// load -- and multiplies them as they arrive.  The waves' partial sums meet in
// LDS at the end and are added in wave order, so results do not change
// between calls.  Eight waves per 16 or 32 weight rows instead of one each:
// at N = 8192 that is 4096 waves, 16 per CU, which is what it takes to keep
// enough loads in flight: M = 1, N = K = 8192 reads its 67 MB at 4.4 TB/s
// (15.3 us), 16384 x 4096 16.6 us, 4096 x 4096 7.1 us.
#include <type_traits>

#include "fp8_tile.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

using namespace fp8;

constexpr int64_t kCUs = 256;

__device__ __forceinline__ i32x8 load_fragment(__amdgpu_buffer_rsrc_t r, uint32_t lo, uint32_t hi,
                                               uint32_t soff) {
  const auto a = __builtin_amdgcn_raw_buffer_load_b128(r, lo, soff, 0);
  const auto b = __builtin_amdgcn_raw_buffer_load_b128(r, hi, soff, 0);
  return join(__builtin_bit_cast(u32x4, a), __builtin_bit_cast(u32x4, b));
}

template <int BM, int BN, int UNROLL, int WAVES, bool BROWS, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void fp8_stream_kernel(int64_t M, int64_t N, int64_t K,
                                                                Fp8Operand a, Fp8Operand b, Fp8Out y) {
  constexpr int FM = BM / 16, FN = BN / 16;
  __shared__ __attribute__((aligned(16))) float part[WAVES][BM][BN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const int64_t tiles_n = (N + BN - 1) / BN;
  const int64_t m0 = blockIdx.x / tiles_n * BM, n0 = blockIdx.x % tiles_n * BN;
  const int rm = (int)min((int64_t)BM, M - m0), rn = (int)min((int64_t)BN, N - n0);
  const int nk = (int)((K + kBlock - 1) / kBlock);
  const uint32_t ld = (uint32_t)K, end = (uint32_t)K - (uint32_t)(nk - 1) * kBlock;
  const bool lo_past = (uint32_t)lg * 16 >= end, hi_past = (uint32_t)(lg + 4) * 16 >= end;
  const auto ra = make_rsrc(a.q + m0 * K, (uint32_t)rm * ld);
  const auto rb = make_rsrc(b.q + n0 * K, (uint32_t)rn * ld);
  uint32_t a_off[FM], b_off[FN];
#pragma unroll
  for (int j = 0; j < FM; ++j) a_off[j] = (uint32_t)(16 * j + li) * ld + lg * 16;
#pragma unroll
  for (int i = 0; i < FN; ++i) {
    // two fragments give a lane eight neighbouring columns (one: four)
    const int r = FN == 1 ? li : 32 * (i >> 1) + 8 * (li >> 2) + (li & 3) + 4 * (i & 1);
    b_off[i] = (uint32_t)r * ld + lg * 16;
  }
  f32x4 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t nb = (N + kBlock - 1) / kBlock;

  for (int k0 = wave; k0 < nk; k0 += WAVES * UNROLL) {
    i32x8 bf[UNROLL][FN], af[UNROLL][FM];
    float sa[UNROLL][FM];
    f32x4 sb[UNROLL][BROWS ? FN : 1];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int kb = k0 + u * WAVES;
      const bool none = kb >= nk, cut = kb == nk - 1;
      const uint32_t soff = (uint32_t)kb * kBlock;
#pragma unroll
      for (int i = 0; i < FN; ++i)
        bf[u][i] = load_fragment(rb, none || (cut && lo_past) ? kNoRow : b_off[i],
                                 none || (cut && hi_past) ? kNoRow : b_off[i] + 64, soff);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int kb = k0 + u * WAVES;
      const bool none = kb >= nk, cut = kb == nk - 1;
      const uint32_t soff = (uint32_t)kb * kBlock;
      const int64_t at = none ? 0 : kb;
      const auto rsa = make_rsrc(a.s + at * M + m0, none ? 0u : (uint32_t)rm * 4);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        af[u][j] = load_fragment(ra, none || (cut && lo_past) ? kNoRow : a_off[j],
                                 none || (cut && hi_past) ? kNoRow : a_off[j] + 64, soff);
        sa[u][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsa, (uint32_t)(16 * j + li) * 4, 0, 0));
      }
      if constexpr (BROWS) {
        const auto rsb = make_rsrc(b.s + at * N + n0, none ? 0u : (uint32_t)rn * 4);
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          const int n = FN == 1 ? 4 * lg : 32 * (i >> 1) + 8 * lg + 4 * (i & 1);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sb[u][i][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsb, (uint32_t)(n + e) * 4, 0, 0));
        }
      } else {
        sb[u][0][0] = b.s[at * nb + n0 / kBlock];
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (k0 + u * WAVES >= nk) break;
      if constexpr (!BROWS) {
#pragma unroll
        for (int j = 0; j < FM; ++j) sa[u][j] *= sb[u][0][0];
      }
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const auto bw = fragment<WIDE>(bf[u][i]);
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          const f32x4 c = mfma_block(bw, fragment<WIDE>(af[u][j]));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j][e] = __builtin_fmaf(c[e], BROWS ? sb[u][BROWS ? i : 0][e] * sa[u][j] : sa[u][j], acc[i][j][e]);
        }
      }
    }
  }

#pragma unroll
  for (int j = 0; j < FM; ++j)
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const int n = FN == 1 ? 4 * lg : 32 * (i >> 1) + 8 * lg + 4 * (i & 1);
      *reinterpret_cast<f32x4*>(&part[wave][16 * j + li][n]) = acc[i][j];
    }
  __syncthreads();
  const TileOut out{(uint8_t*)y.y + (m0 * y.ld + n0) * (y.dtype == 0 ? 4 : 2), y.ld, rm, rn, y.dtype, y.add, y.vec};
  for (int t = tid; t < BM * BN / 8; t += 64 * WAVES) {
    const int m = t / (BN / 8), n = t % (BN / 8) * 8;
    if (m >= rm || n >= rn) continue;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const f32x4 lo = *reinterpret_cast<const f32x4*>(&part[w][m][n]);
      const f32x4 hi = *reinterpret_cast<const f32x4*>(&part[w][m][n + 4]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] += lo[e];
        v[4 + e] += hi[e];
      }
    }
    store8(out, m, n, v);
  }
}

// Workgroups of a tile size.
template <int BM, int BN>
int64_t outputs(int64_t M, int64_t N) {
  return ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
}

template <int BM, int BN, int UNROLL, int WAVES, bool BROWS, bool WIDE>
hipError_t stream_cfg(int64_t M, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b, Fp8Out y,
                      hipStream_t stream) {
  const int64_t tiles = outputs<BM, BN>(M, N);
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  fp8_stream_kernel<BM, BN, UNROLL, WAVES, BROWS, WIDE>
      <<<(unsigned)tiles, 64 * WAVES, 0, stream>>>(M, N, K, a, b, y);
  return hipGetLastError();
}

template <bool BROWS, bool WIDE>
hipError_t stream_rows(int64_t M, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b, Fp8Out y,
                       hipStream_t stream) {
  // Outputs per workgroup: the smallest tile that still gives every CU at most
  // one workgroup, since the time is then that of one loop over K (32 rows,
  // N = 2048, K = 6144: 16 x 16 9.1 us, 16 x 32 11.4, 32 x 32 15.1; N = K =
  // 4096: 11.6, 9.1, 11.0; M = 64: 18.3, 14.8, 11.2).  With more workgroups
  // than CUs the re-reads of A decide: 16 weight rows a workgroup up to M = 8
  // (N = K = 8192: M = 1 15.6, with 32 17.2), 32 from there (M = 16: 17.2,
  // with 16 22.1).
  const bool one16 = outputs<16, 16>(M, N) <= kCUs;
  // Sixteen waves pay when a few rows leave the loop to loads' latency and
  // each still has two blocks (M = 1, 4096 x 4096 7.7 -> 7.0 us, M = 16
  // 7.7 -> 8.2; 2560 x 2048 4.1 -> 4.3).
  if (M <= 4 && K >= 32 * kBlock)
    return stream_cfg<16, 16, 2, 16, BROWS, WIDE>(M, N, K, a, b, y, stream);
  if (M <= 8 || one16) return stream_cfg<16, 16, 4, 8, BROWS, WIDE>(M, N, K, a, b, y, stream);
  if (M <= 16 || outputs<16, 32>(M, N) <= kCUs)
    return stream_cfg<16, 32, 2, 8, BROWS, WIDE>(M, N, K, a, b, y, stream);
  return stream_cfg<32, 32, 2, 8, BROWS, WIDE>(M, N, K, a, b, y, stream);
}

}  // namespace

bool fp8_streams(int64_t M, int64_t N) { return M <= 16 || outputs<32, 32>(M, N) <= kCUs; }

hipError_t launch_fp8_stream(int64_t M, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b,
                             int b_block_rows, Fp8Out y, hipStream_t stream) {
  if (y.dtype == 0)
    return b_block_rows == 1 ? stream_rows<true, true>(M, N, K, a, b, y, stream)
                             : stream_rows<false, true>(M, N, K, a, b, y, stream);
  return b_block_rows == 1 ? stream_rows<true, false>(M, N, K, a, b, y, stream)
                           : stream_rows<false, false>(M, N, K, a, b, y, stream);
}

}  // namespace nvfp4
