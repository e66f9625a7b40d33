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
// between calls.  Eight or sixteen waves per 16 or 32 weight rows instead of
// one each are what it takes to keep enough loads in flight: M = 1, N = K =
// 8192 reads its 67 MB by 512 workgroups of 16 waves in 13.6 us (4.9 TB/s; the
// card reads 6.6 TB/s from a few GB in one launch), 4096 x 4096 takes 7.0 us.
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

// Rows of A that a workgroup multiplies: lane li of fragment j takes row
// 16 j + li, whose bytes and scale are at the offsets (kNoRow: zeros).
template <int FM>
struct StreamRows {
  const uint8_t* q;
  const float* s;
  int64_t s_ld;
  uint32_t q_bytes, s_bytes;
  uint32_t q_off[FM], s_off[FM];
};

// BM x BN outputs from rn rows of B at bq (scales of block 0 at bs, s_ld
// apart) and the rows of A.
template <int BM, int BN, int UNROLL, int WAVES, bool BROWS, bool WIDE>
__device__ __forceinline__ void stream_outputs(const StreamRows<BM / 16>& A, const uint8_t* bq,
                                               const float* bs, int64_t bs_ld, int rn, int64_t K,
                                               const TileOut& out) {
  constexpr int FM = BM / 16, FN = BN / 16;
  __shared__ __attribute__((aligned(16))) float part[WAVES][BM][BN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const int nk = (int)((K + kBlock - 1) / kBlock);
  const uint32_t ld = (uint32_t)K, end = (uint32_t)K - (uint32_t)(nk - 1) * kBlock;
  const bool lo_past = (uint32_t)lg * 16 >= end, hi_past = (uint32_t)(lg + 4) * 16 >= end;
  const auto ra = make_rsrc(A.q, A.q_bytes);
  const auto rb = make_rsrc(bq, (uint32_t)rn * ld);
  uint32_t a_off[FM], b_off[FN];
#pragma unroll
  for (int j = 0; j < FM; ++j) a_off[j] = A.q_off[j] + lg * 16;
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
      const auto rsa = make_rsrc(A.s + at * A.s_ld, none ? 0u : A.s_bytes);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        af[u][j] = load_fragment(ra, none || (cut && lo_past) ? kNoRow : a_off[j],
                                 none || (cut && hi_past) ? kNoRow : a_off[j] + 64, soff);
        sa[u][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsa, A.s_off[j], 0, 0));
      }
      if constexpr (BROWS) {
        const auto rsb = make_rsrc(bs + at * bs_ld, none ? 0u : (uint32_t)rn * 4);
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          const int n = FN == 1 ? 4 * lg : 32 * (i >> 1) + 8 * lg + 4 * (i & 1);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sb[u][i][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsb, (uint32_t)(n + e) * 4, 0, 0));
        }
      } else {
        sb[u][0][0] = bs[at * bs_ld];
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
  for (int t = tid; t < BM * BN / 8; t += 64 * WAVES) {
    const int m = t / (BN / 8), n = t % (BN / 8) * 8;
    if (m >= out.m || n >= out.n) continue;
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

__device__ __forceinline__ TileOut out_of(const Fp8Out& y, int64_t m0, int64_t n0, int m, int n) {
  return {(uint8_t*)y.y + (m0 * y.ld + n0) * (y.dtype == 0 ? 4 : 2), y.ld, m, n, y.dtype, y.add, y.vec};
}

// Rows m0 .. m0 + n of a K-block-major operand with `rows` rows.
template <int FM>
__device__ __forceinline__ StreamRows<FM> rows_from(const Fp8Operand& a, int64_t rows, int64_t m0,
                                                    int n, int64_t K) {
  StreamRows<FM> r{a.q + m0 * K, a.s + m0, rows, (uint32_t)n * (uint32_t)K, (uint32_t)n * 4, {}, {}};
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const uint32_t row = 16 * j + (threadIdx.x & 15);
    r.q_off[j] = row * (uint32_t)K;
    r.s_off[j] = row * 4;
  }
  return r;
}

template <int BM, int BN, int UNROLL, int WAVES, bool BROWS, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void fp8_stream_kernel(int64_t M, int64_t N, int64_t K,
                                                                Fp8Operand a, Fp8Operand b, Fp8Out y) {
  const int64_t tiles_n = (N + BN - 1) / BN;
  const int64_t m0 = blockIdx.x / tiles_n * BM, n0 = blockIdx.x % tiles_n * BN;
  const int rm = (int)min((int64_t)BM, M - m0), rn = (int)min((int64_t)BN, N - n0);
  const int64_t s_ld = BROWS ? N : (N + kBlock - 1) / kBlock;
  stream_outputs<BM, BN, UNROLL, WAVES, BROWS, WIDE>(
      rows_from<BM / 16>(a, M, m0, rm, K), b.q + n0 * K, b.s + (BROWS ? n0 : n0 / kBlock), s_ld, rn, K,
      out_of(y, m0, n0, rm, rn));
}

// Experts' products of few rows: the workgroup's (expert, tile column, tile
// row) in a list that is known on the device only, 64 experts' running counts
// in a wave's lanes at a time.  Eight tile columns of an expert's rows in
// turn, so that the rows of one column share its XCD's L2.
template <int BM, int BN, int UNROLL, int WAVES, bool GATHER, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void fp8_grouped_stream_kernel(
    int G, const int32_t* __restrict__ offsets, const int32_t* __restrict__ row_index,
    int64_t total_m, int64_t a_rows, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b, Fp8Out y) {
  const int lane = threadIdx.x & 63;
  const int64_t tiles_n = (N + BN - 1) / BN, nb = (N + kBlock - 1) / kBlock, kb = (K + kBlock - 1) / kBlock;
  int64_t v = blockIdx.x;
  int e0 = 0;
  Segment sg;
  uint32_t upto, all;
  for (;;) {
    sg = e0 + lane < G ? segment(offsets, e0 + lane, total_m) : Segment{0, 0};
    upto = wave_scan((uint32_t)((sg.n + BM - 1) / BM));
    all = __builtin_amdgcn_readlane(upto, 63);
    if (v < all * tiles_n) break;
    v -= all * tiles_n;
    e0 += 64;
    if (e0 >= G) return;
  }
  // first lane whose running count passes the tile
  const int l = __builtin_ctzll(__ballot((int64_t)upto * tiles_n > v));
  const int64_t start = l == 0 ? 0 : (int64_t)__builtin_amdgcn_readlane(upto, l - 1);
  const int32_t lo = __builtin_amdgcn_readlane(sg.lo, l), n = __builtin_amdgcn_readlane(sg.n, l);
  const int32_t te = (n + BM - 1) / BM;
  const int64_t w = v - start * tiles_n, eight = w / (8 * te) * 8;
  const int32_t in = (int32_t)(w - eight * te), cols = (int32_t)min(tiles_n - eight, (int64_t)8);
  const int32_t tm = in / cols;
  const int64_t e = e0 + l, m0 = lo + (int64_t)tm * BM, n0 = (eight + in % cols) * BN;
  const int rm = min(BM, n - tm * BM), rn = (int)min((int64_t)BN, N - n0);
  StreamRows<BM / 16> A;
  if constexpr (GATHER) {
    A = {a.q, a.s, a_rows, (uint32_t)(a_rows * K), (uint32_t)a_rows * 4, {}, {}};
#pragma unroll
    for (int j = 0; j < BM / 16; ++j) {
      const int r = 16 * j + (lane & 15);
      const int32_t row = r < rm ? row_index[m0 + r] : -1;
      const bool ok = row >= 0 && row < a_rows;
      A.q_off[j] = ok ? (uint32_t)row * (uint32_t)K : kNoRow;
      A.s_off[j] = ok ? (uint32_t)row * 4 : kNoRow;
    }
  } else {
    A = rows_from<BM / 16>(a, total_m, m0, rm, K);
  }
  stream_outputs<BM, BN, UNROLL, WAVES, false, WIDE>(A, b.q + (e * N + n0) * K, b.s + e * kb * nb + n0 / kBlock,
                                                     nb, rn, K, out_of(y, m0, n0, rm, rn));
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
  if (!grid_fits(tiles, 64 * WAVES)) return hipErrorNotSupported;
  fp8_stream_kernel<BM, BN, UNROLL, WAVES, BROWS, WIDE>
      <<<(unsigned)tiles, 64 * WAVES, 0, stream>>>(M, N, K, a, b, y);
  return hipGetLastError();
}

// WIDE: how 32-row tiles multiply.  16-row tiles always take the 16-bit
// instructions and their fp32 sums, bf16 outputs too: the loads hide them, or
// most of them (us, 8-bit and wide: 1 x 8192 x 8192 14.6 / 14.6, 16 x 4096 x 4096
// 7.6 / 7.5, 32 x 4096 x 4096 8.9 / 9.2, 16 x 32768 x 4096 30.8 / 32.5; experts, 16
// tokens top 2 of 8, 4096 x 14336 83 / 87; of 32-row tiles 64 x 4096 x 4096 10.9 /
// 14.3).
template <bool BROWS, bool WIDE>
hipError_t stream_rows(int64_t M, int64_t N, int64_t K, Fp8Operand a, Fp8Operand b, Fp8Out y,
                       hipStream_t stream) {
  // Outputs per workgroup: the smallest tile that still gives every CU at most
  // one workgroup, since the time is then that of one loop over K (bf16, 32
  // rows, N = 2048, K = 6144: 16 x 16 8.9 us, 16 x 32 11.4, 32 x 32 14.9; N = K =
  // 4096: 11.3, 9.1, 10.8; M = 64: 18.4, 14.7, 10.9).  With more workgroups
  // than CUs the re-reads of A decide: 16 weight rows a workgroup up to M = 8
  // (N = K = 8192: M = 1 15.1, with 32 16.7; M = 8 16.9 and 17.0), 32 from there
  // (M = 12: 17.0, with 16 19.1; M = 16: 17.0 and 21.1).
  const bool one16 = outputs<16, 16>(M, N) <= kCUs;
  // Sixteen waves pay when few rows leave a long loop to the loads' latency
  // (M = 1, 16 and 8 waves: 12288 x 6144 15.7 / 16.6, 8192 x 8192 14.6 / 15.2, 4096
  // x 14336 12.9 / 15.0, 2048 x 16384 12.7 / 14.9, though 5120 x 8192 13.8 / 13.0;
  // M = 4 13.4 / 15.3 at 4096 x 14336; but 6144 x 4096 8.9 / 8.4, 14336 x 4096
  // 15.1 / 15.0; 2560 x 2048 4.4 / 4.1; M = 9 16.9 / 17.0, in 16 x 32, at 8192 x 8192).
  if (M <= 4 && K >= 48 * kBlock)
    return stream_cfg<16, 16, 2, 16, BROWS, true>(M, N, K, a, b, y, stream);
  if (M <= 8 || one16) return stream_cfg<16, 16, 4, 8, BROWS, true>(M, N, K, a, b, y, stream);
  if (M <= 16 || outputs<16, 32>(M, N) <= kCUs)
    return stream_cfg<16, 32, 2, 8, BROWS, true>(M, N, K, a, b, y, stream);
  return stream_cfg<32, 32, 2, 8, BROWS, WIDE>(M, N, K, a, b, y, stream);
}

// Outputs per workgroup of the experts' product, from the workgroups to be
// expected: one tile row for every expert that can have rows, or the rows'
// worth and half a tile more for each.  16 x 16 while they do not fill the
// card (2 experts with a row each, N = 1024, K = 4096: 6.2 us, 16 x 32 7.4,
// 64 x 128 in the ring 16.4).  Then 16 x 32 where one tile holds an expert's
// rows, else 32 x 32, up to four workgroups a CU: all of them run at once, so
// the time is little more than that of one loop over K.  More workgroups have
// their starts and ends to pay, those of experts without rows too, which 16 x 32
// makes good while there are at most twice as many as elements of a long K.
// Time in the ring over the time here, mean over routers' uneven rows (top 2 to
// 8 of 8 to 256 experts, N = 512 to 4096), by workgroups up to
//                 K    512  1024  2048  4096  8192  16384
//   16 x 32     512   1.42  1.17  0.81  0.73  0.62   0.52
//              2048   1.88  1.31  0.99  1.05  0.98   0.91
//              4096   1.79  1.31  1.15  1.22  1.15   1.06
//              6144   1.97  1.32  1.00  1.05  1.02   0.96
//     fp32     2048   2.32  1.56  1.08  1.16  1.10   0.99
//              6144   2.45  1.53  1.06  1.14  1.11   1.01
//   32 x 32     512   1.40  1.13  0.73  0.58  0.43
//              6144   1.81  1.28  0.86  0.70  0.47
//     fp32     2048   1.86  1.26  0.84  0.65  0.46
enum GroupedOutputs { kTiles, kRows16x16, kRows16x32, kRows32x32 };
GroupedOutputs grouped_outputs(int64_t G, int64_t total_m, int64_t N, int64_t K) {
  const int64_t live = G < total_m ? G : total_m;
  const int64_t more = total_m / 16 + live / 2, rows = more > live ? more : live;
  const int64_t more32 = total_m / 32 + live / 2, rows32 = more32 > live ? more32 : live;
  const int64_t n16 = (N + 15) / 16, n32 = (N + 31) / 32;
  if (rows * n16 <= kCUs) return kRows16x16;
  if (rows * n32 <= kCUs) return kRows16x32;
  if (more <= live) return rows * n32 <= (K >= 2048 ? 2 * K : 4 * kCUs) ? kRows16x32 : kTiles;
  return rows32 * n32 <= 4 * kCUs ? kRows32x32 : kTiles;
}

template <int BM, int BN, int UNROLL, int WAVES, bool GATHER, bool WIDE>
hipError_t grouped_cfg(int32_t G, const int32_t* m_offsets, const int32_t* row_index,
                       int64_t total_m, int64_t a_rows, int64_t N, int64_t K, Fp8Operand a,
                       Fp8Operand b, Fp8Out y, hipStream_t stream) {
  // an expert ends at most one tile that is not full
  const int64_t tiles = (total_m / BM + (G < total_m ? G : total_m)) * ((N + BN - 1) / BN);
  if (!grid_fits(tiles, 64 * WAVES)) return hipErrorNotSupported;
  fp8_grouped_stream_kernel<BM, BN, UNROLL, WAVES, GATHER, WIDE>
      <<<(unsigned)tiles, 64 * WAVES, 0, stream>>>(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y);
  return hipGetLastError();
}

template <bool GATHER, bool WIDE>
hipError_t grouped_rows(int32_t G, const int32_t* m_offsets, const int32_t* row_index,
                        int64_t total_m, int64_t a_rows, int64_t N, int64_t K, Fp8Operand a,
                        Fp8Operand b, Fp8Out y, hipStream_t stream) {
  switch (grouped_outputs(G, total_m, N, K)) {
    case kRows16x16:
      return grouped_cfg<16, 16, 4, 8, GATHER, true>(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y, stream);
    case kRows16x32:
      return grouped_cfg<16, 32, 2, 8, GATHER, true>(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y, stream);
    default:
      return grouped_cfg<32, 32, 2, 8, GATHER, WIDE>(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y, stream);
  }
}

}  // namespace

bool fp8_grouped_streams(int64_t G, int64_t total_m, int64_t N, int64_t K) {
  return grouped_outputs(G, total_m, N, K) != kTiles;
}

hipError_t launch_fp8_grouped_stream(int32_t G, const int32_t* m_offsets, const int32_t* row_index,
                                     int64_t total_m, int64_t a_rows, int64_t N, int64_t K,
                                     Fp8Operand a, Fp8Operand b, Fp8Out y, hipStream_t stream) {
  auto go = [&](auto wide) {
    constexpr bool W = decltype(wide)::value;
    return row_index != nullptr
               ? grouped_rows<true, W>(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y, stream)
               : grouped_rows<false, W>(G, m_offsets, row_index, total_m, a_rows, N, K, a, b, y, stream);
  };
  return y.dtype == 0 ? go(std::true_type{}) : go(std::false_type{});
}

// Up to 16 rows the weights' stream is all that counts (us, here and in tiles,
// bf16, then fp32 outputs: 1 x 16384 x 4096 15.7 16.7, 15.5 17.8; 16 x 4096 x 4096
// 7.6 11.3, 7.3 15.0; 16 x 65536 x 4096 60 69, 63 69; the most against it: 16 x
// 65536 x 2048 32.3 28.8, 32.5 33.1).  Otherwise as long as 32 x 32 outputs give
// every CU at most one workgroup (64 x 4096 x 512 4.4 4.8, 4.6 5.5; 64 x 4096 x
// 4096 11.1 13.6, 14.4 15.9; 512 x 512 x 8192 17.7 19.7, 22.3 26.6; the most
// against it: 32 x 8192 x 4096 12.8 13.2, 16.0 15.6; past it 32 x 12288 x 4096
// 20.3 15.8, 23.4 17.7; 128 x 4096 x 2048 11.0 8.6, 12.6 10.6; 512 x 1024 x 512
// 5.3 5.0, 6.0 5.7).  So one border serves both types.
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
