// Gated feed-forward block on FP8 operands, dense and per expert:
//
//   h = act(x Wg^T) * (x Wu^T),   W = [Wg; Wu] [2F, K]
//
// one product of 2F weight rows whose tiles take gate and up rows of the same
// outputs (fp8_tile.h), so both factors of an output meet in one lane and only h
// leaves; for training the two products leave too, in bf16.  Bound as the
// product of N = 2F is: by the matrix cores for many rows, by the weights'
// stream for few.
//
// Few rows: a workgroup owns BM x BC outputs, 2 BC weight rows, and its waves
// take the blocks of K in turn, straight into fragment registers; their partial
// sums meet in LDS and are added in wave order, as in fp8_stream.hip.
#include <type_traits>

#include "fp8_launch.h"

namespace nvfp4 {
namespace {

using namespace fp8;

// Outputs of rows m0 .. m0 + m, columns n0 .. n0 + n of h.
__device__ __forceinline__ TileOut out_of(const GatedOutput& y, int64_t m0, int64_t n0, int m, int n) {
  TileOut o{(uint8_t*)y.h.y + (m0 * y.h.ld + n0) * (y.h.dtype == 0 ? 4 : 2), y.h.ld, m, n, y.h.dtype, false, y.h.vec};
  o.act = y.act;
  if (y.gate_up != nullptr) {
    o.gate = reinterpret_cast<uint16_t*>(y.gate_up) + m0 * y.ld2 + n0;
    o.upto = reinterpret_cast<uint16_t*>(y.gate_up) + m0 * y.ld2 + y.F + n0;
    o.ld2 = y.ld2;
    o.vec2 = y.vec2;
  }
  return o;
}

// Rows n0 .. n0 + n of both projections of a weight [2F, K] with s_ld scales
// per block of K, one for each 2^shift rows.
__device__ __forceinline__ TileOperand weight_of(const uint8_t* q, const float* s, int64_t s_ld, int shift,
                                                 int64_t n0, int n, int64_t F, int64_t K) {
  TileOperand b{q + n0 * K, s, s_ld, (uint32_t)(n * K), (uint32_t)s_ld * 4, nullptr, 0, 0};
  b.up_q = F * K;
  b.row0 = n0;
  b.up = F;
  b.shift = shift;
  return b;
}

__device__ __forceinline__ TileOperand rows_of(const Fp8Operand& a, int64_t rows, int64_t m0, int m, int64_t K) {
  return {a.q + m0 * K, a.s + m0, rows, (uint32_t)(m * K), (uint32_t)m * 4, nullptr, 0, 0};
}

// BM x BN / 2 outputs.
template <int BM, int BN, int WM, int WN, int STAGES, bool BROWS, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN, 2) void gated_dense_kernel(int64_t M, int64_t F, int64_t K, Fp8Operand a,
                                                                     Fp8Operand b, int64_t s_ld, int shift,
                                                                     GatedOutput y) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int BC = BN / 2;
  const int tiles_m = (int)ceil_div(M, BM), tiles_n = (int)ceil_div(F, BC);
  // groups of 8 tile rows, walked column by column
  const int pid = xcd_run(blockIdx.x, gridDim.x);
  const int group = pid / (8 * tiles_n), first = group * 8, gsz = min(tiles_m - first, 8);
  const int in = pid - group * 8 * tiles_n;
  const int64_t m0 = (int64_t)(first + in % gsz) * BM, n0 = (int64_t)(in / gsz) * BC;
  const int rm = (int)min((int64_t)BM, M - m0), rn = (int)min((int64_t)BC, F - n0);
  using T = Tile<BM, BN, WM, WN, STAGES, 1, BROWS, WIDE, true>;
  T::template run<false>(rows_of(a, M, m0, rm, K), weight_of(b.q, b.s, s_ld, shift, n0, rn, F, K), (uint32_t)K,
                         (uint32_t)K, out_of(y, m0, n0, rm, rn), smem);
}

// A tile in the list of (expert, tile column, tile row) tiles, which only the
// device knows: each wave keeps 64 experts' running tile counts in its lanes and
// finds a tile's expert by one ballot.
template <int BM>
struct ExpertTiles {
  int G;
  const int32_t* offsets;
  int64_t total_m, tiles_n;
  int64_t before = 0;  // tile rows of the experts below e0
  int e0 = 0;
  Segment sg;
  uint32_t upto;

  __device__ __forceinline__ void load() {
    const int e = e0 + (threadIdx.x & 63);
    sg = e < G ? segment(offsets, e, total_m) : Segment{0, 0};
    upto = wave_scan((uint32_t)((sg.n + BM - 1) / BM));
  }
  // Finds tile u (not below the last one asked for): its expert, the expert's
  // rows and tile rows, and its place among the expert's tiles.
  __device__ __forceinline__ bool find(int64_t u, int& e, int32_t& lo, int32_t& n, int32_t& rows, int32_t& at) {
    uint32_t all = __builtin_amdgcn_readlane(upto, 63);
    while (u >= (before + all) * tiles_n) {
      before += all;
      e0 += 64;
      if (e0 >= G) return false;
      load();
      all = __builtin_amdgcn_readlane(upto, 63);
    }
    const int64_t v = u - before * tiles_n;
    const int l = __builtin_ctzll(__ballot((int64_t)upto * tiles_n > v));
    const int64_t start = l == 0 ? 0 : (int64_t)__builtin_amdgcn_readlane(upto, l - 1);
    lo = __builtin_amdgcn_readlane(sg.lo, l);
    n = __builtin_amdgcn_readlane(sg.n, l);
    rows = (n + BM - 1) / BM;
    at = (int32_t)(v - start * tiles_n);
    e = e0 + l;
    return true;
  }
};

// Experts' rows: workgroups walk the tiles, tile rows fastest so that
// neighbours share a weight tile.  (The walk and three outputs' addresses spill 56 to
// 70 scalar registers into lanes of vector registers in every shape, where the plain
// experts' product spills 21 to 35, and 6 to 12 vector registers in the 256 x 256 shape:
// stored before and read after a tile's loop over K, never in it.  The dense kernels
// spill nothing.)
template <int BM, int BN, int WM, int WN, int STAGES, bool GATHER, bool BROWS, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN, 2) void gated_grouped_kernel(
    int G, const int32_t* __restrict__ offsets, const int32_t* __restrict__ row_index, int64_t total_m,
    int64_t a_rows, int64_t F, int64_t K, Fp8Operand a, Fp8Operand b, GatedOutput y) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int BC = BN / 2;
  using T = Tile<BM, BN, WM, WN, STAGES, 1, BROWS, WIDE, true>;
  const int64_t nb = ceil_div(2 * F, kBlock), kb = ceil_div(K, kBlock);
  ExpertTiles<BM> tiles{G, offsets, total_m, ceil_div(F, BC)};
  tiles.load();
  for (int64_t u = xcd_run(blockIdx.x, gridDim.x);; u += gridDim.x) {
    int e;
    int32_t lo, n, te, w;
    if (!tiles.find(u, e, lo, n, te, w)) return;
    const int32_t tm = w % te, tn = w / te;
    const int64_t m0 = lo + (int64_t)tm * BM, n0 = (int64_t)tn * BC;
    const int rm = min(BM, n - tm * BM), rn = (int)min((int64_t)BC, F - n0);
    TileOperand A;
    if constexpr (GATHER)
      A = {a.q, a.s, a_rows, (uint32_t)(a_rows * K), (uint32_t)a_rows * 4, row_index + m0, rm, (int32_t)a_rows};
    else
      A = rows_of(a, total_m, m0, rm, K);
    const TileOperand B = weight_of(b.q + (int64_t)e * 2 * F * K, b.s + e * kb * nb, nb, 7, n0, rn, F, K);
    T::template run<GATHER>(A, B, (uint32_t)K, (uint32_t)K, out_of(y, m0, n0, rm, rn), smem);
    workgroup_barrier();  // every wave is past its last fragment reads
  }
}

// ---- few rows ---------------------------------------------------------------

__device__ __forceinline__ i32x8 load_fragment(__amdgpu_buffer_rsrc_t r, uint32_t lo, uint32_t hi, uint32_t soff) {
  const auto a = __builtin_amdgcn_raw_buffer_load_b128(r, lo, soff, 0);
  const auto b = __builtin_amdgcn_raw_buffer_load_b128(r, hi, soff, 0);
  return join(__builtin_bit_cast(u32x4, a), __builtin_bit_cast(u32x4, b));
}

// Rows of A: lane li of fragment j takes row 16 j + li, whose bytes and scale
// are at the offsets (kNoRow: zeros).
template <int FM>
struct StreamRows {
  const uint8_t* q;
  const float* s;
  int64_t s_ld;
  uint32_t q_bytes, s_bytes;
  uint32_t q_off[FM], s_off[FM];
};

template <int FM>
__device__ __forceinline__ StreamRows<FM> stream_rows_of(const Fp8Operand& a, int64_t rows, int64_t m0, int n,
                                                         int64_t K) {
  StreamRows<FM> r{a.q + m0 * K, a.s + m0, rows, (uint32_t)n * (uint32_t)K, (uint32_t)n * 4, {}, {}};
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const uint32_t row = 16 * j + (threadIdx.x & 15);
    r.q_off[j] = row * (uint32_t)K;
    r.s_off[j] = row * 4;
  }
  return r;
}

// BM x BC outputs: fragment i holds 16 weight rows of the gate (i < BC / 16) or
// the up projection.
template <int BM, int BC, int UNROLL, int WAVES, bool BROWS, bool WIDE>
__device__ __forceinline__ void stream_gated(const StreamRows<BM / 16>& A, const TileOperand& B, int64_t K,
                                             const TileOut& out) {
  constexpr int FM = BM / 16, FH = BC / 16, FN = 2 * FH;
  __shared__ __attribute__((aligned(16))) float part[WAVES][BM][2 * BC];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const int nk = (int)((K + kBlock - 1) / kBlock);
  const uint32_t ld = (uint32_t)K, end = (uint32_t)K - (uint32_t)(nk - 1) * kBlock;
  const bool lo_past = (uint32_t)lg * 16 >= end, hi_past = (uint32_t)(lg + 4) * 16 >= end;
  const auto ra = make_rsrc(A.q, A.q_bytes);
  const auto rg = make_rsrc(B.q, B.q_bytes), ru = make_rsrc(B.q + B.up_q, B.q_bytes);
  uint32_t a_off[FM], b_off[FN], bs_off[FN];
#pragma unroll
  for (int j = 0; j < FM; ++j) a_off[j] = A.q_off[j] + lg * 16;
#pragma unroll
  for (int i = 0; i < FN; ++i) {
    b_off[i] = (uint32_t)(16 * (i % FH) + li) * ld + lg * 16;
    // of the first of a lane's four outputs
    const int64_t row = B.row0 + 16 * (i % FH) + 4 * lg + (i >= FH ? B.up : 0);
    bs_off[i] = (uint32_t)row;
  }
  f32x4 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int k0 = wave; k0 < nk; k0 += WAVES * UNROLL) {
    i32x8 bf[UNROLL][FN], af[UNROLL][FM];
    float sa[UNROLL][FM], sw[UNROLL][2];
    f32x4 sb[UNROLL][BROWS ? FN : 1];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int kb = k0 + u * WAVES;
      const bool none = kb >= nk, cut = kb == nk - 1;
#pragma unroll
      for (int i = 0; i < FN; ++i)
        bf[u][i] = load_fragment(i < FH ? rg : ru, none || (cut && lo_past) ? kNoRow : b_off[i],
                                 none || (cut && hi_past) ? kNoRow : b_off[i] + 64, (uint32_t)kb * kBlock);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int kb = k0 + u * WAVES;
      const bool none = kb >= nk, cut = kb == nk - 1;
      const int64_t at = none ? 0 : kb;
      const auto rsa = make_rsrc(A.s + at * A.s_ld, none ? 0u : A.s_bytes);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        af[u][j] = load_fragment(ra, none || (cut && lo_past) ? kNoRow : a_off[j],
                                 none || (cut && hi_past) ? kNoRow : a_off[j] + 64, (uint32_t)kb * kBlock);
        sa[u][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsa, A.s_off[j], 0, 0));
      }
      const float* s = B.s + at * B.s_ld;
      if constexpr (BROWS) {
        const auto rsb = make_rsrc(s, none ? 0u : B.s_bytes);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sb[u][i][e] = __uint_as_float(
                __builtin_amdgcn_raw_buffer_load_b32(rsb, ((bs_off[i] + e) >> B.shift) * 4, 0, 0));
      } else {
        // a workgroup's rows of either projection lie in one block of 128
        sw[u][0] = s[B.row0 >> 7];
        sw[u][1] = s[(B.row0 + B.up) >> 7];
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (k0 + u * WAVES >= nk) break;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const auto bw = fragment<WIDE>(bf[u][i]);
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          const f32x4 c = mfma_block(bw, fragment<WIDE>(af[u][j]));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j][e] = __builtin_fmaf(c[e], sa[u][j] * (BROWS ? sb[u][BROWS ? i : 0][e] : sw[u][i / FH]), acc[i][j][e]);
        }
      }
    }
  }

#pragma unroll
  for (int j = 0; j < FM; ++j)
#pragma unroll
    for (int i = 0; i < FN; ++i)
      *reinterpret_cast<f32x4*>(&part[wave][16 * j + li][16 * i + 4 * lg]) = acc[i][j];
  __syncthreads();
  const TileOut gate{out.gate, out.ld2, out.m, out.n, 1, false, out.vec2};
  const TileOut up{out.upto, out.ld2, out.m, out.n, 1, false, out.vec2};
  for (int t = tid; t < BM * BC / 8; t += 64 * WAVES) {
    const int m = t / (BC / 8), n = t % (BC / 8) * 8;
    if (m >= out.m || n >= out.n) continue;
    float g[8], p[8], v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = p[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        g[e] += part[w][m][n + e];
        p[e] += part[w][m][BC + n + e];
      }
    gated8(out.act, g, p, v);
    store8(out, m, n, v);
    if (out.gate != nullptr) {
      store8(gate, m, n, g);
      store8(up, m, n, p);
    }
  }
}

template <int BM, int BC, int UNROLL, int WAVES, bool BROWS, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void gated_stream_kernel(int64_t M, int64_t F, int64_t K, Fp8Operand a,
                                                                  Fp8Operand b, int64_t s_ld, int shift,
                                                                  GatedOutput y) {
  const int64_t tiles_n = (F + BC - 1) / BC;
  const int64_t m0 = blockIdx.x / tiles_n * BM, n0 = blockIdx.x % tiles_n * BC;
  const int rm = (int)min((int64_t)BM, M - m0), rn = (int)min((int64_t)BC, F - n0);
  stream_gated<BM, BC, UNROLL, WAVES, BROWS, WIDE>(stream_rows_of<BM / 16>(a, M, m0, rm, K),
                                                        weight_of(b.q, b.s, s_ld, shift, n0, rn, F, K), K,
                                                        out_of(y, m0, n0, rm, rn));
}

// Experts' few rows, eight tile columns of an expert's rows in turn, so that
// the rows of one column share its XCD's L2.
template <int BM, int BC, int UNROLL, int WAVES, bool GATHER, bool BROWS, bool WIDE>
__global__ __launch_bounds__(64 * WAVES) void gated_grouped_stream_kernel(
    int G, const int32_t* __restrict__ offsets, const int32_t* __restrict__ row_index, int64_t total_m,
    int64_t a_rows, int64_t F, int64_t K, Fp8Operand a, Fp8Operand b, GatedOutput y) {
  const int lane = threadIdx.x & 63;
  const int64_t tiles_n = (F + BC - 1) / BC, nb = (2 * F + kBlock - 1) / kBlock, kb = (K + kBlock - 1) / kBlock;
  ExpertTiles<BM> tiles{G, offsets, total_m, tiles_n};
  tiles.load();
  int e;
  int32_t lo, n, te, w;
  if (!tiles.find(blockIdx.x, e, lo, n, te, w)) return;
  const int64_t eight = w / (8 * te) * 8;
  const int32_t in = (int32_t)(w - eight * te), cols = (int32_t)min(tiles_n - eight, (int64_t)8);
  const int32_t tm = in / cols;
  const int64_t m0 = lo + (int64_t)tm * BM, n0 = (eight + in % cols) * BC;
  const int rm = min(BM, n - tm * BM), rn = (int)min((int64_t)BC, F - n0);
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
    A = stream_rows_of<BM / 16>(a, total_m, m0, rm, K);
  }
  stream_gated<BM, BC, UNROLL, WAVES, BROWS, WIDE>(
      A, weight_of(b.q + (int64_t)e * 2 * F * K, b.s + e * kb * nb, nb, 7, n0, rn, F, K), K, out_of(y, m0, n0, rm, rn));
}

// ---- launches ---------------------------------------------------------------

struct Dense {
  int64_t M, F, K;
  Fp8Operand a, b;
  int64_t s_ld;
  int shift;
  GatedOutput y;
  hipStream_t stream;
};

struct Grouped {
  int32_t G;
  const int32_t *m_offsets, *row_index;
  int64_t total_m, a_rows, F, K;
  Fp8Operand a, b;
  GatedOutput y;
  hipStream_t stream;
};

template <typename S, bool BROWS, bool WIDE>
hipError_t dense(const Dense& d) {
  using T = Tile<S::BM, S::BN, S::WM, S::WN, S::S, 1, BROWS, WIDE, true>;
  auto kern = gated_dense_kernel<S::BM, S::BN, S::WM, S::WN, S::S, BROWS, WIDE>;
  const int64_t tiles = tiles_of(d.M, d.F, S::BM, S::BN / 2);
  if (!grid_fits(tiles, T::kThreads)) return hipErrorNotSupported;
  static std::atomic<uint64_t> done{0};
  const hipError_t err = allow_lds(kern, T::kSmem, done);
  if (err != hipSuccess) return err;
  kern<<<(unsigned)tiles, T::kThreads, T::kSmem, d.stream>>>(d.M, d.F, d.K, d.a, d.b, d.s_ld, d.shift, d.y);
  return hipGetLastError();
}

template <int BM, int BC, int UNROLL, int WAVES, bool BROWS, bool WIDE>
hipError_t stream(const Dense& d) {
  const int64_t tiles = tiles_of(d.M, d.F, BM, BC);
  if (!grid_fits(tiles, 64 * WAVES)) return hipErrorNotSupported;
  gated_stream_kernel<BM, BC, UNROLL, WAVES, BROWS, WIDE>
      <<<(unsigned)tiles, 64 * WAVES, 0, d.stream>>>(d.M, d.F, d.K, d.a, d.b, d.s_ld, d.shift, d.y);
  return hipGetLastError();
}

// The FP8 products' times at N = 2F (fp8_stream.hip, fp8_gemm.hip), since loads and
// loops are theirs; no border was measured here.  Their shapes for 17 to some 600
// rows are missing: 64 x 64 and 128 x 64, whose waves take 32 weight rows and split K
// in two (a wave's 64 rows hold both projections here).  By those times M = 32, F = K =
// 8192 takes 128 tiles of 64 x 128 and 0.60 us a block of K, where the plain product of
// 2F columns takes 0.35: 38 us against 22 and an activation.  16-row tiles take the
// 16-bit instructions and their fp32 sums, as there.
template <bool BROWS, bool WIDE>
hipError_t dense_any(const Dense& d) {
  const int64_t M = d.M, F = d.F;
  if (M <= 4 && d.K >= 48 * kBlock) return stream<16, 16, 1, 16, BROWS, true>(d);
  if (M <= 16) return stream<16, 16, 2, 8, BROWS, true>(d);
  if (tiles_of(M, F, 32, 16) <= 256) return stream<32, 16, 2, 8, BROWS, WIDE>(d);
  if constexpr (WIDE) {
    const int64_t small = tiles_cost(tiles_of(M, F, 64, 64), 90, 140);
    const int64_t middle = tiles_cost(tiles_of(M, F, 128, 64), 126, 206);
    return middle < small ? dense<S128x128, BROWS, true>(d) : dense<S64x128, BROWS, true>(d);
  } else {
    const int64_t cost[4] = {tiles_cost(tiles_of(M, F, 64, 64), 60, 97), tiles_cost(tiles_of(M, F, 128, 64), 90, 122),
                             tiles_cost(tiles_of(M, F, 128, 128), 118, 236),
                             tiles_cost(tiles_of(M, F, 256, 128), 170, 340)};
    int best = 0;
    for (int i = 1; i < 4; ++i)
      if (cost[i] < cost[best]) best = i;
    if (best == 3) return dense<S256x256, BROWS, false>(d);
    if (best == 2) return dense<S128x256, BROWS, false>(d);
    if (best == 1) return dense<S128x128, BROWS, false>(d);
    return dense<S64x128, BROWS, false>(d);
  }
}

template <typename S, bool GATHER, bool BROWS, bool WIDE>
hipError_t grouped(const Grouped& g) {
  using T = Tile<S::BM, S::BN, S::WM, S::WN, S::S, 1, BROWS, WIDE, true>;
  auto kern = gated_grouped_kernel<S::BM, S::BN, S::WM, S::WN, S::S, GATHER, BROWS, WIDE>;
  static std::atomic<uint64_t> done{0};
  const hipError_t err = allow_lds(kern, T::kSmem, done);
  if (err != hipSuccess) return err;
  constexpr unsigned per_cu = T::kSmem > 80 * 1024 ? 1 : 2;
  kern<<<256 * per_cu, T::kThreads, T::kSmem, g.stream>>>(g.G, g.m_offsets, g.row_index, g.total_m, g.a_rows, g.F, g.K,
                                                         g.a, g.b, g.y);
  return hipGetLastError();
}

template <int BM, int BC, int UNROLL, int WAVES, bool GATHER, bool BROWS, bool WIDE>
hipError_t grouped_stream(const Grouped& g) {
  // an expert ends at most one tile that is not full
  const int64_t tiles = (g.total_m / BM + (g.G < g.total_m ? g.G : g.total_m)) * ((g.F + BC - 1) / BC);
  if (!grid_fits(tiles, 64 * WAVES)) return hipErrorNotSupported;
  gated_grouped_stream_kernel<BM, BC, UNROLL, WAVES, GATHER, BROWS, WIDE>
      <<<(unsigned)tiles, 64 * WAVES, 0, g.stream>>>(g.G, g.m_offsets, g.row_index, g.total_m, g.a_rows, g.F, g.K,
                                                     g.a, g.b, g.y);
  return hipGetLastError();
}

// The counts are on the device.  Expected tile rows: one for every expert that
// can have rows, or the rows' worth and half a tile more for each.  The borders are
// those of the experts' FP8 products at N = 2F, not timed here.
template <bool GATHER, bool BROWS, bool WIDE>
hipError_t grouped_any(const Grouped& g) {
  const int64_t live = g.G < g.total_m ? g.G : g.total_m;
  auto rows = [&](int64_t bm) {
    const int64_t more = g.total_m / bm + live / 2;
    return more > live ? more : live;
  };
  const int64_t outs = (g.F + 15) / 16;
  if (g.total_m / 16 + live / 2 <= live ? rows(16) * outs <= (g.K >= 2048 ? 2 * g.K : 1024) : rows(16) * outs <= 256)
    return grouped_stream<16, 16, 2, 8, GATHER, BROWS, true>(g);
  if (rows(32) * outs <= 1024) return grouped_stream<32, 16, 2, 8, GATHER, BROWS, WIDE>(g);
  auto cost = [&](int64_t bm, int64_t bc, int64_t t1, int64_t t2) {
    return tiles_cost(rows(bm) * ((g.F + bc - 1) / bc), t1, t2);
  };
  const int64_t small = WIDE ? cost(64, 64, 90, 140) : cost(64, 64, 60, 97);
  const int64_t middle = WIDE ? cost(128, 64, 126, 206) : cost(128, 64, 90, 122);
  if constexpr (!WIDE) {
    const int64_t large = cost(256, 128, 170, 340);
    if (large < small && large < middle) return grouped<S256x256, GATHER, BROWS, WIDE>(g);
  }
  if (middle < small) return grouped<S128x128, GATHER, BROWS, WIDE>(g);
  return grouped<S64x128, GATHER, BROWS, WIDE>(g);
}

// Calls f with the kind of weight scales and the output's width as constants.
template <typename F>
hipError_t by_kind(bool brows, int dtype, F&& f) {
  auto wide = [&](auto b) { return dtype == 0 ? f(b, std::true_type{}) : f(b, std::false_type{}); };
  return brows ? wide(std::true_type{}) : wide(std::false_type{});
}

}  // namespace

hipError_t launch_fp8_gated(int64_t M, int64_t F, int64_t K, Fp8Operand a, Fp8Operand b, int b_block_rows,
                            GatedOutput y, hipStream_t st) {
  // one scale for a tile's rows of a projection only where F is a multiple of
  // 32; elsewhere a block of 128 rows can end inside them
  const bool brows = b_block_rows == 1 || F % 32 != 0;
  const int64_t s_ld = b_block_rows == 1 ? 2 * F : (2 * F + kBlock - 1) / kBlock;
  const Dense d{M, F, K, a, b, s_ld, b_block_rows == 1 ? 0 : 7, y, st};
  return by_kind(brows, y.h.dtype,
                 [&](auto b_, auto w) { return dense_any<decltype(b_)::value, decltype(w)::value>(d); });
}

hipError_t launch_fp8_grouped_gated(int32_t G, const int32_t* m_offsets, const int32_t* row_index, int64_t total_m,
                                    int64_t a_rows, int64_t F, int64_t K, Fp8Operand a, Fp8Operand b, GatedOutput y,
                                    hipStream_t st) {
  const Grouped g{G, m_offsets, row_index, total_m, a_rows, F, K, a, b, y, st};
  return by_kind(F % 32 != 0, y.h.dtype, [&](auto b_, auto w) {
    constexpr bool B = decltype(b_)::value, W = decltype(w)::value;
    return row_index != nullptr ? grouped_any<true, B, W>(g) : grouped_any<false, B, W>(g);
  });
}

}  // namespace nvfp4
