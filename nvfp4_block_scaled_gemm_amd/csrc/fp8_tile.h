// One output tile of an FP8 block-128 product on the gfx950 matrix cores:
//
//   y[m, n] = sum_kb sa[kb, m] * sb[kb, n / b_rows] * sum_{k in block kb} qa[m, k] qb[n, k]
//
// E4M3 products are exact in fp32 and v_mfma_f32_16x16x128_f8f6f4 takes one
// whole block of 128 per instruction, so each instruction starts from zero
// and its result is one block's sum; the two fp32 scales multiply that sum
// on the vector unit as it is added to the fp32 accumulator (4 v_fma per
// matrix instruction of 32 cycles: 16 cycles on the vector unit, which runs
// beside the matrix core).  The 8-bit matrix rate is only reached through
// this instruction: the older 16x16x32 form runs at the 16-bit rate.
//
//  * A stage is one block of K: BM + BN rows of 128 bytes and one fp32 scale
//    per row, moved HBM -> LDS by direct loads into a ring.  Rows are
//    XOR-swizzled in 16-byte chunks so fragment reads spread over the banks;
//    the swizzle is applied to each lane's source address.
//  * The weights are the instruction's row operand and the activations its
//    column operand, so a lane's four results are four neighbouring output
//    columns of one token and the token's scale is one value per lane.  Rows
//    of W are dealt to the fragments so that two fragments give a lane eight
//    neighbouring columns: one 16-byte store of bf16.
//  * The accumulators must live in the 256 vector registers the vector unit
//    reaches (it adds into them), which bounds a wave to 128 x 64 outputs.
//  * WIDE (fp32 outputs) runs the block on the fp16 instructions instead,
//    which keep fp32 sums, at half the rate (fp8_device.h has the figures).
//  * Rows past the operand read as zeros by the descriptors' range; a last
//    block shorter than 128 reads zeros past K in both operands (K % 16 == 0,
//    so a 16-byte chunk is wholly inside or outside).
//
// Two other products run in the same tile:
//  * GATED, a gated block's: the weight rows are taken 32 of the gate, 32 of
//    the up projection in turn, so a wave's 64 rows give both factors of 32
//    outputs in the same lane, and the epilogue writes act(gate) * up (and the
//    two products, if they are kept).  The main loop differs in the two weight
//    scales alone.
//  * INT8, with one scale for each row of either operand: the sums are 32-bit
//    integers that stay in the accumulators to the end, the scales are applied
//    as the tile goes out, and a stage holds no scales.
// Both write eight neighbouring outputs a lane: whole 16-byte pieces of aligned rows
// (fp32 ones in pairs), else element by element.  The plain product's runs, and its
// column a lane for rows off 16 bytes, are not theirs.
#pragma once

#include "fp8_device.h"
#include "gated_act.h"

namespace nvfp4 {
namespace fp8 {

// One operand of a tile: rows of `q` (row stride `ld` bytes, given to run())
// and the scales of block kb at s + kb * s_ld.
struct TileOperand {
  const uint8_t* q;      // tile's first row (gathered: the whole operand)
  const float* s;        // scale of the tile's first row, block 0 (gathered: of row 0)
  int64_t s_ld;          // scales per block of K
  uint32_t q_bytes;      // readable bytes from q
  uint32_t s_bytes;      // readable bytes from s + kb * s_ld
  const int32_t* index;  // gathered rows (nullptr: rows in order)
  int32_t index_n;       // rows of the tile
  int32_t index_max;     // rows of the operand
  // gated weights: q points at the tile's first gate row, s at block 0 of the
  // whole weight's scales
  int64_t up_q = 0;       // bytes from a gate row to its up row
  int64_t row0 = 0;       // the tile's first gate row
  int64_t up = 0;         // rows from a gate row to its up row
  int shift = 0;          // rows per scale, as a power of two
};

struct TileOut {
  void* y;        // element (0, 0) of the tile
  int64_t ld;     // elements
  int32_t m, n;   // rows and columns of the tile that exist
  int dtype;      // 0 fp32, 1 bf16
  bool add;       // fp32: y += product
  bool vec;       // rows are 16-byte aligned
  // gated: where the two products go in bf16 (nullptr: nowhere)
  void* gate = nullptr;
  void* upto = nullptr;
  int64_t ld2 = 0;
  bool vec2 = false;
  int act = kSilu;
};

  // Eight neighbouring outputs of one row (those below out.n).
  __device__ __forceinline__ void store8(const TileOut& out, int m, int n, const float* v) {
    const int64_t at = (int64_t)m * out.ld + n;
    if (out.vec && n + 8 <= out.n) {
      if (out.dtype == 1) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(
                                                  f32x2{v[2 * e], v[2 * e + 1]}, bf16x2));
        *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(out.y) + at) = w;
      } else {
        f32x4* p = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(out.y) + at);
        f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
        if (out.add) {
          lo += p[0];
          hi += p[1];
        }
        p[0] = lo;
        p[1] = hi;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < out.n) {
          if (out.dtype == 1) {
            reinterpret_cast<__bf16*>(out.y)[at + e] = (__bf16)v[e];
          } else {
            float* p = reinterpret_cast<float*>(out.y) + at + e;
            *p = out.add ? *p + v[e] : v[e];
          }
        }
    }
  }

// KG: groups of WM x WN waves that take the blocks of K in turn, each with a
// ring of its own, and add their sums at the end (in group order): small
// tiles spend a step mostly on meeting and on LDS latency, so fewer steps with
// two waves on each SIMD pay.
template <int BM, int BN, int WM, int WN, int STAGES, int KG, bool BROWS, bool WIDE,
          bool GATED = false, bool INT8 = false>
struct Tile {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves * KG;
  static constexpr int TM = BM / WM, TN = BN / WN;
  static constexpr int FM = TM / 16, FN = TN / 16;
  static constexpr int kALoads = BM / 8 / kWaves, kBLoads = BN / 8 / kWaves;
  static constexpr int kScales = INT8 ? 0 : (BM + BN) / 64;  // scale-load instructions of a stage
  static constexpr int kSLoads = (kScales + kWaves - 1) / kWaves;
  static constexpr int kLoads = kALoads + kBLoads + kSLoads;  // per wave and stage
  static constexpr int kAOff = 0, kBOff = BM * kBlock, kSOff = (BM + BN) * kBlock;
  static constexpr int kStage = kSOff + (INT8 ? 0 : (BM + BN) * 4);
  static constexpr int kSmem = KG * STAGES * kStage;
  static_assert((KG - 1) * BM * BN * 4 <= kSmem, "the groups' sums fit the rings");
  static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "whole loads per wave");
  static_assert((kALoads & (kALoads - 1)) == 0 && (kBLoads & (kBLoads - 1)) == 0,
                "the loads' row bits are disjoint");
  static_assert(BM % 64 == 0 && BN % 64 == 0 && TN % 32 == 0 && TM % 16 == 0, "fragment shapes");
  static_assert(BROWS || 128 % TN == 0, "one weight scale per wave and block");
  static_assert(FM % 2 == 0 && FN >= 2, "pairs of fragments");
  static_assert((STAGES - 1) * kLoads < 64, "vmcnt range");
  static_assert(!GATED || (TN == 64 && kBLoads <= 4), "a wave's weight loads are all of one projection");
  static_assert(!INT8 || (!BROWS && !WIDE && !GATED), "integers have one kind of product");
  using Acc = std::conditional_t<INT8, i32x4, f32x4>;

  // 16 lanes of an activation fragment read rows r .. r + 15: two rows share
  // a 256-byte bank line, so the chunk moves with row / 2.
  static __device__ __forceinline__ int swz_a(int r) { return (r >> 1) & 7; }
  // 16 lanes of a weight fragment read rows 8 * (l / 4) + l % 4 (+ 4): the
  // chunk moves with row bits 1, 3 and 4.
  static __device__ __forceinline__ int swz_b(int r) { return ((r >> 1) & 1) | ((r >> 2) & 6); }

  // K: elements of the sum; ld: bytes between rows of both operands.
  template <bool GATHER>
  static __device__ __forceinline__ void run(const TileOperand& A, const TileOperand& B, uint32_t K,
                                             uint32_t ld, const TileOut& out, uint8_t* smem_all) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave = wave_all % kWaves, kg = wave_all / kWaves;
    uint8_t* const smem = smem_all + kg * STAGES * kStage;
    const int wm = wave / WN, wn = wave % WN;
    const int li = lane & 15, lg = lane >> 4;
    const int nk = (int)((K + kBlock - 1) / kBlock), steps = (nk + KG - 1) / KG;
    // plain copies: a choice between two fields stays a choice of registers
    const uint8_t* const aq = A.q;
    // gated: this wave loads 32 (16) rows of one of the projections
    const bool up_wave = GATED && (wave * kBLoads * 8) % 64 >= 32;
    const uint8_t* const bq = B.q + (GATED && up_wave ? B.up_q : 0);
    const float *const as = A.s, *const bs = B.s;
    const int64_t as_ld = A.s_ld, bs_ld = B.s_ld;
    const uint32_t aq_bytes = A.q_bytes, bq_bytes = B.q_bytes, as_bytes = A.s_bytes, bs_bytes = B.s_bytes;

    uint32_t a_off[kALoads], b_off[kBLoads], s_off[kSLoads ? kSLoads : 1];
    // a load's 16-byte chunk of its rows; rows 8 apart only flip fixed bits
    const int lr = lane >> 3;
    const uint32_t a_chunk = (uint32_t)(((lane & 7) ^ swz_a(wave * kALoads * 8 + lr)) << 4);
    const uint32_t b_chunk = (uint32_t)(((lane & 7) ^ swz_b(wave * kBLoads * 8 + lr)) << 4);
#pragma unroll
    for (int i = 0; i < kALoads; ++i) {
      const int r = (wave * kALoads + i) * 8 + (lane >> 3);
      uint32_t row = (uint32_t)r;
      bool ok = true;
      if constexpr (GATHER) {
        const int32_t v = r < A.index_n ? A.index[r] : -1;
        ok = v >= 0 && v < A.index_max;
        row = (uint32_t)v;
      }
      a_off[i] = ok ? row * ld + (a_chunk ^ (swz_a(i * 8) << 4)) : kNoRow;
    }
#pragma unroll
    for (int i = 0; i < kBLoads; ++i) {
      const int r = (wave * kBLoads + i) * 8 + (lane >> 3);
      const int row = GATED ? (r >> 6) * 32 + (r & 31) : r;
      b_off[i] = (uint32_t)row * ld + (b_chunk ^ (swz_b(i * 8) << 4));
    }
    // chunks of the last block that lie past K: lane masks in scalar
    // registers, so a stage's loads need no branch (one would let the
    // compiler move the products' additions across it)
    const uint32_t end = K - (uint32_t)(nk - 1) * kBlock;
    bool a_past[kALoads], b_past[kBLoads];
#pragma unroll
    for (int i = 0; i < kALoads; ++i) a_past[i] = (a_chunk ^ (uint32_t)(swz_a(i * 8) << 4)) >= end;
#pragma unroll
    for (int i = 0; i < kBLoads; ++i) b_past[i] = (b_chunk ^ (uint32_t)(swz_b(i * 8) << 4)) >= end;
    // scale loads: instruction j < BM / 64 takes the activations' rows, the
    // others the weights'; waves past the last repeat one (same bytes, same
    // place), so every wave issues the same number of loads
    bool s_is_a[kSLoads ? kSLoads : 1];
    int s_slot[kSLoads ? kSLoads : 1];
#pragma unroll
    for (int i = 0; i < kSLoads; ++i) {
      const int j = (wave * kSLoads + i) % (kScales ? kScales : 1);
      s_slot[i] = j;
      s_is_a[i] = j < BM / 64;
      const int r = (s_is_a[i] ? j : j - BM / 64) * 64 + lane;
      if (s_is_a[i]) {
        uint32_t row = (uint32_t)r;
        bool ok = true;
        if constexpr (GATHER) {
          const int32_t v = r < A.index_n ? A.index[r] : -1;
          ok = v >= 0 && v < A.index_max;
          row = (uint32_t)v;
        }
        s_off[i] = ok ? row * 4 : kNoRow;
      } else if constexpr (GATED) {
        const int64_t row = B.row0 + (r >> 6) * 32 + (r & 31) + ((r & 32) ? B.up : 0);
        s_off[i] = (uint32_t)(row >> B.shift) * 4;
      } else {
        s_off[i] = (uint32_t)(BROWS ? r : r / kBlock) * 4;
      }
    }

    // load number J (0 .. kLoads - 1) of stage s into ring slot `slot`; past
    // the last block every lane is out of range (zeros into a slot that is
    // not read again)
    auto load_one = [&](int s, int slot, auto jc) {
      constexpr int J = decltype(jc)::value;
      uint8_t* base = smem + slot * kStage;
      const int kb = s * KG + kg;
      const bool live = kb < nk, cut = kb == nk - 1;
      const uint32_t soff = (uint32_t)kb * kBlock;
      if constexpr (J < kBLoads) {
        constexpr int i = J;
        load_lds16(make_rsrc(bq, live ? bq_bytes : 0u), base + kBOff + (wave * kBLoads + i) * 1024,
                   cut && b_past[i] ? kNoRow : b_off[i], soff);
      } else if constexpr (J < kBLoads + kALoads) {
        constexpr int i = J - kBLoads;
        load_lds16(make_rsrc(aq, live ? aq_bytes : 0u), base + kAOff + (wave * kALoads + i) * 1024,
                   cut && a_past[i] ? kNoRow : a_off[i], soff);
      } else {
        constexpr int i = J - kBLoads - kALoads;
        const float* p = s_is_a[i] ? as : bs;
        const int64_t at = (int64_t)max(min(kb, nk - 1), 0) * (s_is_a[i] ? as_ld : bs_ld);
        const uint32_t bytes = s_is_a[i] ? as_bytes : bs_bytes;
        load_lds4(make_rsrc(p + at, live ? bytes : 0u), base + kSOff + s_slot[i] * 256, s_off[i], 0);
      }
    };
    auto issue = [&](int s, int slot, auto n) {
      static_for<decltype(n)::value>([&](auto jc) { load_one(s, slot, jc); });
    };

    Acc acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = Acc{0, 0, 0, 0};

    // fragments: a lane takes chunks lg and lg + 4 of its row in both
    // operands (the swizzles do not depend on the fragment's number)
    const int b_row0 = wn * TN + 8 * (li >> 2) + (li & 3), a_row0 = wm * TM + li;
    const int b_sw = swz_b(b_row0), a_sw = swz_a(a_row0);
    const int b_at = kBOff + b_row0 * kBlock, a_at = kAOff + a_row0 * kBlock;
    auto read = [&](const uint8_t* p, int sw) {
      return join(*reinterpret_cast<const u32x4*>(p + ((lg ^ sw) << 4)),
                  *reinterpret_cast<const u32x4*>(p + (((lg + 4) ^ sw) << 4)));
    };
    auto read_b = [&](const uint8_t* st, int i) {
      return read(st + b_at + (32 * (i >> 1) + 4 * (i & 1)) * kBlock, b_sw);
    };
    auto read_a = [&](const uint8_t* st, int j) { return read(st + a_at + 16 * j * kBlock, a_sw); };
    auto scales = [&](const uint8_t* st) { return reinterpret_cast<const float*>(st + kSOff); };

    // The loop works on pairs of activation fragments: a pair meets all FN
    // weight fragments while the next pair is read.  In a stage's last pair
    // the workgroup meets (the next stage has landed, this one has been read
    // by all), its slot is refilled and the next stage's first pair and
    // weight fragments are read, each into the registers of the fragment just
    // used -- so the matrix core does not wait for LDS at a stage's start.
    // The refill goes out one load at a time over the Q / 2 products from the
    // meeting on (into the next stage): a wave that issues all of them at
    // once waits for the address unit with its products behind it.
    // A product's result is added two products later, when it is ready.
    using Frag = decltype(fragment<WIDE>(i32x8{}));
    constexpr int PAIRS = FM / 2, PER = 2 * FN, Q = PAIRS * PER;
    i32x8 br[FN], ar[2];
    float fw[GATED ? 2 : 1];
    f32x4 fb[BROWS ? FN : 1];
    f32x4 cq[3];
    Frag bw[FN], aw[2];

    constexpr int MEET = (PAIRS - 1) * PER, SPREAD = Q / 2;
    constexpr int EARLY = ((Q - MEET) * kLoads + SPREAD - 1) / SPREAD < kLoads
                              ? ((Q - MEET) * kLoads + SPREAD - 1) / SPREAD
                              : kLoads;  // loads that go out in the stage of the meeting
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) issue(s, s, std::integral_constant<int, kLoads>{});
    issue(STAGES - 1, STAGES - 1, std::integral_constant<int, EARLY>{});
    wait_vmcnt<(STAGES - 2) * kLoads + EARLY>();
    workgroup_barrier();
    if (wm * TM >= out.m || wn * (GATED ? TN / 2 : TN) >= out.n) {
      // no output of this wave exists (a group's last rows): it only loads
      // and meets the others, and leaves the matrix core to the wave beside it
      int slot = 0;
      for (int s = 0; s < steps; ++s) {
        static_for<kLoads - EARLY>([&](auto nc) {
          load_one(s + STAGES - 1, slot == 0 ? STAGES - 1 : slot - 1, std::integral_constant<int, EARLY + decltype(nc)::value>{});
        });
        wait_vmcnt<(STAGES - 2) * kLoads>();
        workgroup_barrier();
        issue(s + STAGES, slot, std::integral_constant<int, EARLY>{});
        slot = slot + 1 == STAGES ? 0 : slot + 1;
      }
      wait_vmcnt<0>();
      workgroup_barrier();  // the others' turn to the ring for their outputs
      if constexpr (KG > 1) workgroup_barrier();
      return;
    }
#pragma unroll
    for (int i = 0; i < FN; ++i) br[i] = read_b(smem, i);
#pragma unroll
    for (int h = 0; h < 2; ++h) ar[h] = read_a(smem, h);
    int slot = 0;
    for (int s = 0; s < steps; ++s) {
      const uint8_t* st = smem + slot * kStage;
      const int next = slot + 1 == STAGES ? 0 : slot + 1;
      const uint8_t* nst = smem + next * kStage;
      const float* sc = scales(st);
      // scale of a row of A times that of W's block; gated: of either projection
      float fall[GATED && !BROWS ? 2 : 1][FM];
      if constexpr (INT8) {
      } else if constexpr (BROWS) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
          fb[i] = *reinterpret_cast<const f32x4*>(sc + BM + wn * TN + 32 * (i >> 1) + 8 * lg + 4 * (i & 1));
      } else {
        fw[0] = sc[BM + wn * TN];
        if constexpr (GATED) fw[1] = sc[BM + wn * TN + 32];
      }
      if constexpr (!INT8) {
#pragma unroll
        for (int j = 0; j < FM; ++j) fall[0][j] = sc[a_row0 + 16 * j];
      }
      i32x8 an[2];
      auto add = [&](auto qc) {
        constexpr int q = decltype(qc)::value, p = q / PER, i = (q % PER) / 2, h = q % 2, j = 2 * p + h;
        if constexpr (!INT8) {
          const f32x4& c = cq[q % 3];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float f = BROWS ? fb[BROWS ? i : 0][e] * fall[0][j] : fall[GATED && !BROWS ? i >> 1 : 0][j];
            acc[i][j][e] = __builtin_fmaf(c[e], f, acc[i][j][e]);
          }
        }
      };
      static_for<Q>([&](auto qc) {
        constexpr int q = decltype(qc)::value, p = q / PER, r = q % PER, i = r / 2, h = r % 2;
        constexpr bool last = p == PAIRS - 1;
        if constexpr (r == 0) {
          if constexpr (last) {
            // this wave's reads of the stage are done, its loads of the next
            // one have landed
            wait_lgkmcnt0();
            wait_vmcnt<(STAGES - 2) * kLoads>();
          }
          aw[0] = fragment<WIDE>(ar[0]);
          aw[1] = fragment<WIDE>(ar[1]);
        }
        if constexpr (p == 0 && h == 0) bw[i] = fragment<WIDE>(br[i]);
        if constexpr (p == 0 && r == 0 && !BROWS && !INT8) {
#pragma unroll
          for (int j = 0; j < FM; ++j) {
            if constexpr (GATED) fall[1][j] = fall[0][j] * fw[1];
            fall[0][j] *= fw[0];
          }
        }
        if constexpr (INT8) {
          // the block's halves in turn over the pair, so that a sum is used
          // again two instructions later
#pragma unroll
          for (int k = 0; k < 2; ++k) acc[i][2 * p + k] = mfma_half<h>(bw[i], aw[k], acc[i][2 * p + k]);
        } else {
          cq[q % 3] = mfma_block(bw[i], aw[h]);
        }
        if constexpr (q >= 2) add(std::integral_constant<int, q - 2>{});
        if constexpr (last && r == 0) workgroup_barrier();
        // refill: load n at MEET + n * SPREAD / kLoads, counted on into the
        // next stage
        static_for<kLoads>([&](auto nc) {
          constexpr int n = decltype(nc)::value, at = MEET + n * SPREAD / kLoads;
          if constexpr (at == q) load_one(s + STAGES, slot, nc);
          if constexpr (at - Q == q) load_one(s + STAGES - 1, slot == 0 ? STAGES - 1 : slot - 1, nc);
        });
        // the next pair (of this stage or the next), then the next stage's
        // weights behind their last use
        if constexpr (!last) {
          if constexpr (r == 0) an[0] = read_a(st, 2 * p + 2);
          if constexpr (r == 1) an[1] = read_a(st, 2 * p + 3);
        } else {
          if constexpr (r == 1) an[0] = read_a(nst, 0);
          if constexpr (r == 3) an[1] = read_a(nst, 1);
          if constexpr (h == 1) br[i] = read_b(nst, i);
        }
        if constexpr (r == PER - 1) {
          ar[0] = an[0];
          ar[1] = an[1];
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      add(std::integral_constant<int, Q - 2>{});
      add(std::integral_constant<int, Q - 1>{});
      slot = next;
    }
    // the ring's last loads land before the slots can be written again
    wait_vmcnt<0>();

    // The wave's tile goes out through its own part of the idle ring, in
    // passes of 32 rows: lanes write what they hold, then read whole row
    // pieces, so that a store covers runs of TN elements instead of four.
    // (LDS accesses of one wave complete in order.)
    workgroup_barrier();
    if constexpr (KG > 1) {
      // the other groups' sums, each lane's own outputs
      Acc* sums = reinterpret_cast<Acc*>(smem_all) + wave * (FM * FN * 64) + lane;
      constexpr int kGroupSums = kWaves * FM * FN * 64;
      if (kg > 0) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j) sums[(kg - 1) * kGroupSums + (i * FM + j) * 64] = acc[i][j];
      }
      __syncthreads();
      if (kg > 0) return;
#pragma unroll
      for (int g = 0; g < KG - 1; ++g)
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j) acc[i][j] += sums[g * kGroupSums + (i * FM + j) * 64];
    }
    constexpr int RS = TN + 4;  // floats per staged row; + 4 spreads the banks
    constexpr int kStageAt = (KG - 1) * BM * BN;  // floats: behind the groups' sums
    static_assert((kStageAt + kWaves * 32 * RS) * 4 <= kSmem, "staging fits the ring");
    float* stage = reinterpret_cast<float*>(smem_all) + kStageAt + wave * 32 * RS;
    if constexpr (GATED) {
      // eight outputs a lane: their gates and, 32 columns on, their ups
      const TileOut gate{out.gate, out.ld2, out.m, out.n, 1, false, out.vec2};
      const TileOut up{out.upto, out.ld2, out.m, out.n, 1, false, out.vec2};
#pragma unroll
      for (int j2 = 0; j2 < FM / 2; ++j2) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < FN; ++i)
            *reinterpret_cast<f32x4*>(stage + (16 * h + li) * RS + 32 * (i >> 1) + 8 * lg + 4 * (i & 1)) = acc[i][2 * j2 + h];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int r = p * 16 + lane / 4, c = lane % 4 * 8;
          const int m = wm * TM + 32 * j2 + r, n = wn * 32 + c;
          float g[8], u[8], v[8];
          const f32x4* at = reinterpret_cast<const f32x4*>(stage + r * RS + c);
          const f32x4 g0 = at[0], g1 = at[1], u0 = at[8], u1 = at[9];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            g[e] = g0[e];
            g[4 + e] = g1[e];
            u[e] = u0[e];
            u[4 + e] = u1[e];
          }
          gated8(out.act, g, u, v);
          if (m < out.m) {
            store8(out, m, n, v);
            if (out.gate != nullptr) {
              store8(gate, m, n, g);
              store8(up, m, n, u);
            }
          }
        }
      }
      return;
    }
    constexpr int LPR = TN / 8, RPI = 64 / LPR;  // lanes per row, rows per read
    constexpr int NP = 32 / RPI;
    // Whole aligned rows leave in 16-byte pieces, fp32 ones as two runs TN / 2
    // columns apart (what they add to is read ahead of everything, in one
    // go); other rows element by element, a lane a column.
    const bool runs = out.vec && (wn + 1) * TN <= out.n;
    float col_scale[8];
    if constexpr (INT8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) col_scale[e] = B.s[min(wn * TN + 8 * (lane % LPR) + e, out.n - 1)];
    }
    float* const y32 = reinterpret_cast<float*>(out.y) + wn * TN + 4 * (lane % LPR);
    f32x4 old[WIDE ? FM / 2 : 1][WIDE ? NP : 1][2];
    if constexpr (WIDE) {
      if (runs && out.add) {
#pragma unroll
        for (int j2 = 0; j2 < FM / 2; ++j2)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const int m = min(wm * TM + 32 * j2 + p * RPI + lane / LPR, out.m - 1);
            const float* y = y32 + (int64_t)m * out.ld;
            old[j2][p][0] = *reinterpret_cast<const f32x4*>(y);
            old[j2][p][1] = *reinterpret_cast<const f32x4*>(y + TN / 2);
          }
      } else {
#pragma unroll
        for (int j2 = 0; j2 < FM / 2; ++j2)
#pragma unroll
          for (int p = 0; p < NP; ++p) old[j2][p][0] = old[j2][p][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
#pragma unroll
    for (int j2 = 0; j2 < FM / 2; ++j2) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < FN; ++i)
          *reinterpret_cast<Acc*>(stage + (16 * h + li) * RS + 32 * (i >> 1) + 8 * lg + 4 * (i & 1)) = acc[i][2 * j2 + h];
      if constexpr (INT8) {
        // eight outputs a lane, each an integer times its row's and its column's scale
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int r = p * RPI + lane / LPR, c = 8 * (lane % LPR);
          const int m = wm * TM + 32 * j2 + r, n = wn * TN + c;
          const i32x4 lo = *reinterpret_cast<const i32x4*>(stage + r * RS + c);
          const i32x4 hi = *reinterpret_cast<const i32x4*>(stage + r * RS + c + 4);
          if (m < out.m) {
            const float sm = A.s[m];
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)(e < 4 ? lo[e & 3] : hi[e & 3]) * sm * col_scale[e];
            store8(out, m, n, v);
          }
        }
      } else if (runs) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int r = p * RPI + lane / LPR, c = lane % LPR;
          const int m = wm * TM + 32 * j2 + r;
          if constexpr (WIDE) {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(stage + r * RS + 4 * c);
            const f32x4 hi = *reinterpret_cast<const f32x4*>(stage + r * RS + TN / 2 + 4 * c);
            if (m < out.m) {
              float* y = y32 + (int64_t)m * out.ld;
              *reinterpret_cast<f32x4*>(y) = lo + old[j2][p][0];
              *reinterpret_cast<f32x4*>(y + TN / 2) = hi + old[j2][p][1];
            }
          } else {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(stage + r * RS + 8 * c);
            const f32x4 hi = *reinterpret_cast<const f32x4*>(stage + r * RS + 8 * c + 4);
            const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            if (m < out.m) store8(out, m, wn * TN + 8 * c, v);
          }
        }
      } else {
#pragma unroll 4
        for (int e = lane; e < 32 * TN; e += 64) {
          const int r = e / TN, c = e % TN;
          const int m = wm * TM + 32 * j2 + r, n = wn * TN + c;
          if (m >= out.m || n >= out.n) continue;
          const int64_t at = (int64_t)m * out.ld + n;
          const float v = stage[r * RS + c];
          if constexpr (WIDE) {
            float* y = reinterpret_cast<float*>(out.y) + at;
            *y = out.add ? *y + v : v;
          } else {
            reinterpret_cast<__bf16*>(out.y)[at] = (__bf16)v;
          }
        }
      }
    }
  }
};

}  // namespace fp8
}  // namespace nvfp4
