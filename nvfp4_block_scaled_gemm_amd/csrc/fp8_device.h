// Device-side helpers shared by the FP8 block-128 kernels (gfx950 only).
//
// Operand format: E4M3FN bytes q [rows, K] and one fp32 scale per 128
// elements of K for each row (block_rows 1) or each 128 rows (block_rows
// 128), stored K-block-major: s [ceil(K / 128), ceil(rows / block_rows)].
// K-block-major, because a product's step over one block of 128 then reads
// the scales of its rows as one contiguous run.
#pragma once

#include "nvfp4_device.h"

namespace nvfp4 {
namespace fp8 {

constexpr int kBlock = 128;      // elements of K under one scale

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_void_ptr;

// An offset no buffer of these kernels reaches (every descriptor covers less
// than 2^31 bytes): such a lane reads zeros.
constexpr uint32_t kNoRow = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

// Direct buffer -> LDS loads: lane L's 16 (4) bytes land at lds + L * 16 (4);
// offsets past the descriptor's range write zeros.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t voff,
                                           uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_ptr)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t voff,
                                          uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_ptr)lds, 4, voff, soff, 0, 0);
}

// s_waitcnt with only vmcnt constrained.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}
// s_waitcnt with only lgkmcnt constrained to 0.
__device__ __forceinline__ void wait_lgkmcnt0() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
}
// Workgroup barrier that is a compiler memory barrier too, without draining
// the loads in flight (each wave waits for its own before arriving).
__device__ __forceinline__ void workgroup_barrier() { asm volatile("s_barrier" ::: "memory"); }

// 16 x 16 product over one whole block of 128 E4M3 elements, from zero: lane
// L gives 32 bytes of row (column) L % 16 of each operand and receives rows
// 4 * (L / 16) + 0..3 of column L % 16.  Which 32 of the 128 elements a lane
// gives is free as long as both operands agree (a sum has no order).  The
// format codes 0 select E4M3; the unit scales (0) select the unscaled form.
__device__ __forceinline__ f32x4 mfma_block(const i32x8& a, const i32x8& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                                                          0, 0, 0);
}

__device__ __forceinline__ i32x8 join(const u32x4& lo, const u32x4& hi) {
  return __builtin_shufflevector(__builtin_bit_cast(i32x4, lo), __builtin_bit_cast(i32x4, hi), 0, 1,
                                 2, 3, 4, 5, 6, 7);
}

// The same block on the 16-bit matrix instructions: E4M3 values are fp16
// values, so converting loses nothing, and these instructions keep fp32
// sums.  The 8-bit ones align the products of a block to the largest of their
// running sums and cut each 2^-16 below it (the same for all four 8-bit
// forms): at most 127 * 2^-16 < 2^-9 of the sum of the block's magnitudes.
// Measured, of that sum: 2^-12 for random codes, 2^-10.2 for outliers that
// cancel in pairs; 1.5e-5 of the result for normal data.  A bf16 result's own
// rounding, up to 2^-8, hides that unless large products cancel; an fp32
// result would show it.
// Step t of four takes dwords 2t and 2t + 1 of the lane's 32 bytes.
struct F16Block {
  f16x8 v[4];
};
__device__ __forceinline__ F16Block widen(const i32x8& w) {
  F16Block o;
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)w[d], 1.0f, false);
    const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)w[d], 1.0f, true);
    o.v[d >> 1][4 * (d & 1) + 0] = lo[0];
    o.v[d >> 1][4 * (d & 1) + 1] = lo[1];
    o.v[d >> 1][4 * (d & 1) + 2] = hi[0];
    o.v[d >> 1][4 * (d & 1) + 3] = hi[1];
  }
  return o;
}
__device__ __forceinline__ f32x4 mfma_block(const F16Block& a, const F16Block& b) {
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < 4; ++t) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[t], b.v[t], c, 0, 0, 0);
  return c;
}

// The same block in 8-bit integers, one half of it (64 elements) added to 32-bit
// sums: half h is the lane's chunk h of 16 bytes in both operands.
template <int H>
__device__ __forceinline__ i32x4 mfma_half(const i32x8& a, const i32x8& b, const i32x4& c) {
  const i32x4 x = __builtin_shufflevector(a, a, 4 * H, 4 * H + 1, 4 * H + 2, 4 * H + 3);
  const i32x4 y = __builtin_shufflevector(b, b, 4 * H, 4 * H + 1, 4 * H + 2, 4 * H + 3);
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, y, c, 0, 0, 0);
}

// A fragment as the matrix instructions take it.
template <bool WIDE>
__device__ __forceinline__ auto fragment(const i32x8& w) {
  if constexpr (WIDE) return widen(w);
  else return w;
}

// Four fp32 -> four E4M3 bytes, round to nearest even (inputs within +-448
// after rounding).
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

// Group e of a list of offsets, kept inside [0, total] whatever they hold.
struct Segment {
  int32_t lo, n;
};
__device__ __forceinline__ Segment segment(const int32_t* __restrict__ off, int32_t e,
                                           int64_t total) {
  int64_t lo = off[e], hi = off[e + 1];
  lo = lo < 0 ? 0 : (lo > total ? total : lo);
  hi = hi > total ? total : hi;
  return {(int32_t)lo, (int32_t)(hi > lo ? hi - lo : 0)};
}

// Inclusive sum over the 64 lanes of a wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  const int lane = __lane_id();
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(v, d, 64);
    if (lane >= d) v += o;
  }
  return v;
}

}  // namespace fp8
}  // namespace nvfp4
