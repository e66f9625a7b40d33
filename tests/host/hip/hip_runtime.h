// Stand-in for the HIP runtime and for the gfx950 builtins that the FP8, INT8 and
// gradient kernels use, so that their sources compile for the host and run there
// (lanes.cpp runs the lanes).  For tests of indexing, waits and arithmetic without
// a GPU; it knows nothing of time, of the order of memory between waves beyond
// barriers, or of how the hardware rounds inside a matrix instruction.
#pragma once
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <functional>
#include <tuple>
#include <utility>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __shared__ static  // workgroups run one after another
#define __forceinline__ inline __attribute__((always_inline))
#define __launch_bounds__(...)

using std::max;
using std::min;
inline int64_t min(int64_t a, int b) { return a < b ? a : b; }
inline int64_t min(int a, int64_t b) { return a < b ? a : b; }

typedef int hipError_t;
typedef void* hipStream_t;
enum { hipSuccess = 0, hipErrorInvalidValue = 1, hipErrorNotSupported = 801 };
enum hipFuncAttribute { hipFuncAttributeMaxDynamicSharedMemorySize = 8 };
inline hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
inline hipError_t hipGetLastError() { return hipSuccess; }
inline hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }

namespace lanes {

struct Index {
  unsigned x, y, z;
};
extern Index block, grid;
Index thread();
int lane();
[[noreturn]] void fail(const char* what);

// ---- what lanes do together -----------------------------------------------

void barrier();
// One value of `size` bytes (at most 64) from every lane of the wave; returns the
// wave's values in lane order and a mask of the lanes that gave one.  Lanes that
// meet in exchanges of different sizes, or never, end the program.
const uint8_t* exchange(const void* value, size_t size, uint64_t* gave);
inline void wave_sync() {
  const uint8_t none = 0;
  uint64_t gave;
  exchange(&none, 1, &gave);
}

template <typename T>
inline T from_lane(T v, int l) {
  uint64_t gave;
  const uint8_t* all = exchange(&v, sizeof(T), &gave);
  if (!(gave >> l & 1)) fail("a value of a lane that is gone");
  T o;
  memcpy(&o, all + l * sizeof(T), sizeof(T));
  return o;
}
template <typename T>
inline T shfl_xor(T v, int d) {
  return from_lane(v, lane() ^ d);
}
template <typename T>
inline T shfl_up(T v, int d) {
  return from_lane(v, lane() >= d ? lane() - d : lane());
}
inline int readlane(int v, int l) { return from_lane(v, l); }
inline int readfirstlane(int v) {
  uint64_t gave;
  const uint8_t* all = exchange(&v, 4, &gave);
  int o;
  memcpy(&o, all + __builtin_ctzll(gave) * 4, 4);
  return o;
}
inline uint64_t ballot(bool p) {
  uint64_t gave, o = 0;
  const uint8_t b = p;
  const uint8_t* all = exchange(&b, 1, &gave);
  for (int i = 0; i < 64; ++i)
    if (gave >> i & 1 && all[i]) o |= 1ull << i;
  return o;
}
// The one data-parallel move in use: a rotation inside rows of 16 lanes.
inline int rotate16(int, int v, int control, int, int, bool) {
  if ((control & ~15) != 0x120) fail("a data-parallel move other than a rotation");
  return from_lane(v, (lane() & ~15) | ((lane() - (control & 15)) & 15));
}

// ---- buffers and LDS --------------------------------------------------------

uint8_t* dynamic_lds();
// A direct load's bytes: they land at once, or, in the late mode, when a wait asks
// for them.
void land(void* dst, const void* src, size_t n);
void wait_loads(int left);

struct Buffer {
  const uint8_t* p;
  uint32_t bytes;
};
inline Buffer make_buffer(const void* p, short, int bytes, int) { return {(const uint8_t*)p, (uint32_t)bytes}; }
// Words outside the buffer read as zeros.
inline void fetch(Buffer r, uint32_t at, uint32_t more, void* to, uint32_t n) {
  const uint64_t off = (uint64_t)at + more;
  for (uint32_t i = 0; i < n; i += 4) {
    uint8_t w[4] = {0, 0, 0, 0};
    if (off + i + 4 <= r.bytes)
      for (int k = 0; k < 4; ++k) w[k] = *(const volatile uint8_t*)(r.p + off + i + k);
    memcpy((uint8_t*)to + i, w, 4);
  }
}
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
inline u4 load128(Buffer r, uint32_t at, uint32_t more, int) {
  u4 w;
  fetch(r, at, more, &w, 16);
  return w;
}
inline uint32_t load32(Buffer r, uint32_t at, uint32_t more, int) {
  uint32_t w;
  fetch(r, at, more, &w, 4);
  return w;
}
inline void load_lds(Buffer r, void* lds, int n, uint32_t at, uint32_t more, int, int) {
  uint8_t b[16];
  fetch(r, at, more, b, n);
  land((uint8_t*)lds + lane() * n, b, n);
}
inline void waitcnt(int c) {
  const int loads = (c & 15) | ((c >> 14 & 3) << 4);
  if (loads < 63) wait_loads(loads);
}

// ---- arithmetic -------------------------------------------------------------

typedef float f4 __attribute__((ext_vector_type(4)));
typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

float e4m3(uint32_t b);
uint8_t to_e4m3(float v);
f4 mfma_fp8(i8 a, i8 b, f4 c, int, int, int, int, int, int);
f4 mfma_f16(h8 a, h8 b, f4 c, int, int, int);
i4 mfma_i8(i4 a, i4 b, i4 c, int, int, int);

inline int pack_fp8(float a, float b, int old, bool high) {
  const uint32_t w = to_e4m3(a) | (uint32_t)to_e4m3(b) << 8;
  return high ? (old & 0xFFFF) | (int)(w << 16) : (old & (int)0xFFFF0000) | (int)w;
}
inline h2 unpack_fp8(uint32_t w, float, bool high) {
  const uint32_t h = high ? w >> 16 : w;
  return h2{(_Float16)e4m3(h & 255), (_Float16)e4m3(h >> 8 & 255)};
}
// exp2 and the reciprocal as the hardware has them: inputs and results below the
// normal numbers are zeros.  (It is off by up to one unit in the last place more.)
inline float flush(float v) { return fabsf(v) < 0x1p-126f ? copysignf(0.f, v) : v; }
inline float rcp(float x) { return flush((float)(1.0 / (double)flush(x))); }
inline float exp2_(float x) { return flush((float)exp2((double)flush(x))); }

// ---- launches ---------------------------------------------------------------

void run(unsigned grid, unsigned threads, size_t lds, const std::function<void()>& kernel);

template <typename... P>
struct Launch {
  void (*kernel)(P...);
  unsigned grid, threads;
  size_t lds;
  void operator()(P... a) const {
    const std::tuple<P...> args{a...};
    run(grid, threads, lds, [&] { std::apply(kernel, args); });
  }
};
template <typename... P>
Launch<P...> launch(void (*kernel)(P...), unsigned grid, unsigned threads, size_t lds, hipStream_t) {
  return {kernel, grid, threads, lds};
}

}  // namespace lanes

inline float __uint_as_float(uint32_t u) {
  float f;
  memcpy(&f, &u, 4);
  return f;
}
inline uint32_t __float_as_uint(float f) {
  uint32_t u;
  memcpy(&u, &f, 4);
  return u;
}

#define threadIdx (lanes::thread())
#define blockIdx (lanes::block)
#define gridDim (lanes::grid)
#define __syncthreads() lanes::barrier()
#define __lane_id() lanes::lane()
#define __shfl_xor(v, d, width) lanes::shfl_xor(v, d)
#define __shfl_up(v, d, width) lanes::shfl_up(v, d)
#define __ballot(p) lanes::ballot(p)
#define __amdgpu_buffer_rsrc_t lanes::Buffer
#define __builtin_amdgcn_make_buffer_rsrc lanes::make_buffer
#define __builtin_amdgcn_raw_ptr_buffer_load_lds lanes::load_lds
#define __builtin_amdgcn_raw_buffer_load_b128 lanes::load128
#define __builtin_amdgcn_raw_buffer_load_b32 lanes::load32
#define __builtin_amdgcn_s_waitcnt lanes::waitcnt
#define __builtin_amdgcn_sched_barrier(mask) ((void)0)
#define __builtin_amdgcn_readlane lanes::readlane
#define __builtin_amdgcn_readfirstlane lanes::readfirstlane
#define __builtin_amdgcn_update_dpp lanes::rotate16
#define __builtin_amdgcn_cvt_pk_fp8_f32 lanes::pack_fp8
#define __builtin_amdgcn_cvt_scalef32_pk_f16_fp8 lanes::unpack_fp8
#define __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(...) (lanes::fail("an FP4 conversion"), lanes::h2{0, 0})
#define __builtin_amdgcn_cvt_f32_fp8(v, byte) lanes::e4m3((v) & 255)
#define __builtin_amdgcn_rcpf(x) lanes::rcp(x)
#define __builtin_amdgcn_exp2f(x) lanes::exp2_(x)
#define __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4 lanes::mfma_fp8
#define __builtin_amdgcn_mfma_f32_16x16x32_f16 lanes::mfma_f16
#define __builtin_amdgcn_mfma_i32_16x16x64_i8 lanes::mfma_i8
