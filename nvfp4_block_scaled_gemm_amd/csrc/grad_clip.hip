// Norm and clipping of many gradients:
//
//   n2 = sum over all tensors of g^2,   g' = g * (max_norm / sqrt(n2))  where sqrt(n2) > max_norm
//
// Bound by HBM: two reads and a write, a few operations an element.  Squares,
// sums, the coefficient and the product are fp64 (the vector unit's fp64 rate is
// several times what the reads need): nothing overflows or is lost in a long
// sum, and a value is rounded once, on its way out.
//
// A launch takes a table of up to kPiece tensors as its argument.  All of
// their elements, in units of kUnit, are dealt to the workgroups in equal
// contiguous runs, so one search of the table serves a run and tensors of any
// size keep the card busy (up to 2048 workgroups: two rounds of the norm's 110 registers;
// the scaling's 66 leave 256 of them to a second one).  Each workgroup leaves one partial sum; whoever
// needs the norm adds the partials in the same fixed order, so results do not
// change between calls and no atomics are needed.
#include "nvfp4_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 112;         // tensors of a launch (the table is an argument: below 4 KB)
constexpr int64_t kUnit = 2048;     // elements: eight a thread
constexpr int kGroups = 2048;       // workgroups of a launch, partial sums of a piece

struct Table {
  const void* g[kPiece];
  void* out[kPiece];
  int64_t n[kPiece];
  uint32_t first[kPiece + 1];  // units before the tensor
  uint8_t types[kPiece];       // bit 0: g is bf16, bit 1: out is bf16
  int count;
};
static_assert(sizeof(Table) <= 3840, "kernel arguments stay below 4 KB");

// Tensor of unit u: the last one that starts at or before it (tensors without
// elements share their start with the next one).
__device__ __forceinline__ int tensor_of(const Table& t, uint32_t u) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Calls f(tensor, first element, end element) for each piece of a tensor in
// this workgroup's run of units.
template <typename F>
__device__ __forceinline__ void for_runs(const Table& t, F&& f) {
  const uint32_t units = t.first[t.count];
  const uint32_t u0 = (uint32_t)((uint64_t)units * blockIdx.x / gridDim.x);
  const uint32_t u1 = (uint32_t)((uint64_t)units * (blockIdx.x + 1) / gridDim.x);
  if (u0 >= u1) return;
  int i = tensor_of(t, u0);
  for (uint32_t u = u0; u < u1; ++i) {
    const uint32_t a = t.first[i], b = t.first[i + 1];
    const uint32_t to = b < u1 ? b : u1;
    if (u < to) {
      const int64_t e0 = (int64_t)(u - a) * kUnit;
      int64_t e1 = (int64_t)(to - a) * kUnit;
      if (e1 > t.n[i]) e1 = t.n[i];
      f(i, e0, e1);
      u = to;
    }
  }
}

__device__ __forceinline__ float bf16_at(const void* p, int64_t i) {
  return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16);
}

// Adds the 64 lanes' values, the same for every lane.
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Sum over the workgroup in a fixed order (all threads receive it).
__device__ __forceinline__ double group_sum(double v) {
  __shared__ double part[kThreads / 64];
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) s += part[i];
  return s;
}

// Elements of p before the first 16-byte border (at most `n`).
template <int ES>
__device__ __forceinline__ int64_t head_of(const void* p, int64_t n) {
  const int64_t h = (int64_t)((16 - ((uintptr_t)p & 15)) & 15) / ES;
  return h < n ? h : n;
}

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (DT == 1) return bf16_at(p, i);
  else return reinterpret_cast<const float*>(p)[i];
}

template <int DT>
__device__ __forceinline__ void square16(const u32x4& w, double* acc) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == 1) {
      const double a = __uint_as_float(w[k] << 16), b = __uint_as_float(w[k] & 0xFFFF0000u);
      acc[0] = __builtin_fma(a, a, acc[0]);
      acc[1] = __builtin_fma(b, b, acc[1]);
    } else {
      const double a = __uint_as_float(w[k]);
      acc[k & 1] = __builtin_fma(a, a, acc[k & 1]);
    }
  }
}

template <int DT>
__device__ __forceinline__ void square_run(const void* g, int64_t e0, int64_t e1, double* acc) {
  constexpr int ES = DT == 1 ? 2 : 4, V = 16 / ES, U = 8;
  const uint8_t* p = reinterpret_cast<const uint8_t*>(g) + e0 * ES;
  const int64_t n = e1 - e0, h = head_of<ES>(p, n), body = (n - h) / V, tail = h + body * V;
  const int tid = threadIdx.x;
  for (int64_t i = tid; i < h + (n - tail); i += kThreads) {
    const double a = load1<DT>(p, i < h ? i : tail + i - h);
    acc[0] = __builtin_fma(a, a, acc[0]);
  }
  const u32x4* v = reinterpret_cast<const u32x4*>(p + h * ES);
  int64_t i = tid;
  for (; i + (U - 1) * kThreads < body; i += U * kThreads) {
    u32x4 w[U];
#pragma unroll
    for (int k = 0; k < U; ++k) w[k] = v[i + k * kThreads];
#pragma unroll
    for (int k = 0; k < U; ++k) square16<DT>(w[k], acc);
  }
  for (; i < body; i += kThreads) square16<DT>(v[i], acc);
}

__global__ __launch_bounds__(kThreads) void grad_square_kernel(const Table t, double* __restrict__ partial) {
  double acc[2] = {0, 0};
  for_runs(t, [&](int i, int64_t e0, int64_t e1) {
    if (t.types[i] & 1) square_run<1>(t.g[i], e0, e1, acc);
    else square_run<0>(t.g[i], e0, e1, acc);
  });
  const double s = group_sum(acc[0] + acc[1]);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// Sum of the partials, in an order that depends on their number alone.
__device__ __forceinline__ double total_of(const double* __restrict__ partial, int64_t count) {
  double s = 0;
  for (int64_t i = threadIdx.x; i < count; i += kThreads) s += partial[i];
  return group_sum(s);
}

__global__ __launch_bounds__(kThreads) void grad_total_kernel(const double* __restrict__ partial, int64_t count,
                                                              double* __restrict__ norm_sq) {
  const double s = total_of(partial, count);
  if (threadIdx.x == 0) *norm_sq = s;
}

// A run of one tensor, 16-byte pieces on both sides where both reach a border
// after the same few elements; else element by element.
template <int DI, int DO>
__device__ __forceinline__ void scale_run(const void* g, void* out, int64_t e0, int64_t e1, double c) {
  constexpr int EI = DI == 1 ? 2 : 4, EO = DO == 1 ? 2 : 4;
  constexpr int E = 16 / (EI < EO ? EI : EO);      // elements a thread takes at once
  constexpr int NI = E * EI / 16, NO = E * EO / 16, U = 16 / E;
  const uint8_t* p = reinterpret_cast<const uint8_t*>(g) + e0 * EI;
  uint8_t* q = reinterpret_cast<uint8_t*>(out) + e0 * EO;
  const int64_t n = e1 - e0;
  const int tid = threadIdx.x;
  auto one = [&](int64_t i) {
    const float v = (float)(load1<DI>(p, i) * c);
    if constexpr (DO == 1) reinterpret_cast<__bf16*>(q)[i] = (__bf16)v;
    else reinterpret_cast<float*>(q)[i] = v;
  };
  int64_t h = 0;
  while (h < 8 && ((((uintptr_t)p + h * EI) | ((uintptr_t)q + h * EO)) & 15) != 0) ++h;
  if (h == 8 || h > n) {
    for (int64_t i = tid; i < n; i += kThreads) one(i);
    return;
  }
  const int64_t body = (n - h) / E, tail = h + body * E;
  for (int64_t i = tid; i < h + (n - tail); i += kThreads) one(i < h ? i : tail + i - h);
  const u32x4* v = reinterpret_cast<const u32x4*>(p + h * EI);
  u32x4* w = reinterpret_cast<u32x4*>(q + h * EO);
  auto put = [&](int64_t i, const u32x4* r) {
    float f[E];
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const uint32_t w32 = DI == 1 ? (k & 1 ? r[0][k >> 1] & 0xFFFF0000u : r[0][k >> 1] << 16) : r[DI == 1 ? 0 : k >> 2][k & 3];
      f[k] = (float)(__uint_as_float(w32) * c);
    }
#pragma unroll
    for (int j = 0; j < NO; ++j) {
      u32x4 o;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (DO == 1)
          o[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{f[2 * k], f[2 * k + 1]}, bf16x2));
        else
          o[k] = __float_as_uint(f[4 * j + k]);
      }
      w[i * NO + j] = o;
    }
  };
  int64_t i = tid;
  for (; i + (U - 1) * kThreads < body; i += U * kThreads) {
    u32x4 r[U][NI];
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int j = 0; j < NI; ++j) r[k][j] = v[(i + k * kThreads) * NI + j];
#pragma unroll
    for (int k = 0; k < U; ++k) put(i + k * kThreads, r[k]);
  }
  for (; i < body; i += kThreads) {
    u32x4 r[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) r[j] = v[i * NI + j];
    put(i, r);
  }
}

// count > 0: the sum of squares is that of the partials; else *norm_sq.
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const Table t, const double* __restrict__ sums,
                                                              int64_t count, double max_norm,
                                                              float* __restrict__ norm_out) {
  const double n2 = count > 0 ? total_of(sums, count) : *sums;
  const double norm = __builtin_sqrt(n2);
  if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  const bool clip = norm > max_norm && norm < __builtin_inf();
  const double c = clip ? max_norm / norm : 1.0;
  for_runs(t, [&](int i, int64_t e0, int64_t e1) {
    const void* g = t.g[i];
    void* out = t.out[i];
    if (!clip && out == g) return;
    switch (t.types[i]) {
      case 0: return scale_run<0, 0>(g, out, e0, e1, c);
      case 1: return scale_run<1, 0>(g, out, e0, e1, c);
      case 2: return scale_run<0, 1>(g, out, e0, e1, c);
      default: return scale_run<1, 1>(g, out, e0, e1, c);
    }
  });
}

// The tables of a list, piece by piece: f(table, workgroups).  An empty list
// is one empty piece.
template <typename F>
hipError_t for_pieces(int64_t count, const nvfp4_grad* grads, F&& f) {
  Table t;
  int64_t at = 0;
  do {
    t.count = 0;
    uint64_t units = 0;
    t.first[0] = 0;
    for (; at < count && t.count < kPiece; ++at) {
      const nvfp4_grad& g = grads[at];
      t.g[t.count] = g.g;
      t.out[t.count] = g.out != nullptr ? g.out : g.g;
      t.n[t.count] = g.n;
      t.types[t.count] = (uint8_t)((int)g.g_dtype | ((int)g.out_dtype << 1));
      units += (uint64_t)((g.n + kUnit - 1) / kUnit);
      t.first[++t.count] = (uint32_t)units;
    }
    const unsigned groups = (unsigned)(units < kGroups ? (units > 0 ? units : 1) : kGroups);
    const hipError_t e = f(t, groups);
    if (e != hipSuccess) return e;
  } while (at < count);
  return hipSuccess;
}

hipError_t launch_partials(int64_t count, const nvfp4_grad* grads, double* partial, int64_t* made,
                           hipStream_t stream) {
  *made = 0;
  return for_pieces(count, grads, [&](const Table& t, unsigned groups) {
    grad_square_kernel<<<groups, kThreads, 0, stream>>>(t, partial + *made);
    *made += groups;
    return hipGetLastError();
  });
}

}  // namespace

// Partial sums of every piece, and their total.
size_t grad_workspace_bytes(int64_t count) {
  const int64_t pieces = count > kPiece ? (count + kPiece - 1) / kPiece : 1;
  return (size_t)(pieces * kGroups + 1) * sizeof(double);
}

hipError_t launch_grad_norm_sq(int64_t count, const nvfp4_grad* grads, double* norm_sq, double* workspace,
                               hipStream_t stream) {
  int64_t made = 0;
  const hipError_t e = launch_partials(count, grads, workspace, &made, stream);
  if (e != hipSuccess) return e;
  grad_total_kernel<<<1, kThreads, 0, stream>>>(workspace, made, norm_sq);
  return hipGetLastError();
}

hipError_t launch_clip_grads(int64_t count, const nvfp4_grad* grads, double max_norm, const double* norm_sq,
                             float* norm, double* workspace, hipStream_t stream) {
  // The workgroups that scale add the partials themselves: one launch less.
  // Those of many pieces are added once instead.
  int64_t made = 0;
  if (norm_sq == nullptr) {
    hipError_t e = launch_partials(count, grads, workspace, &made, stream);
    if (e != hipSuccess) return e;
    norm_sq = workspace;
    if (made > 2 * kGroups) {
      double* total = workspace + grad_workspace_bytes(count) / sizeof(double) - 1;
      grad_total_kernel<<<1, kThreads, 0, stream>>>(workspace, made, total);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      norm_sq = total;
      made = 0;
    }
  }
  return for_pieces(count, grads, [&](const Table& t, unsigned groups) {
    grad_scale_kernel<<<groups, kThreads, 0, stream>>>(t, norm_sq, made, max_norm, norm);
    norm = nullptr;  // once is enough
    return hipGetLastError();
  });
}

}  // namespace nvfp4
