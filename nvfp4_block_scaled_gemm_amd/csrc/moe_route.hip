// Expert router: top-k choice, expert-sorted order, per-expert counts and the
// balance loss, and the gradient of the logits.
//
//   p[t, :] = softmax(x[t, :])             chosen: the k largest x, ties to the lowest expert
//   f_e = counts_e / (n k),  P_e = (1 / n) sum_t p[t, e],  loss = E sum_e f_e P_e
//   dx[t, e] = p (c_e - <p, c>) + share of the chosen weights' gradients,
//              c_e = dloss E f_e / n  (f is a count: no gradient flows through it)
//
// with n the tokens that chose any expert (a token is masked, or an expert
// is at -inf, and then never chosen).
//
// Forward, two launches (one token costs one pass over its logits):
//  1. route_choose_kernel: LPT lanes hold a token's logits in registers, NPL
//     neighbouring experts each, so the lowest lane of a tie holds the lowest
//     expert.  Each of the k rounds is a maximum over NPL registers and a
//     few lane rotations.  A workgroup takes a chunk of tokens; within 256
//     tokens the choice of an expert is one bit, so a token's place among
//     its expert's tokens is a population count: no atomics whose order
//     could matter, and the order is by token.
//  2. route_place_kernel: every workgroup sums the chunks' counts itself (at
//     most 256 chunks) and writes its own tokens' places; the first also
//     writes offsets, counts and the loss.
// Backward, one launch: the softmax again from the logits (one read, one
// write); the chosen weights' gradients meet their experts through LDS.
#include "nvfp4_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kMaxChunks = 256, kSub = 256, kSubWords = kSub / 32;
constexpr int kMaxExperts = 1024;

__host__ __device__ inline int64_t chunk_tokens(int64_t T) {
  int64_t c = (T + kMaxChunks - 1) / kMaxChunks;
  return c < 16 ? 16 : (c + 15) / 16 * 16;
}

// Order-keeping map of fp32 to unsigned; 0 for what is never chosen (-inf,
// NaN), which no finite value maps to.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  if (!(x > -__builtin_inff())) return 0;
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Rotation inside each row of 16 lanes.
template <int N>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}

template <int LPT, typename T, typename F>
__device__ __forceinline__ T group_reduce(T v, F&& f) {
  auto bits = [](T a) { return __builtin_bit_cast(uint32_t, a); };
  auto back = [](uint32_t a) { return __builtin_bit_cast(T, a); };
  v = f(v, back(ror16<8>(bits(v))));
  v = f(v, back(ror16<4>(bits(v))));
  v = f(v, back(ror16<2>(bits(v))));
  v = f(v, back(ror16<1>(bits(v))));
  if constexpr (LPT >= 32) v = f(v, back((uint32_t)__shfl_xor((int)bits(v), 16, 64)));
  if constexpr (LPT >= 64) v = f(v, back((uint32_t)__shfl_xor((int)bits(v), 32, 64)));
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<LPT>(v, [](float a, float b) { return a + b; });
}

// The lane's NPL logits of one row (-inf past the last expert).
template <int NPL>
__device__ __forceinline__ void load_logits(const void* __restrict__ x, int dtype, int64_t row_at,
                                            int e0, int E, bool vec, bool in, float* v) {
  if (vec && in && e0 + NPL <= E) {
    if (dtype == 1) {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(x) + row_at + e0;
      if constexpr (NPL >= 8) {
#pragma unroll
        for (int i = 0; i < NPL / 8; ++i) {
          const u32x4 w = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
          }
        }
      } else {
        const u32x2 w = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v[2 * j] = __uint_as_float(w[j] << 16);
          v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
      }
    } else {
      const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(x) + row_at + e0);
#pragma unroll
      for (int i = 0; i < NPL / 4; ++i) {
        const f32x4 w = p[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] = w[j];
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    v[i] = -__builtin_inff();
    if (in && e0 + i < E)
      v[i] = dtype == 1 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(x)[row_at + e0 + i] << 16)
                        : reinterpret_cast<const float*>(x)[row_at + e0 + i];
  }
}

// Partial results of the chunks: counts and probability sums [chunks][E],
// routed tokens [chunks].
struct Partials {
  int32_t* counts;
  float* psum;
  int32_t* routed;
};
__host__ inline Partials partials_at(void* ws, int64_t chunks, int64_t E) {
  int32_t* c = reinterpret_cast<int32_t*>(ws);
  float* p = reinterpret_cast<float*>(c + chunks * E);
  return {c, p, reinterpret_cast<int32_t*>(p + chunks * E)};
}

template <int LPT, int NPL>
__global__ __launch_bounds__(1024) void route_choose_kernel(
    int64_t T, int E, int k, const void* __restrict__ x, int dtype, int64_t ld, bool vec,
    const uint8_t* __restrict__ mask, bool renorm, int64_t per_chunk, RouteOut out, Partials part) {
  constexpr int TPW = 64 / LPT;  // tokens of a wave
  __shared__ uint32_t bits[LPT * NPL][kSubWords];
  __shared__ int32_t before[LPT * NPL];
  __shared__ float psum[LPT * NPL];
  __shared__ int32_t routed;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int lg = lane % LPT, grp = lane / LPT, e0 = lg * NPL;
  const int64_t c0 = (int64_t)blockIdx.x * per_chunk, c1 = min(T, c0 + per_chunk);
  for (int i = tid; i < LPT * NPL; i += blockDim.x) {
    before[i] = 0;
    psum[i] = 0.f;
  }
  if (tid == 0) routed = 0;
  float ps[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) ps[i] = 0.f;
  int mine = 0;  // tokens routed, counted by lane 0 of each group
  for (int64_t s0 = c0; s0 < c1; s0 += kSub) {
    const int here = (int)min((int64_t)kSub, c1 - s0);
    for (int i = tid; i < LPT * NPL * kSubWords; i += blockDim.x) (&bits[0][0])[i] = 0;
    __syncthreads();
    for (int base = wave * TPW; base < here; base += waves * TPW) {
      const int tk = base + grp;
      const int64_t t = s0 + tk;
      const bool in = tk < here && (mask == nullptr || mask[t] != 0);
      float v[NPL];
      load_logits<NPL>(x, dtype, t * ld, e0, E, vec, in, v);
      uint32_t key[NPL];
#pragma unroll
      for (int i = 0; i < NPL; ++i) key[i] = key_of(v[i]);
      float top = 0.f, chosen_sum = 0.f, val = -__builtin_inff();
      int32_t got = -1;
      for (int j = 0; j < k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < NPL; ++i) m = max(m, key[i]);
        const uint32_t g = group_max<LPT>(m);
        const uint64_t tie = __ballot(m == g && g != 0);
        const uint64_t grp_tie = LPT == 64 ? tie : (tie >> (grp * LPT)) & ((1ull << (LPT & 63)) - 1);
        if (j == 0) top = g != 0 ? value_of(g) : 0.f;
        const int win = grp_tie != 0 ? __builtin_ctzll(grp_tie) : -1;
        int e = -1;
        if (lg == win) {
#pragma unroll
          for (int i = NPL - 1; i >= 0; --i)
            if (key[i] == g) e = i;
#pragma unroll
          for (int i = 0; i < NPL; ++i)
            if (i == e) key[i] = 0;
          e += e0;
          atomicOr(&bits[e][tk >> 5], 1u << (tk & 31));
        }
        const int won = __shfl(e, win < 0 ? lane : grp * LPT + win, 64);
        if (lg == j) {
          got = win < 0 ? -1 : won;
          val = g != 0 ? value_of(g) : -__builtin_inff();
        }
      }
      // softmax over all, and over the chosen (lane j holds the j-th)
      const bool active = group_max<LPT>(lg < k && got >= 0 ? 1u : 0u) != 0;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        v[i] = active ? __expf(v[i] - top) : 0.f;
        sum += v[i];
      }
      sum = group_sum<LPT>(sum);
      const float inv = active ? 1.0f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) ps[i] += v[i] * inv;
      const float ez = got >= 0 ? __expf(val - top) : 0.f;
      chosen_sum = group_sum<LPT>(ez);
      if (tk < here && lg < k) {
        const int64_t at = t * k + lg;
        out.expert_index[at] = got;
        out.weights[at] = renorm ? (active ? ez / chosen_sum : 0.f) : ez * inv;
      }
      if (lg == 0 && active) ++mine;
    }
    __syncthreads();
    // places within the chunk, by token
    for (int i = tid; i < here * k; i += blockDim.x) {
      const int tk = i / k;
      const int64_t at = s0 * k + i;
      const int e = out.expert_index[at];
      int32_t place = -1;
      if (e >= 0) {
        place = before[e];
#pragma unroll
        for (int w = 0; w < kSubWords; ++w) {
          const uint32_t b = bits[e][w];
          const int d = tk - 32 * w;
          place += __builtin_popcount(d >= 32 ? b : (d > 0 ? b & ((1u << d) - 1u) : 0u));
        }
      }
      out.pair_row[at] = place;
    }
    __syncthreads();
    for (int e = tid; e < E; e += blockDim.x) {
      int32_t n = 0;
#pragma unroll
      for (int w = 0; w < kSubWords; ++w) n += __builtin_popcount(bits[e][w]);
      before[e] += n;
    }
    __syncthreads();
  }
  // probability sums: the wave's groups, then the waves in order
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    if constexpr (LPT <= 16) ps[i] += __shfl_xor(ps[i], 16, 64);
    if constexpr (LPT <= 32) ps[i] += __shfl_xor(ps[i], 32, 64);
  }
  for (int w = 0; w < waves; ++w) {
    if (wave == w && grp == 0) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) psum[e0 + i] += ps[i];
    }
    __syncthreads();
  }
  if (mine != 0) atomicAdd(&routed, mine);
  __syncthreads();
  for (int e = tid; e < E; e += blockDim.x) {
    part.counts[(int64_t)blockIdx.x * E + e] = before[e];
    part.psum[(int64_t)blockIdx.x * E + e] = psum[e];
  }
  if (tid == 0) part.routed[blockIdx.x] = routed;
}

__global__ __launch_bounds__(1024) void route_place_kernel(int64_t T, int E, int k, int chunks,
                                                           int64_t per_chunk, RouteOut out,
                                                           Partials part) {
  __shared__ int32_t total[kMaxExperts], lower[kMaxExperts], offset[kMaxExperts + 1];
  __shared__ double mean[kMaxExperts];
  __shared__ int32_t wave_sum[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool first = blockIdx.x == 0;
  for (int e = tid; e < E; e += 1024) {
    total[e] = 0;
    lower[e] = 0;
  }
  __syncthreads();
  // chunk counts: `parts` threads an expert
  const int parts = max(1, min(chunks, 1024 / E));
  if (tid < parts * E) {
    const int e = tid % E, p = tid / E;
    int32_t all = 0, low = 0;
    for (int c = p; c < chunks; c += parts) {
      const int32_t n = part.counts[(int64_t)c * E + e];
      all += n;
      low += c < (int)blockIdx.x ? n : 0;
    }
    atomicAdd(&total[e], all);
    atomicAdd(&lower[e], low);
  }
  __syncthreads();
  // offsets: inclusive scan over the experts (E <= 1024 threads)
  int32_t v = tid < E ? total[tid] : 0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(v, d, 64);
    if (lane >= d) v += o;
  }
  if (lane == 63) wave_sum[wave] = v;
  __syncthreads();
  int32_t add = 0;
  for (int w = 0; w < wave; ++w) add += wave_sum[w];
  if (tid < E) offset[tid + 1] = v + add;
  if (tid == 0) offset[0] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * per_chunk, c1 = min(T, c0 + per_chunk);
  for (int64_t i = c0 * k + tid; i < c1 * k; i += 1024) {
    const int32_t e = out.expert_index[i];
    if (e < 0) continue;
    const int32_t at = offset[e] + lower[e] + out.pair_row[i];
    out.pair_row[i] = at;
    out.row_index[at] = (int32_t)(i / k);
  }
  // rows behind the last expert name no token
  for (int64_t i = offset[E] + (int64_t)blockIdx.x * 1024 + tid; i < T * k; i += (int64_t)gridDim.x * 1024)
    out.row_index[i] = -1;
  if (!first) return;
  if (tid < E) {
    out.counts[tid] = total[tid];
    out.m_offsets[tid + 1] = offset[tid + 1];
    double s = 0.0;
    for (int c = 0; c < chunks; ++c) s += (double)part.psum[(int64_t)c * E + tid];
    mean[tid] = s * (double)total[tid];
  }
  if (tid == 0) out.m_offsets[0] = 0;
  __syncthreads();
  if (wave == 0) {
    double s = 0.0;
    int64_t n = 0;
    for (int e = lane; e < E; e += 64) s += mean[e];
    for (int c = lane; c < chunks; c += 64) n += part.routed[c];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      s += __shfl_xor(s, d, 64);
      n += __shfl_xor(n, d, 64);
    }
    if (lane == 0) {
      out.routed[0] = (int32_t)n;
      out.loss[0] = n > 0 ? (float)((double)E * s / ((double)n * (double)n * k)) : 0.f;
    }
  }
}

template <int LPT, int NPL>
__global__ __launch_bounds__(256) void route_backward_kernel(
    int64_t T, int E, int k, const void* __restrict__ x, int dtype, int64_t ld, bool vec,
    const uint8_t* __restrict__ mask, bool renorm, const int32_t* __restrict__ expert_index,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ routed,
    const float* __restrict__ d_weights, const float* __restrict__ d_loss, void* __restrict__ dx,
    int64_t ld_d, bool vec_d) {
  constexpr int GROUPS = 256 / LPT;
  __shared__ __attribute__((aligned(16))) float add[GROUPS][LPT * NPL];
  const int lane = threadIdx.x & 63, lg = lane % LPT, e0 = lg * NPL;
  const int g = threadIdx.x / LPT;
  float* row = add[g];
  const float n = (float)routed[0];
  const float coef = d_loss != nullptr && n > 0.f ? d_loss[0] * (float)E / (n * n * (float)k) : 0.f;
  float c[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    c[i] = e0 + i < E ? coef * (float)counts[e0 + i] : 0.f;
    row[e0 + i] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  const int64_t first = (int64_t)blockIdx.x * GROUPS;
  for (int64_t b = first; b < T; b += step) {
    const int64_t t = b + g;
    const bool in = t < T && (mask == nullptr || mask[t] != 0);
    float v[NPL];
    load_logits<NPL>(x, dtype, t * ld, e0, E, vec, in, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) m = max(m, key_of(v[i]));
    m = group_max<LPT>(m);
    const bool active = m != 0;
    const float top = active ? value_of(m) : 0.f;
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      v[i] = active ? __expf(v[i] - top) : 0.f;
      sum += v[i];
    }
    sum = group_sum<LPT>(sum);
    const float inv = active ? 1.0f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      v[i] *= inv;
      dot += v[i] * c[i];
    }
    // lane j takes the j-th chosen expert
    int32_t e = -1;
    float dw = 0.f, ez = 0.f;
    if (active && lg < k && d_weights != nullptr) {
      e = expert_index[t * k + lg];
      if (e < 0 || e >= E) e = -1;
      if (e >= 0) {
        dw = d_weights[t * k + lg];
        const float xe = dtype == 1 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(x)[t * ld + e] << 16)
                                    : reinterpret_cast<const float*>(x)[t * ld + e];
        ez = __expf(xe - top);
      }
    }
    float a;
    if (renorm) {
      const float cs = group_sum<LPT>(ez);
      const float w = e >= 0 ? ez / cs : 0.f;
      a = w * (dw - group_sum<LPT>(w * dw));
    } else {
      a = ez * inv * dw;
      dot += a;
    }
    dot = group_sum<LPT>(dot);
    if (e >= 0) atomicAdd(&row[e], a);  // experts of a token differ: one addend each
    __builtin_amdgcn_wave_barrier();
    float o[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) o[i] = v[i] * (c[i] - dot) + row[e0 + i];
    __builtin_amdgcn_wave_barrier();
    if (e >= 0) row[e] = 0.f;
    __builtin_amdgcn_wave_barrier();
    if (t < T) {
      if (vec_d && e0 + NPL <= E) {
        if (dtype == 1) {
          uint32_t w[NPL / 2];
#pragma unroll
          for (int i = 0; i < NPL / 2; ++i)
            w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{o[2 * i], o[2 * i + 1]}, bf16x2));
          uint16_t* p = reinterpret_cast<uint16_t*>(dx) + t * ld_d + e0;
          if constexpr (NPL >= 8) {
#pragma unroll
            for (int i = 0; i < NPL / 8; ++i)
              reinterpret_cast<u32x4*>(p)[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
          } else {
            *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
          }
        } else {
          f32x4* p = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(dx) + t * ld_d + e0);
#pragma unroll
          for (int i = 0; i < NPL / 4; ++i) p[i] = f32x4{o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]};
        }
      } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          if (e0 + i < E) {
            if (dtype == 1) reinterpret_cast<__bf16*>(dx)[t * ld_d + e0 + i] = (__bf16)o[i];
            else reinterpret_cast<float*>(dx)[t * ld_d + e0 + i] = o[i];
          }
      }
    }
  }
}

bool rows_vec(const void* p, int dtype, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * (dtype == 0 ? 4 : 2)) % 16 == 0;
}

// Lanes per token and experts per lane: as few lanes as hold the experts with
// at most 16 each, so that a wave works on up to four tokens at once.
template <typename F>
hipError_t by_experts(int64_t E, F&& f) {
  if (E <= 64) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
  if (E <= 128) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
  if (E <= 256) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 16>{});
  if (E <= 512) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}

}  // namespace

size_t moe_route_workspace_bytes(int64_t T, int64_t E) {
  const int64_t per = chunk_tokens(T);
  const int64_t chunks = T > 0 ? (T + per - 1) / per : 1;
  return (size_t)(chunks * E * 8 + chunks * 4);
}

hipError_t launch_moe_route(int64_t T, int64_t E, int topk, const void* logits, int dtype,
                            int64_t ld, const uint8_t* mask, bool renorm, RouteOut out,
                            void* workspace, hipStream_t stream) {
  const int64_t per = chunk_tokens(T);
  const int chunks = T > 0 ? (int)((T + per - 1) / per) : 1;  // no token: one empty chunk
  const Partials part = partials_at(workspace, chunks, E);
  const bool vec = rows_vec(logits, dtype, ld);
  const hipError_t err = by_experts(E, [&](auto lpt, auto npl) {
    constexpr int LPT = decltype(lpt)::value, NPL = decltype(npl)::value;
    // a wave for each LPT-lane group of the chunk, up to 16 waves
    int64_t waves = (per * LPT + 63) / 64;
    waves = waves > 16 ? 16 : (waves < 4 ? 4 : waves);
    route_choose_kernel<LPT, NPL><<<(unsigned)chunks, (unsigned)(64 * waves), 0, stream>>>(
        T, (int)E, topk, logits, dtype, ld, vec, mask, renorm, per, out, part);
    return hipGetLastError();
  });
  if (err != hipSuccess) return err;
  route_place_kernel<<<(unsigned)chunks, 1024, 0, stream>>>(T, (int)E, topk, chunks, per, out, part);
  return hipGetLastError();
}

hipError_t launch_moe_route_backward(int64_t T, int64_t E, int topk, const void* logits, int dtype,
                                     int64_t ld, const uint8_t* mask, bool renorm,
                                     const int32_t* expert_index, const int32_t* counts,
                                     const int32_t* routed, const float* d_weights,
                                     const float* d_loss, void* d_logits, int64_t ld_d,
                                     hipStream_t stream) {
  const bool vec = rows_vec(logits, dtype, ld), vec_d = rows_vec(d_logits, dtype, ld_d);
  return by_experts(E, [&](auto lpt, auto npl) {
    constexpr int LPT = decltype(lpt)::value, NPL = decltype(npl)::value;
    const int64_t groups = 256 / LPT;
    int64_t grid = (T + groups - 1) / groups;
    if (grid > 2048) grid = 2048;
    route_backward_kernel<LPT, NPL><<<(unsigned)grid, 256, 0, stream>>>(
        T, (int)E, topk, logits, dtype, ld, vec, mask, renorm, expert_index, counts, routed,
        d_weights, d_loss, d_logits, ld_d, vec_d);
    return hipGetLastError();
  });
}

}  // namespace nvfp4
