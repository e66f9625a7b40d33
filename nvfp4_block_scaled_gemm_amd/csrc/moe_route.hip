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
// Forward, two launches, or one for few tokens (a token costs one pass over
// its logits):
//  1. route_choose_kernel: LPT lanes hold a token's logits in registers, NPL
//     neighbouring experts each.  A logit and its expert make one 31-bit key
//     (the order-keeping image of the logit, cut to leave room for the
//     expert, lower experts larger), so keys differ and a round of the choice
//     is "the largest key below the last": with 31-bit keys, key - last wraps
//     to the top half exactly for the keys below, so one subtraction and half
//     a three-way maximum per logit and four lane rotations do it, nothing is
//     removed and nothing is compared for ties.  bf16 logits fit whole.  fp32
//     logits lose their last bits: a token two of whose chosen (or the first
//     not chosen) agree in what is left is done again by an exact search.
//     A workgroup takes a chunk of tokens; within 256 tokens the choice of an
//     expert is one bit, so a token's place among its expert's tokens is a
//     population count: no atomics whose order could matter.
//  2. route_place_kernel: every workgroup sums the chunks' counts itself (at
//     most 256 chunks, read in batches) and writes its own tokens' places;
//     one more per 64 experts sums their share of the loss.
// Backward, one launch: the softmax again from the logits (one read, one
// write); the chosen weights' gradients meet their experts through LDS.
//
// The choice is bound by the vector unit (1.5 k instructions a logit besides
// the softmax's); of the placement, each workgroup's reading of all chunks'
// counts (256 KB from L2 at 65536 x 256) before it places a token; the rest by
// launches.  Measured, bf16, 256 experts, top 8, replayed from a graph: 1 token
// 6.1 us forward and 3.5 backward, 4096 tokens 15.9 and 4.3, 65536 38.0 (34 MB
// of logits) and 17.9 (67 MB, 3.7 TB/s); there, profiled one kernel at a time,
// choice 29, placement 12 and backward 21.
#include "nvfp4_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace {

constexpr int kMaxChunks = 256, kSub = 256, kSubWords = kSub / 32;
constexpr int kMaxExperts = 1024, kMaxTop = 16;

__host__ __device__ inline int64_t chunk_tokens(int64_t T) {
  int64_t c = (T + kMaxChunks - 1) / kMaxChunks;
  return c < 16 ? 16 : (c + 15) / 16 * 16;
}

// Order-keeping map of fp32 to unsigned; zeros of either sign are one value
// (-0 + 0 is +0, and without that the image of -0 would lie below that of +0).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
// The image of -inf: what is not above it is never chosen.
constexpr uint32_t kNever = 0x007FFFFFu;

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

// exp(d), d <= 0, within 2^-22 relative however far d is.  The instruction
// raises 2 to t = d log2(e), whose rounding alone is up to 2^-24 |t| (5e-6 of
// the result at d = -88): what t loses is kept in r and put back as
// 2^t (1 + r ln 2).  |r| stays below 2^-16 wherever 2^t is not 0; the bounds
// keep it a number where t is -inf (a median drops a NaN of its arguments), and
// a NaN in d comes out through 2^t.
__device__ __forceinline__ float exp_below(float d) {
  constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596303e-8f, kLn2 = 0.693147181f;
  const float t = d * kLog2e;
  const float r = __builtin_fmaf(d, kLog2eRest, __builtin_fmaf(d, kLog2e, -t));
  const float y = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(y, __builtin_amdgcn_fmed3f(r, -1.0f, 1.0f) * kLn2, y);
}

// A logit as fp32.
template <int DT>
__device__ __forceinline__ float logit(const void* __restrict__ x, int64_t at) {
  if constexpr (DT == 1) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(x)[at] << 16);
  else return reinterpret_cast<const float*>(x)[at];
}

// The lane's NPL logits of one row (-inf past the last expert, or all of
// them).  VEC: whole lanes (E % NPL == 0), aligned rows.
template <int NPL, int DT, bool VEC>
__device__ __forceinline__ void load_logits(const void* __restrict__ x, int64_t row_at, int e0,
                                            int E, bool in, float* v) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = -__builtin_inff();
    if (!in || e0 >= E) return;
    if constexpr (DT == 1) {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(x) + row_at + e0;
#pragma unroll
      for (int i = 0; i < NPL / 4; ++i) {
        const u32x2 w = reinterpret_cast<const u32x2*>(p)[i];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v[4 * i + 2 * j] = __uint_as_float(w[j] << 16);
          v[4 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
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
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      v[i] = in && e0 + i < E ? logit<DT>(x, row_at + e0 + i) : -__builtin_inff();
  }
}

// The k largest of a token's logits, lane j receiving the j-th expert (-1:
// none left).  Returns whether the keys could not tell two of them apart
// (fp32 logits only; some lane of the group says so).
template <int LPT, int NPL, int DT>
__device__ __forceinline__ bool choose_by_keys(const float* v, int e0, int lg, int k, int32_t& got) {
  constexpr bool wide = DT == 0;
  constexpr uint32_t kExpert = LPT * NPL - 1;  // the expert's bits of a key
  constexpr uint32_t kNone = (kNever >> 1) | kExpert;  // keys up to here: an expert at -inf
  uint32_t key[NPL], g = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    key[i] = ((key_of(v[i]) >> 1) & ~kExpert) | (kExpert - (uint32_t)(e0 + i));
    g = max(g, key[i]);
  }
  g = group_max<LPT>(g);
  bool same = false;
  for (int j = 0; j < k; ++j) {
    if (lg == j && g > kNone) got = (int32_t)(kExpert - (g & kExpert));
    if (j == k - 1 && !wide) break;  // fp32 looks at one more
    uint32_t m = key[0] - g;
#pragma unroll
    for (int i = 1; i < NPL; ++i) m = max(m, key[i] - g);
    m = group_max<LPT>(m);
    // no key below the last one: the search is over
    const uint32_t next = (int32_t)m < 0 ? m + g : 0u;
    same = same || (next > kNone && ((next ^ g) & ~kExpert) == 0);
    g = next;
  }
  return same && wide;
}

// The same by whole fp32 values: rounds of maximum, first holder, removal.
template <int LPT, int NPL>
__device__ __forceinline__ int32_t choose_exactly(const float (&v)[NPL], int e0, int lg, int grp,
                                                  int k) {
  int32_t got = -1;
  uint32_t key[NPL];  // 0: never chosen, or chosen already
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    key[i] = key_of(v[i]);
    if (key[i] <= kNever) key[i] = 0;
  }
  for (int j = 0; j < k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) m = max(m, key[i]);
    const uint32_t g = group_max<LPT>(m);
    const uint64_t tie = __ballot(m == g && g != 0);
    const uint64_t grp_tie = LPT == 64 ? tie : (tie >> (grp * LPT)) & ((1ull << (LPT & 63)) - 1);
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
    }
    const int won = __shfl(e, win < 0 ? (int)__lane_id() : grp * LPT + win, 64);
    if (lg == j) got = win < 0 ? -1 : won;
  }
  return got;
}

// Partial results of the chunks: counts and probability sums [chunks][E],
// routed tokens [chunks]; then the loss's parts [kMaxExperts / 64] and the
// count of those that are written (cleared by the first launch).
struct Partials {
  int32_t* counts;
  float* psum;
  int32_t* routed;
  float* loss;
  uint32_t* written;
};
constexpr int kLossParts = kMaxExperts / 64;
__host__ inline Partials partials_at(void* ws, int64_t chunks, int64_t E) {
  int32_t* c = reinterpret_cast<int32_t*>(ws);
  float* p = reinterpret_cast<float*>(c + chunks * E);
  int32_t* r = reinterpret_cast<int32_t*>(p + chunks * E);
  float* l = reinterpret_cast<float*>(r + chunks);
  return {c, p, r, l, reinterpret_cast<uint32_t*>(l + 2 * kLossParts)};
}

// Choices are walked as (token, slot) pairs of kMaxTop slots a token, so no
// index is divided by k.  ONE: at most kSub tokens, and the workgroup finishes
// the call by itself.
template <int LPT, int NPL, int DT, bool VEC, bool ONE>
__global__ __launch_bounds__(1024) void route_choose_kernel(
    int T, int E, int k, const void* __restrict__ x, int64_t ld, const uint8_t* __restrict__ mask, bool renorm, int per_chunk, RouteOut out, Partials part) {
  constexpr int TPW = 64 / LPT;  // tokens of a wave
  constexpr int EP = LPT * NPL;
  __shared__ uint32_t bits[EP][kSubWords];
  __shared__ int16_t chosen[kSub][kMaxTop];
  __shared__ int32_t before[EP];
  __shared__ float psum[4][EP];
  __shared__ int32_t routed;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int lg = lane % LPT, grp = lane / LPT, e0 = lg * NPL;
  const int c0 = blockIdx.x * per_chunk, c1 = min(T, c0 + per_chunk);
  for (int i = tid; i < EP; i += blockDim.x) {
    before[i] = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) psum[q][i] = 0.f;
  }
  if (tid == 0) {
    routed = 0;
    if (!ONE && blockIdx.x == 0) *part.written = 0;
  }
  if constexpr (ONE) {
    for (int i = tid; i < EP * kSubWords; i += blockDim.x) (&bits[0][0])[i] = 0;
    __syncthreads();
  }
  // place of token tk of the 256 among the expert's tokens
  auto place_of = [&](int e, int tk) {
    if (e < 0) return -1;
    int32_t place = before[e];
#pragma unroll
    for (int w = 0; w < kSubWords; ++w) {
      const uint32_t b = bits[e][w];
      const int d = tk - 32 * w;
      place += __builtin_popcount(d >= 32 ? b : (d > 0 ? b & ((1u << d) - 1u) : 0u));
    }
    return place;
  };
  auto chosen_by = [&](int e) {
    int32_t n = 0;
#pragma unroll
    for (int w = 0; w < kSubWords; ++w) n += __builtin_popcount(bits[e][w]);
    return n;
  };
  float ps[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) ps[i] = 0.f;
  int mine = 0;  // tokens routed, counted by lane 0 of each group
  for (int s0 = c0; s0 < c1; s0 += kSub) {
    const int here = min(kSub, c1 - s0);
    if constexpr (!ONE) {
      for (int i = tid; i < EP * kSubWords; i += blockDim.x) (&bits[0][0])[i] = 0;
      __syncthreads();
    }
    // one turn ahead of itself: a turn loads the next tokens' logits and then
    // works on its own (the first only loads)
    float nv[NPL];
    for (int base = wave * TPW - waves * TPW; base < here; base += waves * TPW) {
      float v[NPL];
#pragma unroll
      for (int i = 0; i < NPL; ++i) v[i] = nv[i];
      const int nt = base + waves * TPW + grp;
      load_logits<NPL, DT, VEC>(x, (s0 + nt) * ld, e0, E, nt < here && (mask == nullptr || mask[s0 + nt] != 0), nv);
      if (base < 0) continue;
      const int tk = base + grp, t = s0 + tk;
      int32_t got = -1;  // lane j: the j-th chosen expert
      const bool again = choose_by_keys<LPT, NPL, DT>(v, e0, lg, k, got);
      if constexpr (DT == 0) {
        if (__any(again)) {
          const int32_t exact = choose_exactly<LPT, NPL>(v, e0, lg, grp, k);
          if (group_max<LPT>(again ? 1u : 0u) != 0) got = exact;
        }
      }
      float val = -__builtin_inff();
      if (got >= 0) {
        atomicOr(&bits[got][tk >> 5], 1u << (tk & 31));
        val = logit<DT>(x, t * ld + got);
      }
      float top = v[0];
#pragma unroll
      for (int i = 1; i < NPL; ++i) top = fmaxf(top, v[i]);
      top = group_reduce<LPT>(top, [](float p, float q) { return fmaxf(p, q); });
      // softmax over all, and over the chosen (lane j holds the j-th).  The
      // sum's terms may take the plain instruction, whose error grows with a
      // term's distance d from the top: it adds up to 2^-24 times the mean
      // distance under p, which is at most ln E.  (exp_below here: 40.3 instead
      // of 38.0 us for 65536 x 256 bf16.)
      const bool active = top > -__builtin_inff();
      if (!active) top = 0.f;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        v[i] = __expf(v[i] - top);  // an inactive row's -inf gives 0
        sum += v[i];
      }
      sum = group_sum<LPT>(sum);
      const float inv = active ? 1.0f / sum : 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) ps[i] += v[i] * inv;
      const float ez = got >= 0 ? exp_below(val - top) : 0.f;
      const float chosen_sum = group_sum<LPT>(ez);
      if (tk < here && lg < k) {
        chosen[tk][lg] = (int16_t)got;
        const int64_t at = (int64_t)t * k + lg;
        out.expert_index[at] = got;
        out.weights[at] = renorm ? (active ? ez / chosen_sum : 0.f) : ez * inv;
      }
      if (lg == 0 && active) ++mine;
    }
    __syncthreads();
    if constexpr (ONE) break;
    // places within the chunk, by token
    for (int i = tid; i < here * kMaxTop; i += blockDim.x) {
      const int tk = i / kMaxTop, j = i % kMaxTop;
      if (j >= k) continue;
      out.pair_row[(int64_t)(s0 + tk) * k + j] = place_of(chosen[tk][j], tk);
    }
    __syncthreads();
    for (int e = tid; e < E; e += blockDim.x) before[e] += chosen_by(e);
    __syncthreads();
  }
  // probability sums: the wave's groups, then every fourth wave in order
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    if constexpr (LPT <= 16) ps[i] += __shfl_xor(ps[i], 16, 64);
    if constexpr (LPT <= 32) ps[i] += __shfl_xor(ps[i], 32, 64);
  }
  if (mine != 0) atomicAdd(&routed, mine);
  for (int w = 0; w < waves; w += 4) {
    if (wave / 4 == w / 4 && grp == 0) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) psum[wave & 3][e0 + i] += ps[i];
    }
    __syncthreads();
  }
  auto mass = [&](int e) { return (psum[0][e] + psum[1][e]) + (psum[2][e] + psum[3][e]); };
  if constexpr (ONE) {
    __shared__ int32_t wave_sum[16];
    __shared__ double wave_loss[16];
    int32_t end = 0;  // rows of the experts so far
    double loss = 0.0;
    for (int b = 0; b < E; b += blockDim.x) {
      const int e = b + tid;
      const int32_t n = e < E ? chosen_by(e) : 0;
      int32_t v = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(v, d, 64);
        if (lane >= d) v += o;
      }
      if (lane == 63) wave_sum[wave] = v;
      __syncthreads();
      v += end;
      for (int w = 0; w < waves; ++w) {
        if (w < wave) v += wave_sum[w];
        end += wave_sum[w];
      }
      if (e < E) {
        before[e] = v - n;
        out.counts[e] = n;
        out.m_offsets[e + 1] = v;
        loss += (double)n * (double)mass(e);
      }
      __syncthreads();
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) loss += __shfl_xor(loss, d, 64);
    if (lane == 0) wave_loss[wave] = loss;
    for (int i = tid; i < T * kMaxTop; i += blockDim.x) {
      const int t = i / kMaxTop, j = i % kMaxTop;
      if (j >= k) continue;
      const int32_t place = place_of(chosen[t][j], t);
      out.pair_row[t * k + j] = place;
      if (place >= 0) out.row_index[place] = t;
    }
    for (int i = end + tid; i < T * k; i += blockDim.x) out.row_index[i] = -1;
    __syncthreads();
    if (tid != 0) return;
    loss = 0.0;
    for (int w = 0; w < waves; ++w) loss += wave_loss[w];
    out.m_offsets[0] = 0;
    out.routed[0] = routed;
    out.loss[0] = routed > 0 ? (float)((double)E * loss / ((double)routed * (double)routed * k)) : 0.f;
    return;
  }
  for (int e = tid; e < E; e += blockDim.x) {
    part.counts[(int64_t)blockIdx.x * E + e] = before[e];
    part.psum[(int64_t)blockIdx.x * E + e] = mass(e);
  }
  if (tid == 0) part.routed[blockIdx.x] = routed;
}

// Sum over chunks c = p, p + parts, .. of column e of a [chunks][E] array, 16
// loads at a time; `low` takes those of chunks below `limit`.
__device__ __forceinline__ int32_t column_sum(const int32_t* __restrict__ a, int E, int e, int p,
                                              int parts, int chunks, int limit, int32_t& low) {
  int32_t all = 0;
  for (int c = p; c < chunks; c += 16 * parts) {
    int32_t v[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const int cc = c + u * parts;
      v[u] = cc < chunks ? a[(int64_t)cc * E + e] : 0;
    }
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      all += v[u];
      low += c + u * parts < limit ? v[u] : 0;
    }
  }
  return all;
}

// The loss, 64 experts a workgroup and 16 threads an expert (a chunk run of
// each, so one batch of loads): their part of sum_e counts_e sum_t p[t, e] in
// fp64, kept as a pair of fp32 words; whoever finishes last adds the parts in
// order.
__device__ __forceinline__ void loss_part(int E, int k, int chunks, int b, int parts, RouteOut out,
                                          Partials part) {
  __shared__ double mass[16][64];
  __shared__ int32_t load[64];
  const int tid = threadIdx.x, lane = tid & 63, p = tid >> 6, e = b * 64 + lane;
  if (tid < 64) load[tid] = 0;
  __syncthreads();
  double s = 0.0;
  if (e < E) {
    int32_t low = 0;
    const int32_t n = column_sum(part.counts, E, e, p, 16, chunks, 0, low);
    float v[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const int c = p + 16 * u;
      v[u] = c < chunks ? part.psum[(int64_t)c * E + e] : 0.f;
    }
    float f = 0.f;  // 16 chunks' sums, pairwise
#pragma unroll
    for (int u = 0; u < 16; u += 4) f += (v[u] + v[u + 1]) + (v[u + 2] + v[u + 3]);
    s = (double)f;
    atomicAdd(&load[lane], n);
  }
  mass[p][lane] = s;
  __syncthreads();
  if (p != 0) return;
  s = 0.0;
  for (int q = 0; q < 16; ++q) s += mass[q][lane];
  s *= (double)load[lane];
  int32_t n = 0;
  for (int c = lane; c < chunks; c += 64) n += part.routed[c];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    s += __shfl_xor(s, d, 64);
    n += __shfl_xor(n, d, 64);
  }
  if (lane != 0) return;
  const uint64_t w = __builtin_bit_cast(uint64_t, s);
  uint32_t* mine = reinterpret_cast<uint32_t*>(part.loss) + 2 * b;
  __hip_atomic_store(mine, (uint32_t)w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(mine + 1, (uint32_t)(w >> 32), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint32_t before = __hip_atomic_fetch_add(part.written, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  if (before != (uint32_t)parts - 1) return;
  double t = 0.0;
  for (int q = 0; q < parts; ++q) {
    uint32_t* at = reinterpret_cast<uint32_t*>(part.loss) + 2 * q;
    const uint64_t lo = __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint64_t hi = __hip_atomic_load(at + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    t += __builtin_bit_cast(double, lo | (hi << 32));
  }
  const double m = (double)n * (double)n * k;
  out.routed[0] = n;
  out.loss[0] = n > 0 ? (float)((double)E * t / m) : 0.f;
}

// The first `parts` workgroups: the loss.  The others: the places of one
// chunk's tokens; the first of them writes counts and offsets too.
__global__ __launch_bounds__(1024) void route_place_kernel(int T, int E, int k, int chunks,
                                                           int per_chunk, int loss_parts,
                                                           RouteOut out, Partials part) {
  __shared__ int32_t total[kMaxExperts], lower[kMaxExperts], offset[kMaxExperts + 1];
  __shared__ int32_t wave_sum[16];
  if ((int)blockIdx.x < loss_parts) {
    loss_part(E, k, chunks, blockIdx.x, loss_parts, out, part);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunk = blockIdx.x - loss_parts;
  for (int e = tid; e < E; e += 1024) {
    total[e] = 0;
    lower[e] = 0;
  }
  // the chunk's own choices are on their way meanwhile (thread: token of 64,
  // slot of kMaxTop)
  const int c0 = chunk * per_chunk, c1 = min(T, c0 + per_chunk);
  const int slot = tid % kMaxTop;
  int t = slot >= k ? c1 : c0 + tid / kMaxTop;
  int32_t e_next = t < c1 ? out.expert_index[(int64_t)t * k + slot] : -1;
  int32_t p_next = t < c1 ? out.pair_row[(int64_t)t * k + slot] : 0;
  __syncthreads();
  // chunk counts: `parts` threads an expert
  const int parts = max(1, min(chunks, 1024 / E));
  if (tid < parts * E) {
    const int e = tid % E, p = tid / E;
    int32_t low = 0;
    const int32_t all = column_sum(part.counts, E, e, p, parts, chunks, chunk, low);
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
  if (chunk == 0) {
    if (tid < E) {
      out.counts[tid] = total[tid];
      out.m_offsets[tid + 1] = offset[tid + 1];
    }
    if (tid == 0) out.m_offsets[0] = 0;
  }
  // rows behind the last expert name no token
  for (int64_t i = max(offset[E], 0) + (int64_t)chunk * 1024 + tid; i < (int64_t)T * k; i += (int64_t)chunks * 1024)
    out.row_index[i] = -1;
  while (t < c1) {
    const int64_t i = (int64_t)t * k + slot;
    const int32_t e = e_next, p = p_next;
    const int tn = t + 1024 / kMaxTop;
    if (tn < c1) {
      e_next = out.expert_index[(int64_t)tn * k + slot];
      p_next = out.pair_row[(int64_t)tn * k + slot];
    }
    if (e >= 0 && e < E) {
      // inside the rows even if another call writes the same workspace
      const uint32_t at = (uint32_t)(offset[e] + lower[e] + p);
      if (at < (uint32_t)T * (uint32_t)k) {
        out.pair_row[i] = (int32_t)at;
        out.row_index[at] = t;
      }
    }
    t = tn;
  }
}

template <int LPT, int NPL, int DT, bool VEC>
__global__ __launch_bounds__(256) void route_backward_kernel(
    int64_t T, int E, int k, const void* __restrict__ x, int64_t ld, const uint8_t* __restrict__ mask, bool renorm, const int32_t* __restrict__ expert_index,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ routed,
    const float* __restrict__ d_weights, const float* __restrict__ d_loss, void* __restrict__ dx,
    int64_t ld_d) {
  constexpr int GROUPS = 256 / LPT;
  __shared__ __attribute__((aligned(16))) float add[GROUPS][LPT * NPL];
  const int lane = threadIdx.x & 63, lg = lane % LPT, e0 = lg * NPL;
  const int g = threadIdx.x / LPT;
  float* row = add[g];
  __shared__ __attribute__((aligned(16))) float table[LPT * NPL];
  const float n = (float)routed[0];
  const float coef = d_loss != nullptr && n > 0.f ? d_loss[0] * (float)E / (n * n * (float)k) : 0.f;
  for (int e = threadIdx.x; e < LPT * NPL; e += 256) table[e] = e < E ? coef * (float)counts[e] : 0.f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) row[e0 + i] = 0.f;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  const int64_t first = (int64_t)blockIdx.x * GROUPS;
  __syncthreads();
  float nv[NPL], c[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) c[i] = table[e0 + i];
  // one turn ahead of itself, as in the choice
  for (int64_t b = first - step; b < T; b += step) {
    const int64_t t = b + g, nt = t + step;
    float v[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = nv[i];
    load_logits<NPL, DT, VEC>(x, nt * ld, e0, E, nt < T && (mask == nullptr || mask[nt] != 0), nv);
    if (b < first) continue;
    float top = v[0];
#pragma unroll
    for (int i = 1; i < NPL; ++i) top = fmaxf(top, v[i]);
    top = group_reduce<LPT>(top, [](float p, float q) { return fmaxf(p, q); });
    const bool active = top > -__builtin_inff();
    if (!active) top = 0.f;
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      v[i] = exp_below(v[i] - top);  // an inactive row's -inf gives 0
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
        ez = exp_below(logit<DT>(x, t * ld + e) - top);
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
    if (t >= T || e0 >= E) continue;
    if constexpr (VEC && DT == 1) {
      u32x2* p = reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(dx) + t * ld_d + e0);
#pragma unroll
      for (int i = 0; i < NPL / 4; ++i)
        p[i] = u32x2{__builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{o[4 * i], o[4 * i + 1]}, bf16x2)),
                     __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{o[4 * i + 2], o[4 * i + 3]}, bf16x2))};
    } else if constexpr (VEC) {
      f32x4* p = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(dx) + t * ld_d + e0);
#pragma unroll
      for (int i = 0; i < NPL / 4; ++i) p[i] = f32x4{o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (e0 + i < E) {
          if constexpr (DT == 1) reinterpret_cast<__bf16*>(dx)[t * ld_d + e0 + i] = (__bf16)o[i];
          else reinterpret_cast<float*>(dx)[t * ld_d + e0 + i] = o[i];
        }
    }
  }
}

// Rows that a lane reads (writes) NPL neighbours of at once: 16-byte aligned
// and of whole lanes.
bool rows_vec(const void* p, int dtype, int64_t ld, int64_t E, int npl) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * (dtype == 0 ? 4 : 2)) % 16 == 0 && E % npl == 0;
}

template <int N>
using Int = std::integral_constant<int, N>;

// Lanes per token and experts per lane: as few lanes as hold the experts with
// at most 16 each, so that a wave works on up to four tokens at once.
template <typename F>
hipError_t by_experts(int64_t E, F&& f) {
  if (E <= 64) return f(Int<16>{}, Int<4>{});
  if (E <= 128) return f(Int<16>{}, Int<8>{});
  if (E <= 256) return f(Int<16>{}, Int<16>{});
  if (E <= 512) return f(Int<32>{}, Int<16>{});
  return f(Int<64>{}, Int<16>{});
}
// The logits' type and whether rows are read whole lanes at a time.
template <typename F>
hipError_t by_rows(int dtype, bool vec, F&& f) {
  if (dtype == 1) return vec ? f(Int<1>{}, std::true_type{}) : f(Int<1>{}, std::false_type{});
  return vec ? f(Int<0>{}, std::true_type{}) : f(Int<0>{}, std::false_type{});
}

}  // namespace

size_t moe_route_workspace_bytes(int64_t T, int64_t E) {
  const int64_t per = chunk_tokens(T);
  const int64_t chunks = T > 0 ? (T + per - 1) / per : 1;
  return (size_t)(chunks * E * 8 + chunks * 4 + 2 * kLossParts * 4 + 4);
}

hipError_t launch_moe_route(int64_t T, int64_t E, int topk, const void* logits, int dtype,
                            int64_t ld, const uint8_t* mask, bool renorm, RouteOut out,
                            void* workspace, hipStream_t stream) {
  // One workgroup takes the whole call where it needs about one turn for it,
  // and up to 256 experts only while the rounds of its 16 waves' choices do not
  // outweigh the second launch (us, one launch and two, bf16 / fp32: 1 x 256
  // top 8 6.2 / 9.5; 48 x 256 top 8 9.3 10.2 / 12.7 13.3; 64 x 256 top 2 9.5 9.8 / 9.7
  // 10.2, but top 8 10.9 10.2 / 11.2 10.5 and top 16 12.8 11.1; 64 x 128 top 8
  // 8.6 9.0 / 8.8 9.4, but top 16 9.8 9.8 / 10.3 9.8; 96 x 128 top 8 9.8 9.3; 32 x
  // 512 top 16 12.4 13.2 / 13.0 13.6, but 48 x 512 14.8 13.2; 16 x 1024 top 16
  // 12.8 18.2, but 32 x 1024 19.6 18.3).
  const bool one = T <= 64 && T * E <= 16384 && (E > 256 || T * (E + 16 * topk) < 24576);
  const int64_t per = one ? T : chunk_tokens(T);
  const int chunks = one ? 1 : (int)((T + per - 1) / per);
  const Partials part = partials_at(workspace, chunks, E);
  const hipError_t err = by_experts(E, [&](auto lpt, auto npl) {
    constexpr int LPT = decltype(lpt)::value, NPL = decltype(npl)::value;
    // a wave for each LPT-lane group of the chunk, up to 16 waves
    int64_t waves = (per * LPT + 63) / 64;
    waves = waves > 16 ? 16 : (waves < 4 ? 4 : waves);
    return by_rows(dtype, rows_vec(logits, dtype, ld, E, NPL), [&](auto dt, auto vec) {
      auto choose = [&](auto whole_call) {
        route_choose_kernel<LPT, NPL, decltype(dt)::value, decltype(vec)::value, decltype(whole_call)::value>
            <<<(unsigned)chunks, (unsigned)(64 * waves), 0, stream>>>(
                (int)T, (int)E, topk, logits, ld, mask, renorm, (int)per, out, part);
      };
      if (one) choose(std::true_type{});
      else choose(std::false_type{});
      return hipGetLastError();
    });
  });
  if (err != hipSuccess || one) return err;
  const int loss_parts = (int)((E + 63) / 64);
  route_place_kernel<<<(unsigned)(chunks + loss_parts), 1024, 0, stream>>>(
      (int)T, (int)E, topk, chunks, (int)per, loss_parts, out, part);
  return hipGetLastError();
}

hipError_t launch_moe_route_backward(int64_t T, int64_t E, int topk, const void* logits, int dtype,
                                     int64_t ld, const uint8_t* mask, bool renorm,
                                     const int32_t* expert_index, const int32_t* counts,
                                     const int32_t* routed, const float* d_weights,
                                     const float* d_loss, void* d_logits, int64_t ld_d,
                                     hipStream_t stream) {
  return by_experts(E, [&](auto lpt, auto npl) {
    constexpr int LPT = decltype(lpt)::value, NPL = decltype(npl)::value;
    const int64_t groups = 256 / LPT;
    int64_t grid = (T + groups - 1) / groups;
    // four workgroups a CU, several tokens each (65536 x 256: 512 workgroups 22.1
    // us, 1024 17.3, 2048 18.6, 4096 20.6)
    if (grid > 1024) grid = 1024;
    const bool whole = rows_vec(logits, dtype, ld, E, NPL) && rows_vec(d_logits, dtype, ld_d, E, NPL);
    return by_rows(dtype, whole, [&](auto dt, auto vec) {
      route_backward_kernel<LPT, NPL, decltype(dt)::value, decltype(vec)::value>
          <<<(unsigned)grid, 256, 0, stream>>>(T, (int)E, topk, logits, ld, mask, renorm, expert_index,
                                               counts, routed, d_weights, d_loss, d_logits, ld_d);
      return hipGetLastError();
    });
  });
}

}  // namespace nvfp4
