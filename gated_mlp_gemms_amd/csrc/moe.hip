// Kernels of the mixture-of-experts layer around the experts' products: the router and its
// gradient, the counting sort of token choices by expert, and the rows there and back.
#include "common.hpp"
#include "launch.hpp"
#include "moe.h"
#include "rows.hpp"

#include <algorithm>

namespace gmlp {

namespace {

// ---- router ------------------------------------------------------------------------------------

// An unsigned key that orders as the scores do (-0 with +0, every NaN above +inf), and back. 0 is
// no score's key.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.0f);   // -0 + 0 = +0
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// A 16-bit score's key and its expert in one word that orders by score, then lowest expert first.
template <typename T> __device__ __forceinline__ uint32_t packed_key(float x, int e) {
  const float y = x + 0.0f;
  uint32_t h;   // y's own 16 bits, which it came from
  if constexpr (__is_same(T, bf16)) h = __float_as_uint(y) >> 16;
  else h = Bits16<T>::from_f32(y);
  const uint32_t key = x != x ? 0xffffu : h ^ ((h >> 15) ? 0xffffu : 0x8000u);
  return (key << 16) | (uint32_t)(0xffff - e);
}
template <typename T> __device__ __forceinline__ float packed_score(uint32_t m) {
  const uint32_t key = m >> 16;
  return Bits16<T>::to_f32(key ^ ((key >> 15) ? 0x8000u : 0xffffu));
}

constexpr int kRouteThreads = 256;

// The sigmoid of s and its complement, both to a few roundings of themselves: 1 - q from a rounded q cancels, and is 0
// from s = 17.4 on.
struct Sigmoid { float q, rest; };
__device__ __forceinline__ Sigmoid sigmoid_of(float s) {
  const float t = expf(-fabsf(s)), r = 1.0f / (1.0f + t);
  return s < 0.0f ? Sigmoid{t * r, r} : Sigmoid{r, t * r};
}

// Sigmoids divided by their sum over L lanes (`mine`: of those that take part; top: their largest score), as the
// exponentials that they are below 0, scaled by the largest: sigmoids themselves run out of range at -88, where
// their ratios are as they are elsewhere. Below -104 the largest counts as 0 (2^-150), and all weights are 0.
template <int L> __device__ __forceinline__ float sigmoid_share(float s, bool mine, float top) {
  const float shift = fminf(top, 0.0f);
  const float v = s < 0.0f ? expf(s - shift) / (1.0f + expf(s)) : sigmoid_of(s).q;
  const float w = mine ? v : 0.0f, total = group_sum<L>(w);
  return top < -104.0f ? 0.0f : w / total;
}

template <typename T, int C> struct ScorePart {   // C scores as one aligned piece
  static constexpr int B = C * (int)sizeof(T);
  struct alignas(B < 4 ? 4 : B < 16 ? B : 16) type { uint32_t w[(B + 3) / 4]; };
};

// The scores of lane `lane`'s experts lane C .. lane C + C - 1 of a row of E; `pad` past the row. Where C
// divides E a lane's scores are one aligned piece, loaded whole.
template <typename T, int C>
__device__ __forceinline__ void load_scores(const void* logits, int64_t row, int E, int lane, bool live, float pad,
                                            float (&x)[C]) {
  const int e0 = lane * C;
  if (C > 1 && E % C == 0) {
    using Part = typename ScorePart<T, C>::type;
    Part part = {};
    const bool in = live && e0 < E;
    if (in) part = *reinterpret_cast<const Part*>(reinterpret_cast<const char*>(logits) + (row * E + e0) * (int64_t)sizeof(T));
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if constexpr (sizeof(T) == 4) x[j] = in ? __uint_as_float(part.w[j]) : pad;
      else x[j] = in ? Bits16<T>::to_f32(j & 1 ? part.w[j / 2] >> 16 : part.w[j / 2] & 0xffffu) : pad;
    }
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j) x[j] = live && e0 + j < E ? load1<T>(logits, row * E + e0 + j) : pad;
  }
}

// L lanes a token, C scores a lane (lane l holds experts l C .. l C + C - 1). Each of the k rounds
// takes the largest key left, lowest expert first, and clears it. A 16-bit score and its expert fit one
// 32-bit key (upper half of the score's key, lower half counting experts down), so a round is one
// reduction; fp32 scores take a second one for the expert.
// 16384 tokens x 128 scores, k = 8: bound by the rounds' instructions (reading the scores takes 1 us).
template <typename T, int L, int C>
__device__ __forceinline__ void route_token(const void* __restrict__ logits, int64_t t, int64_t tokens, int E, int k,
                                            int sigmoid, int renorm, int* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & (L - 1);
  const bool live = t < tokens;
  constexpr bool PACKED = sizeof(T) == 2;
  float x[C];
  uint32_t key[C];
  load_scores<T, C>(logits, t, E, lane, live, 0.0f, x);
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int e = lane * C + j;
    if constexpr (PACKED) key[j] = e < E ? packed_key<T>(x[j], e) : 0u;
    else key[j] = e < E ? score_key(x[j]) : 0u;
  }

  int my_id = 0;
  float my_score = 0.0f, top = 0.0f;
  for (int i = 0; i < k; ++i) {
    uint32_t m = key[0];
#pragma unroll
    for (int j = 1; j < C; ++j) m = max(m, key[j]);
    m = group_max<L>(m);
    uint32_t at;
    float s;
    if constexpr (PACKED) {
#pragma unroll
      for (int j = 0; j < C; ++j) key[j] = key[j] == m ? 0u : key[j];   // keys are distinct
      at = 0xffffu - (m & 0xffffu);
      s = packed_score<T>(m);
    } else {
      at = 0xffffffffu;
#pragma unroll
      for (int j = C - 1; j >= 0; --j) at = key[j] == m ? (uint32_t)(lane * C + j) : at;
      at = group_min<L>(at);
#pragma unroll
      for (int j = 0; j < C; ++j) key[j] = at == (uint32_t)(lane * C + j) ? 0u : key[j];
      s = key_score(m);
    }
    if (i == 0) top = s;
    if (i == lane) {
      my_id = (int)at;
      my_score = s;
    }
  }
  const bool mine = lane < k;
  float w = 0.0f;
  if (sigmoid) {
    if (renorm) w = sigmoid_share<L>(my_score, mine, top);
    else w = mine ? sigmoid_of(my_score).q : 0.0f;
  } else if (top == -INFINITY) {   // every score is -inf: no expert has a probability
    w = 0.0f;
  } else {
    w = mine ? expf(my_score - top) : 0.0f;
    float part = 0.0f;
    if (renorm) {
      part = w;
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j) part += lane * C + j < E ? expf(x[j] - top) : 0.0f;
    }
    w /= group_sum<L>(part);
  }
  if (live && mine) {
    ids[t * k + lane] = my_id;
    weights[t * k + lane] = w;
  }
}
template <typename T, int L, int C>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const void* __restrict__ logits, int64_t tokens, int E,
                                                              int k, int sigmoid, int renorm, int* __restrict__ ids,
                                                              float* __restrict__ weights) {
  constexpr int R = kRouteThreads / L;
  for (int64_t t0 = (int64_t)blockIdx.x * R; t0 < tokens; t0 += (int64_t)gridDim.x * R)
    route_token<T, L, C>(logits, t0 + threadIdx.x / L, tokens, E, k, sigmoid, renorm, ids, weights);
}

// f(id, coefficient) of choice I, I + 1, .. k - 1, which lane I of the group holds. Lane I of 16 reaches its
// row as a DPP operand (row broadcast); wider groups shuffle.
template <int L, int I, typename F>
__device__ __forceinline__ void each_choice(int k, int id, float coef, F f) {
  if constexpr (I < 16) {
    if (I < k) {   // uniform
      if constexpr (L == 16)
        f((int)dpp<0x150 + I>((uint32_t)id), __uint_as_float(dpp<0x150 + I>(__float_as_uint(coef))));
      else
        f(__shfl(id, I, L), __shfl(coef, I, L));
      each_choice<L, I + 1>(k, id, coef, f);
    }
  }
}

// The gradient, same lanes. With w the weights and m = sum_i g_i w_i:
//   softmax, renormalised: a softmax of the chosen alone, dx_i = w_i (g_i - m) at the chosen ones;
//   softmax:               dx_e = [e chosen] w g - p_e m, p over every expert;
//   sigmoid, renormalised: dx_i = w_i (1 - q_i) (g_i - m);   sigmoid: q_i (1 - q_i) g_i.
// d: the gradient of the lane's C scores, which is added to.
template <typename T, int L, int C>
__device__ __forceinline__ void route_grad(const void* __restrict__ logits, const int* __restrict__ ids,
                                           const float* __restrict__ dweights, int64_t t, bool live, int E, int k,
                                           int sigmoid, int renorm, float (&d)[C]) {
  const int lane = threadIdx.x & (L - 1);
  int id = -1;
  float g = 0.0f, s = -INFINITY;
  if (live && lane < k) {
    id = ids[t * k + lane];
    if (id < 0 || id >= E) id = -1;
    else {
      g = dweights[t * k + lane];
      s = load1<T>(logits, t * E + id);
    }
  }
  const bool chosen = id >= 0;
  float coef = 0.0f;
  if (sigmoid) {
    const Sigmoid p = sigmoid_of(s);
    if (renorm) {
      const float top = key_score(group_max<L>(chosen ? score_key(s) : score_key(-INFINITY)));
      const float w = sigmoid_share<L>(s, chosen, top);
      const float mean = group_sum<L>(g * w);
      coef = w * p.rest * (g - mean);
    } else {
      coef = chosen ? p.q * p.rest * g : 0.0f;
    }
  } else if (renorm) {
    const float top = key_score(group_max<L>(chosen ? score_key(s) : score_key(-INFINITY)));
    if (top != -INFINITY) {
      const float e = chosen ? expf(s - top) : 0.0f;
      const float w = e / group_sum<L>(e);
      coef = w * (g - group_sum<L>(g * w));
    }
  } else {
    float x[C];
    uint32_t m = 0u;
    load_scores<T, C>(logits, t, E, lane, live, -INFINITY, x);
#pragma unroll
    for (int j = 0; j < C; ++j) m = max(m, score_key(x[j]));
    const float top = key_score(group_max<L>(m));
    if (top != -INFINITY) {
      float part = 0.0f;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        x[j] = expf(x[j] - top);
        part += x[j];
      }
      const float total = group_sum<L>(part);
      const float w = chosen ? expf(s - top) / total : 0.0f;
      const float mean = group_sum<L>(g * w);
      coef = w * g;
#pragma unroll
      for (int j = 0; j < C; ++j) d[j] += -(x[j] / total) * mean;   // what every expert gets, chosen or not
    }
  }
  each_choice<L, 0>(k, id, coef, [&](int at, float c) {
#pragma unroll
    for (int j = 0; j < C; ++j) d[j] += at == lane * C + j ? c : 0.0f;
  });
}

// The lane's C values of row t of an [tokens, E] tensor (load_scores' other way).
template <typename T, int C>
__device__ __forceinline__ void store_scores(void* __restrict__ dlogits, int64_t t, int E, int lane, const float (&d)[C]) {
  if (C > 1 && E % C == 0) {   // a lane's gradients are one aligned piece
    using Part = typename ScorePart<T, C>::type;
    Part part;
#pragma unroll
    for (int j = 0; j < (int)(sizeof part.w / 4); ++j) {
      if constexpr (sizeof(T) == 4) part.w[j] = __float_as_uint(d[j]);
      else part.w[j] = pack16x2<T>(d[2 * j], d[C > 1 ? 2 * j + 1 : 0]);
    }
    if (lane * C < E)
      *reinterpret_cast<Part*>(reinterpret_cast<char*>(dlogits) + (t * E + lane * C) * (int64_t)sizeof(T)) = part;
    return;
  }
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int e = lane * C + j;
    if (e < E) store1<T>(dlogits, t * E + e, d[j]);
  }
}
template <typename T, int L, int C>
__global__ __launch_bounds__(kRouteThreads) void route_bwd_kernel(const void* __restrict__ logits,
                                                                  const int* __restrict__ ids,
                                                                  const float* __restrict__ dweights, int64_t tokens,
                                                                  int E, int k, int sigmoid, int renorm,
                                                                  void* __restrict__ dlogits) {
  constexpr int R = kRouteThreads / L;
  for (int64_t t0 = (int64_t)blockIdx.x * R; t0 < tokens; t0 += (int64_t)gridDim.x * R) {
    const int64_t t = t0 + threadIdx.x / L;
    float d[C] = {};
    route_grad<T, L, C>(logits, ids, dweights, t, t < tokens, E, k, sigmoid, renorm, d);
    if (t < tokens) store_scores<T, C>(dlogits, t, E, threadIdx.x & (L - 1), d);
  }
}

// f(L, C) for the lanes a token and scores a lane that E takes.
template <typename F> hipError_t route_shape(int64_t E, F f) {
  using std::integral_constant;
  if (E <= 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (E <= 32) return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  if (E <= 64) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  if (E <= 128) return f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  if (E <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 8>{});
  if (E <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  return f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

// ---- balance loss ------------------------------------------------------------------------------

// A token's probabilities, in place of its C scores a lane (-inf past the row): softmax, or each expert's sigmoid divided by their
// sum (as sigmoid_share). A token without any, and a lane past the row, has zeros; a NaN makes its whole token NaN, through the
// sum, as the maximum passes it over. The exponentials are the hardware's, off by the
// rounding of their argument, |x| half steps (expf is a dozen instructions; 16384 x 128: 8.5 -> 7.1 us, the gradient 12.0 -> 11.2).
// A kernel a score function: short straight code, as every launch fetches it anew (with a branch a score and score_key's maximum
// the loss and the gradient together 22.6 us, so 20.8).
template <int L, int C, bool SIGMOID> __device__ __forceinline__ void balance_probs(float (&x)[C]) {
  float top = x[0];
#pragma unroll
  for (int j = 1; j < C; ++j) top = fmaxf(top, x[j]);
  top = __uint_as_float(group_reduce<L>(__float_as_uint(top), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
  const bool none = SIGMOID ? top < -104.0f : top == -INFINITY;
  const float shift = none ? 0.0f : SIGMOID ? fminf(top, 0.0f) : top;
  float part = 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    if constexpr (SIGMOID) x[j] = x[j] < 0.0f ? __expf(x[j] - shift) / (1.0f + __expf(x[j])) : 1.0f / (1.0f + __expf(-x[j]));
    else x[j] = __expf(x[j] - shift);
    part += x[j];
  }
  const float total = group_sum<L>(part);
  const float r = none && total == total ? 0.0f : 1.0f / total;
#pragma unroll
  for (int j = 0; j < C; ++j) x[j] *= r;
}

// The parts' sums added up, by one workgroup of 1024 threads: 2^sh >= E threads an expert's run of parts beside one another,
// joined in order.
__device__ __forceinline__ void balance_finish(const float* part_p, const int* part_c, int parts, int E, int k, int sh,
                                               int* __restrict__ counts, float* __restrict__ shares,
                                               float* __restrict__ loss) {
  __shared__ float ps[1024];
  __shared__ int cs[1024];
  __shared__ int live;
  __shared__ float waves[16];
  const int tid = threadIdx.x, e = tid & ((1 << sh) - 1), slice = tid >> sh, slices = 1024 >> sh;
  if (tid == 0) live = 0;
  __syncthreads();
  float p = 0.0f;
  int c = 0, n = 0;
  if (e < E) {
#pragma unroll 8
    for (int g = slice; g < parts; g += slices) {
      p += part_p[(int64_t)g * E + e];
      c += part_c[(int64_t)g * (E + 1) + e];
    }
  }
  for (int g = tid; g < parts; g += 1024) n += part_c[(int64_t)g * (E + 1) + E];
  if (n != 0) atomicAdd(&live, n);
  ps[tid] = p;
  cs[tid] = c;
  __syncthreads();
  n = live;
  float v = 0.0f;
  if (slice == 0 && e < E) {
    for (int s = 1; s < slices; ++s) {
      p += ps[tid + (s << sh)];
      c += cs[tid + (s << sh)];
    }
    p = n > 0 ? p / (float)n : 0.0f;
    counts[e] = c;
    shares[e] = p;
    v = n > 0 ? p * ((float)c / ((float)n * (float)k)) : 0.0f;
  }
  v = group_sum<64>(v);
  if ((tid & 63) == 0) waves[tid >> 6] = v;
  __syncthreads();
  if (tid != 0) return;
  v = 0.0f;
  for (int w = 0; w < 16; ++w) v += waves[w];
  counts[E] = n;
  loss[0] = (float)E * v;
}
__global__ __launch_bounds__(1024) void balance_join_kernel(const float* __restrict__ part_p, const int* __restrict__ part_c,
                                                            int parts, int E, int k, int sh, int* __restrict__ counts,
                                                            float* __restrict__ shares, float* __restrict__ loss) {
  balance_finish(part_p, part_c, parts, E, k, sh, counts, shares, loss);
}

// The workgroup's share of the tokens, `chunk` of them: its sums of the probabilities into part_p [E], its tokens an
// expert and its tokens that count into part_c [E + 1]. A lane has the same experts in every token, so their
// sums stay in registers; the groups of a wave, then the waves, are joined in order. A workgroup that has every token
// finishes by itself. 16384 x 128: bound by its trips to memory, so kBalanceAtOnce tokens of a group are under way at once, and
// the mask, read beside them, only chooses what is added (256 threads, a token at a time 15.6 us).
constexpr int kBalanceThreads = 1024, kBalanceAtOnce = 2;
template <typename T, int L, int C, bool SIGMOID>
__global__ __launch_bounds__(kBalanceThreads) void balance_kernel(const void* __restrict__ logits, const int* __restrict__ ids,
                                                                  const uint8_t* __restrict__ mask, int64_t tokens, int E,
                                                                  int k, int64_t chunk, float* part_p,
                                                                  int* part_c, int sh, int* __restrict__ counts,
                                                                  float* __restrict__ shares, float* __restrict__ loss) {
  constexpr int R = kBalanceThreads / L, W = kBalanceThreads / 64, U = kBalanceAtOnce;
  __shared__ int cnt[MOE_MAX_EXPERTS + 1];
  __shared__ float sums[W][L * C];
  const int tid = threadIdx.x, lane = tid & (L - 1);
  for (int e = tid; e <= E; e += kBalanceThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t beg = blockIdx.x * chunk, end = min(tokens, beg + chunk);
  float acc[C] = {};
  int seen = 0;
  for (int64_t t0 = beg; t0 < end; t0 += R * U) {
    float x[U][C];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * R + tid / L;
      load_scores<T, C>(logits, t, E, lane, t < end, -INFINITY, x[u]);
      live[u] = t < end && (mask == nullptr || mask[t] != 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      balance_probs<L, C, SIGMOID>(x[u]);
#pragma unroll
      for (int j = 0; j < C; ++j) acc[j] += live[u] ? x[u][j] : 0.0f;
      seen += live[u] ? 1 : 0;
    }
  }
  for (int64_t i = beg * k + tid; i < end * k; i += kBalanceThreads) {
    const int id = ids[i];
    const bool live = mask == nullptr || mask[i / k] != 0;
    if ((uint32_t)id < (uint32_t)E && live) atomicAdd(&cnt[id], 1);
  }
  if (lane == 0) atomicAdd(&cnt[E], seen);
#pragma unroll
  for (int j = 0; j < C; ++j) {
#pragma unroll
    for (int o = L; o < 64; o <<= 1) acc[j] += __shfl_xor(acc[j], o);
    if ((tid & 63) < L) sums[tid >> 6][lane * C + j] = acc[j];
  }
  __syncthreads();
  for (int e = tid; e < E; e += kBalanceThreads) {
    float s = sums[0][e];
#pragma unroll
    for (int w = 1; w < W; ++w) s += sums[w][e];
    part_p[(int64_t)blockIdx.x * E + e] = s;
  }
  for (int e = tid; e <= E; e += kBalanceThreads) part_c[(int64_t)blockIdx.x * (E + 1) + e] = cnt[e];
  if (gridDim.x > 1) return;
  __syncthreads();
  balance_finish(part_p, part_c, 1, E, k, sh, counts, shares, loss);
}

// The gradient: with a_e = dloss E counts_e / (n^2 k) and m = sum_e p_e a_e, p_e (a_e - m), of sigmoid scores times
// 1 - q_e; on top of the chosen weights' (dweights NULL: none), both rounded once.
template <typename T, int L, int C, bool SIGMOID>
__global__ __launch_bounds__(kRouteThreads) void balance_bwd_kernel(const void* __restrict__ logits, const int* __restrict__ ids,
                                                                    const uint8_t* __restrict__ mask,
                                                                    const int* __restrict__ counts,
                                                                    const float* __restrict__ dloss,
                                                                    const float* __restrict__ dweights, int64_t tokens,
                                                                    int E, int k, int renorm,
                                                                    void* __restrict__ dlogits) {
  constexpr int R = kRouteThreads / L;
  const int lane = threadIdx.x & (L - 1);
  int c[C];   // loaded at once, whatever is past the experts
#pragma unroll
  for (int j = 0; j < C; ++j) c[j] = counts[min(lane * C + j, E)];
  const float n = (float)counts[E];
  const float each = n > 0.0f ? (dloss != nullptr ? dloss[0] : 1.0f) * ((float)E / (n * (float)k)) / n : 0.0f;
  float a[C];
#pragma unroll
  for (int j = 0; j < C; ++j) a[j] = lane * C + j < E ? each * (float)c[j] : 0.0f;
  for (int64_t t0 = (int64_t)blockIdx.x * R; t0 < tokens; t0 += (int64_t)gridDim.x * R) {
    const int64_t t = t0 + threadIdx.x / L;
    const bool in = t < tokens, live = in && (mask == nullptr || mask[t] != 0);
    float x[C], d[C], rest[C];
    load_scores<T, C>(logits, t, E, lane, in, -INFINITY, x);   // (not `live`: the mask would be one more trip to memory first)
#pragma unroll
    for (int j = 0; j < C; ++j) rest[j] = SIGMOID ? sigmoid_of(x[j]).rest : 1.0f;
    balance_probs<L, C, SIGMOID>(x);
    float part = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) part = __builtin_fmaf(x[j], a[j], part);
    const float m = group_sum<L>(part);
#pragma unroll
    for (int j = 0; j < C; ++j) d[j] = live ? x[j] * rest[j] * (a[j] - m) : 0.0f;
    if (dweights != nullptr) route_grad<T, L, C>(logits, ids, dweights, t, in, E, k, SIGMOID, renorm, d);
    if (in) store_scores<T, C>(dlogits, t, E, lane, d);
  }
}

// ---- tokens by expert ----------------------------------------------------------------------------

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSortBins = MOE_MAX_EXPERTS + 1;   // one an expert, and the dropped

__device__ __forceinline__ int sort_bin(int id, int E) { return id < 0 || id >= E ? E : id; }

// counts[chunk][bin] of the chunk's ids.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const int* __restrict__ ids, int n, int E, int chunk,
                                                                  int* __restrict__ counts) {
  __shared__ int cnt[kSortBins];
  const int nb = E + 1;
  for (int b = threadIdx.x; b < nb; b += kSortThreads) cnt[b] = 0;
  __syncthreads();
  const int beg = blockIdx.x * chunk, end = min(n, beg + chunk);
  for (int i = beg + (int)threadIdx.x; i < end; i += kSortThreads) atomicAdd(&cnt[sort_bin(ids[i], E)], 1);
  __syncthreads();
  for (int b = threadIdx.x; b < nb; b += kSortThreads) counts[(int64_t)blockIdx.x * nb + b] = cnt[b];
}

// One workgroup a chunk of ids: the rows of its slots. A bin's first row is the count of lower bins
// (every chunk) plus the bin's count in earlier chunks; inside the chunk each wave owns a run of
// consecutive ids, counts its bins (integer atomics: any order gives the same sums), and after a
// scan over the waves places its ids 64 at a time, equal bins ranked by lane. Chunks are taken in
// order throughout, so the sort is stable and the same on every run.
// counts: per-chunk counts of sort_count_kernel, or NULL with a single chunk.
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const int* __restrict__ ids, int n, int E, int bits,
                                                                  int chunk, const int* __restrict__ counts,
                                                                  int* __restrict__ offsets, int* __restrict__ row_of,
                                                                  int* __restrict__ slot_of) {
  __shared__ int cnt[kSortWaves][kSortBins];   // a wave's count of a bin, then its next row
  __shared__ int wave_sum[kSortWaves];
  const int nb = E + 1, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int beg = blockIdx.x * chunk, end = min(n, beg + chunk);
  const int run = chunk / kSortWaves;   // a multiple of 64
  const int wbeg = beg + wave * run, wend = min(end, wbeg + run);
  for (int b = lane; b < nb; b += 64) cnt[wave][b] = 0;
  __builtin_amdgcn_wave_barrier();
  for (int i = wbeg + lane; i < wend; i += 64) atomicAdd(&cnt[wave][sort_bin(ids[i], E)], 1);
  __syncthreads();

  // thread b: bin b's count over every chunk and over the chunks before this one
  const int bin = tid;   // nb <= kSortThreads + 1; the bin past the last thread is done by that thread, which holds the scan's total
  auto totals = [&](int b, int& all, int& before) {
    all = before = 0;
    if (b >= nb) return;
    if (counts == nullptr) {
      for (int w = 0; w < kSortWaves; ++w) all += cnt[w][b];
      return;
    }
    const int chunks = (int)gridDim.x, mine = (int)blockIdx.x;
#pragma unroll 8
    for (int c = 0; c < chunks; ++c) {
      const int v = counts[(int64_t)c * nb + b];
      all += v;
      before += c < mine ? v : 0;
    }
  };
  int all, before;
  totals(bin, all, before);
  // exclusive scan of `all` over the workgroup's threads
  int incl = all;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  int base = incl - all;
  for (int w = 0; w < wave; ++w) base += wave_sum[w];
  auto place_bin = [&](int b, int first, int earlier) {
    if (b >= nb) return;
    if (blockIdx.x == 0) offsets[b] = first;   // offsets[E] = the rows of every expert
    int row = first + earlier;
    for (int w = 0; w < kSortWaves; ++w) {
      const int v = cnt[w][b];
      cnt[w][b] = row;
      row += v;
    }
  };
  place_bin(bin, base, before);
  if (nb > kSortThreads && tid == kSortThreads - 1) {   // E = kSortThreads: the bin of the dropped
    int all2, before2;
    totals(kSortThreads, all2, before2);
    place_bin(kSortThreads, base + all, before2);
  }
  __syncthreads();

  for (int i0 = wbeg; i0 < wend; i0 += 64) {   // uniform over the wave
    const int i = i0 + lane;
    const bool live = i < wend;
    const int b = live ? sort_bin(ids[i], E) : 0;
    uint64_t peers = __ballot(live);
    for (int q = 0; q < bits; ++q) {
      const uint64_t one = __ballot((b >> q) & 1);
      peers &= ((b >> q) & 1) ? one : ~one;
    }
    const int rank = __builtin_popcountll(peers & ((1ull << lane) - 1ull));
    const int first = live ? cnt[wave][b] : 0;
    __builtin_amdgcn_wave_barrier();   // every lane has read before the last of each bin advances it
    if (live) {
      if (rank + 1 == __builtin_popcountll(peers)) cnt[wave][b] = first + rank + 1;
      const int row = first + rank;
      row_of[i] = row;
      slot_of[row] = i;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- rows there and back -------------------------------------------------------------------------

constexpr int kRowThreads = 256;

// A row of `pieces` 16-byte pieces is walked by 2^sh threads; kRowThreads >> sh rows a workgroup. (Fewer threads a row
// where they would leave fewer turns idle: 5003 tokens of 259 pieces there and back 108 -> 115 us.)
inline int row_shift(int64_t pieces) {
  int sh = 0;
  while (sh < 8 && (int64_t)(1 << sh) < pieces) ++sh;
  return sh;
}
inline unsigned row_grid(int64_t rows, int sh) { return item_grid(rows, kRowThreads >> sh); }

// Rows that no cache will hold until they are read again are streamed (NT: non-temporal loads of the
// rows read once, non-temporal stores): from 32 MiB of sorted rows on. Bound by HBM. Gather, combine and both gradients
// one after another, rows in caches and streamed (us): 6 rows of 2048 bf16 a token, 20 MB 31.7 and 32.5, 30 MB 46 and 41,
// 45 MB 65 and 56, 104 MB 151 and 124, 200 MB 267 and 222 (gather 68 -> 54, combine 54 -> 43, its gradient 88 -> 84,
// gather's 49 -> 40); 3 rows of 1036 fp32, 20 MB 37.5 and 38.4, 45 MB 77 and 71, 62 MB 98 and 92. The two products between
// gather and combine of a layer do not miss the rows: 2048 x 1376, 4 a token, with them 20 MB 121 and 121, 45 MB 216 and
// 208, 104 MB 388 and 395, 150 MB 554 and 552; 2048 x 256, 6 a token, 20 MB 53 and 55, 62 MB 118 and 105, 150 MB 250 and 230.
constexpr int64_t kStreamBytes = 32 << 20;
inline bool stream_rows(int64_t rows, int pieces) { return rows * pieces * 16 >= kStreamBytes; }

// xs[r] = x[slot_of[r] / k]: a row is moved as it is, in 16-byte pieces.
template <bool NT>
__global__ __launch_bounds__(kRowThreads) void gather_kernel(const u32x4* __restrict__ x,
                                                             const int* __restrict__ slot_of,
                                                             const int* __restrict__ offsets, int n, int E, int k,
                                                             int pieces, int sh, u32x4* __restrict__ xs) {
  const int per = kRowThreads >> sh;
  for (int r = blockIdx.x * per + (threadIdx.x >> sh); r < n; r += gridDim.x * per) {
    const int slot = slot_of[r];
    const bool kept = r < offsets[E] && (uint32_t)slot < (uint32_t)n;
    const u32x4* src = x + (int64_t)(kept ? slot / k : 0) * pieces;
    u32x4* dst = xs + (int64_t)r * pieces;
    for (int c = threadIdx.x & ((1 << sh) - 1); c < pieces; c += 1 << sh)
      store_piece<NT>(dst + c, kept ? src[c] : u32x4{0u, 0u, 0u, 0u});
  }
}

// out[t] = residual[t] + sum_j weights[t][j] ys[row_of[t k + j]] over the kept rows (weights NULL: 1,
// residual NULL: 0). The k rows of a piece are loaded J at a time before they are
// summed in order.
template <typename T, int J, bool NT>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(const u32x4* __restrict__ ys,
                                                              const float* __restrict__ weights,
                                                              const int* __restrict__ row_of,
                                                              const int* __restrict__ offsets, const u32x4* residual,
                                                              int tokens, int E, int k, int pieces, int sh,
                                                              u32x4* out) {
  constexpr int N = Piece<T>::N;
  const int per = kRowThreads >> sh, kept = min(offsets[E], tokens * k);
  for (int t = blockIdx.x * per + (threadIdx.x >> sh); t < tokens; t += gridDim.x * per) {
    for (int c = threadIdx.x & ((1 << sh) - 1); c < pieces; c += 1 << sh) {
      float acc[N];
  #pragma unroll
      for (int q = 0; q < N; ++q) acc[q] = 0.0f;
      for (int j0 = 0; j0 < k; j0 += J) {
        u32x4 v[J];
        float w[J];
        bool ok[J];
  #pragma unroll
        for (int j = 0; j < J; ++j) {
          const int64_t slot = (int64_t)t * k + j0 + j;
          const int row = j0 + j < k ? row_of[slot] : -1;
          ok[j] = row >= 0 && row < kept;
          w[j] = ok[j] && weights != nullptr ? weights[slot] : 1.0f;
          v[j] = ok[j] ? load_piece<NT>(ys + (int64_t)row * pieces + c) : u32x4{0u, 0u, 0u, 0u};
        }
  #pragma unroll
        for (int j = 0; j < J; ++j) {
          if (!ok[j]) continue;
          float f[N];
          Piece<T>::unpack(v[j], f);
  #pragma unroll
          for (int q = 0; q < N; ++q) acc[q] = __builtin_fmaf(w[j], f[q], acc[q]);
        }
      }
      if (residual != nullptr) {
        float f[N];
        Piece<T>::unpack(residual[(int64_t)t * pieces + c], f);
  #pragma unroll
        for (int q = 0; q < N; ++q) acc[q] += f[q];
      }
      store_piece<NT>(out + (int64_t)t * pieces + c, Piece<T>::pack(acc));
    }
  }
}

// A wave a row r: with t the row's token, dys[r] = weight dout[t] and the weight's gradient
// dot(ys[r], dout[t]); zeros for a dropped row.
template <typename T, bool NT>
__global__ __launch_bounds__(kRowThreads) void combine_bwd_kernel(const u32x4* __restrict__ dout,
                                                                  const u32x4* __restrict__ ys,
                                                                  const float* __restrict__ weights,
                                                                  const int* __restrict__ slot_of,
                                                                  const int* __restrict__ offsets, int n, int E, int k,
                                                                  int pieces, u32x4* __restrict__ dys,
                                                                  float* __restrict__ dweights) {
  constexpr int N = Piece<T>::N;
  const int lane = threadIdx.x & 63;
  for (int r = blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6); r < n; r += gridDim.x * (kRowThreads / 64)) {
    const int slot = slot_of[r];
    const bool known = (uint32_t)slot < (uint32_t)n, kept = known && r < offsets[E];
    u32x4* dst = dys + (int64_t)r * pieces;
    float dot = 0.0f;
    if (kept) {
      const float w = weights[slot];
      const u32x4* g = dout + (int64_t)(slot / k) * pieces;
      const u32x4* y = ys + (int64_t)r * pieces;
  #pragma unroll 4
      for (int c = lane; c < pieces; c += 64) {
        float gv[N], yv[N], o[N];
        Piece<T>::unpack(g[c], gv);
        Piece<T>::unpack(load_piece<NT>(y + c), yv);
  #pragma unroll
        for (int q = 0; q < N; ++q) {
          dot = __builtin_fmaf(gv[q], yv[q], dot);
          o[q] = w * gv[q];
        }
        store_piece<NT>(dst + c, Piece<T>::pack(o));
      }
  #pragma unroll
      for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
    } else {
      for (int c = lane; c < pieces; c += 64) dst[c] = u32x4{0u, 0u, 0u, 0u};
    }
    if (known && lane == 0) dweights[slot] = dot;
  }
}

template <typename F> hipError_t by_stream(int64_t rows, int pieces, F f) {
  return stream_rows(rows, pieces) ? f(std::true_type{}) : f(std::false_type{});
}

}  // namespace

hipError_t run_moe_route(DType dt, const void* logits, int64_t T, int E, int k, int sigmoid, int renorm, int* ids,
                         float* weights, hipStream_t s) {
  return by_type(dt, [&](auto v) {
    return route_shape(E, [&](auto l, auto c) {
      constexpr int L = decltype(l)::value, C = decltype(c)::value, R = kRouteThreads / L;
      hipLaunchKernelGGL((route_kernel<decltype(v), L, C>), dim3(item_grid(T, R)), dim3(kRouteThreads), 0, s,
                         logits, T, E, k, sigmoid, renorm, ids, weights);
      return hipGetLastError();
    });
  });
}

hipError_t run_moe_route_bwd(DType dt, const void* logits, const int* ids, const float* dweights, int64_t T, int E,
                             int k, int sigmoid, int renorm, void* dlogits, hipStream_t s) {
  return by_type(dt, [&](auto v) {
    return route_shape(E, [&](auto l, auto c) {
      constexpr int L = decltype(l)::value, C = decltype(c)::value, R = kRouteThreads / L;
      hipLaunchKernelGGL((route_bwd_kernel<decltype(v), L, C>), dim3(item_grid(T, R)), dim3(kRouteThreads), 0,
                         s, logits, ids, dweights, T, E, k, sigmoid, renorm, dlogits);
      return hipGetLastError();
    });
  });
}

// Tokens of a workgroup of balance_kernel: whole turns of its groups, at most kBalanceParts workgroups; few tokens one workgroup.
constexpr int64_t kBalanceParts = 128, kBalanceSingle = 4;   // (turns)
static int64_t balance_chunk(int64_t T, int E) {
  int64_t r = 1;
  (void)route_shape(E, [&](auto l, auto) {
    r = kBalanceThreads / decltype(l)::value;
    return hipSuccess;
  });
  if (T <= kBalanceSingle * r) return kBalanceSingle * r;
  return std::max<int64_t>(kBalanceAtOnce * r, ((T + kBalanceParts - 1) / kBalanceParts + r - 1) / r * r);
}
int moe_balance_parts(int64_t T, int E) {
  const int64_t c = balance_chunk(T, E);
  return (int)((T + c - 1) / c);
}

hipError_t run_moe_balance(DType dt, const void* logits, const int* ids, const uint8_t* mask, int64_t T, int E, int k,
                           int sigmoid, int* counts, float* shares, float* loss, void* ws, hipStream_t s) {
  const int parts = moe_balance_parts(T, E);
  float* part_p = static_cast<float*>(ws);
  int* part_c = reinterpret_cast<int*>(part_p + (int64_t)parts * E);
  int sh = 6;
  while ((1 << sh) < E) ++sh;
  if (parts > 0) {
    const hipError_t e = by_type(dt, [&](auto v) {
      return route_shape(E, [&](auto l, auto c) {
        constexpr int L = decltype(l)::value, C = decltype(c)::value;
        const auto kernel = sigmoid ? balance_kernel<decltype(v), L, C, true> : balance_kernel<decltype(v), L, C, false>;
        hipLaunchKernelGGL(kernel, dim3(parts), dim3(kBalanceThreads), 0, s, logits, ids, mask, T, E, k, balance_chunk(T, E),
                           part_p, part_c, sh, counts, shares, loss);
        return hipGetLastError();
      });
    });
    if (e != hipSuccess || parts == 1) return e;
  }
  hipLaunchKernelGGL(balance_join_kernel, dim3(1), dim3(1024), 0, s, part_p, part_c, parts, E, k, sh, counts, shares, loss);
  return hipGetLastError();
}

hipError_t run_moe_balance_bwd(DType dt, const void* logits, const int* ids, const uint8_t* mask, const int* counts,
                               const float* dloss, const float* dweights, int64_t T, int E, int k, int sigmoid, int renorm,
                               void* dlogits, hipStream_t s) {
  return by_type(dt, [&](auto v) {
    return route_shape(E, [&](auto l, auto c) {
      constexpr int L = decltype(l)::value, C = decltype(c)::value, R = kRouteThreads / L;
      const auto kernel = sigmoid ? balance_bwd_kernel<decltype(v), L, C, true> : balance_bwd_kernel<decltype(v), L, C, false>;
      hipLaunchKernelGGL(kernel, dim3(item_grid(T, R)), dim3(kRouteThreads), 0, s, logits, ids, mask, counts, dloss, dweights, T,
                         E, k, renorm, dlogits);
      return hipGetLastError();
    });
  });
}

// Ids a chunk: one workgroup's worth up to kSortSingle, else about 64 chunks of at least 1024.
constexpr int64_t kSortSingle = 4096;
static int64_t sort_chunk(int64_t n) {
  if (n <= kSortSingle) return kSortSingle;
  return std::max<int64_t>(1024, ((n + 63) / 64 + 1023) / 1024 * 1024);
}
size_t moe_sort_counts_bytes(int64_t n, int E) {
  const int64_t c = sort_chunk(n);
  return n <= kSortSingle ? 0 : (size_t)((n + c - 1) / c) * (E + 1) * sizeof(int);
}

hipError_t run_moe_sort(const int* ids, int64_t n, int E, int* offsets, int* row_of, int* slot_of, int* counts,
                        hipStream_t s) {
  const int chunk = (int)sort_chunk(n), chunks = (int)std::max<int64_t>(1, (n + chunk - 1) / chunk);
  int bits = 0;
  while ((1 << bits) <= E) ++bits;   // bins 0 .. E
  if (chunks > 1) {
    hipLaunchKernelGGL(sort_count_kernel, dim3(chunks), dim3(kSortThreads), 0, s, ids, (int)n, E, chunk, counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(sort_place_kernel, dim3(chunks), dim3(kSortThreads), 0, s, ids, (int)n, E, bits, chunk,
                     chunks > 1 ? counts : nullptr, offsets, row_of, slot_of);
  return hipGetLastError();
}

hipError_t run_moe_gather(const void* x, const int* slot_of, const int* offsets, int n, int E, int k, int pieces,
                          void* xs, hipStream_t s) {
  const int sh = row_shift(pieces);
  return by_stream(n, pieces, [&](auto nt) {
    hipLaunchKernelGGL((gather_kernel<decltype(nt)::value>), dim3(row_grid(n, sh)), dim3(kRowThreads), 0, s,
                       static_cast<const u32x4*>(x), slot_of, offsets, n, E, k, pieces, sh, static_cast<u32x4*>(xs));
    return hipGetLastError();
  });
}

hipError_t run_moe_combine(DType dt, const void* ys, const float* weights, const int* row_of, const int* offsets,
                           const void* residual, int T, int E, int k, int pieces, void* out, hipStream_t s) {
  const int sh = row_shift(pieces);
  return by_type(dt, [&](auto v) {
    auto launch = [&](auto j) {   // J: rows of a token in flight at once
      return by_stream((int64_t)T * k, pieces, [&](auto nt) {
        hipLaunchKernelGGL((combine_kernel<decltype(v), decltype(j)::value, decltype(nt)::value>),
                           dim3(row_grid(T, sh)), dim3(kRowThreads), 0, s, static_cast<const u32x4*>(ys),
                           weights, row_of, offsets, static_cast<const u32x4*>(residual), T, E, k, pieces, sh,
                           static_cast<u32x4*>(out));
        return hipGetLastError();
      });
    };
    using std::integral_constant;
    if (k <= 2) return launch(integral_constant<int, 2>{});
    return k <= 4 ? launch(integral_constant<int, 4>{}) : launch(integral_constant<int, 8>{});
  });
}

hipError_t run_moe_combine_bwd(DType dt, const void* dout, const void* ys, const float* weights, const int* slot_of,
                               const int* offsets, int n, int E, int k, int pieces, void* dys, float* dweights,
                               hipStream_t s) {
  return by_type(dt, [&](auto v) {
    return by_stream(n, pieces, [&](auto nt) {
      hipLaunchKernelGGL((combine_bwd_kernel<decltype(v), decltype(nt)::value>), dim3(item_grid(n, kRowThreads / 64)),
                         dim3(kRowThreads), 0, s, static_cast<const u32x4*>(dout), static_cast<const u32x4*>(ys),
                         weights, slot_of, offsets, n, E, k, pieces, static_cast<u32x4*>(dys), dweights);
      return hipGetLastError();
    });
  });
}

}  // namespace gmlp
