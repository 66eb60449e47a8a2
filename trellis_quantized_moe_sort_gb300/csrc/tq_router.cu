// Scored router: softmax or sigmoid scores, a bias that balances the choice,
// groups of experts, top-k and renormalised weights; and its gradient.
//
// One warp per token.  Lane l holds the experts l * PL .. l * PL + PL - 1 of
// the row (PL a power of two, 32 PL >= E), so that a row is read in 16-byte
// pieces and the lowest lane of a tie holds the lowest expert.
//
// The choice compares fp32 values, and a token whose candidates are an ulp
// apart changes its experts with the order of a sum.  So every operation on
// the way to the comparison has one order: the sigmoid is 1 / (1 + exp(-x)),
// the reciprocal rounded to nearest, no contraction; the softmax's denominator is a
// balanced tree over neighbouring experts (a power of two of them, absent ones
// zero), first in a lane's registers, then across lanes 1, 2, 4, 8 and 16
// apart; a group's value is one addition.  The result depends on the token's
// row alone, not on the batch or the launch.
//
// Bound: 8192 x 256 fp32 logits are 8.4 MB, 1.3 us of HBM time, so both
// directions are bound by the issue of a row's instructions (eight exponentials
// and reciprocals a lane, then the rounds of the choice) and by the launch:
// 10.6 us forward (top-6 of 256 in 8 groups, biased sigmoid), 6.7 us backward
// (softmax; sigmoid 5.7).  One row per warp, 64 registers, so 32 warps live on an SM; held to
// 48 or 40 registers it took 0.2 and 0.6 us more.
#include <cuda_runtime.h>

#include <algorithm>

#include "tq_device.cuh"
#include "tq_internal.h"
#include "tq_types.cuh"

namespace tq {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRouterThreads = 128;
constexpr int kRouterWarps = kRouterThreads / 32;
constexpr uint32_t kKeyMasked = 0x007fffffu;   // order_key(-infinity)

// Order-preserving map of fp32 (no NaN, no negative zero) to uint32.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

// x[i] = logit of expert lane * PL + i, -infinity where it is not finite or
// past the row.  `vec`: every lane's piece starts on a 16-byte boundary (or is
// the whole of a narrower, naturally aligned piece).
template <typename T, int PL>
__device__ __forceinline__ void load_row(const T* __restrict__ row, int E, int lane, bool vec, float (&x)[PL]) {
  const int e0 = lane * PL;
  constexpr int kVec = PL * static_cast<int>(sizeof(T)) >= 16 ? 16 / static_cast<int>(sizeof(T)) : PL;
#pragma unroll
  for (int i = 0; i < PL; i += kVec) {
    if (vec && kVec * sizeof(T) == 16 && e0 + i + kVec <= E) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(row + e0 + i));
      const T* const t = reinterpret_cast<const T*>(&q);
#pragma unroll
      for (int j = 0; j < kVec; ++j) x[i + j] = widen(t[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) x[i + j] = e0 + i + j < E ? widen(row[e0 + i + j]) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) x[i] = fabsf(x[i]) < INFINITY ? x[i] : -INFINITY;   // false for NaN too
}

// 1 / (1 + exp(-x)); 0 for a masked logit.
__device__ __forceinline__ float sigmoid_score(float x) {
  return x == -INFINITY ? 0.f : __frcp_rn(__fadd_rn(1.f, expf(-x)));
}

// The softmax's numerator; 0 for a masked logit.
__device__ __forceinline__ float softmax_term(float x, float top) {
  return x == -INFINITY ? 0.f : expf(__fsub_rn(x, top));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Largest logit of the row and the tree sum of the softmax's terms; the terms
// replace x.
template <int PL>
__device__ __forceinline__ void softmax_terms(float (&x)[PL], float* top, float* total) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < PL; ++i) m = fmaxf(m, x[i]);
  m = warp_max(m);
  float t[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) t[i] = x[i] = softmax_term(x[i], m);
#pragma unroll
  for (int w = 1; w < PL; w <<= 1) {
#pragma unroll
    for (int i = 0; i < PL; i += 2 * w) t[i] = __fadd_rn(t[i], t[i + w]);
  }
  float s = t[0];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(kAll, s, o));
  *top = m;
  *total = s;
}

// term / total rounded to nearest, r = 1 / total rounded to nearest (total is 1
// to 1024): by the residual of the product with r, which is exact in an FMA
// (Markstein 1990), where nothing underflows.
__device__ __forceinline__ float softmax_score(float term, float total, float r) {
  if (term < 0x1p-100f) return term > 0.f ? __fdiv_rn(term, total) : 0.f;
  const float q = __fmul_rn(term, r);
  return __fmaf_rn(__fmaf_rn(-q, total, term), r, q);
}

// The score of one expert's logit, as the row's scores were computed.
__device__ __forceinline__ float one_score(float x, int score, float top, float total) {
  if (!(fabsf(x) < INFINITY)) return 0.f;
  return score == TQ_SCORE_SIGMOID ? sigmoid_score(x) : softmax_score(softmax_term(x, top), total, __frcp_rn(total));
}

// Two largest of the four values in (a1 >= a2) and (b1 >= b2).
__device__ __forceinline__ void merge_top2(float& a1, float& a2, float b1, float b2) {
  const float hi = fmaxf(a1, b1), lo = fminf(a1, b1);
  a2 = fmaxf(lo, fmaxf(a2, b2));
  a1 = hi;
}

// Bit g * W of the result: group g stays.  c: the row's selection values in
// shared memory.  W = the largest power of two of lanes that each of `groups`
// groups can have; lane g * W + s takes every W-th value of group g, starting
// g * W values in so that the lanes of different groups meet in different banks.
__device__ __forceinline__ unsigned choose_groups(const float* c, int groups, int size, int top_groups, int W,
                                                  int lane) {
  const int g = lane / W, s = lane & (W - 1);
  float a1 = -INFINITY, a2 = -INFINITY;
  if (g < groups) {
    const float* const mine = c + g * size;
    int at = s < size ? (s + g * W) % size : 0;
    for (int i = s; i < size; i += W) {
      merge_top2(a1, a2, mine[at], -INFINITY);
      at += W;
      while (at >= size) at -= size;
    }
  }
  for (int o = 1; o < W; o <<= 1)
    merge_top2(a1, a2, __shfl_xor_sync(kAll, a1, o), __shfl_xor_sync(kAll, a2, o));
  float value = size > 1 ? __fadd_rn(a1, a2) : a1;
  if (!(value == value)) value = -INFINITY;
  int better = 0;
  for (int i = 0; i < groups; ++i) {
    const float other = __shfl_sync(kAll, value, i * W);
    better += (other > value || (other == value && i < g)) ? 1 : 0;
  }
  return __ballot_sync(kAll, g < groups && s == 0 && better < top_groups);
}

// The same for groups of whole lanes (PL divides their size and `lanes`, the
// lanes of one, is a power of two), from the values in registers; true in every
// lane of a group that stays.
template <int PL>
__device__ __forceinline__ bool choose_lane_groups(const float (&c)[PL], int groups, int top_groups, int lanes,
                                                   int lane) {
  float a1 = c[0], a2 = -INFINITY;
#pragma unroll
  for (int i = 1; i < PL; ++i) {
    a2 = fmaxf(a2, fminf(a1, c[i]));
    a1 = fmaxf(a1, c[i]);
  }
  for (int o = 1; o < lanes; o <<= 1)
    merge_top2(a1, a2, __shfl_xor_sync(kAll, a1, o), __shfl_xor_sync(kAll, a2, o));
  float value = PL * lanes > 1 ? __fadd_rn(a1, a2) : a1;
  if (!(value == value)) value = -INFINITY;
  // lanes past the last group have the lowest key
  uint32_t key = lane < groups * lanes ? order_key(__fadd_rn(value, 0.f)) : 0u;
  bool stays = false;
  for (int i = 0; i < top_groups; ++i) {
    const uint32_t best = __reduce_max_sync(kAll, key);
    const int first = __ffs(__ballot_sync(kAll, key == best)) - 1;   // the lowest group that has it
    if ((lane ^ first) < lanes) {   // of the same group
      stays = true;
      key = 0u;
    }
  }
  return stays;
}

// The top_k largest keys, by rounds over at most 32 of them, one per lane: those
// that are no smaller than the top_k-th largest of the lanes' maxima, which at
// least top_k keys are.  Lane j gets the j-th of the order (the lower expert
// first where keys tie).  False, with nothing chosen, where more keys are left
// (ties, or a choice confined to a few lanes by its groups).  At 8192 rows of 256
// a round over the lanes' whole pieces costs 0.65 us, one of these 0.18 and their
// gathering 0.6: 10.9 -> 9.4 us for top-6, 14.9 -> 10.3 for top-12, 7.7 -> 8.5 for
// top-1, so one or two experts are taken from the whole pieces.
template <int PL>
__device__ __forceinline__ bool choose_from_few(const uint32_t (&key)[PL], int top_k, int lane, uint2* few, int* e,
                                                uint32_t* k) {
  uint32_t head = key[0];
#pragma unroll
  for (int i = 1; i < PL; ++i) head = max(head, key[i]);
  uint32_t least = 0;
  for (int j = 0; j < top_k; ++j) {
    least = __reduce_max_sync(kAll, head);
    if (head == least) head = 0u;
  }
  if (least <= kKeyMasked) return false;
  const unsigned below = (1u << lane) - 1u;
  int count = 0;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const bool in = key[i] >= least;
    const unsigned all = __ballot_sync(kAll, in);
    const int at = count + __popc(all & below);
    if (in && at < 32) few[at] = make_uint2(key[i], lane * PL + i);
    count += __popc(all);
  }
  __syncwarp();
  if (count > 32) return false;
  uint2 mine = lane < count ? few[lane] : make_uint2(0u, 0u);
  __syncwarp();   // read before the next row's are written
  for (int j = 0; j < top_k; ++j) {
    const uint32_t best = __reduce_max_sync(kAll, mine.x);
    const uint32_t which = __reduce_min_sync(kAll, mine.x == best ? mine.y : 0xffffffffu);
    if (mine.x == best && mine.y == which) mine.x = 0u;
    if (lane == j) {
      *e = static_cast<int>(which);
      *k = best;
    }
  }
  return true;
}

template <typename T, int PL>
__global__ void __launch_bounds__(kRouterThreads)
router_scored_kernel(const T* __restrict__ logits, long long stride, const float* __restrict__ bias, int n, int E,
                     int top_k, int score, int groups, int top_groups, int lane_groups, int group_lanes, int renorm,
                     float scale, bool vec, int32_t* __restrict__ ids, float* __restrict__ w) {
  extern __shared__ float rows[];   // [warps][E], with groups only
  __shared__ uint2 few[kRouterWarps][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e0 = lane * PL;
  float b[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) b[i] = bias && e0 + i < E ? __ldg(bias + e0 + i) : 0.f;
  for (long long t = blockIdx.x * kRouterWarps + warp; t < n; t += gridDim.x * kRouterWarps) {
    const T* const row = logits + t * stride;
    float x[PL];
    load_row<T, PL>(row, E, lane, vec, x);
    uint32_t live = 0;   // finite logits
#pragma unroll
    for (int i = 0; i < PL; ++i) live |= (x[i] != -INFINITY ? 1u : 0u) << i;
    float top = 0.f, total = 0.f;
    if (score == TQ_SCORE_SOFTMAX) {
      softmax_terms<PL>(x, &top, &total);
      const float r = __frcp_rn(total);
#pragma unroll
      for (int i = 0; i < PL; ++i) x[i] = softmax_score(x[i], total, r);
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i) x[i] = sigmoid_score(x[i]);
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      if (bias) x[i] = __fadd_rn(x[i], b[i]);
      if (!((live >> i) & 1u) || !(x[i] == x[i])) x[i] = -INFINITY;
    }
    if (lane_groups > 0) {
      if (!choose_lane_groups<PL>(x, groups, top_groups, lane_groups, lane)) {
#pragma unroll
        for (int i = 0; i < PL; ++i) x[i] = -INFINITY;
      }
    } else if (groups > 1) {
      float* const c = rows + warp * E;
      const int size = E / groups;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        if (e0 + i < E) c[e0 + i] = x[i];
      }
      __syncwarp();
      const unsigned keep = choose_groups(c, groups, size, top_groups, group_lanes, lane);
      __syncwarp();
      int g = e0 / size, at = e0 - g * size;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        if (e0 + i < E && !((keep >> (g * group_lanes)) & 1u)) x[i] = -INFINITY;
        if (++at == size) {
          at = 0;
          ++g;
        }
      }
    }
    uint32_t key[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) key[i] = e0 + i < E ? order_key(x[i]) : 0u;
    int mine_e = 0;
    uint32_t mine_key = 0;
    bool chosen = false;
    if constexpr (PL >= 4) chosen = top_k > 2 && choose_from_few<PL>(key, top_k, lane, few[warp], &mine_e, &mine_key);
    for (int j = 0; j < top_k && !chosen; ++j) {
      // largest key of the lane, by a tree; then of the warp; the lowest lane
      // that has it, and its lowest expert
      uint32_t m[PL];
#pragma unroll
      for (int i = 0; i < PL; ++i) m[i] = key[i];
#pragma unroll
      for (int w = 1; w < PL; w <<= 1) {
#pragma unroll
        for (int i = 0; i < PL; i += 2 * w) m[i] = max(m[i], m[i + w]);
      }
      const uint32_t best = __reduce_max_sync(kAll, m[0]);
      uint32_t has = 0;
#pragma unroll
      for (int i = 0; i < PL; ++i) has |= (key[i] == best ? 1u : 0u) << i;
      const int src = __ffs(__ballot_sync(kAll, has != 0)) - 1;
      has = lane == src ? has & (0u - has) : 0u;   // its lowest bit
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        if ((has >> i) & 1u) key[i] = 0u;
      }
      const int e = __shfl_sync(kAll, e0 + __ffs(has) - 1, src);
      if (lane == j) {
        mine_e = e;
        mine_key = best;
      }
    }
    // lane j < top_k: the j-th chosen expert's weight
    float v = 0.f;
    if (lane < top_k && mine_key > kKeyMasked) v = one_score(widen(row[mine_e]), score, top, total);
    if (renorm) {
      const float sum = warp_sum(v);
      v = sum > 0.f ? v / sum : 0.f;
    }
    if (lane < top_k) {
      ids[static_cast<size_t>(t) * top_k + lane] = mine_e;
      w[static_cast<size_t>(t) * top_k + lane] = v * scale;
    }
  }
}

// The gradient of the logits.  Chosen experts with a weight of zero (masked
// fillers) take and give none.  A row is first written as every expert's own
// part (-p_i sum_j dp_j p_j for softmax scores, 0 for sigmoid ones and with
// renormalised weights, which depend on the chosen alone), then the chosen
// experts' values go over it.
template <typename T, int PL>
__global__ void __launch_bounds__(kRouterThreads)
router_scored_backward_kernel(const T* __restrict__ logits, long long stride, const int32_t* __restrict__ ids,
                              const float* __restrict__ w, const float* __restrict__ grad_w, int n, int E, int top_k,
                              int score, int renorm, float scale, bool vec, bool vec_out, T* __restrict__ grad,
                              int* err) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (long long t = blockIdx.x * kRouterWarps + warp; t < n; t += gridDim.x * kRouterWarps) {
    const T* const row = logits + t * stride;
    const size_t at = static_cast<size_t>(t) * top_k + lane;
    int e = -1;
    float g = 0.f;
    if (lane < top_k) {
      e = ids[at];
      if (e < 0 || e >= E) {
        record_error(err, TQ_ERR_INVALID_ARG, kWhereRouter);
        e = -1;
      }
      if (e >= 0 && w[at] != 0.f) g = grad_w[at] * scale;
    }
    const bool live = lane < top_k && e >= 0 && w[at] != 0.f;
    float x[PL];
    float top = 0.f, total = 0.f;
    if (score == TQ_SCORE_SOFTMAX) {
      load_row<T, PL>(row, E, lane, vec, x);
      softmax_terms<PL>(x, &top, &total);
    }
    const float logit = live ? widen(row[e]) : -INFINITY;
    const float p = one_score(logit, score, top, total);
    float own, dot = 0.f;
    if (renorm) {
      // q (g - sum_j g_j q_j) with q = p / sum: no step exceeds g, where g / sum
      // may overflow for scores near fp32's smallest.  Its sum over the chosen is 0.
      const float sum = warp_sum(p);
      const float q = sum > 0.f ? (live ? p : sum) / sum : 0.f;   // g is 0 in the other lanes; 0 / sum divides slowly
      own = q * (g - warp_sum(g * q));
    } else if (score == TQ_SCORE_SOFTMAX) {
      dot = warp_sum(g * p);
      own = p * (g - dot);
    } else {
      own = g * p;
    }
    // 1 - p as p exp(-x): the difference loses its bits as p nears 1
    if (score == TQ_SCORE_SIGMOID && p > 0.f) own *= p * expf(-logit);
    const float r = __frcp_rn(total);   // of a row without finite logits infinite, and its terms are 0
    T* const out = grad + static_cast<size_t>(t) * E;
    const int e0 = lane * PL;
    constexpr int kVec = PL * static_cast<int>(sizeof(T)) >= 16 ? 16 / static_cast<int>(sizeof(T)) : PL;
#pragma unroll
    for (int i = 0; i < PL; i += kVec) {
      T v[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        v[j] = narrow<T>(score == TQ_SCORE_SOFTMAX ? -softmax_score(x[i + j], total, r) * dot : 0.f);
      if (vec_out && kVec * sizeof(T) == 16 && e0 + i + kVec <= E) {
        uint4 q;
        memcpy(&q, v, 16);
        *reinterpret_cast<uint4*>(out + e0 + i) = q;
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          if (e0 + i + j < E) out[e0 + i + j] = v[j];
        }
      }
    }
    __syncwarp();   // the row before the chosen experts' values
    if (live) out[e] = narrow<T>(own);
    __syncwarp();
  }
}

int pieces(int E) {   // experts per lane
  int pl = 1;
  while (32 * pl < E) pl <<= 1;
  return pl;
}

// The stride and base keep every lane's 16-byte piece aligned.
bool rows_aligned(const void* p, long long stride, size_t size) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (stride % 16 * static_cast<long long>(size)) % 16 == 0;
}

int router_blocks(int64_t n) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((n + kRouterWarps - 1) / kRouterWarps,
                                                                 static_cast<int64_t>(sm_count()) * 16)));
}

template <typename T, int PL>
int run_forward(const RouterArgs& a, const T* logits, int32_t* ids, float* w, cudaStream_t s) {
  int lanes = 32;
  while (lanes * a.groups > 32) lanes >>= 1;
  // groups of a power of two of whole lanes are chosen from registers (8192 x
  // 256 in 8 groups: 15.0 -> 11.9 us when it came in), others through shared memory
  const int size = a.E / a.groups, whole = size % PL == 0 ? size / PL : 0;
  const int lane_groups = a.groups > 1 && whole > 0 && (whole & (whole - 1)) == 0 ? whole : 0;
  const size_t smem = a.groups > 1 && !lane_groups ? sizeof(float) * kRouterWarps * a.E : 0;
  return launch_pdl(router_scored_kernel<T, PL>, dim3(router_blocks(a.n)), dim3(kRouterThreads), smem, s, logits,
                    a.stride, a.bias, static_cast<int>(a.n), a.E, a.top_k, a.score, a.groups, a.top_groups, lane_groups,
                    lanes, a.renorm, a.scale, rows_aligned(logits, a.stride, sizeof(T)), ids, w);
}

template <typename T, int PL>
int run_backward(const RouterArgs& a, const T* logits, const int32_t* ids, const float* w, const float* grad_w,
                 T* grad, int* err, cudaStream_t s) {
  return launch_pdl(router_scored_backward_kernel<T, PL>, dim3(router_blocks(a.n)), dim3(kRouterThreads), 0, s,
                    logits, a.stride, ids, w, grad_w, static_cast<int>(a.n), a.E, a.top_k, a.score, a.renorm, a.scale,
                    rows_aligned(logits, a.stride, sizeof(T)), rows_aligned(grad, a.E, sizeof(T)), grad, err);
}

// f(T value, integral_constant PL) for the element type and row width.
template <typename T, typename F>
int by_width(int E, F&& f) {
  switch (pieces(E)) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    case 16: return f(std::integral_constant<int, 16>());
    default: return f(std::integral_constant<int, 32>());
  }
}

template <typename T>
int forward_typed(const RouterArgs& a, const void* logits, int32_t* ids, float* w, cudaStream_t s) {
  return by_width<T>(a.E, [&](auto pl) {
    return run_forward<T, decltype(pl)::value>(a, static_cast<const T*>(logits), ids, w, s);
  });
}

template <typename T>
int backward_typed(const RouterArgs& a, const void* logits, const int32_t* ids, const float* w, const float* grad_w,
                   void* grad, int* err, cudaStream_t s) {
  return by_width<T>(a.E, [&](auto pl) {
    return run_backward<T, decltype(pl)::value>(a, static_cast<const T*>(logits), ids, w, grad_w,
                                                static_cast<T*>(grad), err, s);
  });
}

bool bad_router_args(const RouterArgs& a, int type) {
  constexpr int64_t kMost = static_cast<int64_t>(1) << 31;
  return a.E < 1 || a.E > 1024 || a.top_k < 1 || a.top_k > 32 || a.top_k > a.E || a.n < 0 || a.n >= kMost ||
         a.n * a.top_k >= kMost || a.stride < a.E || bad_type(type) ||
         (a.score != TQ_SCORE_SOFTMAX && a.score != TQ_SCORE_SIGMOID);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

int tq_router_scored(const void* logits, int logits_type, int64_t logits_stride, const float* bias, int64_t n, int E,
                     int top_k, int score, int groups, int top_groups, int renormalize, float scale,
                     int32_t* topk_ids, float* topk_w, tq_stream_t stream) {
  const RouterArgs a{n, logits_stride, bias, E, top_k, score, groups, top_groups, renormalize, scale};
  if (bad_router_args(a, logits_type)) return TQ_ERR_INVALID_ARG;
  if (groups < 1 || groups > 32 || E % groups != 0 || top_groups < 1 || top_groups > groups ||
      top_k > top_groups * (E / groups))
    return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!logits || !topk_ids || !topk_w)) return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int rc = require_sm103(s);
  if (rc != TQ_OK) return rc;
  if (n == 0) return TQ_OK;
  const int st = logits_type == TQ_FP32   ? forward_typed<float>(a, logits, topk_ids, topk_w, s)
                 : logits_type == TQ_BF16 ? forward_typed<__nv_bfloat16>(a, logits, topk_ids, topk_w, s)
                                          : forward_typed<__half>(a, logits, topk_ids, topk_w, s);
  if (st == TQ_OK) count_launch(kCntRouterScored);
  return st;
}

int tq_router_scored_backward(const void* logits, int logits_type, int64_t logits_stride, const int32_t* topk_ids,
                              const float* topk_w, const float* grad_w, int64_t n, int E, int top_k, int score,
                              int renormalize, float scale, void* grad_logits, tq_stream_t stream) {
  const RouterArgs a{n, logits_stride, nullptr, E, top_k, score, 1, 1, renormalize, scale};
  if (bad_router_args(a, logits_type)) return TQ_ERR_INVALID_ARG;
  if (n > 0 && (!logits || !topk_ids || !topk_w || !grad_w || !grad_logits)) return TQ_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int rc = require_sm103(s);
  if (rc != TQ_OK) return rc;
  if (n == 0) return TQ_OK;
  int* err = error_word(&rc);
  if (!err) return rc;
  const int st =
      logits_type == TQ_FP32
          ? backward_typed<float>(a, logits, topk_ids, topk_w, grad_w, grad_logits, err, s)
      : logits_type == TQ_BF16
          ? backward_typed<__nv_bfloat16>(a, logits, topk_ids, topk_w, grad_w, grad_logits, err, s)
          : backward_typed<__half>(a, logits, topk_ids, topk_w, grad_w, grad_logits, err, s);
  if (st == TQ_OK) count_launch(kCntRouterScoredBackward);
  return st;
}

}  // extern "C"
