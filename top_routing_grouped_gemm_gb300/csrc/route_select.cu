// Routing by softmax or sigmoid scores with a balance bias and groups, and its gradient
// (include/moe_block.h has the formulas).
#include <math.h>

#include <type_traits>

#include "moe_internal.h"
#include "overlap.cuh"
#include "ptx.cuh"
#include "route.h"
#include "two_floats.cuh"

#include "../../include/moe_block.h"

namespace moe {
namespace {

constexpr int kWarps = 8;  // a token to each: the 8 tokens of a row of prob_partials
constexpr int kMaxE = 1024;

struct Select {
  int T, E, k, groups, kept, best, group_size, lanes;  // lanes of a group: 32 / (groups, up to 2^n)
  int sigmoid, renormalise;
  float scale;
  const void* logits;
  long long ld;
  const float* bias;
  int* idx;
  float* gate;
  float* partials;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
__device__ __forceinline__ Two warp_sum(Two v) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    v = v + Two{__shfl_xor_sync(~0u, v.hi, o), __shfl_xor_sync(~0u, v.lo, o)};
  return v;
}

// A logit; what is not a number counts as -inf.
template <typename T>
__device__ __forceinline__ float logit(const T* row, int e) {
  const float v = static_cast<float>(row[e]);
  return v == v ? v : -INFINITY;
}

__device__ __forceinline__ float sigmoid(float l) {
  const float e = expf(-fabsf(l)), t = e / (1.f + e);
  return l < 0.f ? t : 1.f / (1.f + e);
}

// A score, where only its share in a sum is wanted: softmax scores without their sum, and sigmoid
// scores, where all are far below 1, times exp(-most), so that they do not vanish.  most: the largest
// logit.
__device__ __forceinline__ float unscaled(float l, float most, bool sigmoid_scores) {
  if (l == -INFINITY) return 0.f;
  if (sigmoid_scores) return most > -40.f ? sigmoid(l) : expf(l - most) / (1.f + expf(l));
  return expf(l - most);
}

// The scores of a row's selected experts over their sum, one to a lane (0 for lanes that hold none: l
// = -inf), and 0 where that sum is.
__device__ __forceinline__ float share(float l, bool sigmoid_scores) {
  const float v = unscaled(l, warp_max(l), sigmoid_scores);
  const float sum = warp_sum(v);
  return sum == 0.f ? 0.f : v / sum;  // (a NaN stays one)
}

// One warp to a token.  Its lanes are parted among the groups; lane i of a group has every
// lanes'th of its experts from i on, VPL of them at most.
template <typename T, int VPL>
__global__ void __launch_bounds__(kWarps * 32) route_select_kernel(const Select s) {
  extern __shared__ float shares[];  // [kWarps][E]
  after_previous();
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + warp;
  float* mine = shares + warp * s.E;
  if (t < s.T) {
    const T* row = static_cast<const T*>(s.logits) + t * s.ld;
    const int group = lane / s.lanes, sub = lane % s.lanes;
    const bool have = group < s.groups;
    const auto in = [&](int j) { return have && sub + j * s.lanes < s.group_size; };
    const auto expert = [&](int j) { return group * s.group_size + sub + j * s.lanes; };
    float l[VPL], lo[VPL];
    float most = -INFINITY, sum = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      l[j] = in(j) ? logit(row, expert(j)) : -INFINITY;
      most = fmaxf(most, l[j]);
    }
    most = warp_max(most);
    // scores for the sums over tokens, in fp32
    const float shift = most == -INFINITY ? 0.f : most;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (in(j)) sum += unscaled(l[j], most, s.sigmoid);
    sum = warp_sum(sum);
    if (s.partials) {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (in(j)) {
          const float v = unscaled(l[j], most, s.sigmoid);
          mine[expert(j)] = sum == 0.f ? 0.f : v / sum;
        }
    }
    // what is compared: scores (+ bias) as two floats, in l and lo
    Two total{0.f, 0.f};
    const bool by_logit = !s.bias;
    const auto score = [&](int j) -> Two {
      if (s.sigmoid) return two_sigmoid(l[j]);
      const Two e = two_exp(two_sum(l[j], -shift));
      return most == INFINITY ? Two{NAN, 0.f} : e / total;
    };
    if (!s.sigmoid && (s.bias || s.groups > 1)) {
#pragma unroll 1
      for (int j = 0; j < VPL; ++j)
        if (in(j)) total = total + two_exp(two_sum(l[j], -shift));
      total = warp_sum(total);
      if (total.hi == 0.f) total.hi = 1.f;
    }
    uint64_t key[VPL];
    uint64_t top[2] = {0, 0};  // the lane's largest two, of the group's then
    Two value[2] = {{-INFINITY, 0.f}, {-INFINITY, 0.f}};
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      key[j] = 0;
      if (!in(j)) continue;
      Two c{l[j], 0.f};
      if (s.bias || s.groups > 1) c = score(j);
      if (s.bias) {
        const float b = s.bias[expert(j)];
        const Two w = two_sum(c.hi, b);
        c = quick_sum(w.hi, __fadd_rn(w.lo, c.lo));
        if (isinf(w.hi) || w.hi != w.hi) c = {w.hi == w.hi ? w.hi : -INFINITY, 0.f};
      }
      const uint64_t of = two_key(c);
      key[j] = by_logit ? two_key({l[j], 0.f}) : of;
      if (s.groups > 1) {
        if (c.hi != c.hi) c = {-INFINITY, 0.f};
        if (of > top[0]) {
          top[1] = top[0], value[1] = value[0];
          top[0] = of, value[0] = c;
        } else if (of > top[1]) {
          top[1] = of, value[1] = c;
        }
      }
    }
    bool in_kept = have;
    if (s.groups > 1) {
      for (int o = s.lanes / 2; o; o >>= 1) {
        uint64_t other[2];
        Two theirs[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          other[i] = __shfl_xor_sync(~0u, top[i], o);
          theirs[i].hi = __shfl_xor_sync(~0u, value[i].hi, o);
          theirs[i].lo = __shfl_xor_sync(~0u, value[i].lo, o);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (other[i] > top[0]) {
            top[1] = top[0], value[1] = value[0];
            top[0] = other[i], value[0] = theirs[i];
          } else if (other[i] > top[1]) {
            top[1] = other[i], value[1] = theirs[i];
          }
      }
      Two worth = value[0];
      if (s.best == 2) {
        worth = isinf(value[0].hi) || isinf(value[1].hi)
                    ? Two{value[0].hi + value[1].hi, 0.f}
                    : value[0] + value[1];
      }
      const uint64_t v = two_key(worth);
      int before = 0;
      for (int g = 0; g < s.groups; ++g) {
        const uint64_t other = __shfl_sync(~0u, v, g * s.lanes);
        before += other > v || (other == v && g < group);
      }
      in_kept = have && before < s.kept;
    }
    // k rounds: the warp's largest key (of equal ones the lowest expert) goes to lane r
    uint64_t head = 0;
    int head_expert = kMaxE;
    const auto next = [&](uint64_t below, int after) {
      head = 0, head_expert = kMaxE;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (in_kept && key[j] && (key[j] < below || (key[j] == below && expert(j) > after)) &&
            key[j] > head)
          head = key[j], head_expert = expert(j);
    };
    next(~0ull, -1);
    int chosen = 0;
    for (int r = 0; r < s.k; ++r) {
      const uint32_t hi = __reduce_max_sync(~0u, static_cast<uint32_t>(head >> 32));
      const uint32_t low = __reduce_max_sync(
          ~0u, static_cast<uint32_t>(head >> 32) == hi ? static_cast<uint32_t>(head) : 0u);
      const uint64_t best = static_cast<uint64_t>(hi) << 32 | low;
      const int e = __reduce_min_sync(~0u, head == best ? head_expert : kMaxE);
      if (lane == r) chosen = e;
      if (head_expert == e) next(best, e);
    }
    const bool slot = lane < s.k;
    const float of = slot ? logit(row, chosen) : -INFINITY;
    float g;
    if (s.renormalise)
      g = share(of, s.sigmoid);
    else if (s.sigmoid)
      g = sigmoid(of);
    else
      g = sum == 0.f ? 0.f : unscaled(of, most, false) / sum;
    if (slot) {
      s.idx[t * s.k + lane] = chosen;
      s.gate[t * s.k + lane] = s.scale * g;
    }
  }
  if (!s.partials) return;
  __syncthreads();
  const int tokens = static_cast<int>(min(static_cast<long long>(kWarps),
                                          s.T - static_cast<long long>(blockIdx.x) * kWarps));
  for (int e = threadIdx.x; e < s.E; e += kWarps * 32) {
    float sum = 0.f;
    for (int w = 0; w < tokens; ++w) sum += shares[w * s.E + e];
    s.partials[static_cast<long long>(blockIdx.x) * s.E + e] = sum;
  }
}

struct SelectGrad {
  int T, E, k;
  int sigmoid, renormalise;
  float scale;
  const void* logits;
  long long ld;
  const int* idx;
  const float* dgate;
  void* dlogits;
  float* dlogits_topk;
  int* dev_status;
};

// With w the selected scores over their sum, d = scale dgate and s' = s (1 - s) or s:
//   renormalised: dl_j = w_j (1 - s_j) (d_j - sum_i w_i d_i)   (softmax without the second factor)
//   else, sigmoid: dl_j = s_j (1 - s_j) d_j;  softmax: dl_e = s_e (d_e - sum_i s_i d_i) for all e.
// One warp to a token.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) route_select_backward_kernel(const SelectGrad s) {
  after_previous();
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (t >= s.T) return;
  const T* row = static_cast<const T*>(s.logits) + t * s.ld;
  int e = -1;
  float d = 0.f;
  if (lane < s.k) {
    e = s.idx[t * s.k + lane];
    d = s.scale * s.dgate[t * s.k + lane];
    if (e < 0 || e >= s.E) {
      report_status(s.dev_status, MOE_ERR_BAD_INDEX);
      e = -1;
    }
  }
  const float l = e >= 0 ? logit(row, e) : -INFINITY;
  if (e < 0) d = 0.f;
  float v, dot = 0.f, most = 0.f, inv = 0.f;
  if (s.renormalise) {
    const float w = share(l, s.sigmoid);
    v = w * (d - warp_sum(w * d));
    if (s.sigmoid) v *= sigmoid(-l);
  } else if (s.sigmoid) {
    v = sigmoid(l) * sigmoid(-l) * d;
  } else {
    most = -INFINITY;
    for (int i = lane; i < s.E; i += 32) most = fmaxf(most, logit(row, i));
    most = warp_max(most);
    if (most == -INFINITY) most = 0.f;
    float sum = 0.f;
    for (int i = lane; i < s.E; i += 32) sum += expf(logit(row, i) - most);
    sum = warp_sum(sum);
    inv = sum == 0.f ? 0.f : 1.f / sum;
    const float p = e >= 0 ? expf(l - most) * inv : 0.f;
    dot = warp_sum(p * d);
    v = p * d;
  }
  if (e < 0) v = 0.f;
  if (s.dlogits_topk && lane < s.k) s.dlogits_topk[t * s.k + lane] = v;
  if (!s.dlogits) return;
  T* out = static_cast<T*>(s.dlogits) + t * s.E;
  const bool dense = !s.renormalise && !s.sigmoid;
  for (int i = lane; i < s.E; i += 32)
    out[i] = static_cast<T>(dense ? -dot * (expf(logit(row, i) - most) * inv) : 0.f);
  __syncwarp();
  // the parts of an expert that is named twice are added in the slots' order by the first of them
  const unsigned same = __match_any_sync(~0u, e);
  float sum = 0.f;
  for (int j = 0; j < s.k; ++j) {
    const float other = __shfl_sync(~0u, v, j);
    if (same >> j & 1) sum += other;
  }
  if (e < 0 || (same & ((1u << lane) - 1))) return;
  if (dense) sum = fmaf(-dot, expf(l - most) * inv, sum);
  out[e] = static_cast<T>(sum);
}

// ------------------------------------------------------------------------ host side

int check(int T, int E, int k, const moe_route_rule* r, int dtype, const void* logits,
          long long ld) {
  if (!r || !logits || T <= 0 || E <= 0 || k <= 0) return MOE_ERR_INVALID_ARG;
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (r->groups <= 0 || E % r->groups || r->groups_kept <= 0 || r->groups_kept > r->groups)
    return MOE_ERR_INVALID_ARG;
  if (r->groups > 1 &&
      (r->group_best < 1 || r->group_best > 2 || r->group_best > E / r->groups))
    return MOE_ERR_INVALID_ARG;
  if (!(fabsf(r->scale) <= 3.4028235e38f)) return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || k > 32 || r->groups > 32 || T > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (k > r->groups_kept * (E / r->groups)) return MOE_ERR_INVALID_ARG;
  if (T > 1 && ld != 0 && ld < E) return MOE_ERR_INVALID_ARG;
  if (ld > (1ll << 32)) return MOE_ERR_UNSUPPORTED;
  return misaligned(logits, dtype == MOE_F32 ? 4 : 2) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int blocks_of(int T) { return route_num_partials(T); }

// Calls f(VPL) for what a lane holds.
template <typename F>
void with_values(int per_lane, F f) {
  using std::integral_constant;
  if (per_lane <= 4)
    f(integral_constant<int, 4>{});
  else if (per_lane <= 8)
    f(integral_constant<int, 8>{});
  else if (per_lane <= 16)
    f(integral_constant<int, 16>{});
  else if (per_lane <= 28)
    f(integral_constant<int, 28>{});
  else if (per_lane <= 32)
    f(integral_constant<int, 32>{});
  else
    f(integral_constant<int, 64>{});
}

}  // namespace
}  // namespace moe

extern "C" {

using namespace moe;

int moe_route_select(int32_t T, int32_t E, int32_t k, const moe_route_rule* rule, int32_t dtype,
                     const void* logits, int64_t ld_logits, const float* select_bias,
                     int32_t* topk_idx, float* topk_gate, float* prob_partials,
                     moe_stream_t stream) {
  if (int e = check(T, E, k, rule, dtype, logits, ld_logits)) return e;
  if (!topk_idx || !topk_gate) return MOE_ERR_INVALID_ARG;
  if (misaligned(select_bias, 4) || misaligned(topk_idx, 4) || misaligned(topk_gate, 4) ||
      misaligned(prob_partials, 4))
    return MOE_ERR_UNSUPPORTED;
  Select s{};
  s.T = T, s.E = E, s.k = k;
  s.groups = rule->groups, s.kept = rule->groups_kept, s.best = rule->group_best;
  s.group_size = E / s.groups;
  s.lanes = 32;
  for (int g = 1; g < s.groups; g *= 2) s.lanes /= 2;
  s.sigmoid = rule->score == MOE_SCORE_SIGMOID;
  s.renormalise = rule->renormalise != 0;
  s.scale = rule->scale;
  s.logits = logits, s.ld = T == 1 ? 0 : ld_logits, s.bias = select_bias;
  s.idx = topk_idx, s.gate = topk_gate, s.partials = prob_partials;
  mark_before(MOE_KERNEL_ROUTE_SELECT, stream);
  cudaError_t err = cudaSuccess;
  with_values((s.group_size + s.lanes - 1) / s.lanes, [&](auto v) {
    constexpr int VPL = decltype(v)::value;
    const int smem = prob_partials ? kWarps * E * 4 : 0;
    if (dtype == MOE_F32)
      err = launch_behind(route_select_kernel<float, VPL>, blocks_of(T), kWarps * 32, smem, stream, s);
    else
      err = launch_behind(route_select_kernel<__nv_bfloat16, VPL>, blocks_of(T), kWarps * 32, smem,
                          stream, s);
  });
  mark_after(MOE_KERNEL_ROUTE_SELECT, stream);
  count_launches(1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_route_select_backward(int32_t T, int32_t E, int32_t k, const moe_route_rule* rule,
                              int32_t dtype, const void* logits, int64_t ld_logits,
                              const int32_t* topk_idx, const float* dgate, void* dlogits,
                              float* dlogits_topk, int32_t* dev_status, moe_stream_t stream) {
  if (int e = check(T, E, k, rule, dtype, logits, ld_logits)) return e;
  if (!topk_idx || !dgate || (!dlogits && !dlogits_topk)) return MOE_ERR_INVALID_ARG;
  if (dlogits_topk && rule->score == MOE_SCORE_SOFTMAX && !rule->renormalise)
    return MOE_ERR_INVALID_ARG;
  if (misaligned(topk_idx, 4) || misaligned(dgate, 4) || misaligned(dlogits_topk, 4) ||
      misaligned(dev_status, 4) || misaligned(dlogits, dtype == MOE_F32 ? 4 : 2))
    return MOE_ERR_UNSUPPORTED;
  SelectGrad s{};
  s.T = T, s.E = E, s.k = k;
  s.sigmoid = rule->score == MOE_SCORE_SIGMOID;
  s.renormalise = rule->renormalise != 0;
  s.scale = rule->scale;
  s.logits = logits, s.ld = T == 1 ? 0 : ld_logits;
  s.idx = topk_idx, s.dgate = dgate, s.dlogits = dlogits, s.dlogits_topk = dlogits_topk;
  s.dev_status = dev_status;
  mark_before(MOE_KERNEL_ROUTE_SELECT_BWD, stream);
  const cudaError_t err =
      dtype == MOE_F32
          ? launch_behind(route_select_backward_kernel<float>, blocks_of(T), kWarps * 32, 0, stream, s)
          : launch_behind(route_select_backward_kernel<__nv_bfloat16>, blocks_of(T), kWarps * 32, 0,
                          stream, s);
  mark_after(MOE_KERNEL_ROUTE_SELECT_BWD, stream);
  count_launches(1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
