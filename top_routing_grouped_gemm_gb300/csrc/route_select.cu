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
  int T, E, k, groups, kept, best, group_size;
  int lanes, lanes_log2;  // of a group: 32 / (groups, up to 2^n)
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
// A logit; what is not a number counts as -inf.
template <typename T>
__device__ __forceinline__ float logit(const T* row, int e) {
  return fmaxf(static_cast<float>(row[e]), -INFINITY);
}

__device__ __forceinline__ float sigmoid(float l) {
  const float e = expf(-fabsf(l)), t = e / (1.f + e);
  return l < 0.f ? t : 1.f / (1.f + e);
}
// The same by the hardware's approximations, 2^x off by 2^-22 of it and 1 / x by 2^-23: exp(l) is off by
// (|l| + 4) 2^-24 of it, which leaves the score off by 8 x 2^-24 at most (|l| e^-|l| < 0.4).  What would
// be subnormal is 0.
__device__ __forceinline__ float quick_exp(float l) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * 1.44269504f));
  return e;
}
__device__ __forceinline__ float quick_sigmoid(float l) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + quick_exp(-l)));
  return r;
}

// A score, where only its share in a sum is wanted: softmax scores without their sum, and sigmoid
// scores, where all are far below 1, times exp(-most), so that they do not vanish.  most: the largest
// logit.
__device__ __forceinline__ float unscaled(float l, float most, bool sigmoid_scores) {
  if (l == -INFINITY) return 0.f;
  if (sigmoid_scores) return most > -40.f ? sigmoid(l) : expf(l - most) / (1.f + expf(l));
  return expf(l - most);
}

template <int VEC>
__device__ __forceinline__ void load_logits(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
    v[0] = *p;
  }
}
template <int VEC>
__device__ __forceinline__ void store_scores(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 4)
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *p = v[0];
}
template <int VEC>
__device__ __forceinline__ void load_logits(const __nv_bfloat16* p, float (&v)[VEC]) {
  if constexpr (VEC == 4) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
  } else {
    v[0] = static_cast<float>(*p);
  }
}

// The scores of a row's selected experts over their sum, one to a lane (0 for lanes that hold none: l
// = -inf), and 0 where that sum is.
__device__ __forceinline__ float share(float l, bool sigmoid_scores) {
  const float v = unscaled(l, warp_max(l), sigmoid_scores);
  const float sum = warp_sum(v);
  return sum == 0.f ? 0.f : v / sum;  // (a NaN stays one)
}

// What a lane of a token's warp holds: the lanes are parted among the groups, and a group's lanes take
// `vec` neighbouring ones of its experts in turn.
struct Share {
  int group, first, step, vec, count;  // its first expert, from one of its vecs to the next, how many
  bool have;
  __device__ __forceinline__ Share(const Select& s, int vec_) : vec(vec_) {
    const int lane = threadIdx.x & 31;
    group = lane >> s.lanes_log2;
    have = group < s.groups;
    const int sub = (lane & (s.lanes - 1)) * vec;
    first = group * s.group_size + sub;
    step = s.lanes * vec;
    count = have && sub < s.group_size ? ((s.group_size - sub + step - 1) / vec >> s.lanes_log2) * vec : 0;
  }
  __device__ __forceinline__ int expert(int j) const { return first + j / vec * step + j % vec; }
};

// Whether the lane's group is among those kept, `worth` being the key of its value.
__device__ __forceinline__ bool group_kept(const Select& s, uint64_t worth, int group) {
  int before = 0;
  for (int g = 0; g < s.groups; ++g) {
    const uint64_t other = __shfl_sync(~0u, worth, g * s.lanes);
    before += other > worth || (other == worth && g < group);
  }
  return group < s.groups && before < s.kept;
}

__device__ __forceinline__ uint64_t warp_most(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(~0u, static_cast<uint32_t>(v >> 32));
  const uint32_t lo =
      __reduce_max_sync(~0u, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return static_cast<uint64_t>(hi) << 32 | lo;
}

// Scores (and biases) as two floats.  What follows up to the kernel runs for few tokens, on an SM
// whose instruction cache has not got it: short code and loops that are not unrolled matter more than
// the number of instructions.  (Unrolled, three tokens of 16384 that came here took 50 us.)
__device__ __noinline__ Two exact_score(float l, float most, bool sigmoid, Two total, float bias) {
  const float shift = most == -INFINITY ? 0.f : most;
  const Two e = two_exp(sigmoid ? Two{-fabsf(l), 0.f} : two_sum(l, -shift));
  // sigmoid: e / (1 + e), or what that lacks to 1, which keeps its own precision; softmax: e / total
  const Two one = quick_sum(1.f, e.hi);
  Two c = e / (sigmoid ? quick_sum(one.hi, __fadd_rn(one.lo, e.lo)) : total);
  if (sigmoid && l >= 0.f) {
    const Two rest = quick_sum(1.f, -c.hi);
    c = quick_sum(rest.hi, __fsub_rn(rest.lo, c.lo));
  }
  if (!sigmoid && most == INFINITY) c = {NAN, 0.f};
  const Two w = two_sum(c.hi, bias);
  c = quick_sum(w.hi, __fadd_rn(w.lo, c.lo));
  if (isinf(w.hi)) c = {w.hi, 0.f};
  return w.hi != w.hi ? Two{-INFINITY, 0.f} : c;
}

struct Exact {
  Two total;  // of softmax's exponentials
  float most;
  const float* bias;
  bool sigmoid;
  template <typename T>
  __device__ __forceinline__ Exact(const Select& s, const Share& mine, const T* row, float most_)
      : total{0.f, 0.f}, most(most_), bias(s.bias), sigmoid(s.sigmoid) {
    if (sigmoid) return;
    const float shift = most == -INFINITY ? 0.f : most;
#pragma unroll 1
    for (int j = 0; j < mine.count; ++j)
      total = total + two_exp(two_sum(logit(row, mine.expert(j)), -shift));
#pragma unroll 1
    for (int o = 16; o; o >>= 1)
      total = total + Two{__shfl_xor_sync(~0u, total.hi, o), __shfl_xor_sync(~0u, total.lo, o)};
    if (total.hi == 0.f) total.hi = 1.f;
  }
  __device__ __forceinline__ Two score(float l, int e) const {
    return exact_score(l, most, sigmoid, total, bias ? bias[e] : 0.f);
  }
};

// The selection by such scores: lane r gets the r-th expert.  Rarely called: short code and few
// registers (its keys are in local memory) matter more than its time, several times that of the
// selection in fp32.
template <typename T>
__device__ __noinline__ int select_exactly(const Select& s, const T* row, float most, int vec) {
  Share mine(s, vec);
  const int lane = threadIdx.x & 31;
  const Exact exact(s, mine, row, most);
  uint64_t key[64];
  uint64_t top[2] = {0, 0};  // the lane's largest two, of the group's then
  Two value[2] = {{-INFINITY, 0.f}, {-INFINITY, 0.f}};
  const auto put = [&](uint64_t of, Two c) {
    if (of > top[0]) {
      top[1] = top[0], value[1] = value[0];
      top[0] = of, value[0] = c;
    } else if (of > top[1]) {
      top[1] = of, value[1] = c;
    }
  };
#pragma unroll 1
  for (int j = 0; j < mine.count; ++j) {
    const float l = logit(row, mine.expert(j));
    const Two c = exact.score(l, mine.expert(j));
    const uint64_t of = two_key(c);
    key[j] = s.bias ? of : two_key({l, 0.f});
    put(of, c);
  }
  if (s.groups > 1) {
#pragma unroll 1
    for (int o = s.lanes / 2; o; o >>= 1) {
      const uint64_t k0 = __shfl_xor_sync(~0u, top[0], o), k1 = __shfl_xor_sync(~0u, top[1], o);
      const Two v0{__shfl_xor_sync(~0u, value[0].hi, o), __shfl_xor_sync(~0u, value[0].lo, o)};
      const Two v1{__shfl_xor_sync(~0u, value[1].hi, o), __shfl_xor_sync(~0u, value[1].lo, o)};
      put(k0, v0);
      put(k1, v1);
    }
    Two worth = value[0];
    if (s.best == 2)
      worth = isinf(value[0].hi) || isinf(value[1].hi) ? Two{value[0].hi + value[1].hi, 0.f}
                                                       : value[0] + value[1];
    if (!group_kept(s, two_key(worth), mine.group)) mine.count = 0;
  }
  // k rounds: the lane whose first it was (of equal ones the lowest expert) looks for its next
  uint64_t head = ~0ull;
  int expert = -1, chosen = 0;
  const auto next = [&] {
    const uint64_t below = head;
    const int after = expert;
    head = 0, expert = kMaxE;
#pragma unroll 1
    for (int j = 0; j < mine.count; ++j)
      if ((key[j] < below || (key[j] == below && mine.expert(j) > after)) && key[j] > head)
        head = key[j], expert = mine.expert(j);
  };
  next();
#pragma unroll 1
  for (int r = 0; r < s.k; ++r) {
    const uint64_t best = warp_most(head);
    const int e = __reduce_min_sync(~0u, head == best ? expert : kMaxE);
    if (lane == r) chosen = e;
    if (expert == e) next();
  }
  return chosen;
}

// Whether the lane's group is among those kept, by exact values: those of the experts from `least` on
// (of their scores in fp32, times `scale`, and biases), which are in `list` then, 64 at most: -1 for
// more.  One to a lane and turn.
template <typename T>
__device__ __noinline__ int keep_exactly(const Select& s, const T* row, const float* row_scores,
                                         float scale, float most, float least, int vec, int* list,
                                         Two* values) {
  const Share mine(s, vec);
  const Exact exact(s, mine, row, most);
  const int lane = threadIdx.x & 31;
  const auto wanted = [&](int j) {
    const int e = mine.expert(j);
    return fmaxf(row_scores[e] * scale + (s.bias ? s.bias[e] : 0.f), -INFINITY) >= least;
  };
  int to = 0;
#pragma unroll 1
  for (int j = 0; j < mine.count; ++j) to += wanted(j);
  const int own = to;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int before = __shfl_up_sync(~0u, to, o);
    if (lane >= o) to += before;
  }
  const int n = __shfl_sync(~0u, to, 31);
  if (n > 64) return -1;
  to -= own;
#pragma unroll 1
  for (int j = 0; j < mine.count; ++j)
    if (wanted(j)) list[to++] = mine.expert(j);
  __syncwarp();
#pragma unroll 1
  for (int i = lane; i < n; i += 32)
    values[i] = exact.score(logit(row, list[i]), list[i]);
  __syncwarp();
  Two top[2] = {{-INFINITY, 0.f}, {-INFINITY, 0.f}};
#pragma unroll 1
  for (int i = 0; i < n; ++i)
    if (static_cast<unsigned>(list[i] - mine.group * s.group_size) < static_cast<unsigned>(s.group_size)) {
      const Two c = values[i];
      if (two_key(c) > two_key(top[0]))
        top[1] = top[0], top[0] = c;
      else if (two_key(c) > two_key(top[1]))
        top[1] = c;
    }
  __syncwarp();  // (the list is used again)
  Two worth = top[0];
  if (s.best == 2)
    worth = isinf(top[0].hi) || isinf(top[1].hi) ? Two{top[0].hi + top[1].hi, 0.f} : top[0] + top[1];
  return group_kept(s, two_key(worth), mine.group);
}

// The selection from candidates, up to two to a lane (kMaxE: none), which hold all that can be chosen.
template <typename T>
__device__ __noinline__ int order_exactly(const Select& s, const T* row, float most, int vec,
                                          int expert0, int expert1) {
  const Exact exact(s, Share(s, vec), row, most);
  uint64_t key0 = 0, key1 = 0;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    key1 = key0;
    const int e = i ? expert0 : expert1;
    if (__any_sync(~0u, e < kMaxE)) {
      const int at = min(e, s.E - 1);
      key0 = two_key(exact.score(logit(row, at), at));
    }
    if (e >= kMaxE) key0 = 0;
  }
  if (key1 > key0 || (key1 == key0 && expert1 < expert0)) {
    const uint64_t key = key0;
    const int expert = expert0;
    key0 = key1, expert0 = expert1;
    key1 = key, expert1 = expert;
  }
  int chosen = 0;
#pragma unroll 1
  for (int r = 0; r < s.k; ++r) {
    const uint64_t best = warp_most(key0);
    const int e = __reduce_min_sync(~0u, key0 == best ? expert0 : kMaxE);
    if (static_cast<int>(threadIdx.x & 31) == r) chosen = e;
    if (expert0 == e) key0 = key1, expert0 = expert1, key1 = 0, expert1 = kMaxE;
  }
  return chosen;
}

// One warp to a token, VPL experts to a lane at most.  The scores are formed in fp32 and selected by;
// where two that stand next to each other in the order (or the last group kept and the first one left
// out) are nearer than their rounding, the token is selected again with scores as two floats.  Equal
// logits with equal biases have equal scores and need that not.  Bound by instructions: 1860 of a warp
// for 896 logits with a bias, 840 of them at half rate; 16384 x 896 in fp32 38 us (68 MB, 10 us of
// reading).  (Conditional stores of candidates and k rounds of a warp's maximum: 2400, 50 us.  Four
// blocks to an SM, of 64 registers, spill: 38.4 us.)
template <typename T, int VPL, int VEC, bool SIGMOID>
__global__ void __launch_bounds__(kWarps * 32, VPL <= 16 ? 4 : VPL <= 32 ? 3 : 2)
    route_select_kernel(const __grid_constant__ Select s) {
  extern __shared__ __align__(16) float scores[];  // [kWarps][E], as they are formed
  __shared__ uint2 candidates[kWarps][68 + 33];
  __shared__ float share_of[kWarps];  // 1 / their sum
  after_previous();
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (t < s.T) {
    const T* row = static_cast<const T*>(s.logits) + t * s.ld;
    float* row_scores = scores + warp * s.E;
    const Share mine(s, VEC);
    float v[VPL];  // logits, then what is compared; NaN: none
    float most = -INFINITY, sum = 0.f, inv = 1.f;
#pragma unroll
    for (int j = 0; j < VPL; j += VEC) {
      float q[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) q[i] = NAN;
      if (j < mine.count) load_logits<VEC>(row + mine.expert(j), q);
      const float floor = j < mine.count ? -INFINITY : NAN;
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j + i] = fmaxf(q[i], floor);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) most = fmaxf(most, v[j]);
    most = warp_max(most);
    bool exact = true;
    const bool small = SIGMOID && !(most > -40.f);  // scores below 2^-57
    const bool by_score = s.bias || s.groups > 1;
    if (s.partials || by_score || (!SIGMOID && !s.renormalise)) {
      const float shift = most == -INFINITY ? 0.f : most;
#pragma unroll
      for (int j = 0; j < VPL; j += VEC) {
        float q[VEC], of = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          q[i] = SIGMOID ? quick_sigmoid(v[j + i]) : quick_exp(v[j + i] - shift);
          of += q[i];
        }
        if (j < mine.count) {  // (short, so that it takes no branches)
          sum += of;
          store_scores<VEC>(row_scores + mine.expert(j), q);
        }
      }
      if (small) {  // what is added up over tokens is their shares
        sum = 0.f;
#pragma unroll 1
        for (int j = 0; j < mine.count; ++j) {
          const float q = unscaled(logit(row, mine.expert(j)), most, true);
          sum += q;
          row_scores[mine.expert(j)] = q;
        }
        if (s.bias) exact = false;  // they need more than fp32 beside it
      }
      sum = warp_sum(sum);
      inv = sum == 0.f ? 0.f : __fdividef(1.f, sum);
      if (lane == 0) share_of[warp] = inv;
    }
    // Errors of scores are at most `step` of their size: 8 halves of an fp32 step of sigmoid's, and
    // for softmax |l - most| + VPL + 20 of them; of the sum with a bias one more.
    const float step = SIGMOID ? 0x1p-21f : 0x1p-17f;
    const float largest = SIGMOID ? 1.f : inv;  // what no score is above
    const auto compared = [&](float q, float b, float floor) {
      return fmaxf(SIGMOID ? q + b : fmaf(q, inv, b), floor);
    };
    bool kept = true;
    if (by_score) {
      float top[2] = {-INFINITY, -INFINITY};
      const bool by_logit = !s.bias && s.best == 1;  // the order of the largest scores
      if (!by_logit) {
#pragma unroll
        for (int j = 0; j < VPL; j += VEC) {
          float q[VEC], b[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) q[i] = NAN, b[i] = 0.f;
          if (j < mine.count) load_logits<VEC>(row_scores + mine.expert(j), q);
          if (s.bias && j < mine.count) load_logits<VEC>(s.bias + mine.expert(j), b);
          const float floor = j < mine.count ? -INFINITY : NAN;
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            float c = SIGMOID ? q[i] : q[i] * inv;
            if (s.bias) v[j + i] = c = compared(q[i], b[i], floor);
            if (s.groups > 1) {
              c = fmaxf(c, -INFINITY);  // (none there)
              top[1] = fmaxf(top[1], fminf(top[0], c));
              top[0] = fmaxf(top[0], c);
            }
          }
        }
      }
      if (s.groups > 1) {
        if (by_logit)
#pragma unroll
          for (int j = 0; j < VPL; ++j) top[0] = fmaxf(top[0], v[j]);
        for (int o = s.lanes / 2; o; o >>= 1) {
          const float a = __shfl_xor_sync(~0u, top[0], o), b = __shfl_xor_sync(~0u, top[1], o);
          top[1] = fmaxf(fmaxf(top[1], b), fminf(top[0], a));
          top[0] = fmaxf(top[0], a);
        }
        const float worth = fmaxf(s.best == 2 ? top[0] + top[1] : top[0], -INFINITY);
        kept = group_kept(s, ordered_bits(worth), mine.group);
        if (!by_logit && s.kept < s.groups) {
          const float last = -warp_max(kept ? -worth : -INFINITY);
          const float next = warp_max(mine.have && !kept ? worth : -INFINITY);
          // two sums of one or two scores (and biases)
          const float size = 2.f * s.best * largest + fabsf(last) + fabsf(next);
          if (!(last - next > size * step)) {
            // experts that may be among the largest of their group
            // (an infinite one as it is: inf - inf would leave out all of them)
            const float least = s.best == 2 ? top[1] : top[0];
            const float margin = isinf(least) ? 0.f : (2.f * largest + 0.5f * fabsf(least)) * step;
            const int by_value = keep_exactly(
                s, row, row_scores, SIGMOID ? 1.f : inv, most, least - margin, VEC,
                reinterpret_cast<int*>(candidates[warp]),
                reinterpret_cast<Two*>(candidates[warp] + 32));
            if (__any_sync(~0u, by_value < 0))
              exact = false;
            else
              kept = by_value;
          }
        }
        if (!kept)
#pragma unroll
          for (int j = 0; j < VPL; ++j) v[j] = NAN;
      }
    }
    // Candidates: all from a threshold on that leaves k + 1 of them at least, and 64 at most.  At
    // least as many are above it as there are lanes' halves whose largest is: bisected until those
    // are few.  (As keys in the values' order; 0: none.)
    float half[2] = {NAN, NAN};
#pragma unroll
    for (int j = 0; j < VPL; ++j) half[j >= VPL / 2] = fmaxf(half[j >= VPL / 2], v[j]);
    const uint32_t key0 = half[0] == half[0] ? ordered_bits(half[0]) : 0;
    const uint32_t key1 = half[1] == half[1] ? ordered_bits(half[1]) : 0;
    const auto above = [&](uint32_t from) {
      return __popc(__ballot_sync(~0u, key0 >= from)) + __popc(__ballot_sync(~0u, key1 >= from));
    };
    const uint32_t low = min(key0, key1);
    uint32_t over = __reduce_max_sync(~0u, max(key0, key1));
    uint32_t least = __reduce_min_sync(~0u, low ? low : ~0u);
    constexpr uint32_t kLowest = 0x007fffffu;  // of -inf
    if (above(least) <= s.k) least = kLowest;
    for (int i = 0; i < 12 && least < over; ++i) {
      const uint32_t middle = least + (over - least + 1) / 2;
      const int n = above(middle);
      if (n <= s.k) {
        over = middle - 1;
      } else {
        least = middle;
        if (n <= s.k + 8) break;
      }
    }
    float from;
    uint64_t own;  // the lane's values from there on, a bit to each
    int n;
    // Counted; and, where they are more than 64 (rare), bisected on by their own number.
    uint32_t under = least, most_key = __reduce_max_sync(~0u, max(key0, key1));
    for (;;) {
      from = ordered_value(least);
      uint32_t low_bits = 0, high_bits = 0;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (v[j] >= from) (j < 32 ? low_bits : high_bits) |= 1u << (j & 31);
      own = low_bits | static_cast<uint64_t>(high_bits) << 32;
      n = __reduce_add_sync(~0u, __popc(low_bits) + __popc(high_bits));
      if (n > 64)
        under = least;
      else if (n <= s.k && least > under)
        most_key = least - 1;
      else
        break;
      if (under >= most_key) break;
      least = under + (most_key - under + 1) / 2;
    }
    int chosen = 0;
    if (n > 64 || (n <= s.k && least > kLowest)) {  // (equal ones are not parted)
      exact = false;
    } else if (exact) {
      const int count = __popcll(own);
      int to = count;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int before = __shfl_up_sync(~0u, to, o);
        if (lane >= o) to += before;
      }
      to -= count;
      // as (the expert's complement, key), which as 64 bits are in the order wanted; read again, since
      // which of v they are is not known to the compiler (28 conditional stores took more)
      uint2* list = candidates[warp];
      for (; own; own &= own - 1) {
        const int e = mine.expert(__ffsll(own) - 1);
        float c;
        if (s.bias)
          c = compared(row_scores[e], s.bias[e], -INFINITY);
        else
          c = fmaxf(logit(row, e), -INFINITY);
        list[to++] = make_uint2(~static_cast<uint32_t>(e), ordered_bits(c));
      }
      if (lane < 4) list[n + lane] = make_uint2(0, 0);
      uint2* sorted = list + 68;
      sorted[lane] = make_uint2(~static_cast<uint32_t>(kMaxE), 0);
      if (lane == 0) sorted[32] = sorted[0];
      __syncwarp();
      // Up to two to a lane; each one's place is the number of those before it.
      const uint2 first = lane < n ? list[lane] : make_uint2(~static_cast<uint32_t>(kMaxE), 0);
      const uint2 second = lane + 32 < n ? list[lane + 32] : make_uint2(~static_cast<uint32_t>(kMaxE), 0);
      const auto both = [](uint2 c) { return c.x | static_cast<uint64_t>(c.y) << 32; };
      const uint64_t mine0 = both(first), mine1 = both(second);
      int place0 = 0, place1 = 0;
      for (int i = 0; i < n; i += 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t other = both(list[i + j]);
          place0 += other > mine0;
          if (n > 32) place1 += other > mine1;
        }
      }
      if (lane < n && place0 <= s.k) sorted[place0] = first;
      if (lane + 32 < n && place1 <= s.k) sorted[place1] = second;
      __syncwarp();
      const int expert0 = static_cast<int>(~first.x), expert1 = static_cast<int>(~second.x);
      chosen = static_cast<int>(~sorted[lane].x);
      const uint32_t of = sorted[lane].y, after = lane < s.k ? sorted[lane + 1].y : 0;
      if (s.bias) {
        bool near = false, edge = false;
        if (lane < s.k && after) {
          const float a = ordered_value(of), b = ordered_value(after);
          const float size = 2.f * largest + (fabsf(a) + fabsf(b)) * 0.25f;
          near = !(a - b > size * step);
          // candidates end too near to the last one chosen
          edge = lane == s.k - 1 && !(a - from > size * step);
        }
        if (__any_sync(~0u, near)) {
          if (__any_sync(~0u, edge))
            exact = false;
          else
            chosen = order_exactly(s, row, most, VEC, expert0, expert1);
        }
      }
    }
    if (!exact) chosen = select_exactly(s, row, most, VEC);
    const bool slot = lane < s.k;
    const float l = slot ? logit(row, chosen) : -INFINITY;
    float g;
    if (s.renormalise)
      g = share(l, SIGMOID);
    else if (SIGMOID)
      g = sigmoid(l);
    else
      g = sum == 0.f ? 0.f : unscaled(l, most, false) / sum;
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
    if (tokens == kWarps) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum = fmaf(scores[w * s.E + e], share_of[w], sum);
    } else {
#pragma unroll 1
      for (int w = 0; w < tokens; ++w) sum = fmaf(scores[w * s.E + e], share_of[w], sum);
    }
    s.partials[static_cast<long long>(blockIdx.x) * s.E + e] = sum;
  }
}

struct SelectGrad {
  int T, E, k;
  int sigmoid, renormalise;
  int wide;  // 16 bytes of dlogits to a store
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
// One warp to a token.  Bound by the round trips idx -> logit and the stores of zeros: 8192 x 896 in fp32
// 9 us (29 MB written, 4 us).
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
  if (dense)
    for (int i = lane; i < s.E; i += 32)
      out[i] = static_cast<T>(-dot * (expf(logit(row, i) - most) * inv));
  else if (s.wide)
    for (int i = lane; i < s.E * static_cast<int>(sizeof(T)) / 16; i += 32)
      reinterpret_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
  else
    for (int i = lane; i < s.E; i += 32) out[i] = static_cast<T>(0.f);
  __syncwarp();
  // the parts of an expert that is named twice are added in the slots' order by the first of them
  const unsigned same = __match_any_sync(~0u, e);
  float sum = v;
  if (__any_sync(~0u, e >= 0 && (same & (same - 1)))) {
    sum = 0.f;
    for (int j = 0; j < s.k; ++j) {
      const float other = __shfl_sync(~0u, v, j);
      if (same >> j & 1) sum += other;
    }
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

// Calls f(VPL, VEC) for what a lane holds.
template <typename F>
void with_values(int per_lane, bool fours, F f) {
  const auto with = [&](auto v) {
    if (fours)
      f(v, std::integral_constant<int, 4>{});
    else
      f(v, std::integral_constant<int, 1>{});
  };
  if (per_lane <= 4)
    with(std::integral_constant<int, 4>{});
  else if (per_lane <= 8)
    with(std::integral_constant<int, 8>{});
  else if (per_lane <= 16)
    with(std::integral_constant<int, 16>{});
  else if (per_lane <= 28)
    with(std::integral_constant<int, 28>{});
  else if (per_lane <= 32)
    with(std::integral_constant<int, 32>{});
  else
    with(std::integral_constant<int, 64>{});
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
  s.lanes_log2 = 5;
  for (int g = 1; g < s.groups; g *= 2) s.lanes /= 2, --s.lanes_log2;
  s.sigmoid = rule->score == MOE_SCORE_SIGMOID;
  s.renormalise = rule->renormalise != 0;
  s.scale = rule->scale;
  s.logits = logits, s.ld = T == 1 ? 0 : ld_logits, s.bias = select_bias;
  s.idx = topk_idx, s.gate = topk_gate, s.partials = prob_partials;
  mark_before(MOE_KERNEL_ROUTE_SELECT, stream);
  cudaError_t err = cudaSuccess;
  // four neighbours to a load where rows and groups begin on such boundaries
  const int bytes = dtype == MOE_F32 ? 16 : 8;
  const bool fours = s.group_size % 4 == 0 && s.ld % 4 == 0 && !misaligned(logits, bytes) &&
                     !misaligned(select_bias, 16);
  const int vec = fours ? 4 : 1, per = s.lanes * vec;
  with_values((s.group_size + per - 1) / per * vec, fours, [&](auto v, auto c) {
    constexpr int VPL = decltype(v)::value, VEC = decltype(c)::value;
    const bool stored = prob_partials || s.bias || s.groups > 1 || (!s.sigmoid && !s.renormalise);
    const int smem = stored ? kWarps * E * 4 : 0;
    const auto launch = [&](auto kernel) {
      err = launch_behind(kernel, blocks_of(T), kWarps * 32, smem, stream, s);
    };
    const auto with = [&](auto type) {
      using L = decltype(type);
      if (s.sigmoid)
        launch(route_select_kernel<L, VPL, VEC, true>);
      else
        launch(route_select_kernel<L, VPL, VEC, false>);
    };
    if (dtype == MOE_F32)
      with(float{});
    else
      with(__nv_bfloat16{});
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
  s.wide = !misaligned(dlogits, 16) && E * (dtype == MOE_F32 ? 4 : 2) % 16 == 0;
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
