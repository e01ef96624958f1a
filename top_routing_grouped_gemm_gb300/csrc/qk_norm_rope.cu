// Norm of query and key heads with the rotation by position, forward and backward
// (include/linear_attention.h has the formulas).
#include <math.h>
#include <stdlib.h>

#include <algorithm>
#include <type_traits>

#include "moe_internal.h"
#include "overlap.cuh"
#include "ptx.cuh"

#include "../../include/linear_attention.h"

namespace moe {
namespace {

constexpr int kMaxD = 256, kMaxHeads = 4096;
// Of the GPU that the cuts are made for.  (Not asked of the driver: the workspace's size follows from
// the cuts, and has to be the same wherever and before whatever it is asked for.)
constexpr int kSms = 152;

// One group of heads (q or k) as the kernels see it.
struct Side {
  const void* x;
  const void* dy;
  void* out;  // y, or dx
  const float* weight;
  long long x_ts, x_hs, dy_ts, dy_hs, o_ts, o_hs;
  int w_hs;  // values between the weight rows of two heads: D, or 0 for one shared row
  int heads;
};

// A lane holds two quads of a row (a token's head): with halves paired, values 4 j .. 4 j + 3 of
// the first half and their partners in the second, so that a rotation stays within the lane; with
// neighbours paired, and for the values that are not rotated, eight consecutive ones.
template <typename T>
struct Raw;  // as loaded

template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int far) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p + far));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

template <>
struct Raw<__nv_bfloat16> {
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int far) {
    a = __ldcs(reinterpret_cast<const uint2*>(p));
    b = __ldcs(reinterpret_cast<const uint2*>(p + far));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

__device__ __forceinline__ void store(float* p, int far, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(p + far), make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store(__nv_bfloat16* p, int far, const float (&v)[8]) {
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])));
  __stcs(reinterpret_cast<uint2*>(p + far),
         make_uint2(pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
}

// A block takes some heads of a range of tokens, in tiles.  D / 8 neighbouring lanes of a warp hold a
// row, as many rows as the warp has room for, and always the same head, so that its weight stays in
// registers and its weight gradient gathers there.  (On a power of two of lanes, rows of 80 values
// leave 6 of 16 idle: 62500 tokens x 20 heads of 80 bf16 took 130 us so, 86 us now.)  The
// block forms the tile's sines and cosines once, in shared memory, for all its heads.
constexpr int kThreads = 256;
// Rows of 8 values that a lane has on their way; the forward, which shares the registers among more
// blocks, has fewer of them in fp32 (9765 tokens x 40 heads x 128 took 69.3 us with four, 66.4 us with
// two).
constexpr int kRows = 4;
template <typename T>
constexpr int kForwardRows = sizeof(T) == 4 ? 2 : kRows;
constexpr int kIdle = 1 << 20;  // a token that no tile has
constexpr int kForwardBlocks = 4, kBackwardBlocks = 2;  // to an SM

struct Shape {
  int N, D, rot, interleaved, heads_per_block, tokens_per_block, tile;
  float eps;
  const int* pos;
  const double* inv_freq;
};

// The tile's angles.  A thread keeps one pair: its frequency in turns a token, as a 64-bit fraction
// of a turn.  Times the position in whole numbers that wraps as turns do, so the angle is exact but
// for the frequency's own rounding (2^-53 of it, times the position), at any position; a product in
// 64-bit floating point would be as exact, at a thirtieth of the rate on this GPU.  The upper 32
// bits go on to the sine and cosine in fp32.  A lane rotates four pairs: place j holds pairs
// 4 j .. 4 j + 3 as two float4 (cos, sin, cos, sin), the first ones of all places before the
// second ones, so that the lanes of a row read without conflicts.
struct Angles {
  unsigned long long fraction;
  int pair, token, step, to;  // its pair, first token, tokens between, and place in a token's table

  __device__ __forceinline__ explicit Angles(const Shape& s) {
    const int half = s.rot / 2;
    step = kThreads / max(half, 1);
    token = threadIdx.x / max(half, 1);
    pair = threadIdx.x - token * half;
    to = (pair % 4 / 2 * (half / 4) + pair / 4) * 2 + pair % 2;
    if (token >= step || half == 0) {
      token = kIdle;
      return;
    }
    double f = s.inv_freq[pair] * 0.15915494309189533577;
    f -= floor(f);
    fraction = static_cast<unsigned long long>(f * 18446744073709551616.0);
  }

  __device__ __forceinline__ void fill(float4* table, const Shape& s, long long t0, int n) const {
    for (int t = token; t < n; t += step) {
      const long long pos = s.pos[t0 + t];
      const int turns = static_cast<int>(fraction * static_cast<unsigned long long>(pos) >> 32);
      float2 cs;
      sincospif(static_cast<float>(turns) * 4.656612873077393e-10f, &cs.y, &cs.x);  // 2^-31
      reinterpret_cast<float2*>(table)[t * (s.rot / 2) + to] = cs;
    }
  }
};

// What a lane has to do.  The lanes of a row are L = D / 8 of them (FULL), or L is the least power of
// two that is not less.
template <int L, bool FULL>
struct Lane {
  int near, far;     // its first quad, and the second from there
  int place, lanes;  // among the lanes of its row
  int head, slot;    // head of all heads; tokens slot, slot + stride, ... of a tile
  int group, stride;
  bool turns;        // rotates its values

  __device__ __forceinline__ Lane(const Shape& s, int heads) {
    lanes = FULL ? L : s.D / 8;
    const int lane = threadIdx.x & 31, per_warp = 32 / lanes, row = lane / lanes;
    place = lane - row * lanes;
    group = threadIdx.x / 32 * per_warp + row;
    stride = kThreads / 32 * per_warp / s.heads_per_block;
    slot = group / s.heads_per_block;
    head = blockIdx.y * s.heads_per_block + group % s.heads_per_block;
    // lanes without a row read what another row's lanes read
    if (row >= per_warp || slot >= stride || head >= heads)
      slot = kIdle, head = heads - 1, group = -1;
    turns = place * 8 < s.rot;
    const bool halves = turns && !s.interleaved;
    near = place * (halves ? 4 : 8);
    far = halves ? s.rot / 2 : 4;
  }

  // The sum over the row's lanes.
  __device__ __forceinline__ float row_sum(float v) const {
    if constexpr (FULL) {
#pragma unroll
      for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
      return v;
    } else {
#pragma unroll
      for (int o = L / 2; o; o >>= 1) {  // the first o lanes get those behind them
        const float behind = __shfl_down_sync(~0u, v, o);
        if (place + o < lanes) v += behind;
      }
      return __shfl_sync(~0u, v, (threadIdx.x & 31) - place);
    }
  }
};

// R(th) v, or R(-th) v (BACK).
template <bool BACK>
__device__ __forceinline__ void rotate(float (&v)[8], const float4* cs, const Shape& s) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float4 w = cs[c * (s.rot / 8)];
    const float cosv[2] = {w.x, w.z}, sinv[2] = {BACK ? -w.y : w.y, BACK ? -w.w : w.w};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * c + e;
      if (s.interleaved) {
        const float x0 = v[2 * i], x1 = v[2 * i + 1];
        v[2 * i] = x0 * cosv[e] - x1 * sinv[e];
        v[2 * i + 1] = x1 * cosv[e] + x0 * sinv[e];
      } else {
        const float x0 = v[i], x1 = v[i + 4];
        v[i] = x0 * cosv[e] - x1 * sinv[e];
        v[i + 4] = x1 * cosv[e] + x0 * sinv[e];
      }
    }
  }
}

template <int L, bool FULL>
__device__ __forceinline__ void load_weight(const Side& side, int h, const Lane<L, FULL>& me,
                                            float (&w)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e] = side.weight ? side.weight[static_cast<long long>(h) * side.w_hs + me.near +
                                     (e < 4 ? e : me.far + e - 4)]
                       : 1.f;
}

// Every row is read and written once: 32768 tokens x 32 heads x 128 bf16 take 89.8 us, 0.89 of the
// rate of a plain copy, with 63 % of the issue slots used (2.5 us more with addresses from each row's
// index, which cost instructions that these 64-bit steps do not).  Two or three rows on their way instead of four, and three or five blocks
// to an SM instead of kForwardBlocks, take 5 to 12 % longer; partners in other lanes, with shuffles,
// and blocks in several waves took 131 us.
template <typename T, int L, bool FULL>
__global__ void __launch_bounds__(kThreads, kForwardBlocks)
    rope_forward_kernel(const Shape s, const Side q, const Side k) {
  extern __shared__ float4 table[];  // [2][tile][rot / 4]
  after_previous();
  const Angles angles(s);
  const Lane<L, FULL> me(s, q.heads + k.heads);
  const Side& side = me.head < q.heads ? q : k;
  const int h = me.head < q.heads ? me.head : me.head - q.heads;
  float w[8];
  load_weight(side, h, me, w);
  const T* x = static_cast<const T*>(side.x) + h * side.x_hs + me.near;
  T* y = static_cast<T*>(side.out) + h * side.o_hs + me.near;
  const long long x_step = me.stride * side.x_ts, o_step = me.stride * side.o_ts;
  const int cs_step = me.stride * (s.rot / 4);
  const int lo = blockIdx.x * s.tokens_per_block, hi = min(lo + s.tokens_per_block, s.N);
  const float inv_D = 1.f / s.D;
  int buf = 0;
  for (int t0 = lo; t0 < hi; t0 += s.tile, buf ^= 1) {
    const int n = min(s.tile, hi - t0);
    const float4* cs = table + buf * s.tile * (s.rot / 4);
    angles.fill(table + buf * s.tile * (s.rot / 4), s, t0, n);
    __syncthreads();  // (the other buffer's readers are done when they come here again)
    const T* from = x + (t0 + min(me.slot, n - 1)) * side.x_ts;
    T* to = y + (t0 + me.slot) * side.o_ts;
    cs += me.slot * (s.rot / 4) + me.place;
    // the same number of rounds for all lanes: they shuffle
    for (int left = n - me.slot, round = 0; round < n; round += kForwardRows<T> * me.stride) {
      Raw<T> raw[kForwardRows<T>];
#pragma unroll
      for (int u = 0; u < kForwardRows<T>; ++u) {
        raw[u].load(from, me.far);
        if (left > (u + 1) * me.stride) from += x_step;  // past the last row: that row again
      }
#pragma unroll
      for (int u = 0; u < kForwardRows<T>; ++u, left -= me.stride, to += o_step, cs += cs_step) {
        float v[8], sum = 0.f;
        raw[u].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
        const float rstd = rsqrtf(fmaf(me.row_sum(sum), inv_D, s.eps));
        if (left > 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= rstd * w[e];
          if (me.turns) rotate<false>(v, cs, s);
          store(to, me.far, v);
        }
      }
    }
  }
}

// x and dy are read once and dx is written once; with dy in fp32 the same rows take 173.5 us, 0.93
// of the rate of a copy (fewer rows on their way or more blocks to an SM: 5 to 11 % longer).  The weights'
// gradients stay in registers over all of a block's tokens, and no atomic orders their sums.
// partial: [blocks][2][D] (the shared weights of q and k) or [gridDim.x][heads][D] (a row for each
// head), the sums of the block's rows; null: not wanted.
template <typename T, typename G, int L, bool FULL>
__global__ void __launch_bounds__(kThreads, kBackwardBlocks)
    rope_backward_kernel(const Shape s, const Side q, const Side k, float* partial) {
  extern __shared__ float4 table[];  // [2][tile][rot / 4]
  __shared__ float sums[kThreads * 8];  // [group][D]
  after_previous();
  const Angles angles(s);
  const int heads = q.heads + k.heads;
  const Lane<L, FULL> me(s, heads);
  const Side& side = me.head < q.heads ? q : k;
  const int h = me.head < q.heads ? me.head : me.head - q.heads;
  float w[8], dw[8] = {};
  load_weight(side, h, me, w);
  const T* x = static_cast<const T*>(side.x) + h * side.x_hs + me.near;
  const G* dy = static_cast<const G*>(side.dy) + h * side.dy_hs + me.near;
  T* dx = static_cast<T*>(side.out) + h * side.o_hs + me.near;
  const long long lo = static_cast<long long>(blockIdx.x) * s.tokens_per_block;
  const long long hi = min(lo + s.tokens_per_block, static_cast<long long>(s.N));
  const float inv_D = 1.f / s.D;
  int buf = 0;
  for (long long t0 = lo; t0 < hi; t0 += s.tile, buf ^= 1) {
    float4* now = table + buf * s.tile * (s.rot / 4);
    const int n = static_cast<int>(min(static_cast<long long>(s.tile), hi - t0));
    angles.fill(now, s, t0, n);
    __syncthreads();
    for (int t = 0; t < n; t += kRows * me.stride) {
      const int first = t + me.slot;
      Raw<T> raw[kRows];
      Raw<G> raw_d[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const long long at = t0 + min(first + u * me.stride, n - 1);
        raw[u].load(x + at * side.x_ts, me.far);
        raw_d[u].load(dy + at * side.dy_ts, me.far);
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int at = first + u * me.stride;
        float v[8], d[8];
        raw[u].get(v);
        raw_d[u].get(d);
        if (me.turns) rotate<true>(d, now + min(at, n - 1) * (s.rot / 4) + me.place, s);
        // both sums of the row at once: u = w dn; mean(u x^) = rstd mean(u x)
        float sum = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum = fmaf(v[e], v[e], sum);
          dot = fmaf(d[e] * w[e], v[e], dot);
        }
        const float rstd = rsqrtf(fmaf(me.row_sum(sum), inv_D, s.eps));
        const float c = me.row_sum(dot) * inv_D * rstd * rstd;
        if (at < n) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dw[e] = fmaf(d[e], v[e] * rstd, dw[e]);
            d[e] = rstd * fmaf(-c, v[e], d[e] * w[e]);
          }
          store(dx + (t0 + at) * side.o_ts, me.far, d);
        }
      }
    }
  }
  if (!partial) return;
  if (me.group >= 0)
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[me.group * s.D + me.near + (e < 4 ? e : me.far + e - 4)] = dw[e];
  __syncthreads();
  const int groups = me.stride * s.heads_per_block;
  const int first = blockIdx.y * s.heads_per_block;
  if (q.w_hs || k.w_hs) {  // a row for each head: its groups, every heads_per_block'th
    for (int i = threadIdx.x; i < s.heads_per_block * s.D; i += kThreads) {
      const int head = i / s.D, e = i % s.D;
      if (first + head >= heads) continue;
      float sum = 0.f;
      for (int g = head; g < groups; g += s.heads_per_block) sum += sums[g * s.D + e];
      partial[(static_cast<long long>(blockIdx.x) * heads + first + head) * s.D + e] = sum;
    }
  } else {
    for (int i = threadIdx.x; i < 2 * s.D; i += kThreads) {
      const int of_k = i / s.D, e = i % s.D;
      float sum = 0.f;
      for (int g = 0; g < groups; ++g) {
        const int head = first + g % s.heads_per_block;
        if (head < heads && (head >= q.heads) == of_k) sum += sums[g * s.D + e];
      }
      partial[(static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * s.D + i] = sum;
    }
  }
}

// The weight gradients of one side from the blocks' sums: row b of its `rows` (of D values) is the sum
// of rows b + j + i `step` of `from`, j < inner, i < outer.
struct Sums {
  const float* from;
  float* dweight;
  int rows, outer, inner;
};

// 32 columns of one row, of q or of k, to a block; its 32 warps take every 32nd of the rows to add each
// and are then added in order.
__global__ void __launch_bounds__(1024)
    rope_dweight_kernel(const Sums q, const Sums k, int step, int D) {
  __shared__ float sums[32][33];
  after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  const bool of_k = static_cast<int>(blockIdx.y) >= q.rows;
  const Sums& side = of_k ? k : q;
  const long long row = blockIdx.y - (of_k ? q.rows : 0);
  const float* from = side.from + row * D + i;
  const int outer = side.outer, inner = side.inner;
  float sum = 0.f;
  if (i < D)
#pragma unroll 4
    for (int r = warp; r < outer * inner; r += 32)
      sum += from[(static_cast<long long>(r / inner) * step + r % inner) * D];
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int v = 1; v < 32; ++v) sum += sums[v][lane];
  if (i < D) side.dweight[row * D + i] = sum;
}

// ------------------------------------------------------------------------ host side

// Rows that a block has at once: 8 values to a lane.
int rows_of(int D) { return kThreads / 32 * (32 / (D / 8)); }

// Heads of a block: what leaves fewest lanes idle (of a block's lanes, and of the last part's
// heads), against the angles that each part of the heads forms anew.  In instructions a row, about
// 90 for each lane and 50 for each pair's angle, all values of a head taken as turned: the workspace's
// size, which follows the same cut, is asked for without rotary_dim.  (16 + 4 heads of 96, 16 rows to a block: two parts
// of 10 heads leave 3 / 8 of the lanes idle, four of 5 leave 1 / 16; the backward of 26041 tokens
// in bf16 takes 125 and 108 us.)
int heads_of_block(int D, int heads) {
  const int rows = rows_of(D);
  int best = 1;
  double least = 1e30;
  for (int h = 1; h <= std::min(heads, rows); ++h) {
    const int parts = (heads + h - 1) / h;
    const double busy = static_cast<double>(rows / h * h) / rows * heads / (parts * h);
    const double cost = 90.0 * kThreads / rows / busy + D / 2 * 50.0 / h;
    if (cost <= least) least = cost, best = h;
  }
  return best;
}

// The heads in parts, and the tokens in as many parts as fill the GPU once, or fewer if there are
// fewer tokens.
// A tile is what a block's lanes take in a few rounds of kRows rows each, or less where its angles
// would not fit 32 KB twice.
struct Cuts {
  int heads_per_block, head_parts, tokens_per_block, token_parts, at_once;

  int tile(int rot) const {
    const int round = kRows * at_once, fit = rot ? 4096 / rot : round;
    if (round <= fit) return round * std::max(1, std::min(16, fit) / round);
    return std::max(at_once, fit / at_once * at_once);
  }
};

Cuts cuts_of(int N, int D, int heads, int blocks_per_sm) {
  Cuts c;
  const int rows = rows_of(D);
  c.heads_per_block = heads_of_block(D, heads);
  c.head_parts = (heads + c.heads_per_block - 1) / c.heads_per_block;
  c.at_once = rows / c.heads_per_block;  // tokens
  const long long parts = std::max(1, blocks_per_sm * kSms / c.head_parts);
  const long long per = (N + parts - 1) / parts;
  c.tokens_per_block = static_cast<int>((per + c.at_once - 1) / c.at_once * c.at_once);
  c.token_parts = static_cast<int>((static_cast<long long>(N) + c.tokens_per_block - 1) / c.tokens_per_block);
  return c;
}

bool bad_align(const void* p) { return misaligned(p, 16); }

// Whether the rows [N, heads] of D values at these strides overlap.
bool overlap(long long N, long long heads, long long D, long long ts, long long hs) {
  if (N == 1) ts = heads * llabs(hs) + D;
  if (heads == 1) hs = N * llabs(ts) + D;
  const bool token_major = hs >= D && ts >= (heads - 1) * hs + D;
  const bool head_major = ts >= D && hs >= (N - 1) * ts + D;
  return !(token_major || head_major);
}

int check_common(int N, int D, int rot, int dtype, float eps, const void* pos, const void* freq) {
  if (N <= 0 || D <= 0 || rot < 0 || rot > D || !(eps > 0.f) || !(eps <= 3e38f))
    return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (rot > 0 && (!pos || !freq)) return MOE_ERR_INVALID_ARG;
  if (D % 8 || D > kMaxD || rot % 16 || N > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (misaligned(pos, 4) || misaligned(freq, 8)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_rows(const void* p, long long ts, long long hs) {
  if (!p) return MOE_ERR_INVALID_ARG;
  return bad_align(p) || ts % 8 || hs % 8 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int check_heads(int N, int heads, const float* weight) {
  if (heads <= 0) return MOE_ERR_INVALID_ARG;
  if (heads > kMaxHeads || bad_align(weight)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int side_of(int N, int D, const moe_qk_rows* r, Side* s) {
  if (int e = check_heads(N, r->heads, r->weight)) return e;
  if (int e = check_rows(r->x, r->x_token_stride, r->x_head_stride)) return e;
  if (int e = check_rows(r->y, r->y_token_stride, r->y_head_stride)) return e;
  if (overlap(N, r->heads, D, r->y_token_stride, r->y_head_stride)) return MOE_ERR_INVALID_ARG;
  *s = Side{r->x, nullptr, r->y, r->weight, r->x_token_stride, r->x_head_stride, 0, 0,
            r->y_token_stride, r->y_head_stride, r->weight_per_head ? D : 0, r->heads};
  return MOE_OK;
}

int side_of(int N, int D, const moe_qk_grads* r, Side* s) {
  if (int e = check_heads(N, r->heads, r->weight)) return e;
  if (int e = check_rows(r->x, r->x_token_stride, r->x_head_stride)) return e;
  if (int e = check_rows(r->dy, r->dy_token_stride, r->dy_head_stride)) return e;
  if (int e = check_rows(r->dx, r->dx_token_stride, r->dx_head_stride)) return e;
  if (bad_align(r->dweight)) return MOE_ERR_UNSUPPORTED;
  if (overlap(N, r->heads, D, r->dx_token_stride, r->dx_head_stride)) return MOE_ERR_INVALID_ARG;
  *s = Side{r->x, r->dy, r->dx, r->weight, r->x_token_stride, r->x_head_stride,
            r->dy_token_stride, r->dy_head_stride, r->dx_token_stride, r->dx_head_stride,
            r->weight_per_head ? D : 0, r->heads};
  return MOE_OK;
}

// Rows of the partial sums: two for each block, or one for each head and part of the tokens.
size_t backward_ws(int N, int D, int q_heads, int k_heads) {
  const Cuts c = cuts_of(N, D, q_heads + k_heads, kBackwardBlocks);
  return up256(static_cast<size_t>(c.token_parts) *
               std::max(2 * c.head_parts, q_heads + k_heads) * D * 4);
}

// Calls f(L, FULL) for the lanes of a row.
template <typename F>
void with_lanes(int D, F f) {
  const int lanes = D / 8;
  const auto with = [&](auto L) {
    if (lanes == L)
      f(L, std::true_type{});
    else
      f(L, std::false_type{});
  };
  if (lanes > 16)
    with(std::integral_constant<int, 32>{});
  else if (lanes > 8)
    with(std::integral_constant<int, 16>{});
  else
    with(std::integral_constant<int, 8>{});
}

}  // namespace
}  // namespace moe

extern "C" {

using namespace moe;

int moe_qk_norm_rope(int32_t N, int32_t D, int32_t rotary_dim, int32_t interleaved, int32_t dtype,
                     float eps, const int32_t* positions, const double* inv_freq,
                     const moe_qk_rows* q, const moe_qk_rows* k, moe_stream_t stream) {
  if (!q) return MOE_ERR_INVALID_ARG;
  if (int e = check_common(N, D, rotary_dim, dtype, eps, positions, inv_freq)) return e;
  Side sq{}, sk{};
  if (int e = side_of(N, D, q, &sq)) return e;
  if (k)
    if (int e = side_of(N, D, k, &sk)) return e;
  const Cuts c = cuts_of(N, D, sq.heads + sk.heads, kForwardBlocks);
  const Shape s{N, D, rotary_dim, interleaved != 0, c.heads_per_block, c.tokens_per_block,
                c.tile(rotary_dim), eps, positions, inv_freq};
  const dim3 grid(c.token_parts, c.head_parts);
  const int smem = 2 * s.tile * rotary_dim * 4;
  mark_before(MOE_KERNEL_QK_NORM_ROPE, stream);
  cudaError_t err = cudaSuccess;
  with_lanes(D, [&](auto lanes, auto full) {
    constexpr int L = decltype(lanes)::value;
    constexpr bool FULL = decltype(full)::value;
    if (dtype == MOE_BF16)
      err = launch_behind(rope_forward_kernel<__nv_bfloat16, L, FULL>, grid, kThreads, smem, stream,
                          s, sq, sk);
    else
      err = launch_behind(rope_forward_kernel<float, L, FULL>, grid, kThreads, smem, stream,
                          s, sq, sk);
  });
  mark_after(MOE_KERNEL_QK_NORM_ROPE, stream);
  count_launches(1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_qk_norm_rope_backward_workspace_size(int32_t N, int32_t D, int32_t q_heads,
                                                int32_t k_heads) {
  if (N <= 0 || N > (1 << 30) || D <= 0 || D > kMaxD || D % 8 || q_heads <= 0 ||
      q_heads > kMaxHeads || k_heads < 0 || k_heads > kMaxHeads)
    return 0;
  return backward_ws(N, D, q_heads, k_heads);
}

int moe_qk_norm_rope_backward(int32_t N, int32_t D, int32_t rotary_dim, int32_t interleaved,
                              int32_t dtype, int32_t dy_dtype, float eps,
                              const int32_t* positions, const double* inv_freq,
                              const moe_qk_grads* q, const moe_qk_grads* k, void* workspace,
                              size_t workspace_bytes, moe_stream_t stream) {
  if (!q || (dy_dtype != MOE_F32 && dy_dtype != dtype)) return MOE_ERR_INVALID_ARG;
  if (int e = check_common(N, D, rotary_dim, dtype, eps, positions, inv_freq)) return e;
  Side sq{}, sk{};
  if (int e = side_of(N, D, q, &sq)) return e;
  if (k)
    if (int e = side_of(N, D, k, &sk)) return e;
  const int heads = sq.heads + sk.heads;
  const bool weights = q->dweight || (k && k->dweight);
  float* partial = nullptr;
  if (weights) {
    if (!workspace || workspace_bytes < backward_ws(N, D, sq.heads, sk.heads))
      return MOE_ERR_WORKSPACE;
    if (bad_align(workspace)) return MOE_ERR_UNSUPPORTED;
    partial = static_cast<float*>(workspace);
  }
  const Cuts c = cuts_of(N, D, heads, kBackwardBlocks);
  const Shape s{N, D, rotary_dim, interleaved != 0, c.heads_per_block, c.tokens_per_block,
                c.tile(rotary_dim), eps, positions, inv_freq};
  const dim3 grid(c.token_parts, c.head_parts);
  const int smem = 2 * s.tile * rotary_dim * 4;
  mark_before(MOE_KERNEL_QK_NORM_ROPE_BWD, stream);
  cudaError_t err = cudaSuccess;
  with_lanes(D, [&](auto lanes, auto full) {
    constexpr int L = decltype(lanes)::value;
    constexpr bool FULL = decltype(full)::value;
    using B = __nv_bfloat16;
    if (dtype == MOE_F32)
      err = launch_behind(rope_backward_kernel<float, float, L, FULL>, grid, kThreads, smem, stream,
                          s, sq, sk, partial);
    else if (dy_dtype == MOE_F32)
      err = launch_behind(rope_backward_kernel<B, float, L, FULL>, grid, kThreads, smem, stream,
                          s, sq, sk, partial);
    else
      err = launch_behind(rope_backward_kernel<B, B, L, FULL>, grid, kThreads, smem, stream,
                          s, sq, sk, partial);
  });
  if (weights) {
    // rows of partial: two for each block, or, if either side has a weight for each head, one for
    // each head (a shared weight's are then added over its heads)
    const bool by_head = sq.w_hs || sk.w_hs;
    const auto sums = [&](const moe_qk_grads* side, int place, int first_head) {
      if (!side || !side->dweight) return Sums{};
      return Sums{partial + static_cast<size_t>(by_head ? first_head : place) * D, side->dweight,
                  side->weight_per_head ? side->heads : 1,
                  by_head ? c.token_parts : c.token_parts * c.head_parts,
                  by_head && !side->weight_per_head ? side->heads : 1};
    };
    const Sums of_q = sums(q, 0, 0), of_k = sums(k, 1, sq.heads);
    if (err == cudaSuccess)
      err = launch_behind(rope_dweight_kernel, dim3((D + 31) / 32, of_q.rows + of_k.rows), 1024, 0,
                          stream, of_q, of_k, by_head ? heads : 2, D);
  }
  mark_after(MOE_KERNEL_QK_NORM_ROPE_BWD, stream);
  count_launches(weights ? 2 : 1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
