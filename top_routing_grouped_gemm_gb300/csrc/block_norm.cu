// The norms before and after a block with its gate, residual scale and residual sum, forward and
// backward (include/moe_block.h has the formulas).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "moe_internal.h"
#include "overlap.cuh"
#include "ptx.cuh"

#include "../../include/moe_block.h"

namespace moe {
namespace {

constexpr int kMaxD = 16384;
// Of the GPU that the cuts are made for (the workspace's size follows from them, and has to be the
// same wherever it is asked for).
constexpr int kSms = 152;

// What the forward and the backward read.
struct Block {
  int N, D;
  float eps, scale;
  int gate_kind, gate_sigmoid, post_norm;
  const void *x, *y, *gate;
  long long ld_x, ld_y, ld_gate;
  const float *w_post, *w_pre;
};

struct Grads {
  const void *dz, *dn;
  void *dx, *dy, *dgate;
  long long ld_dz, ld_dn, ld_dx, ld_dy, ld_dgate;
  float* partial;  // [blocks][3][D]: dw_pre, dw_post, dgate of a gate [D]; null: none wanted
};

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 q = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void weight8(const float* w, int at, float (&v)[8]) {
  if (w)
    load8(w + at, v);
  else
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.f;
}

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + __expf(-v)); }

// A row is held by WARPS warps, C pieces of 8 values to a lane: piece c of thread i has values
// (c * 32 * WARPS + i) * 8 on.  Rows of up to 512 values take one warp.
template <int WARPS, int C>
struct Lanes {
  static constexpr int kRowThreads = WARPS * 32;
  static constexpr int kThreads = kRowThreads > 256 ? kRowThreads : 256;
  static constexpr int kGroups = kThreads / kRowThreads;  // rows that a block has at once

  int thread, group;

  __device__ __forceinline__ Lanes()
      : thread(threadIdx.x % kRowThreads), group(threadIdx.x / kRowThreads) {}
  __device__ __forceinline__ int at(int c) const { return (c * kRowThreads + thread) * 8; }

  // Sums over the row's threads, the same in all of them.  `sums` is the group's, of the call's
  // own: three in turn are enough, as nobody is two barriers ahead.
  __device__ __forceinline__ float2 sum(float2 v, float2* sums) const {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      v.x += __shfl_xor_sync(~0u, v.x, o);
      v.y += __shfl_xor_sync(~0u, v.y, o);
    }
    if constexpr (WARPS > 1) {
      if (thread % 32 == 0) sums[thread / 32] = v;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kRowThreads) : "memory");
      v = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v.x += sums[w].x, v.y += sums[w].y;
    }
    return v;
  }
  __device__ __forceinline__ float sum(float v, float2* sums) const {
    return sum(make_float2(v, 0.f), sums).x;
  }
};

// a(gate) of 8 values; of a gate [N] the same for all.
template <typename T>
__device__ __forceinline__ void gate8(const Block& b, long long row, int at, float token,
                                      float (&a)[8]) {
  if (b.gate_kind == MOE_GATE_VALUE)
    load8(static_cast<const T*>(b.gate) + row * b.ld_gate + at, a);
  else if (b.gate_kind == MOE_GATE_CHANNEL)
    load8(static_cast<const float*>(b.gate) + at, a);
  else
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = token;
  if (b.gate_sigmoid && b.gate_kind >= MOE_GATE_CHANNEL && b.gate_kind != MOE_GATE_TOKEN)
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = sigmoid(a[e]);
}

// a(gate) of a gate [N], 1 without a gate.
__device__ __forceinline__ float token_gate(const Block& b, long long row) {
  if (b.gate_kind != MOE_GATE_TOKEN) return 1.f;
  const float g = static_cast<const float*>(b.gate)[row];
  return b.gate_sigmoid ? sigmoid(g) : g;
}

template <typename S, typename T, int WARPS, int C>
__global__ void __launch_bounds__(Lanes<WARPS, C>::kThreads)
    block_norm_kernel(const Block b, void* z_, long long ld_z, void* n_, long long ld_n) {
  using L = Lanes<WARPS, C>;
  __shared__ float2 sums[3][L::kGroups][WARPS];
  after_previous();
  const L me;
  const float inv_D = 1.f / b.D;
  const long long step = static_cast<long long>(gridDim.x) * L::kGroups;
  for (long long row = static_cast<long long>(blockIdx.x) * L::kGroups + me.group; row < b.N;
       row += step) {
    const S* x = static_cast<const S*>(b.x) + row * b.ld_x;
    const T* y = static_cast<const T*>(b.y) + row * b.ld_y;
    float z[C][8], u[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (me.at(c) < b.D) {
        load8(x + me.at(c), z[c]);
        if (b.y) load8(y + me.at(c), u[c]);
      }
    if (b.y) {
      const float token = token_gate(b, row);
      float ry = 1.f;
      if (b.post_norm) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (me.at(c) < b.D)
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(u[c][e], u[c][e], s);
        ry = rsqrtf(fmaf(me.sum(s, sums[0][me.group]), inv_D, b.eps));
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (me.at(c) < b.D) {
          float w[8], a[8];
          weight8(b.post_norm ? b.w_post : nullptr, me.at(c), w);
          gate8<T>(b, row, me.at(c), token, a);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            z[c][e] = fmaf(b.scale * a[e], w[e] * (u[c][e] * ry), z[c][e]);
        }
    }
    if (z_)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (me.at(c) < b.D) store8(static_cast<S*>(z_) + row * ld_z + me.at(c), z[c]);
    if (n_) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (me.at(c) < b.D)
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(z[c][e], z[c][e], s);
      const float rz = rsqrtf(fmaf(me.sum(s, sums[1][me.group]), inv_D, b.eps));
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (me.at(c) < b.D) {
          float w[8];
          weight8(b.w_pre, me.at(c), w);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] *= z[c][e] * rz;
          store8(static_cast<T*>(n_) + row * ld_n + me.at(c), w);
        }
    }
    // the next row's first sums go where this row's readers may still be: one more barrier's worth
    if (WARPS > 1 && !(b.y && b.post_norm && n_))
      asm volatile("bar.sync %0, %1;" ::"r"(1 + me.group), "n"(L::kRowThreads) : "memory");
  }
}

// z is formed again.  With z^ = z / rms(z) and y^ = y / rms(y),
//   dz' = dz + (w_pre dn - z^ mean(w_pre dn z^)) / rms(z) = dx
//   t   = scale a dz',   da = scale dz' u
//   dy  = (w_post t - y^ mean(w_post t y^)) / rms(y), or t
// The sums over rows (of dn z^, t y^, da) stay in shared memory, each thread's values in places of
// its own, over all rows of a block.
template <typename S, typename T, typename G, int WARPS, int C>
__global__ void __launch_bounds__(Lanes<WARPS, C>::kThreads)
    block_norm_backward_kernel(const Block b, const Grads g) {
  using L = Lanes<WARPS, C>;
  __shared__ float2 sums[3][L::kGroups][WARPS];
  extern __shared__ float acc[];  // [3][C][8][threads]
  after_previous();
  const L me;
  const float inv_D = 1.f / b.D;
  const auto place = [&](int which, int c, int e) -> float& {
    return acc[((which * C + c) * 8 + e) * L::kThreads + threadIdx.x];
  };
  if (g.partial)
    for (int i = 0; i < 3 * C * 8; ++i) acc[i * L::kThreads + threadIdx.x] = 0.f;
  const long long step = static_cast<long long>(gridDim.x) * L::kGroups;
  for (long long row = static_cast<long long>(blockIdx.x) * L::kGroups + me.group; row < b.N;
       row += step) {
    const S* x = static_cast<const S*>(b.x) + row * b.ld_x;
    const T* y = static_cast<const T*>(b.y) + row * b.ld_y;
    const S* dz_row = static_cast<const S*>(g.dz) + row * g.ld_dz;
    const G* dn_row = static_cast<const G*>(g.dn) + row * g.ld_dn;
    float z[C][8], v[C][8], dz[C][8], dn[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (me.at(c) < b.D) {
        load8(x + me.at(c), z[c]);
        if (b.y) load8(y + me.at(c), v[c]);
        if (g.dz) {
          load8(dz_row + me.at(c), dz[c]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) dz[c][e] = 0.f;
        }
        if (g.dn) load8(dn_row + me.at(c), dn[c]);
      }
    const float token = b.y ? token_gate(b, row) : 0.f;
    float ry = 1.f;
    if (b.y) {
      if (b.post_norm) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (me.at(c) < b.D)
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(v[c][e], v[c][e], s);
        ry = rsqrtf(fmaf(me.sum(s, sums[0][me.group]), inv_D, b.eps));
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (me.at(c) < b.D) {
          float w[8], a[8];
          weight8(b.post_norm ? b.w_post : nullptr, me.at(c), w);
          gate8<T>(b, row, me.at(c), token, a);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            z[c][e] = fmaf(b.scale * a[e], w[e] * (v[c][e] * ry), z[c][e]);
        }
    }
    if (g.dn) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (me.at(c) < b.D) {
          float w[8];
          weight8(b.w_pre, me.at(c), w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            s.x = fmaf(z[c][e], z[c][e], s.x);
            s.y = fmaf(w[e] * dn[c][e], z[c][e], s.y);
          }
        }
      s = me.sum(s, sums[1][me.group]);
      const float rz = rsqrtf(fmaf(s.x, inv_D, b.eps));
      const float m = s.y * inv_D * rz * rz;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (me.at(c) < b.D) {
          float w[8];
          weight8(b.w_pre, me.at(c), w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (g.partial) place(0, c, e) += dn[c][e] * (z[c][e] * rz);
            dz[c][e] += rz * fmaf(-m, z[c][e], w[e] * dn[c][e]);
          }
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (me.at(c) < b.D) store8(static_cast<S*>(g.dx) + row * g.ld_dx + me.at(c), dz[c]);
    if (!b.y) {
      if (WARPS > 1 && g.dn)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + me.group), "n"(L::kRowThreads) : "memory");
      continue;
    }
    float2 s = make_float2(0.f, 0.f);  // of w_post t y, and of dz' u
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (me.at(c) < b.D) {
        float w[8], a[8], da[8];
        weight8(b.post_norm ? b.w_post : nullptr, me.at(c), w);
        gate8<T>(b, row, me.at(c), token, a);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = b.scale * dz[c][e], u = w[e] * (v[c][e] * ry);
          da[e] = d * u;
          s.y += da[e];
          const float t = d * a[e];
          s.x = fmaf(t * w[e], v[c][e], s.x);
          if (g.partial) place(1, c, e) += t * (v[c][e] * ry);
          dz[c][e] = t * w[e];
          if (b.gate_sigmoid) da[e] *= a[e] * (1.f - a[e]);
          if (g.partial && b.gate_kind == MOE_GATE_CHANNEL) place(2, c, e) += da[e];
        }
        if (b.gate_kind == MOE_GATE_VALUE && g.dgate)
          store8(static_cast<T*>(g.dgate) + row * g.ld_dgate + me.at(c), da);
      }
    s = me.sum(s, sums[2][me.group]);
    if (b.gate_kind == MOE_GATE_TOKEN && g.dgate && me.thread == 0)
      static_cast<float*>(g.dgate)[row] = s.y * (b.gate_sigmoid ? token * (1.f - token) : 1.f);
    if (g.dy) {
      const float m = b.post_norm ? s.x * inv_D * ry * ry : 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (me.at(c) < b.D) {
          float d[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = ry * fmaf(-m, v[c][e], dz[c][e]);
          store8(static_cast<T*>(g.dy) + row * g.ld_dy + me.at(c), d);
        }
    }
    // without a sum before it the next row's could meet this one's readers
    if (WARPS > 1 && !b.post_norm && !g.dn)
      asm volatile("bar.sync %0, %1;" ::"r"(1 + me.group), "n"(L::kRowThreads) : "memory");
  }
  if (!g.partial) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 3 * b.D; i += L::kThreads) {
    const int which = i / b.D, col = i % b.D;
    const int piece = col / 8, c = piece / L::kRowThreads, thread = piece % L::kRowThreads;
    float sum = 0.f;
    for (int group = 0; group < L::kGroups; ++group)
      sum += acc[((which * C + c) * 8 + col % 8) * L::kThreads + group * L::kRowThreads + thread];
    g.partial[static_cast<long long>(blockIdx.x) * 3 * b.D + i] = sum;
  }
}

// The blocks' sums added: 32 columns to a block, whose 32 warps take every 32nd of the rows each and
// are then added in order.
__global__ void __launch_bounds__(1024)
    block_norm_sums_kernel(const float* partial, int blocks, int D, float* out0, float* out1,
                           float* out2) {
  __shared__ float sums[32][33];
  after_previous();
  float* out = blockIdx.y == 0 ? out0 : blockIdx.y == 1 ? out1 : out2;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (col < D)
#pragma unroll 4
    for (int r = warp; r < blocks; r += 32)
      sum += partial[(static_cast<long long>(r) * 3 + blockIdx.y) * D + col];
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int w = 1; w < 32; ++w) sum += sums[w][lane];
  if (col < D) out[col] = sum;
}

// ------------------------------------------------------------------------ host side

// Calls f(WARPS, C) for the warps of a row and the pieces of a lane.
template <typename F>
auto with_lanes(int D, F f) {
  using std::integral_constant;
  if (D <= 256) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (D <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (D <= 1024) return f(integral_constant<int, 2>{}, integral_constant<int, 2>{});
  if (D <= 2048) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (D <= 4096) return f(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  if (D <= 8192) return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  return f(integral_constant<int, 32>{}, integral_constant<int, 2>{});
}

// Blocks of a launch: the rows in turn over what the GPU holds at once.
template <int WARPS, int C>
int blocks_of(int N, int threads_per_sm) {
  using L = Lanes<WARPS, C>;
  const long long most = static_cast<long long>(kSms) * std::max(1, threads_per_sm / L::kThreads);
  return static_cast<int>(std::min<long long>(most, (N + L::kGroups - 1ll) / L::kGroups));
}

constexpr int kForwardThreads = 1024, kBackwardThreads = 512;  // to an SM

int backward_blocks(int N, int D) {
  return with_lanes(D, [&](auto warps, auto c) {
    return blocks_of<decltype(warps)::value, decltype(c)::value>(N, kBackwardThreads);
  });
}

size_t backward_ws(int N, int D) {
  return up256(static_cast<size_t>(backward_blocks(N, D)) * 3 * D * 4);
}

bool finite(float v) { return v == v && fabsf(v) <= 3.4028235e38f; }

// A matrix [N, D]: its stride, which of a single row means nothing.
int rows_status(const void* p, int N, int D, long long* ld, bool output) {
  if (misaligned(p, 16)) return MOE_ERR_UNSUPPORTED;
  if (N == 1) {
    *ld = D;
    return MOE_OK;
  }
  if (*ld % 8) return MOE_ERR_UNSUPPORTED;
  if (output ? *ld < D : (*ld != 0 && *ld < D)) return MOE_ERR_INVALID_ARG;
  return *ld > (1ll << 32) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

#define BLOCK_TRY(expr)                    \
  do {                                     \
    const int status_ = (expr);            \
    if (status_ != MOE_OK) return status_; \
  } while (0)

bool types_ok(int stream, int dtype) {
  return (stream == MOE_F32 && (dtype == MOE_F32 || dtype == MOE_BF16)) ||
         (stream == MOE_BF16 && dtype == MOE_BF16);
}

int block_of(const moe_block_in* in, Block* b) {
  if (!in || !in->x || in->N <= 0 || in->D <= 0) return MOE_ERR_INVALID_ARG;
  if (!(in->eps > 0.f) || !finite(in->eps) || !finite(in->scale)) return MOE_ERR_INVALID_ARG;
  if (in->gate_kind < MOE_GATE_NONE || in->gate_kind > MOE_GATE_VALUE) return MOE_ERR_INVALID_ARG;
  if ((in->gate_kind == MOE_GATE_NONE) != !in->gate) return MOE_ERR_INVALID_ARG;
  if (!in->y && (in->gate || in->post_norm)) return MOE_ERR_INVALID_ARG;
  if (in->w_post && !in->post_norm) return MOE_ERR_INVALID_ARG;
  if (in->stream_dtype < MOE_BF16 || in->stream_dtype > MOE_F32 || in->dtype < MOE_BF16 ||
      in->dtype > MOE_F32)
    return MOE_ERR_INVALID_ARG;
  if (!types_ok(in->stream_dtype, in->dtype)) return MOE_ERR_UNSUPPORTED;
  if (in->D % 8 || in->D > kMaxD || in->N > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  *b = Block{in->N, in->D, in->eps, in->scale, in->gate_kind,
             in->gate_kind != MOE_GATE_NONE && in->gate_sigmoid, in->post_norm != 0, in->x, in->y,
             in->gate, in->ld_x, in->ld_y, in->ld_gate, in->w_post, in->w_pre};
  BLOCK_TRY(rows_status(in->x, in->N, in->D, &b->ld_x, false));
  if (in->y) BLOCK_TRY(rows_status(in->y, in->N, in->D, &b->ld_y, false));
  if (in->gate_kind == MOE_GATE_VALUE)
    BLOCK_TRY(rows_status(in->gate, in->N, in->D, &b->ld_gate, false));
  if (misaligned(in->gate, in->gate_kind == MOE_GATE_TOKEN ? 4 : 16) ||
      misaligned(in->w_post, 16) || misaligned(in->w_pre, 16))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Calls f(S, T) with values of the types of the stream and of the blocks.
template <typename F>
void with_types(int stream, int dtype, F f) {
  if (stream == MOE_BF16)
    f(__nv_bfloat16{}, __nv_bfloat16{});
  else if (dtype == MOE_BF16)
    f(float{}, __nv_bfloat16{});
  else
    f(float{}, float{});
}

}  // namespace
}  // namespace moe

extern "C" {

using namespace moe;

int moe_block_norm(const moe_block_in* in, void* z, int64_t ld_z, void* n, int64_t ld_n,
                   moe_stream_t stream) {
  Block b{};
  BLOCK_TRY(block_of(in, &b));
  if ((!z && (b.y || !n)) || (!n && b.w_pre)) return MOE_ERR_INVALID_ARG;
  long long lz = ld_z, ln = ld_n;
  if (z) BLOCK_TRY(rows_status(z, b.N, b.D, &lz, true));
  if (n) BLOCK_TRY(rows_status(n, b.N, b.D, &ln, true));
  mark_before(MOE_KERNEL_BLOCK_NORM, stream);
  cudaError_t err = cudaSuccess;
  with_types(in->stream_dtype, in->dtype, [&](auto s, auto t) {
    with_lanes(b.D, [&](auto warps, auto c) {
      constexpr int W = decltype(warps)::value, C = decltype(c)::value;
      err = launch_behind(block_norm_kernel<decltype(s), decltype(t), W, C>,
                          blocks_of<W, C>(b.N, kForwardThreads), Lanes<W, C>::kThreads, 0, stream,
                          b, z, lz, n, ln);
    });
  });
  mark_after(MOE_KERNEL_BLOCK_NORM, stream);
  count_launches(1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_block_norm_backward_workspace_size(int32_t N, int32_t D, int32_t gate_kind) {
  if (N <= 0 || N > (1 << 30) || D <= 0 || D > kMaxD || D % 8 || gate_kind < MOE_GATE_NONE ||
      gate_kind > MOE_GATE_VALUE)
    return 0;
  return backward_ws(N, D);
}

int moe_block_norm_backward(const moe_block_in* in, const moe_block_grads* grads,
                            void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  Block b{};
  BLOCK_TRY(block_of(in, &b));
  const moe_block_grads* r = grads;
  if (!r || !r->dx || (!r->dz && !r->dn)) return MOE_ERR_INVALID_ARG;
  if (!b.y && (r->dy || r->dgate || r->dw_post)) return MOE_ERR_INVALID_ARG;
  if ((r->dgate && !b.gate) || (r->dw_post && !b.post_norm)) return MOE_ERR_INVALID_ARG;
  if (r->dn && r->dn_dtype != MOE_F32 && r->dn_dtype != in->dtype) return MOE_ERR_INVALID_ARG;
  Grads g{r->dz, r->dn, r->dx, r->dy, r->dgate, r->ld_dz, r->ld_dn, r->ld_dx, r->ld_dy,
          r->ld_dgate, nullptr};
  if (r->dz) BLOCK_TRY(rows_status(r->dz, b.N, b.D, &g.ld_dz, false));
  if (r->dn) BLOCK_TRY(rows_status(r->dn, b.N, b.D, &g.ld_dn, false));
  BLOCK_TRY(rows_status(r->dx, b.N, b.D, &g.ld_dx, true));
  if (r->dy) BLOCK_TRY(rows_status(r->dy, b.N, b.D, &g.ld_dy, true));
  if (r->dgate && b.gate_kind == MOE_GATE_VALUE)
    BLOCK_TRY(rows_status(r->dgate, b.N, b.D, &g.ld_dgate, true));
  if (misaligned(r->dgate, 4) || misaligned(r->dw_post, 4) || misaligned(r->dw_pre, 4))
    return MOE_ERR_UNSUPPORTED;
  const bool channel = r->dgate && b.gate_kind == MOE_GATE_CHANNEL;
  const bool partial = r->dw_pre || r->dw_post || channel;
  if (partial) {
    if (!workspace || workspace_bytes < backward_ws(b.N, b.D)) return MOE_ERR_WORKSPACE;
    if (misaligned(workspace, 16)) return MOE_ERR_UNSUPPORTED;
    g.partial = static_cast<float*>(workspace);
  }
  const int blocks = backward_blocks(b.N, b.D);
  mark_before(MOE_KERNEL_BLOCK_NORM_BWD, stream);
  cudaError_t err = cudaSuccess;
  with_types(in->stream_dtype, in->dtype, [&](auto s, auto t) {
    with_lanes(b.D, [&](auto warps, auto c) {
      constexpr int W = decltype(warps)::value, C = decltype(c)::value;
      using S = decltype(s);
      using T = decltype(t);
      const int threads = Lanes<W, C>::kThreads, smem = partial ? 3 * C * 8 * threads * 4 : 0;
      const auto launch = [&](auto kernel) {
        err = launched(cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * C * 8 * threads * 4));
        if (err == cudaSuccess) err = launch_behind(kernel, blocks, threads, smem, stream, b, g);
      };
      if (std::is_same<T, float>::value || r->dn_dtype == MOE_F32)
        launch(block_norm_backward_kernel<S, T, float, W, C>);
      else
        launch(block_norm_backward_kernel<S, T, T, W, C>);
    });
  });
  if (partial && err == cudaSuccess)
    err = launch_behind(block_norm_sums_kernel, dim3((b.D + 31) / 32, 3), 1024, 0, stream,
                        g.partial, blocks, b.D, r->dw_pre, r->dw_post,
                        channel ? static_cast<float*>(r->dgate) : nullptr);
  mark_after(MOE_KERNEL_BLOCK_NORM_BWD, stream);
  count_launches(partial ? 2 : 1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
