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
  float* partial;  // [blocks][2][D]: sums of the blocks' rows; null: none wanted
};

// V neighbouring values: 8, or 4 where the residual stream is fp32, so that 16 bytes of it follow 16
// bytes of the next lane (8 values to a lane, in two pieces 32 bytes apart, leave half of every
// 32-byte sector to another instruction: 8192 x 4096 forward 86 us at 4.0 TB/s).
__device__ __forceinline__ void unpack(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xffff0000u);
}
template <int V>
__device__ __forceinline__ void load(const float* p, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float4 q = reinterpret_cast<const float4*>(p)[i / 4];
    v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
  }
}
template <int V>
__device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const uint2 q = reinterpret_cast<const uint2*>(p)[i / 4];
    unpack(q.x, v[i], v[i + 1]);
    unpack(q.y, v[i + 2], v[i + 3]);
  }
}
template <int V>
__device__ __forceinline__ void store(float* p, const float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4)
    reinterpret_cast<float4*>(p)[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int V>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[V]) {
  if constexpr (V == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// 1 / (1 + exp(-v)): the hardware's reciprocal and one step of Newton's, which leaves the last rounding
// (and no branch, which a division has for what does not occur here).
__device__ __forceinline__ float sigmoid(float v) {
  const float x = 1.f + expf(-v);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return x < 1e38f ? fmaf(r, fmaf(-x, r, 1.f), r) : r;  // (infinite: 0)
}

// A row is held by WARPS warps, C pieces of V values to a lane: piece c of thread i has values
// (c * 32 * WARPS + i) * V on.  Rows of up to 512 values take one warp.
// FULL: the rows have just as many, and no piece is beyond their end.
template <int WARPS, int C, int V, bool FULL>
struct Lanes {
  static constexpr int kRowThreads = WARPS * 32, kPieces = C, kValues = V;
  static constexpr bool kFull = FULL;
  static constexpr int kThreads = kRowThreads > 256 ? kRowThreads : 256;
  static constexpr int kGroups = kThreads / kRowThreads;  // rows that a block has at once

  int thread, group;

  __device__ __forceinline__ Lanes()
      : thread(threadIdx.x % kRowThreads), group(threadIdx.x / kRowThreads) {}
  __device__ __forceinline__ int at(int c) const { return (c * kRowThreads + thread) * V; }
  __device__ __forceinline__ bool in(int c, int D) const { return FULL || at(c) < D; }

  // Sums over the row's threads, the same in all of them.  `sums` is the group's, of the call's
  // own: three in turn are enough, as nobody is two barriers ahead.
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N], float (*sums)[WARPS]) const {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(~0u, v[i], o);
    if constexpr (WARPS > 1) {
      if (thread % 32 == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) sums[i][thread / 32] = v[i];
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kRowThreads) : "memory");
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v[i] += sums[i][w];
      }
    }
  }
  __device__ __forceinline__ float sum(float v, float (*sums)[WARPS]) const {
    float one[1] = {v};
    sum(one, sums);
    return one[0];
  }
};

// Rows on their way: every thread copies the 16-byte pieces that it will read itself into places of
// its own in shared memory, some rows ahead, so that nothing but its own wait stands between.
// (Loaded when they were wanted, 2 blocks of 256 threads to an SM had too few bytes under way:
// 16384 x 4096 bf16 169 us.)  V values of type X take V * sizeof(X) bytes of each of THREADS threads,
// in pieces of 8 or 16 bytes; piece i of all threads follows piece i - 1 of all.
template <int THREADS, int V, typename X>
struct Piece {
  static constexpr int kBytes = V * sizeof(X) < 16 ? 8 : 16, kCount = V * sizeof(X) / kBytes;
  static constexpr int kAll = THREADS * V * sizeof(X);  // bytes of a piece of V values of all threads

  static __device__ __forceinline__ void copy(uint32_t to, const X* from) {
    to += threadIdx.x * kBytes;
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const X* at = from + i * (V / kCount);
      if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * (THREADS * 16)), "l"(at)
                     : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(at) : "memory");
    }
  }
  static __device__ __forceinline__ void read(uint32_t from, float (&v)[V]) {
    from += threadIdx.x * kBytes;
    uint32_t w[V * sizeof(X) / 4];
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      uint32_t(&q)[V * sizeof(X) / 4] = w;
      if constexpr (kBytes == 16)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q[4 * i]), "=r"(q[4 * i + 1]), "=r"(q[4 * i + 2]), "=r"(q[4 * i + 3])
                     : "r"(from + i * (THREADS * 16))
                     : "memory");
      else
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q[0]), "=r"(q[1]) : "r"(from) : "memory");
    }
#pragma unroll
    for (int i = 0; i < static_cast<int>(V * sizeof(X) / 4); ++i)
      if constexpr (sizeof(X) == 4)
        v[i] = __uint_as_float(w[i]);
      else
        unpack(w[i], v[2 * i], v[2 * i + 1]);
  }
};
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void wait_for_copies(int but) {
  if (but == 3)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (but == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (but == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Where the pieces of a row are, in bytes: x, y, a gate [N, D], then dz and dn.
template <typename S, typename T, typename G, int THREADS, int C, int V, bool BACKWARD>
struct Places {
  static constexpr int kS = Piece<THREADS, V, S>::kAll, kT = Piece<THREADS, V, T>::kAll;
  static constexpr int kG = Piece<THREADS, V, G>::kAll;
  static constexpr int kY = C * kS, kGate = kY + C * kT;
  static constexpr int dz(bool gates) { return kGate + (gates ? C * kT : 0); }
  static constexpr int dn(bool gates) { return dz(gates) + (BACKWARD ? C * kS : 0); }
  static constexpr int all(bool gates) { return dn(gates) + (BACKWARD ? C * kG : 0); }
};

// a(gate) of a gate [N], 1 without a gate.
__device__ __forceinline__ float token_gate(const Block& b, long long row) {
  if (b.gate_kind != MOE_GATE_TOKEN) return 1.f;
  const float g = static_cast<const float*>(b.gate)[row];
  return b.gate_sigmoid ? sigmoid(g) : g;
}

// Rows of more than 8192 values are read where they are, again for each time that they are wanted.
template <int WARPS>
constexpr bool kDirect = WARPS == 32;

// A row in shared memory (or, kDirect, in its matrices), as one thread sees it.
template <typename S, typename T, typename G, int WARPS, int C, int V, bool FULL, bool BACKWARD>
struct Row {
  using L = Lanes<WARPS, C, V, FULL>;
  using P = Places<S, T, G, L::kThreads, C, V, BACKWARD>;
  uint32_t at;
  long long r;
  int first, gates;  // the thread's first column

  __device__ __forceinline__ int col(int c) const { return first + c * (L::kRowThreads * V); }
  template <typename X>
  __device__ __forceinline__ void get(int place, const void* p, long long ld, int c,
                                      float (&v)[V]) const {
    if constexpr (kDirect<WARPS>)
      load(static_cast<const X*>(p) + r * ld + col(c), v);
    else
      Piece<L::kThreads, V, X>::read(at + place + c * Piece<L::kThreads, V, X>::kAll, v);
  }
  template <typename X>
  __device__ __forceinline__ void put(int place, const void* p, long long ld, int c) const {
    Piece<L::kThreads, V, X>::copy(at + place + c * Piece<L::kThreads, V, X>::kAll,
                                   static_cast<const X*>(p) + r * ld + col(c));
  }
  __device__ __forceinline__ void x(const Block& b, int c, float (&v)[V]) const {
    get<S>(0, b.x, b.ld_x, c, v);
  }
  __device__ __forceinline__ void y(const Block& b, int c, float (&v)[V]) const {
    get<T>(P::kY, b.y, b.ld_y, c, v);
  }
  __device__ __forceinline__ void dz(const Grads& g, int c, float (&v)[V]) const {
    get<S>(P::dz(gates), g.dz, g.ld_dz, c, v);
  }
  __device__ __forceinline__ void dn(const Grads& g, int c, float (&v)[V]) const {
    get<G>(P::dn(gates), g.dn, g.ld_dn, c, v);
  }
  // a(gate) of a gate [N, D].
  __device__ __forceinline__ void gate(const Block& b, int c, float (&a)[V]) const {
    get<T>(P::kGate, b.gate, b.ld_gate, c, a);
    if (b.gate_sigmoid)
#pragma unroll
      for (int e = 0; e < V; ++e) a[e] = sigmoid(a[e]);
  }
  __device__ __forceinline__ void copy_block(const Block& b) const {
    if constexpr (kDirect<WARPS>) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!FULL && col(c) >= b.D) continue;
      put<S>(0, b.x, b.ld_x, c);
      if (b.y) put<T>(P::kY, b.y, b.ld_y, c);
      if (gates) put<T>(P::kGate, b.gate, b.ld_gate, c);
    }
  }
  __device__ __forceinline__ void copy_grads(const Block& b, const Grads& g) const {
    if constexpr (kDirect<WARPS>) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!FULL && col(c) >= b.D) continue;
      if (g.dz) put<S>(P::dz(gates), g.dz, g.ld_dz, c);
      if (g.dn) put<G>(P::dn(gates), g.dn, g.ld_dn, c);
    }
  }
};

// What the thread's columns have in all rows: scale w_post a (of a gate [D]), and w_pre.
template <int WARPS, int C, int V, bool FULL>
struct Columns {
  float post[C][V], pre[C][V];
  __device__ __forceinline__ Columns(const Block& b, const Lanes<WARPS, C, V, FULL>& me) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int e = 0; e < V; ++e) post[c][e] = b.scale, pre[c][e] = 1.f;
      if (!me.in(c, b.D)) continue;
      float a[V];
      if (b.w_post) times(static_cast<const float*>(b.w_post), me.at(c), post[c]);
      if (b.gate_kind == MOE_GATE_CHANNEL) {
        load(static_cast<const float*>(b.gate) + me.at(c), a);
#pragma unroll
        for (int e = 0; e < V; ++e) post[c][e] *= b.gate_sigmoid ? sigmoid(a[e]) : a[e];
      }
      if (b.w_pre) times(static_cast<const float*>(b.w_pre), me.at(c), pre[c]);
    }
  }
  static __device__ __forceinline__ void times(const float* w, int at, float (&v)[V]) {
    float f[V];
    load(w + at, f);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] *= f[e];
  }
};

// The weights of the thread's columns stay in registers over the block's rows, and everything that
// is one number for a row is multiplied together first: two fused products to a value of z, and one
// product less for the norms than for weights and factors one by one (515 instructions for a warp's
// part of a row of 4096 then).  8192 x 4096, an fp32 stream with bf16 values: 73 us (402 MB: 59 at the
// rate of a copy); 16384 x 4096 in bf16 95 us (79): blocks wait for a row's sum and its memory in turn.
template <typename S, typename T, int WARPS, int C, int V, bool FULL>
__global__ void __launch_bounds__(Lanes<WARPS, C, V, FULL>::kThreads,
                                  Lanes<WARPS, C, V, FULL>::kThreads > 256 ? 1 : 2)
    block_norm_kernel(const Block b, void* z_, long long ld_z, void* n_, long long ld_n, int ahead) {
  using L = Lanes<WARPS, C, V, FULL>;
  using R = Row<S, T, T, WARPS, C, V, FULL, false>;
  __shared__ float sums[2][L::kGroups][1][WARPS];
  extern __shared__ __align__(16) uint8_t shared[];
  after_previous();
  const L me;
  const int gates = b.gate_kind == MOE_GATE_VALUE;
  const uint32_t ring = smem_u32(shared);
  const int row_bytes = R::P::all(gates);
  const float inv_D = 1.f / b.D;
  const long long step = static_cast<long long>(gridDim.x) * L::kGroups;
  const long long first = static_cast<long long>(blockIdx.x) * L::kGroups + me.group;
  for (int i = 0; i < ahead; ++i) {
    if (first + i * step < b.N) {
      const R row{ring + i * row_bytes, first + i * step, me.at(0), gates};
      row.copy_block(b);
    }
    commit_copies();
  }
  const Columns<WARPS, C, V, FULL> columns(b, me);
  int now = 0, next = ahead;
  for (long long r = first; r < b.N; r += step) {
    if (r + ahead * step < b.N) {
      const R coming{ring + next * row_bytes, r + ahead * step, me.at(0), gates};
      coming.copy_block(b);
    }
    commit_copies();
    const float token = b.y ? token_gate(b, r) : 0.f;
    wait_for_copies(ahead);
    const R row{ring + now * row_bytes, r, me.at(0), gates};
    if (++now > ahead) now = 0;
    if (++next > ahead) next = 0;
    float z[C][V], y[C][V];
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (me.in(c, b.D)) {
        row.x(b, c, z[c]);
        if (b.y) {
          row.y(b, c, y[c]);
#pragma unroll
          for (int e = 0; e < V; ++e) s = fmaf(y[c][e], y[c][e], s);
        }
      }
    if (b.y) {
      float by = token;
      if (b.post_norm) by *= rsqrtf(fmaf(me.sum(s, sums[0][me.group]), inv_D, b.eps));
      s = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (me.in(c, b.D)) {
#pragma unroll
          for (int e = 0; e < V; ++e) y[c][e] *= by;
          if (gates) {
            float a[V];
            row.gate(b, c, a);
#pragma unroll
            for (int e = 0; e < V; ++e) y[c][e] *= a[e];
          }
#pragma unroll
          for (int e = 0; e < V; ++e) z[c][e] = fmaf(columns.post[c][e], y[c][e], z[c][e]);
        }
    }
    s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (me.in(c, b.D)) {
        if (z_) store(static_cast<S*>(z_) + r * ld_z + me.at(c), z[c]);
#pragma unroll
        for (int e = 0; e < V; ++e) s = fmaf(z[c][e], z[c][e], s);
      }
    if (n_) {
      const float rz = rsqrtf(fmaf(me.sum(s, sums[1][me.group]), inv_D, b.eps));
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (me.in(c, b.D)) {
#pragma unroll
          for (int e = 0; e < V; ++e) z[c][e] *= rz * columns.pre[c][e];
          store(static_cast<T*>(n_) + r * ld_n + me.at(c), z[c]);
        }
    }
    // the next row's first sums go where this row's readers may still be: one more barrier's worth
    if (WARPS > 1 && !(b.y && b.post_norm && n_))
      asm volatile("bar.sync %0, %1;" ::"r"(1 + me.group), "n"(L::kRowThreads) : "memory");
  }
}

// z is formed again.  With z^ = z / rms(z), y^ = y / rms(y), p = scale w_post a (of a gate [D]) and a
// gate [N]'s a apart,
//   dz' = dz + (w_pre dn - z^ mean(w_pre dn z^)) / rms(z) = dx
//   dy  = (a p dz' - y^ mean(a p dz' y^)) / rms(y), or a p dz'
// and with Q = sum over rows of a dz' y^, what the gradients of w_post and of a gate [D] are made of
// (scale a Q and scale w_post a' Q), and sum(p dz' y^) the gradient of a gate [N] before a'.  The sums
// over rows stay in registers over all rows of a block.  8192 x 4096 as above 127 us (604 MB: 89).
template <typename S, typename T, typename G, int WARPS, int C, int V, bool FULL>
__global__ void __launch_bounds__(Lanes<WARPS, C, V, FULL>::kThreads,
                                  Lanes<WARPS, C, V, FULL>::kThreads > 256 ? 1 : 2)
    block_norm_backward_kernel(const Block b, const Grads g, int ahead) {
  using L = Lanes<WARPS, C, V, FULL>;
  using R = Row<S, T, G, WARPS, C, V, FULL, true>;
  __shared__ float sums[3][L::kGroups][2][WARPS];
  extern __shared__ __align__(16) uint8_t shared[];
  after_previous();
  const L me;
  const int gates = b.gate_kind == MOE_GATE_VALUE;
  const uint32_t ring = smem_u32(shared);
  const int row_bytes = R::P::all(gates);
  const float inv_D = 1.f / b.D;
  const long long step = static_cast<long long>(gridDim.x) * L::kGroups;
  const long long first = static_cast<long long>(blockIdx.x) * L::kGroups + me.group;
  for (int i = 0; i < ahead; ++i) {
    if (first + i * step < b.N) {
      const R row{ring + i * row_bytes, first + i * step, me.at(0), gates};
      row.copy_block(b);
      row.copy_grads(b, g);
    }
    commit_copies();
  }
  const Columns<WARPS, C, V, FULL> columns(b, me);
  float of_pre[C][V] = {}, of_post[C][V] = {};  // sums of dn z^, and Q
  int now = 0, next = ahead;
  for (long long r = first; r < b.N; r += step) {
    if (r + ahead * step < b.N) {
      const R coming{ring + next * row_bytes, r + ahead * step, me.at(0), gates};
      coming.copy_block(b);
      coming.copy_grads(b, g);
    }
    commit_copies();
    const float token = b.y ? token_gate(b, r) : 0.f;
    wait_for_copies(ahead);
    const R row{ring + now * row_bytes, r, me.at(0), gates};
    if (++now > ahead) now = 0;
    if (++next > ahead) next = 0;
    float ry = 1.f;
    if (b.y && b.post_norm) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (me.in(c, b.D)) {
          float y[V];
          row.y(b, c, y);
#pragma unroll
          for (int e = 0; e < V; ++e) s = fmaf(y[e], y[e], s);
        }
      ry = rsqrtf(fmaf(me.sum(s, sums[0][me.group]), inv_D, b.eps));
    }
    const float by = ry * token;
    float z[C][V];
    float s[2] = {0.f, 0.f};  // of z z, and of w_pre dn z
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (me.in(c, b.D)) {
        row.x(b, c, z[c]);
        if (b.y) {
          float y[V];
          row.y(b, c, y);
#pragma unroll
          for (int e = 0; e < V; ++e) y[e] *= by;
          if (gates) {
            float a[V];
            row.gate(b, c, a);
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] *= a[e];
          }
#pragma unroll
          for (int e = 0; e < V; ++e) z[c][e] = fmaf(columns.post[c][e], y[e], z[c][e]);
        }
        if (g.dn) {
          float dn[V];
          row.dn(g, c, dn);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            s[0] = fmaf(z[c][e], z[c][e], s[0]);
            s[1] = fmaf(columns.pre[c][e] * dn[e], z[c][e], s[1]);
          }
        }
      }
    float rz = 0.f, m = 0.f;
    if (g.dn) {
      me.sum(s, sums[1][me.group]);
      rz = rsqrtf(fmaf(s[0], inv_D, b.eps));
      m = s[1] * inv_D * rz * rz * rz;
    }
    float sum = 0.f;  // of p dz' y (with a gate [N, D]'s a)
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (me.in(c, b.D)) {
        float dz[V];
        if (g.dz) {
          row.dz(g, c, dz);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) dz[e] = 0.f;
        }
        if (g.dn) {
          float dn[V];
          row.dn(g, c, dn);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            of_pre[c][e] = fmaf(dn[e] * rz, z[c][e], of_pre[c][e]);
            dz[e] = fmaf(columns.pre[c][e] * dn[e], rz, fmaf(-m, z[c][e], dz[e]));
          }
        }
        store(static_cast<S*>(g.dx) + r * g.ld_dx + me.at(c), dz);
        if (!b.y) continue;
        float y[V];
        row.y(b, c, y);
        if (gates) {
          float a[V], da[V];
          row.gate(b, c, a);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            da[e] = columns.post[c][e] * dz[e] * (y[e] * ry);
            if (b.gate_sigmoid) da[e] *= a[e] * (1.f - a[e]);
            dz[e] *= a[e];
          }
          if (g.dgate) store(static_cast<T*>(g.dgate) + r * g.ld_dgate + me.at(c), da);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          of_post[c][e] = fmaf(dz[e], y[e] * by, of_post[c][e]);
          z[c][e] = columns.post[c][e] * dz[e];  // what dy is made of
          sum = fmaf(z[c][e], y[e], sum);
        }
      }
    if (b.y) {
      sum = me.sum(sum, sums[2][me.group]);
      if (b.gate_kind == MOE_GATE_TOKEN && g.dgate && me.thread == 0)
        static_cast<float*>(g.dgate)[r] = sum * ry * (b.gate_sigmoid ? token * (1.f - token) : 1.f);
      if (g.dy) {
        const float my = b.post_norm ? sum * token * inv_D * ry * ry * ry : 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (me.in(c, b.D)) {
            float y[V];
            row.y(b, c, y);
#pragma unroll
            for (int e = 0; e < V; ++e) z[c][e] = fmaf(by, z[c][e], -my * y[e]);
            store(static_cast<T*>(g.dy) + r * g.ld_dy + me.at(c), z[c]);
          }
      }
    }
    // with one sum to a row the next one's could meet this one's readers
    if (WARPS > 1 && (!b.y || (!b.post_norm && !g.dn)))
      asm volatile("bar.sync %0, %1;" ::"r"(1 + me.group), "n"(L::kRowThreads) : "memory");
  }
  if (!g.partial) return;
  // The row groups' sums, added in their order.
  wait_for_copies(0);
  __syncthreads();
  float* all = reinterpret_cast<float*>(shared);  // [groups][values of a row's places] of one of both
  constexpr int kValues = C * L::kRowThreads * V;
  float* to = g.partial + static_cast<long long>(blockIdx.x) * 2 * b.D;
  if (L::kGroups == 1) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (me.in(c, b.D)) {
        store(to + me.at(c), of_pre[c]);
        store(to + b.D + me.at(c), of_post[c]);
      }
    return;
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      store(all + me.group * kValues + me.at(c), which ? of_post[c] : of_pre[c]);
    __syncthreads();
    for (int i = threadIdx.x; i < b.D; i += L::kThreads) {
      float sum = 0.f;
#pragma unroll
      for (int group = 0; group < L::kGroups; ++group) sum += all[group * kValues + i];
      to[which * b.D + i] = sum;
    }
    __syncthreads();
  }
}

// The blocks' sums added, 64 columns to a block, whose 32 warps take every 32nd of the rows each and
// are then added in order; y = 1: Q, of which the gradients of w_post and of a gate [D] are made.
__global__ void __launch_bounds__(1024)
    block_norm_sums_kernel(const Block b, const float* partial, int blocks, float* dw_pre,
                           float* dw_post, float* dgate) {
  __shared__ float2 sums[32][32];
  after_previous();
  if (blockIdx.y == 0 ? !dw_pre : !dw_post && !dgate) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 64 + lane * 2;
  float2 sum = make_float2(0.f, 0.f);
  if (col < b.D)
    for (int r0 = warp; r0 < blocks; r0 += 320) {  // ten rows on their way at once
      float2 v[10];
#pragma unroll
      for (int i = 0; i < 10; ++i) {
        v[i] = make_float2(0.f, 0.f);
        const int r = r0 + i * 32;
        if (r < blocks)
          v[i] = *reinterpret_cast<const float2*>(
              partial + (static_cast<long long>(r) * 2 + blockIdx.y) * b.D + col);
      }
#pragma unroll
      for (int i = 0; i < 10; ++i) sum.x += v[i].x, sum.y += v[i].y;
    }
  sums[warp][lane] = sum;
  __syncthreads();
  if (warp || col >= b.D) return;
#pragma unroll
  for (int w = 1; w < 32; ++w) sum.x += sums[w][lane].x, sum.y += sums[w][lane].y;
  const float q[2] = {sum.x, sum.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (blockIdx.y == 0) {
      dw_pre[col + i] = q[i];
      continue;
    }
    float a = 1.f, da = 1.f;
    if (b.gate_kind == MOE_GATE_CHANNEL) {
      a = static_cast<const float*>(b.gate)[col + i];
      if (b.gate_sigmoid) a = sigmoid(a), da = a * (1.f - a);
    }
    if (dgate) dgate[col + i] = b.scale * (b.w_post ? b.w_post[col + i] : 1.f) * da * q[i];
    if (dw_post) dw_post[col + i] = b.scale * a * q[i];
  }
}

// ------------------------------------------------------------------------ host side

template <typename P>
using LanesOf = std::remove_pointer_t<typename P::value_type>;

// Calls f(a Lanes) for rows of D values, V to a piece.
template <int V, typename F>
auto with_lanes(int D, F f) {
  const auto with = [&](auto warps, auto eights) {
    constexpr int W = decltype(warps)::value, E = decltype(eights)::value;
    return D == W * 32 * E * 8 ? f(std::integral_constant<Lanes<W, E * 8 / V, V, true>*, nullptr>{})
                               : f(std::integral_constant<Lanes<W, E * 8 / V, V, false>*, nullptr>{});
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  if (D <= 256) return with(one, one);
  if (D <= 512) return with(one, two);
  if (D <= 1024) return with(two, two);
  if (D <= 2048) return with(std::integral_constant<int, 4>{}, two);
  if (D <= 4096) return with(std::integral_constant<int, 8>{}, two);
  // (6554 rows of 4104, 5120 and 6144 forward and back, an fp32 stream: 264, 292 and 299 us; by 16 warps,
  // of whose lanes up to half have nothing, 295, 310 and 340)
  if (D <= 6144) return with(std::integral_constant<int, 12>{}, two);
  if (D <= 8192) return with(std::integral_constant<int, 16>{}, two);
  return with(std::integral_constant<int, 32>{}, two);
}

// Blocks of a launch: the rows in turn over what the GPU holds at once.
int blocks_of(int N, int groups, int per_sm) {
  return static_cast<int>(
      std::min<long long>(static_cast<long long>(kSms) * per_sm, (N + groups - 1ll) / groups));
}

constexpr int kSharedPerSm = 228 * 1024;

// Rows under way beside the one at work, and the shared memory of a block for them.
struct Ahead {
  int rows, bytes;
};
// At most `most`, and so many that `blocks` of them fit an SM, or one if not even two rows do.
template <int WARPS>
Ahead ahead_of(int row_bytes, int most, int blocks) {
  if (kDirect<WARPS>) return {0, 0};
  int rows = most;
  while (rows > 1 && (row_bytes * (rows + 1) + 2048) * blocks > kSharedPerSm) --rows;
  while (rows && row_bytes * (rows + 1) > 224 * 1024) --rows;
  return {rows, row_bytes * (rows + 1)};
}

// Three rows at most, of places P with a gate [N, D] or without.
template <typename L, typename P>
Ahead ahead_with(bool gates) {
  return ahead_of<L::kRowThreads / 32>(P::all(gates), 3, L::kThreads > 256 ? 1 : 2);
}

// How much shared memory a kernel may be launched with.  That is the kernel's, for all threads of the
// process: what any call wants, so that no call takes it down while another one is about to launch.
template <typename L, typename P>
cudaError_t allow_shared(const void* kernel) {
  return launched(
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           std::max(ahead_with<L, P>(false).bytes, ahead_with<L, P>(true).bytes)));
}

// (The backward's blocks write partial sums, so their number is the same for all types.)
int backward_blocks(int N, int D) {
  return with_lanes<8>(D, [&](auto lanes) {
    using L = LanesOf<decltype(lanes)>;
    return blocks_of(N, L::kGroups, L::kThreads > 256 ? 1 : 2);
  });
}

size_t backward_ws(int N, int D) {
  return up256(static_cast<size_t>(backward_blocks(N, D)) * 2 * D * 4);
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
    using S = decltype(s);
    using T = decltype(t);
    with_lanes<sizeof(S) == 4 ? 4 : 8>(b.D, [&](auto lanes) {
      using L = LanesOf<decltype(lanes)>;
      constexpr int W = L::kRowThreads / 32, C = L::kPieces, V = L::kValues, threads = L::kThreads;
      constexpr bool FULL = L::kFull;
      using P = Places<S, T, T, threads, C, V, false>;
      const Ahead ahead = ahead_with<L, P>(b.gate_kind == MOE_GATE_VALUE);
      const int blocks = threads > 256 ? 1 : std::max(1, std::min(2, kSharedPerSm / (ahead.bytes + 2048)));
      const auto kernel = block_norm_kernel<S, T, W, C, V, FULL>;
      err = allow_shared<L, P>(reinterpret_cast<const void*>(kernel));
      if (err == cudaSuccess)
        err = launch_behind(kernel, blocks_of(b.N, L::kGroups, blocks), threads, ahead.bytes, stream, b,
                            z, lz, n, ln, ahead.rows);
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
    using S = decltype(s);
    using T = decltype(t);
    with_lanes<sizeof(S) == 4 ? 4 : 8>(b.D, [&](auto lanes) {
      using L = LanesOf<decltype(lanes)>;
      constexpr int W = L::kRowThreads / 32, C = L::kPieces, V = L::kValues, threads = L::kThreads;
      constexpr bool FULL = L::kFull;
      const auto launch = [&](auto kernel, auto dn) {
        using P = Places<S, T, decltype(dn), threads, C, V, true>;
        const Ahead ahead = ahead_with<L, P>(b.gate_kind == MOE_GATE_VALUE);
        err = allow_shared<L, P>(reinterpret_cast<const void*>(kernel));
        if (err == cudaSuccess)
          err = launch_behind(kernel, blocks, threads, ahead.bytes, stream, b, g, ahead.rows);
      };
      if (std::is_same<T, float>::value || r->dn_dtype == MOE_F32)
        launch(block_norm_backward_kernel<S, T, float, W, C, V, FULL>, float{});
      else
        launch(block_norm_backward_kernel<S, T, T, W, C, V, FULL>, T{});
    });
  });
  if (partial && err == cudaSuccess)
    err = launch_behind(block_norm_sums_kernel, dim3((b.D + 63) / 64, 2), 1024, 0, stream, b, g.partial,
                        blocks, r->dw_pre, r->dw_post,
                        channel ? static_cast<float*>(r->dgate) : nullptr);
  mark_after(MOE_KERNEL_BLOCK_NORM_BWD, stream);
  count_launches(partial ? 2 : 1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
