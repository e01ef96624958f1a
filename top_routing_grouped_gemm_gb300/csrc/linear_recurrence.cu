// Gated linear recurrence over packed sequences, forward, backward and one token
// (include/linear_recurrence.h has the formulas).
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "moe_internal.h"
#include "ptx.cuh"
#include "slots.cuh"

#include "../../include/linear_recurrence.h"

namespace moe {
namespace {

constexpr int kChunk = 64;      // rows between the kept states
constexpr int kWarps = 8;       // warps of a scan block
constexpr int kMaxCluster = 8;  // blocks of a cluster (the portable limit)

__device__ __forceinline__ float ld(const float* p, long long i) { return p[i]; }
__device__ __forceinline__ float ld(const __nv_bfloat16* p, long long i) {
  return __bfloat162float(p[i]);
}
__device__ __forceinline__ void st(float* p, long long i, float v) { p[i] = v; }
__device__ __forceinline__ void st(__nv_bfloat16* p, long long i, float v) {
  p[i] = __float2bfloat16_rn(v);
}

// ------------------------------------------------------------------ what a lane moves at once
//
// CH channels of one row: two bf16 (4 bytes), one bf16 (rows that are not 4-byte aligned) or
// one fp32; a warp covers 32 CH neighbouring channels.
template <typename T, int CH>
struct Piece;

template <>
struct Piece<float, 1> {
  float bits;
  __device__ __forceinline__ void load(const float* p) { bits = __ldcs(p); }
  __device__ __forceinline__ void clear() { bits = 0.f; }
  __device__ __forceinline__ float get(int) const { return bits; }
  static __device__ __forceinline__ void store(float* p, const float (&v)[1]) { __stcs(p, v[0]); }
};

template <>
struct Piece<__nv_bfloat16, 1> {
  unsigned short bits;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    bits = __ldcs(reinterpret_cast<const unsigned short*>(p));
  }
  __device__ __forceinline__ void clear() { bits = 0; }
  __device__ __forceinline__ float get(int) const {
    return __uint_as_float(static_cast<unsigned>(bits) << 16);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[1]) {
    *p = __float2bfloat16_rn(v[0]);
  }
};

template <>
struct Piece<__nv_bfloat16, 2> {
  unsigned bits;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    bits = __ldcs(reinterpret_cast<const unsigned*>(p));
  }
  __device__ __forceinline__ void clear() { bits = 0; }
  __device__ __forceinline__ float get(int c) const {
    return __uint_as_float(c ? bits & 0xffff0000u : bits << 16);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[2]) {
    __stcs(reinterpret_cast<unsigned*>(p), pack_bf16x2(v[0], v[1]));
  }
};

// exp(g) as 2^(g log2(e)): two instructions.  The product's rounding costs |g| 2^-24 of the
// result, which matters little where a state is forgotten that fast.  ex2.approx is below the
// true value by 2.3e-8 on average for small arguments, as long memories have them (measured over
// [-0.2, 0]: mean -2.3e-8, rms 3.8e-8; the library's expf, of four times the instructions, has
// -1.6e-9 and 3.1e-8), which would add up over the ~1 / |g| steps that a state lives; the
// exponent carries log2(1 + 2.3e-8) against it.
__device__ __forceinline__ float decay_of(float g) {
  float a;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(fmaf(g, 1.4426950408889634f, 3.3e-8f)));
  return a;
}

// 1 - exp(g) for g <= 0, given a = exp(g): near 0, where the difference cancels, the series
// -g (1 + g/2 + g^2/6 + ...) to g^5 / 6! (the next term is 4.8e-8 at the border).
__device__ __forceinline__ float one_minus(float g, float a) {
  float p = 1.f / 720.f;
  p = fmaf(p, g, 1.f / 120.f);
  p = fmaf(p, g, 1.f / 24.f);
  p = fmaf(p, g, 1.f / 6.f);
  p = fmaf(p, g, 0.5f);
  p = fmaf(p, g, 1.f);
  return g > -0.25f ? -g * p : 1.f - a;
}

// ------------------------------------------------------------------ packed sequences

struct Packed {
  int N, n_seq;
  const int* off;  // null: n_seq sequences of len rows
  int len;
};

__device__ __forceinline__ int bound_of(const Packed& q, int j) {
  return q.off ? min(max(q.off[j], 0), q.N) : j * q.len;
}

// Reports offsets that break the rules (one block of the grid calls this).
__device__ __forceinline__ void check_offsets(const Packed& q, int* dev_status) {
  if (!q.off || !dev_status) return;
  int bad = threadIdx.x == 0 && q.off[0] != 0;
  for (int s = threadIdx.x; s < q.n_seq; s += blockDim.x)
    bad |= q.off[s] > q.off[s + 1] || q.off[s] < 0 || q.off[s + 1] > q.N;
  if (__syncthreads_or(bad) && threadIdx.x == 0) atomicCAS(dev_status, 0, MOE_ERR_BAD_INDEX);
}

// First row of part p of `parts`: the start of the first sequence that begins at or after row
// p N / parts.  Whole sequences go to one part, and every block finds the same cuts.
__device__ __forceinline__ int part_begin(const Packed& q, int p, int parts) {
  if (p == 0) return 0;
  if (p == parts) return bound_of(q, q.n_seq);
  const int target = static_cast<int>(static_cast<long long>(p) * q.N / parts);
  if (!q.off) return min((target + q.len - 1) / q.len, q.n_seq) * q.len;
  int before = 0;
  for (int s = 0; s < q.n_seq; s += blockDim.x) {
    const int i = s + threadIdx.x;
    before += __syncthreads_count(i < q.n_seq && q.off[i] < target);
  }
  return bound_of(q, before);
}

// Sequences that begin and end in the rows [t0, t0 + ROWS) of a tile: first[r], last[r] = the
// sequence whose first or last row is t0 + r, else -1.
template <int ROWS>
struct Marks {
  int first[ROWS], last[ROWS];
};

// Walks the bounds of the sequences beside tiles that come in ascending (DOWN: descending)
// order.  The state is the same in all threads of the block.
template <bool DOWN, int ROWS>
struct Walker {
  int cursor;  // bounds passed (DOWN: bounds left)
  int next;    // the nearest bound that is not passed

  __device__ __forceinline__ void start(const Packed& q) {
    cursor = DOWN ? q.n_seq + 1 : 0;
    next = DOWN ? 0x7fffffff : -1;
  }

  // Whether a sequence begins or ends in the tile at t0; then the marks are written, and the
  // block has to meet before it reads them, and again before the next call.
  __device__ __forceinline__ bool mark(const Packed& q, int t0, Marks<ROWS>& m) {
    if (!q.off) {
      // the first multiple of len that is not before the tile
      const long long at = t0 <= 0 ? 0 : (static_cast<long long>(t0) + q.len - 1) / q.len * q.len;
      if (at > t0 + ROWS) return false;
    } else if (DOWN ? next < t0 : next > t0 + ROWS) {
      return false;
    }
    for (int r = threadIdx.x; r < ROWS; r += blockDim.x) m.first[r] = m.last[r] = -1;
    __syncthreads();
    if (!q.off) {
      for (int r = threadIdx.x; r <= ROWS; r += blockDim.x) {
        const int t = t0 + r;
        if (t >= 0 && t <= q.N && t % q.len == 0) {
          if (r < ROWS && t < q.N) m.first[r] = t / q.len;
          if (r > 0 && t > 0) m.last[r - 1] = t / q.len - 1;
        }
      }
      return true;
    }
    while (true) {
      const int j = DOWN ? cursor - 1 - static_cast<int>(threadIdx.x)
                         : cursor + static_cast<int>(threadIdx.x);
      bool passed = false;
      if (j >= 0 && j <= q.n_seq) {
        const int b = bound_of(q, j);
        if (b >= t0 && b < t0 + ROWS && j < q.n_seq && bound_of(q, j + 1) > b) m.first[b - t0] = j;
        if (b > t0 && b <= t0 + ROWS && j > 0 && bound_of(q, j - 1) < b) m.last[b - t0 - 1] = j - 1;
        passed = DOWN ? b > t0 : b < t0 + ROWS;
      }
      const int n = __syncthreads_count(passed);
      cursor += DOWN ? -n : n;
      if (n < static_cast<int>(blockDim.x)) break;
    }
    if (DOWN)
      next = cursor > 0 ? bound_of(q, cursor - 1) : -0x7fffffff;
    else
      next = cursor <= q.n_seq ? bound_of(q, cursor) : 0x7fffffff;
    return true;
  }
};

// ------------------------------------------------------------------ joining spans of time
//
// h -> a h + b is associative in pairs (A, H): h -> A h + H.  The time axis is cut into tiles of
// 8 warps x R rows; the blocks of a cluster take neighbouring tiles, cluster after cluster of
// them.  Each warp runs its R rows twice in registers: once for their pair, and, when the pairs
// before it are known, once more from the state that these give.  Pairs are joined within a
// block through shared memory and within the cluster through distributed shared memory, always
// in the order of the recurrence.  A is -1 for a span in which a sequence begins: what came
// before is then not used at all, not even multiplied by zero.

template <int CH>
struct Pair {
  float A[CH], H[CH];
};

template <int CH>
__device__ __forceinline__ void follow(float (&h)[CH], const Pair<CH>& p) {
#pragma unroll
  for (int c = 0; c < CH; ++c) h[c] = p.A[c] < 0.f ? p.H[c] : fmaf(p.A[c], h[c], p.H[c]);
}

template <int CH>
__device__ __forceinline__ void append(Pair<CH>& s, const Pair<CH>& p) {
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    s.H[c] = p.A[c] < 0.f ? p.H[c] : fmaf(p.A[c], s.H[c], p.H[c]);
    s.A[c] = fminf(p.A[c], s.A[c]) < 0.f ? -1.f : s.A[c] * p.A[c];
  }
}

// What the warps of a block and the blocks of a cluster exchange, double-buffered by the parity
// of the step.  A block writes step n + 2 over step n only after it has every block's pair of
// step n + 1, and a block publishes that only when all its warps have read step n.
template <int CH>
struct Exchange {
  Pair<CH> warps[2][kWarps][32];
  Pair<CH> blocks[2][kMaxCluster][32];
  uint64_t full[2];
  int abort;
};

template <int CH>
__device__ __forceinline__ void exchange_init(Exchange<CH>& x, int cluster) {
  if (threadIdx.x == 0) {
    mbar_init(&x.full[0], 1);
    mbar_init(&x.full[1], 1);
    x.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (cluster > 1) cluster_sync();  // every block runs, its barriers set, before one writes there
}

// Sends a warp's joined pair to every block of the cluster (itself too), where it counts towards
// the barrier of the step.
template <int CH>
__device__ __forceinline__ void publish(Exchange<CH>& x, int buf, const Pair<CH>& p, int rank,
                                        int cluster, int lane) {
  for (int q = 0; q < cluster; ++q) {
    const uint32_t to = cluster_addr(&x.blocks[buf][rank][lane], q);
    const uint32_t bar = cluster_addr(&x.full[buf], q);
    if constexpr (CH == 2)
      asm volatile(
          "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, "
          "[%5];" ::"r"(to),
          "r"(__float_as_uint(p.A[0])), "r"(__float_as_uint(p.A[1])), "r"(__float_as_uint(p.H[0])),
          "r"(__float_as_uint(p.H[1])), "r"(bar)
          : "memory");
    else
      asm volatile(
          "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::
              "r"(to),
          "r"(__float_as_uint(p.A[0])), "r"(__float_as_uint(p.H[0])), "r"(bar)
          : "memory");
  }
}

// Joins the pairs of step `it`: `carry` becomes the state in front of this warp's span, `state`
// goes on over the whole step.  `order` is the warp's place in the order of the recurrence.  The
// wait is bounded: when it runs out the rest of the launch goes on without waiting (its results
// are then wrong, and reported), so every barrier still gets all its threads.
template <int CH>
__device__ __forceinline__ void join(Exchange<CH>& x, int it, const Pair<CH>& mine, int order,
                                     int rank, int cluster, int lane, float (&state)[CH],
                                     float (&carry)[CH], int* dev_status) {
  const int buf = it & 1;
  x.warps[buf][order][lane] = mine;
  if (cluster > 1 && threadIdx.x == 0)
    mbar_arrive_expect_tx(&x.full[buf], cluster * 32 * sizeof(Pair<CH>));
  __syncthreads();
  if (cluster > 1) {
    if (order == 0) {
      Pair<CH> sum = mine;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) append(sum, x.warps[buf][w][lane]);
      publish(x, buf, sum, rank, cluster, lane);
    }
    if (!mbar_wait(&x.full[buf], (it >> 1) & 1, &x.abort)) {
      *reinterpret_cast<volatile int*>(&x.abort) = 1;
      report_status(dev_status, MOE_ERR_TIMEOUT);
    }
#pragma unroll
    for (int q = 0; q < kMaxCluster; ++q) {
      if (q == rank)
#pragma unroll
        for (int c = 0; c < CH; ++c) carry[c] = state[c];
      if (q < cluster) follow(state, x.blocks[buf][q][lane]);
    }
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
      if (w < order) follow(carry, x.warps[buf][w][lane]);
  } else {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == order)
#pragma unroll
        for (int c = 0; c < CH; ++c) carry[c] = state[c];
      follow(state, x.warps[buf][w][lane]);
    }
  }
}

// R rows from row t0 at channel d; rows outside [lo, hi) as zeros.
template <typename T, int CH, int R>
__device__ __forceinline__ void fetch(Piece<T, CH> (&v)[R], const T* base, long long stride, int d,
                                      int t0, int lo, int hi) {
  const T* at = base + t0 * stride + d;
  if (t0 >= lo && t0 + R <= hi) {
#pragma unroll
    for (int r = 0; r < R; ++r, at += stride) v[r].load(at);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v[r].clear();
      if (t0 + r >= lo && t0 + r < hi) v[r].load(at + r * stride);
    }
  }
}

// ------------------------------------------------------------------ forward

template <typename T>
struct ForwardArgs {
  Packed seq;
  int D, parts, cluster;
  const T *g, *x;
  long long ld_g, ld_x;
  const float* h0;  // may be h_T
  T* h;
  float *h_T, *h_chunks;
  int* dev_status;
};

template <typename T, int CH, bool MIX>
__global__ void __launch_bounds__(32 * kWarps, 2) glr_forward_kernel(const ForwardArgs<T> p) {
  constexpr int R = 16, ROWS = kWarps * R;
  __shared__ Exchange<CH> xch;
  __shared__ Marks<ROWS> marks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.cluster, part = blockIdx.x / p.cluster;
  const int d0 = (blockIdx.y * 32 + lane) * CH;
  const bool on = d0 < p.D;
  const int d = on ? d0 : p.D - CH;  // lanes past the last channel load it too
  const long long D = p.D;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seq, p.dev_status);
  const int lo = part_begin(p.seq, part, p.parts), hi = part_begin(p.seq, part + 1, p.parts);

  if (p.seq.off && p.h_T && on)  // empty sequences hand their state on
    for (int s = blockIdx.x * kWarps + warp; s < p.seq.n_seq; s += gridDim.x * kWarps)
      if (bound_of(p.seq, s) >= bound_of(p.seq, s + 1))
#pragma unroll
        for (int c = 0; c < CH; ++c) p.h_T[s * D + d + c] = p.h0 ? p.h0[s * D + d + c] : 0.f;

  const int base = lo / ROWS * ROWS, step = ROWS * p.cluster;
  const int steps = hi > lo ? (hi - base + step - 1) / step : 0;
  Piece<T, CH> g[R], x[R];
  Walker<false, ROWS> walk;
  walk.start(p.seq);
  float state[CH] = {};
  if (steps) {
    fetch(g, p.g, p.ld_g, d, base + rank * ROWS + warp * R, lo, hi);
    fetch(x, p.x, p.ld_x, d, base + rank * ROWS + warp * R, lo, hi);
  }
  exchange_init(xch, p.cluster);
  for (int it = 0; it < steps; ++it) {
    const int tile = base + (it * p.cluster + rank) * ROWS, t0 = tile + warp * R;
    unsigned firsts = 0, lasts = 0;
    const bool marked = walk.mark(p.seq, tile, marks);
    if (marked) {
      __syncthreads();
      const int mine = warp * R + (lane & (R - 1));
      firsts = __ballot_sync(~0u, marks.first[mine] >= 0) & ((1u << R) - 1);
      lasts = __ballot_sync(~0u, marks.last[mine] >= 0) & ((1u << R) - 1);
    }

    // the span's pair; a[r], b[r] stay for the second pass
    float a[R][CH], b[R][CH], h[CH];
    Pair<CH> pair;
#pragma unroll
    for (int c = 0; c < CH; ++c) pair.A[c] = 1.f, pair.H[c] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const float lg = g[r].get(c), xv = x[r].get(c);
        a[r][c] = decay_of(lg);
        b[r][c] = MIX ? one_minus(lg, a[r][c]) * xv : xv;
        pair.A[c] *= a[r][c];
        pair.H[c] = fmaf(a[r][c], pair.H[c], b[r][c]);
      }
    if (it + 1 < steps) {
      fetch(g, p.g, p.ld_g, d, t0 + step, lo, hi);
      fetch(x, p.x, p.ld_x, d, t0 + step, lo, hi);
    }
    if (firsts) {  // again, with the initial states
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if ((firsts >> r & 1) && p.h0)
            b[r][c] = fmaf(a[r][c], p.h0[marks.first[warp * R + r] * D + d + c], b[r][c]);
          pair.H[c] = firsts >> r & 1 ? b[r][c] : fmaf(a[r][c], pair.H[c], b[r][c]);
        }
#pragma unroll
      for (int c = 0; c < CH; ++c) pair.A[c] = -1.f;
    }

    join(xch, it, pair, warp, rank, p.cluster, lane, state, h, p.dev_status);

    if (p.h_chunks && on && t0 % kChunk == 0 && t0 >= lo && t0 < hi)
#pragma unroll
      for (int c = 0; c < CH; ++c) p.h_chunks[t0 / kChunk * D + d + c] = firsts & 1 ? 0.f : h[c];
    T* out = p.h + t0 * D + d;
    if (!marked && t0 >= lo && t0 + R <= hi) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int c = 0; c < CH; ++c) h[c] = fmaf(a[r][c], h[c], b[r][c]);
        if (on) Piece<T, CH>::store(out, h);
        out += D;
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
          h[c] = firsts >> r & 1 ? b[r][c] : fmaf(a[r][c], h[c], b[r][c]);
        if (on && t0 + r >= lo && t0 + r < hi) {
          Piece<T, CH>::store(out + r * D, h);
          if ((lasts >> r & 1) && p.h_T)
#pragma unroll
            for (int c = 0; c < CH; ++c) p.h_T[marks.last[warp * R + r] * D + d + c] = h[c];
        }
      }
    }
    if (marked) __syncthreads();  // the marks are rewritten
  }
  if (p.cluster > 1) cluster_sync();  // no block leaves while another may still write to it
}

// ------------------------------------------------------------------ backward
//
// lam_t = dh_t + back_t, back_{t-1} = a_t lam_t runs the same scan with time reversed: pairs
// (A, H) of back over a span, the last row first.  A tile is one 64-row piece between kept
// states, so the states in front of its rows are formed again from the kept one within the
// block, beside the pairs of the gradient.

template <typename T>
struct BackwardArgs {
  Packed seq;
  int D, parts, cluster;
  const T *g, *x, *dh;
  long long ld_g, ld_x;
  const float *h0, *h_chunks, *dh_T;  // dh_T may be dh0
  T *dg, *dx;
  float* dh0;
  int* dev_status;
};

template <typename T, int CH, bool MIX>
__global__ void __launch_bounds__(32 * kWarps, 2) glr_backward_kernel(const BackwardArgs<T> p) {
  constexpr int R = 8, ROWS = kWarps * R;
  static_assert(ROWS == kChunk, "a tile begins at a kept state");
  __shared__ Exchange<CH> xch;
  __shared__ Pair<CH> ahead[2][kWarps][32];  // the forward pairs of the warps
  __shared__ Marks<ROWS> marks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.cluster, part = blockIdx.x / p.cluster;
  const int d0 = (blockIdx.y * 32 + lane) * CH;
  const bool on = d0 < p.D;
  const int d = on ? d0 : p.D - CH;
  const long long D = p.D;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seq, p.dev_status);
  const int lo = part_begin(p.seq, part, p.parts), hi = part_begin(p.seq, part + 1, p.parts);

  if (p.seq.off && p.dh0 && on)  // empty sequences hand their gradient on
    for (int s = blockIdx.x * kWarps + warp; s < p.seq.n_seq; s += gridDim.x * kWarps)
      if (bound_of(p.seq, s) >= bound_of(p.seq, s + 1))
#pragma unroll
        for (int c = 0; c < CH; ++c) p.dh0[s * D + d + c] = p.dh_T ? p.dh_T[s * D + d + c] : 0.f;

  const int top = (hi + ROWS - 1) / ROWS * ROWS, step = ROWS * p.cluster;
  const int steps = hi > lo ? (top - lo / ROWS * ROWS + step - 1) / step : 0;
  Piece<T, CH> g[R], x[R], dh[R];
  float kept[CH] = {};
  const auto fetch_tile = [&](Piece<T, CH>(&gt)[R], Piece<T, CH>(&xt)[R], Piece<T, CH>(&dt)[R],
                              float(&kt)[CH], int tile) {
    fetch(gt, p.g, p.ld_g, d, tile + warp * R, lo, hi);
    fetch(xt, p.x, p.ld_x, d, tile + warp * R, lo, hi);
    fetch(dt, p.dh, D, d, tile + warp * R, lo, hi);
    if (tile >= 0 && tile < hi)
#pragma unroll
      for (int c = 0; c < CH; ++c) kt[c] = p.h_chunks[tile / kChunk * D + d + c];
  };
  Walker<true, ROWS> walk;
  walk.start(p.seq);
  float state[CH] = {};
  if (steps) fetch_tile(g, x, dh, kept, top - (rank + 1) * ROWS);
  exchange_init(xch, p.cluster);
  for (int it = 0; it < steps; ++it) {
    const int tile = top - (it * p.cluster + rank + 1) * ROWS, t0 = tile + warp * R;
    unsigned firsts = 0, lasts = 0;
    const bool marked = walk.mark(p.seq, tile, marks);
    if (marked) {
      __syncthreads();
      const int mine = warp * R + (lane & (R - 1));
      firsts = __ballot_sync(~0u, marks.first[mine] >= 0) & ((1u << R) - 1);
      lasts = __ballot_sync(~0u, marks.last[mine] >= 0) & ((1u << R) - 1);
    }
    const auto state_before = [&](int r, int c) {  // of the sequence that begins in row r
      return p.h0 ? p.h0[marks.first[warp * R + r] * D + d + c] : 0.f;
    };
    const auto grad_after = [&](int r, int c) {  // of the sequence that ends in row r
      return p.dh_T ? p.dh_T[marks.last[warp * R + r] * D + d + c] : 0.f;
    };

    float a[R][CH], om[MIX ? R : 1][CH] = {};  // exp(g), 1 - exp(g)
    const auto input = [&](int r, int c) { return MIX ? om[r][c] * x[r].get(c) : x[r].get(c); };
    Pair<CH> fwd, rev;
#pragma unroll
    for (int c = 0; c < CH; ++c) fwd.A[c] = 1.f, fwd.H[c] = rev.H[c] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const float lg = g[r].get(c);
        a[r][c] = decay_of(lg);
        if (MIX) om[r][c] = one_minus(lg, a[r][c]);
        fwd.A[c] *= a[r][c];
        fwd.H[c] = fmaf(a[r][c], fwd.H[c], input(r, c));
      }
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
#pragma unroll
      for (int c = 0; c < CH; ++c) rev.H[c] = a[r][c] * (dh[r].get(c) + rev.H[c]);
#pragma unroll
    for (int c = 0; c < CH; ++c) rev.A[c] = fwd.A[c];
    if (firsts) {  // again, from the initial states
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (firsts >> r & 1) fwd.H[c] = state_before(r, c);
          fwd.H[c] = fmaf(a[r][c], fwd.H[c], input(r, c));
          fwd.A[c] = -1.f;
        }
    }
    if (lasts) {  // again, from the final states' gradients
#pragma unroll
      for (int r = R - 1; r >= 0; --r)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (lasts >> r & 1) rev.H[c] = grad_after(r, c);
          rev.H[c] = a[r][c] * (dh[r].get(c) + rev.H[c]);
          rev.A[c] = -1.f;
        }
    }
    ahead[it & 1][warp][lane] = fwd;
    Piece<T, CH> g_next[R], x_next[R], dh_next[R];
    float kept_next[CH] = {};
    if (it + 1 < steps) fetch_tile(g_next, x_next, dh_next, kept_next, tile - step);

    float back[CH];
    join(xch, it, rev, kWarps - 1 - warp, rank, p.cluster, lane, state, back, p.dev_status);

    float h[CH], before[R][CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) h[c] = kept[c];
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
      if (w < warp) follow(h, ahead[it & 1][w][lane]);
    T* dg = p.dg + (t0 + R - 1) * p.ld_g + d;
    T* dx = p.dx + (t0 + R - 1) * p.ld_x + d;
    if (!marked && t0 >= lo && t0 + R <= hi) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          before[r][c] = MIX ? h[c] - x[r].get(c) : h[c];
          h[c] = fmaf(a[r][c], h[c], input(r, c));
        }
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        float o_g[CH], o_x[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const float lam = dh[r].get(c) + back[c];
          back[c] = a[r][c] * lam;
          o_x[c] = MIX ? om[r][c] * lam : lam;
          o_g[c] = back[c] * before[r][c];
        }
        if (on) {
          Piece<T, CH>::store(dg, o_g);
          Piece<T, CH>::store(dx, o_x);
        }
        dg -= p.ld_g;
        dx -= p.ld_x;
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (firsts >> r & 1) h[c] = state_before(r, c);
          before[r][c] = MIX ? h[c] - x[r].get(c) : h[c];
          h[c] = fmaf(a[r][c], h[c], input(r, c));
        }
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        float o_g[CH], o_x[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (lasts >> r & 1) back[c] = grad_after(r, c);
          const float lam = dh[r].get(c) + back[c];
          back[c] = a[r][c] * lam;
          o_x[c] = MIX ? om[r][c] * lam : lam;
          o_g[c] = back[c] * before[r][c];
        }
        if (on && t0 + r >= lo && t0 + r < hi) {
          Piece<T, CH>::store(dg - (R - 1 - r) * p.ld_g, o_g);
          Piece<T, CH>::store(dx - (R - 1 - r) * p.ld_x, o_x);
          if ((firsts >> r & 1) && p.dh0)
#pragma unroll
            for (int c = 0; c < CH; ++c) p.dh0[marks.first[warp * R + r] * D + d + c] = back[c];
        }
      }
    }
    if (marked) __syncthreads();  // the marks are rewritten
#pragma unroll
    for (int r = 0; r < R; ++r) g[r] = g_next[r], x[r] = x_next[r], dh[r] = dh_next[r];
#pragma unroll
    for (int c = 0; c < CH; ++c) kept[c] = kept_next[c];
  }
  if (p.cluster > 1) cluster_sync();  // no block leaves while another may still write to it
}

template <typename T, bool MIX>
__global__ void __launch_bounds__(128)
    glr_step_kernel(int D, const T* g, long long ld_g, const T* x, long long ld_x,
                    const int* slot, int n_slots, float* state, T* h, int* dev_status) {
  const int b = blockIdx.y, d = blockIdx.x * 128 + threadIdx.x;
  const int row = claimed_slot(b, slot, n_slots, dev_status);
  if (row < 0 || d >= D) return;
  float* s = state + static_cast<long long>(row) * D + d;
  const float lg = ld(g, b * ld_g + d), xv = ld(x, b * ld_x + d);
  const float now = fmaf(expf(lg), *s, MIX ? -expm1f(lg) * xv : xv);
  *s = now;
  st(h, static_cast<long long>(b) * D + d, now);
}

// ------------------------------------------------------------------------ host side

bool misaligned(const void* p, int size) {
  return reinterpret_cast<uintptr_t>(p) & static_cast<unsigned>(size - 1);
}

int check_rows(int N, int D, int n_seq, const int* seq_off, int mode, int dtype, const void* g,
               long long ld_g, const void* x, long long ld_x, const void* out, bool grads) {
  if (N <= 0 || D <= 0 || n_seq <= 0 || !g || !x || !out) return MOE_ERR_INVALID_ARG;
  if (mode != MOE_GLR_ADD && mode != MOE_GLR_MIX) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_BF16 && dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (!seq_off && N % n_seq) return MOE_ERR_INVALID_ARG;
  for (long long ld : {ld_g, ld_x})
    if (N > 1 && ld < D && (grads || ld != 0)) return MOE_ERR_INVALID_ARG;
  const int size = dtype == MOE_BF16 ? 2 : 4;
  if (misaligned(g, size) || misaligned(x, size) || misaligned(out, size))
    return MOE_ERR_UNSUPPORTED;
  if (n_seq > (1 << 24) || N > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Blocks of a scan: strips of `width` channels, each a row of clusters over time.
struct Grid {
  int strips, cluster, parts;
};

Grid grid_of(int N, int D, int n_seq, int width, int rows) {
  Grid g;
  g.strips = (D + width - 1) / width;
  const int want = 2 * num_sms();  // two blocks of 8 warps on every SM
  const int tiles = (N + rows - 1) / rows;
  g.cluster = std::max(1, std::min({kMaxCluster, tiles, want / g.strips}));
  g.parts = std::max(1, std::min({n_seq, tiles, want / (g.strips * g.cluster)}));
  return g;
}

template <typename Args>
int launch(void (*kernel)(Args), const Grid& g, const Args& args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(g.cluster * g.parts, g.strips);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = g.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = g.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Calls f(T{}, channels per lane, mode) for the call's type: two bf16 channels per lane where
// every row of every tensor is 4-byte aligned, else one.
template <typename F>
int dispatch(int D, int mode, int dtype, std::initializer_list<const void*> ptrs,
             std::initializer_list<long long> strides, F f) {
  using std::integral_constant;
  const auto with_mode = [&](auto type, auto ch) {
    return mode == MOE_GLR_MIX ? f(type, ch, std::true_type{}) : f(type, ch, std::false_type{});
  };
  if (dtype == MOE_F32) return with_mode(float{}, integral_constant<int, 1>{});
  bool two = D % 2 == 0;
  for (const void* q : ptrs) two = two && !misaligned(q, 4);
  for (long long s : strides) two = two && s % 2 == 0;
  return two ? with_mode(__nv_bfloat16{}, integral_constant<int, 2>{})
             : with_mode(__nv_bfloat16{}, integral_constant<int, 1>{});
}

}  // namespace
}  // namespace moe

#define GLR_LAUNCH(KERNEL, GRID, BLOCK, ...)                                        \
  do {                                                                              \
    if (dtype == MOE_BF16) {                                                        \
      using T = __nv_bfloat16;                                                      \
      if (mode == MOE_GLR_MIX) KERNEL<T, true><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__); \
      else KERNEL<T, false><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__);               \
    } else {                                                                        \
      using T = float;                                                              \
      if (mode == MOE_GLR_MIX) KERNEL<T, true><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__); \
      else KERNEL<T, false><<<GRID, BLOCK, 0, stream>>>(__VA_ARGS__);               \
    }                                                                               \
  } while (0)

extern "C" {

using namespace moe;

int moe_glr_forward(int32_t N, int32_t D, int32_t n_seq, const int32_t* seq_off, int32_t mode,
                    int32_t dtype, const void* g, int64_t ld_g, const void* x, int64_t ld_x,
                    const float* h0, void* h, float* h_T, float* h_chunks, int32_t* dev_status,
                    moe_stream_t stream) {
  if (int e = check_rows(N, D, n_seq, seq_off, mode, dtype, g, ld_g, x, ld_x, h, false)) return e;
  const Packed seq{N, n_seq, seq_off, seq_off ? 0 : N / n_seq};
  mark_before(MOE_KERNEL_GLR_FWD, stream);
  const int e = dispatch(
      D, mode, dtype, {g, x, h}, {ld_g, ld_x, D}, [&](auto type, auto ch, auto mix) {
        using T = decltype(type);
        constexpr int CH = decltype(ch)::value;
        const Grid gr = grid_of(N, D, n_seq, 32 * CH, 16 * kWarps);
        const ForwardArgs<T> a{seq,  D,    gr.parts, gr.cluster, static_cast<const T*>(g),
                               static_cast<const T*>(x), ld_g,   ld_x, h0, static_cast<T*>(h),
                               h_T,  h_chunks, dev_status};
        return launch(glr_forward_kernel<T, CH, decltype(mix)::value>, gr, a, stream);
      });
  mark_after(MOE_KERNEL_GLR_FWD, stream);
  count_launches(1);
  return e;
}

int moe_glr_backward(int32_t N, int32_t D, int32_t n_seq, const int32_t* seq_off, int32_t mode,
                     int32_t dtype, const void* g, int64_t ld_g, const void* x, int64_t ld_x,
                     const float* h0, const float* h_chunks, const void* dh, const float* dh_T,
                     void* dg, void* dx, float* dh0, int32_t* dev_status, moe_stream_t stream) {
  if (int e = check_rows(N, D, n_seq, seq_off, mode, dtype, g, ld_g, x, ld_x, dg, true)) return e;
  if (!h_chunks || !dh || !dx) return MOE_ERR_INVALID_ARG;
  const int size = dtype == MOE_BF16 ? 2 : 4;
  if (misaligned(dh, size) || misaligned(dx, size)) return MOE_ERR_UNSUPPORTED;
  const Packed seq{N, n_seq, seq_off, seq_off ? 0 : N / n_seq};
  mark_before(MOE_KERNEL_GLR_BWD, stream);
  const int e = dispatch(
      D, mode, dtype, {g, x, dh, dg, dx}, {ld_g, ld_x, D}, [&](auto type, auto ch, auto mix) {
        using T = decltype(type);
        constexpr int CH = decltype(ch)::value;
        const Grid gr = grid_of(N, D, n_seq, 32 * CH, kChunk);
        const BackwardArgs<T> a{seq, D, gr.parts, gr.cluster, static_cast<const T*>(g),
                                static_cast<const T*>(x), static_cast<const T*>(dh), ld_g, ld_x,
                                h0, h_chunks, dh_T, static_cast<T*>(dg), static_cast<T*>(dx), dh0,
                                dev_status};
        return launch(glr_backward_kernel<T, CH, decltype(mix)::value>, gr, a, stream);
      });
  mark_after(MOE_KERNEL_GLR_BWD, stream);
  count_launches(1);
  return e;
}

int moe_glr_step(int32_t B, int32_t D, int32_t mode, int32_t dtype, const void* g, int64_t ld_g,
                 const void* x, int64_t ld_x, const int32_t* slot, int32_t n_slots, float* state,
                 void* h, int32_t* dev_status, moe_stream_t stream) {
  if (int e = check_rows(B, D, 1, nullptr, mode, dtype, g, ld_g, x, ld_x, h, false)) return e;
  if (!state || n_slots <= 0 || (!slot && B > n_slots)) return MOE_ERR_INVALID_ARG;
  if (B > 65535) return MOE_ERR_UNSUPPORTED;
  const dim3 grid((D + 127) / 128, B);
  mark_before(MOE_KERNEL_GLR_STEP, stream);
  GLR_LAUNCH(glr_step_kernel, grid, 128, D, static_cast<const T*>(g), ld_g,
             static_cast<const T*>(x), ld_x, slot, n_slots, state, static_cast<T*>(h),
             dev_status);
  const cudaError_t err = cudaGetLastError();
  mark_after(MOE_KERNEL_GLR_STEP, stream);
  count_launches(1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
