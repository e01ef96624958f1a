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
constexpr int kWarps = 8;       // warps of a scan block, beside the one that joins
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kRows = 8;        // rows of a warp in a tile
constexpr int kTile = kWarps * kRows;
constexpr int kStages = 3;      // tiles in shared memory
constexpr int kMaxCluster = 8;  // blocks of a cluster (the portable limit)
constexpr int kBounds = 512;    // bounds of sequences that a block keeps in shared memory

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
__device__ __forceinline__ float get(const uint32_t& bits, int c, __nv_bfloat16) {
  return __uint_as_float(c ? bits & 0xffff0000u : bits << 16);
}
__device__ __forceinline__ float get(const uint32_t& bits, int, float) {
  return __uint_as_float(bits);
}

__device__ __forceinline__ void put(float* p, const float (&v)[1]) { __stcs(p, v[0]); }
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&v)[1]) {
  *p = __float2bfloat16_rn(v[0]);
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&v)[2]) {
  __stcs(reinterpret_cast<unsigned*>(p), pack_bf16x2(v[0], v[1]));
}

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

// Part p of `parts` begins with the first sequence that begins at or after row p N / parts: its
// index (off only) and its first row.  Whole sequences go to one part, and every block finds the
// same cuts.  Called by whole blocks.
struct Cut {
  int seq, row;
};

__device__ __forceinline__ Cut part_begin(const Packed& q, int p, int parts) {
  if (p == 0) return {0, 0};
  if (p == parts) return {q.n_seq, bound_of(q, q.n_seq)};
  const int target = static_cast<int>(static_cast<long long>(p) * q.N / parts);
  if (!q.off) {
    const int s = min((target + q.len - 1) / q.len, q.n_seq);
    return {s, s * q.len};
  }
  int before = 0;
  for (int s = 0; s < q.n_seq; s += blockDim.x) {
    const int i = s + threadIdx.x;
    before += __syncthreads_count(i < q.n_seq && q.off[i] < target);
  }
  return {before, bound_of(q, before)};
}

// What begins and ends in the kRows rows of a warp: bit r of firsts and lasts for row r, and the
// sequences (one warp's own words of shared memory).
struct Marks {
  int first[kRows], last[kRows];
};

// Walks the bounds of the sequences beside a warp's rows, which come in ascending (DOWN:
// descending) order.  The state is the same in all lanes.
template <bool DOWN>
struct Walker {
  int cursor;  // bounds passed (DOWN: bounds left)
  int next;    // the nearest bound that is not passed

  __device__ __forceinline__ void start(const Cut& from) {
    cursor = DOWN ? from.seq + 1 : from.seq;
    next = from.row;
  }

  __device__ __forceinline__ void mark(const Packed& q, int t0, int lane, Marks& m,
                                       unsigned& firsts, unsigned& lasts) {
    firsts = lasts = 0;
    if (!q.off) {
      // the first multiple of len that is not before the rows
      if (t0 > 0 && (t0 + q.len - 1ll) / q.len * q.len > t0 + kRows) return;
      __syncwarp();  // the words may still be read
      const int t = t0 + lane;
      const bool bound = lane <= kRows && t >= 0 && t <= q.N && t % q.len == 0;
      const bool first = bound && lane < kRows && t < q.N, last = bound && lane > 0 && t > 0;
      if (first) m.first[lane] = t / q.len;
      if (last) m.last[lane - 1] = t / q.len - 1;
      firsts = __ballot_sync(~0u, first);
      lasts = __ballot_sync(~0u, last) >> 1;
      __syncwarp();
      return;
    }
    if (DOWN ? next < t0 : next > t0 + kRows) return;
    __syncwarp();
    while (true) {
      const int j = DOWN ? cursor - 1 - lane : cursor + lane;
      bool passed = false;
      unsigned first = 0, last = 0;
      if (j >= 0 && j <= q.n_seq) {
        const int b = bound_of(q, j), r = b - t0;
        if (r >= 0 && r < kRows && j < q.n_seq && bound_of(q, j + 1) > b) {
          m.first[r] = j;
          first = 1u << r;
        }
        if (r > 0 && r <= kRows && j > 0 && bound_of(q, j - 1) < b) {
          m.last[r - 1] = j - 1;
          last = 1u << (r - 1);
        }
        passed = DOWN ? r > 0 : r < kRows;
      }
      firsts |= __reduce_or_sync(~0u, first);
      lasts |= __reduce_or_sync(~0u, last);
      const int n = __popc(__ballot_sync(~0u, passed));
      cursor += DOWN ? -n : n;
      if (n < 32) break;
    }
    if (DOWN)
      next = cursor > 0 ? bound_of(q, cursor - 1) : -0x7fffffff;
    else
      next = cursor <= q.n_seq ? bound_of(q, cursor) : 0x7fffffff;
    __syncwarp();
  }
};

// ------------------------------------------------------------------ joining spans of time
//
// h -> a h + b is associative in pairs (A, H): h -> A h + H.  The time axis is cut into tiles of
// 8 warps x kRows rows; the blocks of a cluster take neighbouring tiles, cluster after cluster of
// them.  Each warp runs its rows twice in registers: once for their pair, and, when the pairs
// before it are known, once more from the state that these give.  A ninth warp joins the pairs,
// always in the order of the recurrence: over the warps, over the blocks of the cluster (through
// distributed shared memory) and from step to step; meanwhile the others form the pairs of the
// next tile.  A is -1 for a span in which a sequence begins: what came before is then not used at
// all, not even multiplied by zero.

// (Aligned for the vector store that carries it.)
template <int CH>
struct alignas(8 * CH) Pair {
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
// of the step.  A warp forms its pair of step n + 2 after it has its state of step n, which the
// joining warp gives when it has read the pairs of step n; and that warp joins step n + 2 when
// every warp has formed its pair, after using its state of step n.  A block sends its pair of
// step n + 2 when it has every block's of step n + 1, and a block sends that after it has read
// all of step n.
template <int CH, int PAIRS>
struct Exchange {
  Pair<CH> warps[2][PAIRS][kWarps][32];
  Pair<CH> blocks[2][kMaxCluster][32];
  float states[2][PAIRS][kWarps][32 * CH];
  uint64_t formed[2], joined[2], received[2];
  uint64_t loaded[kStages], freed[kStages];  // tiles
  int abort;
};

// Waits, with a limit.  When it runs out the rest of the launch goes on without waiting (its
// results are then wrong, and reported).
__device__ __forceinline__ void wait_for(uint64_t* bar, int n, int* abort, int* dev_status) {
  if (!mbar_wait(bar, n & 1, abort)) {
    *reinterpret_cast<volatile int*>(abort) = 1;
    report_status(dev_status, MOE_ERR_TIMEOUT);
  }
}

// One lane's arrival for its warp.
__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

template <typename X>
__device__ __forceinline__ void exchange_init(X& x, int cluster) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&x.formed[i], kWarps);
      mbar_init(&x.joined[i], 1);
      mbar_init(&x.received[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&x.loaded[i], 1);
      mbar_init(&x.freed[i], kWarps);
    }
    x.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (cluster > 1) cluster_sync();  // every block runs, its barriers set, before one writes there
}

// Sends a block's pair to every block of the cluster (itself too), where it counts towards the
// barrier of the step.
template <int CH>
__device__ __forceinline__ void publish(Pair<CH>* slot, uint64_t* received, const Pair<CH>& p,
                                        int cluster) {
  for (int q = 0; q < cluster; ++q) {
    const uint32_t to = cluster_addr(slot, q), bar = cluster_addr(received, q);
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

// The joining warp's part of a step: `pairs` (order w is at warps[PAIR][DOWN ? 7 - w : w]) give
// every warp its state in states[PAIR] and move `state` over the whole step.
template <bool DOWN, int PAIR, int CH, int PAIRS>
__device__ __forceinline__ void join(Exchange<CH, PAIRS>& x, int it, int rank, int cluster,
                                     int lane, float (&state)[CH], int* dev_status) {
  const int buf = it & 1;
  Pair<CH> pairs[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) pairs[w] = x.warps[buf][PAIR][DOWN ? kWarps - 1 - w : w][lane];
  float carry[CH];
  if (cluster > 1) {
    Pair<CH> sum = pairs[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) append(sum, pairs[w]);
    if (lane == 0) mbar_arrive_expect_tx(&x.received[buf], cluster * 32 * sizeof(Pair<CH>));
    publish(&x.blocks[buf][rank][lane], &x.received[buf], sum, cluster);
    wait_for(&x.received[buf], it >> 1, &x.abort, dev_status);
#pragma unroll
    for (int q = 0; q < kMaxCluster; ++q) {
      if (q == rank)
#pragma unroll
        for (int c = 0; c < CH; ++c) carry[c] = state[c];
      if (q < cluster) follow(state, x.blocks[buf][q][lane]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) carry[c] = state[c];
  }
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    float* to = &x.states[buf][PAIR][DOWN ? kWarps - 1 - w : w][lane * CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) to[c] = carry[c];
    follow(carry, pairs[w]);
  }
  if (cluster == 1)
#pragma unroll
    for (int c = 0; c < CH; ++c) state[c] = carry[c];
}

// ------------------------------------------------------------------ tiles in shared memory
//
// kStages tiles of ARRAYS inputs, each [kTile][32] words: the word of a lane holds its CH
// channels.  Where rows begin on 16-byte boundaries, the joining warp has TMA copy whole tiles
// ahead (ASYNC); elsewhere each warp copies its rows through registers when they are asked for.
template <int ARRAYS>
__device__ __forceinline__ uint32_t* tile_at(uint32_t* ring, int it, int array) {
  return ring + (it % kStages * ARRAYS + array) * kTile * 32;
}

// One thread: the copies of step `it`, the tile at row t0 of the strip at channel d0.
template <int ARRAYS>
__device__ __forceinline__ void load_tile(uint32_t* ring, uint64_t* loaded, const CUtensorMap* maps,
                                          int it, int d0, int t0) {
  uint64_t* bar = &loaded[it % kStages];
  mbar_arrive_expect_tx(bar, ARRAYS * kTile * 128);
  const uint64_t policy = l2_policy_evict_first();
  for (int i = 0; i < ARRAYS; ++i)
    tma_load_2d(tile_at<ARRAYS>(ring, it, i), &maps[i], bar, d0, t0, policy);
}

// One thread, after a launch that gave up: the copies still in flight (again with a limit).
__device__ __forceinline__ void drain(uint64_t* loaded, int steps, volatile int* abort) {
  if (!*abort) return;
  int never = 0;
  for (int it = max(0, steps - kStages); it < steps; ++it)
    mbar_wait(&loaded[it % kStages], (it / kStages) & 1, &never);
}

// A warp's rows from row t0, those outside [lo, hi) as zeros; words[r 32] is row r's.
template <typename T>
__device__ __forceinline__ void copy_rows(uint32_t* words, const T* base, long long stride, int t0,
                                          int lo, int hi, bool on) {
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    uint32_t bits = 0;
    if (on && t0 + r >= lo && t0 + r < hi) {
      const T v = base[(t0 + r) * stride];
      memcpy(&bits, &v, sizeof v);
    }
    words[r * 32] = bits;
  }
}

// Dynamic shared memory from its first 128-byte boundary on, as TMA wants it (the launch asks for
// kAlign bytes more).
constexpr int kAlign = 128;
__device__ __forceinline__ uint32_t* aligned_128(uint32_t* p) {
  return p + (((smem_u32(p) + 127u) & ~127u) - smem_u32(p)) / 4;
}

// The bounds of the sequences, from shared memory where they fit.
__device__ __forceinline__ Packed near(const Packed& q, int* bounds) {
  if (!q.off || q.n_seq >= kBounds) return q;
  for (int i = threadIdx.x; i <= q.n_seq; i += kThreads) bounds[i] = q.off[i];
  __syncthreads();
  return {q.N, q.n_seq, bounds, q.len};
}

// to = from for the sequences without rows, from null: zero (a part of them for each warp).
template <int CH>
__device__ __forceinline__ void hand_on_empty(const Packed& q, const float* from, float* to,
                                              long long D, int d, int warp) {
  for (int s = blockIdx.x * kWarps + warp; s < q.n_seq; s += gridDim.x * kWarps)
    if (bound_of(q, s) >= bound_of(q, s + 1))
#pragma unroll
      for (int c = 0; c < CH; ++c) to[s * D + d + c] = from ? from[s * D + d + c] : 0.f;
}

// ------------------------------------------------------------------ forward

template <typename T>
struct ForwardArgs {
  CUtensorMap maps[2];  // g, x (ASYNC)
  Packed seq;
  int D, parts, cluster;
  const T *g, *x;
  long long ld_g, ld_x;
  const float* h0;  // may be h_T
  T* h;
  float *h_T, *h_chunks;
  int* dev_status;
};

template <typename T, int CH, bool MIX, bool ASYNC>
__global__ void __launch_bounds__(kThreads, 2)
    glr_forward_kernel(const __grid_constant__ ForwardArgs<T> p) {
  extern __shared__ uint32_t dynamic[];
  uint32_t* ring = aligned_128(dynamic);
  __shared__ Exchange<CH, 1> xch;
  __shared__ Marks marks[2][kWarps];
  __shared__ int bounds[kBounds];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.cluster, part = blockIdx.x / p.cluster;
  const int d = (blockIdx.y * 32 + lane) * CH;
  const bool on = d < p.D;
  const long long D = p.D;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seq, p.dev_status);
  const Packed seq = near(p.seq, bounds);
  const Cut from = part_begin(seq, part, p.parts);
  const int lo = from.row, hi = part_begin(seq, part + 1, p.parts).row;
  const int base = lo / kTile * kTile, step = kTile * p.cluster;
  const int steps = hi > lo ? (hi - base + step - 1) / step : 0;
  const auto tile_row = [&](int it) { return base + (it * p.cluster + rank) * kTile; };
  exchange_init(xch, p.cluster);

  if (warp == kWarps) {  // the joining warp
    const auto load = [&](int it) {
      if (ASYNC && lane == 0 && it < steps)
        load_tile<2>(ring, xch.loaded, p.maps, it, blockIdx.y * 32 * CH, tile_row(it));
    };
    for (int it = 0; it < kStages; ++it) load(it);
    float state[CH] = {};
    for (int it = 0; it < steps; ++it) {
      wait_for(&xch.formed[it & 1], it >> 1, &xch.abort, p.dev_status);
      load(it + kStages);  // every warp has read this step's tile
      join<false, 0>(xch, it, rank, p.cluster, lane, state, p.dev_status);
      arrive_warp(&xch.joined[it & 1], lane);
    }
    if (ASYNC && lane == 0) drain(xch.loaded, steps, &xch.abort);
  } else {
    if (seq.off && p.h_T && on) hand_on_empty<CH>(seq, p.h0, p.h_T, D, d, warp);
    struct Span {
      float a[kRows][CH], b[kRows][CH];
      unsigned firsts, lasts;
    };
    Walker<false> walk;
    walk.start(from);

    // the pair of the span of step `it`
    const auto form = [&](int it, Span& s) {
      const int t0 = tile_row(it) + warp * kRows;
      const Marks& m = marks[it & 1][warp];
      walk.mark(seq, t0, lane, marks[it & 1][warp], s.firsts, s.lasts);
      uint32_t* g = tile_at<2>(ring, it, 0) + warp * kRows * 32 + lane;
      uint32_t* x = tile_at<2>(ring, it, 1) + warp * kRows * 32 + lane;
      if (ASYNC) {
        wait_for(&xch.loaded[it % kStages], it / kStages, &xch.abort, p.dev_status);
        if (t0 < lo || t0 + kRows > hi) {  // rows of others and padding: the state goes through
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (t0 + r < lo || t0 + r >= hi) g[r * 32] = x[r * 32] = 0;
          fence_proxy_async_smem();  // TMA writes these words next
        }
      } else {
        copy_rows(g, p.g + d, p.ld_g, t0, lo, hi, on);
        copy_rows(x, p.x + d, p.ld_x, t0, lo, hi, on);
      }
      Pair<CH> pair;
#pragma unroll
      for (int c = 0; c < CH; ++c) pair.A[c] = 1.f, pair.H[c] = 0.f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const uint32_t wg = g[r * 32], wx = x[r * 32];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const float lg = get(wg, c, T()), xv = get(wx, c, T());
          s.a[r][c] = decay_of(lg);
          s.b[r][c] = MIX ? one_minus(lg, s.a[r][c]) * xv : xv;
          pair.A[c] *= s.a[r][c];
          pair.H[c] = fmaf(s.a[r][c], pair.H[c], s.b[r][c]);
        }
      }
      if (s.firsts) {  // again, with the initial states
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            if ((s.firsts >> r & 1) && p.h0 && on)
              s.b[r][c] = fmaf(s.a[r][c], p.h0[m.first[r] * D + d + c], s.b[r][c]);
            pair.H[c] = s.firsts >> r & 1 ? s.b[r][c] : fmaf(s.a[r][c], pair.H[c], s.b[r][c]);
            pair.A[c] = -1.f;
          }
      }
      xch.warps[it & 1][0][warp][lane] = pair;
      arrive_warp(&xch.formed[it & 1], lane);
    };

    // the rows of step `it` from the state in front of them
    const auto finish = [&](int it, Span& s) {
      const int t0 = tile_row(it) + warp * kRows;
      const Marks& m = marks[it & 1][warp];
      wait_for(&xch.joined[it & 1], it >> 1, &xch.abort, p.dev_status);
      float h[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) h[c] = xch.states[it & 1][0][warp][lane * CH + c];
      if (p.h_chunks && on && t0 % kChunk == 0 && t0 >= lo && t0 < hi)
#pragma unroll
        for (int c = 0; c < CH; ++c)
          p.h_chunks[t0 / kChunk * D + d + c] = s.firsts & 1 ? 0.f : h[c];
      T* out = p.h + t0 * D + d;
      if (!(s.firsts | s.lasts) && t0 >= lo && t0 + kRows <= hi) {
#pragma unroll
        for (int r = 0; r < kRows; ++r, out += D) {
#pragma unroll
          for (int c = 0; c < CH; ++c) h[c] = fmaf(s.a[r][c], h[c], s.b[r][c]);
          if (on) put(out, h);
        }
        return;
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r, out += D) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
          h[c] = s.firsts >> r & 1 ? s.b[r][c] : fmaf(s.a[r][c], h[c], s.b[r][c]);
        if (on && t0 + r >= lo && t0 + r < hi) {
          put(out, h);
          if ((s.lasts >> r & 1) && p.h_T)
#pragma unroll
            for (int c = 0; c < CH; ++c) p.h_T[m.last[r] * D + d + c] = h[c];
        }
      }
    };

    Span even, odd;
    for (int it = -1; it < steps; it += 2) {
      if (it + 1 < steps) form(it + 1, even);
      if (it >= 0) finish(it, odd);
      if (it + 2 < steps) form(it + 2, odd);
      if (it + 1 < steps) finish(it + 1, even);
    }
  }
  __syncwarp();
  if (p.cluster > 1) cluster_sync();  // no block leaves while another may still write to it
}

// ------------------------------------------------------------------ backward
//
// lam_t = dh_t + back_t, back_{t-1} = a_t lam_t runs the same scan with time reversed: pairs
// (A, H) of back over a span, the last row first.  A tile is one 64-row piece between kept
// states, so the states in front of its rows are formed again from the kept one within the
// block, by pairs of their own.

template <typename T>
struct BackwardArgs {
  CUtensorMap maps[3];  // g, x, dh (ASYNC)
  Packed seq;
  int D, parts, cluster;
  const T *g, *x, *dh;
  long long ld_g, ld_x;
  const float *h0, *h_chunks, *dh_T;  // dh_T may be dh0
  T *dg, *dx;
  float* dh0;
  int* dev_status;
};

template <typename T, int CH, bool MIX, bool ASYNC>
__global__ void __launch_bounds__(kThreads, 2)
    glr_backward_kernel(const __grid_constant__ BackwardArgs<T> p) {
  static_assert(kTile == kChunk, "a tile begins at a kept state");
  extern __shared__ uint32_t dynamic[];
  uint32_t* ring = aligned_128(dynamic);
  __shared__ Exchange<CH, 2> xch;  // the gradient's pairs, the state's
  __shared__ Marks marks[2][kWarps];
  __shared__ int bounds[kBounds];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.cluster, part = blockIdx.x / p.cluster;
  const int d = (blockIdx.y * 32 + lane) * CH;
  const bool on = d < p.D;
  const long long D = p.D;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seq, p.dev_status);
  const Packed seq = near(p.seq, bounds);
  const Cut until = part_begin(seq, part + 1, p.parts);
  const int lo = part_begin(seq, part, p.parts).row, hi = until.row;
  const int top = (hi + kTile - 1) / kTile * kTile, step = kTile * p.cluster;
  const int steps = hi > lo ? (top - lo / kTile * kTile + step - 1) / step : 0;
  const auto tile_row = [&](int it) { return top - (it * p.cluster + rank + 1) * kTile; };
  exchange_init(xch, p.cluster);

  if (warp == kWarps) {  // the joining warp
    const auto load = [&](int it) {
      if (ASYNC && lane == 0 && it < steps)
        load_tile<3>(ring, xch.loaded, p.maps, it, blockIdx.y * 32 * CH, tile_row(it));
    };
    const auto kept_state = [&](int it, float(&k)[CH]) {
      const int tile = tile_row(it);
#pragma unroll
      for (int c = 0; c < CH; ++c)
        k[c] = on && it < steps && tile >= 0 ? p.h_chunks[tile / kChunk * D + d + c] : 0.f;
    };
    for (int it = 0; it < kStages; ++it) load(it);
    float state[CH] = {}, kept[CH];
    kept_state(0, kept);
    for (int it = 0; it < steps; ++it) {
      wait_for(&xch.formed[it & 1], it >> 1, &xch.abort, p.dev_status);
      join<false, 1>(xch, it, 0, 1, lane, kept, p.dev_status);
      kept_state(it + 1, kept);
      join<true, 0>(xch, it, rank, p.cluster, lane, state, p.dev_status);
      arrive_warp(&xch.joined[it & 1], lane);
      if (ASYNC && it > 0) {  // the step before has been read for the second time
        wait_for(&xch.freed[(it - 1) % kStages], (it - 1) / kStages, &xch.abort, p.dev_status);
        load(it - 1 + kStages);
      }
    }
    if (ASYNC && lane == 0) drain(xch.loaded, steps, &xch.abort);
  } else {
    if (seq.off && p.dh0 && on) hand_on_empty<CH>(seq, p.dh_T, p.dh0, D, d, warp);
    struct Span {
      float a[kRows][CH], om[MIX ? kRows : 1][CH];  // exp(g), 1 - exp(g)
      unsigned firsts, lasts;
    };
    Walker<true> walk;
    walk.start(until);
    const auto words = [&](int it, int array) {
      return tile_at<3>(ring, it, array) + warp * kRows * 32 + lane;
    };
    const auto state_before = [&](const Marks& m, int r, int c) {  // where a sequence begins
      return on && p.h0 ? p.h0[m.first[r] * D + d + c] : 0.f;
    };
    const auto grad_after = [&](const Marks& m, int r, int c) {  // where a sequence ends
      return on && p.dh_T ? p.dh_T[m.last[r] * D + d + c] : 0.f;
    };

    // the pairs of the span of step `it`
    const auto form = [&](int it, Span& s) {
      const int t0 = tile_row(it) + warp * kRows;
      const Marks& m = marks[it & 1][warp];
      walk.mark(seq, t0, lane, marks[it & 1][warp], s.firsts, s.lasts);
      uint32_t *g = words(it, 0), *x = words(it, 1), *dh = words(it, 2);
      if (ASYNC) {
        wait_for(&xch.loaded[it % kStages], it / kStages, &xch.abort, p.dev_status);
        if (t0 < lo || t0 + kRows > hi) {  // rows of others and padding: all goes through
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (t0 + r < lo || t0 + r >= hi) g[r * 32] = x[r * 32] = dh[r * 32] = 0;
          fence_proxy_async_smem();  // TMA writes these words next
        }
      } else {
        copy_rows(g, p.g + d, p.ld_g, t0, lo, hi, on);
        copy_rows(x, p.x + d, p.ld_x, t0, lo, hi, on);
        copy_rows(dh, p.dh + d, D, t0, lo, hi, on);
      }
      const auto input = [&](int r, int c) {
        const float xv = get(x[r * 32], c, T());
        return MIX ? s.om[MIX ? r : 0][c] * xv : xv;
      };
      Pair<CH> fwd, rev;
#pragma unroll
      for (int c = 0; c < CH; ++c) fwd.A[c] = 1.f, fwd.H[c] = rev.H[c] = 0.f;
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const float lg = get(g[r * 32], c, T());
          s.a[r][c] = decay_of(lg);
          if (MIX) s.om[MIX ? r : 0][c] = one_minus(lg, s.a[r][c]);
          fwd.A[c] *= s.a[r][c];
          fwd.H[c] = fmaf(s.a[r][c], fwd.H[c], input(r, c));
        }
#pragma unroll
      for (int r = kRows - 1; r >= 0; --r)
#pragma unroll
        for (int c = 0; c < CH; ++c)
          rev.H[c] = s.a[r][c] * (get(dh[r * 32], c, T()) + rev.H[c]);
#pragma unroll
      for (int c = 0; c < CH; ++c) rev.A[c] = fwd.A[c];
      if (s.firsts) {  // again, from the initial states
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            if (s.firsts >> r & 1) fwd.H[c] = state_before(m, r, c);
            fwd.H[c] = fmaf(s.a[r][c], fwd.H[c], input(r, c));
            fwd.A[c] = -1.f;
          }
      }
      if (s.lasts) {  // again, from the final states' gradients
#pragma unroll
        for (int r = kRows - 1; r >= 0; --r)
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            if (s.lasts >> r & 1) rev.H[c] = grad_after(m, r, c);
            rev.H[c] = s.a[r][c] * (get(dh[r * 32], c, T()) + rev.H[c]);
            rev.A[c] = -1.f;
          }
      }
      xch.warps[it & 1][0][warp][lane] = rev;
      xch.warps[it & 1][1][warp][lane] = fwd;
      arrive_warp(&xch.formed[it & 1], lane);
    };

    // the gradients of step `it`
    const auto finish = [&](int it, Span& s) {
      const int t0 = tile_row(it) + warp * kRows;
      const Marks& m = marks[it & 1][warp];
      const uint32_t *x = words(it, 1), *dh = words(it, 2);
      wait_for(&xch.joined[it & 1], it >> 1, &xch.abort, p.dev_status);
      float back[CH], h[CH], before[kRows][CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        back[c] = xch.states[it & 1][0][warp][lane * CH + c];
        h[c] = xch.states[it & 1][1][warp][lane * CH + c];
      }
      const auto advance = [&](int r, int c) {
        const float xv = get(x[r * 32], c, T());
        before[r][c] = MIX ? h[c] - xv : h[c];
        h[c] = fmaf(s.a[r][c], h[c], MIX ? s.om[MIX ? r : 0][c] * xv : xv);
      };
      T* dg = p.dg + (t0 + kRows - 1) * p.ld_g + d;
      T* dx = p.dx + (t0 + kRows - 1) * p.ld_x + d;
      float o_g[CH], o_x[CH];
      const auto retreat = [&](int r, int c) {
        const float lam = get(dh[r * 32], c, T()) + back[c];
        back[c] = s.a[r][c] * lam;
        o_x[c] = MIX ? s.om[MIX ? r : 0][c] * lam : lam;
        o_g[c] = back[c] * before[r][c];
      };
      if (!(s.firsts | s.lasts) && t0 >= lo && t0 + kRows <= hi) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int c = 0; c < CH; ++c) advance(r, c);
#pragma unroll
        for (int r = kRows - 1; r >= 0; --r, dg -= p.ld_g, dx -= p.ld_x) {
#pragma unroll
          for (int c = 0; c < CH; ++c) retreat(r, c);
          if (on) {
            put(dg, o_g);
            put(dx, o_x);
          }
        }
      } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            if (s.firsts >> r & 1) h[c] = state_before(m, r, c);
            advance(r, c);
          }
#pragma unroll
        for (int r = kRows - 1; r >= 0; --r, dg -= p.ld_g, dx -= p.ld_x) {
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            if (s.lasts >> r & 1) back[c] = grad_after(m, r, c);
            retreat(r, c);
          }
          if (on && t0 + r >= lo && t0 + r < hi) {
            put(dg, o_g);
            put(dx, o_x);
            if ((s.firsts >> r & 1) && p.dh0)
#pragma unroll
              for (int c = 0; c < CH; ++c) p.dh0[m.first[r] * D + d + c] = back[c];
          }
        }
      }
      if (ASYNC) arrive_warp(&xch.freed[it % kStages], lane);
    };

    Span even, odd;
    for (int it = -1; it < steps; it += 2) {
      if (it + 1 < steps) form(it + 1, even);
      if (it >= 0) finish(it, odd);
      if (it + 2 < steps) form(it + 2, odd);
      if (it + 1 < steps) finish(it + 1, even);
    }
  }
  __syncwarp();
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

Grid grid_of(int N, int D, int n_seq, int width) {
  Grid g;
  g.strips = (D + width - 1) / width;
  const int want = 2 * num_sms();  // two blocks of 8 warps on every SM
  const int tiles = (N + kTile - 1) / kTile;
  g.cluster = std::max(1, std::min({kMaxCluster, tiles, want / g.strips}));
  g.parts = std::max(1, std::min({n_seq, tiles, want / (g.strips * g.cluster)}));
  return g;
}

// Launches KERNEL with `ring` bytes of shared memory beside its own.
template <typename Args>
int launch(void (*kernel)(Args), const Grid& g, int ring, const Args& args, cudaStream_t stream) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ring) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(g.cluster * g.parts, g.strips);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = ring;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = g.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = g.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Calls f(T{}, channels per lane, mode, ASYNC) for the call's type.  Tensors whose rows all begin
// on 16-byte boundaries (and do not share one row) are copied by TMA.
template <typename F>
int dispatch(int mode, int dtype, std::initializer_list<const void*> ptrs,
             std::initializer_list<long long> strides, F f) {
  using std::integral_constant;
  using One = integral_constant<int, 1>;
  using Two = integral_constant<int, 2>;
  const int size = dtype == MOE_F32 ? 4 : 2;
  bool aligned = true;
  for (const void* q : ptrs) aligned = aligned && !misaligned(q, 16);
  for (long long s : strides) aligned = aligned && s > 0 && s * size % 16 == 0;
  const auto with_mode = [&](auto type, auto ch, auto async) {
    return mode == MOE_GLR_MIX ? f(type, ch, std::true_type{}, async)
                               : f(type, ch, std::false_type{}, async);
  };
  if (dtype == MOE_F32)
    return aligned ? with_mode(float{}, One{}, std::true_type{})
                   : with_mode(float{}, One{}, std::false_type{});
  return aligned ? with_mode(__nv_bfloat16{}, Two{}, std::true_type{})
                 : with_mode(__nv_bfloat16{}, One{}, std::false_type{});
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
      mode, dtype, {g, x, h}, {ld_g, ld_x, D}, [&](auto type, auto ch, auto mix, auto async) {
        using T = decltype(type);
        constexpr int CH = decltype(ch)::value;
        constexpr bool ASYNC = decltype(async)::value, F32 = sizeof(T) == 4;
        const Grid gr = grid_of(N, D, n_seq, 32 * CH);
        ForwardArgs<T> a{{}, seq, D, gr.parts, gr.cluster, static_cast<const T*>(g),
                         static_cast<const T*>(x), ld_g, ld_x, h0, static_cast<T*>(h), h_T,
                         h_chunks, dev_status};
        if (ASYNC) {
          if (int err = encode_map_rows(&a.maps[0], g, F32, D, N, ld_g, 32 * CH, kTile)) return err;
          if (int err = encode_map_rows(&a.maps[1], x, F32, D, N, ld_x, 32 * CH, kTile)) return err;
        }
        return launch(glr_forward_kernel<T, CH, decltype(mix)::value, ASYNC>, gr,
                      kStages * 2 * kTile * 128 + kAlign, a, stream);
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
      mode, dtype, {g, x, dh, dg, dx}, {ld_g, ld_x, D},
      [&](auto type, auto ch, auto mix, auto async) {
        using T = decltype(type);
        constexpr int CH = decltype(ch)::value;
        constexpr bool ASYNC = decltype(async)::value, F32 = sizeof(T) == 4;
        const Grid gr = grid_of(N, D, n_seq, 32 * CH);
        BackwardArgs<T> a{{}, seq, D, gr.parts, gr.cluster, static_cast<const T*>(g),
                          static_cast<const T*>(x), static_cast<const T*>(dh), ld_g, ld_x, h0,
                          h_chunks, dh_T, static_cast<T*>(dg), static_cast<T*>(dx), dh0,
                          dev_status};
        if (ASYNC) {
          const void* in[3] = {g, x, dh};
          const long long ld[3] = {ld_g, ld_x, D};
          for (int i = 0; i < 3; ++i)
            if (int err = encode_map_rows(&a.maps[i], in[i], F32, D, N, ld[i], 32 * CH, kTile))
              return err;
        }
        return launch(glr_backward_kernel<T, CH, decltype(mix)::value, ASYNC>, gr,
                      kStages * 3 * kTile * 128 + kAlign, a, stream);
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
