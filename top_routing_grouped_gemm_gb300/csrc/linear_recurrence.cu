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
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;  // blocks of a cluster (the portable limit)
constexpr int kForwardRows = 16;  // rows of a warp in a tile
constexpr int kBackwardRows = 8;
constexpr int kForwardStages = 2;   // tiles in shared memory
constexpr int kBackwardStages = 3;  // (one is still read while the next but one arrives)
constexpr int kBounds = 1024;   // bounds of sequences that a block keeps in shared memory

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

// Reports a wait that ran out.  The rest of the launch goes on without waiting (its results are
// then wrong), so every barrier still gets all its threads.
__device__ __forceinline__ void give_up(int* abort, int* dev_status) {
  *reinterpret_cast<volatile int*>(abort) = 1;
  report_status(dev_status, MOE_ERR_TIMEOUT);
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

template <int CH, typename Tiles>
__device__ __forceinline__ void exchange_init(Exchange<CH>& x, int cluster, const Tiles& tiles) {
  tiles.init();
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
// goes on over the whole step.  `order` is the warp's place in the order of the recurrence.  At
// `meet` all warps have read the step's tile once.
template <int CH, typename Meet>
__device__ __forceinline__ void join(Exchange<CH>& x, int it, const Pair<CH>& mine, int order,
                                     int rank, int cluster, int lane, float (&state)[CH],
                                     float (&carry)[CH], int* dev_status, Meet meet) {
  const int buf = it & 1;
  x.warps[buf][order][lane] = mine;
  if (cluster > 1 && threadIdx.x == 0)
    mbar_arrive_expect_tx(&x.full[buf], cluster * 32 * sizeof(Pair<CH>));
  __syncthreads();
  meet();
  if (cluster > 1) {
    if (order == 0) {
      Pair<CH> sum = mine;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) append(sum, x.warps[buf][w][lane]);
      publish(x, buf, sum, rank, cluster, lane);
    }
    if (!mbar_wait(&x.full[buf], (it >> 1) & 1, &x.abort)) give_up(&x.abort, dev_status);
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

// ------------------------------------------------------------------ tiles in shared memory
//
// STAGES tiles of ARRAYS inputs, each [ROWS][32] words: the word of a lane holds its CH channels.
// Where rows begin on 16-byte boundaries, one thread has TMA copy whole tiles two steps ahead
// (ASYNC); elsewhere each warp copies its rows through registers when they are asked for.
template <int ARRAYS, int STAGES, int ROWS, bool ASYNC>
struct Tiles {
  uint32_t* words;
  uint64_t* full;  // [STAGES] barriers (ASYNC)

  __device__ __forceinline__ uint32_t* at(int stage, int array) const {
    return words + (stage * ARRAYS + array) * ROWS * 32;
  }

  __device__ __forceinline__ void init() const {
    if (ASYNC && threadIdx.x == 0)
      for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1);
  }

  // One thread: the copies of step `it`, the tile at row t0 of the strip at channel d0.
  __device__ __forceinline__ void load(int it, const CUtensorMap* maps, int d0, int t0) const {
    const int stage = it % STAGES;
    mbar_arrive_expect_tx(&full[stage], ARRAYS * ROWS * 128);
    const uint64_t policy = l2_policy_evict_first();
    for (int i = 0; i < ARRAYS; ++i) tma_load_2d(at(stage, i), &maps[i], &full[stage], d0, t0, policy);
  }

  __device__ __forceinline__ bool wait(int it, volatile int* abort) const {
    return mbar_wait(&full[it % STAGES], (it / STAGES) & 1, abort);
  }

  // After a launch that gave up: the copies still in flight (again with a limit).
  __device__ __forceinline__ void drain(int steps, volatile int* abort) const {
    if (!*abort || threadIdx.x != 0) return;
    int never = 0;
    for (int it = max(0, steps - STAGES); it < steps; ++it) wait(it, &never);
  }
};

// R rows of one warp from row t0, those outside [lo, hi) as zeros; words[r 32] is row r's.
template <int R, typename T>
__device__ __forceinline__ void copy_rows(uint32_t* words, const T* base, long long stride, int t0,
                                          int lo, int hi, bool on) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
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
  constexpr int R = kForwardRows, ROWS = kWarps * R;
  extern __shared__ uint32_t dynamic[];
  uint32_t* ring = aligned_128(dynamic);
  __shared__ uint64_t full[kForwardStages];
  __shared__ Exchange<CH> xch;
  __shared__ Marks<ROWS> marks;
  __shared__ int bounds[kBounds];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.cluster, part = blockIdx.x / p.cluster;
  const int d = (blockIdx.y * 32 + lane) * CH;
  const bool on = d < p.D;
  const long long D = p.D;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seq, p.dev_status);
  const Packed seq = near(p.seq, bounds);
  const int lo = part_begin(seq, part, p.parts), hi = part_begin(seq, part + 1, p.parts);

  const int base = lo / ROWS * ROWS, step = ROWS * p.cluster;
  const int steps = hi > lo ? (hi - base + step - 1) / step : 0;
  const Tiles<2, kForwardStages, ROWS, ASYNC> tiles{ring, full};
  const auto load = [&](int it) {  // one thread
    if (it < steps)
      tiles.load(it, p.maps, blockIdx.y * 32 * CH, base + (it * p.cluster + rank) * ROWS);
  };
  exchange_init(xch, p.cluster, tiles);
  if (ASYNC && threadIdx.x == 0)
    for (int it = 0; it < kForwardStages; ++it) load(it);

  if (seq.off && p.h_T && on)  // empty sequences hand their state on
    for (int s = blockIdx.x * kWarps + warp; s < seq.n_seq; s += gridDim.x * kWarps)
      if (bound_of(seq, s) >= bound_of(seq, s + 1))
#pragma unroll
        for (int c = 0; c < CH; ++c) p.h_T[s * D + d + c] = p.h0 ? p.h0[s * D + d + c] : 0.f;

  Walker<false, ROWS> walk;
  walk.start(seq);
  float state[CH] = {};
  for (int it = 0; it < steps; ++it) {
    const int tile = base + (it * p.cluster + rank) * ROWS, t0 = tile + warp * R;
    unsigned firsts = 0, lasts = 0;
    const bool marked = walk.mark(seq, tile, marks);
    if (marked) {
      __syncthreads();
      const int mine = warp * R + (lane & (R - 1));
      firsts = __ballot_sync(~0u, marks.first[mine] >= 0) & ((1u << R) - 1);
      lasts = __ballot_sync(~0u, marks.last[mine] >= 0) & ((1u << R) - 1);
    }
    uint32_t* raw_g = tiles.at(it % kForwardStages, 0) + warp * R * 32 + lane;
    uint32_t* raw_x = tiles.at(it % kForwardStages, 1) + warp * R * 32 + lane;
    const bool whole = t0 >= lo && t0 + R <= hi;
    if (ASYNC) {
      if (!tiles.wait(it, &xch.abort)) give_up(&xch.abort, p.dev_status);
      if (!whole) {  // rows of others and padding: the state goes through
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (t0 + r < lo || t0 + r >= hi) raw_g[r * 32] = raw_x[r * 32] = 0;
        fence_proxy_async_smem();  // TMA writes these words next
      }
    } else {
      copy_rows<R>(raw_g, p.g + d, p.ld_g, t0, lo, hi, on);
      copy_rows<R>(raw_x, p.x + d, p.ld_x, t0, lo, hi, on);
    }

    // the span's pair; a[r], b[r] stay for the second pass
    float a[R][CH], b[R][CH], h[CH];
    Pair<CH> pair;
#pragma unroll
    for (int c = 0; c < CH; ++c) pair.A[c] = 1.f, pair.H[c] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t wg = raw_g[r * 32], wx = raw_x[r * 32];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const float lg = get(wg, c, T()), xv = get(wx, c, T());
        a[r][c] = decay_of(lg);
        b[r][c] = MIX ? one_minus(lg, a[r][c]) * xv : xv;
        pair.A[c] *= a[r][c];
        pair.H[c] = fmaf(a[r][c], pair.H[c], b[r][c]);
      }
    }
    if (firsts) {  // again, with the initial states
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if ((firsts >> r & 1) && p.h0 && on)
            b[r][c] = fmaf(a[r][c], p.h0[marks.first[warp * R + r] * D + d + c], b[r][c]);
          pair.H[c] = firsts >> r & 1 ? b[r][c] : fmaf(a[r][c], pair.H[c], b[r][c]);
        }
#pragma unroll
      for (int c = 0; c < CH; ++c) pair.A[c] = -1.f;
    }

    join(xch, it, pair, warp, rank, p.cluster, lane, state, h, p.dev_status, [&] {
      if (ASYNC && threadIdx.x == 0) load(it + kForwardStages);  // over the tile just read
    });

    if (p.h_chunks && on && t0 % kChunk == 0 && t0 >= lo && t0 < hi)
#pragma unroll
      for (int c = 0; c < CH; ++c) p.h_chunks[t0 / kChunk * D + d + c] = firsts & 1 ? 0.f : h[c];
    T* out = p.h + t0 * D + d;
    if (!marked && whole) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int c = 0; c < CH; ++c) h[c] = fmaf(a[r][c], h[c], b[r][c]);
        if (on) put(out, h);
        out += D;
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
          h[c] = firsts >> r & 1 ? b[r][c] : fmaf(a[r][c], h[c], b[r][c]);
        if (on && t0 + r >= lo && t0 + r < hi) {
          put(out + r * D, h);
          if ((lasts >> r & 1) && p.h_T)
#pragma unroll
            for (int c = 0; c < CH; ++c) p.h_T[marks.last[warp * R + r] * D + d + c] = h[c];
        }
      }
    }
    if (marked) __syncthreads();  // the marks are rewritten
  }
  if (ASYNC) tiles.drain(steps, &xch.abort);
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
  constexpr int R = kBackwardRows, ROWS = kWarps * R;
  static_assert(ROWS == kChunk, "a tile begins at a kept state");
  extern __shared__ uint32_t dynamic[];
  uint32_t* ring = aligned_128(dynamic);
  __shared__ uint64_t full[kBackwardStages];
  __shared__ Exchange<CH> xch;
  __shared__ Pair<CH> ahead[2][kWarps][32];  // the forward pairs of the warps
  __shared__ Marks<ROWS> marks;
  __shared__ int bounds[kBounds];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.cluster, part = blockIdx.x / p.cluster;
  const int d = (blockIdx.y * 32 + lane) * CH;
  const bool on = d < p.D;
  const long long D = p.D;
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(p.seq, p.dev_status);
  const Packed seq = near(p.seq, bounds);
  const int lo = part_begin(seq, part, p.parts), hi = part_begin(seq, part + 1, p.parts);

  const int top = (hi + ROWS - 1) / ROWS * ROWS, step = ROWS * p.cluster;
  const int steps = hi > lo ? (top - lo / ROWS * ROWS + step - 1) / step : 0;
  const Tiles<3, kBackwardStages, ROWS, ASYNC> tiles{ring, full};
  const auto load = [&](int it) {  // one thread
    if (it < steps)
      tiles.load(it, p.maps, blockIdx.y * 32 * CH, top - (it * p.cluster + rank + 1) * ROWS);
  };
  exchange_init(xch, p.cluster, tiles);
  if (ASYNC && threadIdx.x == 0)
    for (int it = 0; it < kBackwardStages - 1; ++it) load(it);
  const auto kept_state = [&](int it, float(&k)[CH]) {
    const int tile = top - (it * p.cluster + rank + 1) * ROWS;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      k[c] = on && it < steps && tile >= 0 ? p.h_chunks[tile / kChunk * D + d + c] : 0.f;
  };

  if (seq.off && p.dh0 && on)  // empty sequences hand their gradient on
    for (int s = blockIdx.x * kWarps + warp; s < seq.n_seq; s += gridDim.x * kWarps)
      if (bound_of(seq, s) >= bound_of(seq, s + 1))
#pragma unroll
        for (int c = 0; c < CH; ++c) p.dh0[s * D + d + c] = p.dh_T ? p.dh_T[s * D + d + c] : 0.f;

  Walker<true, ROWS> walk;
  walk.start(seq);
  float state[CH] = {}, kept[CH];
  kept_state(0, kept);
  for (int it = 0; it < steps; ++it) {
    const int tile = top - (it * p.cluster + rank + 1) * ROWS, t0 = tile + warp * R;
    unsigned firsts = 0, lasts = 0;
    const bool marked = walk.mark(seq, tile, marks);
    if (marked) {
      __syncthreads();
      const int mine = warp * R + (lane & (R - 1));
      firsts = __ballot_sync(~0u, marks.first[mine] >= 0) & ((1u << R) - 1);
      lasts = __ballot_sync(~0u, marks.last[mine] >= 0) & ((1u << R) - 1);
    }
    uint32_t* raw[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) raw[i] = tiles.at(it % kBackwardStages, i) + warp * R * 32 + lane;
    const bool whole = t0 >= lo && t0 + R <= hi;
    if (ASYNC) {
      if (!tiles.wait(it, &xch.abort)) give_up(&xch.abort, p.dev_status);
      if (!whole) {  // rows of others and padding: state and gradient go through
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (t0 + r < lo || t0 + r >= hi)
            raw[0][r * 32] = raw[1][r * 32] = raw[2][r * 32] = 0;
        fence_proxy_async_smem();  // TMA writes these words next
      }
    } else {
      copy_rows<R>(raw[0], p.g + d, p.ld_g, t0, lo, hi, on);
      copy_rows<R>(raw[1], p.x + d, p.ld_x, t0, lo, hi, on);
      copy_rows<R>(raw[2], p.dh + d, D, t0, lo, hi, on);
    }
    const auto x = [&](int r, int c) { return get(raw[1][r * 32], c, T()); };
    const auto dh = [&](int r, int c) { return get(raw[2][r * 32], c, T()); };
    const auto state_before = [&](int r, int c) {  // of the sequence that begins in row r
      return on && p.h0 ? p.h0[marks.first[warp * R + r] * D + d + c] : 0.f;
    };
    const auto grad_after = [&](int r, int c) {  // of the sequence that ends in row r
      return on && p.dh_T ? p.dh_T[marks.last[warp * R + r] * D + d + c] : 0.f;
    };

    float a[R][CH], om[MIX ? R : 1][CH] = {};  // exp(g), 1 - exp(g)
    const auto input = [&](int r, int c) { return MIX ? om[r][c] * x(r, c) : x(r, c); };
    Pair<CH> fwd, rev;
#pragma unroll
    for (int c = 0; c < CH; ++c) fwd.A[c] = 1.f, fwd.H[c] = rev.H[c] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const float lg = get(raw[0][r * 32], c, T());
        a[r][c] = decay_of(lg);
        if (MIX) om[r][c] = one_minus(lg, a[r][c]);
        fwd.A[c] *= a[r][c];
        fwd.H[c] = fmaf(a[r][c], fwd.H[c], input(r, c));
      }
#pragma unroll
    for (int r = R - 1; r >= 0; --r)
#pragma unroll
      for (int c = 0; c < CH; ++c) rev.H[c] = a[r][c] * (dh(r, c) + rev.H[c]);
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
          rev.H[c] = a[r][c] * (dh(r, c) + rev.H[c]);
          rev.A[c] = -1.f;
        }
    }
    ahead[it & 1][warp][lane] = fwd;
    float kept_next[CH];
    kept_state(it + 1, kept_next);

    float back[CH];
    join(xch, it, rev, kWarps - 1 - warp, rank, p.cluster, lane, state, back, p.dev_status, [&] {
      if (ASYNC && threadIdx.x == 0) load(it + kBackwardStages - 1);  // over the step before's tile
    });

    float h[CH], before[R][CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) h[c] = kept[c];
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
      if (w < warp) follow(h, ahead[it & 1][w][lane]);
    T* dg = p.dg + (t0 + R - 1) * p.ld_g + d;
    T* dx = p.dx + (t0 + R - 1) * p.ld_x + d;
    if (!marked && whole) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          before[r][c] = MIX ? h[c] - x(r, c) : h[c];
          h[c] = fmaf(a[r][c], h[c], input(r, c));
        }
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        float o_g[CH], o_x[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const float lam = dh(r, c) + back[c];
          back[c] = a[r][c] * lam;
          o_x[c] = MIX ? om[r][c] * lam : lam;
          o_g[c] = back[c] * before[r][c];
        }
        if (on) {
          put(dg, o_g);
          put(dx, o_x);
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
          before[r][c] = MIX ? h[c] - x(r, c) : h[c];
          h[c] = fmaf(a[r][c], h[c], input(r, c));
        }
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        float o_g[CH], o_x[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (lasts >> r & 1) back[c] = grad_after(r, c);
          const float lam = dh(r, c) + back[c];
          back[c] = a[r][c] * lam;
          o_x[c] = MIX ? om[r][c] * lam : lam;
          o_g[c] = back[c] * before[r][c];
        }
        if (on && t0 + r >= lo && t0 + r < hi) {
          put(dg - (R - 1 - r) * p.ld_g, o_g);
          put(dx - (R - 1 - r) * p.ld_x, o_x);
          if ((firsts >> r & 1) && p.dh0)
#pragma unroll
            for (int c = 0; c < CH; ++c) p.dh0[marks.first[warp * R + r] * D + d + c] = back[c];
        }
      }
    }
    if (marked) __syncthreads();  // the marks are rewritten
#pragma unroll
    for (int c = 0; c < CH; ++c) kept[c] = kept_next[c];
  }
  if (ASYNC) tiles.drain(steps, &xch.abort);
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
        constexpr int CH = decltype(ch)::value, ROWS = kForwardRows * kWarps;
        constexpr bool ASYNC = decltype(async)::value, F32 = sizeof(T) == 4;
        const Grid gr = grid_of(N, D, n_seq, 32 * CH, ROWS);
        ForwardArgs<T> a{{}, seq, D, gr.parts, gr.cluster, static_cast<const T*>(g),
                         static_cast<const T*>(x), ld_g, ld_x, h0, static_cast<T*>(h), h_T,
                         h_chunks, dev_status};
        if (ASYNC) {
          if (int err = encode_map_rows(&a.maps[0], g, F32, D, N, ld_g, 32 * CH, ROWS)) return err;
          if (int err = encode_map_rows(&a.maps[1], x, F32, D, N, ld_x, 32 * CH, ROWS)) return err;
        }
        return launch(glr_forward_kernel<T, CH, decltype(mix)::value, ASYNC>, gr,
                      kForwardStages * 2 * ROWS * 128 + kAlign, a, stream);
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
        const Grid gr = grid_of(N, D, n_seq, 32 * CH, kChunk);
        BackwardArgs<T> a{{}, seq, D, gr.parts, gr.cluster, static_cast<const T*>(g),
                          static_cast<const T*>(x), static_cast<const T*>(dh), ld_g, ld_x, h0,
                          h_chunks, dh_T, static_cast<T*>(dg), static_cast<T*>(dx), dh0,
                          dev_status};
        if (ASYNC) {
          const void* in[3] = {g, x, dh};
          const long long ld[3] = {ld_g, ld_x, D};
          for (int i = 0; i < 3; ++i)
            if (int err = encode_map_rows(&a.maps[i], in[i], F32, D, N, ld[i], 32 * CH, kChunk))
              return err;
        }
        return launch(glr_backward_kernel<T, CH, decltype(mix)::value, ASYNC>, gr,
                      kBackwardStages * 3 * kChunk * 128 + kAlign, a, stream);
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
