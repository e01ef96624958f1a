// Gated linear recurrence over packed sequences, forward, backward and one token
// (include/linear_recurrence.h has the formulas).
#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "cluster_room.h"
#include "moe_internal.h"
#include "overlap.cuh"
#include "ptx.cuh"
#include "slots.cuh"

#include "../../include/linear_recurrence.h"

namespace moe {
namespace {

constexpr int kChunk = 64;      // rows between the kept states
constexpr int kWarps = 8;       // warps of a scan block, beside two that join what these form
constexpr int kThreads = 32 * (kWarps + 2);
constexpr int kRows = 8;        // rows of a warp in a tile
constexpr int kTile = kWarps * kRows;
constexpr int kStages = 3;      // tiles in shared memory
constexpr int kBounds = 512;    // bounds of sequences that a block keeps in shared memory

// ------------------------------------------------------------------ what a lane works on
//
// CH channels of one row: two bf16 (one 4-byte word), one bf16 (rows that do not begin on 4-byte
// boundaries) or one fp32; a warp covers 32 CH neighbouring channels.  Two channels are worked on by
// packed fp32 instructions, which halve the issue slots that bound these kernels.
template <int CH>
struct Vec;

template <>
struct Vec<1> {
  float v;
  __device__ __forceinline__ float operator[](int) const { return v; }
};

template <>
struct Vec<2> {
  unsigned long long v;
  __device__ __forceinline__ float operator[](int c) const {
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
    return c ? hi : lo;
  }
};

__device__ __forceinline__ Vec<2> pack(float lo, float hi) {
  Vec<2> r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}

template <int CH>
__device__ __forceinline__ Vec<CH> all(float f) {
  if constexpr (CH == 2)
    return pack(f, f);
  else
    return {f};
}

__device__ __forceinline__ Vec<1> fma(Vec<1> a, Vec<1> b, Vec<1> c) { return {fmaf(a.v, b.v, c.v)}; }
__device__ __forceinline__ Vec<1> operator*(Vec<1> a, Vec<1> b) { return {a.v * b.v}; }
__device__ __forceinline__ Vec<1> operator+(Vec<1> a, Vec<1> b) { return {a.v + b.v}; }
__device__ __forceinline__ Vec<2> fma(Vec<2> a, Vec<2> b, Vec<2> c) {
  Vec<2> r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Vec<2> operator*(Vec<2> a, Vec<2> b) {
  Vec<2> r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Vec<2> operator+(Vec<2> a, Vec<2> b) {
  Vec<2> r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
template <int CH>
__device__ __forceinline__ Vec<CH> operator-(Vec<CH> a, Vec<CH> b) {
  return fma(b, all<CH>(-1.f), a);
}

// The channels of a word of shared memory, of global memory, and back.
template <typename T, int CH>
__device__ __forceinline__ Vec<CH> of_word(uint32_t bits) {
  if constexpr (CH == 2)
    return pack(__uint_as_float(bits << 16), __uint_as_float(bits & 0xffff0000u));
  else
    return {__uint_as_float(sizeof(T) == 4 ? bits : bits << 16)};
}

template <int CH>
__device__ __forceinline__ Vec<CH> read(const float* p) {
  if constexpr (CH == 2)
    return pack(p[0], p[1]);
  else
    return {p[0]};
}
template <int CH>
__device__ __forceinline__ void write(float* p, Vec<CH> v) {
#pragma unroll
  for (int c = 0; c < CH; ++c) p[c] = v[c];
}

__device__ __forceinline__ void put(float* p, Vec<1> v) { __stcs(p, v.v); }
__device__ __forceinline__ void put(__nv_bfloat16* p, Vec<1> v) { *p = __float2bfloat16_rn(v.v); }
__device__ __forceinline__ void put(__nv_bfloat16* p, Vec<2> v) {
  __stcs(reinterpret_cast<unsigned*>(p), pack_bf16x2(v[0], v[1]));
}

// exp(g) as 2^(g log2(e)): two instructions.  The product's rounding costs |g| 2^-24 of the
// result, which matters little where a state is forgotten that fast.  ex2.approx is below the
// true value by 2.3e-8 on average for small arguments, as long memories have them (measured over
// [-0.2, 0]: mean -2.3e-8, rms 3.8e-8; the library's expf, of four times the instructions, has
// -1.6e-9 and 3.1e-8), which would add up over the ~1 / |g| steps that a state lives; the
// exponent carries log2(1 + 2.3e-8) against it.
__device__ __forceinline__ float exp2_approx(float t) {
  float a;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(t));
  return a;
}
template <int CH>
__device__ __forceinline__ Vec<CH> decay_of(Vec<CH> g) {
  const Vec<CH> t = fma(g, all<CH>(1.4426950408889634f), all<CH>(3.3e-8f));
  if constexpr (CH == 2)
    return pack(exp2_approx(t[0]), exp2_approx(t[1]));
  else
    return {exp2_approx(t[0])};
}

// 1 - exp(g) for g <= 0, given a = exp(g).  Near 0, where the difference cancels, -g q(g) with q
// the interpolation of (exp(g) - 1) / g at the five Chebyshev points of [-0.35, 0] (off by 1.4e-8
// at most; 1.1e-7 with the roundings of fp32); beyond, the difference is off by 3.2e-7 at most.
// One channel at a time: the packed instructions run on one of the two fp32 pipes alone, and this
// is where they would fill it (32768 x 2048, mixed, 87 us: a sixth more time packed).
__device__ __forceinline__ float one_minus(float g, float a) {
  float q = fmaf(-0.007211245596408844f, g, -0.04133187234401703f);
  q = fmaf(q, g, -0.16662530601024628f);
  q = fmaf(q, g, -0.49999821186065674f);
  q = fmaf(q, g, -1.f);
  return g > -0.35f ? q * g : 1.f - a;
}
__device__ __forceinline__ Vec<1> one_minus(Vec<1> g, Vec<1> a) { return {one_minus(g.v, a.v)}; }
__device__ __forceinline__ Vec<2> one_minus(Vec<2> g, Vec<2> a) {
  return pack(one_minus(g[0], a[0]), one_minus(g[1], a[1]));
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
  bool bad = q.off[0] != 0;
  for (int s = threadIdx.x; s < q.n_seq; s += blockDim.x)
    bad |= q.off[s] > q.off[s + 1] || q.off[s] < 0 || q.off[s + 1] > q.N;
  if (bad) atomicCAS(dev_status, 0, MOE_ERR_BAD_INDEX);
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

// The sequences that begin and end in the kRows rows of a warp (in shared memory; the walker's
// masks say which rows).
struct Marks {
  int first[kRows], last[kRows];
};

// Walks the bounds of the sequences beside a warp's rows, which come in ascending (DOWN:
// descending) order.  The state is the same in all lanes.  (Others wait meanwhile, for 2 s at most: 2^24
// empty sequences beside the same rows, the most there can be, take 0.18 s.)
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
      if (t0 > 0 && (t0 + q.len - 1u) / q.len * q.len > static_cast<unsigned>(t0 + kRows)) return;
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
// before it are known, once more from the state that these give.  Two more warps join the pairs,
// always in the order of the recurrence: over the warps, over the blocks of the cluster (through
// distributed shared memory) and from step to step; meanwhile the others form the pairs of the
// next tile.  A is -1 for a span in which a sequence begins: what came before is then not used at
// all, not even multiplied by zero.

// (Aligned for the vector store that carries it.)
template <int CH>
struct alignas(8 * CH) Pair {
  Vec<CH> A, H;
  __device__ __forceinline__ bool cut() const { return A[0] < 0.f; }  // of all channels alike
};

template <int CH>
__device__ __forceinline__ void follow(Vec<CH>& h, const Pair<CH>& p) {
  const Vec<CH> on = fma(p.A, h, p.H);
  h = p.cut() ? p.H : on;
}

template <int CH>
__device__ __forceinline__ void append(Pair<CH>& s, const Pair<CH>& p) {
  const Vec<CH> A = s.A * p.A;
  s.A = s.cut() || p.cut() ? all<CH>(-1.f) : A;
  follow(s.H, p);
}

// The clusters' barriers wait for no memory: the first one orders the set-up of the mbarriers, the last
// one the numbers of pairs sent, and both of these have fences of their own (waiting for the copies and
// stores in flight there cost 1 us of a launch).  A warp's threads, one of which may have copied tiles
// on its own, come there together.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A warp's end: no block leaves while another may still write to it.
__device__ __forceinline__ void leave_together(int cluster) {
  if (cluster > 1) {
    cluster_arrive();
    cluster_wait();
  }
}

// What the warps of a block and the blocks of a cluster exchange.  Step n uses the buffers n % 2
// between the warps of a block.  A warp forms its pair of step n + 2 after it has used what the
// joining warps gave it for step n, and they go to step n + 2 when every warp has formed its pair.
// Between blocks it uses the buffers n % 4: a block sends its pair of step n + 4 when its warps
// have used step n + 2, for which it had every block's pair; each block sent that when its warps
// had used step n.  (Those are in dynamic shared memory, behind the tiles: [4][cluster][32].)
template <int CH, int PAIRS>
struct Exchange {
  Pair<CH> warps[2][PAIRS][kWarps][32];
  Vec<CH> state[2][32];  // in front of the block's tile
  Marks marks[2][kWarps];
  uint64_t formed[2], joined[2], received[4];
  uint64_t loaded[kStages], freed[kStages];  // tiles
  int sent[kMaxCluster];  // pairs that each block of the cluster has sent, known from the last barrier on
  int abort;
};

// Position in the ring of tiles, and the parity of its current use.
struct Turn {
  int at = 0;
  unsigned use = 0;
  __device__ __forceinline__ void next() {
    if (++at == kStages) at = 0, use ^= 1;
  }
};

// How long a launch waits.  (drill_*: in the self-test, that warp of the blocks of that rank leaves
// at that step as if a wait of its own had run out.)
struct Waits {
  uint64_t limit_ns = kWaitTimeoutNs;
  int* dev_status = nullptr;
  int drill_rank = -1, drill_warp = -1, drill_step = 0;

  __device__ __forceinline__ int steps_of(int rank, int warp, int steps) const {
    return rank == drill_rank && warp == drill_warp ? min(steps, drill_step) : steps;
  }
  __device__ __forceinline__ void give_up(int* abort) const {
    *reinterpret_cast<volatile int*>(abort) = 1;
    report_status(dev_status, MOE_ERR_TIMEOUT);
  }
};

// Waits, with a limit.  A warp whose wait runs out arrives nowhere and starts no copy any more, so
// nobody who depends on it goes on either, and no buffer is written again before it has been read.
// What is under way then is waited for at the end (drain, drain_pairs).  A joining warp, whose lanes
// all send, leaves at once, its lanes deciding together; a working warp, one lane of which arrives for
// it, goes through its rows in vain, 8 us a step (deciding together at every wait takes 1 % of the
// scans' time, and looking at `abort` once a step as much).
// (Trying again and again without a look at the clock between takes issue slots from the warps that
// work: 2 to 6 %.)
[[nodiscard]] __device__ __forceinline__ bool wait_for(uint64_t* bar, unsigned parity, int* abort,
                                                       const Waits& w) {
  return __all_sync(~0u, mbar_wait(bar, parity, abort, w.limit_ns));
}

// The same for a barrier that other blocks of the cluster complete: what they wrote is acquired at
// their scope.
[[nodiscard]] __device__ __forceinline__ bool wait_for_cluster(uint64_t* bar, unsigned parity,
                                                               int* abort, const Waits& w) {
  return __all_sync(~0u, mbar_wait_cluster(bar, parity, abort, w.limit_ns));
}

// A working warp's lane waits; `alive` becomes false when that runs out.
__device__ __forceinline__ void wait_alive(bool& alive, uint64_t* bar, unsigned parity, int* abort,
                                           const Waits& w) {
  if (!mbar_wait(bar, parity, abort, w.limit_ns)) {
    w.give_up(abort);
    alive = false;
  }
}

// One lane's arrival for its warp.
__device__ __forceinline__ void arrive_warp(uint64_t* bar, bool arrives) {
  __syncwarp();
  if (arrives) mbar_arrive(bar);
}

template <int CH, int PAIRS>
__device__ __forceinline__ void exchange_init(Exchange<CH, PAIRS>& x) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&x.formed[i], kWarps);
      mbar_init(&x.joined[i], 2);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&x.received[i], 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&x.loaded[i], 1);
      mbar_init(&x.freed[i], kWarps);
    }
    x.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
}

// Two warps join.  This is the first one's part of step `it`: the pairs of the block's warps (in
// the order of the recurrence) become the pairs of all that comes before them in the tile; the
// whole tile's is sent to every block of the cluster, this one too, where its bytes count towards
// the barrier of the step.
template <bool DOWN, int CH, int PAIRS>
__device__ __forceinline__ void join_warps(Exchange<CH, PAIRS>& x, Pair<CH>* blocks, int it,
                                           int rank, int cluster, int lane) {
  Pair<CH> pairs[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) pairs[w] = x.warps[it & 1][0][DOWN ? kWarps - 1 - w : w][lane];
  Pair<CH> sum{all<CH>(1.f), all<CH>(0.f)};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    x.warps[it & 1][0][DOWN ? kWarps - 1 - w : w][lane] = sum;
    if (w == 0)
      sum = pairs[0];
    else
      append(sum, pairs[w]);
  }
  Pair<CH>* slot = &blocks[((it & 3) * cluster + rank) * 32 + lane];
  uint64_t* received = &x.received[it & 3];
  if (cluster == 1) {
    *slot = sum;
    arrive_warp(received, lane == 0);
  } else {
    if (lane == 0) mbar_arrive_expect_tx(received, cluster * 32 * sizeof(Pair<CH>));
    for (int q = 0; q < cluster; ++q) {
      const uint32_t to = cluster_addr(slot, q), bar = cluster_addr(received, q);
      if constexpr (CH == 2)
        asm volatile(
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::
                "r"(to),
            "l"(sum.A.v), "l"(sum.H.v), "r"(bar)
            : "memory");
      else
        asm volatile(
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::
                "r"(to),
            "r"(__float_as_uint(sum.A.v)), "r"(__float_as_uint(sum.H.v)), "r"(bar)
            : "memory");
    }
  }
  arrive_warp(&x.joined[it & 1], lane == 0);
}

// The second one's: the state in front of this block's tile, from `state` in front of the step's
// first tile, which moves on over the whole step.
template <int CH, int PAIRS>
[[nodiscard]] __device__ __forceinline__ bool join_blocks(Exchange<CH, PAIRS>& x,
                                                          const Pair<CH>* blocks, int it, int rank,
                                                          int cluster, int lane, Vec<CH>& state,
                                                          const Waits& waits) {
  if (!wait_for_cluster(&x.received[it & 3], it >> 2 & 1, &x.abort, waits)) return false;
  Vec<CH> mine = state;
  const Pair<CH>* pairs = &blocks[(it & 3) * cluster * 32 + lane];
#pragma unroll 4
  for (int q = 0; q < cluster; ++q) {
    if (q == rank) mine = state;
    follow(state, pairs[q * 32]);
  }
  x.state[it & 1][lane] = mine;
  arrive_warp(&x.joined[it & 1], lane == 0);
  return true;
}

// Before the last barrier of the cluster, the first joining warp's part: tells every block how many
// pairs this one has sent.
template <int CH, int PAIRS>
__device__ __forceinline__ void publish_sent(Exchange<CH, PAIRS>& x, int sent, int rank, int cluster,
                                             int lane) {
  if (lane < cluster) st_cluster(cluster_addr(&x.sent[rank], lane), sent);
  fence_cluster();  // (the barrier itself orders nothing)
}

// After it, the second one's in a block that has seen the pairs of `got` steps only: waits, again with
// a limit, for those that are still under way to it, so that none comes when the block has gone.  They
// belong to the four steps from `got` on, as no block sends its pair of step n + 4 before all have used
// step n; the barrier of a step then counts the blocks that did send theirs.
template <int CH, int PAIRS>
__device__ __forceinline__ void drain_pairs(Exchange<CH, PAIRS>& x, int got, int steps, int rank,
                                            int cluster, int lane) {
  if (lane) return;
  constexpr int kBytes = 32 * sizeof(Pair<CH>);
  for (int n = got; n < min(steps, got + 4); ++n) {
    int senders = 0;
    for (int q = 0; q < cluster; ++q) senders += x.sent[q] > n;
    if (senders == 0) continue;
    uint64_t* received = &x.received[n & 3];
    if (x.sent[rank] <= n)
      mbar_arrive_expect_tx(received, senders * kBytes);
    else if (senders < cluster)  // it expects all of them
      mbar_complete_tx(received, (cluster - senders) * kBytes);
    int never = 0;
    mbar_wait_cluster(received, n >> 2 & 1, &never);
  }
}

// ------------------------------------------------------------------ tiles in shared memory
//
// kStages tiles of ARRAYS inputs, each [kTile][32] words: the word of a lane holds its CH channels.
// Where rows begin on 16-byte boundaries, TMA copies whole tiles ahead (ASYNC); elsewhere each
// warp copies its rows through registers when they are asked for.
template <int ARRAYS>
__device__ __forceinline__ uint32_t* tile_at(uint32_t* ring, int stage, int array) {
  return ring + (stage * ARRAYS + array) * kTile * 32;
}

// One thread: the copies of step `it`, the tile at row t0 of the strip at channel d0.
template <int ARRAYS>
__device__ __forceinline__ void load_tile(uint32_t* ring, uint64_t* loaded, const CUtensorMap* maps,
                                          int it, int d0, int t0) {
  const int stage = it % kStages;
  mbar_arrive_expect_tx(&loaded[stage], ARRAYS * kTile * 128);
  const uint64_t policy = l2_policy_evict_first();
  for (int i = 0; i < ARRAYS; ++i)
    tma_load_2d(tile_at<ARRAYS>(ring, stage, i), &maps[i], &loaded[stage], d0, t0, policy);
}

// The same thread at the end, after the copies of the first `issued` steps: none is in flight when the
// block goes, not even in a launch that gave up (again with a limit).
__device__ __forceinline__ void drain(uint64_t* loaded, int issued) {
  int never = 0;
  for (int it = max(0, issued - kStages); it < issued; ++it)
    mbar_wait(&loaded[it % kStages], it / kStages & 1, &never);
}

// A warp's rows from row t0, those outside [lo, hi) as zeros; words[r 32] is row r's.  (Plain loads: the
// kernel is alive before the one in front of it has ended, which may still write these rows then.)
template <int CH, typename T>
__device__ __forceinline__ void copy_rows(uint32_t* words, const T* base, long long stride, int t0,
                                          int lo, int hi, bool on) {
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    uint32_t bits = 0;
    if (on && t0 + r >= lo && t0 + r < hi) {
      const T* from = base + (t0 + r) * stride;
      if constexpr (CH * sizeof(T) == 4) {
        bits = *reinterpret_cast<const uint32_t*>(from);
      } else {
        const T v = *from;
        memcpy(&bits, &v, sizeof v);
      }
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
  for (int i = threadIdx.x; i <= q.n_seq; i += blockDim.x) bounds[i] = q.off[i];
  __syncthreads();
  return {q.N, q.n_seq, bounds, q.len};
}

// to = from for the sequences without rows, from null: zero.  32 of every 32 `groups` sequences; called
// by whole warps.
template <int CH>
__device__ __forceinline__ void hand_on_empty(const Packed& q, const float* from, float* to,
                                              long long D, int d, bool on, int lane, int group,
                                              int groups) {
  for (int s = group * 32; s < q.n_seq; s += groups * 32) {
    const int mine = s + lane;
    unsigned empty =
        __ballot_sync(~0u, mine < q.n_seq && bound_of(q, mine) >= bound_of(q, mine + 1));
    for (; empty; empty &= empty - 1) {
      const long long at = (s + __ffs(empty) - 1) * D + d;
      if (on) write(to + at, from ? read<CH>(from + at) : all<CH>(0.f));
    }
  }
}

// The scans do that when their rows are done (nobody waits for it then), if there are 32 sequences or
// fewer to each of the warps that do it; else this kernel does it behind them, which has blocks by the
// number of sequences (2000 x 256 bf16 in 1000 sequences: 12.4 us with it, 10.4 without).
constexpr int kEmptyThreads = 256;

__global__ void __launch_bounds__(kEmptyThreads)
    glr_empty_kernel(const Packed q, const float* from, float* to, int D) {
  after_previous();
  const int lane = threadIdx.x & 31, warps = kEmptyThreads / 32;
  const int d = blockIdx.y * 32 + lane;
  hand_on_empty<1>(q, from, to, D, d, d < D, lane, blockIdx.x * warps + threadIdx.x / 32,
                   gridDim.x * warps);
}

// ------------------------------------------------------------------ forward
//
// g and x are read once and h is written once.  32768 x 2048 bf16 take 71.0 us, 0.85 of the rate of
// a plain copy (16276 x 2048 fp32 64.1 us, 0.93): what holds the bf16 form back is waiting, between
// instructions (two channels to unpack and gate for each word) and for the other blocks, with 53 %
// of the issue slots used.  24 sequences in as many rows take 81 us, as tiles with bounds go through
// a path of their own.  (16 rows to a warp, without the pairs of the next tile in between: 4 % less
// time with one sequence, 8 % more with 24.)

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
  bool hands_on;  // the states of empty sequences
  Waits waits;
};

template <typename T, int CH, bool MIX, bool ASYNC>
__global__ void __launch_bounds__(kThreads, 2)
    glr_forward_kernel(const __grid_constant__ ForwardArgs<T> p) {
  static_assert(kTile == kChunk, "a tile begins at a kept state");
  extern __shared__ uint32_t dynamic[];
  uint32_t* ring = aligned_128(dynamic);
  Pair<CH>* blocks = reinterpret_cast<Pair<CH>*>(ring + kStages * 2 * kTile * 32);
  __shared__ Exchange<CH, 1> xch;
  __shared__ int bounds[kBounds];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.cluster, part = blockIdx.x / p.cluster;
  const int d = (blockIdx.y * 32 + lane) * CH;
  bool on = d < p.D;  // (of a working warp's first lane: and it has waited for everything)
  const long long D = p.D;
  exchange_init(xch);
  if (p.cluster > 1) cluster_arrive();  // (its way there and back, while the bounds come)
  after_previous();
  const Packed seq = near(p.seq, bounds);
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(seq, p.waits.dev_status);
  const Cut from = part_begin(seq, part, p.parts);
  const int lo = from.row, hi = part_begin(seq, part + 1, p.parts).row;
  const int base = lo / kTile * kTile, step = kTile * p.cluster;
  const int steps = hi > lo ? (hi - base + step - 1) / step : 0;
  const auto tile_row = [&](int it) { return base + (it * p.cluster + rank) * kTile; };
  int issued = 0;  // tiles (the loading warp's)
  const auto load = [&](int it) {
    if (!ASYNC || it >= steps) return;
    if (lane == 0)
      load_tile<2>(ring, xch.loaded, p.maps, it, blockIdx.y * 32 * CH, tile_row(it));
    issued = it + 1;
  };
  // a warp that ends before the last step has given up
  const int own_steps = p.waits.steps_of(rank, warp, steps);
  int done = 0;
  if (warp == kWarps)
    for (int it = 0; it < kStages; ++it) load(it);
  const auto hand_on = [&](int group, int groups) {
    if (p.hands_on) hand_on_empty<CH>(seq, p.h0, p.h_T, D, d, on, lane, group, groups);
  };
  if (p.cluster > 1) cluster_wait();  // every block runs, its barriers set, before one sends

  if (warp == kWarps) {  // joins the warps, and has the tiles loaded
    for (; done < own_steps; ++done) {
      if (!wait_for(&xch.formed[done & 1], done >> 1 & 1, &xch.abort, p.waits)) break;
      join_warps<false>(xch, blocks, done, rank, p.cluster, lane);
      load(done + kStages);  // over the tile that every warp has read
    }
    if (p.cluster > 1) publish_sent(xch, done, rank, p.cluster, lane);
  } else if (warp > kWarps) {  // joins the blocks
    Vec<CH> state = all<CH>(0.f);
    while (done < own_steps &&
           join_blocks(xch, blocks, done, rank, p.cluster, lane, state, p.waits))
      ++done;
    // (without TMA the working warps are short of registers: 8191 x 2046 bf16 38.8 us there, 33.9 here)
    if (!ASYNC) hand_on(blockIdx.x, gridDim.x);
  } else {
    struct Span {
      Vec<CH> a[kRows], b[kRows];  // the rows' decays and inputs
      unsigned firsts, lasts;
    };
    if (own_steps < steps) report_status(p.waits.dev_status, MOE_ERR_TIMEOUT);
    Walker<false> walk;
    walk.start(from);

    // the pair of the span of step `it`
    const auto form = [&](int it, int buf, Span& s) {
      const int t0 = tile_row(it) + warp * kRows;
      Marks& m = xch.marks[buf][warp];
      walk.mark(seq, t0, lane, m, s.firsts, s.lasts);
      uint32_t* g = tile_at<2>(ring, it % kStages, 0) + warp * kRows * 32 + lane;
      uint32_t* x = tile_at<2>(ring, it % kStages, 1) + warp * kRows * 32 + lane;
      if (ASYNC) {
        wait_alive(on, &xch.loaded[it % kStages], it / kStages & 1, &xch.abort, p.waits);
        if (t0 < lo || t0 + kRows > hi) {  // rows of others and padding: the state goes through
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (t0 + r < lo || t0 + r >= hi) g[r * 32] = x[r * 32] = 0;
          fence_proxy_async_smem();  // TMA writes these words next
        }
      } else {
        copy_rows<CH>(g, p.g + d, p.ld_g, t0, lo, hi, on);
        copy_rows<CH>(x, p.x + d, p.ld_x, t0, lo, hi, on);
      }
      Pair<CH> pair{all<CH>(1.f), all<CH>(0.f)};
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const Vec<CH> lg = of_word<T, CH>(g[r * 32]);
        s.b[r] = of_word<T, CH>(x[r * 32]);
        s.a[r] = decay_of(lg);
        if constexpr (MIX) s.b[r] = one_minus(lg, s.a[r]) * s.b[r];
        pair.A = pair.A * s.a[r];
        pair.H = fma(s.a[r], pair.H, s.b[r]);
      }
      if (s.firsts) {  // again, with the initial states
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if ((s.firsts >> r & 1) && p.h0 && on)
            s.b[r] = fma(s.a[r], read<CH>(p.h0 + m.first[r] * D + d), s.b[r]);
          const Vec<CH> next = fma(s.a[r], pair.H, s.b[r]);
          pair.H = s.firsts >> r & 1 ? s.b[r] : next;
        }
        pair.A = all<CH>(-1.f);
      }
      xch.warps[buf][0][warp][lane] = pair;
      arrive_warp(&xch.formed[buf], on && lane == 0);
    };

    // the rows of step `it` from the state in front of them
    const auto finish = [&](int it, int buf, Span& s) {
      const int t0 = tile_row(it) + warp * kRows;
      const Marks& m = xch.marks[buf][warp];
      wait_alive(on, &xch.joined[buf], it >> 1 & 1, &xch.abort, p.waits);
      Vec<CH> h = xch.state[buf][lane];
      follow(h, xch.warps[buf][0][warp][lane]);
      if (warp == 0 && p.h_chunks && on && t0 >= lo && t0 < hi)  // kTile == kChunk
        write(p.h_chunks + t0 / kChunk * D + d, s.firsts & 1 ? all<CH>(0.f) : h);
      T* to = p.h + t0 * D + d;
      if (!(s.firsts | s.lasts) && t0 >= lo && t0 + kRows <= hi) {
#pragma unroll
        for (int r = 0; r < kRows; ++r, to += D) {
          h = fma(s.a[r], h, s.b[r]);
          if (on) put(to, h);
        }
      } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r, to += D) {
          const Vec<CH> next = fma(s.a[r], h, s.b[r]);
          h = s.firsts >> r & 1 ? s.b[r] : next;
          if (on && t0 + r >= lo && t0 + r < hi) {
            put(to, h);
            if ((s.lasts >> r & 1) && p.h_T) write(p.h_T + m.last[r] * D + d, h);
          }
        }
      }
    };

    // always one step's pairs ahead of the states
    Span even, odd;
    for (int it = -1; it < own_steps; it += 2) {
      if (it + 1 < own_steps) form(it + 1, 0, even);
      if (it >= 0) finish(it, 1, odd);
      if (it + 2 < own_steps) form(it + 2, 1, odd);
      if (it + 1 < own_steps) finish(it + 1, 0, even);
    }
    if (ASYNC) hand_on(blockIdx.x * kWarps + warp, gridDim.x * kWarps);
  }
  if (warp >= kWarps && done < steps) p.waits.give_up(&xch.abort);
  if (ASYNC && warp == kWarps && lane == 0) drain(xch.loaded, issued);
  if (p.cluster > 1) {  // no block leaves while another may still write to it
    cluster_arrive();
    cluster_wait();
    if (warp > kWarps && done < steps) drain_pairs(xch, done, steps, rank, p.cluster, lane);
  }
}

// ------------------------------------------------------------------ backward
//
// lam_t = dh_t + back_t, back_{t-1} = a_t lam_t runs the same scan with time reversed: pairs
// (A, H) of back over a span, the last row first.  A tile is one 64-row piece between kept
// states, so the states in front of its rows are formed again from the kept one within the
// block, by pairs of their own.
//
// g, x and dh are read once and dg and dx are written once.  8192 x 4096 bf16 in 6 sequences, mixed,
// take 79 us after the forward's 46 us (124.7 us together, 0.64 of a copy's rate), bound by
// instructions: 65 % of the issue slots, 78 % of the busiest scheduler's.  The gates are formed
// twice; holding them in registers until the pairs are known leaves no room for the overlap of two
// tiles (3 % more).

template <typename T>
struct BackwardArgs {
  CUtensorMap maps[3];  // g, x, dh (ASYNC)
  Packed seq;
  int D, parts, cluster;
  const T *g, *x, *dh;
  long long ld_g, ld_x;
  const float *h0, *h_chunks, *dh_T;
  T *dg, *dx;
  float* dh0;
  bool hands_on;
  Waits waits;
};

template <typename T, int CH, bool MIX, bool ASYNC>
__global__ void __launch_bounds__(kThreads, 2)
    glr_backward_kernel(const __grid_constant__ BackwardArgs<T> p) {
  static_assert(kTile == kChunk, "a tile begins at a kept state");
  extern __shared__ uint32_t dynamic[];
  uint32_t* ring = aligned_128(dynamic);
  Pair<CH>* blocks = reinterpret_cast<Pair<CH>*>(ring + kStages * 3 * kTile * 32);
  // the gradient's pairs, the state's
  __shared__ Exchange<CH, 2> xch;
  __shared__ int bounds[kBounds];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % p.cluster, part = blockIdx.x / p.cluster;
  const int d = (blockIdx.y * 32 + lane) * CH;
  const bool on = d < p.D;
  const long long D = p.D;
  exchange_init(xch);
  if (p.cluster > 1) cluster_arrive();  // (its way there and back, while the bounds come)
  after_previous();
  const Packed seq = near(p.seq, bounds);
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(seq, p.waits.dev_status);
  const Cut until = part_begin(seq, part + 1, p.parts);
  const int lo = part_begin(seq, part, p.parts).row, hi = until.row;
  const int top = (hi + kTile - 1) / kTile * kTile, step = kTile * p.cluster;
  const int steps = hi > lo ? (top - lo / kTile * kTile + step - 1) / step : 0;
  const auto tile_row = [&](int it) { return top - (it * p.cluster + rank + 1) * kTile; };
  int issued = 0;  // tiles (the loading warp's)
  const auto load = [&](int it) {
    if (!ASYNC || it >= steps) return;
    if (lane == 0)
      load_tile<3>(ring, xch.loaded, p.maps, it, blockIdx.y * 32 * CH, tile_row(it));
    issued = it + 1;
  };
  // a warp that ends before the last step has given up
  const int own_steps = p.waits.steps_of(rank, warp, steps);
  int done = 0;
  if (warp == kWarps)
    for (int it = 0; it < kStages; ++it) load(it);
  if (p.cluster > 1) cluster_wait();  // every block runs, its barriers set, before one sends

  if (warp == kWarps) {  // joins the gradient's pairs of the warps, and has the tiles loaded
    while (done < own_steps) {
      if (!wait_for(&xch.formed[done & 1], done >> 1 & 1, &xch.abort, p.waits)) break;
      join_warps<true>(xch, blocks, done, rank, p.cluster, lane);
      const int before = done++ - 1;
      if (ASYNC && before >= 0) {  // that step has been read for the second time
        if (!wait_for(&xch.freed[before % kStages], before / kStages & 1, &xch.abort, p.waits)) break;
        load(before + kStages);
      }
    }
    if (done < steps) p.waits.give_up(&xch.abort);
    if (p.cluster > 1) publish_sent(xch, done, rank, p.cluster, lane);
    if (ASYNC && lane == 0) drain(xch.loaded, issued);
    leave_together(p.cluster);
  } else if (warp > kWarps) {  // joins the state's pairs of the warps, and the blocks
    const auto kept_state = [&](int it) {
      const int tile = tile_row(it);
      return on && it < steps && tile >= 0 ? read<CH>(p.h_chunks + tile / kChunk * D + d)
                                           : all<CH>(0.f);
    };
    Vec<CH> state = all<CH>(0.f), kept = kept_state(0);
    for (; done < own_steps; ++done) {
      if (!wait_for(&xch.formed[done & 1], done >> 1 & 1, &xch.abort, p.waits)) break;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {  // the state in front of each warp's rows, as A
        const Pair<CH> pair = xch.warps[done & 1][1][w][lane];
        xch.warps[done & 1][1][w][lane].A = kept;
        follow(kept, pair);
      }
      kept = kept_state(done + 1);
      if (!join_blocks(xch, blocks, done, rank, p.cluster, lane, state, p.waits)) break;
    }
    if (done < steps) p.waits.give_up(&xch.abort);
    leave_together(p.cluster);
    if (p.cluster > 1 && done < steps) drain_pairs(xch, done, steps, rank, p.cluster, lane);
  } else {
    if (own_steps < steps) report_status(p.waits.dev_status, MOE_ERR_TIMEOUT);
    bool arrives = lane == 0;
    Walker<true> walk;
    walk.start(until);
    const auto state_before = [&](const Marks& m, int r) {  // where a sequence begins
      return on && p.h0 ? read<CH>(p.h0 + m.first[r] * D + d) : all<CH>(0.f);
    };
    const auto grad_after = [&](const Marks& m, int r) {  // where a sequence ends
      return on && p.dh_T ? read<CH>(p.dh_T + m.last[r] * D + d) : all<CH>(0.f);
    };
    // exp(g) of the rows, and 1 - exp(g) where it is needed
    const auto gates = [&](const uint32_t* g, Vec<CH>(&a)[kRows], Vec<CH>(&om)[MIX ? kRows : 1]) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const Vec<CH> lg = of_word<T, CH>(g[r * 32]);
        a[r] = decay_of(lg);
        if constexpr (MIX) om[r] = one_minus(lg, a[r]);
      }
    };

    // the pairs of the span of step `it`
    struct Masks {
      unsigned firsts, lasts;
    };
    Turn form_tile, tile;
    const auto form = [&](int it, int buf, Masks& s) {
      const int t0 = tile_row(it) + warp * kRows;
      Marks& m = xch.marks[buf][warp];
      walk.mark(seq, t0, lane, m, s.firsts, s.lasts);
      Vec<CH> early_s = all<CH>(0.f), early_g = early_s;
      if (s.firsts) early_s = state_before(m, __ffs(s.firsts) - 1);
      if (s.lasts) early_g = grad_after(m, 31 - __clz(s.lasts));
      uint32_t *g = tile_at<3>(ring, form_tile.at, 0) + warp * kRows * 32 + lane,
               *x = tile_at<3>(ring, form_tile.at, 1) + warp * kRows * 32 + lane,
               *dh = tile_at<3>(ring, form_tile.at, 2) + warp * kRows * 32 + lane;
      if (ASYNC) {
        wait_alive(arrives, &xch.loaded[form_tile.at], form_tile.use, &xch.abort, p.waits);
        if (t0 < lo || t0 + kRows > hi) {  // rows of others and padding: all goes through
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (t0 + r < lo || t0 + r >= hi) g[r * 32] = x[r * 32] = dh[r * 32] = 0;
          fence_proxy_async_smem();  // TMA writes these words next
        }
      } else {
        copy_rows<CH>(g, p.g + d, p.ld_g, t0, lo, hi, on);
        copy_rows<CH>(x, p.x + d, p.ld_x, t0, lo, hi, on);
        copy_rows<CH>(dh, p.dh + d, D, t0, lo, hi, on);
      }
      Vec<CH> a[kRows], om[MIX ? kRows : 1];
      gates(g, a, om);
      const auto input = [&](int r) {
        const Vec<CH> xv = of_word<T, CH>(x[r * 32]);
        if constexpr (MIX)
          return om[r] * xv;
        else
          return xv;
      };
      Pair<CH> fwd{all<CH>(1.f), all<CH>(0.f)}, rev = fwd;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        fwd.A = fwd.A * a[r];
        fwd.H = fma(a[r], fwd.H, input(r));
      }
#pragma unroll
      for (int r = kRows - 1; r >= 0; --r) rev.H = a[r] * (of_word<T, CH>(dh[r * 32]) + rev.H);
      rev.A = fwd.A;
      if (const unsigned firsts = s.firsts) {  // again, from the initial states
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (firsts >> r & 1) fwd.H = firsts & ((1 << r) - 1) ? state_before(m, r) : early_s;
          fwd.H = fma(a[r], fwd.H, input(r));
        }
        fwd.A = all<CH>(-1.f);
      }
      if (const unsigned lasts = s.lasts) {  // again, from the final states' gradients
#pragma unroll
        for (int r = kRows - 1; r >= 0; --r) {
          if (lasts >> r & 1) rev.H = lasts >> r > 1 ? grad_after(m, r) : early_g;
          rev.H = a[r] * (of_word<T, CH>(dh[r * 32]) + rev.H);
        }
        rev.A = all<CH>(-1.f);
      }
      xch.warps[buf][0][warp][lane] = rev;
      xch.warps[buf][1][warp][lane] = fwd;
      arrive_warp(&xch.formed[buf], arrives);
      form_tile.next();
    };

    // the gradients of step `it`
    const auto finish = [&](int it, int buf, const Masks& s) {
      const int t0 = tile_row(it) + warp * kRows;
      const Marks& m = xch.marks[buf][warp];
      const unsigned firsts = s.firsts, lasts = s.lasts;
      const uint32_t *g = tile_at<3>(ring, tile.at, 0) + warp * kRows * 32 + lane,
                     *x = tile_at<3>(ring, tile.at, 1) + warp * kRows * 32 + lane,
                     *dh = tile_at<3>(ring, tile.at, 2) + warp * kRows * 32 + lane;
      Vec<CH> a[kRows], om[MIX ? kRows : 1];
      gates(g, a, om);
      wait_alive(arrives, &xch.joined[buf], it >> 1 & 1, &xch.abort, p.waits);
      Vec<CH> back = xch.state[buf][lane], h = xch.warps[buf][1][warp][lane].A;
      follow(back, xch.warps[buf][0][warp][lane]);
      Vec<CH> before[kRows], o_g, o_x;
      const auto advance = [&](int r) {
        const Vec<CH> xv = of_word<T, CH>(x[r * 32]);
        if constexpr (MIX) {
          before[r] = h - xv;
          h = fma(a[r], h, om[r] * xv);
        } else {
          before[r] = h;
          h = fma(a[r], h, xv);
        }
      };
      const auto retreat = [&](int r) {
        const Vec<CH> lam = of_word<T, CH>(dh[r * 32]) + back;
        back = a[r] * lam;
        o_x = lam;
        if constexpr (MIX) o_x = om[r] * lam;
        o_g = back * before[r];
      };
      T* dg = p.dg + (t0 + kRows - 1) * p.ld_g + d;
      T* dx = p.dx + (t0 + kRows - 1) * p.ld_x + d;
      if (!(firsts | lasts) && t0 >= lo && t0 + kRows <= hi) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) advance(r);
#pragma unroll
        for (int r = kRows - 1; r >= 0; --r, dg -= p.ld_g, dx -= p.ld_x) {
          retreat(r);
          if (on) {
            put(dg, o_g);
            put(dx, o_x);
          }
        }
      } else {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (firsts >> r & 1) h = state_before(m, r);
          advance(r);
        }
#pragma unroll
        for (int r = kRows - 1; r >= 0; --r, dg -= p.ld_g, dx -= p.ld_x) {
          if (lasts >> r & 1) back = grad_after(m, r);
          retreat(r);
          if (on && t0 + r >= lo && t0 + r < hi) {
            put(dg, o_g);
            put(dx, o_x);
            if ((firsts >> r & 1) && p.dh0) write(p.dh0 + m.first[r] * D + d, back);
          }
        }
      }
      if (ASYNC) arrive_warp(&xch.freed[tile.at], arrives);
      tile.next();
    };

    // always one step's pairs ahead of the states (one copy of the code: with two, it no longer
    // fits the instruction cache)
    Masks now{}, next{};
    for (int it = -1; it < own_steps; ++it) {
      if (it + 1 < own_steps) form(it + 1, (it + 1) & 1, next);
      if (it >= 0) finish(it, it & 1, now);
      now = next;
    }
    if (p.hands_on)
      hand_on_empty<CH>(seq, p.dh_T, p.dh0, D, d, on, lane, blockIdx.x * kWarps + warp,
                        gridDim.x * kWarps);
    leave_together(p.cluster);
  }
}

// ------------------------------------------------------------------ one token

// Four channels of a row, or one.
__device__ __forceinline__ void get(const float* p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ void get(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xffff0000u);
  v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xffff0000u);
}
__device__ __forceinline__ void get(const float* p, float (&v)[1]) { v[0] = *p; }
__device__ __forceinline__ void get(const __nv_bfloat16* p, float (&v)[1]) {
  v[0] = __bfloat162float(*p);
}
__device__ __forceinline__ void set(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void set(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void set(float* p, const float (&v)[1]) { *p = v[0]; }
__device__ __forceinline__ void set(__nv_bfloat16* p, const float (&v)[1]) {
  *p = __float2bfloat16_rn(v[0]);
}

// V channels to a thread; 64 requests x 4096 channels take 1.9 us in a graph of twelve steps, two
// dependent round trips to memory; 512 requests 4.9 us (0.90 of a copy's rate; L2 holds their states).
// Gates and inputs are on their way while the request's row is looked up, and the state while the
// requests before it are searched for the same row.
constexpr int kStepThreads = 128;

template <typename T, bool MIX, int V>
__global__ void __launch_bounds__(kStepThreads)
    glr_step_kernel(int D, const T* g, long long ld_g, const T* x, long long ld_x,
                    const int* slot, int n_slots, float* state, T* h, int* dev_status) {
  const int b = blockIdx.y, d = (blockIdx.x * kStepThreads + threadIdx.x) * V;
  const bool on = d < D;
  after_previous();
  const int row = slot ? slot[b] : b;
  float lg[V], xv[V], s[V];
  if (on) {
    get(g + b * ld_g + d, lg);
    get(x + b * ld_x + d, xv);
  }
  if (row < 0 || row >= n_slots) {
    if (row != -1 && threadIdx.x == 0 && dev_status) atomicCAS(dev_status, 0, MOE_ERR_BAD_INDEX);
    return;
  }
  float* at = state + static_cast<long long>(row) * D + d;
  if (on) get(at, s);
  if ((slot && named_before(b, row, slot, dev_status)) || !on) return;
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const float a = expf(lg[c]);
    s[c] = fmaf(a, s[c], MIX ? one_minus(lg[c], a) * xv[c] : xv[c]);
  }
  set(at, s);
  set(h + static_cast<long long>(b) * D + d, s);
}

// ------------------------------------------------------------------------ host side

// The self-test's settings, of the calling thread.
thread_local Waits test_waits;

Waits waits_of(int* dev_status) {
  Waits w = test_waits;
  w.dev_status = dev_status;
  return w;
}

// Of fp32 and int32 arrays.
bool misaligned_words(std::initializer_list<const void*> ptrs) {
  return std::any_of(ptrs.begin(), ptrs.end(), [](const void* p) { return misaligned(p, 4); });
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
  if (n_seq > (1 << 24) || N > (1 << 30) || D > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Dynamic shared memory of a scan of `arrays` inputs with clusters of the given size.
template <int CH>
int dynamic_bytes(int arrays, int cluster) {
  return kAlign + kStages * arrays * kTile * 128 + 4 * cluster * 32 * static_cast<int>(sizeof(Pair<CH>));
}

cudaLaunchAttribute cluster_of(int c) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = c;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  return attr;
}

// A cluster beyond what the GPU has room for beside the others would wait for a second round (40
// strips of clusters of 7, where 38 fit, took half as long again as clusters of 6), so the driver
// is asked how many clusters of each size run at once, for each kernel and device the first time that
// this succeeds.  Sizes that it refuses are left out.
template <auto KERNEL, int CH, int ARRAYS>
const ClusterRoom* room_for() {
  static ClusterRoom rooms[64];
  static std::atomic<bool> known[64];
  static std::mutex mu;
  int dev = 0;
  if (launched(cudaGetDevice(&dev)) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  if (known[dev].load(std::memory_order_acquire)) return &rooms[dev];
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev].load(std::memory_order_relaxed)) return &rooms[dev];
  if (launched(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    dynamic_bytes<CH>(ARRAYS, kMaxCluster))) != cudaSuccess)
    return nullptr;
  launched(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
  rooms[dev] = ask_room([](int c, int* n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = dynamic_bytes<CH>(ARRAYS, c);
    cudaLaunchAttribute attr = cluster_of(c);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return launched(cudaOccupancyMaxActiveClusters(n, KERNEL, &cfg)) == cudaSuccess;
  });
  known[dev].store(true, std::memory_order_release);
  return &rooms[dev];
}

int launch_empty(const Packed& seq, const float* from, float* to, int D, cudaStream_t stream) {
  const dim3 grid((seq.n_seq + kEmptyThreads - 1) / kEmptyThreads, (D + 31) / 32);
  return launch_behind(glr_empty_kernel, grid, kEmptyThreads, 0, stream, seq, from, to, D) ==
                 cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

// Launches KERNEL, and behind it, if need be, the one for the empty sequences, which go from `from` to
// `to` (null: not wanted).  HANDS warps of a block hand states on themselves.
template <auto KERNEL, int CH, int ARRAYS, int HANDS, typename Args>
int launch(int N, int D, int n_seq, Args& args, const float* from, float* to, cudaStream_t stream,
           int* launches) {
  const ClusterRoom* room = room_for<KERNEL, CH, ARRAYS>();
  if (!room) return MOE_ERR_CUDA;
  const int strips = (D + 32 * CH - 1) / (32 * CH), tiles = (N + kTile - 1) / kTile;
  const ClusterChoice choice = choose_clusters(*room, strips, tiles, n_seq);
  const int cluster = args.cluster = choice.cluster;
  args.parts = choice.parts;
  const bool empty = args.seq.off && to;
  args.hands_on = empty && n_seq <= 32ll * HANDS * cluster * args.parts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster * args.parts, strips);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = dynamic_bytes<CH>(ARRAYS, cluster);
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2] = {behind_previous(), cluster_of(cluster)};
  cfg.attrs = attrs;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  ++*launches;
  if (launched(cudaLaunchKernelEx(&cfg, KERNEL, args)) != cudaSuccess) return MOE_ERR_CUDA;
  if (!empty || args.hands_on) return MOE_OK;
  ++*launches;
  return launch_empty(args.seq, from, to, D, stream);
}

// Calls f(T{}, channels per lane, mode, ASYNC) for the call's type.  Tensors whose rows all begin
// on 16-byte boundaries (and do not share one row) are copied by TMA; a lane has two bf16 where they
// all begin on 4-byte boundaries (8191 x 2046, forward: 62 us with one, 34 us with two).
template <typename F>
int dispatch(int mode, int dtype, std::initializer_list<const void*> ptrs,
             std::initializer_list<long long> strides, F f) {
  using std::integral_constant;
  using One = integral_constant<int, 1>;
  using Two = integral_constant<int, 2>;
  const int size = dtype == MOE_F32 ? 4 : 2;
  bool aligned = true, even = true;
  for (const void* q : ptrs) aligned = aligned && !misaligned(q, 16), even = even && !misaligned(q, 4);
  for (long long s : strides) aligned = aligned && s > 0 && s * size % 16 == 0, even = even && s % 2 == 0;
  const auto with_mode = [&](auto type, auto ch, auto async) {
    return mode == MOE_GLR_MIX ? f(type, ch, std::true_type{}, async)
                               : f(type, ch, std::false_type{}, async);
  };
  if (dtype == MOE_F32)
    return aligned ? with_mode(float{}, One{}, std::true_type{})
                   : with_mode(float{}, One{}, std::false_type{});
  if (aligned) return with_mode(__nv_bfloat16{}, Two{}, std::true_type{});
  return even ? with_mode(__nv_bfloat16{}, Two{}, std::false_type{})
              : with_mode(__nv_bfloat16{}, One{}, std::false_type{});
}

}  // namespace
}  // namespace moe

extern "C" {

using namespace moe;

int moe_glr_forward(int32_t N, int32_t D, int32_t n_seq, const int32_t* seq_off, int32_t mode,
                    int32_t dtype, const void* g, int64_t ld_g, const void* x, int64_t ld_x,
                    const float* h0, void* h, float* h_T, float* h_chunks, int32_t* dev_status,
                    moe_stream_t stream) {
  if (int e = check_rows(N, D, n_seq, seq_off, mode, dtype, g, ld_g, x, ld_x, h, false)) return e;
  if (misaligned_words({seq_off, h0, h_T, h_chunks, dev_status})) return MOE_ERR_UNSUPPORTED;
  if (N == 1) ld_g = ld_x = D;  // whatever they are
  const Packed seq{N, n_seq, seq_off, seq_off ? 0 : N / n_seq};
  mark_before(MOE_KERNEL_GLR_FWD, stream);
  int launches = 0;
  const int e = dispatch(
      mode, dtype, {g, x, h}, {ld_g, ld_x, D}, [&](auto type, auto ch, auto mix, auto async) {
        using T = decltype(type);
        constexpr int CH = decltype(ch)::value;
        constexpr bool ASYNC = decltype(async)::value, F32 = sizeof(T) == 4;
        ForwardArgs<T> a{{}, seq, D, 1, 1, static_cast<const T*>(g), static_cast<const T*>(x), ld_g, ld_x, h0, static_cast<T*>(h), h_T,
                         h_chunks, false, waits_of(dev_status)};
        if (ASYNC) {
          if (int err = encode_map_rows(&a.maps[0], g, F32, D, N, ld_g, 32 * CH, kTile)) return err;
          if (int err = encode_map_rows(&a.maps[1], x, F32, D, N, ld_x, 32 * CH, kTile)) return err;
        }
        return launch<glr_forward_kernel<T, CH, decltype(mix)::value, ASYNC>, CH, 2,
                      ASYNC ? kWarps : 1>(N, D, n_seq, a, h0, h_T, stream, &launches);
      });
  mark_after(MOE_KERNEL_GLR_FWD, stream);
  count_launches(launches);
  return e;
}

int moe_glr_backward(int32_t N, int32_t D, int32_t n_seq, const int32_t* seq_off, int32_t mode,
                     int32_t dtype, const void* g, int64_t ld_g, const void* x, int64_t ld_x,
                     const float* h0, const float* h_chunks, const void* dh, const float* dh_T,
                     void* dg, void* dx, float* dh0, int32_t* dev_status, moe_stream_t stream) {
  if (int e = check_rows(N, D, n_seq, seq_off, mode, dtype, g, ld_g, x, ld_x, dg, true)) return e;
  if (!h_chunks || !dh || !dx) return MOE_ERR_INVALID_ARG;
  const int size = dtype == MOE_BF16 ? 2 : 4;
  if (misaligned(dh, size) || misaligned(dx, size) ||
      misaligned_words({seq_off, h0, h_chunks, dh_T, dh0, dev_status}))
    return MOE_ERR_UNSUPPORTED;
  if (N == 1) ld_g = ld_x = D;
  const Packed seq{N, n_seq, seq_off, seq_off ? 0 : N / n_seq};
  mark_before(MOE_KERNEL_GLR_BWD, stream);
  int launches = 0;
  const int e = dispatch(
      mode, dtype, {g, x, dh, dg, dx}, {ld_g, ld_x, D},
      [&](auto type, auto ch, auto mix, auto async) {
        using T = decltype(type);
        constexpr int CH = decltype(ch)::value;
        constexpr bool ASYNC = decltype(async)::value, F32 = sizeof(T) == 4;
        BackwardArgs<T> a{{}, seq, D, 1, 1, static_cast<const T*>(g),
                          static_cast<const T*>(x), static_cast<const T*>(dh), ld_g, ld_x, h0,
                          h_chunks, dh_T, static_cast<T*>(dg), static_cast<T*>(dx), dh0,
                          false, waits_of(dev_status)};
        if (ASYNC) {
          const void* in[3] = {g, x, dh};
          const long long ld[3] = {ld_g, ld_x, D};
          for (int i = 0; i < 3; ++i)
            if (int err = encode_map_rows(&a.maps[i], in[i], F32, D, N, ld[i], 32 * CH, kTile))
              return err;
        }
        return launch<glr_backward_kernel<T, CH, decltype(mix)::value, ASYNC>, CH, 3, kWarps>(
            N, D, n_seq, a, dh_T, dh0, stream, &launches);
      });
  mark_after(MOE_KERNEL_GLR_BWD, stream);
  count_launches(launches);
  return e;
}

int moe_glr_step(int32_t B, int32_t D, int32_t mode, int32_t dtype, const void* g, int64_t ld_g,
                 const void* x, int64_t ld_x, const int32_t* slot, int32_t n_slots, float* state,
                 void* h, int32_t* dev_status, moe_stream_t stream) {
  if (int e = check_rows(B, D, 1, nullptr, mode, dtype, g, ld_g, x, ld_x, h, false)) return e;
  if (!state || n_slots <= 0 || (!slot && B > n_slots)) return MOE_ERR_INVALID_ARG;
  if (misaligned_words({slot, state, dev_status})) return MOE_ERR_UNSUPPORTED;
  if (B > kMaxSlots) return MOE_ERR_UNSUPPORTED;  // (and no more fit a grid's second dimension)
  // four channels to a thread where every row begins on the boundary of four values (64 requests x
  // 4096 channels, bf16, in a graph of twelve steps: 2.5 us with one, 1.9 us with four; 512 requests:
  // 10.9 and 4.9)
  const int size = dtype == MOE_BF16 ? 2 : 4;
  const bool four = D % 4 == 0 && ld_g % 4 == 0 && ld_x % 4 == 0 && !misaligned(g, 4 * size) &&
                    !misaligned(x, 4 * size) && !misaligned(h, 4 * size) && !misaligned(state, 16);
  const int width = kStepThreads * (four ? 4 : 1);
  const dim3 grid((D + width - 1) / width, B);
  mark_before(MOE_KERNEL_GLR_STEP, stream);
  cudaError_t err = cudaSuccess;
  const auto run = [&](auto type, auto mix, auto v) {
    using T = decltype(type);
    err = launch_behind(glr_step_kernel<T, decltype(mix)::value, decltype(v)::value>, grid, kStepThreads,
                        0, stream, D, static_cast<const T*>(g), ld_g, static_cast<const T*>(x), ld_x,
                        slot, n_slots, state, static_cast<T*>(h), dev_status);
  };
  const auto with_width = [&](auto type, auto mix) {
    if (four)
      run(type, mix, std::integral_constant<int, 4>{});
    else
      run(type, mix, std::integral_constant<int, 1>{});
  };
  const auto with_mode = [&](auto type) {
    if (mode == MOE_GLR_MIX)
      with_width(type, std::true_type{});
    else
      with_width(type, std::false_type{});
  };
  if (dtype == MOE_BF16)
    with_mode(__nv_bfloat16{});
  else
    with_mode(float{});
  mark_after(MOE_KERNEL_GLR_STEP, stream);
  count_launches(1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_selftest_recurrence_waits(int32_t limit_ms, int32_t rank, int32_t warp, int32_t step) {
  if (limit_ms < 0 || limit_ms > 2000 || (limit_ms && step < 0)) return MOE_ERR_INVALID_ARG;
  test_waits = Waits{};
  if (limit_ms) {
    test_waits.limit_ns = limit_ms * 1000000ull;
    test_waits.drill_rank = rank;
    test_waits.drill_warp = warp;
    test_waits.drill_step = step;
  }
  return MOE_OK;
}

}  // extern "C"
