// The experts' products with 4-bit weights for few tokens (include/moe_block.h has the formulas).
//
// A weight w = s (c - z) is read once for all rows (tokens) of its expert, and the time is that of
// reading; what has to be small beside it is the number of instructions for each weight.  The products
// run on the tensor cores with 16 weight rows against 8 tokens, 16 columns at a time, fp16 operands and
// fp32 sums: a code 0 .. 15 in the lowest bits of a half-word IS the fp16 value code 2^-24 (a subnormal
// one), and in the next four bits 16 times that, so eight codes become operands by one shift and four
// masks.  A token's values are scaled beforehand by a power of two (x by one for its row, h by one for
// each 64 values), so that fp16 holds what bf16 had; those that go with the 16-fold codes are divided by
// 16.  Zeros are taken off the sums: sum s (c - z) x = s (sum c x - z sum x), the sums of x being formed
// once beforehand.  (Codes made 16 + code in bf16, less 16 + zero, took 71 instructions for 16 x 64
// weights, where half the pipes' rate holds for 40 of them.  e4m3 operands, which a code in a byte is too,
// are turned into others first on this GPU: 108 instructions.)
//
// Now it is 56 for gate and up, 80 for down, whose operand has two parts.  One token through 16 of 896
// experts of 4096 x 1024 takes 31.5 us (104 MB, 15 us of reading), 64 tokens that crowd on few experts
// 500 us (358), 32 tokens through experts of 2048 x 512 with zeros 157 us (97): warps are issuing half of
// the time, in turn with what they wait for.
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "moe_internal.h"
#include "overlap.cuh"
#include "ptx.cuh"

#include "../../include/moe_block.h"

namespace moe {
namespace {

constexpr int kStrip = 16;       // weight rows of a product
constexpr int kTile = 64;        // weights of a row that a lane's 16 bytes are part of
constexpr int kMaxSlots = 16384;
constexpr int kMaxWidth = 1 << 20;
constexpr int kMaxExperts = 1024;
// Rows of an expert that its weights are read once for; more of them are taken in several chunks.  (Where
// experts have many rows the second reading is of the L2: 32 rows to a chunk, with as many values to
// wait for as a lane then has, took 160 us instead of 94 for 16 tokens x 8 of 64 experts, 4096 x 1024,
// 252 instead of 138 for 64 and 4153 instead of 2654 for 2048.)
constexpr int kChunk = 8;
constexpr int kXParts = 1, kHParts = 2;  // fp16 values for one of x, of h
constexpr int kWarps = 8, kMaxWarps = 16;  // to a block
constexpr int kSharedPerSm = 228 * 1024, kSharedPerBlock = 227 * 1024;
constexpr int kDrillGroup = 32;  // of the weights (without zeros) that the waits are tested with

// ---------------------------------------------------------------- layout
// A tile of 16 rows x 64 columns takes 512 bytes, 16 to a lane: lane 4 g + t holds rows g and g + 8,
// columns 8 t .. 8 t + 7 of each half of the tile, as the words (g, first half), (g + 8, first half),
// (g, second half), (g + 8, second half).  Within a word column 2 p + i of its eight is nibble
// p + 4 i.  (The order of the columns means nothing to a product, as long as the tokens' operand has the
// same.)  A tile's rows are those of a strip; strips, then experts follow one another.  Scales: for 16
// rows and a group of columns, 4096 times the scales of rows g and g + 8 for each g; with zeros, each
// scale is followed by its zero, in bf16.

__global__ void w4_pack_kernel(int rows, int cols, long long words, const uint8_t* codes,
                               uint32_t* out) {
  after_previous();
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < words;
       i += step) {
    const int word = static_cast<int>(i & 3), lane = static_cast<int>(i >> 2 & 31);
    const long long tile = i >> 7;
    const int tiles = cols / kTile;
    const long long strip = tile / tiles;  // over all experts: rows is a multiple of 16
    const long long row = strip * kStrip + lane / 4 + word % 2 * 8;
    const int col = static_cast<int>(tile % tiles) * kTile + word / 2 * 32 + lane % 4 * 8;
    const uint8_t* from = codes + (row * cols + col) / 2;
    uint32_t w = 0;
    for (int c = 0; c < 8; ++c) w |= (from[c / 2] >> (c % 2 * 4) & 15u) << (c / 2 * 4 + c % 2 * 16);
    out[i] = w;
  }
}

__global__ void w4_pack_scales_kernel(int groups, long long entries, const __nv_bfloat16* scales,
                                      const uint8_t* zeros, __nv_bfloat16* out) {
  after_previous();
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; i < entries;
       i += step) {
    const int in = static_cast<int>(i & 15);  // 2 g + half
    const long long at = i >> 4;
    const long long row = at / groups * kStrip + in / 2 + in % 2 * 8;
    const long long from = row * groups + at % groups;
    const __nv_bfloat16 scale = __float2bfloat16_rn(4096.f * __bfloat162float(scales[from]));
    if (zeros) {
      out[2 * i] = scale;
      out[2 * i + 1] = __float2bfloat16_rn(static_cast<float>(zeros[from] & 15));
    } else {
      out[i] = scale;
    }
  }
}

// ---------------------------------------------------------------- the slots by expert
// Chunks of at most kChunk rows of one expert; a row is a slot, in the slots' order within an expert.
struct Groups {
  const int* idx;  // [slots] the slots' experts; a single token's slots are chunks as they are
  const float* gate;
  int slots, E, single;
  int* count;     // [1] chunks
  int* expert;    // [E + slots / kChunk]
  int* first;     // [...] its first row
  int* rows;      // [...] how many
  int* row_slot;  // [slots]
  float* row_gate;
  int* slot_row;  // [slots], -1 for a bad expert

  __device__ __forceinline__ bool good(int slot) const { return idx[slot] >= 0 && idx[slot] < E; }
  __device__ __forceinline__ int chunks() const { return single ? slots : *count; }
  // The expert of chunk c, its first row and how many there are (none for a bad expert).
  __device__ __forceinline__ int expert_of(int c) const {
    return single ? (good(c) ? idx[c] : 0) : expert[c];
  }
  __device__ __forceinline__ int first_of(int c) const { return single ? c : first[c]; }
  __device__ __forceinline__ int rows_of(int c) const { return single ? good(c) : rows[c]; }
  __device__ __forceinline__ int slot_of(int row) const { return single ? row : row_slot[row]; }
  __device__ __forceinline__ float gate_of(int row) const { return single ? gate[row] : row_gate[row]; }
};

__device__ __forceinline__ int block_scan(int v, int* sums) {  // exclusive, 1024 threads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int in = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int below = __shfl_up_sync(~0u, in, o);
    if (lane >= o) in += below;
  }
  if (lane == 31) sums[warp] = in;
  __syncthreads();
  if (warp == 0) {
    int all = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int below = __shfl_up_sync(~0u, all, o);
      if (lane >= o) all += below;
    }
    sums[lane] = all;
  }
  __syncthreads();
  const int before = warp ? sums[warp - 1] : 0;
  __syncthreads();
  return before + in - v;
}

// One block of 1024.  The first `warps` of its warps have a part of the slots each, 32 at a time.
__device__ void group_slots(const Groups& g, int warps, int* dev_status) {
  extern __shared__ unsigned short seen[];  // [warps][E]: slots of the expert in the warp's part
  __shared__ int sums[32], start[kMaxExperts];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = g.E;
  const int part = (g.slots + warps * 32 - 1) / (warps * 32) * 32;
  for (int i = threadIdx.x; i < warps * E; i += 1024) seen[i] = 0;
  __syncthreads();
  const int lo = warp * part, hi = warp < warps ? min(lo + part, g.slots) : 0;
  const auto pass = [&](auto put) {
    for (int at = lo; at < hi; at += 32) {
      const int slot = at + lane;
      const int e = slot < hi && g.good(slot) ? g.idx[slot] : -1;
      const unsigned same = __match_any_sync(~0u, e);
      const int rank = __popc(same & ((1u << lane) - 1));
      const int before = e >= 0 ? seen[warp * E + e] : 0;
      __syncwarp();
      if (e >= 0 && rank == 0) seen[warp * E + e] = before + __popc(same);
      __syncwarp();
      if (slot < hi) put(slot, e, before + rank);
    }
  };
  pass([&](int slot, int, int) {
    if (!g.good(slot)) report_status(dev_status, MOE_ERR_BAD_INDEX);
  });
  __syncthreads();
  int all = 0;
  const int e = threadIdx.x;
  if (e < E)
    for (int w = 0; w < warps; ++w) {
      const int n = seen[w * E + e];
      seen[w * E + e] = all;
      all += n;
    }
  const int chunks = (all + kChunk - 1) / kChunk;
  const int both = block_scan(all | chunks << 16, sums);  // (each up to 16384)
  const int row = both & 0xffff, at = both >> 16;
  if (threadIdx.x == 1023) *g.count = at + chunks;
  for (int c = 0; c < chunks; ++c) {
    g.expert[at + c] = e;
    g.first[at + c] = row + c * kChunk;
    g.rows[at + c] = min(kChunk, all - c * kChunk);
  }
  if (e < E) start[e] = row;
  __syncthreads();
  pass([&](int slot, int of, int rank) {
    const int r = of < 0 ? -1 : start[of] + rank;
    g.slot_row[slot] = r;
    if (r < 0) return;
    g.row_slot[r] = slot;
    g.row_gate[r] = g.gate[slot];
  });
}

// The same for few slots: every slot looks at all others, which has two barriers where the above has
// ten (7 tokens x 4 of 64 experts, 512 x 256: 17.1 -> 15.7 us).  Experts in the order of their first
// slots.  One block of 1024.
constexpr int kFewSlots = 256;
__device__ void group_few_slots(const Groups& g, int* dev_status) {
  __shared__ __align__(16) int expert[kFewSlots], rows_of[kFewSlots];  // (of an expert's first slots)
  const int i = threadIdx.x, slots = g.slots;
  int e = -1;
  if (i < slots) {
    if (g.good(i))
      e = g.idx[i];
    else
      report_status(dev_status, MOE_ERR_BAD_INDEX);
  }
  if (i < kFewSlots) expert[i] = e;
  __syncthreads();
  int first = i, rank = 0, rows = 0;  // of the slots of this expert
  if (e >= 0)
    for (int j = 0; j < slots; j += 4) {
      const int4 q = reinterpret_cast<const int4*>(expert)[j / 4];
      const int others[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool same = others[c] == e;
        if (same && rows == 0) first = j + c;
        rows += same;
        rank += same && j + c < i;
      }
    }
  if (i < kFewSlots) rows_of[i] = e >= 0 && first == i ? rows : 0;
  __syncthreads();
  if (i >= slots) return;
  int row = rank, at = 0, all = 0;  // chunks before the expert's, and of all
  for (int j = 0; j < slots; j += 4) {
    const int4 q = reinterpret_cast<const int4*>(rows_of)[j / 4];
    const int others[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int chunks = (others[c] + kChunk - 1) / kChunk;
      all += chunks;
      if (j + c < first) row += others[c], at += chunks;
    }
  }
  if (i == 0) *g.count = all;
  g.slot_row[i] = e >= 0 ? row : -1;
  if (e < 0) return;
  g.row_slot[row] = i;
  g.row_gate[row] = g.gate[i];
  if (rank % kChunk) return;
  at += rank / kChunk;
  g.expert[at] = e, g.first[at] = row, g.rows[at] = min(kChunk, rows - rank);
}

// ---------------------------------------------------------------- the tokens' values
// Rows of values as operands: PARTS fp16 values to each, and for every 64 columns (a tile) the sums of
// the values themselves and the factor that the products' sums are scaled by, which x has one of for a
// whole row.
template <int PARTS>
struct Rows {
  uint8_t* parts;  // [rows][tiles][PARTS][4 lanes][2 halves of a tile][8] fp16
  float4* info;    // [rows][tiles]: the factor; sums / 4096 over the halves and the tile
  int tiles;

  __device__ __forceinline__ const uint8_t* row(int r) const {
    return parts + static_cast<long long>(r) * (PARTS * kTile * 2 * tiles);
  }
  __device__ __forceinline__ const float4* info_row(int r) const {
    return info + static_cast<long long>(r) * tiles;
  }

  // Four neighbouring lanes (t = 0 .. 3) write a tile of a row: v[c][j] is column 32 c + 8 t + j, and
  // `most` the largest of what shares the factor.  u = v 2^e, |u| < 2^15, divided by 16 for j = 2, 3, 6,
  // 7, is part 0 + part 1 / 2048: fp16 has 11 bits, so one part is off by at most 2^-12 of it (bf16
  // values not at all) and two by 2^-24; and the small ones, whose bits end at 2^-24, by 2^-25 or 2^-36
  // in that scale, 2^-35 or 2^-46 of the largest.  Where that is not finite the factor is NaN, and so
  // becomes all that it scales.
  __device__ __forceinline__ void write(int r, int tile, const float (&v)[2][8], float most,
                                        bool whole_row) const {
    const int t = threadIdx.x & 3;
    const int exponent = max((__float_as_int(most) >> 23) - 127, -120);  // of the largest
    float left[2][8], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = ldexpf(v[c][j], 14 - exponent);
        sum[c] += u;
        left[c][j] = j & 2 ? u * 0.0625f : u;
      }
#pragma unroll
    for (int o = 1; o < 4; o *= 2) {
      sum[0] += __shfl_xor_sync(~0u, sum[0], o);
      sum[1] += __shfl_xor_sync(~0u, sum[1], o);
    }
    uint8_t* to = parts + (static_cast<long long>(r) * tiles + tile) * (PARTS * kTile * 2) + t * 32;
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t word[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 p = __floats2half2_rn(left[c][2 * i], left[c][2 * i + 1]);
          left[c][2 * i] = (left[c][2 * i] - __low2float(p)) * 2048.f;
          left[c][2 * i + 1] = (left[c][2 * i + 1] - __high2float(p)) * 2048.f;
          word[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        *reinterpret_cast<uint4*>(to + q * (kTile * 2) + c * 16) =
            make_uint4(word[0], word[1], word[2], word[3]);
      }
    if (t == 0) {
      const float factor = most <= 3.4028235e38f ? ldexpf(1.f, exponent - 2) : NAN;
      // the sums are of 4096ths; a whole row's are less its factor, which the results are multiplied by
      const int scale = whole_row ? -24 : exponent - 26;
      const float lo = ldexpf(sum[0], scale), hi = ldexpf(sum[1], scale);
      info[static_cast<long long>(r) * tiles + tile] = make_float4(factor, lo, hi, lo + hi);
    }
  }
  // Of 16 values; infinity if one is not a number.
  static __device__ __forceinline__ float largest(const float (&v)[2][8]) {
    float most = 0.f;
    bool good = true;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        most = fmaxf(most, fabsf(v[c][j]));
        good &= v[c][j] == v[c][j];
      }
    return good ? most : INFINITY;
  }
};

__device__ __forceinline__ void load16(const __nv_bfloat16* x, float (&v)[2][8]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint4 q = *reinterpret_cast<const uint4*>(x + c * 32);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[c][2 * j] = __uint_as_float(w[j] << 16);
      v[c][2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

// The tokens' values as operands, 256 threads to a row, and (the last block) the slots by expert;
// counters set to zero.
__global__ void __launch_bounds__(1024)
    w4_prepare_kernel(const __nv_bfloat16* x, int T, Rows<kXParts> rows, int* counters,
                      int n_counters, const Groups g, int warps, int* dev_status) {
  __shared__ float largest[4][8];
  after_previous();
  // (gate and up are set up beside this: one token 32.1 -> 31.9 us, 32 tokens 161 -> 157, 64 499 -> 500)
  let_next_start();
  const int blocks = g.single ? gridDim.x : gridDim.x - 1;
  if (blockIdx.x == blocks) {
    if (g.slots <= kFewSlots)
      group_few_slots(g, dev_status);
    else
      group_slots(g, warps, dev_status);
    return;
  }
  const int me = blockIdx.x * 1024 + threadIdx.x, all = blocks * 1024;
  for (int i = me; i < n_counters; i += all) counters[i] = 0;
  if (g.single && me < g.slots && !g.good(me)) report_status(dev_status, MOE_ERR_BAD_INDEX);
  const int team = threadIdx.x / 256, lane = threadIdx.x % 256;
  for (int r = blockIdx.x * 4 + team; r < T; r += blocks * 4) {
    const __nv_bfloat16* from = x + static_cast<long long>(r) * rows.tiles * kTile + lane % 4 * 8;
    float v[2][8], most = 0.f;
    for (int tile = lane / 4; tile < rows.tiles; tile += 64) {
      load16(from + tile * kTile, v);
      most = fmaxf(most, Rows<kXParts>::largest(v));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
    if (lane % 32 == 0) largest[team][lane / 32] = most;
    asm volatile("bar.sync %0, 256;" ::"r"(1 + team) : "memory");
#pragma unroll
    for (int w = 0; w < 8; ++w) most = fmaxf(most, largest[team][w]);
    asm volatile("bar.sync %0, 256;" ::"r"(1 + team) : "memory");
    // whole warps: lanes behind the row's end write its last tile again
    for (int tile = lane / 4; tile - lane % 32 / 4 < rows.tiles; tile += 64) {
      const int at = min(tile, rows.tiles - 1);
      load16(from + at * kTile, v);
      rows.write(r, at, v, most, true);
    }
  }
}

// ---------------------------------------------------------------- products
//
// `split` warps (1 to 8) take a strip of 16 weight rows (of both matrices, for gate and up), each every
// split'th piece of 256 of its columns.  Pieces come by bulk copies into a ring that is the warp's own,
// one piece or more ahead of the products and on into the warp's next strip.  (16 bytes to a lane by
// cp.async took about as many instructions for the copies as for the products: 1738 us -> 1161 us for
// 64 tokens, at 2.1 TB/s with 60 % of the issue slots used.)

// d = a b + c
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                    float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
        "f"(c3));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                    bool first) {
  if (first)
    mma(d, a, b0, b1, 0.f, 0.f, 0.f, 0.f);
  else
    mma(d, a, b0, b1, d[0], d[1], d[2], d[3]);
}

// True for one lane of a whole warp.  (Of a lane that the compiler knows to be one, operands of a bulk
// copy go to the uniform registers at once; `lane == 0` made a loop over the lanes of each copy.)
__device__ __forceinline__ bool one_lane() {
  uint32_t one;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(one));
  return one != 0;
}

// A bulk copy into shared memory; its bytes are counted at `bar`.
__device__ __forceinline__ void bulk_load(uint32_t to, const void* from, uint32_t bytes, uint32_t bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, "
      "[%3], %4;" ::"r"(to), "l"(from), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

// Whether the barrier's phase completed, for the whole warp; gives up after a limit.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
    while (!(ok = mbar_try_wait(bar, parity)) && globaltimer_ns() - t0 < limit_ns) {
    }
  }
  return __all_sync(~0u, ok);
}

// Self-test of those waits, of launches by the thread that asks for it: they wait this long at most, and
// one copy of one warp is expected to be longer than it is, so that its wait runs out.
struct Drill {
  uint64_t limit_ns;  // 0: none
  int block, warp, copy;
};
thread_local Drill drill_of_gateup, drill_of_down;

struct Weights {
  const void* codes;
  const void* scales;
  int group;
};

// Strips of one or two matrices [E, rows, cols] for the slots' chunks.
struct Problem {
  Groups g;
  Weights w[2];
  int rows, cols, split;
  int* dev_status;
  Drill drill;
};

// The tasks of a team of warps, one after the other: task i is strip i % strips of chunk i / strips.
struct Tasks {
  int chunk, strip, strips, chunk_step, strip_step;
  __device__ __forceinline__ Tasks(int first, int step, int strips_)
      : chunk(first / strips_), strip(first % strips_), strips(strips_),
        chunk_step(step / strips_), strip_step(step % strips_) {}
  __device__ __forceinline__ void next() {
    chunk += chunk_step, strip += strip_step;
    if (strip >= strips) strip -= strips, ++chunk;
  }
};

// MATS strips of weights with 8 tokens at most; ZEROS: zeros are given; GROUP columns to a scale.
// Gate and up take x, whose rows have one factor, and a strip of each.  DOWN takes h, which has a
// factor for each tile, and one strip or two neighbouring ones (which share the loads of h and wait for
// them half as often: 32 tokens, 2048 x 512: 170 -> 158 us).  ONE: a single token, whose values come
// with the weights' pieces and stand in all columns.  DRILL: the waits' self-test.  (Read from the L2 by each lane, a tile ahead, they
// were what down waited for: 34 -> 30 us.)
template <bool DOWN, int MATS, bool ZEROS, int GROUP, bool ONE = false, bool DRILL = false>
struct Product {
  static constexpr bool kFactors = DOWN, FINE = GROUP == 32;
  static constexpr int PARTS = DOWN ? kHParts : kXParts;
  static constexpr int kPieceTiles = MATS == 2 ? 4 : 8;
  static constexpr int kRows = DOWN ? MATS * kStrip : kStrip;  // of a matrix, to a task
  static constexpr int kWords = ZEROS ? 2 : 1;                  // of a group's scales, to a lane
  static constexpr int kCodes = kPieceTiles * 512;              // bytes of a piece and matrix
  static constexpr int of_scales(int tiles) { return tiles * (2048 * kWords / GROUP); }
  static constexpr int kValues = kCodes + of_scales(kPieceTiles);  // where ONE's values are in a place
  static constexpr int kInfo = kValues + kPieceTiles * (PARTS * kTile * 2);
  static constexpr int kPlace = ONE ? kInfo + kPieceTiles * 16 : kValues;
  static constexpr int kSums = MATS * 4;  // to a lane
  static constexpr int with_places(int n) { return n * MATS * kPlace + kSums * 128 + 32; }
  static constexpr int kBlocks = 2;  // to an SM
  // Of the ring, one less of them on their way: three for the shorter pieces of gate and up, if two
  // blocks still fit (with one, 32 tokens with zeros and groups of 64 took 81 us there instead of 66).
  static constexpr int kPlaces =
      MATS == 2 && kBlocks * (kWarps * with_places(3) + 1024) <= kSharedPerSm ? 3 : 2;
  static constexpr int kRing = kPlaces * MATS * kPlace;
  static constexpr int kWarpBytes = with_places(kPlaces), kBytes = kWarps * kWarpBytes;
  // Tiles that one scale is multiplied with at once: two where their sums can wait for it.
  static constexpr int kTogether = GROUP == 128 && !kFactors ? 2 : 1;

  // Issues the copies of pieces; all of a warp's lanes know where it stands, one issues them.
  struct Copies {
    const Problem& p;
    uint32_t ring, bars;
    int tiles, place;  // tiles: of a strip
    uint64_t policy;
    int copies = 0;  // (DRILL)

    __device__ __forceinline__ Copies(const Problem& p_, uint8_t* ring_, uint64_t* bars_)
        : p(p_), ring(smem_u32(ring_)), bars(smem_u32(bars_)), tiles(p_.cols / kTile), place(0),
          policy(l2_policy_evict_first()) {}
    // n tiles from `tile` on of all that a matrix has (fewer than 2^31).
    __device__ __forceinline__ void issue(int tile, int n, const void* values = nullptr,
                                          const void* infos = nullptr) {
      const uint32_t to = ring + place * (MATS * kPlace), bar = bars + place * 8;
      const uint32_t bytes = n * 512, of = of_scales(n);
      const uint32_t parts = n * (PARTS * kTile * 2), info = n * 16;
      uint32_t more = 0;
      if (DRILL && blockIdx.x == p.drill.block && threadIdx.x / 32 == p.drill.warp &&
          copies++ == p.drill.copy)
        more = 16;
      if (one_lane()) {
        expect(bar, MATS * (bytes + of) + (ONE ? parts + info : 0) + more);
        if (ONE) {
          bulk_load(to + kValues, values, parts, bar, policy);
          bulk_load(to + kInfo, infos, info, bar, policy);
        }
#pragma unroll
        for (int i = 0; i < MATS; ++i) {
          const Weights& w = p.w[DOWN ? 0 : i];
          const long long at = tile + (DOWN ? i * tiles : 0);
          bulk_load(to + i * kPlace, static_cast<const uint8_t*>(w.codes) + at * 512, bytes, bar, policy);
          bulk_load(to + i * kPlace + kCodes, static_cast<const uint8_t*>(w.scales) + at * of_scales(1),
                    of, bar, policy);
        }
      }
      if (++place == kPlaces) place = 0;
    }
  };

  // The pieces of a team's strips, one warp's share, ahead of the products.
  struct Ahead : Copies {
    Tasks at;
    int chunks, tile, left, skip;  // tiles from the piece on; tiles of the team's pieces before

    __device__ __forceinline__ Ahead(const Problem& p_, uint8_t* ring_, uint64_t* bars_,
                                     const Tasks& at_, int chunks_, int first)
        : Copies(p_, ring_, bars_), at(at_), chunks(chunks_), skip(first * kPieceTiles) {
      begin();
    }
    __device__ __forceinline__ void begin() {
      if (at.chunk >= chunks) return;
      tile = (this->p.g.expert_of(at.chunk) * at.strips + at.strip) * (kRows / kStrip) * this->tiles + skip;
      left = this->tiles - skip;
    }
    __device__ __forceinline__ void next() {
      if (at.chunk >= chunks) return;
      this->issue(tile, min(kPieceTiles, left));
      const int step = this->p.split * kPieceTiles;
      tile += step, left -= step;
      if (left <= 0) {
        at.next();
        begin();
      }
    }
  };

  // A warp's share of the pieces of one strip of a single token's slots after one another, those of bad
  // experts left out; the same in the block's next strips.
  struct Pieces {
    int chunk, piece, pieces, chunk_step, piece_step;
    uint32_t good;  // slots, a bit to each (32 at most)
    __device__ __forceinline__ Pieces(int first, int step, int pieces_, uint32_t good_)
        : chunk(first / pieces_), piece(first % pieces_), pieces(pieces_),
          chunk_step(step / pieces_), piece_step(step % pieces_), good(good_) {
      while (bad()) step_on();
    }
    __device__ __forceinline__ void next() {
      do step_on();
      while (bad());
    }
    __device__ __forceinline__ bool left() const { return chunk < 32 && good >> chunk; }

   private:
    __device__ __forceinline__ bool bad() const { return left() && !(good >> chunk & 1); }
    __device__ __forceinline__ void step_on() {
      chunk += chunk_step, piece += piece_step;
      if (piece >= pieces) piece -= pieces, ++chunk;
    }
  };
  struct AheadInStrips : Copies {
    Pieces start, at;
    int strip, strips, expert;
    const Rows<PARTS>& values;

    __device__ __forceinline__ AheadInStrips(const Problem& p_, const Rows<PARTS>& values_,
                                             uint8_t* ring_, uint64_t* bars_, const Pieces& at_)
        : Copies(p_, ring_, bars_), start(at_), at(at_), strip(blockIdx.x), strips(p_.rows / kStrip),
          values(values_) {
      if (!at.left()) strip = strips;  // more warps than pieces
      if (strip < strips) expert = p_.g.expert_of(at.chunk);
    }
    __device__ __forceinline__ void next() {
      if (strip >= strips) return;
      const int skip = at.piece * kPieceTiles;
      const int tile = (expert * strips + strip) * this->tiles + skip;
      const int n = min(kPieceTiles, this->tiles - skip);
      this->issue(tile, n, values.row(at.chunk) + skip * (PARTS * kTile * 2),
                  values.info_row(at.chunk) + skip);
      at.next();
      if (!at.left()) at = start, strip += gridDim.x;
      if (strip < strips) expert = this->p.g.expert_of(at.chunk);  // (wanted at the next call)
    }
  };

  struct Scale {
    float s[2], z[2];  // of rows g and g + 8
    __device__ __forceinline__ void load(const uint32_t* from) {
      if constexpr (ZEROS) {
        const uint2 v = *reinterpret_cast<const uint2*>(from);
        s[0] = __uint_as_float(v.x << 16), s[1] = __uint_as_float(v.y << 16);
        z[0] = __uint_as_float(v.x & 0xffff0000u), z[1] = __uint_as_float(v.y & 0xffff0000u);
      } else {
        const uint32_t v = *from;
        s[0] = __uint_as_float(v << 16), s[1] = __uint_as_float(v & 0xffff0000u);
        z[0] = z[1] = 8.f;
      }
    }
  };

  // A tile's weights as operands, for each 16 of its columns.
  struct Operands {
    uint32_t a[4][4];
    __device__ __forceinline__ void load(const uint8_t* codes) {
      const uint4 w = *reinterpret_cast<const uint4*>(codes + (threadIdx.x & 31) * 16);
      const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // row g + i % 2 * 8, half i / 2
        const uint32_t next = words[i] >> 8;
        a[i / 2 * 2][i % 2] = words[i] & 0x000f000fu, a[i / 2 * 2][i % 2 + 2] = words[i] & 0x00f000f0u;
        a[i / 2 * 2 + 1][i % 2] = next & 0x000f000fu, a[i / 2 * 2 + 1][i % 2 + 2] = next & 0x00f000f0u;
      }
    }
  };

  // Where a lane finds the values of eight tokens: the parts of token lane / 4, and what goes with the
  // sums of tokens lane % 4 * 2 and the one after.
  struct From {
    const uint8_t* parts;
    const float4* info[2];
    __device__ __forceinline__ void advance(int n) {
      parts += n * (PARTS * kTile * 2), info[0] += n, info[1] += n;
    }
  };
  // Those values, for a tile.
  struct Values {
    uint4 v[PARTS][2];
    float factor[2], sum[FINE ? 2 : 1][2];
    __device__ __forceinline__ void load(const From& x, int tile) {
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          v[q][c] = reinterpret_cast<const uint4*>(x.parts + (tile * PARTS + q) * (kTile * 2))[c];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4* info = x.info[i] + tile;
        if (kFactors) {
          const float4 all = *info;
          factor[i] = all.x, sum[0][i] = FINE ? all.y : all.w;
          if (FINE) sum[FINE][i] = all.z;
        } else if (FINE) {
          sum[0][i] = info->y, sum[FINE][i] = info->z;
        } else {
          sum[0][i] = info->w;
        }
      }
    }
  };

  // acc += s (part - z sum), for what `part` and `sum` have of a group's columns.
  static __device__ __forceinline__ void add(const uint8_t* scales, int group,
                                             const float (&part)[PARTS][4], const float (&factor)[2],
                                             const float (&sum)[2], float (&acc)[4]) {
    Scale s;
    s.load(reinterpret_cast<const uint32_t*>(scales + group * (32 * kWords)) +
           (threadIdx.x & 31) / 4 * kWords);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float v = part[PARTS - 1][r];
#pragma unroll
      for (int q = PARTS - 2; q >= 0; --q) v = fmaf(v, 1.f / 2048.f, part[q][r]);
      if (kFactors)
        v = fmaf(factor[r % 2], v, -s.z[r / 2] * sum[r % 2]);
      else
        v = fmaf(-s.z[r / 2], sum[r % 2], v);
      acc[r] = fmaf(s.s[r / 2], v, acc[r]);
    }
  }

  // Tile u of a piece (`at` in `from`), the i-th of kTogether.
  static __device__ __forceinline__ void multiply(const Operands& w, const Values& x,
                                                  const uint8_t* scales, int u, int i,
                                                  float (&part)[PARTS][4], float (&before)[2],
                                                  float (&acc)[4]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
        mma(part[q], w.a[2 * c], x.v[q][c].x, x.v[q][c].y, (c == 0 && i == 0) || FINE);
        mma(part[q], w.a[2 * c + 1], x.v[q][c].z, x.v[q][c].w, false);
      }
      if (FINE) add(scales, 2 * u + c, part, x.factor, x.sum[FINE ? c : 0], acc);
    }
    if (FINE) return;
    const float sum[2] = {i ? before[0] + x.sum[0][0] : x.sum[0][0],
                          i ? before[1] + x.sum[0][1] : x.sum[0][1]};
    if (i + 1 == kTogether)
      add(scales, GROUP == 128 ? u / 2 : u, part, x.factor, sum, acc);
    else
      before[0] = sum[0], before[1] = sum[1];
  }

  // N tiles of a piece from its tile u0 on, for which x stands at the values.  `now` has those of the
  // first one, and is left with those of the tile after the last if there is `more` to come.
  template <int N>
  static __device__ __forceinline__ void tiles_of(const uint8_t* from, int u0, From& x, bool more,
                                                  Values& now, float (&acc)[MATS][4]) {
    static_assert(N % kTogether == 0, "whole groups");
    float part[MATS][PARTS][4], before[2];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int u = u0 + k;
      Operands w[MATS];
#pragma unroll
      for (int i = 0; i < MATS; ++i) w[i].load(from + i * kPlace + u * 512);
      const Values mine = now;
      if (k + 1 < N || more) now.load(x, k + 1);
#pragma unroll
      for (int i = 0; i < MATS; ++i) {
        float sums[2] = {before[0], before[1]};
        multiply(w[i], mine, from + i * kPlace + kCodes, u, k % kTogether, part[i], sums, acc[i]);
        if (i + 1 == MATS) before[0] = sums[0], before[1] = sums[1];
      }
    }
    x.advance(N);
  }
  // The n tiles of a piece, for which x stands at the values and `now` has those of the first.
  static __device__ __forceinline__ void piece(const uint8_t* from, int n, From& x, Values& now,
                                               float (&acc)[MATS][4]) {
    if (n == kPieceTiles) {
#pragma unroll 1
      for (int u = 0; u < kPieceTiles; u += 4)
        tiles_of<4>(from, u, x, u + 4 < kPieceTiles, now, acc);
    } else {
#pragma unroll 1
      for (int u = 0; u < n; u += kTogether)
        tiles_of<kTogether>(from, u, x, u + kTogether < n, now, acc);
    }
  }

  // All of the warp's strips.  value_row(r) is the row of x of a chunk's row r; put(chunk, first, rows,
  // strip, sums) gets the sums: place r of a lane is row lane / 4 + r / 2 * 8 of the strip, token
  // lane % 4 * 2 + r % 2 of the chunk.  (Columns of tokens that there are not repeat the first one's; a
  // product's columns have nothing to do with each other.)
  template <typename RowOf, typename Put>
  static __device__ __forceinline__ void run(const Problem& p, const Rows<PARTS>& values,
                                             uint8_t* shared, RowOf value_row, Put put) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, split = p.split;
    const int team = warp / split, me = warp % split, teams = kWarps / split;
    uint8_t* ring = shared + warp * kRing;
    float* sums = reinterpret_cast<float*>(shared + kWarps * kRing);  // [warp][kSums][32]
    uint64_t* bars =
        reinterpret_cast<uint64_t*>(shared + kWarps * (kRing + kSums * 128)) + warp * kPlaces;
    if (lane == 0) {
      for (int i = 0; i < kPlaces; ++i) mbar_init(bars + i, 1);
      fence_barrier_init();
    }
    __syncwarp();
    after_previous();
    const int strips = p.rows / kRows, tiles = p.cols / kTile, chunks = p.g.chunks();
    Tasks task(blockIdx.x * teams + team, gridDim.x * teams, strips);
    Ahead ahead(p, ring, bars, task, chunks, me);
    for (int i = 0; i < kPlaces - 1; ++i) ahead.next();
    int place = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (; task.chunk < chunks; task.next()) {
      const int first = p.g.first_of(task.chunk), rows = p.g.rows_of(task.chunk);
      const auto row = [&](int token) { return value_row(first + (token < rows ? token : 0)); };
      From x{values.row(row(lane / 4)) + lane % 4 * 32,
             {values.info_row(row(lane % 4 * 2)), values.info_row(row(lane % 4 * 2 + 1))}};
      float acc[MATS][4] = {};
      x.advance(me * kPieceTiles);
      for (int left = tiles - me * kPieceTiles; left > 0 && ok; left -= split * kPieceTiles) {
        Values now;
        now.load(x, 0);
        if (!wait_for(bars + place, parity, limit(p))) {
          ok = false;
          break;
        }
        ahead.next();
        __syncwarp();
        piece(ring + place * (MATS * kPlace), min(left, kPieceTiles), x, now, acc);
        if (split > 1) x.advance((split - 1) * kPieceTiles);  // (not read behind the end)
        if (++place == kPlaces) place = 0, parity ^= 1;
        __syncwarp();  // the place is read before it is copied into again
      }
      if (split > 1) {  // the team's sums, added in its order by its first warp
        const auto sync = [&] {
          asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(split * 32) : "memory");
        };
        if (me)
#pragma unroll
          for (int i = 0; i < kSums; ++i)
            sums[(warp * kSums + i) * 32 + lane] = acc[i / 4][i % 4];
        sync();
        if (!me)
          for (int o = 1; o < split; ++o)
#pragma unroll
            for (int i = 0; i < kSums; ++i)
              acc[i / 4][i % 4] += sums[((warp + o) * kSums + i) * 32 + lane];
        sync();
      }
      if (!me) put(task.chunk, first, rows, task.strip, acc);
    }
    drain(p, ok, ahead.place, bars, place, parity);
  }

  // All of the block's strips, for a single token: the sums over its experts stay in the products' sums.
  // put(strip, row, sum).
  template <typename Put>
  static __device__ __forceinline__ void run_strips(const Problem& p, const Rows<PARTS>& values,
                                                    uint8_t* shared, Put put) {
    static_assert(ONE && MATS == 1, "one strip, one token");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32;
    uint8_t* ring = shared + warp * kRing;
    float* sums = reinterpret_cast<float*>(shared + warps * kRing);  // [warp][4][32]
    uint64_t* bars =
        reinterpret_cast<uint64_t*>(shared + warps * (kRing + kSums * 128)) + warp * kPlaces;
    if (lane == 0) {
      for (int i = 0; i < kPlaces; ++i) mbar_init(bars + i, 1);
      fence_barrier_init();
    }
    __syncwarp();
    after_previous();
    const int strips = p.rows / kStrip, tiles = p.cols / kTile;
    const uint32_t good = __ballot_sync(~0u, lane < p.g.slots && p.g.good(lane));
    const Pieces start(warp, warps, (tiles + kPieceTiles - 1) / kPieceTiles, good);
    AheadInStrips ahead(p, values, ring, bars, start);
    for (int i = 0; i < kPlaces - 1; ++i) ahead.next();
    int place = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (int strip = blockIdx.x; strip < strips; strip += gridDim.x) {
      float acc[1][4] = {};
      for (Pieces at = start; at.left() && ok; at.next()) {
        if (!wait_for(bars + place, parity, limit(p))) {
          ok = false;
          break;
        }
        ahead.next();
        const uint8_t* from = ring + place * kPlace;
        const float4* infos = reinterpret_cast<const float4*>(from + kInfo);
        From x{from + kValues + lane % 4 * 32, {infos, infos}};
        Values now;
        now.load(x, 0);
        __syncwarp();
        piece(from, min(tiles - at.piece * kPieceTiles, kPieceTiles), x, now, acc);
        if (++place == kPlaces) place = 0, parity ^= 1;
        __syncwarp();  // the place is read before it is copied into again
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[(warp * 4 + r) * 32 + lane] = acc[0][r];
      __syncthreads();
      if (threadIdx.x < 128 && lane % 4 == 0 && warp % 2 == 0) {  // (all columns are the same)
        float sum = 0.f;
        for (int w = 0; w < warps; ++w) sum += sums[w * 128 + threadIdx.x];
        put(strip, lane / 4 + warp / 2 * 8, sum);
      }
      __syncthreads();
    }
    drain(p, ok, ahead.place, bars, place, parity);
  }

  static __device__ __forceinline__ uint64_t limit(const Problem& p) {
    return DRILL ? p.drill.limit_ns : kWaitTimeoutNs;
  }
  // After a wait that ran out: what is on its way arrives before the block's memory is given up.
  static __device__ __forceinline__ void drain(const Problem& p, bool ok, int issued,
                                               uint64_t* bars, int place, uint32_t parity) {
    if (ok) return;
    if ((threadIdx.x & 31) == 0) report_status(p.dev_status, MOE_ERR_TIMEOUT);
    while (place != issued) {
      wait_for(bars + place, parity, limit(p));
      if (++place == kPlaces) place = 0, parity ^= 1;
    }
  }
};

struct GateUp {
  Problem p;
  Rows<kXParts> x;
  float* h;       // [slots][F], times the gate
  Rows<kHParts> parts;  // the same as operands
  int* counters;  // [chunks][F / 64]: strips of a tile that are done
  int k;
};

// h goes to memory in fp32; the warp that brings the last of a tile's four strips makes operands of it.
template <bool ZEROS, int GROUP, bool DRILL>
__global__ void __launch_bounds__(kWarps * 32, Product<false, 2, ZEROS, GROUP>::kBlocks)
    w4_gateup_kernel(const GateUp a) {
  using Of = Product<false, 2, ZEROS, GROUP, false, DRILL>;
  extern __shared__ __align__(16) uint8_t shared[];
  const int F = a.p.rows, lane = threadIdx.x & 31;
  Of::run(
      a.p, a.x, shared, [&](int r) { return a.p.g.slot_of(r) / a.k; },
      [&](int chunk, int first, int rows, int strip, const float (&acc)[2][4]) {
        if (rows == 0) return;  // a single token's bad expert: it has no row, and down none of h to read
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int token = lane % 4 * 2 + r % 2;
          if (token >= rows) continue;
          // (a factor of the whole row of x)
          const float f = a.x.info_row(a.p.g.slot_of(first + token) / a.k)->x;
          const float v = f * acc[0][r];
          const float h = a.p.g.gate_of(first + token) * (v / (1.f + expf(-v)) * (f * acc[1][r]));
          __stcg(a.h + (first + token) * static_cast<long long>(F) + strip * kStrip + lane / 4 +
                     r / 2 * 8, h);
        }
        const int tile = strip / 4;
        __threadfence();
        __syncwarp();
        int before = 0;
        if (lane == 0)
          before = atomicAdd(a.counters + static_cast<long long>(chunk) * (F / kTile) + tile, 1);
        if (__shfl_sync(~0u, before, 0) != 3) return;
        __threadfence();
        const int r = first + min(lane / 4, rows - 1);  // (the last one again)
        float v[2][8];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 q = __ldcg(reinterpret_cast<const float4*>(
                a.h + r * static_cast<long long>(F) + tile * kTile + c * 32 + lane % 4 * 8 + j));
            v[c][j] = q.x, v[c][j + 1] = q.y, v[c][j + 2] = q.z, v[c][j + 3] = q.w;
          }
        float most = Rows<kHParts>::largest(v);
        most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
        most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
        a.parts.write(r, tile, v, most, false);
      });
}

struct Down {
  Problem p;
  Rows<kHParts> h;
  float* out;  // [slots][d], a row to a slot
  __nv_bfloat16* y;
};

// A single token: y at once.
template <bool ZEROS, int GROUP, bool DRILL>
__global__ void __launch_bounds__(kMaxWarps * 32) w4_down_kernel(const Down a) {
  using Of = Product<true, 1, ZEROS, GROUP, true, DRILL>;
  extern __shared__ __align__(16) uint8_t shared[];
  Of::run_strips(a.p, a.h, shared, [&](int strip, int row, float sum) {
    a.y[strip * kStrip + row] = __float2bfloat16_rn(sum);
  });
}

// More tokens: the rows' parts of it, which w4_combine_kernel adds.
template <bool ZEROS, int GROUP, bool DRILL>
__global__ void __launch_bounds__(kWarps * 32, Product<true, 2, ZEROS, GROUP>::kBlocks)
    w4_down_rows_kernel(const Down a) {
  extern __shared__ __align__(16) uint8_t shared[];
  const int d = a.p.rows, lane = threadIdx.x & 31;
  Product<true, 2, ZEROS, GROUP, false, DRILL>::run(
      a.p, a.h, shared, [&](int r) { return r; },
      [&](int, int first, int rows, int strip, const float (&acc)[2][4]) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int token = lane % 4 * 2 + r % 2;
          if (token < rows)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              a.out[(first + token) * static_cast<long long>(d) + (strip * 2 + i) * kStrip + lane / 4 +
                    r / 2 * 8] = acc[i][r];
        }
      });
}

// y_t = sum_j out[row of slot (t, j)], in the slots' order: 4 columns to a thread.
__global__ void __launch_bounds__(128)
    w4_combine_kernel(const int* slot_row, const float* out, int d, int k, __nv_bfloat16* y) {
  __shared__ int rows[32];
  after_previous();
  const long long t = blockIdx.x;
  if (threadIdx.x < 32) rows[threadIdx.x] = threadIdx.x < k ? slot_row[t * k + threadIdx.x] : -1;
  __syncthreads();
  for (int c = (blockIdx.y * 128 + threadIdx.x) * 4; c < d; c += gridDim.y * 512) {
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < k; j0 += 8) {
      float4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (rows[j0 + j] >= 0)
          v[j] = *reinterpret_cast<const float4*>(out + static_cast<long long>(rows[j0 + j]) * d + c);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        sum.x += v[j].x, sum.y += v[j].y, sum.z += v[j].z, sum.w += v[j].w;
    }
    *reinterpret_cast<uint2*>(y + t * d + c) =
        make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
  }
}

// ------------------------------------------------------------------------ host side

constexpr int kSms = 152;
// Warps to a strip: what takes least time, in pieces, with one more for each strip's beginning and end;
// the strips are taken in rounds.
int split_of(long long strips, int pieces, int warps) {
  int best = 1;
  long long least = -1;
  for (int split = 1; split <= kWarps && split <= pieces; split *= 2) {
    const long long teams = warps / split, rounds = (strips + teams - 1) / teams;
    const long long cost = rounds * ((pieces + split - 1) / split + 1);
    if (least < 0 || cost < least) least = cost, best = split;
  }
  return best;
}

struct Workspace {
  Groups g;
  Rows<kXParts> x;
  Rows<kHParts> parts;
  int* counters;
  int n_counters;
  float* h;
  float* out;
  size_t bytes;
};

Workspace carve(const moe_problem* p, void* base) {
  const size_t slots = static_cast<size_t>(p->T) * p->k;
  const size_t chunks = std::min<size_t>(p->E, slots) + slots / kChunk;
  Workspace w{};
  uint8_t* at = static_cast<uint8_t*>(base);
  const auto take = [&](size_t bytes) {
    uint8_t* got = at + w.bytes;
    w.bytes += up256(bytes);
    return got;
  };
  w.g.count = reinterpret_cast<int*>(take(4));
  w.g.expert = reinterpret_cast<int*>(take(chunks * 4));
  w.g.first = reinterpret_cast<int*>(take(chunks * 4));
  w.g.rows = reinterpret_cast<int*>(take(chunks * 4));
  w.g.row_slot = reinterpret_cast<int*>(take(slots * 4));
  w.g.row_gate = reinterpret_cast<float*>(take(slots * 4));
  w.g.slot_row = reinterpret_cast<int*>(take(slots * 4));
  const size_t x_tiles = p->d / kTile, h_tiles = p->F / kTile;
  w.x.tiles = p->d / kTile, w.parts.tiles = p->F / kTile;
  w.x.parts = take(p->T * x_tiles * (kXParts * kTile * 2));
  w.x.info = reinterpret_cast<float4*>(take(p->T * x_tiles * 16));
  w.parts.parts = take(slots * h_tiles * (kHParts * kTile * 2));
  w.parts.info = reinterpret_cast<float4*>(take(slots * h_tiles * 16));
  w.n_counters = static_cast<int>((p->T == 1 ? slots : chunks) * h_tiles);
  w.counters = reinterpret_cast<int*>(take(w.n_counters * 4));
  w.h = reinterpret_cast<float*>(take(slots * p->F * 4));
  w.out = reinterpret_cast<float*>(take(p->T == 1 ? 0 : slots * p->d * 4));
  return w;
}

// 2^40 weights of a matrix, whose tiles are counted in 31 bits.
bool too_many(long long E, long long rows, long long cols) { return E * rows > (1ll << 40) / cols; }

int check_w4(const moe_problem* p) {
  if (int e = check_problem(p)) return e;
  if (p->r || static_cast<long long>(p->T) * p->k > kMaxSlots) return MOE_ERR_UNSUPPORTED;
  if (std::max(p->d, p->F) > kMaxWidth || too_many(p->E, p->d, p->F)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool bad_group(int group, int cols) {
  return (group != 32 && group != 64 && group != 128) || cols % group;
}

int check_weights(const moe_w4* w, int cols) {
  if (!w || !w->codes || !w->scales) return MOE_ERR_INVALID_ARG;
  if (bad_group(w->group, cols) || misaligned(w->codes, 16) || misaligned(w->scales, 16))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" {

using namespace moe;

int moe_w4_pack(int32_t E, int32_t rows, int32_t cols, int32_t group, const uint8_t* codes,
                const moe_bf16* scales, const uint8_t* zeros, void* packed_codes,
                void* packed_scales, moe_stream_t stream) {
  if (E <= 0 || rows <= 0 || cols <= 0 || !codes || !scales || !packed_codes || !packed_scales)
    return MOE_ERR_INVALID_ARG;
  if (rows % kStrip || cols % kTile || bad_group(group, cols)) return MOE_ERR_UNSUPPORTED;
  if (misaligned(scales, 2) || misaligned(packed_codes, 16) || misaligned(packed_scales, 16))
    return MOE_ERR_UNSUPPORTED;
  const long long weights = static_cast<long long>(E) * rows * cols;
  if (too_many(E, rows, cols)) return MOE_ERR_UNSUPPORTED;
  const auto grid = [](long long n) {
    return static_cast<int>(std::min<long long>((n + 255) / 256, 8ll * kSms));
  };
  cudaError_t err = launch_behind(w4_pack_kernel, grid(weights / 8), 256, 0, stream, rows, cols,
                                  weights / 8, codes, static_cast<uint32_t*>(packed_codes));
  if (err == cudaSuccess)
    err = launch_behind(w4_pack_scales_kernel, grid(weights / group), 256, 0, stream, cols / group,
                        weights / group, reinterpret_cast<const __nv_bfloat16*>(scales), zeros,
                        static_cast<__nv_bfloat16*>(packed_scales));
  count_launches(2);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_w4_expert_ffn_workspace_size(const moe_problem* p) {
  return check_w4(p) == MOE_OK ? carve(p, nullptr).bytes : 0;
}

int moe_w4_expert_ffn(const moe_problem* p, const moe_bf16* x, const int32_t* topk_idx,
                      const float* topk_gate, const moe_w4* w_gate, const moe_w4* w_up,
                      const moe_w4* w_down, moe_bf16* y, void* workspace, size_t workspace_bytes,
                      int32_t* dev_status, moe_stream_t stream) {
  if (int e = check_w4(p)) return e;
  if (!x || !topk_idx || !topk_gate || !y) return MOE_ERR_INVALID_ARG;
  if (int e = check_weights(w_gate, p->d)) return e;
  if (int e = check_weights(w_up, p->d)) return e;
  if (int e = check_weights(w_down, p->F)) return e;
  const bool zeros = w_gate->has_zeros != 0;
  if (w_gate->group != w_up->group || w_gate->group != w_down->group ||
      zeros != (w_up->has_zeros != 0) || zeros != (w_down->has_zeros != 0))
    return MOE_ERR_UNSUPPORTED;
  if (misaligned(x, 16) || misaligned(y, 16) || misaligned(topk_idx, 4) ||
      misaligned(topk_gate, 4) || misaligned(dev_status, 4))
    return MOE_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < carve(p, nullptr).bytes) return MOE_ERR_WORKSPACE;
  if (misaligned(workspace, 16)) return MOE_ERR_UNSUPPORTED;
  const Workspace ws = carve(p, workspace);
  const int slots = p->T * p->k;
  const auto of = [](const moe_w4* w) { return Weights{w->codes, w->scales, w->group}; };
  Groups g = ws.g;
  g.idx = topk_idx, g.gate = topk_gate, g.slots = slots, g.E = p->E, g.single = p->T == 1;
  const int chunks = std::max(std::min(p->E, slots), slots / kChunk);  // about
  const Drill drill_up = drill_of_gateup, drill_down = drill_of_down;
  const bool drill = drill_up.limit_ns || drill_down.limit_ns;
  if (drill && (zeros || w_gate->group != kDrillGroup)) return MOE_ERR_UNSUPPORTED;
  GateUp up{{g, {of(w_gate), of(w_up)}, p->F, p->d, 1, dev_status, drill_up}, ws.x, ws.h, ws.parts,
            ws.counters, p->k};
  Down down{{g, {of(w_down), {}}, p->d, p->F, 1, dev_status, drill_down}, ws.parts, ws.out,
            reinterpret_cast<__nv_bfloat16*>(y)};
  cudaError_t err = cudaSuccess;
  // (The limit is the kernel's, for all threads of the process: the most that any call wants, so that
  // no call takes it down while another one is about to launch.)
  const auto launch = [&](auto kernel, int blocks, int warps, int bytes, int limit, auto& args) {
    if (err == cudaSuccess)
      err = launched(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, limit));
    if (err == cudaSuccess) err = launch_behind(kernel, blocks, warps * 32, bytes, stream, args);
  };
  const auto by_strips = [&](auto kernel, auto product, auto& args) {
    using Of = decltype(product);
    const int blocks = std::min(Of::kBlocks, kSharedPerSm / (Of::kBytes + 1024)) * kSms;
    args.p.split = split_of(chunks * static_cast<long long>(args.p.rows / Of::kRows),
                            (args.p.cols / kTile + Of::kPieceTiles - 1) / Of::kPieceTiles,
                            blocks * kWarps);
    launch(kernel, blocks, kWarps, Of::kBytes, Of::kBytes, args);
  };
  mark_before(MOE_KERNEL_W4_GATEUP, stream);
  {
    const int warps = std::min(32, (slots + 31) / 32);
    const int blocks = std::min((p->T + 3) / 4, kSms - 1);
    err = launched(cudaFuncSetAttribute(
        w4_prepare_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 32 * kMaxExperts * 2));
    if (err == cudaSuccess)
      err = launch_behind(w4_prepare_kernel, blocks + !g.single, 1024,
                          slots <= kFewSlots ? 0 : warps * p->E * 2, stream,
                          reinterpret_cast<const __nv_bfloat16*>(x), p->T, ws.x, ws.counters,
                          ws.n_counters, g, warps, dev_status);
  }
  const auto with = [&](auto z, auto of_group, auto drilled) {
    constexpr bool Z = decltype(z)::value, DRILL = decltype(drilled)::value;
    constexpr int GROUP = decltype(of_group)::value;
    by_strips(w4_gateup_kernel<Z, GROUP, DRILL>, Product<false, 2, Z, GROUP>{}, up);
    mark_after(MOE_KERNEL_W4_GATEUP, stream);
    mark_before(MOE_KERNEL_W4_DOWN, stream);
    if (g.single) {
      using Of = Product<true, 1, Z, GROUP, true>;
      constexpr int kMost = std::min(kMaxWarps, kSharedPerBlock / Of::kWarpBytes);
      const int strips = p->d / kStrip, warps = strips > kSms ? kWarps : kMost;
      launch(w4_down_kernel<Z, GROUP, DRILL>, std::min(strips, 2 * kSms * kWarps / warps), warps,
             warps * Of::kWarpBytes, kMost * Of::kWarpBytes, down);
    } else {
      by_strips(w4_down_rows_kernel<Z, GROUP, DRILL>, Product<true, 2, Z, GROUP>{}, down);
    }
    if (!g.single && err == cudaSuccess)
      err = launch_behind(w4_combine_kernel, dim3(p->T, std::min(64, (p->d + 511) / 512)), 128, 0,
                          stream, ws.g.slot_row, ws.out, p->d, p->k, down.y);
  };
  const auto with_group = [&](auto z) {
    if (w_gate->group == 32)
      with(z, std::integral_constant<int, 32>{}, std::false_type{});
    else if (w_gate->group == 64)
      with(z, std::integral_constant<int, 64>{}, std::false_type{});
    else
      with(z, std::integral_constant<int, 128>{}, std::false_type{});
  };
  if (drill)
    with(std::false_type{}, std::integral_constant<int, kDrillGroup>{}, std::true_type{});
  else if (zeros)
    with_group(std::true_type{});
  else
    with_group(std::false_type{});
  mark_after(MOE_KERNEL_W4_DOWN, stream);
  count_launches(3 + !g.single);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_selftest_w4_waits(int32_t limit_ms, int32_t down, int32_t block, int32_t warp, int32_t copy) {
  if (limit_ms < 0 || limit_ms > 2000 || (limit_ms && (block < 0 || warp < 0 || copy < 0)))
    return MOE_ERR_INVALID_ARG;
  drill_of_gateup = drill_of_down = Drill{};
  if (!limit_ms) return MOE_OK;
  const uint64_t limit_ns = limit_ms * 1000000ull;
  drill_of_gateup = {limit_ns, down ? -1 : block, warp, copy};
  drill_of_down = {limit_ns, down ? block : -1, warp, copy};
  return MOE_OK;
}

}  // extern "C"
