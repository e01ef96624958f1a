// The experts' products with 4-bit weights for few tokens (include/moe_block.h has the formulas).
//
// A weight w = s (c - z) is read once for all rows (tokens) of its expert, and the time is that of
// reading.  The products run on the tensor cores with 16 weight rows against 8 tokens (m16n8k16, bf16
// operands, fp32 sums): codes less zeros are whole numbers that bf16 holds exactly, and a group's sum
// is multiplied by its scale in fp32 afterwards.
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
constexpr int kMaxExperts = 1024;
constexpr int kWarps = 8;

// ---------------------------------------------------------------- layout
// A tile of 16 rows x 64 columns takes 512 bytes, 16 to a lane: lane 4 g + t holds rows g and g + 8,
// columns 8 t .. 8 t + 7 of each half of the tile, as the words (g, first half), (g + 8, first half),
// (g, second half), (g + 8, second half).  Within a word column 2 p + i of its eight is nibble
// p + 4 i, so that a shift and a mask leave two neighbouring columns in the halves of a word, as the
// product's operands want them (the order of the columns means nothing to it, as long as the tokens'
// operand has the same: column 8 t + j of a half is in lane t there too).  A tile's rows are those
// of a strip; strips, then experts follow one another.  Scales: for 16 rows and a group of columns,
// (row g, row g + 8) for each g; with zeros, each scale is followed by 128 + zero, in bf16.

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
    for (int p = 0; p < 4; ++p) {
      const uint32_t two = from[p];
      w |= (two & 15) << (4 * p) | (two >> 4) << (4 * p + 16);
    }
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
    if (zeros) {
      out[2 * i] = scales[from];
      out[2 * i + 1] = __float2bfloat16_rn(128.f + (zeros[from] & 15));
    } else {
      out[i] = scales[from];
    }
  }
}

// ---------------------------------------------------------------- the slots by expert
// Chunks of at most `chunk` rows of one expert; a row is a slot, in the slots' order within an
// expert.  One block.
struct Groups {
  int* count;      // [1] chunks
  int* expert;     // [E + slots / chunk]
  int* first;      // [...] its first row
  int* rows;       // [...] how many
  int* row_slot;   // [slots]
  int* slot_row;   // [slots], -1 for a bad expert
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

__global__ void __launch_bounds__(1024)
    w4_group_kernel(const int* idx, int slots, int E, int chunk, Groups g, int* dev_status) {
  extern __shared__ unsigned short seen[];  // [32][E]: slots of the expert in the warp's part
  __shared__ int sums[32];
  after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = (slots + 1023) / 1024 * 32;  // slots of a warp
  for (int i = threadIdx.x; i < 32 * E; i += 1024) seen[i] = 0;
  __syncthreads();
  const int lo = warp * part, hi = min(lo + part, slots);
  const auto pass = [&](auto put) {
    for (int at = lo; at < hi; at += 32) {
      const int slot = at + lane;
      int e = -1;
      if (slot < hi) {
        e = idx[slot];
        if (e < 0 || e >= E) e = -1;
      }
      const unsigned same = __match_any_sync(~0u, e);
      const int rank = __popc(same & ((1u << lane) - 1));
      const int before = e >= 0 ? seen[warp * E + e] : 0;
      __syncwarp();
      if (e >= 0 && rank == 0) seen[warp * E + e] = before + __popc(same);
      __syncwarp();
      if (slot < hi) put(slot, e, before + rank);
    }
  };
  pass([&](int, int e, int) {
    if (e < 0) report_status(dev_status, MOE_ERR_BAD_INDEX);
  });
  __syncthreads();
  int all = 0;
  const int e = threadIdx.x;
  if (e < E)
    for (int w = 0; w < 32; ++w) {
      const int n = seen[w * E + e];
      seen[w * E + e] = all;
      all += n;
    }
  const int chunks = (all + chunk - 1) / chunk;
  const int row = block_scan(all, sums), at = block_scan(chunks, sums);
  if (threadIdx.x == 1023) *g.count = at + chunks;
  for (int c = 0; c < chunks; ++c) {
    g.expert[at + c] = e;
    g.first[at + c] = row + c * chunk;
    g.rows[at + c] = min(chunk, all - c * chunk);
  }
  __shared__ int start[kMaxExperts];
  if (e < E) start[e] = row;
  __syncthreads();
  pass([&](int slot, int of, int rank) {
    const int r = of < 0 ? -1 : start[of] + rank;
    g.slot_row[slot] = r;
    if (r >= 0) g.row_slot[r] = slot;
  });
}

// ---------------------------------------------------------------- products

__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t less(uint32_t codes, uint32_t zero) {
  __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&codes),
                             *reinterpret_cast<__nv_bfloat162*>(&zero));
  return *reinterpret_cast<uint32_t*>(&v);
}

// Two codes of a word (those 2 p and 2 p + 1) as 128 + code in bf16, less 128 + zero.
__device__ __forceinline__ uint32_t two_codes(uint32_t word, int p, uint32_t zero) {
  return less((word >> (4 * p) & 0x000f000fu) | 0x43004300u, zero);
}

// One strip's weights, as the kernels read them.
struct Matrix {
  const uint4* codes;
  const uint32_t* scales;
};

struct Weights {
  const void* codes;
  const void* scales;
  int group;
};

// Scales (and zeros) of rows g and g + 8 in a group of columns.
template <bool ZEROS>
struct Scale {
  float s0, s1;
  uint32_t z0, z1;
  __device__ __forceinline__ void load(const uint32_t* scales, long long group, int g) {
    if constexpr (ZEROS) {
      const uint2 v = reinterpret_cast<const uint2*>(scales)[group * 8 + g];
      s0 = __uint_as_float(v.x << 16), s1 = __uint_as_float(v.y << 16);
      z0 = __byte_perm(v.x, 0, 0x3232), z1 = __byte_perm(v.y, 0, 0x3232);
    } else {
      const uint32_t v = scales[group * 8 + g];
      s0 = __uint_as_float(v << 16), s1 = __uint_as_float(v & 0xffff0000u);
      z0 = z1 = 0x43084308u;  // 136
    }
  }
};

// acc += W x^T over the tiles first, first + step, ... of a strip, for MATS matrices against NT x 8
// tokens, whose values are given in PIECES parts to add.  x[i]: the row of token 8 i + g (its tile
// begins at column 0), null for none; the second piece is `piece` values behind.
template <int MATS, int NT, int PIECES, bool ZEROS>
__device__ __forceinline__ void product(const Matrix (&m)[MATS], int group, int tiles, int first,
                                        int step, const __nv_bfloat16* const (&x)[NT],
                                        long long piece, float (&acc)[MATS][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr int U = 2;  // tiles on their way
  for (int tile = first; tile < tiles; tile += U * step) {
    uint4 w[U][MATS];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MATS; ++i)
        if (tile + u * step < tiles)
          w[u][i] = load_stream(m[i].codes + (tile + u * step) * 32ll + lane);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = tile + u * step;
      if (at >= tiles) break;
      uint4 v[2][NT][PIECES];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < PIECES; ++q) {
            v[c][n][q] = make_uint4(0, 0, 0, 0);
            if (x[n])
              v[c][n][q] = *reinterpret_cast<const uint4*>(x[n] + q * piece + at * kTile + c * 32 +
                                                           t * 8);
          }
#pragma unroll
      for (int i = 0; i < MATS; ++i) {
        Scale<ZEROS> s;
        float part[NT][4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c == 0 || group == 32) {
            s.load(m[i].scales, group == 32 ? at * 2 + c : group == 64 ? at : at >> 1, g);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r) part[n][r] = 0.f;
          }
          const uint32_t w0 = c ? w[u][i].z : w[u][i].x, w1 = c ? w[u][i].w : w[u][i].y;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a0 = two_codes(w0, 2 * h, s.z0), a1 = two_codes(w1, 2 * h, s.z1);
            const uint32_t a2 = two_codes(w0, 2 * h + 1, s.z0), a3 = two_codes(w1, 2 * h + 1, s.z1);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int q = 0; q < PIECES; ++q)
                mma(part[n], a0, a1, a2, a3, h ? v[c][n][q].z : v[c][n][q].x,
                    h ? v[c][n][q].w : v[c][n][q].y);
          }
          if (c == 1 || group == 32) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              acc[i][n][0] = fmaf(s.s0, part[n][0], acc[i][n][0]);
              acc[i][n][1] = fmaf(s.s0, part[n][1], acc[i][n][1]);
              acc[i][n][2] = fmaf(s.s1, part[n][2], acc[i][n][2]);
              acc[i][n][3] = fmaf(s.s1, part[n][3], acc[i][n][3]);
            }
          }
        }
      }
    }
  }
}

template <int MATS, bool ZEROS>
__device__ __forceinline__ Matrix strip_of(const Weights& w, int e, int rows, int cols, int strip) {
  const long long strips = rows / kStrip, at = e * strips + strip;
  return {static_cast<const uint4*>(w.codes) + at * (cols / kTile) * 32,
          static_cast<const uint32_t*>(w.scales) + at * (cols / w.group) * (ZEROS ? 16 : 8)};
}

// The warps of a block share a strip's tiles; their sums are added in the warps' order.
// put(i, row, token, sums of the MATS matrices) for all 16 x 8 NT of them.
template <int MATS, int NT, int PIECES, bool ZEROS, typename Put>
__device__ __forceinline__ void strip_product(const Matrix (&m)[MATS], int group, int cols,
                                              const __nv_bfloat16* const (&x)[NT],
                                              long long piece, float* sums, Put put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float acc[MATS][NT][4] = {};
  product<MATS, NT, PIECES, ZEROS>(m, group, cols / kTile, warp, kWarps, x, piece, acc);
  __syncthreads();  // (the last strip's readers are done)
#pragma unroll
  for (int i = 0; i < MATS; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        sums[(((warp * MATS + i) * NT + n) * 4 + r) * 32 + lane] = acc[i][n][r];
  __syncthreads();
  // place (n, r, lane) is row lane / 4 + r / 2 * 8, token 8 n + lane % 4 * 2 + r % 2
  for (int p = threadIdx.x; p < NT * 128; p += kWarps * 32) {
    float v[MATS] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
#pragma unroll
      for (int i = 0; i < MATS; ++i) v[i] += sums[(w * MATS + i) * NT * 128 + p];
    const int l = p & 31, r = p >> 5 & 3, n = p >> 7;
    put(l / 4 + r / 2 * 8, n * 8 + l % 4 * 2 + r % 2, v);
  }
}

struct GateUp {
  Groups g;
  Weights gate, up;
  const __nv_bfloat16* x;
  __nv_bfloat16* h;  // [2][slots][F]: two pieces
  int d, F, k, slots;
};

template <int NT, bool ZEROS>
__device__ __forceinline__ void gateup_task(const GateUp& p, int c, int strip, float* sums) {
  const int e = p.g.expert[c], first = p.g.first[c], rows = p.g.rows[c];
  const int g = (threadIdx.x & 31) >> 2;
  const Matrix m[2] = {strip_of<2, ZEROS>(p.gate, e, p.F, p.d, strip),
                       strip_of<2, ZEROS>(p.up, e, p.F, p.d, strip)};
  const __nv_bfloat16* x[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = n * 8 + g;
    x[n] = r < rows ? p.x + static_cast<long long>(p.g.row_slot[first + r] / p.k) * p.d : nullptr;
  }
  strip_product<2, NT, 1, ZEROS>(
      m, p.gate.group, p.d, x, 0, sums, [&](int row, int token, const float (&v)[2]) {
        if (token >= rows) return;
        const float a = v[0], h = a / (1.f + expf(-a)) * v[1];
        const __nv_bfloat16 hi = __float2bfloat16_rn(h);
        __nv_bfloat16* to = p.h + (first + token) * static_cast<long long>(p.F) + strip * kStrip + row;
        to[0] = hi;
        to[static_cast<long long>(p.slots) * p.F] = __float2bfloat16_rn(h - __bfloat162float(hi));
      });
}

template <int NT, bool ZEROS>
__global__ void __launch_bounds__(kWarps * 32) w4_gateup_kernel(const GateUp p) {
  __shared__ float sums[kWarps * 2 * NT * 128];
  after_previous();
  const int strips = p.F / kStrip;
  const long long tasks = static_cast<long long>(*p.g.count) * strips;
  for (long long task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int c = static_cast<int>(task / strips), strip = static_cast<int>(task % strips);
    gateup_task<NT, ZEROS>(p, c, strip, sums);
  }
}

struct Down {
  Groups g;
  Weights down;
  const __nv_bfloat16* h;
  float* out;  // [slots][d], a row to a slot, before the gates
  int d, F, slots;
};

template <int NT, bool ZEROS>
__global__ void __launch_bounds__(kWarps * 32) w4_down_kernel(const Down p) {
  __shared__ float sums[kWarps * NT * 128];
  after_previous();
  const int strips = p.d / kStrip;
  const long long tasks = static_cast<long long>(*p.g.count) * strips;
  const int g = (threadIdx.x & 31) >> 2;
  for (long long task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int c = static_cast<int>(task / strips), strip = static_cast<int>(task % strips);
    const int e = p.g.expert[c], first = p.g.first[c], rows = p.g.rows[c];
    const Matrix m[1] = {strip_of<1, ZEROS>(p.down, e, p.d, p.F, strip)};
    const __nv_bfloat16* x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      x[n] = n * 8 + g < rows ? p.h + (first + n * 8 + g) * static_cast<long long>(p.F) : nullptr;
    strip_product<1, NT, 2, ZEROS>(
        m, p.down.group, p.F, x, static_cast<long long>(p.slots) * p.F, sums,
        [&](int row, int token, const float (&v)[1]) {
          if (token < rows)
            p.out[(first + token) * static_cast<long long>(p.d) + strip * kStrip + row] = v[0];
        });
  }
}

// y_t = sum_j gate_j out[row of slot (t, j)], in the slots' order.
__global__ void __launch_bounds__(256)
    w4_combine_kernel(const float* out, const int* slot_row, const float* gate, int T, int d, int k,
                      __nv_bfloat16* y) {
  after_previous();
  const long long pairs = static_cast<long long>(T) * d / 2;
  const long long step = gridDim.x * 256ll;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < pairs; i += step) {
    const int t = static_cast<int>(i / (d / 2)), c = static_cast<int>(i % (d / 2)) * 2;
    float2 sum = make_float2(0.f, 0.f);
    for (int j = 0; j < k; ++j) {
      const int r = slot_row[t * k + j];
      if (r < 0) continue;
      const float w = gate[t * k + j];
      const float2 v = *reinterpret_cast<const float2*>(out + static_cast<long long>(r) * d + c);
      sum.x = fmaf(w, v.x, sum.x);
      sum.y = fmaf(w, v.y, sum.y);
    }
    *reinterpret_cast<uint32_t*>(y + static_cast<long long>(t) * d + c) =
        pack_bf16x2(sum.x, sum.y);
  }
}

// ------------------------------------------------------------------------ host side

constexpr int kSms = 152;
constexpr int kBlocks = 4;  // to an SM

// Rows of an expert that its weights are read once for; more of them are taken in several chunks.
int chunk_of(int T) { return T <= 8 ? 8 : T <= 16 ? 16 : 32; }

struct Workspace {
  Groups g;
  __nv_bfloat16* h;
  float* out;
  size_t bytes;
};

Workspace carve(const moe_problem* p, void* base) {
  const size_t slots = static_cast<size_t>(p->T) * p->k, chunk = chunk_of(p->T);
  const size_t chunks = std::min<size_t>(p->E, slots) + slots / chunk;
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
  w.g.slot_row = reinterpret_cast<int*>(take(slots * 4));
  w.h = reinterpret_cast<__nv_bfloat16*>(take(slots * p->F * 4));
  w.out = reinterpret_cast<float*>(take(slots * p->d * 4));
  return w;
}

int check_w4(const moe_problem* p) {
  if (int e = check_problem(p)) return e;
  if (p->r || static_cast<long long>(p->T) * p->k > kMaxSlots) return MOE_ERR_UNSUPPORTED;
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
  if (static_cast<long long>(E) * rows > (1ll << 40) / cols) return MOE_ERR_UNSUPPORTED;
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
  if (w_gate->group != w_up->group || zeros != (w_up->has_zeros != 0) ||
      zeros != (w_down->has_zeros != 0))
    return MOE_ERR_UNSUPPORTED;
  if (misaligned(x, 16) || misaligned(y, 16) || misaligned(topk_idx, 4) ||
      misaligned(topk_gate, 4) || misaligned(dev_status, 4))
    return MOE_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < carve(p, nullptr).bytes) return MOE_ERR_WORKSPACE;
  if (misaligned(workspace, 16)) return MOE_ERR_UNSUPPORTED;
  const Workspace ws = carve(p, workspace);
  const int slots = p->T * p->k, chunk = chunk_of(p->T);
  const auto of = [](const moe_w4* w) { return Weights{w->codes, w->scales, w->group}; };
  const GateUp up{ws.g, of(w_gate), of(w_up), reinterpret_cast<const __nv_bfloat16*>(x), ws.h,
                  p->d, p->F, p->k, slots};
  const Down down{ws.g, of(w_down), ws.h, ws.out, p->d, p->F, slots};
  const int smem = 32 * p->E * 2;
  cudaError_t err = launched(cudaFuncSetAttribute(
      w4_group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 32 * kMaxExperts * 2));
  mark_before(MOE_KERNEL_W4_GATEUP, stream);
  if (err == cudaSuccess)
    err = launch_behind(w4_group_kernel, 1, 1024, smem, stream, topk_idx, slots, p->E, chunk, ws.g,
                        dev_status);
  const auto run = [&](auto nt, auto z) {
    constexpr int NT = decltype(nt)::value;
    constexpr bool Z = decltype(z)::value;
    if (err == cudaSuccess)
      err = launch_behind(w4_gateup_kernel<NT, Z>, kBlocks * kSms, kWarps * 32, 0, stream, up);
    mark_after(MOE_KERNEL_W4_GATEUP, stream);
    mark_before(MOE_KERNEL_W4_DOWN, stream);
    if (err == cudaSuccess)
      err = launch_behind(w4_down_kernel<NT, Z>, kBlocks * kSms, kWarps * 32, 0, stream, down);
  };
  const auto with_chunk = [&](auto z) {
    if (chunk == 8)
      run(std::integral_constant<int, 1>{}, z);
    else if (chunk == 16)
      run(std::integral_constant<int, 2>{}, z);
    else
      run(std::integral_constant<int, 4>{}, z);
  };
  if (zeros)
    with_chunk(std::true_type{});
  else
    with_chunk(std::false_type{});
  if (err == cudaSuccess) {
    const long long pairs = static_cast<long long>(p->T) * p->d / 2;
    err = launch_behind(w4_combine_kernel,
                        static_cast<int>(std::min<long long>((pairs + 255) / 256, 8ll * kSms)), 256, 0, stream,
                        ws.out, ws.g.slot_row, topk_gate, p->T, p->d, p->k,
                        reinterpret_cast<__nv_bfloat16*>(y));
  }
  mark_after(MOE_KERNEL_W4_DOWN, stream);
  count_launches(4);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
