// Norm of query and key heads with the rotation by position, forward and backward
// (include/linear_attention.h has the formulas).
#include <math.h>

#include "moe_internal.h"

#include "../../include/linear_attention.h"

namespace moe {
namespace {

constexpr int kMaxD = 256;

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

__device__ __forceinline__ float ld(const float* p, long long i) { return p[i]; }
__device__ __forceinline__ float ld(const __nv_bfloat16* p, long long i) {
  return __bfloat162float(p[i]);
}
__device__ __forceinline__ void st(float* p, long long i, float v) { p[i] = v; }
__device__ __forceinline__ void st(__nv_bfloat16* p, long long i, float v) {
  p[i] = __float2bfloat16_rn(v);
}

// cos and sin of pos * inv_freq: the angle in turns, in 64 bits, less its whole turns; what is
// left (at most half a turn) is exact to 2^-25 of a turn in fp32.
__device__ __forceinline__ float2 cos_sin(int pos, double inv_freq) {
  double turns = static_cast<double>(pos) * (inv_freq * 0.15915494309189533577);
  turns -= rint(turns);
  float2 cs;
  sincospif(2.f * static_cast<float>(turns), &cs.y, &cs.x);
  return cs;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// One warp per (token, head).
template <typename T>
__global__ void __launch_bounds__(256) rope_forward_kernel(int N, int D, int rot, int interleaved,
                                                           float eps, const int* pos,
                                                           const double* inv_freq, Side q, Side k) {
  __shared__ float rows[8][kMaxD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = q.heads + k.heads;
  const long long r = static_cast<long long>(blockIdx.x) * 8 + warp;
  if (r >= static_cast<long long>(N) * heads) return;
  const int t = static_cast<int>(r / heads);
  int h = static_cast<int>(r % heads);
  const Side& s = h < q.heads ? q : k;
  if (h >= q.heads) h -= q.heads;
  const T* x = static_cast<const T*>(s.x) + t * s.x_ts + h * s.x_hs;
  T* y = static_cast<T*>(s.out) + t * s.o_ts + h * s.o_hs;
  float* n = rows[warp];
  float sum = 0.f;
  for (int i = lane; i < D; i += 32) {
    n[i] = ld(x, i);
    sum += n[i] * n[i];
  }
  const float rstd = rsqrtf(warp_sum(sum) / D + eps);
  for (int i = lane; i < D; i += 32)
    n[i] *= rstd * (s.weight ? s.weight[static_cast<long long>(h) * s.w_hs + i] : 1.f);
  __syncwarp();
  for (int i = lane; i < rot / 2; i += 32) {
    const int a = interleaved ? 2 * i : i, b = interleaved ? 2 * i + 1 : i + rot / 2;
    const float2 cs = cos_sin(pos[t], inv_freq[i]);
    st(y, a, n[a] * cs.x - n[b] * cs.y);
    st(y, b, n[b] * cs.x + n[a] * cs.y);
  }
  for (int i = rot + lane; i < D; i += 32) st(y, i, n[i]);
}

// Blocks (split, head): each of the 8 warps takes every 8th token of the split, so the weight
// gradient of a head gathers in registers; partial [splits][heads][D] holds the blocks' sums.
template <typename T, typename G>
__global__ void __launch_bounds__(256) rope_backward_kernel(int N, int D, int rot, int interleaved,
                                                            float eps, const int* pos,
                                                            const double* inv_freq, Side q, Side k,
                                                            int per_split, float* partial) {
  __shared__ float rows[8][kMaxD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.y;
  const Side& s = c < q.heads ? q : k;
  const int h = c < q.heads ? c : c - q.heads;
  const long long lo = static_cast<long long>(blockIdx.x) * per_split;
  const long long hi = min(lo + per_split, static_cast<long long>(N));
  float* n = rows[warp];
  float w[kMaxD / 32], dw[kMaxD / 32];
#pragma unroll
  for (int j = 0; j < kMaxD / 32; ++j) {
    const int i = lane + 32 * j;
    w[j] = i < D && s.weight ? s.weight[static_cast<long long>(h) * s.w_hs + i] : 1.f;
    dw[j] = 0.f;
  }
  for (long long t = lo + warp; t < hi; t += 8) {
    const T* x = static_cast<const T*>(s.x) + t * s.x_ts + h * s.x_hs;
    const G* dy = static_cast<const G*>(s.dy) + t * s.dy_ts + h * s.dy_hs;
    T* dx = static_cast<T*>(s.out) + t * s.o_ts + h * s.o_hs;
    for (int i = lane; i < rot / 2; i += 32) {
      const int a = interleaved ? 2 * i : i, b = interleaved ? 2 * i + 1 : i + rot / 2;
      const float2 cs = cos_sin(pos[t], inv_freq[i]);
      const float da = ld(dy, a), db = ld(dy, b);
      n[a] = da * cs.x + db * cs.y;
      n[b] = db * cs.x - da * cs.y;
    }
    for (int i = rot + lane; i < D; i += 32) n[i] = ld(dy, i);
    float xv[kMaxD / 32], sum = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxD / 32; ++j) {
      const int i = lane + 32 * j;
      xv[j] = i < D ? ld(x, i) : 0.f;
      sum += xv[j] * xv[j];
    }
    const float rstd = rsqrtf(warp_sum(sum) / D + eps);
    __syncwarp();
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxD / 32; ++j) {
      const int i = lane + 32 * j;
      if (i < D) {
        xv[j] *= rstd;
        dw[j] += n[i] * xv[j];
        dot += n[i] * w[j] * xv[j];
      }
    }
    dot = warp_sum(dot) / D;
#pragma unroll
    for (int j = 0; j < kMaxD / 32; ++j) {
      const int i = lane + 32 * j;
      if (i < D) st(dx, i, rstd * (n[i] * w[j] - xv[j] * dot));
    }
    __syncwarp();
  }
  if (!partial) return;
#pragma unroll
  for (int j = 0; j < kMaxD / 32; ++j)
    if (lane + 32 * j < D) n[lane + 32 * j] = dw[j];
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += 256) {
    float sum = 0.f;
    for (int v = 0; v < 8; ++v) sum += rows[v][i];
    partial[(static_cast<long long>(blockIdx.x) * gridDim.y + c) * D + i] = sum;
  }
}

// dweight from the blocks' sums: one thread per value, the splits (and, for a shared row, the
// heads) in order.
__global__ void rope_dweight_kernel(const float* partial, int splits, int heads, int D,
                                    int first_head, int n_heads, int per_head, float* dweight) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (per_head ? n_heads : 1) * D) return;
  const int h0 = per_head ? i / D : 0, h1 = per_head ? h0 + 1 : n_heads;
  float sum = 0.f;
  for (int s = 0; s < splits; ++s)
    for (int h = h0; h < h1; ++h)
      sum += partial[(static_cast<long long>(s) * heads + first_head + h) * D + i % D];
  dweight[i] = sum;
}

// ------------------------------------------------------------------------ host side

int per_split_of(int N) { return N <= 64 * 64 ? 64 : (N + 63) / 64; }
int splits_of(int N) { return (N + per_split_of(N) - 1) / per_split_of(N); }

bool bad_align(const void* p) { return reinterpret_cast<uintptr_t>(p) & 15u; }

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
  if (D % 8 || D > kMaxD || rot % 16) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_rows(const void* p, long long ts, long long hs) {
  if (!p) return MOE_ERR_INVALID_ARG;
  return bad_align(p) || ts % 8 || hs % 8 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

int check_heads(int N, int heads, const float* weight) {
  if (heads <= 0) return MOE_ERR_INVALID_ARG;
  if (heads > 4096 || bad_align(weight)) return MOE_ERR_UNSUPPORTED;
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

size_t backward_ws(int N, int D, int q_heads, int k_heads) {
  return up256(static_cast<size_t>(splits_of(N)) * (q_heads + k_heads) * D * 4);
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
  const long long rows = static_cast<long long>(N) * (sq.heads + sk.heads);
  if ((rows + 7) / 8 > 0x7fffffffll) return MOE_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  mark_before(MOE_KERNEL_QK_NORM_ROPE, stream);
  if (dtype == MOE_BF16)
    rope_forward_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(
        N, D, rotary_dim, interleaved, eps, positions, inv_freq, sq, sk);
  else
    rope_forward_kernel<float><<<grid, 256, 0, stream>>>(N, D, rotary_dim, interleaved, eps,
                                                         positions, inv_freq, sq, sk);
  const cudaError_t err = cudaGetLastError();
  mark_after(MOE_KERNEL_QK_NORM_ROPE, stream);
  count_launches(1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_qk_norm_rope_backward_workspace_size(int32_t N, int32_t D, int32_t q_heads,
                                                int32_t k_heads) {
  if (N <= 0 || D <= 0 || q_heads <= 0 || k_heads < 0) return 0;
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
  const dim3 grid(splits_of(N), heads);
  const int per = per_split_of(N);
  mark_before(MOE_KERNEL_QK_NORM_ROPE_BWD, stream);
  if (dtype == MOE_F32)
    rope_backward_kernel<float, float><<<grid, 256, 0, stream>>>(
        N, D, rotary_dim, interleaved, eps, positions, inv_freq, sq, sk, per, partial);
  else if (dy_dtype == MOE_F32)
    rope_backward_kernel<__nv_bfloat16, float><<<grid, 256, 0, stream>>>(
        N, D, rotary_dim, interleaved, eps, positions, inv_freq, sq, sk, per, partial);
  else
    rope_backward_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, 256, 0, stream>>>(
        N, D, rotary_dim, interleaved, eps, positions, inv_freq, sq, sk, per, partial);
  int launches = 1;
  const auto reduce = [&](float* dw, int first, int n, int per_head) {
    const int values = (per_head ? n : 1) * D;
    rope_dweight_kernel<<<(values + 127) / 128, 128, 0, stream>>>(partial, grid.x, heads, D, first,
                                                                  n, per_head, dw);
    ++launches;
  };
  if (q->dweight) reduce(q->dweight, 0, sq.heads, q->weight_per_head != 0);
  if (k && k->dweight) reduce(k->dweight, sq.heads, sk.heads, k->weight_per_head != 0);
  const cudaError_t err = cudaGetLastError();
  mark_after(MOE_KERNEL_QK_NORM_ROPE_BWD, stream);
  count_launches(launches);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
