// Gated linear recurrence over packed sequences, forward, backward and one token
// (include/linear_recurrence.h has the formulas).
#include "moe_internal.h"
#include "slots.cuh"

#include "../../include/linear_recurrence.h"

namespace moe {
namespace {

constexpr int kChunk = 64;  // rows between the kept states

__device__ __forceinline__ float ld(const float* p, long long i) { return p[i]; }
__device__ __forceinline__ float ld(const __nv_bfloat16* p, long long i) {
  return __bfloat162float(p[i]);
}
__device__ __forceinline__ void st(float* p, long long i, float v) { p[i] = v; }
__device__ __forceinline__ void st(__nv_bfloat16* p, long long i, float v) {
  p[i] = __float2bfloat16_rn(v);
}

struct Range {
  int lo, hi;
};

// Rows of sequence s, inside [0, N] whatever seq_off holds.
__device__ __forceinline__ Range rows_of(int s, int N, int n_seq, const int* seq_off) {
  if (!seq_off) return {s * (N / n_seq), (s + 1) * (N / n_seq)};
  const int lo = max(seq_off[s], 0), hi = min(seq_off[s + 1], N);
  return {lo, hi};
}

__device__ __forceinline__ void check_offsets(int s, int N, int n_seq, const int* seq_off,
                                              int* dev_status) {
  if (!seq_off || !dev_status) return;
  const int lo = seq_off[s], hi = seq_off[s + 1];
  if (lo > hi || lo < 0 || hi > N || (s == 0 && lo != 0))
    atomicCAS(dev_status, 0, MOE_ERR_BAD_INDEX);
}

// One thread per sequence and channel.
template <typename T, bool MIX>
__global__ void glr_forward_kernel(int N, int D, int n_seq, const int* seq_off, const T* g,
                                   long long ld_g, const T* x, long long ld_x, const float* h0,
                                   T* h, float* h_T, float* h_chunks, int* dev_status) {
  const int s = blockIdx.y, d = blockIdx.x * blockDim.x + threadIdx.x;
  if (d == 0) check_offsets(s, N, n_seq, seq_off, dev_status);
  if (d >= D) return;
  const Range r = rows_of(s, N, n_seq, seq_off);
  float now = h0 ? h0[static_cast<long long>(s) * D + d] : 0.f;
  for (int t = r.lo; t < r.hi; ++t) {
    if (h_chunks && t % kChunk == 0)
      h_chunks[static_cast<long long>(t / kChunk) * D + d] = t == r.lo ? 0.f : now;
    const float lg = ld(g, t * ld_g + d), xv = ld(x, t * ld_x + d);
    now = fmaf(expf(lg), now, MIX ? -expm1f(lg) * xv : xv);
    st(h, static_cast<long long>(t) * D + d, now);
  }
  if (h_T) h_T[static_cast<long long>(s) * D + d] = now;
}

// One thread per sequence and channel: 64-row pieces from the last to the first, the states in
// front of each row formed again from the kept one.
template <typename T, bool MIX>
__global__ void glr_backward_kernel(int N, int D, int n_seq, const int* seq_off, const T* g,
                                    long long ld_g, const T* x, long long ld_x, const float* h0,
                                    const float* h_chunks, const T* dh, const float* dh_T, T* dg,
                                    T* dx, float* dh0, int* dev_status) {
  const int s = blockIdx.y, d = blockIdx.x * blockDim.x + threadIdx.x;
  if (d == 0) check_offsets(s, N, n_seq, seq_off, dev_status);
  if (d >= D) return;
  const Range r = rows_of(s, N, n_seq, seq_off);
  const long long sd = static_cast<long long>(s) * D + d;
  float back = dh_T ? dh_T[sd] : 0.f;
  float before[kChunk];
  for (int hi = r.hi; hi > r.lo;) {
    const int lo = max(r.lo, (hi - 1) / kChunk * kChunk);
    float now = lo == r.lo ? (h0 ? h0[sd] : 0.f)
                           : h_chunks[static_cast<long long>(lo / kChunk) * D + d];
    for (int t = lo; t < hi; ++t) {
      const float lg = ld(g, t * ld_g + d), xv = ld(x, t * ld_x + d);
      before[t - lo] = now;
      now = fmaf(expf(lg), now, MIX ? -expm1f(lg) * xv : xv);
    }
    for (int t = hi - 1; t >= lo; --t) {
      const float lg = ld(g, t * ld_g + d), xv = ld(x, t * ld_x + d);
      const float lam = ld(dh, static_cast<long long>(t) * D + d) + back;
      back = expf(lg) * lam;
      st(dx, t * ld_x + d, MIX ? -expm1f(lg) * lam : lam);
      st(dg, t * ld_g + d, back * (MIX ? before[t - lo] - xv : before[t - lo]));
    }
    hi = lo;
  }
  if (dh0) dh0[sd] = back;
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
  if (n_seq > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
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
  if (n_seq > 65535) return MOE_ERR_UNSUPPORTED;
  const dim3 grid((D + 63) / 64, n_seq);
  mark_before(MOE_KERNEL_GLR_FWD, stream);
  GLR_LAUNCH(glr_forward_kernel, grid, 64, N, D, n_seq, seq_off, static_cast<const T*>(g), ld_g,
             static_cast<const T*>(x), ld_x, h0, static_cast<T*>(h), h_T, h_chunks, dev_status);
  const cudaError_t err = cudaGetLastError();
  mark_after(MOE_KERNEL_GLR_FWD, stream);
  count_launches(1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_glr_backward(int32_t N, int32_t D, int32_t n_seq, const int32_t* seq_off, int32_t mode,
                     int32_t dtype, const void* g, int64_t ld_g, const void* x, int64_t ld_x,
                     const float* h0, const float* h_chunks, const void* dh, const float* dh_T,
                     void* dg, void* dx, float* dh0, int32_t* dev_status, moe_stream_t stream) {
  if (int e = check_rows(N, D, n_seq, seq_off, mode, dtype, g, ld_g, x, ld_x, dg, true)) return e;
  if (!h_chunks || !dh || !dx) return MOE_ERR_INVALID_ARG;
  const int size = dtype == MOE_BF16 ? 2 : 4;
  if (misaligned(dh, size) || misaligned(dx, size)) return MOE_ERR_UNSUPPORTED;
  if (n_seq > 65535) return MOE_ERR_UNSUPPORTED;
  const dim3 grid((D + 63) / 64, n_seq);
  mark_before(MOE_KERNEL_GLR_BWD, stream);
  GLR_LAUNCH(glr_backward_kernel, grid, 64, N, D, n_seq, seq_off, static_cast<const T*>(g), ld_g,
             static_cast<const T*>(x), ld_x, h0, h_chunks, static_cast<const T*>(dh), dh_T,
             static_cast<T*>(dg), static_cast<T*>(dx), dh0, dev_status);
  const cudaError_t err = cudaGetLastError();
  mark_after(MOE_KERNEL_GLR_BWD, stream);
  count_launches(1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
