// One token of the gated delta rule for a batch of requests (include/linear_attention.h).
#include "moe_internal.h"
#include "slots.cuh"

#include "../../include/linear_attention.h"

namespace moe {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Value rows of the state do not depend on one another: with r = v - a S k^ (a = exp(g)) each
// row does S <- a S + beta r k^ and o = scale (a S q^ + beta r (k^ . q^)), so both products of
// the old row are taken in one pass over it.  One warp per value row.
template <int DK>
__global__ void __launch_bounds__(256)
    gdr_step_kernel(int B, int H, int dv, const __nv_bfloat16* q, const __nv_bfloat16* k,
                    const __nv_bfloat16* v, const float* beta, const float* g, const int* slot,
                    int n_slots, float scale, float* S, __nv_bfloat16* o, int* dev_status) {
  constexpr int NV = DK / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / H, h = blockIdx.x % H;
  const int row = claimed_slot(b, slot, n_slots, dev_status);
  if (row < 0) return;
  const long long bh = static_cast<long long>(b) * H + h;
  float qv[NV], kv[NV], qq = 0.f, kk = 0.f, kq = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    qv[j] = __bfloat162float(q[bh * DK + lane + 32 * j]);
    kv[j] = __bfloat162float(k[bh * DK + lane + 32 * j]);
    qq += qv[j] * qv[j];
    kk += kv[j] * kv[j];
  }
  qq = warp_sum(qq);
  kk = warp_sum(kk);
  const float rq = qq > 0.f ? rsqrtf(qq) : 0.f, rk = kk > 0.f ? rsqrtf(kk) : 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    qv[j] *= rq;
    kv[j] *= rk;
    kq += qv[j] * kv[j];
  }
  kq = warp_sum(kq);
  const float a = expf(g[bh]), bt = beta[bh];
  float* Sh = S + (static_cast<long long>(row) * H + h) * dv * DK;
  for (int i = warp; i < dv; i += 8) {
    float s[NV], sk = 0.f, sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      s[j] = a * Sh[i * DK + lane + 32 * j];
      sk += s[j] * kv[j];
      sq += s[j] * qv[j];
    }
    sk = warp_sum(sk);
    sq = warp_sum(sq);
    const float w = bt * (__bfloat162float(v[bh * dv + i]) - sk);
#pragma unroll
    for (int j = 0; j < NV; ++j) Sh[i * DK + lane + 32 * j] = s[j] + w * kv[j];
    if (lane == 0) o[bh * dv + i] = __float2bfloat16_rn(scale * (sq + w * kq));
  }
}

}  // namespace
}  // namespace moe

extern "C" int moe_gdr_step(int32_t B, int32_t H, int32_t dk, int32_t dv, const moe_bf16* q,
                            const moe_bf16* k, const moe_bf16* v, const float* beta,
                            const float* g, const int32_t* slot, int32_t n_slots, float scale,
                            float* S, moe_bf16* o, int32_t* dev_status, moe_stream_t stream) {
  using namespace moe;
  if (B <= 0 || H <= 0 || n_slots <= 0 || !q || !k || !v || !beta || !g || !S || !o)
    return MOE_ERR_INVALID_ARG;
  if (!slot && B > n_slots) return MOE_ERR_INVALID_ARG;
  if (!((dk == 64 || dk == 128) && (dv == 64 || dv == 128))) return MOE_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H > (1ll << 24)) return MOE_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
       reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(S) |
       reinterpret_cast<uintptr_t>(o)) & 15u)
    return MOE_ERR_UNSUPPORTED;
  const auto* q_ = reinterpret_cast<const __nv_bfloat16*>(q);
  const auto* k_ = reinterpret_cast<const __nv_bfloat16*>(k);
  const auto* v_ = reinterpret_cast<const __nv_bfloat16*>(v);
  auto* o_ = reinterpret_cast<__nv_bfloat16*>(o);
  mark_before(MOE_KERNEL_GDR_STEP, stream);
  if (dk == 128)
    gdr_step_kernel<128><<<B * H, 256, 0, stream>>>(B, H, dv, q_, k_, v_, beta, g, slot, n_slots,
                                                    scale, S, o_, dev_status);
  else
    gdr_step_kernel<64><<<B * H, 256, 0, stream>>>(B, H, dv, q_, k_, v_, beta, g, slot, n_slots,
                                                   scale, S, o_, dev_status);
  const cudaError_t err = cudaGetLastError();
  mark_after(MOE_KERNEL_GDR_STEP, stream);
  count_launches(1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
