// One token of the gated delta rule for a batch of requests (include/linear_attention.h).
#include "moe_internal.h"
#include "overlap.cuh"
#include "slots.cuh"

#include "../../include/linear_attention.h"

namespace moe {
namespace {

// Value rows of the state do not depend on one another: with r = v - a S k^ (a = exp(g)) each
// row does S <- a S + beta r k^ and o = scale (a S q^ + beta r (k^ . q^)), so both products of
// the old row are taken in one pass over it, and the state is read and written once, which bounds
// the step.  DK / 4 lanes hold a row, four values each; a lane has kRows rows on their way at once.
constexpr int kRows = 8;
constexpr int kThreads = 128;

template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Sums of 16 values over W lanes, halving the values with the lanes (16 shuffles instead of 16
// log2(W)): the lane with place p (of W) gets the sum of value p 16 / W.
template <int W>
__device__ __forceinline__ float sums_of_16(float (&v)[16], int lane) {
#pragma unroll
  for (int n = 8, o = W / 2; n; n >>= 1, o >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool up = lane & o;
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(~0u, give, o);
    }
  return W == 32 ? v[0] + __shfl_xor_sync(~0u, v[0], 1) : v[0];
}

__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
  v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
}

template <int DK>
__device__ __forceinline__ float dot(const float (&a)[4], const float (&b)[4]) {
  return fmaf(a[0], b[0], fmaf(a[1], b[1], fmaf(a[2], b[2], a[3] * b[3])));
}

// 256 requests x 16 heads x 128 x 128 (537 MB of states both ways) take 79.8 us, the rate of a
// plain copy; a single request 2.1 us in a graph of such steps, two dependent round trips to memory.
template <int DK>
__global__ void __launch_bounds__(kThreads)
    gdr_step_kernel(int H, int dv, const __nv_bfloat16* q, const __nv_bfloat16* k,
                    const __nv_bfloat16* v, const float* beta, const float* g, const int* slot,
                    int n_slots, float scale, float* S, __nv_bfloat16* o, int* dev_status) {
  constexpr int W = DK / 4;                       // lanes of a row
  constexpr int kBlockRows = kThreads / W * kRows;
  const int parts = dv / kBlockRows;
  const int part = blockIdx.x % parts;
  const long long bh = blockIdx.x / parts;
  const int b = static_cast<int>(bh / H), h = static_cast<int>(bh % H);
  const int lane = threadIdx.x & 31, place = threadIdx.x % W;
  const int first = part * kBlockRows + threadIdx.x / W * kRows;  // value row

  after_previous();
  const int row = slot ? slot[b] : b;
  float qv[4], kv[4];
  load4(q + bh * DK + place * 4, qv);
  load4(k + bh * DK + place * 4, kv);
  const float a = expf(g[bh]), bt = beta[bh];
  // the place p = 2 r + 1 (of 16) will have row r's output
  constexpr int kShare = W / 16;
  const int r_mine = place / kShare / 2;
  const float v_mine = __bfloat162float(v[bh * dv + first + r_mine]);
  if (row < 0 || row >= n_slots) {
    if (row != -1 && threadIdx.x == 0 && dev_status) atomicCAS(dev_status, 0, MOE_ERR_BAD_INDEX);
    return;
  }
  float* Sr = S + ((static_cast<long long>(row) * H + h) * dv + first) * DK + place * 4;
  float4 s[kRows];  // (of a request that is refused below, they are read in vain)
#pragma unroll
  for (int r = 0; r < kRows; ++r) s[r] = *reinterpret_cast<const float4*>(Sr + r * DK);
  if (slot && named_before(b, row, slot, dev_status)) return;

  const float qq = lanes_sum<W>(dot<DK>(qv, qv)), kk = lanes_sum<W>(dot<DK>(kv, kv));
  const float rq = qq > 0.f ? rsqrtf(qq) : 0.f, rk = kk > 0.f ? rsqrtf(kk) : 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) qv[j] *= rq, kv[j] *= rk;
  const float kq = lanes_sum<W>(dot<DK>(qv, kv));
  float sums[16];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    s[r].x *= a, s[r].y *= a, s[r].z *= a, s[r].w *= a;
    const float sv[4] = {s[r].x, s[r].y, s[r].z, s[r].w};
    sums[2 * r] = dot<DK>(sv, kv);
    sums[2 * r + 1] = dot<DK>(sv, qv);
  }
  const float sum = sums_of_16<W>(sums, lane);
  const int base = lane - place;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float sk = __shfl_sync(~0u, sum, base + 2 * r * kShare);
    const float vr = __shfl_sync(~0u, v_mine, base + 2 * r * kShare);
    const float w = bt * (vr - sk);
    *reinterpret_cast<float4*>(Sr + r * DK) =
        make_float4(fmaf(w, kv[0], s[r].x), fmaf(w, kv[1], s[r].y), fmaf(w, kv[2], s[r].z),
                    fmaf(w, kv[3], s[r].w));
  }
  const float sk = __shfl_sync(~0u, sum, base + 2 * r_mine * kShare);
  if (place % (2 * kShare) == kShare)
    o[bh * dv + first + r_mine] = __float2bfloat16_rn(scale * fmaf(bt * (v_mine - sk), kq, sum));
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
  if (slot && B > kMaxSlots) return MOE_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(q), static_cast<const void*>(k),
                        static_cast<const void*>(v), static_cast<const void*>(S),
                        static_cast<const void*>(o)})
    if (misaligned(p, 16)) return MOE_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(beta), static_cast<const void*>(g),
                        static_cast<const void*>(slot), static_cast<const void*>(dev_status)})
    if (misaligned(p, 4)) return MOE_ERR_UNSUPPORTED;
  const auto* q_ = reinterpret_cast<const __nv_bfloat16*>(q);
  const auto* k_ = reinterpret_cast<const __nv_bfloat16*>(k);
  const auto* v_ = reinterpret_cast<const __nv_bfloat16*>(v);
  auto* o_ = reinterpret_cast<__nv_bfloat16*>(o);
  mark_before(MOE_KERNEL_GDR_STEP, stream);
  const auto launch = [&](auto kernel, int lanes) {
    const int parts = dv / (kThreads / lanes * kRows);
    return launch_behind(kernel, dim3(static_cast<unsigned>(B) * H * parts), kThreads, 0, stream, H, dv,
                         q_, k_, v_, beta, g, slot, n_slots, scale, S, o_, dev_status);
  };
  const cudaError_t err =
      dk == 128 ? launch(gdr_step_kernel<128>, 32) : launch(gdr_step_kernel<64>, 16);
  mark_after(MOE_KERNEL_GDR_STEP, stream);
  count_launches(1);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
