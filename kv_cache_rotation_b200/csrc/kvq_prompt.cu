// Causal attention over whole packed prompts (kvq_attend_prompt):
//   out_i = sum_{n <= i} p_n v_n,  p = softmax_n(scale * q_i . k_n)
// in one pass over the keys with the running maximum and sum of the softmax.
#include <cuda_bf16.h>
#include <math.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

template <typename T>
__device__ __forceinline__ float2 to_f2(uint32_t w);
template <>
__device__ __forceinline__ float2 to_f2<__half>(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
template <>
__device__ __forceinline__ float2 to_f2<__nv_bfloat16>(uint32_t w) { return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w)); }

// One warp per (row, query head), a lane per D / 32 channels.
template <typename T, int D>
__global__ void __launch_bounds__(256) k_prompt_rows(const PromptArgs a) {
  constexpr int W = D / 64;  // 32-bit words per lane
  const int lane = threadIdx.x & 31;
  const long long wi = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int row = static_cast<int>(wi / a.q_heads), qh = static_cast<int>(wi % a.q_heads);
  if (row >= a.n_rows) return;
  int r0 = -1;
  for (int s = 0; s < a.n_seqs; ++s) {
    const int b = __ldg(a.cu_rows + s), e = __ldg(a.cu_rows + s + 1);
    if (row >= b && row < e && row - b < a.max_rows) r0 = max(b, 0);
  }
  if (r0 < 0) return;
  const int h = qh / (a.q_heads / a.heads);
  float q[2 * W], o[2 * W], m = -INFINITY, l = 0.0f;
  const uint32_t* qp = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) + row * a.q_stride + qh * D) + lane * W;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float2 f = to_f2<T>(qp[i]);
    q[2 * i] = f.x, q[2 * i + 1] = f.y;
    o[2 * i] = o[2 * i + 1] = 0.0f;
  }
  for (int n = r0; n <= row; ++n) {
    const uint32_t* kp = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.k) + n * a.k_stride + h * D) + lane * W;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 f = to_f2<T>(__ldg(kp + i));
      s = fmaf(q[2 * i], f.x, fmaf(q[2 * i + 1], f.y, s));
    }
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= a.scale;
    const float mn = fmaxf(m, s), f = m == mn ? 1.0f : __expf(m - mn), p = __expf(s - mn);
    m = mn;
    l = fmaf(l, f, p);
    const uint32_t* vp = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.v) + n * a.v_stride + h * D) + lane * W;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 v = to_f2<T>(__ldg(vp + i));
      o[2 * i] = fmaf(o[2 * i], f, p * v.x);
      o[2 * i + 1] = fmaf(o[2 * i + 1], f, p * v.y);
    }
  }
  T* op = static_cast<T*>(a.out) + row * a.out_stride + qh * D + lane * 2 * W;
#pragma unroll
  for (int i = 0; i < 2 * W; ++i) op[i] = static_cast<T>(o[i] / l);
}

}  // namespace

kvq_status launch_attend_prompt(const PromptArgs& p, cudaStream_t st, const LaunchCtx&) {
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(p.n_rows) * p.q_heads + 7) / 8);
  if (p.bf16) {
    if (p.head_dim == 128) k_prompt_rows<__nv_bfloat16, 128><<<grid, 256, 0, st>>>(p);
    else k_prompt_rows<__nv_bfloat16, 64><<<grid, 256, 0, st>>>(p);
  } else {
    if (p.head_dim == 128) k_prompt_rows<__half, 128><<<grid, 256, 0, st>>>(p);
    else k_prompt_rows<__half, 64><<<grid, 256, 0, st>>>(p);
  }
  return launch_status();
}

}  // namespace kvq
