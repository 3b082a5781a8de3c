// kca_prefix.cu -- the merge of attn_decode_prefix: the partial softmax states
// of the prefix that the batch shares (written by the tensor-core prefill
// kernel or the multi-row units, one per run of keys) and of each sequence's
// own keys, combined by log-sum-exp,
//   out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i,   M = max_i m_i.
//
// Bound: memory (1 KiB a partial, mostly in L2) and one chain of loads.  One
// CTA per (sequence, head); warp w takes partials w, w + 8, ..., lane l the
// dims 8 l .. 8 l + 7; the warps' sums meet in shared memory.
#include "kca_common.cuh"
#include "kca_plan.h"
#include "kca_rows.h"

namespace kca {
namespace {

constexpr int kPmWarps = 8;
constexpr float kPmLog2e = 1.4426950408889634f;

__global__ void __launch_bounds__(kPmWarps * 32) prefix_merge_kernel(const PrefixMergeArgs a) {
  __shared__ float sm[kPmWarps], sl[kPmWarps];
  __shared__ float sacc[kPmWarps][kDim];
  const int row = blockIdx.x, b = row / kHeads, h = row % kHeads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t base = (int64_t)(b / a.group) * a.group_step + (b % a.group) * kHeads + h;
  const float* own_ml = a.own + (int64_t)row * 2;
  const float* own_acc = a.own + (int64_t)a.batch * kHeads * 2 + (int64_t)row * kDim;
  // the own keys are one more partial, n_items
  auto m_of = [&](int s) {
    return s < a.n_items ? a.ml[(base + s * a.item_step) * 2] * a.mscale : own_ml[0] * kPmLog2e;
  };
  float M = -INFINITY;
  for (int s = threadIdx.x; s <= a.n_items; s += kPmWarps * 32) M = max_nan(M, m_of(s));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) sm[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPmWarps; ++w) M = max_nan(M, sm[w]);
  const float mu = M == -INFINITY ? 0.f : M;
  float L = 0.f, A[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = warp; s <= a.n_items; s += kPmWarps) {
    const int64_t r = base + s * a.item_step;
    const float f = exp2f(m_of(s) - mu);
    L += f * (s < a.n_items ? a.ml[r * 2 + 1] : own_ml[1]);
    const float4* p = reinterpret_cast<const float4*>((s < a.n_items ? a.acc + r * kDim : own_acc) + 8 * lane);
    const float4 x = p[0], y = p[1];
    A[0] += f * x.x; A[1] += f * x.y; A[2] += f * x.z; A[3] += f * x.w;
    A[4] += f * y.x; A[5] += f * y.y; A[6] += f * y.z; A[7] += f * y.w;
  }
  if (lane == 0) sl[warp] = L;
#pragma unroll
  for (int i = 0; i < 8; ++i) sacc[warp][8 * lane + i] = A[i];
  __syncthreads();
  const int d = threadIdx.x;
  float l = 0.f, x = 0.f;
#pragma unroll
  for (int w = 0; w < kPmWarps; ++w) {
    l += sl[w];
    x += sacc[w][d];
  }
  x = M == -INFINITY && l == 0.f ? 0.f : x / l;   // no key at all: zeros
  if (a.ctx_dev != nullptr) {
    const int64_t c = a.ctx_dev[b];
    if (c < a.ctx_min || c > a.ctx_bound) {
      if (h == 0 && d == 0) record_error(a.status, kSiteCtx, kErrBadCtx, (unsigned)b);
      x = 0.f;
    }
  }
  const int64_t o = (int64_t)row * kDim + d;
  if (a.out_dtype == KCA_F16) static_cast<__half*>(a.out)[o] = __float2half_rn(x);
  else if (a.out_dtype == KCA_BF16) static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(x);
  else static_cast<float*>(a.out)[o] = x;
}
static_assert(kPmWarps * 32 == kDim, "thread d writes dim d");

}  // namespace

cudaError_t launch_prefix_merge(const PrefixMergeArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.batch * kHeads);
  cfg.blockDim = dim3(kPmWarps * 32);
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_merge_kernel, a);
}

}  // namespace kca
