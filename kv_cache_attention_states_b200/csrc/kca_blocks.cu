// kca_blocks.cu -- the two steps before attention over selected key blocks:
// bounds of every finished block of 64 keys (attn_summarize_blocks), and the
// choice of a query's blocks by a cheap score (attn_select_blocks).  The
// attention over the chosen blocks is the decode kernels' own (mode kBlocks
// of kca_decode_mma.cu and kca_rows.cu).
//
// Bounds.  For block j and dim t, hi = max and lo = min of K over the 64 keys;
// a query value q then meets no key value above max(q hi, q lo), and
//   u_j = sum_t max(q_t hi_t, q_t lo_t) >= q . k   for every key k of block j.
// hi and lo are kept as int8 codes under one f32 scale, the query is coded
// the same way, and the sum is taken exactly in integers: the score of a
// block, and with it the list, depends on no order of summation.
#include <atomic>
#include <cuda_runtime.h>

#include "../../include/kca.h"
#include "kca_common.cuh"
#include "kca_plan.h"
#include "kca_rows.h"

namespace kca {
namespace {

constexpr int kBlockKeys = KCA_BLOCK_KEYS;
constexpr int kCodeRow = 2 * kDim;          // codes of a block: 256 of hi, 256 of lo

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// int8 code of x under the scale sx (the quantisation of attn_quantize_k).
__device__ __forceinline__ uint32_t block_code(float x, float sx) {
  if (!(sx > 0.f) || !(sx <= 3.402823466e38f)) return 0u;
  int c = __float2int_rn(__fdiv_rn(x, sx));
  c = c > 127 ? 127 : (c < -127 ? -127 : c);
  return static_cast<uint32_t>(c) & 0xffu;
}

// ---------------------------------------------------------------- summaries
// One CTA per finished block: warp w takes keys 8 w .. 8 w + 7, lane l dims
// 8 l .. 8 l + 7 (eight 16-byte loads in flight per thread for 16-bit keys),
// the warps' bounds meet in shared memory, and thread t quantises dim t.
// Bound: memory (32 KiB of 16-bit keys in, 516 bytes out).
struct SummaryArgs {
  const void* k;
  const int64_t* ctx;
  signed char* codes;
  float* scales;
  DeviceStatus* status;
  int64_t capacity, n_new;
  int32_t n_blocks;        // blocks per sequence of codes / scales
};

template <int KT>
__global__ void __launch_bounds__(256) summarize_kernel(const SummaryArgs a) {
  __shared__ float hi_s[8][kDim], lo_s[8][kDim];
  __shared__ float am_s[8];
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t ctx = a.ctx[b];
  if (ctx < 0 || ctx > a.capacity) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.status, kSiteCtx, kErrBadCtx, (unsigned)b);
    return;
  }
  // finished by the newest positions: ctx - n_new < 64 (j + 1) <= ctx
  const int64_t old = ctx > a.n_new ? ctx - a.n_new : 0;
  const int64_t j = old / kBlockKeys + blockIdx.x;
  if (j >= ctx / kBlockKeys) return;
  const char* rows = static_cast<const char*>(a.k) +
                     (((int64_t)b * a.capacity + j * kBlockKeys + 8 * warp) * kDim + 8 * lane) * ElemBytes<KT>::value;
  float x[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) load8<KT>(rows + (int64_t)i * kDim * ElemBytes<KT>::value, x[i]);
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    float h = x[0][t], l = x[0][t];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      h = max_nan(h, x[i][t]);
      l = min_nan(l, x[i][t]);
    }
    x[0][t] = h;
    x[1][t] = l;
  }
  float4* hd = reinterpret_cast<float4*>(&hi_s[warp][8 * lane]);
  float4* ld = reinterpret_cast<float4*>(&lo_s[warp][8 * lane]);
  hd[0] = make_float4(x[0][0], x[0][1], x[0][2], x[0][3]);
  hd[1] = make_float4(x[0][4], x[0][5], x[0][6], x[0][7]);
  ld[0] = make_float4(x[1][0], x[1][1], x[1][2], x[1][3]);
  ld[1] = make_float4(x[1][4], x[1][5], x[1][6], x[1][7]);
  __syncthreads();
  const int t = threadIdx.x;
  float h = hi_s[0][t], l = lo_s[0][t];
#pragma unroll
  for (int w = 1; w < 8; ++w) {
    h = max_nan(h, hi_s[w][t]);
    l = min_nan(l, lo_s[w][t]);
  }
  float am = max_nan(fabsf(h), fabsf(l));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
  if (lane == 0) am_s[warp] = am;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) am = max_nan(am, am_s[w]);
  const float sx = am * (1.0f / 127.0f);
  const int64_t row = (int64_t)b * a.n_blocks + j;
  a.codes[row * kCodeRow + t] = (signed char)block_code(h, sx);
  a.codes[row * kCodeRow + kDim + t] = (signed char)block_code(l, sx);
  if (t == 0) a.scales[row] = sx;
}

// ---------------------------------------------------------------- selection
// Scores: CTA (i, b) takes blocks 64 i .. 64 i + 63 of sequence b, warp w
// eight of them.  The eight heads' queries are quantised in the CTA (warp h:
// head h) and split into their positive and negative codes; with q+ against
// hi and q- against lo the bound is two int8 products, taken exactly on
// m16n8k32 MMAs (rows 0-7 the heads, columns the eight blocks, 8 + 8 steps of
// 32 dims into one accumulator).  An MMA sums over k in any order, so k is
// permuted on both operands until a thread's share of a code row is whole
// 16-byte pieces, and the codes go from memory to the MMA without passing
// through shared memory.
// Choice: the CTA that draws a sequence's last ticket (nothing waits) holds
// all its scores, eight per thread, as ordered 32-bit keys; a radix search
// over the four bytes finds the smallest key taken, and two counts in index
// order place the blocks.
// Bound: latency (516 bytes a block: 1 MB for 131,072 keys), hence many small
// CTAs and one launch.
constexpr int kSelThreads = 256;
constexpr int kSelBlocks = 64;                       // blocks scored per CTA
constexpr int kSelPer = KCA_MAX_BLOCKS / kSelThreads;  // scores per thread in the choice
static_assert(kSelPer == 8, "two 16-byte loads of scores per thread");

struct SelectArgs {
  const void* q;
  const signed char* codes;
  const float* scales;
  const int64_t* ctx;
  int32_t* out;
  float* scores;           // [batch][KCA_MAX_BLOCKS]
  int32_t* tickets;        // one per sequence, self-resetting
  DeviceStatus* status;
  int64_t blocks_cap, ctx_bound;
  int32_t n_select, n_sink, n_recent;
};

__device__ __forceinline__ void mma_s8_16832(int (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(0u), "r"(a2), "r"(0u), "r"(b0), "r"(b1));
}

// Scores as unsigned keys of the same order: NaN above all numbers.
__device__ __forceinline__ uint32_t order_key(float s) {
  if (s != s) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(s + 0.f);   // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int QT>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a) {
  __shared__ __align__(16) unsigned char qc[kHeads * kDim];   // query codes
  __shared__ float sq_s[kHeads];
  __shared__ int hist[4][256];
  __shared__ int warp_sum[8];
  __shared__ int last;
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) hist[i][threadIdx.x] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int64_t ctx = a.ctx[b];
  if (ctx < 0 || ctx > a.ctx_bound) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.status, kSiteCtx, kErrBadCtx, (unsigned)b);
    ctx = 0;
  }
  const int nb = (int)((ctx + kBlockKeys - 1) / kBlockKeys);
  const int ctas = nb > 0 ? (nb + kSelBlocks - 1) / kSelBlocks : 1;
  if ((int)blockIdx.x >= ctas) return;
  const int k = a.n_select < nb ? a.n_select : nb;
  int32_t* out = a.out + (int64_t)b * a.n_select;
  if (nb <= a.n_select) {   // every block is taken: no score matters
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < a.n_select; i += kSelThreads) out[i] = i < nb ? i : -1;
    return;
  }

  // code rows first: their loads overlap the quantisation of the query
  const int blk = blockIdx.x * kSelBlocks + 8 * warp + g;
  const bool have = blk < nb - 1 && blk < a.blocks_cap;   // the last block is always taken: no summary needed
  const int64_t row = (int64_t)b * a.blocks_cap + blk;
  uint4 hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4* p = reinterpret_cast<const uint4*>(a.codes + row * kCodeRow + 64 * i + 16 * tig);
    hi[i] = have ? p[0] : make_uint4(0u, 0u, 0u, 0u);
    lo[i] = have ? p[kDim / 16] : make_uint4(0u, 0u, 0u, 0u);
  }
  // D columns of this thread: blocks 2 tig and 2 tig + 1 of the warp
  const int c0 = blockIdx.x * kSelBlocks + 8 * warp + 2 * tig;
  float sk[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    sk[i] = c0 + i < nb - 1 && c0 + i < a.blocks_cap ? a.scales[(int64_t)b * a.blocks_cap + c0 + i] : 0.f;
  {
    float x[8];
    load8<QT>(static_cast<const char*>(a.q) + (((int64_t)b * kHeads + warp) * kDim + 8 * lane) * ElemBytes<QT>::value, x);
    float am = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) am = max_nan(am, fabsf(x[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
    const float sx = am * (1.0f / 127.0f);
    if (lane == 0) sq_s[warp] = sx;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = block_code(x[4 * i], sx) | (block_code(x[4 * i + 1], sx) << 8) | (block_code(x[4 * i + 2], sx) << 16) |
             (block_code(x[4 * i + 3], sx) << 24);
    *reinterpret_cast<uint2*>(qc + warp * kDim + 8 * lane) = make_uint2(w[0], w[1]);
  }
  __syncthreads();
  int acc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 qa = *reinterpret_cast<const uint4*>(qc + g * kDim + 64 * i + 16 * tig);
    mma_s8_16832(acc[0], __vmaxs4(qa.x, 0u), __vmaxs4(qa.y, 0u), hi[i].x, hi[i].y);
    mma_s8_16832(acc[1], __vmins4(qa.x, 0u), __vmins4(qa.y, 0u), lo[i].x, lo[i].y);
    mma_s8_16832(acc[0], __vmaxs4(qa.z, 0u), __vmaxs4(qa.w, 0u), hi[i].z, hi[i].w);
    mma_s8_16832(acc[1], __vmins4(qa.z, 0u), __vmins4(qa.w, 0u), lo[i].z, lo[i].w);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {   // head g, block c0 + i; then the best of the 8 heads
    float s = static_cast<float>(acc[0][i] + acc[1][i]) * (sq_s[g] * sk[i]);
    s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, 4));
    s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, 8));
    s = max_nan(s, __shfl_xor_sync(0xffffffffu, s, 16));
    if (g == 0 && c0 + i < nb) a.scores[(int64_t)b * KCA_MAX_BLOCKS + c0 + i] = s;
  }
  // Release: the block's scores, ordered by the barrier before one thread's
  // acq_rel ticket; acquire: the same ticket in the last CTA, then a barrier.
  __syncthreads();
  if (threadIdx.x == 0) {
    int prev;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(prev) : "l"(a.tickets + b) : "memory");
    last = prev == ctas - 1;
    if (last) a.tickets[b] = 0;   // ready for the next call
  }
  __syncthreads();
  if (!last) return;

  uint32_t key[kSelPer];
  {
    const int i0 = threadIdx.x * kSelPer;
    const float4* p = reinterpret_cast<const float4*>(a.scores + (int64_t)b * KCA_MAX_BLOCKS + i0);
    float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0;
    if (i0 < nb) {      // places of the row past nb hold old scores; they are not used
      s0 = __ldcg(p);
      s1 = __ldcg(p + 1);
    }
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int i = 0; i < kSelPer; ++i) {
      const int j = i0 + i;
      key[i] = j >= nb ? 0u : (j < a.n_sink || j >= nb - a.n_recent) ? 0xffffffffu : order_key(s[i]);
    }
  }
  // Radix search, highest byte first: `want` keys are still to be taken among
  // those that share `prefix`; the bin that holds the want-th largest extends
  // the prefix.  Every warp scans the bins itself (lane l: bins 8 l .. 8 l + 7).
  uint32_t prefix = 0;
  int want = k;
#pragma unroll
  for (int pass = 0; pass < 4; ++pass) {
    const int sh = 24 - 8 * pass;
#pragma unroll
    for (int i = 0; i < kSelPer; ++i)
      if (threadIdx.x * kSelPer + i < nb && (pass == 0 || (key[i] >> (sh + 8)) == prefix))
        atomicAdd(&hist[pass][(key[i] >> sh) & 0xffu], 1);
    __syncthreads();
    int h[8], sum = 0;
    const int4 h0 = *reinterpret_cast<const int4*>(&hist[pass][8 * lane]);
    const int4 h1 = *reinterpret_cast<const int4*>(&hist[pass][8 * lane + 4]);
    h[0] = h0.x; h[1] = h0.y; h[2] = h0.z; h[3] = h0.w;
    h[4] = h1.x; h[5] = h1.y; h[6] = h1.z; h[7] = h1.w;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += h[i];
    int above = sum;   // keys in the bins of this lane and of higher lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_down_sync(0xffffffffu, above, o);
      if (lane + o < 32) above += v;
    }
    above -= sum;      // in bins above this lane's
    int bin = -1, rest = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      if (bin < 0 && above < want && above + h[i] >= want) {
        bin = 8 * lane + i;
        rest = want - above;
      }
      above += h[i];
    }
    const unsigned who = __ballot_sync(0xffffffffu, bin >= 0);   // exactly one lane
    const int src = __ffs(who) - 1;
    prefix = (prefix << 8) | (uint32_t)__shfl_sync(0xffffffffu, bin, src);
    want = __shfl_sync(0xffffffffu, rest, src);
  }
  // Taken: every key above `prefix`, and of the keys equal to it the first
  // `want` by index.  Places by a scan in index order of both counts (16 bits
  // each: at most 2,048).
  int cnt = 0;
#pragma unroll
  for (int i = 0; i < kSelPer; ++i) {
    if (threadIdx.x * kSelPer + i >= nb) continue;
    cnt += key[i] > prefix ? 1 : key[i] == prefix ? (1 << 16) : 0;
  }
  int incl = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int before = incl - cnt;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  int gt = before & 0xffff, eq = before >> 16;
#pragma unroll
  for (int i = 0; i < kSelPer; ++i) {
    const int j = threadIdx.x * kSelPer + i;
    if (j >= nb) continue;
    if (key[i] > prefix) {
      out[gt + (eq < want ? eq : want)] = j;
      ++gt;
    } else if (key[i] == prefix) {
      if (eq < want) out[gt + eq] = j;
      ++eq;
    }
  }
}

cudaLaunchConfig_t dependent_launch(dim3 grid, int threads, cudaStream_t s, cudaLaunchAttribute* at) {
  at->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

bool blk_dtype_ok(int32_t d) { return d == KCA_F32 || d == KCA_F16 || d == KCA_BF16; }
bool blk_aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
constexpr size_t kStatusBytes = 256;   // the counters follow the status word in the workspace header

}  // namespace
}  // namespace kca

extern "C" {

int attn_summarize_blocks(const void* k_cache, int32_t kv_dtype, int64_t capacity, int32_t batch,
                          const int64_t* ctx_len_dev, int64_t n_new, int8_t* codes, float* scales, void* workspace,
                          void* stream) {
  using namespace kca;
  if (!k_cache || !ctx_len_dev || !codes || !scales) return KCA_ERR_NULL;
  if (!blk_dtype_ok(kv_dtype)) return KCA_ERR_DTYPE;
  if (capacity < 1 || capacity > KCA_MAX_POSITION || batch < 1 || batch > KCA_MAX_BATCH || n_new < 1 ||
      n_new > capacity)
    return KCA_ERR_RANGE;
  if (!blk_aligned(k_cache, 16) || !blk_aligned(codes, 16) || !blk_aligned(scales, 4) || !blk_aligned(ctx_len_dev, 8) ||
      !blk_aligned(workspace, 4))
    return KCA_ERR_ALIGN;
  SummaryArgs a{k_cache, ctx_len_dev, codes, scales, static_cast<DeviceStatus*>(workspace), capacity, n_new,
                (int32_t)cdiv(capacity, kBlockKeys)};
  cudaLaunchAttribute at;
  // n_new consecutive positions finish at most ceil(n_new / 64) blocks
  const cudaLaunchConfig_t cfg = dependent_launch(dim3((unsigned)cdiv(n_new, kBlockKeys), batch), 256,
                                                  static_cast<cudaStream_t>(stream), &at);
  const cudaError_t e = kv_dtype == KCA_F32   ? cudaLaunchKernelEx(&cfg, summarize_kernel<KCA_F32>, a)
                        : kv_dtype == KCA_F16 ? cudaLaunchKernelEx(&cfg, summarize_kernel<KCA_F16>, a)
                                              : cudaLaunchKernelEx(&cfg, summarize_kernel<KCA_BF16>, a);
  return e == cudaSuccess ? KCA_OK : KCA_ERR_CUDA;
}

size_t attn_select_blocks_workspace_bytes(int32_t batch, int64_t ctx_bound) {
  if (batch < 1 || batch > KCA_MAX_BATCH || ctx_bound < 1 || ctx_bound > KCA_MAX_POSITION) return 0;
  return KCA_WORKSPACE_HEADER + (size_t)batch * KCA_MAX_BLOCKS * sizeof(float);
}

int attn_select_blocks(const void* q, int32_t q_dtype, const int8_t* codes, const float* scales, int64_t blocks_cap,
                       int32_t batch, const int64_t* ctx_len_dev, int64_t ctx_bound, int32_t n_select, int32_t n_sink,
                       int32_t n_recent, int32_t* blocks, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace kca;
  if (!q || !codes || !scales || !ctx_len_dev || !blocks || !workspace) return KCA_ERR_NULL;
  if (!blk_dtype_ok(q_dtype)) return KCA_ERR_DTYPE;
  if (batch < 1 || batch > KCA_MAX_BATCH || ctx_bound < 1 || ctx_bound > KCA_MAX_POSITION) return KCA_ERR_RANGE;
  if (blocks_cap < cdiv(ctx_bound, kBlockKeys) - 1 || blocks_cap < 1 || blocks_cap > KCA_MAX_BLOCKS)
    return KCA_ERR_RANGE;
  if (n_select < 1 || n_select > KCA_MAX_BLOCKS || n_sink < 0 || n_recent < 1 || n_sink > n_select - n_recent)
    return KCA_ERR_RANGE;
  if (!blk_aligned(q, 16) || !blk_aligned(codes, 16) || !blk_aligned(scales, 4) || !blk_aligned(blocks, 4) ||
      !blk_aligned(ctx_len_dev, 8))
    return KCA_ERR_ALIGN;
  if (!blk_aligned(workspace, 256) || workspace_bytes < attn_select_blocks_workspace_bytes(batch, ctx_bound))
    return KCA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  SelectArgs a{q, codes, scales, ctx_len_dev, blocks, reinterpret_cast<float*>(ws + KCA_WORKSPACE_HEADER),
               reinterpret_cast<int32_t*>(ws + kStatusBytes), reinterpret_cast<DeviceStatus*>(ws), blocks_cap, ctx_bound,
               n_select, n_sink, n_recent};
  cudaLaunchAttribute at;
  const cudaLaunchConfig_t cfg =
      dependent_launch(dim3((unsigned)cdiv(cdiv(ctx_bound, kBlockKeys), kSelBlocks), batch), kSelThreads,
                       static_cast<cudaStream_t>(stream), &at);
  const cudaError_t e = q_dtype == KCA_F32   ? cudaLaunchKernelEx(&cfg, select_kernel<KCA_F32>, a)
                        : q_dtype == KCA_F16 ? cudaLaunchKernelEx(&cfg, select_kernel<KCA_F16>, a)
                                             : cudaLaunchKernelEx(&cfg, select_kernel<KCA_BF16>, a);
  return e == cudaSuccess ? KCA_OK : KCA_ERR_CUDA;
}

}  // extern "C"
