// kca_norm_rope.cu -- attn_norm_rope_append: everything between the q / k / v
// projections and the attention calls in one pass over the rows.
//
// For every token, with x a row of 256 (8 query rows, 1 key row, 1 value row):
//   norm      y = x / sqrt(mean(x^2) + eps) * (w + w0)      (q, k; v without w)
//   rotation  a_i = pos[axis(i)] * inv_freq[i],  i < 128
//             z[i]       = y[i] cos a_i - y[i + 128] sin a_i
//             z[i + 128] = y[i + 128] cos a_i + y[i] sin a_i
// then q to its own buffer and k, v to the cache rows the caller names.
//
// Bound: memory.  A token is 10 rows in and 10 out (10 KiB with 16-bit types)
// against ~50 operations per element pair, so the pass over HBM decides for
// many tokens, and the launch plus one chain of loads for few.  Hence one
// warp holds HG rows of a token in registers from load to store (all loads
// issued first), and the cosines and sines of a token are computed once per
// warp, not read: a table of 131,072 positions would be 134 MB, and the 1 KiB
// of it that a token needs another tenth of its traffic.
//
// Angles: pos * inv_freq can be 1e5 radians, where f32 has lost the fraction
// of a turn, so the product is taken in f64 in turns (1 / 2 pi folded in), the
// nearest whole turn subtracted there, and only the remainder (at most half a
// turn) goes to f32.  Sums of squares, norms and rotations are f32; the one
// rounding to fewer bits is the store.
//
// Rows per warp: 10 warps a token (one row each) while that fills no more
// than the GPU's warps, else 2 (five rows each), which share the angles.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/kca.h"
#include "kca_common.cuh"
#include "kca_plan.h"

namespace kca {
namespace {

constexpr int kTokenRows = kHeads + 2;      // q heads, k, v
constexpr int kHalf = kDim / 2;
constexpr int kNormWarps = 8;               // warps per block

struct NormRopeArgs {
  const void* q;            // token t at q + t * q_stride elements, its 8 heads contiguous
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;
  const void* wq;           // [256] of w_dtype, or null (1)
  const void* wk;
  const int64_t* pos;       // [n_axes][n_rows], or null (no rotation)
  const float* inv_freq;    // [128]
  void* q_out;              // [n_rows][8][256]
  void* k_cache;
  void* v_cache;
  const int64_t* dst;       // device destinations, or null: dst0 + token
  int64_t dst0, cache_rows;
  DeviceStatus* status;     // may be null
  float w0, eps;
  int32_t n_rows, n_axes, w_dtype, q_dtype, kv_dtype;
  int32_t norm_qk, norm_v;
  uint32_t axis4[kHalf / 4];   // axis of frequency 4 i + j in byte j of word i
};

// Four consecutive elements from a 16-byte (f32) or 8-byte aligned address.
template <int DT>
__device__ __forceinline__ void get4(const void* row, int dim, float* x) {
  if (DT == KCA_F32) {
    const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + dim);
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(row) + dim);
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 f = DT == KCA_F16 ? __half22float2(*reinterpret_cast<const __half2*>(&w[i]))
                                     : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ void get4(int dt, const void* row, int dim, float* x) {
  if (dt == KCA_F32) get4<KCA_F32>(row, dim, x);
  else if (dt == KCA_F16) get4<KCA_F16>(row, dim, x);
  else get4<KCA_BF16>(row, dim, x);
}
__device__ __forceinline__ void put4(int dt, void* row, int dim, const float* x) {
  if (dt == KCA_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(row) + dim) = make_float4(x[0], x[1], x[2], x[3]);
    return;
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (dt == KCA_F16) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *reinterpret_cast<uint2*>(static_cast<unsigned short*>(row) + dim) = make_uint2(w[0], w[1]);
}

// Weight and offset of a lane's eight dims: 1 where there is no weight.
__device__ __forceinline__ void row_weight(const NormRopeArgs& a, const void* w, int d1, int d2, float (&wt)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) wt[j] = 1.f;
    return;
  }
  get4(a.w_dtype, w, d1, wt);
  get4(a.w_dtype, w, d2, wt + 4);
#pragma unroll
  for (int j = 0; j < 8; ++j) wt[j] += a.w0;
}

// Lane l of a warp holds dims 4 l .. 4 l + 3 and 128 + 4 l .. + 3 of each of
// its rows: the two halves of four rotation pairs, and 256- or 512-byte
// contiguous accesses per warp.
template <int IT, int HG>
__global__ void __launch_bounds__(kNormWarps * 32, HG == 1 ? 1 : 4) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kGroups = kTokenRows / HG;
  constexpr int kIn = ElemBytes<IT>::value;
  const int64_t w = (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5);
  const int64_t token = w / kGroups;
  const int first = (int)(w % kGroups) * HG;
  const int lane = threadIdx.x & 31;
  // Programmatic dependent launch: nothing of the caller's is read before the
  // previous kernel of the stream is done.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (token >= a.n_rows) return;
  const int64_t dst = a.dst != nullptr ? a.dst[token] : a.dst0 + token;
  if (dst < 0 || dst >= a.cache_rows) {
    // -1 marks a padding token; any other value outside the cache is an error
    if (dst != -1 && first == 0 && lane == 0) record_error(a.status, kSiteAppend, kErrBadRow, (unsigned)token);
    return;
  }
  const int d1 = 4 * lane, d2 = kHalf + 4 * lane;
  float x[HG][8];
#pragma unroll
  for (int i = 0; i < HG; ++i) {
    const int r = first + i;
    const char* row = r < kHeads    ? static_cast<const char*>(a.q) + (token * a.q_stride + r * kDim) * kIn
                      : r == kHeads ? static_cast<const char*>(a.k) + token * a.k_stride * kIn
                                    : static_cast<const char*>(a.v) + token * a.v_stride * kIn;
    get4<IT>(row, d1, x[i]);
    get4<IT>(row, d2, x[i] + 4);
  }
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  const bool turn = a.pos != nullptr && first <= kHeads;   // a warp with only the value row needs no angle
  if (turn) {
    const float4 f4 = *reinterpret_cast<const float4*>(a.inv_freq + d1);
    const float f[4] = {f4.x, f4.y, f4.z, f4.w};
    int64_t p0 = a.pos[token];
    const uint32_t ax = a.n_axes > 1 ? a.axis4[lane] : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t p = a.n_axes > 1 ? a.pos[(int64_t)((ax >> (8 * i)) & 0xffu) * a.n_rows + token] : p0;
      double t = (double)p * (double)f[i] * 0.15915494309189533577;   // turns
      t -= rint(t);
      sincospif(2.f * (float)t, &s[i], &c[i]);
    }
  }
  // Sums of squares of the warp's rows, then 1 / sqrt(mean + eps).
  float rs[HG];
#pragma unroll
  for (int i = 0; i < HG; ++i) {
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[i][j], x[i][j], ss);
    rs[i] = ss;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < HG; ++i) rs[i] += __shfl_xor_sync(0xffffffffu, rs[i], o);
  float wt[8];   // the warp's query rows share one weight, read once
  if (a.norm_qk && first < kHeads) row_weight(a, a.wq, d1, d2, wt);
#pragma unroll
  for (int i = 0; i < HG; ++i) {
    const int r = first + i;
    if (r < kTokenRows - 1 ? a.norm_qk : a.norm_v) {
      if (r == kHeads) row_weight(a, a.wk, d1, d2, wt);
      const float f = 1.f / sqrtf(rs[i] * (1.f / kDim) + a.eps);
      const bool weighted = r < kTokenRows - 1;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = weighted ? x[i][j] * f * wt[j] : x[i][j] * f;
    }
    if (r <= kHeads && turn) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float lo = x[i][j], hi = x[i][4 + j];
        x[i][j] = lo * c[j] - hi * s[j];
        x[i][4 + j] = hi * c[j] + lo * s[j];
      }
    }
    const int dt = r < kHeads ? a.q_dtype : a.kv_dtype;
    const int esz = dt == KCA_F32 ? 4 : 2;
    char* out = r < kHeads    ? static_cast<char*>(a.q_out) + (token * kHeads + r) * (kDim * esz)
                : r == kHeads ? static_cast<char*>(a.k_cache) + dst * (kDim * esz)
                              : static_cast<char*>(a.v_cache) + dst * (kDim * esz);
    put4(dt, out, d1, x[i]);
    put4(dt, out, d2, x[i] + 4);
  }
}

template <int IT, int HG>
cudaError_t launch_t(const NormRopeArgs& a, cudaStream_t stream) {
  const int64_t warps = (int64_t)a.n_rows * (kTokenRows / HG);
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + kNormWarps - 1) / kNormWarps));
  cfg.blockDim = dim3(kNormWarps * 32);
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<IT, HG>, a);
}

// Tokens up to which every row gets its own warp (10 warps a token).
constexpr int kOneRowTokens = 512;
template <int IT>
cudaError_t launch_in(const NormRopeArgs& a, cudaStream_t stream) {
  return a.n_rows <= kOneRowTokens ? launch_t<IT, 1>(a, stream) : launch_t<IT, 5>(a, stream);
}

bool norm_dtype_ok(int32_t d) { return d == KCA_F32 || d == KCA_F16 || d == KCA_BF16; }
bool norm_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// A row stride: whole 16-byte units, and rows no further apart than 32-bit
// products of rows and strides stay far from overflowing 64 bits.
bool stride_ok(int64_t s, int32_t dt) {
  return s >= 0 && s <= ((int64_t)1 << 32) && (s * (dt == KCA_F32 ? 4 : 2)) % 16 == 0;
}

}  // namespace
}  // namespace kca

extern "C" int attn_norm_rope_append(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                                     const void* v_new, int64_t v_stride, int32_t in_dtype, int32_t n_rows,
                                     int32_t flags, const void* q_weight, const void* k_weight, int32_t w_dtype,
                                     float weight_offset, float eps, const int64_t* positions, int32_t n_axes,
                                     const uint8_t* freq_axis, const float* inv_freq, void* q_out,
                                     int32_t q_out_dtype, void* k_cache, void* v_cache, int32_t kv_dtype,
                                     int64_t cache_rows, const int64_t* dst_rows_dev, int64_t dst_row0,
                                     void* workspace, void* stream) {
  using namespace kca;
  if (!q || !k_new || !v_new || !q_out || !k_cache || !v_cache) return KCA_ERR_NULL;
  if ((positions == nullptr) != (inv_freq == nullptr)) return KCA_ERR_NULL;
  if (!norm_dtype_ok(in_dtype) || !norm_dtype_ok(q_out_dtype) || !norm_dtype_ok(kv_dtype) || !norm_dtype_ok(w_dtype))
    return KCA_ERR_DTYPE;
  if (n_rows < 1 || cache_rows < 1 || (flags & ~(KCA_NORM_QK | KCA_NORM_V)) != 0) return KCA_ERR_RANGE;
  if (dst_rows_dev == nullptr && (dst_row0 < 0 || dst_row0 > cache_rows - n_rows)) return KCA_ERR_RANGE;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(weight_offset)) return KCA_ERR_RANGE;
  if (n_axes < 1 || n_axes > KCA_MAX_ROPE_AXES) return KCA_ERR_RANGE;
  // in place only where every token writes the bytes it alone has read
  if (q_out == q && (q_out_dtype != in_dtype || (n_rows > 1 && q_stride != kHeads * kDim))) return KCA_ERR_RANGE;
  NormRopeArgs a{};
  for (int i = 0; freq_axis != nullptr && i < kHalf; ++i) {
    if (freq_axis[i] >= n_axes) return KCA_ERR_RANGE;
    a.axis4[i / 4] |= static_cast<uint32_t>(freq_axis[i]) << (8 * (i % 4));
  }
  if (!stride_ok(q_stride, in_dtype) || !stride_ok(k_stride, in_dtype) || !stride_ok(v_stride, in_dtype) ||
      !norm_aligned(q) || !norm_aligned(k_new) || !norm_aligned(v_new) || !norm_aligned(q_out) ||
      !norm_aligned(k_cache) || !norm_aligned(v_cache) || !norm_aligned(q_weight) || !norm_aligned(k_weight) ||
      !norm_aligned(inv_freq) || (reinterpret_cast<uintptr_t>(positions) & 7u) != 0 ||
      (reinterpret_cast<uintptr_t>(dst_rows_dev) & 7u) != 0 || (reinterpret_cast<uintptr_t>(workspace) & 3u) != 0)
    return KCA_ERR_ALIGN;
  a.q = q;
  a.k = k_new;
  a.v = v_new;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.wq = q_weight;
  a.wk = k_weight;
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.dst = dst_rows_dev;
  a.dst0 = dst_row0;
  a.cache_rows = cache_rows;
  a.status = static_cast<DeviceStatus*>(workspace);
  a.w0 = weight_offset;
  a.eps = eps;
  a.n_rows = n_rows;
  a.n_axes = n_axes;
  a.w_dtype = w_dtype;
  a.q_dtype = q_out_dtype;
  a.kv_dtype = kv_dtype;
  a.norm_qk = (flags & KCA_NORM_QK) != 0;
  a.norm_v = (flags & KCA_NORM_V) != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = in_dtype == KCA_F32   ? launch_in<KCA_F32>(a, s)
                        : in_dtype == KCA_F16 ? launch_in<KCA_F16>(a, s)
                                              : launch_in<KCA_BF16>(a, s);
  return e == cudaSuccess ? KCA_OK : KCA_ERR_CUDA;
}
