// norm.cu -- RMSNorm with the residual's addition and an E4M3 output in blocks:
//   s = x (+ r),  y = s / sqrt(mean(s^2) + eps) * w,
//   per block of 64 or 128 values of y: scale = max(amax, 1e-4) * fp32(1/448),
//   codes = E4M3 round-to-nearest-even of clamp(y / scale, -448, 448)
// ("DeepSeek-V4 全面解读" §2.5 RMSNorm, §3.4 act_quant_kernel).  s is kept in
// fp32 for the norm; the residual stream's new value is s rounded to BF16.
//
// One pass: a row stays in registers between its sum of squares and its codes.
// kTpr threads share a row (16 lanes for an indexer head of 128 values, up to
// 512 threads for 16384), each holding kUnits 16-byte units, unit i of a thread
// being unit i kTpr + (its index) of the row, so loads and stores are coalesced
// and a block's 8 or 16 units are neighbouring lanes of one warp: its absmax is
// three or four shuffles.  The grid is resident and walks the rows; the weights
// of a thread's columns are loaded once.  To keep reads in flight a long row's
// successor is loaded before the row is reduced, and short rows go several at a
// time (a row of 128 is one 16-byte load a thread).
#include <atomic>

#include "common.cuh"
#include "dsv4sa_internal.h"

namespace dsv4sa {
namespace {

constexpr float kFp8MaxInv = 1.0f / 448.0f;
constexpr float kAmaxFloor = 1e-4f;

struct NormParams {
  const uint4* x;
  const uint4* r;          // null: no residual
  const float4* w;
  uint4* sum;              // null: not stored
  uint4* y;                // null: not stored
  uint2* codes;            // null: not stored
  float* scale;
  int64_t x_stride;        // in units of 8 values
  int64_t r_stride;
  int32_t n;
  int32_t units;           // dim / 8
  int32_t group_units;     // group / 8: 8 or 16
  float inv_dim;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kTpr, int kUnits, int kRowsAtOnce, bool kRes>
__global__ void __launch_bounds__(kTpr > 256 ? kTpr : 256) rmsnorm_quant_kernel(const NormParams p) {
  constexpr int kThreads = kTpr > 256 ? kTpr : 256;
  constexpr int kRowsPerCta = kThreads / kTpr;
  constexpr int kWarps = kTpr > 32 ? kTpr / 32 : 1;         // warps that share a row
  __shared__ float part[2][kRowsPerCta][kWarps];
  griddep_launch();
  griddep_wait();
  const int tid = static_cast<int>(threadIdx.x);
  const int c = tid % kTpr, sub = tid / kTpr;               // place in the row, row of the CTA
  float w[kUnits][8];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = i * kTpr + c;
    const float4 a = u < p.units ? __ldg(p.w + 2 * u) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 b = u < p.units ? __ldg(p.w + 2 * u + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
    w[i][0] = a.x, w[i][1] = a.y, w[i][2] = a.z, w[i][3] = a.w;
    w[i][4] = b.x, w[i][5] = b.y, w[i][6] = b.z, w[i][7] = b.w;
  }
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRowsPerCta;
  auto load = [&](int64_t row, uint4 (&xv)[kUnits], uint4 (&rv)[kUnits]) {
    const bool live = row < p.n;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = i * kTpr + c;
      const bool in = live && u < p.units;
      xv[i] = in ? __ldcs(p.x + row * p.x_stride + u) : zero;
      if constexpr (kRes) rv[i] = in ? __ldcs(p.r + row * p.r_stride + u) : zero;
    }
  };
  int buf = 0;
  // one row, from the units in xv and rv; `next` loads the row after it in between
  auto process = [&](int64_t row, uint4 (&xv)[kUnits], uint4 (&rv)[kUnits], int64_t next) {
    const bool live = row < p.n;
    float s[kUnits][8];
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      float r[8];
      unpack8(xv[i], s[i]);
      if constexpr (kRes) unpack8(rv[i], r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (kRes) s[i][j] += r[j];
        sq = fmaf(s[i][j], s[i][j], sq);
      }
    }
    if constexpr (kRowsAtOnce == 1) load(next, xv, rv);   // in flight while this row is reduced
#pragma unroll
    for (int o = (kTpr < 32 ? kTpr : 32) / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if constexpr (kWarps > 1) {
      if ((tid & 31) == 0) part[buf][sub][c >> 5] = sq;
      __syncthreads();
      sq = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) sq += part[buf][sub][i];
      buf ^= 1;            // the other copy: no thread writes it before every thread passed this barrier
    }
    const float rstd = __frsqrt_rn(fmaf(sq, p.inv_dim, p.eps));
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = i * kTpr + c;
      const bool in = live && u < p.units;
      if (in && p.sum) __stcs(p.sum + row * p.units + u, pack8(s[i]));
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[i][j] = s[i][j] * rstd * w[i][j];
        amax = fmaxf(amax, fabsf(s[i][j]));
      }
      if (in && p.y) __stcs(p.y + row * p.units + u, pack8(s[i]));
      if (p.codes) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
        if (p.group_units == 16) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
        const float scale = __fmul_rn(fmaxf(amax, kAmaxFloor), kFp8MaxInv);
        // y itself carries fp32 roundings, so a multiply by the rounded
        // reciprocal instead of a division moves a code only where y is already
        // within them of a tie; the conversion saturates at +-448
        const float inv = __frcp_rn(scale);
        uint32_t q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(s[i][4 * h] * inv, s[i][4 * h + 1] * inv),
                                                       __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(s[i][4 * h + 2] * inv, s[i][4 * h + 3] * inv),
                                                       __NV_SATFINITE, __NV_E4M3);
          q[h] = lo | (hi << 16);
        }
        if (in) {
          __stcs(p.codes + row * p.units + u, make_uint2(q[0], q[1]));
          if ((u & (p.group_units - 1)) == 0) p.scale[row * (p.units / p.group_units) + u / p.group_units] = scale;
        }
      }
    }
  };
  // the first row of the CTA decides: every thread takes part in shuffles and barriers
  int64_t first = static_cast<int64_t>(blockIdx.x) * kRowsPerCta;
  uint4 xv[kRowsAtOnce][kUnits], rv[kRowsAtOnce][kUnits];
  if constexpr (kRowsAtOnce == 1) {
    load(first + sub, xv[0], rv[0]);
    for (; first < p.n; first += step) process(first + sub, xv[0], rv[0], first + sub + step);
  } else {
    for (; first < p.n; first += kRowsAtOnce * step) {
#pragma unroll
      for (int k = 0; k < kRowsAtOnce; ++k) load(first + sub + k * step, xv[k], rv[k]);
#pragma unroll
      for (int k = 0; k < kRowsAtOnce; ++k) process(first + sub + k * step, xv[k], rv[k], 0);
    }
  }
}

template <int kTpr, int kUnits, int kRowsAtOnce, bool kRes>
int launch_norm_r(const NormParams& p, cudaStream_t stream) {
  constexpr int kThreads = kTpr > 256 ? kTpr : 256;
  constexpr int kRowsPerCta = kThreads / kTpr;
  static std::atomic<int> cached{0};   // CTAs per SM, a property of the kernel: queried once
  int dev = 0, sms = 0, resident = cached.load(std::memory_order_relaxed);
  if (cudaGetDevice(&dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  if (resident == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(
            &resident, rmsnorm_quant_kernel<kTpr, kUnits, kRowsAtOnce, kRes>, kThreads, 0) != cudaSuccess)
      return DSV4SA_ERR_CUDA;
    if (resident < 1) resident = 1;
    cached.store(resident, std::memory_order_relaxed);
  }
  // A CTA for each kRowsPerCta rows while there are few; a resident grid that keeps
  // the weights in registers for long rows; for short ones (whose weights are a few
  // cached lines) CTAs of a few batches each, which even out better
  const int64_t want = (static_cast<int64_t>(p.n) + kRowsPerCta - 1) / kRowsPerCta;
  const int64_t full = static_cast<int64_t>(sms) * resident * (kRowsAtOnce > 1 ? 4 : 1);
  return launch_pdl(rmsnorm_quant_kernel<kTpr, kUnits, kRowsAtOnce, kRes>,
                    dim3(static_cast<unsigned>(want < full ? want : full)), dim3(kThreads), 0, stream, p) == cudaSuccess
             ? DSV4SA_OK
             : DSV4SA_ERR_CUDA;
}

template <int kTpr, int kUnits, int kRowsAtOnce>
int launch_norm(const NormParams& p, cudaStream_t stream) {
  return p.r ? launch_norm_r<kTpr, kUnits, kRowsAtOnce, true>(p, stream)
             : launch_norm_r<kTpr, kUnits, kRowsAtOnce, false>(p, stream);
}

}  // namespace

int launch_rmsnorm_quant(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                         const float* norm_w, float eps, int32_t n, int32_t dim, int32_t group, void* residual_out,
                         void* y, uint8_t* codes, float* scale, cudaStream_t stream) {
  NormParams p{};
  p.x = static_cast<const uint4*>(x);
  p.r = static_cast<const uint4*>(residual);
  p.w = reinterpret_cast<const float4*>(norm_w);
  p.sum = static_cast<uint4*>(residual_out);
  p.y = static_cast<uint4*>(y);
  p.codes = reinterpret_cast<uint2*>(codes);
  p.scale = scale;
  p.x_stride = x_stride / 8;
  p.r_stride = residual_stride / 8;
  p.n = n;
  p.units = dim / 8;
  p.group_units = group / 8;
  p.inv_dim = 1.0f / static_cast<float>(dim);
  p.eps = eps;
  // the fewest threads whose registers hold the row in at most four units each
  if (dim <= 128) return launch_norm<16, 1, 4>(p, stream);
  if (dim <= 256) return launch_norm<32, 1, 4>(p, stream);
  if (dim <= 512) return launch_norm<32, 2, 2>(p, stream);
  if (dim <= 1024) return launch_norm<32, 4, 1>(p, stream);
  if (dim <= 2048) return launch_norm<128, 2, 1>(p, stream);
  if (dim <= 4096) return launch_norm<128, 4, 1>(p, stream);
  if (dim <= 8192) return launch_norm<256, 4, 1>(p, stream);
  return launch_norm<512, 4, 1>(p, stream);
}

}  // namespace dsv4sa
