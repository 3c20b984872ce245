// norm.cu -- RMSNorm with the residual's addition and an E4M3 output in blocks:
//   s = x (+ r),  y = s / sqrt(mean(s^2) + eps) * w,
//   per block of 64 or 128 values of y: scale = max(amax, 1e-4) * fp32(1/448),
//   codes = E4M3 round-to-nearest-even of clamp(y / scale, -448, 448)
// ("DeepSeek-V4 全面解读" §2.5 RMSNorm, §3.4 act_quant_kernel).  s is kept in
// fp32 for the norm; the residual stream's new value is s rounded to BF16.
//
// One pass: a row stays in registers between its sum of squares and its codes.
// kTpr threads share a row (8 lanes for an indexer head of 128 values, up to
// 512 threads for 16384), each holding kUnits 16-byte units, unit i of a thread
// being unit i kTpr + (its index) of the row, so loads and stores are coalesced
// and a block's 8 or 16 units are neighbouring lanes of one warp: its absmax is
// three or four shuffles.  A CTA walks several rows; the weights
// of a thread's columns are loaded once, and the next row's units before the
// current row is reduced, so reads stay in flight.  Rows of up to 512 are bound by
// their instructions as much as by HBM: two units a thread instead of one halve the
// shuffles and addresses a value, packed fp32 the arithmetic, and 64 registers leave
// 32 warps a multiprocessor (262144 rows of 128: 41 us before these, 20.4 with them, 18.3
// with 32-bit rows and the hardware's reciprocals, 17.8 with rare means apart, 15.2 at the
// measured copy bandwidth; several rows a thread at once took 23 to 31).  With a residual these
// kernels spill 16 bytes.  Long rows are bound by HBM: 8191 rows of 7168 with residual, sum and
// BF16 output 80.5 us, 78.3 at the copy's bandwidth.
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

// 1 / x and 1 / sqrt(x) by the hardware (relative 2^-22 or so; x normal).
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / sqrt(sq inv_dim + eps) where that mean is below 2^-100, infinite or NaN.  The estimate
// takes a mean below the smallest normal number for zero, so it is formed 2^64 times as large.
constexpr uint32_t kLowMean = 0x0D800000u;   // 2^-100
__device__ __forceinline__ float rsqrt_of_rare_mean(float sq, float inv_dim, float eps) {
  const bool low = fmaf(sq, inv_dim, eps) < 0x1p-100f;
  const float up = low ? 0x1p64f : 1.f, down = low ? 0x1p32f : 1.f;
  const float ms = fmaf(sq * up, inv_dim, eps * up), r0 = rsqrt_approx(ms);
  return ms > 0.f && ms < INFINITY ? r0 * fmaf(-0.5f * ms * r0, r0, 1.5f) * down : r0;
}

__device__ __forceinline__ void unpack8(const uint4 v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[i].x, f[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kTpr, int kUnits, bool kRes>
__global__ void __launch_bounds__(kTpr > 256 ? kTpr : 256, kTpr <= 32 && kUnits <= 2 ? 4 : (kTpr <= 256 ? 2 : 1)) rmsnorm_quant_kernel(const NormParams p) {
  constexpr int kThreads = kTpr > 256 ? kTpr : 256;
  constexpr int kRowsPerCta = kThreads / kTpr;
  constexpr int kWarps = kTpr > 32 ? kTpr / 32 : 1;         // warps that share a row
  __shared__ float part[2][kRowsPerCta][kWarps];
  griddep_launch();
  griddep_wait();
  const int tid = static_cast<int>(threadIdx.x);
  const int c = tid % kTpr, sub = tid / kTpr;               // place in the row, row of the CTA
  float2 w[kUnits][4];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = i * kTpr + c;
    const float4 a = u < p.units ? __ldg(p.w + 2 * u) : make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 b = u < p.units ? __ldg(p.w + 2 * u + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
    w[i][0] = make_float2(a.x, a.y), w[i][1] = make_float2(a.z, a.w);
    w[i][2] = make_float2(b.x, b.y), w[i][3] = make_float2(b.z, b.w);
  }
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint32_t n = static_cast<uint32_t>(p.n), step = gridDim.x * kRowsPerCta;   // row + step < 2^32
  auto load = [&](uint32_t row, uint4 (&xv)[kUnits], uint4 (&rv)[kUnits]) {
    const bool live = row < n;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = i * kTpr + c;
      const bool in = live && u < p.units;
      xv[i] = in ? __ldcs(p.x + static_cast<int64_t>(row) * p.x_stride + u) : zero;
      if constexpr (kRes) rv[i] = in ? __ldcs(p.r + static_cast<int64_t>(row) * p.r_stride + u) : zero;
    }
  };
  int buf = 0;
  // one row, from the units in xv and rv; `next` loads the row after it in between
  auto process = [&](uint32_t row, uint4 (&xv)[kUnits], uint4 (&rv)[kUnits], uint32_t next) {
    const bool live = row < n;
    float2 s[kUnits][4];
    float2 sq2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      unpack8(xv[i], s[i]);
      if constexpr (kRes) {
        float2 r[4];
        unpack8(rv[i], r);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = make_float2(s[i][j].x + r[j].x, s[i][j].y + r[j].y);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sq2 = fma2(s[i][j], s[i][j], sq2);
    }
    float sq = sq2.x + sq2.y;
    load(next, xv, rv);    // in flight while this row is reduced
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
    // 1 / sqrt by the hardware's estimate and one Newton step (relative 2^-23)
    const float ms = fmaf(sq, p.inv_dim, p.eps);
    const float r0 = rsqrt_approx(ms);
    float rstd = r0 * fmaf(-0.5f * ms * r0, r0, 1.5f);
    if (__float_as_uint(ms) - kLowMean >= 0x7F800000u - kLowMean) rstd = rsqrt_of_rare_mean(sq, p.inv_dim, p.eps);
    const float2 rstd2 = make_float2(rstd, rstd);
    const int64_t out0 = static_cast<int64_t>(row) * p.units + c;                  // this thread's first unit of the outputs
    float top[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const bool in = live && i * kTpr + c < p.units;
      if (in && p.sum) __stcs(p.sum + out0 + i * kTpr, pack8(s[i]));
      top[i] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = mul2(s[i][j], w[i][j]);                    // t = s w; y = t rstd
        top[i] = fmaxf(top[i], fmaxf(fabsf(s[i][j].x), fabsf(s[i][j].y)));
      }
      if (in && p.y) {
        float2 y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = mul2(s[i][j], rstd2);
        __stcs(p.y + out0 + i * kTpr, pack8(y));
      }
    }
    if (!p.codes) return;
    // absmax of a block: its 8 units are neighbouring lanes, its 16 units twice as many,
    // or with eight threads a row the same lanes' next units
    if (kTpr == 8 && p.group_units == 16) {
#pragma unroll
      for (int i = 0; i + 1 < kUnits; i += 2) top[i] = top[i + 1] = fmaxf(top[i], top[i + 1]);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = i * kTpr + c;
      const bool in = live && u < p.units;
      {
        float amax = top[i];                                 // of t
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
        if (kTpr > 8 && p.group_units == 16) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 8));
        const float scale = __fmul_rn(fmaxf(amax * rstd, kAmaxFloor), kFp8MaxInv);
        // y / scale = t (448 / amax(t)), in which the row's factor cancels (unless the
        // block is below the floor): three roundings from the sum to the code, where
        // norm, weight, scale and quotient in turn take five (of 33.6 million codes 4 to 19
        // differ from those of the exact quotient; 6 to 22 so).  The quotient is the
        // hardware's estimate with its residual added; the conversion saturates.
        // (Of amax / 256: above 2^126 the hardware's quotient would be 0.)
        const float r = rcp_approx(amax * 0x1p-8f) * 0x1p-8f, k0 = 448.f * r;
        const float inv = amax * rstd > kAmaxFloor ? fmaf(fmaf(-amax, k0, 448.f), r, k0) : rstd * (448.f / kAmaxFloor);
        const float2 inv2 = make_float2(inv, inv);
        uint32_t q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(mul2(s[i][2 * h], inv2), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(mul2(s[i][2 * h + 1], inv2), __NV_SATFINITE, __NV_E4M3);
          q[h] = lo | (hi << 16);
        }
        if (in) {
          __stcs(p.codes + out0 + i * kTpr, make_uint2(q[0], q[1]));
          if ((u & (p.group_units - 1)) == 0) p.scale[(out0 + i * kTpr) >> (p.group_units == 16 ? 4 : 3)] = scale;
        }
      }
    }
  };
  // the first row of the CTA decides: every thread takes part in shuffles and barriers
  uint32_t first = blockIdx.x * kRowsPerCta;
  uint4 xv[kUnits], rv[kUnits];
  load(first + sub, xv, rv);
  for (; first < n; first += step) process(first + sub, xv, rv, first + sub + step);
}

template <int kTpr, int kUnits, bool kRes>
int launch_norm_r(const NormParams& p, cudaStream_t stream) {
  constexpr int kThreads = kTpr > 256 ? kTpr : 256;
  constexpr int kRowsPerCta = kThreads / kTpr;
  static std::atomic<int> cached{0};   // CTAs per SM, a property of the kernel: queried once
  int dev = 0, sms = 0, resident = cached.load(std::memory_order_relaxed);
  if (cudaGetDevice(&dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  if (resident == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(
            &resident, rmsnorm_quant_kernel<kTpr, kUnits, kRes>, kThreads, 0) != cudaSuccess)
      return DSV4SA_ERR_CUDA;
    if (resident < 1) resident = 1;
    cached.store(resident, std::memory_order_relaxed);
  }
  const int64_t want = (static_cast<int64_t>(p.n) + kRowsPerCta - 1) / kRowsPerCta;
  // long rows: more CTAs than run at once, a few rows each, so that none is left with more
  // to do than the others (8191 rows of 7168: 81.1 us with eight times the resident ones,
  // 84.8 with these alone); short rows keep their weights and the next row's loads longer
  // (262144 rows of 128: 20.4 us with the resident ones, 23.5 with eight times)
  const int64_t full = static_cast<int64_t>(sms) * resident * (kTpr > 32 ? 8 : 1);
  return launch_pdl(rmsnorm_quant_kernel<kTpr, kUnits, kRes>,
                    dim3(static_cast<unsigned>(want < full ? want : full)), dim3(kThreads), 0, stream, p) == cudaSuccess
             ? DSV4SA_OK
             : DSV4SA_ERR_CUDA;
}

template <int kTpr, int kUnits>
int launch_norm(const NormParams& p, cudaStream_t stream) {
  return p.r ? launch_norm_r<kTpr, kUnits, true>(p, stream)
             : launch_norm_r<kTpr, kUnits, false>(p, stream);
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
  if (dim <= 128) return launch_norm<8, 2>(p, stream);
  if (dim <= 256) return launch_norm<16, 2>(p, stream);
  if (dim <= 512) return launch_norm<32, 2>(p, stream);
  if (dim <= 1024) return launch_norm<32, 4>(p, stream);
  if (dim <= 2048) return launch_norm<128, 2>(p, stream);
  if (dim <= 4096) return launch_norm<128, 4>(p, stream);
  if (dim <= 8192) return launch_norm<256, 4>(p, stream);
  return launch_norm<512, 4>(p, stream);
}

}  // namespace dsv4sa
