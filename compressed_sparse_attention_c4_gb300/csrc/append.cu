// append.cu -- new rows of the KV projection into a paged pool in one pass: RMSNorm, the
// rotation of the last 64 dims at the row's position, quantisation, and the slot.
//   y = x / sqrt(mean(x^2) + eps) * w;   (a, b) -> (a c - b s, b c + a s) for y's last 32 pairs
// ("DeepSeek-V4 全面解读" §2.11 step 2: kv_norm, RoPE, act_quant of the nope part; §2.6; the
// formats of writer.cu.)  y stays in fp32 until it is a code or a BF16 rope value: one
// rounding instead of the three of separate calls.  Without the norm the codes and scales are
// those of the cache writer, bit for bit.
//
// A warp takes a row at a time, lane c holding the 16-byte units c and 32 + c (8 values each): loads
// and stores are contiguous, a 64-value block is eight neighbouring lanes (a 32-value FP4 block
// four), and the rotated units 56-63 are the second ones of lanes 24-31, whole pairs in a lane.
// Norm weights and the row's table entries come from L1 and L2.
#include "common.cuh"
#include "dsv4sa_internal.h"
#include "fp4.cuh"

namespace dsv4sa {
namespace {

constexpr int kThreads = 256;
constexpr float kFp8MaxInv = 1.0f / 448.0f;   // rounded to fp32
constexpr float kAmaxFloor = 1e-4f;
constexpr float kFp4MaxInv = 1.0f / 6.0f;
constexpr float kFp4AmaxFloor = 6.0f * 1.1754943508222875e-38f;   // 6 * 2^-126 (exact)

struct AppendParams {
  const uint4* rows;
  int64_t row_stride;      // in units
  const int32_t* page_table;
  const int32_t* row_seq;
  const int32_t* row_pos;
  const int32_t* row_entry;   // null: from the position
  const int32_t* src_row;     // null: row r is row r of `rows`
  const float4* cs;           // [rope_rows][16], null: not rotated
  const float4* w;            // null: no weights
  uint8_t* base;
  int64_t page_stride, num_pages;
  int32_t pt_stride;
  int32_t pt_rows;            // INT32_MAX where the caller did not say
  int32_t ring;
  int32_t n, n_src;
  int32_t rope_rows;
  int32_t per;                // rows of a warp's batch
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4 v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

// The largest magnitude of eight values, as fp32 bits (NaN above everything).
__device__ __forceinline__ uint32_t top_of(const float2 (&y)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = max(m, max(__float_as_uint(y[i].x) & 0x7FFFFFFFu, __float_as_uint(y[i].y) & 0x7FFFFFFFu));
  return m;
}

// E4M3 codes of y / scale, the quotient rounded to fp32 as a division would round it: the
// product with the rounded reciprocal, corrected by its residual (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).  Where an infinity or a
// NaN is in the block the division itself.
__device__ __forceinline__ uint2 e4m3x8(const float2 (&y)[4], float scale, bool finite) {
  const float rc = __frcp_rn(scale);
  const float2 r2 = make_float2(rc, rc), s2 = make_float2(-scale, -scale);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = mul2(y[i], r2);
    float2 z = fma2(fma2(q, s2, y[i]), r2, q);
    z.x = copysignf(z.x, y[i].x), z.y = copysignf(z.y, y[i].y);   // of a zero
    if (!finite) {
      z.x = fminf(fmaxf(__fdiv_rn(y[i].x, scale), -448.f), 448.f);
      z.y = fminf(fmaxf(__fdiv_rn(y[i].y, scale), -448.f), 448.f);
    }
    c[i] = __nv_cvt_float2_to_fp8x2(z, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// A warp takes `per` consecutive rows.  Lane l looks up row l's slot -- one chain of dependent
// loads for all of them -- and the rows themselves come through shared memory, kStages of them
// on the way at a time: each lane copies, and later reads, its own 16-byte units, so nothing
// has to be waited for but the copy.  65529 FP8 rows with the norm 33.3 us (18.3 at the copy
// bandwidth, 15.8 without the table rows that sequences share), 57.6 with a row a warp and loads
// one after the other; 32749 FP4 rows without it 10.3 (8.0), 17.6 so; 32 rows 2.6.  By the counters
// (caches cold: 36.8 us) the FP8 kernel issues in 56 % of its slots and has 18 warps a
// multiprocessor on average: 80 registers let three CTAs in, and the batches below are sized
// for four, so the last quarter of them runs with most of the GPU idle.  FP4: 59 % and 25.
constexpr int kStages = 4;
constexpr int kMaxRows = 16;             // of a warp's batch
constexpr int kStageBytes = 1024 + 256;  // the row, and its rotation

__device__ __forceinline__ void copy16(uint8_t* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <bool kFp4, bool kNorm>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const AppendParams p) {
  // default page layouts (see dsv4sa.h)
  constexpr int kNopeRow = kFp4 ? 224 : 448, kRopeOff = 64 * kNopeRow, kScaleOff = kRopeOff + 64 * 128;
  __shared__ __align__(16) uint8_t ring[kThreads / 32][kStages][kStageBytes];
  griddep_launch();
  griddep_wait();
  const int c = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  const bool rope_lane = c >= 24;
  float4 w[4];
  if constexpr (kNorm) {
    const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = p.w ? __ldg(p.w + (i >> 1) * 64 + 2 * c + (i & 1)) : one;
  }
  for (int64_t r0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp) * p.per; r0 < p.n;
       r0 += static_cast<int64_t>(gridDim.x) * (kThreads / 32) * p.per) {   // warp-uniform
    const int rows = static_cast<int>(min(static_cast<int64_t>(p.per), p.n - r0));
    // ---- row r0 + lane: its source, position, page (-1: not written) and slot
    int l_src = 0, l_pos = 0, l_page = -1, l_slot = 0;
    if (c < rows) {
      const int64_t r = r0 + c;
      const int seq = __ldg(p.row_seq + r);
      l_pos = p.row_pos ? __ldg(p.row_pos + r) : 0;
      l_src = p.src_row ? __ldg(p.src_row + r) : static_cast<int>(r);
      const int e = p.row_entry ? __ldg(p.row_entry + r) : (p.ring > 0 && l_pos >= 0 ? l_pos % p.ring : l_pos);
      const bool ok = l_src >= 0 && l_src < p.n_src && seq >= 0 && seq < p.pt_rows && e >= 0 && (e >> 6) < p.pt_stride &&
                      (!p.cs || (l_pos >= 0 && l_pos < p.rope_rows));
      if (ok) l_page = __ldg(p.page_table + static_cast<int64_t>(seq) * p.pt_stride + (e >> 6));
      if (l_page < 0 || l_page >= p.num_pages) {
        l_page = -1;
        if (seq != -1) raise_error(kErrIndex);             // -1: padding of the batch
      }
      l_slot = e & 63;
    }
    auto fetch = [&](int i) {            // row r0 + i; an empty group past the last one
      const int src = __shfl_sync(0xffffffffu, l_src, i & 31), pos = __shfl_sync(0xffffffffu, l_pos, i & 31);
      const int page = __shfl_sync(0xffffffffu, l_page, i & 31);
      if (i < rows && page >= 0) {
        uint8_t* at = ring[warp][i % kStages];
        const uint4* from = p.rows + src * p.row_stride + c;
        copy16(at + c * 16, from);
        copy16(at + 512 + c * 16, from + 32);
        if (p.cs && rope_lane) {
          const float4* cs = p.cs + static_cast<int64_t>(pos) * 16 + 2 * (c - 24);
          copy16(at + 1024 + (c - 24) * 32, cs);
          copy16(at + 1040 + (c - 24) * 32, cs + 1);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) fetch(i);
#pragma unroll 1
    for (int i = 0; i < rows; ++i) {
      fetch(i + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      const int page = __shfl_sync(0xffffffffu, l_page, i), slot = __shfl_sync(0xffffffffu, l_slot, i);
      if (page < 0) continue;            // the same in the whole warp
      const uint8_t* at = ring[warp][i % kStages];
      const uint4 v0 = *reinterpret_cast<const uint4*>(at + c * 16), v1 = *reinterpret_cast<const uint4*>(at + 512 + c * 16);
      float2 y0[4], y1[4];
      unpack8(v0, y0);
      unpack8(v1, y1);
      if constexpr (kNorm) {
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = fma2(y1[i], y1[i], fma2(y0[i], y0[i], s2));
        float sq = s2.x + s2.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        const float rstd = rsqrtf(fmaf(sq, 1.0f / 512.0f, p.eps));
        const float2 rstd2 = make_float2(rstd, rstd);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y0[i] = mul2(y0[i], rstd2);
          y1[i] = mul2(y1[i], rstd2);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {      // weights of 1 where there are none
          y0[2 * i] = mul2(y0[2 * i], make_float2(w[i].x, w[i].y)), y0[2 * i + 1] = mul2(y0[2 * i + 1], make_float2(w[i].z, w[i].w));
          y1[2 * i] = mul2(y1[2 * i], make_float2(w[2 + i].x, w[2 + i].y)), y1[2 * i + 1] = mul2(y1[2 * i + 1], make_float2(w[2 + i].z, w[2 + i].w));
        }
      }
      uint32_t m0 = top_of(y0), m1 = top_of(y1);               // m1 of lanes 24-31 is not used
      m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, 1)), m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, 1));
      m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, 2)), m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, 2));
      if constexpr (!kFp4) m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, 4)), m1 = max(m1, __shfl_xor_sync(0xffffffffu, m1, 4));
      uint8_t* pg = p.base + static_cast<int64_t>(page) * p.page_stride;
      uint8_t* nope = pg + slot * kNopeRow;
      if constexpr (kFp4) {
        uint8_t* sc = pg + kScaleOff + slot * 16;
        auto put = [&](const float2 (&y)[4], uint32_t mag, int u) {
          const bool finite = mag < 0x7F800000u;
          // e = ceil(log2(fp32(max(amax, 6 * 2^-126) * fp32(1/6)))), off the fields of that product (a normal number)
          const uint32_t t = __float_as_uint(__fmul_rn(fmaxf(finite ? __uint_as_float(mag) : 0.f, kFp4AmaxFloor), kFp4MaxInv));
          const uint32_t b = (t >> 23) + ((t & 0x7FFFFFu) != 0u ? 1u : 0u);   // the E8M0 byte
          const float inv = __uint_as_float((254u - b) << 23);
          float2 z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = mul2(y[i], make_float2(inv, inv));
          reinterpret_cast<uint32_t*>(nope)[u] = finite ? e2m1x8(z) : 0u;
          if ((c & 3) == 0) sc[u >> 2] = static_cast<uint8_t>(finite ? b : 255u);
        };
        put(y0, m0, c);
        if (!rope_lane) put(y1, m1, 32 + c);
      } else {
        float* sc = reinterpret_cast<float*>(pg + kScaleOff + slot * 32);
        auto put = [&](const float2 (&y)[4], uint32_t mag, int u) {
          const float scale = __fmul_rn(fmaxf(__uint_as_float(mag), kAmaxFloor), kFp8MaxInv);
          reinterpret_cast<uint2*>(nope)[u] = e4m3x8(y, scale, mag < 0x7F800000u);
          if ((c & 7) == 0) sc[u >> 3] = scale;
        };
        put(y0, m0, c);
        if (!rope_lane) put(y1, m1, 32 + c);
      }
      if (rope_lane) {
        float4 z0, z1;
        if (p.cs) {
          z0 = *reinterpret_cast<const float4*>(at + 1024 + (c - 24) * 32);
          z1 = *reinterpret_cast<const float4*>(at + 1040 + (c - 24) * 32);
        }
        const float2 cs[4] = {{z0.x, z0.y}, {z0.z, z0.w}, {z1.x, z1.y}, {z1.z, z1.w}};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = y1[i];
          if (p.cs) y1[i] = make_float2(fmaf(y.x, cs[i].x, -(y.y * cs[i].y)), fmaf(y.y, cs[i].x, y.x * cs[i].y));
          const __nv_bfloat162 v = __floats2bfloat162_rn(y1[i].x, y1[i].y);
          o[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        // neither normed nor rotated: the input's bits
        reinterpret_cast<uint4*>(pg + kRopeOff + slot * 128)[c - 24] = kNorm || p.cs ? make_uint4(o[0], o[1], o[2], o[3]) : v1;
      }
    }
  }
}

template <bool kFp4, bool kNorm>
cudaError_t launch_append(AppendParams& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorUnknown;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return cudaErrorUnknown;
  // batches for four CTAs a multiprocessor (what the 64 registers without the norm allow; with it
  // three fit at a time), as far as there are rows
  constexpr int64_t kWarps = kThreads / 32;
  const int64_t n = p.n, want = (n + sms * 4 * kWarps - 1) / (sms * 4 * kWarps);
  p.per = static_cast<int32_t>(want < 1 ? 1 : (want > kMaxRows ? kMaxRows : want));
  const int64_t blocks = (n + p.per * kWarps - 1) / (p.per * kWarps), cap = static_cast<int64_t>(sms) * 16;
  return launch_pdl(cache_append_kernel<kFp4, kNorm>, dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(kThreads), 0,
                    stream, p);
}

}  // namespace

int launch_cache_append(const dsv4sa_append_args* a, cudaStream_t stream) {
  AppendParams p{};
  p.rows = static_cast<const uint4*>(a->rows);
  p.row_stride = a->row_stride / 8;
  p.page_table = a->page_table;
  p.row_seq = a->row_seq;
  p.row_pos = a->row_pos;
  p.row_entry = a->row_entry;
  p.src_row = a->src_row;
  p.cs = reinterpret_cast<const float4*>(a->rope_cs);
  p.w = a->norm ? reinterpret_cast<const float4*>(a->norm_w) : nullptr;
  p.base = static_cast<uint8_t*>(a->pool->base);
  p.page_stride = a->pool->page_stride;
  p.num_pages = a->pool->num_pages;
  p.pt_stride = a->pt_stride;
  p.pt_rows = a->pt_rows > 0 ? a->pt_rows : INT32_MAX;
  p.ring = a->ring;
  p.n = a->n;
  p.n_src = a->n_src;
  p.rope_rows = a->rope_rows;
  p.eps = a->eps;
  const bool fp4 = a->pool->kind == DSV4SA_POOL_KV_FP4, norm = a->norm != 0;
  const cudaError_t e = fp4 ? (norm ? launch_append<true, true>(p, stream) : launch_append<true, false>(p, stream))
                            : (norm ? launch_append<false, true>(p, stream) : launch_append<false, false>(p, stream));
  return e == cudaSuccess ? DSV4SA_OK : DSV4SA_ERR_CUDA;
}

uint32_t* error_word_append() { return error_word(); }

}  // namespace dsv4sa
