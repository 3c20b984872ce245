// writer.cu -- the KV-cache writer: new BF16 rows quantised into a paged pool.
//
// For each new row (an entry s of the sequence whose page-table row is
// row_seq[r]): every 64-value block of the quantised part gets
// amax = max(max |x|, 1e-4), scale = amax * fp32(1/448) and E4M3 codes
// RNE(clamp(x / scale, -448, 448)), all in fp32 ("DeepSeek-V4 全面解读" §3.4
// act_quant_kernel); the codes and the fp32 scale go to slot s % 64 of page
// page_table[row_seq[r]][s / 64] ("DeepSeek-V4 in SGLang" 概念5
// DeepSeekV4TokenToKVPool).  KV pool: 448 nope values quantised (7 blocks),
// 64 rope values stored as BF16 unchanged.  Indexer-key pool: 128 values
// quantised (2 blocks).
//
// FP4 indexer-key pool ("DeepSeek-V4 全面解读" §3.5 fp4_quant_kernel and §3.3
// fast_round_scale; "tilelang量化内核拆解…" 32-group E8M0 scales): every
// 32-value block gets e = ceil(log2(fp32(max(amax, 6 * 2^-126) * fp32(1/6)))),
// read off the fp32 exponent and mantissa fields, and E2M1 codes
// RNE(clamp(x * 2^-e, -6, 6)) -- x * 2^-e is x / 2^e exactly -- packed two per
// byte, value 2j in the low nibble; the scale is stored as the E8M0 byte e + 127.
//
// Each lane owns 16 consecutive values of a row (one 32-byte load), so a
// 64-value block is four neighbouring lanes (a 32-value FP4 block two) and a
// KV row (512 values) is one warp, an indexer key (128 values) a quarter warp.  The block's absmax is a
// max over the bit patterns of |x| (order-preserving for non-negative floats)
// across those four lanes; the 16 codes of a lane are one 16-byte store, so a
// block's 64 codes leave as one contiguous 64-byte piece.
#include "common.cuh"
#include "dsv4sa_internal.h"
#include "fp4.cuh"

namespace dsv4sa {
namespace {

constexpr int kThreads = 256;
constexpr float kFp8MaxInv = 1.0f / 448.0f;   // fp8_max_inv, rounded to fp32
constexpr float kAmaxFloor = 1e-4f;
constexpr float kFp4MaxInv = 1.0f / 6.0f;                     // fp4_max_inv, rounded to fp32
constexpr float kFp4AmaxFloor = 6.0f * 1.1754943508222875e-38f;   // 6 * 2^-126 (exact)

struct WriterParams {
  const int32_t* page_table;
  const int32_t* row_seq;
  const int32_t* row_entry;
  const uint4* rows;        // bf16 [n][row_len], 16-byte aligned
  uint8_t* base;
  int64_t page_stride;
  int64_t num_pages;
  int64_t nope_off;
  int64_t rope_off;
  int64_t scale_off;
  int32_t nope_row;
  int32_t rope_row;
  int32_t scale_row;
  int32_t pt_stride;
  int32_t n;
};

// A resident grid walks the rows grid-stride; a lane's next row (entry,
// sequence and its 32 bytes of values) is loaded while the current one is
// looked up, converted and stored, so the row loads stay in flight.
template <int kLanesPerRow, int kQuantBlocks>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const WriterParams p) {
  constexpr int kRowsPerWarp = 32 / kLanesPerRow;
  constexpr int kRowLen = kLanesPerRow * 16;
  griddep_launch();
  griddep_wait();   // the rows may come from the previous kernel of the stream
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const int sub = lane / kLanesPerRow;           // row of the warp's group
  const int c = lane % kLanesPerRow;             // 16-value chunk of the row
  const bool rope = c >= kQuantBlocks * 4;       // KV rows: values 448..511
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * kRowsPerWarp;
  int64_t r = ((static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5) * kRowsPerWarp + sub;
  if (r - sub >= p.n) return;                    // warp-uniform
  // clamped rows: every lane loads, so the shuffles below see the full warp
  auto load = [&](int64_t row, int& s, int& seq, uint4& v0, uint4& v1) {
    const int64_t rc = row < p.n ? row : p.n - 1;
    s = __ldg(p.row_entry + rc);
    seq = __ldg(p.row_seq + rc);
    const uint4* src = p.rows + rc * (kRowLen / 8) + c * 2;
    v0 = __ldg(src);
    v1 = __ldg(src + 1);
  };
  int s, seq;
  uint4 v0, v1;
  load(r, s, seq, v0, v1);
  for (; r - sub < p.n; r += stride) {
    bool live = r < p.n;
    const bool ok = s >= 0 && (s >> 6) < p.pt_stride && seq >= 0;
    const int page = __ldg(p.page_table + static_cast<int64_t>(ok ? seq : 0) * p.pt_stride + (ok ? s >> 6 : 0));
    int s_next, seq_next;
    uint4 v0_next, v1_next;
    load(r + stride, s_next, seq_next, v0_next, v1_next);
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t mag = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) mag = max(mag, max((w[j] << 16) & 0x7FFFFFFFu, w[j] & 0x7FFF0000u));
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
    if (live && (!ok || page < 0 || page >= p.num_pages)) {
      if (c == 0) raise_error(kErrIndex);
      live = false;
    }
    if (live) {
      const int slot = s & 63;
      uint8_t* pg = p.base + static_cast<int64_t>(page) * p.page_stride;
      if (rope) {                                 // stored as they are
        uint4* dst = reinterpret_cast<uint4*>(pg + p.rope_off + static_cast<int64_t>(slot) * p.rope_row) +
                     (c - kQuantBlocks * 4) * 2;
        dst[0] = v0;
        dst[1] = v1;
      } else {
        const float scale = __fmul_rn(fmaxf(__uint_as_float(mag), kAmaxFloor), kFp8MaxInv);
        uint32_t codes[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          uint32_t pair = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float x0 = __uint_as_float(w[j + h] << 16), x1 = __uint_as_float(w[j + h] & 0xFFFF0000u);
            const float y0 = fminf(fmaxf(__fdiv_rn(x0, scale), -448.f), 448.f);
            const float y1 = fminf(fmaxf(__fdiv_rn(x1, scale), -448.f), 448.f);
            pair |= static_cast<uint32_t>(static_cast<uint16_t>(
                        __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3)))
                    << (16 * h);
          }
          codes[j / 2] = pair;
        }
        *reinterpret_cast<uint4*>(pg + p.nope_off + static_cast<int64_t>(slot) * p.nope_row + c * 16) =
            make_uint4(codes[0], codes[1], codes[2], codes[3]);
        if ((c & 3) == 0)
          reinterpret_cast<float*>(pg + p.scale_off + static_cast<int64_t>(slot) * p.scale_row)[c >> 2] = scale;
      }
    }
    s = s_next;
    seq = seq_next;
    v0 = v0_next;
    v1 = v1_next;
  }
}

// E2M1 code of an fp32 value in [-6, 6]: the nearest of 0, 0.5, 1, 1.5, 2, 3,
// 4, 6 with ties to the code whose mantissa bit is clear (0.25 -> 0, 0.75 -> 1,
// 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4), counted as the thresholds
// the magnitude passes; bit 3 is the sign (-0 -> 8).
__device__ __forceinline__ uint32_t e2m1_code(float y) {
  const float a = fabsf(y);
  const uint32_t m = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
  return m | ((__float_as_uint(y) >> 28) & 8u);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// fp32 nearest to 128^-0.5, the scale of the order-128 Hadamard rotation.
constexpr float kRot128 = 0x1.6a09e6p-4f;

// fp32 -> BF16 bits, round to nearest, ties to even (finite values).
__device__ __forceinline__ uint32_t bf16_bits_rne(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// The order-128 Hadamard rotation of a key held 16 values a lane across the 8
// lanes of a quarter warp ("DeepSeek-V4 全面解读" §2.9, the compressor's rotate
// path): fp32 butterflies (a + b, a - b) of strides 1, 2, 4, 8 inside the lane,
// then 16, 32, 64 across lanes c ^ 1, c ^ 2, c ^ 4 (the lane holding the lower
// index keeps a + b), then the fp32 scale 128^-0.5 and one rounding to BF16.
// w holds the lane's 16 BF16 values, two per word, and receives the result.
__device__ __forceinline__ void hadamard128_bf16(uint32_t (&w)[8], int c) {
  float v[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
#pragma unroll
  for (int h = 1; h < 16; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if ((i & h) == 0) {
        const float a = v[i], b = v[i + h];
        v[i] = __fadd_rn(a, b);
        v[i + h] = __fsub_rn(a, b);
      }
    }
  }
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) {
    const bool upper = (c & m) != 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float o = __shfl_xor_sync(0xffffffffu, v[i], m);
      v[i] = upper ? __fsub_rn(o, v[i]) : __fadd_rn(v[i], o);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    w[j] = bf16_bits_rne(__fmul_rn(v[2 * j], kRot128)) | (bf16_bits_rne(__fmul_rn(v[2 * j + 1], kRot128)) << 16);
}

// Indexer keys into an IDXK_FP4 pool: a quarter warp per key, 16 values a
// lane, a 32-value block per lane pair; a lane's 16 codes leave as one 8-byte
// store, a key's four exponent bytes as one 4-byte store by its first lane.
// kRotate: each key is first rotated (hadamard128_bf16) and the rotated BF16
// values are quantised.
template <bool kRotate>
__global__ void __launch_bounds__(kThreads) fp4_key_write_kernel(const WriterParams p) {
  griddep_launch();
  griddep_wait();   // the rows may come from the previous kernel of the stream
  const int lane = static_cast<int>(threadIdx.x & 31u);
  const int sub = lane >> 3, c = lane & 7;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * 4;
  for (int64_t r0 = ((static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5) * 4; r0 < p.n;
       r0 += stride) {   // warp-uniform: every lane takes part in the shuffles
    const int64_t r = r0 + sub;
    bool live = r < p.n;
    const int64_t rc = live ? r : p.n - 1;
    const int s = __ldg(p.row_entry + rc), seq = __ldg(p.row_seq + rc);
    const uint4* src = p.rows + rc * 16 + c * 2;
    const uint4 v0 = __ldg(src), v1 = __ldg(src + 1);
    uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    if constexpr (kRotate) hadamard128_bf16(w, c);
    uint32_t mag = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) mag = max(mag, max((w[j] << 16) & 0x7FFFFFFFu, w[j] & 0x7FFF0000u));
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));   // the block's lane pair
    const float t = __fmul_rn(fmaxf(__uint_as_float(mag), kFp4AmaxFloor), kFp4MaxInv);
    const uint32_t tb = __float_as_uint(t);                 // normal: t >= 2^-126
    const int e = static_cast<int>((tb >> 23) & 0xFFu) - 127 + ((tb & 0x7FFFFFu) != 0u ? 1 : 0);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);   // 2^-e, e in [-126, 126]
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x0 = __uint_as_float(w[j] << 16), x1 = __uint_as_float(w[j] & 0xFFFF0000u);
      const uint32_t byte = e2m1_code(fminf(fmaxf(__fmul_rn(x0, inv), -6.f), 6.f)) |
                            (e2m1_code(fminf(fmaxf(__fmul_rn(x1, inv), -6.f), 6.f)) << 4);
      if (j < 4) lo |= byte << (8 * j);
      else hi |= byte << (8 * (j - 4));
    }
    // the four exponent bytes of the key, from lanes 0, 2, 4, 6 of its quarter warp
    const uint32_t eb = static_cast<uint32_t>(e + 127);
    const int q0 = lane & ~7;
    const uint32_t e8 = __shfl_sync(0xffffffffu, eb, q0) | (__shfl_sync(0xffffffffu, eb, q0 + 2) << 8) |
                        (__shfl_sync(0xffffffffu, eb, q0 + 4) << 16) | (__shfl_sync(0xffffffffu, eb, q0 + 6) << 24);
    const bool ok = s >= 0 && (s >> 6) < p.pt_stride && seq >= 0;
    const int page = __ldg(p.page_table + static_cast<int64_t>(ok ? seq : 0) * p.pt_stride + (ok ? s >> 6 : 0));
    if (live && (!ok || page < 0 || page >= p.num_pages)) {
      if (c == 0) raise_error(kErrIndex);
      live = false;
    }
    if (live) {
      const int slot = s & 63;
      uint8_t* pg = p.base + static_cast<int64_t>(page) * p.page_stride;
      *reinterpret_cast<uint2*>(pg + p.nope_off + static_cast<int64_t>(slot) * p.nope_row + c * 8) =
          make_uint2(lo, hi);
      if (c == 0) *reinterpret_cast<uint32_t*>(pg + p.scale_off + static_cast<int64_t>(slot) * p.scale_row) = e8;
    }
  }
}

// KV rows into a KV_FP4 pool: a warp per row, lane c holding the 16-byte units c and
// 32 + c (8 values each), so every load and store of the warp is contiguous.  Units
// 0-55 are the nope part, quantised as the FP4 keys are -- a 32-value block is four
// neighbouring lanes -- and units 56-63 (the second of lanes 24-31) the rope values,
// stored as they are.  A unit's eight codes leave as one 4-byte store, a block's
// exponent as one byte (the last two bytes of the scale row are padding, never
// written).  A block that holds an infinity or a NaN gets the exponent byte 255
// (E8M0 NaN) and codes 0, so it reads back as NaN.  kRowsW rows per warp are in
// flight: the row loads are independent of the entry -> page look-ups.  65529 rows take
// 15.0 us in a graph of such calls, 13.5 being the bytes at the measured copy bandwidth, and
// 32 rows 2.3 (with the grid of launch_rows below, one row a warp takes 14.6 and 1.9, four 15.1
// and 2.9; two were the best of 65529 with eight CTAs a multiprocessor).  The integer pipe is
// nearly as busy (68%).
constexpr int kRowsW = 2;

// Eight values -> eight codes, nearest, ties to even, saturating (as e2m1_code counts out).
__device__ __forceinline__ uint32_t e2m1x8(const float2* y) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0].x), "f"(y[0].y), "f"(y[1].x), "f"(y[1].y), "f"(y[2].x), "f"(y[2].y), "f"(y[3].x), "f"(y[3].y));
  return r;
}

// The codes and the exponent byte of a unit whose block is lanes c, c ^ 1, c ^ 2, c ^ 3.
// The block's absmax is a maximum of BF16 pairs (NaN wins).
__device__ __forceinline__ uint32_t quantise_unit(const uint4 v, uint32_t& exponent) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t a[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] = w[j] & 0x7FFF7FFFu;
  auto max2 = [](uint32_t x, uint32_t y) {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
    return *reinterpret_cast<const uint32_t*>(&m);
  };
  uint32_t m2 = max2(max2(a[0], a[1]), max2(a[2], a[3]));
  m2 = max2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
  m2 = max2(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
  const uint32_t mag = max(m2 << 16, m2 & 0x7FFF0000u);   // as fp32 bits
  const bool finite = mag < 0x7F800000u;
  // e = ceil(log2(max(amax, 6 * 2^-126) * fp32(1/6))).  amax has eight significant bits, so
  // the product is at most a power of two exactly when amax's are at most 1.5: the exponent
  // field goes up by one above that, and by two less than the field's in any case.
  const uint32_t top = max(finite ? mag : 0u, 0x01C00000u);       // 6 * 2^-126
  const uint32_t e = ((top + 0x003FFFFFu) >> 23) - 2u;            // the E8M0 byte: 1 .. 253
  const float inv = __uint_as_float((254u - e) << 23);            // 2^-(e - 127)
  float2 y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    y[j] = mul2(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)), make_float2(inv, inv));
  exponent = finite ? e : 255u;
  return finite ? e2m1x8(y) : 0u;
}

__global__ void __launch_bounds__(kThreads) kv_fp4_write_kernel(const WriterParams p) {
  griddep_launch();
  griddep_wait();   // the rows may come from the previous kernel of the stream
  const int c = static_cast<int>(threadIdx.x & 31u);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * kRowsW;
  for (int64_t r0 = ((static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5) * kRowsW; r0 < p.n;
       r0 += stride) {   // warp-uniform: every lane takes part in the shuffles
    int s[kRowsW], page[kRowsW];
    bool ok[kRowsW];
    uint4 v[kRowsW][2];
#pragma unroll
    for (int k = 0; k < kRowsW; ++k) {   // clamped rows: unconditional loads, all in flight
      const int64_t rc = r0 + k < p.n ? r0 + k : p.n - 1;
      s[k] = __ldg(p.row_entry + rc);
      page[k] = __ldg(p.row_seq + rc);
      v[k][0] = __ldcs(p.rows + rc * 64 + c);
      v[k][1] = __ldcs(p.rows + rc * 64 + 32 + c);
    }
#pragma unroll
    for (int k = 0; k < kRowsW; ++k) {
      ok[k] = s[k] >= 0 && (s[k] >> 6) < p.pt_stride && page[k] >= 0;
      page[k] = __ldg(p.page_table + static_cast<int64_t>(ok[k] ? page[k] : 0) * p.pt_stride + (ok[k] ? s[k] >> 6 : 0));
    }
#pragma unroll
    for (int k = 0; k < kRowsW; ++k) {
      uint32_t e0, e1;
      const uint32_t c0 = quantise_unit(v[k][0], e0);
      const uint32_t c1 = quantise_unit(v[k][1], e1);       // lanes 24-31: rope values, not used
      if (r0 + k >= p.n) continue;
      if (!ok[k] || page[k] < 0 || page[k] >= p.num_pages) {
        if (c == 0) raise_error(kErrIndex);
        continue;
      }
      const int slot = s[k] & 63;
      uint8_t* pg = p.base + static_cast<int64_t>(page[k]) * p.page_stride;
      uint32_t* nope = reinterpret_cast<uint32_t*>(pg + p.nope_off + slot * p.nope_row);
      uint8_t* sc = pg + p.scale_off + slot * p.scale_row;
      nope[c] = c0;
      if ((c & 3) == 0) sc[c >> 2] = static_cast<uint8_t>(e0);
      if (c < 24) {
        nope[32 + c] = c1;
        if ((c & 3) == 0) sc[8 + (c >> 2)] = static_cast<uint8_t>(e1);
      } else {
        reinterpret_cast<uint4*>(pg + p.rope_off + slot * p.rope_row)[c - 24] = v[k][1];
      }
    }
  }
}

// Rows of a KV or KV_FP4 pool back as BF16: value e4m3(code) * scale rounded to
// BF16, or e2m1(code) * 2^(b - 127), which BF16 holds exactly (2 significant
// bits; past its range an infinity, as a product of the two rounds to).  A warp per
// row, lane c writing the 16-byte units c and 32 + c of it as in the writer; kRowsR
// rows per warp in flight.  One: a row is three dependent loads (entry, page id, row), but
// many warps hide them better than many rows a warp do (65529 FP4 rows, in L2 from the
// call before: 15.9 us with one row, 17.3 with two, 17.1 with four), and few rows are read
// sooner (32 rows 1.9 us, 2.3, 2.9).  65529 rows of an FP8 pool take 16.3 us.
constexpr int kRowsR = 1;

struct ReaderParams {
  WriterParams w;          // rows unused
  uint4* out;              // bf16 [n][512]
};

// Eight values: E2M1 codes in x times the scale of byte b, or E4M3 codes in x and y
// times a scale.
__device__ __forceinline__ uint4 read_fp4(uint32_t x, uint32_t b) {
  const BlockScale bs = block_scale(b);
  uint4 v = widen8(x, bs.first);
  if (bs.more) v = scale_up(v, bs.more);
  return v;
}
__device__ __forceinline__ uint4 read_fp8(uint32_t x, uint32_t y, float scale) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(((j < 2 ? x : y) >> (16 * (j & 1))) & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    o[j] = pack2(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool kFp4>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReaderParams q) {
  const WriterParams& p = q.w;
  griddep_launch();
  griddep_wait();
  const int c = static_cast<int>(threadIdx.x & 31u);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads / 32) * kRowsR;
  for (int64_t r0 = ((static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5) * kRowsR; r0 < p.n; r0 += stride) {
    int s[kRowsR], page[kRowsR];
    bool ok[kRowsR];
    uint2 code[kRowsR][2];            // codes of the two units (FP4: in .x)
    uint4 rope[kRowsR];               // lanes 24-31: the second unit
    uint32_t scl[kRowsR][2];          // the scale byte, or the fp32 scale's bits
#pragma unroll
    for (int k = 0; k < kRowsR; ++k) {
      const int64_t rc = r0 + k < p.n ? r0 + k : p.n - 1;
      s[k] = __ldg(p.row_entry + rc);
      page[k] = __ldg(p.row_seq + rc);
    }
#pragma unroll
    for (int k = 0; k < kRowsR; ++k) {
      ok[k] = s[k] >= 0 && (s[k] >> 6) < p.pt_stride && page[k] >= 0;
      page[k] = __ldg(p.page_table + static_cast<int64_t>(ok[k] ? page[k] : 0) * p.pt_stride + (ok[k] ? s[k] >> 6 : 0));
    }
#pragma unroll
    for (int k = 0; k < kRowsR; ++k) {
      const bool bad = !ok[k] || page[k] < 0 || page[k] >= p.num_pages;
      if (bad && s[k] != -1 && r0 + k < p.n && c == 0) raise_error(kErrIndex);   // -1: no row there, zeros
      ok[k] = !bad;
      const int slot = s[k] & 63;
      const uint8_t* pg = p.base + static_cast<int64_t>(ok[k] ? page[k] : 0) * p.page_stride;
      const uint8_t* nope = pg + p.nope_off + slot * p.nope_row;
      const uint8_t* sc = pg + p.scale_off + slot * p.scale_row;
      rope[k] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int u = 32 * h + c;
        code[k][h] = make_uint2(0u, 0u);
        scl[k][h] = 0u;
        if (!ok[k]) continue;
        if (u >= 56) {
          rope[k] = __ldcs(reinterpret_cast<const uint4*>(pg + p.rope_off + slot * p.rope_row) + (u - 56));
        } else if constexpr (kFp4) {
          code[k][h].x = __ldcs(reinterpret_cast<const uint32_t*>(nope) + u);
          scl[k][h] = __ldcs(sc + (u >> 2));
        } else {
          code[k][h] = __ldcs(reinterpret_cast<const uint2*>(nope) + u);
          scl[k][h] = __ldcs(reinterpret_cast<const uint32_t*>(sc) + (u >> 3));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kRowsR; ++k) {
      if (r0 + k >= p.n) continue;
      uint4* dst = q.out + (r0 + k) * 64;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 v;
        if constexpr (kFp4) v = read_fp4(code[k][h].x, scl[k][h]);
        else v = read_fp8(code[k][h].x, code[k][h].y, __uint_as_float(scl[k][h]));
        __stcs(dst + 32 * h + c, h == 1 && c >= 24 ? rope[k] : v);
      }
    }
  }
}

// CTAs of `rows_per_block` rows over n rows, at most 20 a multiprocessor (six run at once):
// enough that none is left with more to do, few enough that starting them does not show
// (65529 FP4 rows written and then read, in a graph: 32.4 us; 64 a multiprocessor, one batch
// each, 33.9, 12 33.3, 8 34.7).
template <class P>
cudaError_t launch_rows(void (*kernel)(P), const P& p, int64_t n, int64_t rows_per_block, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorUnknown;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return cudaErrorUnknown;
  const int64_t want = (n + rows_per_block - 1) / rows_per_block, cap = static_cast<int64_t>(sms) * 20;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)), dim3(kThreads), 0, stream, p);
}

template <int kLanesPerRow, int kQuantBlocks>
cudaError_t launch_writer(const WriterParams& p, cudaStream_t stream) {
  static int resident = 0;                       // CTAs per SM, queried once
  if (resident == 0 &&
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, cache_write_kernel<kLanesPerRow, kQuantBlocks>,
                                                    kThreads, 0) != cudaSuccess)
    return cudaErrorUnknown;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorUnknown;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return cudaErrorUnknown;
  const int64_t rows_per_block = static_cast<int64_t>(kThreads / 32) * (32 / kLanesPerRow);
  const int64_t want = (p.n + rows_per_block - 1) / rows_per_block;
  const int64_t full = static_cast<int64_t>(sms) * (resident > 0 ? resident : 1);
  const int64_t blocks = want < full ? want : full;
  return launch_pdl(cache_write_kernel<kLanesPerRow, kQuantBlocks>, dim3(static_cast<unsigned>(blocks)),
                    dim3(kThreads), 0, stream, p);
}

}  // namespace

static WriterParams pool_params(const dsv4sa_pool_desc* pool, const int32_t* page_table, int32_t pt_stride,
                                const int32_t* row_seq, const int32_t* row_entry, int32_t n) {
  WriterParams p{};
  p.page_table = page_table;
  p.row_seq = row_seq;
  p.row_entry = row_entry;
  p.base = static_cast<uint8_t*>(pool->base);
  p.page_stride = pool->page_stride;
  p.num_pages = pool->num_pages;
  p.nope_off = pool->nope_off;
  p.rope_off = pool->rope_off;
  p.scale_off = pool->scale_off;
  p.nope_row = pool->nope_row;
  p.rope_row = pool->rope_row;
  p.scale_row = pool->scale_row;
  p.pt_stride = pt_stride;
  p.n = n;
  return p;
}

int launch_cache_read(const dsv4sa_pool_desc* pool, const int32_t* page_table, int32_t pt_stride,
                      const int32_t* row_seq, const int32_t* row_entry, void* rows, int32_t n, cudaStream_t stream) {
  const ReaderParams q{pool_params(pool, page_table, pt_stride, row_seq, row_entry, n), static_cast<uint4*>(rows)};
  constexpr int64_t per = (kThreads / 32) * kRowsR;
  const cudaError_t e = pool->kind == DSV4SA_POOL_KV_FP4 ? launch_rows(cache_read_kernel<true>, q, n, per, stream)
                                                         : launch_rows(cache_read_kernel<false>, q, n, per, stream);
  return e == cudaSuccess ? DSV4SA_OK : DSV4SA_ERR_CUDA;
}

int launch_cache_write(const dsv4sa_pool_desc* pool, const int32_t* page_table, int32_t pt_stride,
                       const int32_t* row_seq, const int32_t* row_entry, const void* rows, int32_t n,
                       bool rotate, cudaStream_t stream) {
  WriterParams p = pool_params(pool, page_table, pt_stride, row_seq, row_entry, n);
  p.rows = static_cast<const uint4*>(rows);
  const bool kv = pool->kind == DSV4SA_POOL_KV;
  if (n == 0) return DSV4SA_OK;
  if (pool->kind == DSV4SA_POOL_KV_FP4 && !rotate)
    return launch_rows(kv_fp4_write_kernel, p, n, (kThreads / 32) * kRowsW, stream) == cudaSuccess ? DSV4SA_OK
                                                                                                   : DSV4SA_ERR_CUDA;
  if (pool->kind == DSV4SA_POOL_IDXK_FP4) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
    const int64_t rows_per_block = (kThreads / 32) * 4;
    const int64_t want = (static_cast<int64_t>(n) + rows_per_block - 1) / rows_per_block;
    const int64_t cap = static_cast<int64_t>(sms) * 8;
    const int64_t blocks = want < cap ? want : cap;
    const cudaError_t e =
        rotate ? launch_pdl(fp4_key_write_kernel<true>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0,
                            stream, p)
               : launch_pdl(fp4_key_write_kernel<false>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0,
                            stream, p);
    return e == cudaSuccess ? DSV4SA_OK : DSV4SA_ERR_CUDA;
  }
  if (rotate) return DSV4SA_ERR_UNSUPPORTED;   // rotation is the FP4 key path only
  const cudaError_t e = kv ? launch_writer<32, 7>(p, stream) : launch_writer<8, 2>(p, stream);
  return e == cudaSuccess ? DSV4SA_OK : DSV4SA_ERR_CUDA;
}

uint32_t read_error_word_writer(cudaStream_t stream, bool clear) {
  uint32_t v = 0;
  cudaMemcpyFromSymbolAsync(&v, g_err_word, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  cudaStreamSynchronize(stream);
  if (clear && v) {
    const uint32_t z = 0;
    cudaMemcpyToSymbolAsync(g_err_word, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream);
    cudaStreamSynchronize(stream);
  }
  return v;
}

}  // namespace dsv4sa
