// fp4.cuh -- E2M1 codes with an E8M0 scale (one byte per 32 values) to BF16, exactly.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace dsv4sa {

// The block scale 2^(b - 127) for widen8: `first` = 2^min(b - 1, 127) in BF16, in
// both halves (the codes are placed 2^126 too small), `more` = the exponent still to
// be added for blocks of magnitudes above 12.  Byte 255 is NaN.
struct BlockScale {
  uint32_t first;
  uint32_t more;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t b) {
  const uint32_t e = min(b + 126u, 254u);                 // b = 0: 2^-1
  const uint32_t h = b == 255u ? 0x7FC0u : e << 7;
  return BlockScale{h | (h << 16), b > 128u && b != 255u ? b - 128u : 0u};
}

// Eight E2M1 codes -> eight BF16 values.  The two codes of a byte become one
// register: a multiplication by 2^6 + 2^18 puts the three magnitude bits of either
// where BF16 keeps the last two exponent bits and the first mantissa bit, one by
// 2^12 + 2^24 their signs; as a BF16 number that is the value times 2^-126 (a
// magnitude of 1, 0.5, is subnormal there as here), and the product with the
// scale restores it exactly.  Half of the work is on the FMA pipe, so it does not
// all queue for the ALU, as a table by byte permutations does.
__device__ __forceinline__ uint4 widen8(uint32_t w, uint32_t first) {
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&first);
  uint32_t v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t byte = __byte_perm(w, 0u, 0x4440 + j);
    const uint32_t x = ((byte * 0x00040040u) & 0x01C001C0u) | ((byte * 0x01001000u) & 0x80008000u);
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), s);
    v[j] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// The same in the order 0, 4, 1, 5, 2, 6, 3, 7: codes 16 bits apart share a register from
// the start, so one masked word times 2^6 + 2^12 (or 2^2 + 2^8, a nibble further on) places
// magnitude and sign of both: 17 instructions instead of 24.
__device__ __forceinline__ uint4 widen8_split(uint32_t w, uint32_t first) {
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&first);
  uint32_t v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t part = j < 2 ? w : w >> 8;
    const uint32_t x = ((j & 1) ? (part & 0x00F000F0u) * 0x0104u : (part & 0x000F000Fu) * 0x1040u) & 0x81C081C0u;
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), s);
    v[j] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// Eight values times 2^more (rarely called).
__device__ __forceinline__ uint4 scale_up(uint4 v, uint32_t more) {
  // in two steps: 2^more may pass BF16's range although the product does not
  const uint32_t a = min(more, 64u), c = more - a;
  const uint32_t ha = (127u + a) << 7, hc = (127u + c) << 7;
  const uint32_t fa = ha | (ha << 16), fc = hc | (hc << 16);
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    __nv_bfloat162 x = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&w[j]), *reinterpret_cast<const __nv_bfloat162*>(&fa));
    x = __hmul2(x, *reinterpret_cast<const __nv_bfloat162*>(&fc));
    w[j] = *reinterpret_cast<uint32_t*>(&x);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace dsv4sa
