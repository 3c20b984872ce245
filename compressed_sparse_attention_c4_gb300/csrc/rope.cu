// rope.cu -- rotary positions: the (cos, sin) table of a context, and rows of heads rotated by it.
//
// Table ("DeepSeek-V4 全面解读" §2.6 precompute_freqs_cis): row r, pair i holds (cos, sin) of
// (first + r) w_i, w_i = base^(-2i/d), the low frequencies divided by `factor` where the
// context is scaled (YaRN: w_i / factor below a ramp of pairs, w_i above it).
// Rotation (§2.6 apply_rotary_emb; §2.11: each query head divided by its root mean square,
// without weights, before): (a, b) -> (a c - b s, b c + a s), the inverse with -s.
#include <cmath>

#include "common.cuh"
#include "dsv4sa_internal.h"

namespace dsv4sa {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- table
// An angle is a phase: w_i / 2 pi as a 64-bit fraction of a turn, times the position, modulo
// 2^64.  Whole turns drop out exactly; the fraction is the nearest one, half a step of 2^-64 turn off,
// so position n is off by at most n 2^-62.3 (2^-31 at the last 31-bit position, 2^-24, fp32's own
// rounding, at 2^38).  A frequency in fp64 would be off by n 2^-53.  The nearest quarter turn is
// taken off in whole numbers, too; what is left, at most an eighth of a turn with 64 bits below the
// point, is rounded to fp32 and goes through the Taylor series of sine and cosine (to x^9 and
// x^10: 2^-28 and 2^-32 at pi / 4).  A thread keeps one pair and
// adds a constant phase from row to row.  Bound by HBM (written once) and instructions both: 1M rows
// of 32 pairs 46.4 us, 39.5 at the measured copy bandwidth; CUDA's sincospif took 59.7.
struct TableParams {
  float2* cs;
  int64_t first;
  int64_t rows;
  int32_t pairs;
  int32_t rows_per_block;
  uint64_t turn[DSV4SA_MAX_ROPE_PAIRS];
};

__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ TableParams p) {
  griddep_launch();
  griddep_wait();
  const int i = static_cast<int>(threadIdx.x) % p.pairs, sub = static_cast<int>(threadIdx.x) / p.pairs;
  if (sub >= p.rows_per_block) return;
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.rows_per_block;
  int64_t r = static_cast<int64_t>(blockIdx.x) * p.rows_per_block + sub;
  const uint64_t turn = p.turn[i], turn_step = turn * static_cast<uint64_t>(step);
  uint64_t phase = turn * static_cast<uint64_t>(p.first + r);
  for (; r < p.rows; r += step, phase += turn_step) {
    const uint64_t at = phase + (uint64_t{1} << 61);
    const uint32_t quarter = static_cast<uint32_t>(at >> 62);
    const int64_t rest = static_cast<int64_t>((at & ((uint64_t{1} << 62) - 1)) - (uint64_t{1} << 61));
    // hi 2^32 + lo, each rounded on its own where it is long
    const float part = fmaf(static_cast<float>(static_cast<int32_t>(rest >> 32)), 0x1p32f, static_cast<float>(static_cast<uint32_t>(rest)));
    const float x = part * static_cast<float>(6.283185307179586476925 * 0x1p-64), xx = x * x;
    const float s0 = fmaf(xx, fmaf(xx, fmaf(xx, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6);
    const float c0 = fmaf(xx, fmaf(xx, fmaf(xx, fmaf(xx, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f);
    const float s = fmaf(x * xx, s0, x), c = fmaf(xx, c0, 1.f);
    const uint32_t odd = quarter & 1u;
    const uint32_t a = __float_as_uint(odd ? s : c) ^ ((quarter + 1u & 2u) << 30), b = __float_as_uint(odd ? c : s) ^ ((quarter & 2u) << 30);
    __stcs(p.cs + r * p.pairs + i, make_float2(__uint_as_float(a), __uint_as_float(b)));
  }
}

// ---------------------------------------------------------------- rotation
// A row (one head of one token) is units of 8 values; L lanes share it, lane c holding units
// c, c + L, ... .  Pairs side by side lie in one unit; with the pairs in two halves a lane loads
// its unit's partner too (the neighbours of its group have just asked for the same lines).
// In place and without a norm only the rotated units are touched.  Bound by HBM: 4096 x 64 heads of
// 512, normed, 86.9 us (79.2 at the copy bandwidth), 8191 x 64 of 128 in halves 48.2 (39.8), 32 x 64
// of 512 2.4 (latency: position, table row).
struct RopeParams {
  const uint4* x;
  uint4* out;
  const float4* cs;        // table rows of 2 * ru float4
  const int32_t* pos;
  const float* w;          // null: no weights
  int64_t x_tok, x_head, out_tok, out_head;   // strides in units
  uint32_t rows;           // T H
  uint32_t H;
  int32_t ub, ue;          // units of a row that are read and written
  int32_t u0, ru;          // rotated units [u0, u0 + ru)
  int32_t rope_rows;
  float sign;              // -1: the inverse rotation
  float inv_dim, eps;
};

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void times_weights(float (&f)[8], const float* w) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w)), b = __ldg(reinterpret_cast<const float4*>(w) + 1);
  f[0] *= a.x, f[1] *= a.y, f[2] *= a.z, f[3] *= a.w, f[4] *= b.x, f[5] *= b.y, f[6] *= b.z, f[7] *= b.w;
}

template <int L, int U, bool kNorm, bool kHalves>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  griddep_launch();
  griddep_wait();
  const uint32_t c = threadIdx.x % L, sub = (threadIdx.x & 31u) / L;
  constexpr uint32_t kPerWarp = 32 / L;
  const uint32_t step = gridDim.x * (kThreads / L);
  for (uint32_t r0 = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kPerWarp; r0 < p.rows; r0 += step) {   // warp-uniform
    const bool live = r0 + sub < p.rows;
    const uint32_t row = live ? r0 + sub : p.rows - 1;
    const uint32_t t = row / p.H, h = row - t * p.H;
    const uint4* src = p.x + static_cast<int64_t>(t) * p.x_tok + static_cast<int64_t>(h) * p.x_head;
    const int32_t at = __ldg(p.pos + t);
    uint4 v[U], other[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = p.ub + i * L + static_cast<int>(c), j = u - p.u0;
      v[i] = u < p.ue ? src[u] : make_uint4(0u, 0u, 0u, 0u);
      if (kHalves && j >= 0 && j < p.ru) other[i] = src[p.u0 + (2 * j < p.ru ? j + p.ru / 2 : j - p.ru / 2)];
    }
    float rstd = 1.f;
    if constexpr (kNorm) {
      float sq = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float f[8];
        unpack8(v[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) sq = fmaf(f[k], f[k], sq);
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      rstd = rsqrtf(fmaf(sq, p.inv_dim, p.eps));
    }
    const bool known = at >= 0 && at < p.rope_rows;
    if (!known && live && c == 0) raise_error(kErrIndex);
    const float4* cs = p.cs + static_cast<int64_t>(known ? at : 0) * (2 * p.ru);
    uint4* dst = p.out + static_cast<int64_t>(t) * p.out_tok + static_cast<int64_t>(h) * p.out_head;
    __syncwarp();            // in place: every lane of the row has its values and its partners'
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = p.ub + i * L + static_cast<int>(c), j = u - p.u0;
      const bool turned = j >= 0 && j < p.ru;
      if (!live || u >= p.ue) continue;
      if (!kNorm && !turned) {
        dst[u] = v[i];
        continue;
      }
      float f[8];
      unpack8(v[i], f);
      if constexpr (kNorm) {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= rstd;
        if (p.w) times_weights(f, p.w + 8 * u);
      }
      if (turned && known) {
        if constexpr (kHalves) {
          const bool upper = 2 * j >= p.ru;
          const int k0 = upper ? j - p.ru / 2 : j;
          float g[8];
          unpack8(other[i], g);
          if constexpr (kNorm) {
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] *= rstd;
            if (p.w) times_weights(g, p.w + 8 * (p.u0 + k0 + (upper ? 0 : p.ru / 2)));
          }
          const float sign = upper ? p.sign : -p.sign;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 z = __ldg(cs + 4 * k0 + k);
            f[2 * k] = fmaf(f[2 * k], z.x, g[2 * k] * (sign * z.y));
            f[2 * k + 1] = fmaf(f[2 * k + 1], z.z, g[2 * k + 1] * (sign * z.w));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float4 z = __ldg(cs + 2 * j + k);
            const float s0 = p.sign * z.y, s1 = p.sign * z.w;
            const float a0 = f[4 * k], b0 = f[4 * k + 1], a1 = f[4 * k + 2], b1 = f[4 * k + 3];
            f[4 * k] = fmaf(a0, z.x, -(b0 * s0)), f[4 * k + 1] = fmaf(b0, z.x, a0 * s0);
            f[4 * k + 2] = fmaf(a1, z.z, -(b1 * s1)), f[4 * k + 3] = fmaf(b1, z.z, a1 * s1);
          }
        }
      }
      dst[u] = pack8(f);
    }
  }
}

template <int L, int U, bool kNorm>
cudaError_t launch_rope_l(const RopeParams& p, bool halves, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorUnknown;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return cudaErrorUnknown;
  const int64_t per = kThreads / L, want = (static_cast<int64_t>(p.rows) + per - 1) / per, cap = static_cast<int64_t>(sms) * 32;
  const dim3 grid(static_cast<unsigned>(want < cap ? want : cap));
  return halves ? launch_pdl(rope_kernel<L, U, kNorm, true>, grid, dim3(kThreads), 0, stream, p)
                : launch_pdl(rope_kernel<L, U, kNorm, false>, grid, dim3(kThreads), 0, stream, p);
}
template <int L, int U>
cudaError_t launch_rope_lu(const RopeParams& p, bool norm, bool halves, cudaStream_t stream) {
  return norm ? launch_rope_l<L, U, true>(p, halves, stream) : launch_rope_l<L, U, false>(p, halves, stream);
}

}  // namespace

// Pairs of doubles, hi + lo with |lo| at most half a step of hi: about 100 bits (Dekker, "A
// floating-point technique for extending the available precision", 1971; the product by fma).
struct Two {
  double hi, lo;
};
static Two sum_of(double a, double b) {    // |a| >= |b|
  const double s = a + b;
  return {s, b - (s - a)};
}
static Two add(Two a, Two b) {
  const double s = a.hi + b.hi, t = s - a.hi;
  return sum_of(s, ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo));
}
static Two mul(Two a, Two b) {
  const double p = a.hi * b.hi;
  return sum_of(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
static Two ratio(double a, double b) {
  const double q = a / b;
  return {q, std::fma(-q, b, a) / b};
}

int launch_rope_table(float* cs, int64_t rows, int32_t pairs, int64_t first, double base, double factor,
                      int64_t original_len, double beta_fast, double beta_slow, cudaStream_t stream) {
  constexpr double kPi = 3.14159265358979323846;
  TableParams p{};
  p.cs = reinterpret_cast<float2*>(cs);
  p.first = first;
  p.rows = rows;
  p.pairs = pairs;
  p.rows_per_block = kThreads / pairs;
  // YaRN: pairs that turn more than beta_fast times over the original length keep their
  // frequency, those that turn less than beta_slow times are divided, a ramp between
  const double d = 2.0 * pairs;
  double lo = 0, hi = 0;
  if (original_len > 0) {
    auto border = [&](double beta) { return d * std::log(original_len / (beta * 2 * kPi)) / (2 * std::log(base)); };
    lo = std::fmax(std::floor(border(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(border(beta_slow)), d - 1);
  }
  // base^(-1 / pairs): fp64's, and one step of Newton's on base x^pairs = 1
  const double near = std::pow(base, -1.0 / pairs);
  Two p2 = {near, 0}, power = {base, 0};
  for (int32_t n = pairs; n > 0; n >>= 1, p2 = mul(p2, p2))
    if (n & 1) power = mul(power, p2);
  const Two root = mul({near, 0}, add({1, 0}, {-add(power, {-1, 0}).hi / pairs, 0}));
  const Two shrink = ratio(1.0, factor), per_turn = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};   // 1 / factor, 1 / 2 pi
  Two w = {1, 0};
  for (int32_t i = 0; i < pairs; ++i, w = mul(w, root)) {
    // the part of w that is divided; original_len 0: all (positions interpolated)
    Two part = {1, 0};
    if (original_len > 0) part = i <= lo ? Two{0, 0} : i >= hi ? Two{1, 0} : ratio(i - lo, hi - lo);
    const Two turns = mul(mul(w, add(add({1, 0}, {-part.hi, -part.lo}), mul(shrink, part))), per_turn);
    const double x = std::ldexp(turns.hi, 64), whole = std::floor(x);       // below 2^62
    p.turn[i] = static_cast<uint64_t>(whole) + static_cast<uint64_t>(std::llround((x - whole) + std::ldexp(turns.lo, 64)));
  }
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  const int64_t want = (rows + p.rows_per_block - 1) / p.rows_per_block, cap = static_cast<int64_t>(sms) * 32;
  return launch_pdl(rope_table_kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)), dim3(kThreads), 0, stream, p) ==
                 cudaSuccess
             ? DSV4SA_OK
             : DSV4SA_ERR_CUDA;
}

int launch_rope(const dsv4sa_rope_args* a, cudaStream_t stream) {
  RopeParams p{};
  p.x = static_cast<const uint4*>(a->x);
  p.out = static_cast<uint4*>(a->out);
  p.cs = reinterpret_cast<const float4*>(a->rope_cs);
  p.pos = a->pos;
  p.w = a->norm ? a->norm_w : nullptr;
  p.x_tok = a->x_tok_stride / 8, p.x_head = a->x_head_stride / 8;
  p.out_tok = a->out_tok_stride / 8, p.out_head = a->out_head_stride / 8;
  p.rows = static_cast<uint32_t>(a->T) * static_cast<uint32_t>(a->H);
  p.H = static_cast<uint32_t>(a->H);
  p.u0 = a->rope_off / 8, p.ru = a->rope_dim / 8;
  const bool part = a->x == a->out && !a->norm;      // the other units stay as they are
  p.ub = part ? p.u0 : 0;
  p.ue = part ? p.u0 + p.ru : a->dim / 8;
  p.rope_rows = a->rope_rows;
  p.sign = a->inverse ? -1.f : 1.f;
  p.inv_dim = 1.0f / static_cast<float>(a->dim);
  p.eps = a->eps;
  const bool norm = a->norm != 0, halves = a->layout == DSV4SA_ROPE_HALVES;
  const int units = p.ue - p.ub;
  cudaError_t e;
  if (units <= 8) e = launch_rope_lu<4, 2>(p, norm, halves, stream);
  else if (units <= 16) e = launch_rope_lu<8, 2>(p, norm, halves, stream);
  else if (units <= 32) e = launch_rope_lu<16, 2>(p, norm, halves, stream);
  else if (units <= 64) e = launch_rope_lu<32, 2>(p, norm, halves, stream);
  else e = launch_rope_lu<32, 4>(p, norm, halves, stream);
  return e == cudaSuccess ? DSV4SA_OK : DSV4SA_ERR_CUDA;
}

uint32_t* error_word_rope() { return error_word(); }

}  // namespace dsv4sa
