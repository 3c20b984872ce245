// attn_fp4.cu -- sparse attention with attention sink over gathered rows of a
// 4-bit KV cache (E2M1 codes, one E8M0 scale per 32 values, BF16 rope part).
//
// For query t, head h and the multiset J of valid indices of
// idx_c[t] (compressed pool) ++ the window (raw-token pool):
//   o[t, h] = sum_j e^{a_j} kv_j / (sum_j e^{a_j} + e^{sink_h}),  a_j = scale * q[t, h] . kv_j
// ("DeepSeek-V4 全面解读" §3.7 sparse_attn_kernel, §3.5 fp4_quant_kernel for the
// format; "tilelang量化内核拆解…" sparse_attn 实现拆解: running max starts at -1e30;
// "DeepSeek-V4 in SGLang" MQALayer: one kv tensor is both K and V.)
//
// Work.  An item is one query and a group of HN = 16, 32 or 64 heads.  With one
// CTA per item the grid is persistent and each CTA walks items; else the CS
// CTAs of a thread-block cluster share an item, CTA r taking every CS-th run of
// 32 list positions, and merge at the end.
//
// Pipeline of a CTA.  The valid rows of the lists are packed -- J is a multiset,
// their order is free -- into chunks of 128, so -1 entries cost no tensor work:
//   gather warps (8): index -> page id -> row, 256 positions at a time, the valid
//     ones appended to a ring; a chunk's rows (16-byte pieces, two threads a row)
//     are loaded into registers while the tensor core works on the chunk before,
//     then widened to BF16 and stored in the 128 x 512 tile, 128 dims at a time,
//     each as soon as the previous chunk's PV has read those dims.
//   MMA thread: S^T = KV . Q^T (M = 128 rows, N = HN, K = 512), 128 dims at a time
//     as they arrive; then O^T += V^T . P^T (M = 128 dims x 4, N = HN, K = 128): the
//     tile is read K-major for S and MN-major for PV.
//   softmax warps (8): thread = row, half of the heads.  P in BF16 against a max
//     that is only moved (and O rescaled) when a score passes it by 2^8: a vote
//     replaces the max's reduction in nearly every chunk but the first.  The
//     sum of the probabilities stays with its row's thread until the
//     end.  Then the output is scaled, rotated back and written from TMEM while
//     the next item's S runs.
// Widening is exact: a code's BF16 bits are looked up (two byte permutations for
// four codes) and multiplied by the power of two in BF16.  P is the one operand
// rounded (BF16, 2^-9 of a probability); S, O, maxima, sums and the partial
// results that a cluster exchanges are fp32.
#include "attn_common.cuh"

namespace dsv4sa {
namespace {

using namespace attn;

constexpr int kComputeThreads = 256;     // warps 0-7
constexpr int kGatherThreads = 256;      // warps 8-15
constexpr int kThreads4 = kComputeThreads + kGatherThreads + 32;   // warp 16: MMA
constexpr int kRing = 512;               // located rows waiting for a chunk
constexpr int kRun = 32;                 // list positions a CTA of a cluster takes in a row
constexpr int kFp4RopeOff = 14336;       // KV_FP4 page layout (see dsv4sa.h)
constexpr int kFp4ScaleOff = 22528;
constexpr float kSlack = 8.f;            // log2 units a score may pass the max in use by

constexpr uint32_t kBarCompute4 = 1;     // named barriers
constexpr uint32_t kBarGather4 = 2;

template <int HN>
struct Smem4 {
  static constexpr int kKv = 0;
  static constexpr int kQ = kKvBytes;                    // 8 column blocks x HN rows x 128 B
  static constexpr int kP = kQ + 8 * HN * 128;           // 128 rows x 128 B, or 2 blocks x HN rows x 128 B
  static constexpr int kTiles = kP + kRows * 128;        // end of the tiles (the merge may use all of them)
  static constexpr int kRing_ = kTiles;                  // uint64 [kRing]
  static constexpr int kRed = kRing_ + kRing * 8;        // float [HN][4]
  static constexpr int kM = kRed + HN * 16;              // float [HN] each
  static constexpr int kAlpha = kM + HN * 4;
  static constexpr int kFac = kAlpha + HN * 4;           // float [kMaxClusterSplits][HN]
  static constexpr int kMl = kFac + kMaxClusterSplits * HN * 4;   // float2 [kMaxClusterSplits][HN]
  static constexpr int kCnt = kMl + kMaxClusterSplits * HN * 8;   // int [8]
  static constexpr int kMeta = kCnt + 32;                // int [2]
  static constexpr int kBar = kMeta + 16;                // barriers, see below
  static constexpr int kTmem = kBar + 17 * 8 + 8;
  static constexpr int kBytes = kTmem + 16;
};

// 32 E2M1 codes (16 bytes) times a power of two (BF16, in both halves) -> 32 BF16
// values, out[w] = values 8 w .. 8 w + 7.
__device__ __forceinline__ void widen32(const uint4 codes, uint32_t scale2, uint4* out) {
  const uint32_t w4[4] = {codes.x, codes.y, codes.z, codes.w};
  const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&scale2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = w4[i];
    const uint32_t sel = w & 0x77777777u, sel2 = sel >> 16;
    // BF16 of 0, 0.5, 1, 1.5, 2, 3, 4, 6: high bytes, then low bytes
    const uint32_t h0 = __byte_perm(0x3F3F3F00u, 0x40404040u, sel), l0 = __byte_perm(0xC0800000u, 0xC0804000u, sel);
    const uint32_t h1 = __byte_perm(0x3F3F3F00u, 0x40404040u, sel2), l1 = __byte_perm(0xC0800000u, 0xC0804000u, sel2);
    uint32_t v[4] = {__byte_perm(l0, h0, 0x5140), __byte_perm(l0, h0, 0x7362), __byte_perm(l1, h1, 0x5140),
                     __byte_perm(l1, h1, 0x7362)};
    v[0] |= ((w << 12) & 0x8000u) | ((w << 24) & 0x80000000u);
    v[1] |= ((w << 4) & 0x8000u) | ((w << 16) & 0x80000000u);
    v[2] |= ((w >> 4) & 0x8000u) | ((w << 8) & 0x80000000u);
    v[3] |= ((w >> 12) & 0x8000u) | (w & 0x80000000u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v[j]), s);
      v[j] = *reinterpret_cast<const uint32_t*>(&x);
    }
    out[i] = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// 2^(b - 127) in BF16, in both halves; 255 is NaN.
__device__ __forceinline__ uint32_t e8m0_bf16x2(uint32_t b) {
  const uint32_t h = b == 0u ? 0x0040u : (b == 255u ? 0x7FC0u : b << 7);
  return h | (h << 16);
}

__device__ __forceinline__ bool any_of(bool v, uint32_t id, uint32_t n) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(v ? 1u : 0u), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// 16-byte asynchronous copy into shared memory; bytes = 0 writes zeros.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Positions of a list of n that CTA r of CS takes, and the k-th of them.
__device__ __forceinline__ int share_of(int n, int r, int CS) {
  const int whole = n / (kRun * CS), rest = n - whole * kRun * CS - r * kRun;
  return whole * kRun + min(max(rest, 0), kRun);
}
__device__ __forceinline__ int share_at(int k, int r, int CS) { return ((k / kRun) * CS + r) * kRun + k % kRun; }

template <int HN>
__global__ void __launch_bounds__(kThreads4, 1) sparse_attn_fp4_kernel(const AttnParams p, int groups) {
  using S = Smem4<HN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* kv = smem + S::kKv;
  uint8_t* qs = smem + S::kQ;
  uint8_t* ps = smem + S::kP;
  uint64_t* ring = reinterpret_cast<uint64_t*>(smem + S::kRing_);
  float* red = reinterpret_cast<float*>(smem + S::kRed);
  float* m_used = reinterpret_cast<float*>(smem + S::kM);
  float* alpha = reinterpret_cast<float*>(smem + S::kAlpha);
  float* fac = reinterpret_cast<float*>(smem + S::kFac);
  float2* mlr = reinterpret_cast<float2*>(smem + S::kMl);
  int* wcnt = reinterpret_cast<int*>(smem + S::kCnt);
  volatile int* meta = reinterpret_cast<volatile int*>(smem + S::kMeta);
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + S::kBar);   // [4]: 128 dims of the chunk are in the tile
  uint64_t* bar_free = bar_full + 4;     // [4]: ... have been read by PV
  uint64_t* bar_tok = bar_full + 8;      // [2]: a chunk's (or an item's end's) meta is written
  uint64_t* bar_s = bar_full + 10;       // S is complete
  uint64_t* bar_p = bar_full + 11;       // P is written
  uint64_t* bar_o = bar_full + 12;       // every PV of the item is complete
  uint64_t* bar_q = bar_full + 13;       // the item's Q is in place
  uint64_t* bar_item = bar_full + 14;    // the end of the item has been seen
  uint64_t* bar_recv = bar_full + 15;    // merge: the other splits' partials landed
  uint64_t* bar_ml = bar_full + 16;      // merge: the other splits' (m, l) landed
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + S::kTmem);

  constexpr int HW = HN / 2;             // heads of a softmax thread
  constexpr uint32_t kTmemCols = HN == 64 ? 512u : (HN == 32 ? 256u : 128u);
  constexpr uint32_t kColS = 0, kColO = HN;
  const int CS = p.nsplit;
  const int crank = CS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tid = static_cast<int>(threadIdx.x);
  const uint32_t warp = warp_id(), lane = lane_id();
  const int n_items = p.T * groups, item0 = static_cast<int>(blockIdx.x) / CS;
  const int item_step = static_cast<int>(gridDim.x) / CS;
  const int slice = 512 / CS;            // dims of the output this CTA writes
  const int slot_bytes = slice * HN * 4;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar_full + i, kGatherThreads / 32);
      mbar_init(bar_free + i, 1);
    }
    mbar_init(bar_tok, 1);
    mbar_init(bar_tok + 1, 1);
    mbar_init(bar_s, 1);
    mbar_init(bar_p, kComputeThreads / 32);
    mbar_init(bar_o, 1);
    mbar_init(bar_q, kComputeThreads / 32);
    mbar_init(bar_item, 1);
    mbar_init(bar_recv, 1);
    mbar_init(bar_ml, CS > 1 ? (CS - 1) * HN : 1);
    fence_mbar_init();
    if (CS > 1) mbar_arrive_expect_tx(bar_recv, static_cast<uint32_t>((CS - 1) * slot_bytes));
  }
  if (warp == 16) {
    tmem_alloc(tmem_holder, kTmemCols);
    tmem_relinquish();
  }
  griddep_launch();
  // Without early_window every input may come from the previous kernel of the
  // stream; with it only idx_c does.
  if (!p.early_window) griddep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (CS > 1) cluster_sync();            // every CTA's barriers are initialised before any remote arrival
  const uint32_t tmem = *tmem_holder;
  bool ok = true;                        // no wait of this thread has run out

  if (warp >= 8 && warp < 16) {
    // =========================== gather warps ===========================
    // A wait that runs out is not repeated: the loop, whose length the lists
    // alone decide, goes on without waiting.
    const int gt = tid - kComputeThreads;
    const int row = gt >> 1, half = gt & 1;
    bool waited = !p.early_window;
    int chunk = 0, token = 0, n_item = 0;
    for (int item = item0; item < n_items; item += item_step, ++n_item) {
      const int t = item / groups;
      const int seq = __ldg(p.q_seq + t);
      const int32_t* cpt = p.comp_pt + static_cast<int64_t>(seq) * p.comp_pt_stride;
      const int32_t* wpt = p.win_pt + static_cast<int64_t>(seq) * p.win_pt_stride;
      const int32_t wpos = p.idx_w || p.kw == 0 ? 0 : __ldg(p.win_pos + t);
      const int cw = share_of(p.kw, crank, CS), total = cw + share_of(p.kc, crank, CS);
      int cursor = 0, head = 0, count = 0;      // positions located; ring state
      while (true) {
        // ---- locate rows until a chunk is full or the lists are done
        while (count < kRows && cursor < total) {
          if (!waited && cursor == cw) {
            if (count > 0) break;               // the window's rows go first, before idx_c is there
            griddep_wait();
            waited = true;
          }
          const int end = waited ? total : cw;
          const int pos = cursor + gt;
          uint64_t rp = 0;
          if (pos < end) {
            const bool window = pos < cw;
            const int j = share_at(window ? pos : pos - cw, crank, CS);
            int32_t e;
            if (!window) {
              e = __ldg(p.idx_c + static_cast<int64_t>(t) * p.idx_c_stride + j);
            } else if (p.idx_w) {
              e = __ldg(p.idx_w + static_cast<int64_t>(t) * p.idx_w_stride + j);
            } else {
              const int64_t pw = static_cast<int64_t>(wpos) - p.kw + 1 + j;
              e = pw < 0 ? -1 : static_cast<int32_t>(p.win_ring > 0 ? pw % p.win_ring : pw);
            }
            if (e >= 0) {
              const int64_t lim = static_cast<int64_t>(window ? p.win_pt_stride : p.comp_pt_stride) * 64;
              const int64_t np = window ? p.win_num_pages : p.comp_num_pages;
              const int32_t page = e < lim ? __ldg((window ? wpt : cpt) + (e >> 6)) : -1;
              if (page < 0 || page >= np) {
                raise_error(kErrIndex);
              } else {
                const uint8_t* base = window ? p.win_base : p.comp_base;
                const int64_t stride = window ? p.win_page_stride : p.comp_page_stride;
                rp = reinterpret_cast<uint64_t>(base + page * stride) | static_cast<uint64_t>(e & 63);
              }
            }
          }
          const uint32_t bits = __ballot_sync(0xffffffffu, rp != 0);
          const int w = static_cast<int>(warp) - 8;
          if (lane == 0) wcnt[w] = __popc(bits);
          named_barrier_sync(kBarGather4, kGatherThreads);
          int before = 0, all = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int n = wcnt[i];
            before += i < w ? n : 0;
            all += n;
          }
          if (rp != 0)
            ring[(head + count + before + __popc(bits & ((1u << lane) - 1u))) & (kRing - 1)] = rp;
          named_barrier_sync(kBarGather4, kGatherThreads);
          count += all;
          cursor = min(cursor + kGatherThreads, end);
        }
        const int n = min(count, kRows);
        if (n == 0) break;
        // ---- load: thread (row, half) takes the 16-byte code pieces 2 j + half (one
        // scale block each), four rope pieces and the scale row; rows past n are zero
        uint4 code[7], rope[4], scl;
        {
          const bool in = row < n;
          const uint64_t rp = in ? ring[(head + row) & (kRing - 1)] : 0;
          const uint8_t* page = reinterpret_cast<const uint8_t*>(rp & ~uint64_t(63));
          const int slot = static_cast<int>(rp & 63);
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          const uint4* cp = reinterpret_cast<const uint4*>(page + slot * 224) + half;
          const uint4* rpp = reinterpret_cast<const uint4*>(page + kFp4RopeOff + slot * 128) + 4 * half;
          scl = in ? __ldg(reinterpret_cast<const uint4*>(page + kFp4ScaleOff + slot * 16)) : zero;
#pragma unroll
          for (int j = 0; j < 7; ++j) code[j] = in ? __ldg(cp + 2 * j) : zero;
#pragma unroll
          for (int j = 0; j < 4; ++j) rope[j] = in ? __ldg(rpp + j) : zero;
        }
        head += n;
        count -= n;
        const uint32_t sb[4] = {scl.x, scl.y, scl.z, scl.w};
        // ---- 128 dims at a time, as the previous chunk's PV has read them
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (chunk > 0) {
            bool good = true;
            if (ok && lane == 0) good = mbar_wait(bar_free + b, (chunk - 1) & 1);
            ok = __shfl_sync(0xffffffffu, good ? 1 : 0, 0) != 0 && ok;
          }
          if (b == 0 && gt == 0) {        // the slot's last token has been read: its chunk's PV was issued
            meta[token & 1] = n;
            mbar_arrive(bar_tok + (token & 1));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int j = 2 * b + i;       // column block
            uint8_t* blk = kv + j * kKvBlock;
            if (j < 7) {
              uint4 v[4];                  // scale byte 2 j + half of the row
              widen32(code[j], e8m0_bf16x2((sb[j >> 1] >> (16 * (j & 1) + 8 * half)) & 0xFFu), v);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint4*>(blk + sw128_offset(row, static_cast<uint32_t>(4 * half + x))) = v[x];
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint4*>(blk + sw128_offset(row, static_cast<uint32_t>(4 * half + x))) = rope[x];
            }
          }
          fence_proxy_async_smem();        // the tile is read by the tensor core
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_full + b);
        }
        ++chunk;
        ++token;
      }
      // ---- the item's end; of items without rows, the end before it has been seen
      if (gt == 0) {
        if (n_item > 0 && ok) ok = mbar_wait(bar_item, (n_item - 1) & 1);
        meta[token & 1] = -1;
        mbar_arrive(bar_tok + (token & 1));
      }
      ++token;
    }
  } else if (warp == 16) {
    // =========================== MMA thread ===========================
    if (lane == 0) {
      const uint32_t idesc_s = make_idesc(kFmtBF16, kFmtBF16, 0, 0, 128, HN);
      const uint32_t idesc_o = make_idesc(kFmtBF16, kFmtBF16, 1, HN == 64 ? 1 : 0, 128, HN);
      const uint64_t kvk = smem_desc_sw128(smem_u32(kv), 16, 1024), qk = smem_desc_sw128(smem_u32(qs), 16, 1024);
      const uint64_t kvm = smem_desc_sw128(smem_u32(kv), kKvBlock, 1024);
      // P: [row][64 heads] (N contiguous) for 64 heads, else [head][64 rows] x 2
      const uint64_t pd = smem_desc_sw128(smem_u32(ps), HN == 64 ? kRows * 128 : 16, 1024);
      int chunk = 0, token = 0, n_item = 0;
      for (int item = item0; item < n_items && ok; item += item_step, ++n_item) {
        ok = mbar_wait(bar_q, n_item & 1);
        bool first = true;
        while (ok) {
          ok = mbar_wait(bar_tok + (token & 1), (token >> 1) & 1);
          if (!ok) break;
          const int n = meta[token & 1];
          ++token;
          if (n < 0) break;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            ok = ok && mbar_wait(bar_full + b, chunk & 1);
            tc_fence_after();
#pragma unroll
            for (int kk = 8 * b; kk < 8 * b + 8; ++kk) {
              const uint32_t ao = ((kk >> 2) * kKvBlock + (kk & 3) * 32) >> 4;
              const uint32_t bo = ((kk >> 2) * (HN * 128) + (kk & 3) * 32) >> 4;
              mma_f16(tmem + kColS, kvk + ao, qk + bo, idesc_s, kk > 0 ? 1u : 0u);
            }
          }
          mma_commit(bar_s);
          ok = ok && mbar_wait(bar_p, chunk & 1);
          tc_fence_after();
#pragma unroll
          for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t ao = (2 * mb * kKvBlock + kk * 2048) >> 4;
              const uint32_t bo = (HN == 64 ? kk * 2048 : (kk >> 2) * (HN * 128) + (kk & 3) * 32) >> 4;
              mma_f16(tmem + kColO + mb * HN, kvm + ao, pd + bo, idesc_o, (!first || kk > 0) ? 1u : 0u);
            }
            mma_commit(bar_free + mb);
          }
          first = false;
          ++chunk;
        }
        mma_commit(bar_o);
      }
    }
    __syncwarp();
  } else {
    // =========================== softmax warps ===========================
    const uint32_t g = warp & 3u, hh = warp >> 2;
    const int r = static_cast<int>(g * 32 + lane);          // row of the chunk, and TMEM lane
    const int hb = static_cast<int>(hh) * HW;               // first head of this thread
    const uint32_t ta = tmem + ((g * 32u) << 16);
    bool waited = !p.early_window;
    // Q of an item -> swizzled K-major tile; heads past H are zero
    auto load_q = [&](int item) {
      const int t = item / groups, h0 = (item - t * groups) * HN;
      const uint4* src = reinterpret_cast<const uint4*>(p.q) + static_cast<int64_t>(t) * p.H * 64;
#pragma unroll 4
      for (int u = tid; u < HN * 64; u += kComputeThreads) {
        const int h = u >> 6, v = u & 63;
        cp_async16(qs + (v >> 3) * (HN * 128) + sw128_offset(h, v & 7), src + static_cast<int64_t>(min(h0 + h, p.H - 1)) * 64 + v,
                   h0 + h < p.H ? 16u : 0u);
      }
    };
    auto q_ready = [&]() {
      cp_async_wait();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q);
    };
    if (item0 < n_items) {
      load_q(item0);
      q_ready();
    }
    int chunk = 0, token = 0, n_item = 0;
    bool alive = true;                                      // the same in all compute threads
    for (int item = item0; item < n_items; item += item_step, ++n_item) {
      const int t = item / groups, h0 = (item - t * groups) * HN;
      const int hreal = min(HN, p.H - h0);
      float lsum[HW];
#pragma unroll
      for (int i = 0; i < HW; ++i) lsum[i] = 0.f;
      if (tid < HN) m_used[tid] = -1e30f;
      bool have_o = false;
      while (true) {
        // ---- one thread waits for the chunk's S (or the item's end), the others at the barrier
        bool bad = false;
        if (tid == 0 && alive) {
          bad = !mbar_wait(bar_tok + (token & 1), (token >> 1) & 1);
          if (!bad && meta[token & 1] >= 0) bad = !mbar_wait(bar_s, chunk & 1);
        }
        alive = !any_of(bad, kBarCompute4, kComputeThreads) && alive;
        if (!alive) break;
        const int n = meta[token & 1];
        ++token;
        if (n < 0) break;
        tc_fence_after();
        float sv[HW];
        tmem_load_cols<HW>(ta + kColS + hb, sv);
        const bool rvalid = r < n;
        float over = -INFINITY;
#pragma unroll
        for (int i = 0; i < HW; i += 4) {
          const float4 m = *reinterpret_cast<const float4*>(m_used + hb + i);
          const float mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            sv[i + x] = rvalid ? sv[i + x] * p.scale_log2 : -INFINITY;
            over = fmaxf(over, sv[i + x] - mm[x]);
          }
        }
        if (any_of(over > kSlack, kBarCompute4, kComputeThreads)) {
          // a score passes the max in use: take the chunk's max of those heads, rescale
          float tmp[HW];
#pragma unroll
          for (int i = 0; i < HW; ++i) tmp[i] = sv[i];
          const float m = TransposeReduce<HW>::run(tmp, lane, 16u, OpMax());
          constexpr int kRep = 32 / HW;
          if ((lane & (kRep - 1)) == 0) red[(hb + lane / kRep) * 4 + g] = m;
          named_barrier_sync(kBarCompute4, kComputeThreads);
          if (tid < HN) {
            const float4 q = *reinterpret_cast<const float4*>(red + tid * 4);
            const float mc = fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)), mo = m_used[tid];
            const float mn = mc > mo + kSlack ? mc : mo;
            alpha[tid] = ex2_approx(mo - mn);
            m_used[tid] = mn;
          }
          named_barrier_sync(kBarCompute4, kComputeThreads);
          if (have_o) {                  // S being complete, so is the PV before it
#pragma unroll
            for (int i = 0; i < HW; ++i) lsum[i] *= alpha[hb + i];
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
              const uint32_t to = ta + kColO + (hh * 2 + b) * HN;
#pragma unroll 1
              for (int j0 = 0; j0 < HN; j0 += 16) {
                float v[16];
                tmem_load_cols<16>(to + j0, v);
#pragma unroll
                for (int x = 0; x < 16; ++x) v[x] *= alpha[j0 + x];
                tmem_st16(to + j0, v);
              }
            }
            tmem_st_wait();
          }
        }
        // ---- P, rounded to BF16 for PV; the sum is fp32
#pragma unroll
        for (int i = 0; i < HW; i += 8) {
          const float4 ma = *reinterpret_cast<const float4*>(m_used + hb + i);
          const float4 mb = *reinterpret_cast<const float4*>(m_used + hb + i + 4);
          const float mm[8] = {ma.x, ma.y, ma.z, ma.w, mb.x, mb.y, mb.z, mb.w};
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float a = ex2_approx(sv[i + 2 * x] - mm[2 * x]), b = ex2_approx(sv[i + 2 * x + 1] - mm[2 * x + 1]);
            lsum[i + 2 * x] += a;
            lsum[i + 2 * x + 1] += b;
            w[x] = pack_bf16x2(a, b);
          }
          if constexpr (HN == 64) {
            *reinterpret_cast<uint4*>(ps + sw128_offset(r, static_cast<uint32_t>((hb + i) >> 3))) =
                make_uint4(w[0], w[1], w[2], w[3]);
          } else {
            uint8_t* prow = ps + (r >> 6) * (HN * 128);
            const uint32_t unit = static_cast<uint32_t>((r & 63) >> 3);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              *reinterpret_cast<uint16_t*>(prow + sw128_offset(hb + i + x, unit) + (r & 7) * 2) =
                  static_cast<uint16_t>(w[x >> 1] >> (16 * (x & 1)));
          }
        }
        have_o = true;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p);
        ++chunk;
      }
      if (!alive) break;
      // ---- the item's end: its last S is complete, so Q may be replaced
      if (CS == 1 && item + item_step < n_items) load_q(item + item_step);
      // per-head sums over the rows
      {
        const float l = TransposeReduce<HW>::run(lsum, lane, 16u, OpAdd());
        constexpr int kRep = 32 / HW;
        if ((lane & (kRep - 1)) == 0) red[(hb + lane / kRep) * 4 + g] = l;
      }
      if (!waited) {                     // outputs are written after the previous kernels completed
        griddep_wait();
        waited = true;
      }
      named_barrier_sync(kBarCompute4, kComputeThreads);
      float m_mine = -1e30f, l_mine = 0.f;
      if (tid < HN) {
        const float4 q = *reinterpret_cast<const float4*>(red + tid * 4);
        m_mine = m_used[tid];
        l_mine = (q.x + q.y) + (q.z + q.w);
      }
      if (CS > 1) {
        if (tid < HN) {
#pragma unroll 1
          for (int o = 0; o < CS; ++o) {
            if (o == crank) continue;
            st_cluster_v2f32(cluster_map(smem_u32(mlr + crank * HN + tid), static_cast<uint32_t>(o)), m_mine, l_mine);
            mbar_arrive_remote(cluster_map(smem_u32(bar_ml), static_cast<uint32_t>(o)));
          }
          ok = mbar_wait(bar_ml, 0) && ok;
        }
      }
      if (tid < HN) {
        const float sink2 = tid < hreal ? __ldg(p.sink + h0 + tid) * kLog2e : -INFINITY;
        auto ml_of = [&](int c) { return c == crank ? make_float2(m_mine, l_mine) : mlr[c * HN + tid]; };
        float M = sink2;
        for (int c = 0; c < CS; ++c) {
          const float2 ml = ml_of(c);
          if (!(ml.y == 0.f)) M = fmaxf(M, ml.x);
        }
        float L = sink2 > -INFINITY ? exp2f(sink2 - M) : 0.f;   // a sink of -inf adds nothing
        for (int c = 0; c < CS; ++c) {
          const float2 ml = ml_of(c);
          if (!(ml.y == 0.f)) L += ml.y * exp2f(ml.x - M);
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;             // an empty denominator gives zeros
        for (int c = 0; c < CS; ++c) {
          const float2 ml = ml_of(c);
          fac[c * HN + tid] = ml.y == 0.f ? 0.f : exp2f(ml.x - M) * inv;
        }
        if (p.lse && crank == 0 && tid < hreal)
          p.lse[static_cast<int64_t>(t) * p.H + h0 + tid] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      }
      bool bad = false;
      if (tid == 0) bad = !mbar_wait(bar_o, n_item & 1);
      alive = !any_of(bad, kBarCompute4, kComputeThreads);      // also publishes the factors
      tc_fence_after();
      if (!alive) break;
      if (tid == 0) mbar_arrive(bar_item);                      // the MMA thread has read the end's token, too
      if (CS == 1 && item + item_step < n_items) q_ready();
      if (CS > 1) break;                 // merged below, by all warps of the cluster
      // ---- output: thread = dim, lanes (d, d + 1) pair up to store two values of a head
      const float4* rrow = rope_row(p, t);
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        const int blk = static_cast<int>(hh) * 2 + b;
        const int d = blk * 128 + r;
        uint16_t* orow = p.out + (static_cast<int64_t>(t) * p.H + h0) * 512 + (d & ~1);
        const bool rot = rrow != nullptr && d >= 512 - 64;      // warp-uniform
        const float2 cs = rot ? __ldg(reinterpret_cast<const float2*>(rrow) + ((d - (512 - 64)) >> 1)) : make_float2(1.f, 0.f);
#pragma unroll 1
        for (int j0 = 0; j0 < HN; j0 += 16) {
          float v[16];
          if (have_o) {
            tmem_load_cols<16>(ta + kColO + blk * HN + j0, v);
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) v[x] = 0.f;
          }
#pragma unroll
          for (int x = 0; x < 16; x += 2) {
            float a = v[x] * fac[j0 + x], c = v[x + 1] * fac[j0 + x + 1];
            // even lanes take head x, odd lanes head x + 1, of both dims
            const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? a : c, 1);
            float lo = (lane & 1) ? got : a, hi = (lane & 1) ? c : got;
            if (rot) {
              const float2 z = rotate_back(lo, hi, cs.x, cs.y);
              lo = z.x;
              hi = z.y;
            }
            const int h = j0 + x + static_cast<int>(lane & 1);
            if (h < hreal) *reinterpret_cast<uint32_t*>(orow + static_cast<int64_t>(h) * 512) = pack_bf16x2(lo, hi);
          }
        }
      }
      tc_fence_before();                 // O has been read; the next item's PV follows its bar_p
      named_barrier_sync(kBarCompute4, kComputeThreads);        // m_used, red and fac are free again
    }
    ok = ok && alive;
  }

  if (CS > 1) {
    // =========================== cluster merge ===========================
    // Receive slots of the other CS - 1 splits at [0, R), this CTA's outgoing ones
    // at [R, 2 R), R = (CS - 1) slot_bytes, inside the idle tiles.  A slot is
    // [dim][HN] fp32; its 16-byte units are permuted within 128 bytes by the dim, so
    // that the lanes of a warp (neighbouring dims) hit every bank.
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_arrive();                    // this CTA's tiles are idle: the other CTAs may copy into them
    const int R = (CS - 1) * slot_bytes;
    const int t = item0 / groups, h0 = (item0 - t * groups) * HN;
    const int hreal = min(HN, p.H - h0);
    const uint32_t g = warp & 3u, hh = warp >> 2;
    const uint32_t ta = tmem + ((g * 32u) << 16);
    auto unit_at = [](uint8_t* slot, int dl, int u) {
      const int s = HN >= 32 ? (u ^ (dl & 7)) : (u ^ ((dl >> 1) & 3));
      return reinterpret_cast<float4*>(slot + dl * (HN * 4)) + s;
    };
    const bool compute = warp < 8;
    // fac is zero where this split attended to nothing; its O may then hold anything
    if (compute) {
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        const int blk = static_cast<int>(hh) * 2 + b;
        const int d = blk * 128 + static_cast<int>(g * 32 + lane);
        const int owner = d / slice;     // warp-uniform: a slice is at least 64 aligned dims
        if (owner == crank) continue;
        uint8_t* slot = smem + R + (owner < crank ? owner : owner - 1) * slot_bytes;
#pragma unroll 1
        for (int j0 = 0; j0 < HN; j0 += 16) {
          float v[16];
          tmem_load_cols<16>(ta + kColO + blk * HN + j0, v);
#pragma unroll
          for (int x = 0; x < 16; x += 4)
            *unit_at(slot, d - owner * slice, (j0 + x) / 4) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
        }
      }
    }
    fence_proxy_async_smem();            // the staged slots are read by the bulk-copy engine
    __syncthreads();
    cluster_wait();                      // every CTA's tiles are idle
    if (tid == 0) {
      for (int o = 0; o < CS; ++o) {
        if (o == crank) continue;
        const int at = crank < o ? crank : crank - 1;
        bulk_copy_to_cluster(cluster_map(smem_u32(smem + at * slot_bytes), static_cast<uint32_t>(o)),
                             smem + R + (o < crank ? o : o - 1) * slot_bytes, static_cast<uint32_t>(slot_bytes),
                             cluster_map(smem_u32(bar_recv), static_cast<uint32_t>(o)));
      }
    }
    ok = mbar_wait(bar_recv, 0) && ok;   // the other splits' slots have landed here
    cluster_arrive();                    // ... so their copies out of the senders are complete
    if (compute) {
      const float4* rrow = rope_row(p, t);
#pragma unroll 1
      for (int blk = crank * slice / 128; blk < (crank * slice + slice + 127) / 128; ++blk) {
        const int d = blk * 128 + static_cast<int>(g * 32 + lane), dl = d - crank * slice;
        if (d / slice != crank) continue;                       // warp-uniform (half a block when slice is 64)
        uint16_t* orow = p.out + (static_cast<int64_t>(t) * p.H + h0) * 512 + (d & ~1);
        const bool rot = rrow != nullptr && d >= 512 - 64;
        const float2 cs = rot ? __ldg(reinterpret_cast<const float2*>(rrow) + ((d - (512 - 64)) >> 1)) : make_float2(1.f, 0.f);
#pragma unroll 1
        for (int j0 = static_cast<int>(hh) * HW; j0 < (static_cast<int>(hh) + 1) * HW; j0 += 8) {
          float v[8];
          tmem_load_cols<8>(ta + kColO + blk * HN + j0, v);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float f = fac[crank * HN + j0 + x];
            v[x] = f == 0.f ? 0.f : v[x] * f;
          }
#pragma unroll 1
          for (int c = 0; c < CS; ++c) {
            if (c == crank) continue;
            uint8_t* slot = smem + (c < crank ? c : c - 1) * slot_bytes;
#pragma unroll
            for (int x = 0; x < 8; x += 4) {
              const float4 u = *unit_at(slot, dl, (j0 + x) / 4);
              const float4 f = *reinterpret_cast<const float4*>(fac + c * HN + j0 + x);
              if (f.x != 0.f) v[x] = fmaf(u.x, f.x, v[x]);
              if (f.y != 0.f) v[x + 1] = fmaf(u.y, f.y, v[x + 1]);
              if (f.z != 0.f) v[x + 2] = fmaf(u.z, f.z, v[x + 2]);
              if (f.w != 0.f) v[x + 3] = fmaf(u.w, f.w, v[x + 3]);
            }
          }
#pragma unroll
          for (int x = 0; x < 8; x += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v[x] : v[x + 1], 1);
            float lo = (lane & 1) ? got : v[x], hi = (lane & 1) ? v[x + 1] : got;
            if (rot) {
              const float2 z = rotate_back(lo, hi, cs.x, cs.y);
              lo = z.x;
              hi = z.y;
            }
            const int h = j0 + x + static_cast<int>(lane & 1);
            if (h < hreal && ok) *reinterpret_cast<uint32_t*>(orow + static_cast<int64_t>(h) * 512) = pack_bf16x2(lo, hi);
          }
        }
      }
    }
    cluster_wait();                      // no copy reads this CTA's staging any more
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int HN>
int launch_hn4(const AttnParams& p, int groups, int sms, cudaStream_t stream) {
  constexpr int bytes = Smem4<HN>::kBytes + 1024;   // + alignment slack
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
  if (p.nsplit > 1 && 2 * (p.nsplit - 1) * (512 / p.nsplit) * HN * 4 > Smem4<HN>::kTiles) return DSV4SA_ERR_UNSUPPORTED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  if (!smem_attr_once(dev, 5 + HN / 32, reinterpret_cast<const void*>(sparse_attn_fp4_kernel<HN>), bytes))
    return DSV4SA_ERR_CUDA;
  const int64_t items = static_cast<int64_t>(p.T) * groups;
  if (items * p.nsplit > INT32_MAX) return DSV4SA_ERR_UNSUPPORTED;
  cudaError_t e;
  if (p.nsplit == 1) {
    e = launch_pdl(sparse_attn_fp4_kernel<HN>, dim3(static_cast<unsigned>(items < sms ? items : sms)), dim3(kThreads4),
                   bytes, stream, p, groups);
  } else {
    e = launch_cluster_pdl(sparse_attn_fp4_kernel<HN>, dim3(static_cast<unsigned>(items * p.nsplit)), dim3(kThreads4),
                           bytes, p.nsplit, stream, p, groups);
  }
  return e == cudaSuccess ? DSV4SA_OK : DSV4SA_ERR_CUDA;
}

}  // namespace

namespace attn {

int launch_fp4(int32_t mode, AttnParams& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  int hn = p.H <= 16 ? 16 : (p.H <= 32 ? 32 : 64);
  int groups = (p.H + hn - 1) / hn;
  p.nsplit = 1;
  const int rows = p.kc + p.kw;
  if (mode == DSV4SA_ATTN_DECODE && rows > kRows) {
    const int64_t items = static_cast<int64_t>(p.T) * groups;
    const int most = hn == 64 ? 4 : 8;   // the merge's slots of 64 heads fit in the tiles up to 4 splits
    while (p.nsplit < most && items * p.nsplit * 2 <= sms) p.nsplit *= 2;
  }
  switch (hn) {
    case 16: return launch_hn4<16>(p, groups, sms, stream);
    case 32: return launch_hn4<32>(p, groups, sms, stream);
    default: return launch_hn4<64>(p, groups, sms, stream);
  }
}

}  // namespace attn

uint32_t read_error_word_attn_fp4(cudaStream_t stream, bool clear) {
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
