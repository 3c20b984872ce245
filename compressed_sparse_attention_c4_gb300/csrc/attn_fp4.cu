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
// 32 list positions, and merge at the end.  plan4 below chooses HN and CS.
//
// Pipeline of a CTA.  The valid rows of the lists are packed -- J is a multiset,
// their order is free -- into chunks of 128, so -1 entries cost no tensor work (the window's
// into chunks of their own where full lists make no more chunks so, see window_apart):
//   gather warps (16): index -> page id -> row, 256 positions at a time, the valid
//     ones appended to a ring; a chunk's rows (four threads a row) are loaded into
//     registers while the chunk before is worked on, then widened to BF16 and
//     stored in the 128 x 512 tile (128-byte swizzle) when its PV has read it.  The
//     nope dims lie in the tile in the order that costs least to widen (dim_of), and
//     so do Q's and O's.
//   MMA warp: S^T = KV . Q^T (M = 128 rows, N = HN, K = 512), then O^T += V^T . P^T
//     (M = 128 dims x 4, N = HN, K = 128): the tile is read K-major for S and
//     MN-major for PV.
//   Q warps (3): the next item's Q, once the last S of this one is complete.
//   softmax warps (8): thread = row, half of the heads.  P is BF16 against a max
//     that is only moved (and O rescaled) when a score passes it by 2^8: a vote
//     replaces the max's reduction in nearly every chunk but the first.  The sum
//     of the probabilities stays with its row's thread until the end.  At an
//     item's end these warps write the output while the next item's first chunk
//     is gathered and scored.
// What bounds it.  64 heads: shared memory and the hand-overs.  An MMA of M = 128, N = 64,
// K = 16 reads 6 KB and takes 48 cycles, the 128 bytes a clock of shared memory
// (measured), so while MMAs run other accesses hardly proceed, and the phases of a
// chunk (about 3000 cycles of MMAs, 1000 of stores, the widening's 7168 words of eight codes)
// follow one another: 4096 queries of 640 rows take 582 us, 590 TFLOP/s.  The tile is
// handed over in two halves of its dims: as a whole that call took 687 us, by quarters
// 629, by halves 617 then (a wait drains the tensor pipe).  Two tiles of 64 rows in turn, a
// group of gather warps for each, took 726 against 610: each step from one kind of warp to
// the next costs 400 to 1600 cycles whatever the tile's size.  16 heads: the widening (2.8 us
// a chunk).  One query: the chain of latencies -- lists, page ids, rows, S, softmax, PV, merge.
// Widening is exact (fp4.cuh).  P is the one operand rounded (BF16, 2^-8 of a
// probability at most); S, O, maxima, sums and the partial results that a cluster
// exchanges are fp32.
#include <atomic>

#include "attn_common.cuh"
#include "attn_pipe.cuh"
#include "fp4.cuh"

namespace dsv4sa {
namespace {

using namespace attn;

constexpr int kComputeThreads = 256;     // warps 0-7: softmax, output
constexpr int kGatherThreads = 512;      // warps 8-23
constexpr int kMmaWarp = 24;
constexpr int kThreads4 = kComputeThreads + kGatherThreads + 128;   // the last warpgroup: the MMA warp, then
constexpr int kQThreads = 96;            // its other three warps fetch Q
constexpr int kLocate = 256;             // list positions looked up at a time
constexpr int kRing = 512;               // located rows waiting for a chunk (fewer than 128 + 256)
constexpr int kRun = 32;                 // list positions a CTA of a cluster takes in a row
constexpr int kFp4RopeOff = 14336;       // KV_FP4 page layout (see dsv4sa.h)
constexpr int kFp4ScaleOff = 22528;
constexpr float kSlack = 8.f;            // log2 units a score may pass the max in use by
constexpr int kHalf = 4 * kKvBlock;      // bytes of a half of the tile: 128 rows x 256 dims
constexpr int kLastChunk = 256;          // meta: rows of the chunk (<= 128), and this for an item's last
// Registers per thread (setmaxnreg): the launch gives 896 x 72 = 64512, the three
// kinds of warpgroup then hold 256 x 96 + 512 x 64 + 128 x 56 = 64512, or, for 64 heads,
// whose softmax threads have 32 scores and sums each, 256 x 120 + 512 x 56 + 128 x 40 (4096
// queries of 64 heads, in a graph: 582 us, with 112, 56 and 56 582, with the first shares 599;
// 1024 with a window of 60 rows 153.3, 154.4, 158.8).  With 112, 56 and 56 the smaller items
// take as long (128 ragged queries of 8 heads 31.6 us and 31.5).  The 64-head kernel spills a
// little by the compiler's count, 44 bytes stored and 40 loaded.
template <int HN>
struct Regs4 {
  static constexpr int kCompute = HN == 64 ? 120 : 96, kGather = HN == 64 ? 56 : 64, kMma = HN == 64 ? 40 : 56;
  static_assert(kComputeThreads * kCompute + kGatherThreads * kGather + 128 * kMma <= kThreads4 * 72,
                "the register shares fit in the launch's");
};

constexpr uint32_t kBarCompute4 = 1;     // named barriers
constexpr uint32_t kBarGather4 = 2;

template <int HN>
struct Smem4 {
  // Halves of tiles.  (With 16 heads a third one fits, so that the next chunk is widened
  // while this one is scored: 128 queries of 8 heads, up to 1152 rows, 31.2 us for 32.1 in
  // a graph of such calls then, but 37.2 for 33.3 launched one by one.)
  static constexpr int kSlots = 2;
  static constexpr int kStage = HN == 16 ? 8 : 16;       // heads of an output step
  static constexpr int kKv = 0;
  static constexpr int kQ = kSlots * kHalf;              // 8 column blocks x HN rows x 128 B
  static constexpr int kP = kQ + 8 * HN * 128;           // 128 rows x 128 B, or 2 blocks x HN rows x 128 B; output staging
  static constexpr int kTiles = kP + kStage * 1024;      // end of the tiles (the merge may use all of them)
  static constexpr int kRing_ = kTiles;                  // uint64 [kRing]
  static constexpr int kRed = kRing_ + kRing * 8;        // float [HN][4]
  static constexpr int kM = kRed + HN * 16;              // float [HN] each
  static constexpr int kAlpha = kM + HN * 4;
  static constexpr int kFac = kAlpha + HN * 4;           // float [kMaxClusterSplits][HN]
  static constexpr int kMl = kFac + kMaxClusterSplits * HN * 4;   // float2 [kMaxClusterSplits][HN]
  static constexpr int kCnt = kMl + kMaxClusterSplits * HN * 8;   // int [16]
  static constexpr int kMeta = kCnt + 64;                // int [4]
  static constexpr int kBar = kMeta + 16;                // barriers, see below
  static constexpr int kTmem = kBar + (2 * kSlots + 13) * 8;
  static constexpr int kBytes = kTmem + 16;
};

// Store two floats into another CTA's shared memory, counted as 8 bytes on a barrier
// there.  (A plain store with a releasing remote arrival each took 0.7 us apiece, one
// after the other: 4.7 us for the (m, l) of a cluster of four, 6.4 of eight.)
__device__ __forceinline__ void st_async_v2f32(uint32_t addr, float a, float b, uint32_t mbar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr), "f"(a),
               "f"(b), "r"(mbar)
               : "memory");
}

// Where the tile's column `d` belongs: the nope part is widened in the order 0, 4, 1, 5, 2,
// 6, 3, 7 within eight dims (fp4.cuh), Q is put into that order, too, and O comes out in it.
__device__ __forceinline__ int dim_of(int d) {
  return d < DSV4SA_NOPE_DIM ? (d & ~7) | ((d & 7) >> 1) | ((d & 1) << 2) : d;
}

// Positions of a list of n that CTA r of CS takes, and the k-th of them.
__host__ __device__ __forceinline__ int share_of(int n, int r, int CS) {
  const int whole = n / (kRun * CS), rest = n - whole * kRun * CS - r * kRun;
  return whole * kRun + min(max(rest, 0), kRun);
}
// Whether the window's rows get chunks of their own: where full lists make no more chunks so.
// Sizes alone decide, so a call that may work on the window before the compressed indices are
// there (EARLY_WINDOW) forms the same chunks, and the same sums, as one that may not.
__device__ __forceinline__ bool window_apart(int cw, int cc) {
  return (cw + kRows - 1) / kRows + (cc + kRows - 1) / kRows == (cw + cc + kRows - 1) / kRows;
}
__device__ __forceinline__ int share_at(int k, int r, int CS) { return ((k / kRun) * CS + r) * kRun + k % kRun; }

template <int HN>
__global__ void __launch_bounds__(kThreads4, 1) sparse_attn_fp4_kernel(const AttnParams p, int groups) {
  using S = Smem4<HN>;
  // 128-byte swizzled tiles need 1024-byte aligned bases.  An offset from the array (not
  // a rounded address) lets the compiler see shared memory: 32-bit addresses, no
  // generic loads.
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
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
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + S::kBar);   // [slots]: half of a chunk's dims is in place
  uint64_t* bar_free = bar_full + S::kSlots; // [slots]: ... has been read by PV
  uint64_t* bar_tok = bar_free + S::kSlots;  // [4]: a chunk's (or an item's end's) meta is written
  uint64_t* bar_s = bar_tok + 4;         // S is complete
  uint64_t* bar_p = bar_s + 1;           // P is written
  uint64_t* bar_o = bar_s + 2;           // every PV of the item is complete
  uint64_t* bar_q = bar_s + 3;           // the item's Q has been copied
  uint64_t* bar_item = bar_s + 4;        // the end of the item has been seen
  uint64_t* bar_recv = bar_s + 5;        // merge: the other splits' partials landed
  uint64_t* bar_ml = bar_s + 6;          // merge: the other splits' (m, l) landed
  uint64_t* bar_q0 = bar_s + 7;          // the first item's Q is in order
  uint64_t* bar_qfree = bar_s + 8;       // every S of the item is complete
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
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(bar_full + i, kGatherThreads / 32);
      mbar_init(bar_free + i, 1);
    }
    mbar_init(bar_s, 1);
    mbar_init(bar_p, kComputeThreads / 32);
    for (int i = 0; i < 4; ++i) mbar_init(bar_tok + i, 1);
    mbar_init(bar_o, 1);
    mbar_init(bar_q, kQThreads / 32);
    mbar_init(bar_item, 1);
    mbar_init(bar_recv, 1);
    mbar_init(bar_ml, 1);
    mbar_init(bar_q0, kComputeThreads / 32);
    mbar_init(bar_qfree, 1);
    fence_mbar_init();
    if (CS > 1) {
      mbar_arrive_expect_tx(bar_recv, static_cast<uint32_t>((CS - 1) * slot_bytes));
      mbar_arrive_expect_tx(bar_ml, static_cast<uint32_t>((CS - 1) * HN * 8));
    }
  }
  if (warp == kMmaWarp) {
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
  if (CS > 1) cluster_arrive();          // this CTA's barriers are initialised; waited for before anything remote
  const uint32_t tmem = *tmem_holder;
  bool ok = true;                        // no wait of this thread has run out

  // Q's nope part into the order of the tile's columns, when it has arrived: the first
  // item's by the softmax warps, idle then, the others' by the gather warps.  (By the three
  // warps that copy it, it delayed the first S: decode of 32 x 640 rows 22.3 us, 4096 x 640
  // 630 us; here 20.9 and 606.)
  auto order_q = [&](int n_item, int first, int step) {
    const bool there = warp_wait(bar_q, n_item & 1);
#pragma unroll 1
    for (int u = first; u < HN * (DSV4SA_NOPE_DIM / 8); u += step) {
      const int h = u / (DSV4SA_NOPE_DIM / 8), v = u - h * (DSV4SA_NOPE_DIM / 8);
      uint4* at = reinterpret_cast<uint4*>(qs + (v >> 3) * (HN * 128) + sw128_offset(h, v & 7));
      const uint4 x = *at;
      *at = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                       __byte_perm(x.y, x.w, 0x7632));
    }
    fence_proxy_async_smem();
    __syncwarp();
    return there;
  };

  if (warp >= 8 && warp < kMmaWarp) {
    // =========================== gather warps ===========================
    // A wait that runs out is not repeated: the loop, whose length the lists
    // alone decide, goes on without waiting.
    regs_dec<Regs4<HN>::kGather>();
    const int gt = tid - kComputeThreads;
    const int row = gt >> 2, piece = gt & 3;
    bool waited = !p.early_window;
    int slot = 0, token = 0;                    // the next half's
    uint32_t round = 0;                         // how often all slots have been filled
    int head = 0;                               // ring: first located row not yet loaded
    const int cw = share_of(p.kw, crank, CS), total = cw + share_of(p.kc, crank, CS);   // this CTA's positions of an item
    const int cw_apart = window_apart(cw, total - cw) ? cw : 0;   // the window's, if it gets chunks of its own
    for (int item = item0, n_item = 0; item < n_items; item += item_step, ++n_item) {
      const int t = item / groups;
      int cursor = 0;                           // positions looked up
      int count = 0;                            // rows in the ring; 2^16 up, those of a window that gets chunks of its own
      bool q_ordered = false;
      // look up the next positions, one a thread of half of them
      auto locate = [&]() {
        const int end = min(cursor + kLocate, waited ? total : cw);
        const int pos = cursor + gt;
        uint64_t rp = 0;
        if (gt < kLocate && pos < end) {
          const bool window = pos < cw;
          const int j = share_at(window ? pos : pos - cw, crank, CS);
          int32_t e;
          const int seq = __ldg(p.q_seq + t);   // in flight together with the entry
          if (!window) {
            e = __ldg(p.idx_c + static_cast<int64_t>(t) * p.idx_c_stride + j);
          } else if (p.idx_w) {
            e = __ldg(p.idx_w + static_cast<int64_t>(t) * p.idx_w_stride + j);
          } else {
            const int64_t pw = static_cast<int64_t>(__ldg(p.win_pos + t)) - p.kw + 1 + j;
            e = pw < 0 ? -1 : static_cast<int32_t>(p.win_ring > 0 ? pw % p.win_ring : pw);
          }
          if (e >= 0) {
            const int stride = window ? p.win_pt_stride : p.comp_pt_stride;
            const int32_t* pt = (window ? p.win_pt : p.comp_pt) + static_cast<int64_t>(seq) * stride;
            const int64_t np = window ? p.win_num_pages : p.comp_num_pages;
            const int32_t page = (e >> 6) < stride ? __ldg(pt + (e >> 6)) : -1;
            if (page < 0 || page >= np) {
              raise_error(kErrIndex);
            } else {
              const uint8_t* base = window ? p.win_base : p.comp_base;
              rp = reinterpret_cast<uint64_t>(base + page * (window ? p.win_page_stride : p.comp_page_stride)) |
                   static_cast<uint64_t>(e & 63);
            }
          }
        }
        const uint32_t bits = __ballot_sync(0xffffffffu, rp != 0);
        const int w = static_cast<int>(warp) - 8;
        const uint32_t own_bits = __ballot_sync(0xffffffffu, rp != 0 && pos < cw_apart);
        if (lane == 0) wcnt[w] = __popc(bits) | __popc(own_bits) << 16;
        named_barrier_sync(kBarGather4, kGatherThreads);
        int before = 0, all = 0;
#pragma unroll
        for (int i = 0; i < kLocate / 32; ++i) {
          const int n = wcnt[i];
          before += i < w ? n : 0;
          all += n;
        }
        if (rp != 0) ring[(head + ((count + before) & 0xFFFF) + __popc(bits & ((1u << lane) - 1u))) & (kRing - 1)] = rp;
        named_barrier_sync(kBarGather4, kGatherThreads);
        count += all;
        cursor = end;
      };
      // ---- a chunk's rows in registers: the four threads of a row take its 16-byte code pieces
      // 4 b + piece (a scale block each) of the first three quarters, 8 bytes of codes and 32
      // of rope values of the last; rows past the chunk's are zero
      uint4 code[3], rope[2], scl;
      uint2 code3;
      const uint8_t* page = nullptr;
      int rs = -1;                              // the row's slot in its page, -1: none
      auto take = [&](int n) {                  // the next n rows of the ring
        const uint64_t rp = row < n ? ring[(head + row) & (kRing - 1)] : 0;
        page = reinterpret_cast<const uint8_t*>(rp & ~uint64_t(63));
        rs = row < n ? static_cast<int>(rp & 63) : -1;
        head += n;
        count -= count >= 0x10000 ? n << 16 | n : n;   // the window's come first
      };
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      auto load_scales = [&]() { return rs >= 0 ? __ldg(reinterpret_cast<const uint4*>(page + kFp4ScaleOff + rs * 16)) : zero; };
      auto load_quarter = [&](int b) {
        const uint8_t* cp = page + rs * 224;
        if (b < 3) {
          code[b] = rs >= 0 ? __ldg(reinterpret_cast<const uint4*>(cp) + 4 * b + piece) : zero;
        } else {
          const uint4* rpp = reinterpret_cast<const uint4*>(page + kFp4RopeOff + rs * 128) + 2 * piece;
          code3 = rs >= 0 ? __ldg(reinterpret_cast<const uint2*>(cp + 192) + piece) : make_uint2(0u, 0u);
          rope[0] = rs >= 0 ? __ldg(rpp) : zero;
          rope[1] = rs >= 0 ? __ldg(rpp + 1) : zero;
        }
      };
      while (true) {
        // ---- enough rows for a chunk, or the end of the lists
        while ((count & 0xFFFF) < kRows && cursor < total) {
          if (cursor >= cw) {
            if (count >= 0x10000) break;        // the window's rows go first, before idx_c is there
            if (!waited) griddep_wait();
            waited = true;
          }
          locate();
        }
        const int n = min(count >= 0x10000 ? count >> 16 : count, kRows);
        if (n == 0) break;
        take(n);
        scl = load_scales();
#pragma unroll
        for (int b = 0; b < 4; ++b) load_quarter(b);
        // ---- look ahead while the loads are in flight
        if ((count & 0xFFFF) < kRows && cursor < total && (waited || cursor < cw)) locate();
        // no row of the item is left to come: the softmax may replace Q once this chunk's S is complete
        const bool last = count == 0 && cursor >= total;
        // ---- into the tile, half by half, when the half that was there has been read by its PV
        // the four bytes of the scales that this thread's pieces need
        const uint32_t sb = __byte_perm(__byte_perm(scl.x, scl.y, piece * 0x11 + 0x40),
                                        __byte_perm(scl.z, scl.w, piece + ((piece >> 1) + 4) * 0x10), 0x5410);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if ((b & 1) == 0 && round > 0 && ok) ok = warp_wait(bar_free + slot, (round - 1) & 1);
          uint8_t* half = kv + slot * kHalf;
          if (b < 3) {
            // 32 values: units 4 (piece & 1) + x of column block 2 b + (piece >> 1).  The
            // upper two pieces take x in the order 2, 3, 0, 1, so that the eight lanes of
            // two rows hit eight different bank groups.  (Eight lanes with eight rows of the
            // same piece would, too, but load eight half-used sectors: 644 us for 578 then.)
            const BlockScale bs = block_scale((sb >> (8 * b)) & 0xFFu);
            uint8_t* blk = half + (2 * (b & 1) + (piece >> 1)) * kKvBlock;
            const uint32_t c4[4] = {code[b].x, code[b].y, code[b].z, code[b].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w = piece >= 2 ? c4[i ^ 2] : c4[i];
              const uint32_t x = static_cast<uint32_t>(i) ^ (piece & 2);
              uint4 v = widen8_split(w, bs.first);
              if (bs.more) v = scale_up(v, bs.more);
              *reinterpret_cast<uint4*>(blk + sw128_offset(row, static_cast<uint32_t>(4 * (piece & 1)) + x)) = v;
            }
          } else {
            const BlockScale bs = block_scale(sb >> 24);
            const uint32_t u = static_cast<uint32_t>(2 * piece);
            uint4 v0 = widen8_split(code3.x, bs.first), v1 = widen8_split(code3.y, bs.first);
            if (bs.more) {
              v0 = scale_up(v0, bs.more);
              v1 = scale_up(v1, bs.more);
            }
            *reinterpret_cast<uint4*>(half + 2 * kKvBlock + sw128_offset(row, u)) = v0;
            *reinterpret_cast<uint4*>(half + 2 * kKvBlock + sw128_offset(row, u + 1)) = v1;
            *reinterpret_cast<uint4*>(half + 3 * kKvBlock + sw128_offset(row, u)) = rope[0];
            *reinterpret_cast<uint4*>(half + 3 * kKvBlock + sw128_offset(row, u + 1)) = rope[1];
          }
          if ((b & 1) == 1) {
            if (!q_ordered && n_item > 0 && ok) ok = order_q(n_item, gt, kGatherThreads);   // Q comes once the last S is complete
            q_ordered = true;
            fence_proxy_async_smem();      // the tile is read by the tensor core
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_full + slot);
            slot = slot + 1 == S::kSlots ? 0 : slot + 1;
            round += slot == 0 ? 1u : 0u;
          }
          if (b == 0 && gt == 0) {         // the meta slot's last token, four ago, has been read
            meta[token & 3] = n | (last ? kLastChunk : 0);
            mbar_arrive(bar_tok + (token & 3));
          }
        }
        __syncwarp();
        ++token;
      }
      if (!q_ordered) {                         // an item without rows: its phase of the barrier passes, too,
        ok = ok && warp_wait(bar_q, n_item & 1);
        named_barrier_sync(kBarGather4, kGatherThreads);   // ... for every warp before the next Q may come
      }
      // ---- the item's end, once the end before it has been seen
      if (gt == 0) {
        if (n_item > 0 && ok) ok = bar_wait(bar_item, (n_item - 1) & 1);
        meta[token & 3] = -1;
        mbar_arrive(bar_tok + (token & 3));
      }
      __syncwarp();
      ++token;
    }
    if (CS > 1) {
      ok = ok && warp_wait(bar_o, 0);    // the MMAs no longer read the tiles
      tc_fence_after();
      cluster_wait();
      cluster_arrive();
    }
  } else if (warp >= kMmaWarp) {
    // =========================== MMA warp ===========================
    regs_dec<Regs4<HN>::kMma>();
    if (warp == kMmaWarp) {
      const uint32_t idesc_s = make_idesc(kFmtBF16, kFmtBF16, 0, 0, 128, HN);
      const uint32_t idesc_o = make_idesc(kFmtBF16, kFmtBF16, 1, HN == 64 ? 1 : 0, 128, HN);
      const uint32_t hi = static_cast<uint32_t>(smem_desc_sw128(0, 16, 1024) >> 32);   // stride, version, swizzle
      const uint32_t kvk = static_cast<uint32_t>(smem_desc_sw128(smem_u32(kv), 16, 1024));
      const uint32_t qk = static_cast<uint32_t>(smem_desc_sw128(smem_u32(qs), 16, 1024));
      const uint32_t kvm = static_cast<uint32_t>(smem_desc_sw128(smem_u32(kv), kKvBlock, 1024));
      // P: [row][64 heads] (N contiguous) for 64 heads, else [head][64 rows] x 2
      const uint32_t pd = static_cast<uint32_t>(smem_desc_sw128(smem_u32(ps), HN == 64 ? kRows * 128 : 16, 1024));
      int chunk = 0, token = 0, n_item = 0;
      int slot = 0;
      uint32_t round = 0;
      for (int item = item0; item < n_items && ok; item += item_step, ++n_item) {
        if (n_item == 0) ok = warp_wait(bar_q0, 0);   // a later item's Q is in order when its tile is
        bool first = true, q_freed = false;
        while (ok) {
          ok = warp_wait(bar_tok + (token & 3), (token >> 2) & 1);
          if (!ok) break;
          const int word = meta[token & 3];
          ++token;
          if (word < 0) break;
          int at[2];                       // the chunk's halves
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && warp_wait(bar_full + slot, round & 1);
            tc_fence_after();
            at[h] = slot * kHalf;
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {  // not unrolled: the descriptors would not fit in registers
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_f16_elect(tmem + kColS, kvk + ((at[h] + b * kKvBlock + kk * 32) >> 4), qk + (((4 * h + b) * HN * 128 + kk * 32) >> 4),
                              hi, idesc_s, h > 0 || b > 0 || kk > 0 ? 1u : 0u);
            }
            slot = slot + 1 == S::kSlots ? 0 : slot + 1;
            round += slot == 0 ? 1u : 0u;
          }
          mma_commit_elect(bar_s);
          if ((word & kLastChunk) != 0) {
            mma_commit_elect(bar_qfree);
            q_freed = true;
          }
          ok = ok && warp_wait(bar_p, chunk & 1);
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll 1
            for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint32_t bo = (HN == 64 ? kk * 2048 : (kk >> 2) * (HN * 128) + (kk & 3) * 32) >> 4;
                mma_f16_elect(tmem + kColO + (2 * h + mb) * HN, kvm + ((at[h] + 2 * mb * kKvBlock + kk * 2048) >> 4), pd + bo, hi,
                              idesc_o, (!first || kk > 0) ? 1u : 0u);
              }
            }
            mma_commit_elect(bar_free + at[h] / kHalf);
          }
          first = false;
          ++chunk;
        }
        if (!q_freed) mma_commit_elect(bar_qfree);
        mma_commit_elect(bar_o);
      }
    } else {
      // ---- the warpgroup's other three warps fetch Q: the next item's, as soon as an
      // item's last S is complete (it is brought into L2 when the item begins).
      // Swizzled K-major tile; heads past the item's are zero.
      const int qt = tid - (kMmaWarp + 1) * 32;
      auto load_q = [&](int item) {
        const int t = item / groups, h0 = (item - t * groups) * HN;
        const int hreal = min(HN, p.H - h0);
        const uint4* src = reinterpret_cast<const uint4*>(p.q) + (static_cast<int64_t>(t) * p.H + h0) * 64;
#pragma unroll 4
        for (int u = qt; u < HN * 64; u += kQThreads) {
          const int h = u >> 6, v = u & 63;
          cp_async16(qs + (v >> 3) * (HN * 128) + sw128_offset(h, v & 7), src + min(h, hreal - 1) * 64 + v, h < hreal ? 16u : 0u);
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
      for (int item = item0, n_item = 0; item + item_step < n_items && ok; item += item_step, ++n_item) {
        const int next = item + item_step;
        if (qt == 0) {
          const int t = next / groups, h0 = (next - t * groups) * HN;
          prefetch_l2(p.q + (static_cast<int64_t>(t) * p.H + h0) * 512, static_cast<uint32_t>(min(HN, p.H - h0)) * 1024u);
        }
        ok = warp_wait(bar_qfree, n_item & 1);
        if (ok) {
          load_q(next);
          q_ready();
        }
      }
      cp_async_wait();
    }
    __syncwarp();
    if (CS > 1) {
      cluster_wait();
      cluster_arrive();
    }
  } else {
    // =========================== softmax warps ===========================
    regs_inc<Regs4<HN>::kCompute>();
    const uint32_t g = warp & 3u, hh = warp >> 2;
    const int r = static_cast<int>(g * 32 + lane);          // row of the chunk, and TMEM lane
    const int hb = static_cast<int>(hh) * HW;               // first head of this thread
    const uint32_t ta = tmem + ((g * 32u) << 16);
    bool waited = !p.early_window;
    if (tid < HN) m_used[tid] = -1e30f;
    if (item0 < n_items && order_q(0, tid, kComputeThreads) && lane == 0) mbar_arrive(bar_q0);
    named_barrier_sync(kBarCompute4, kComputeThreads);
    int chunk = 0, token = 0, n_item = 0;
    bool alive = true;                                      // the same in all compute threads
    bool arrived = false;                                   // at the cluster's second barrier
    for (int item = item0; item < n_items; item += item_step, ++n_item) {
      const int t = item / groups, h0 = (item - t * groups) * HN;
      const int hreal = min(HN, p.H - h0);
      float lsum[HW];
#pragma unroll
      for (int i = 0; i < HW; ++i) lsum[i] = 0.f;
      // the head's sink now: at the end it would be a cold load
      const float sink = tid < hreal ? __ldg(p.sink + h0 + tid) : -INFINITY;
      bool have_o = false;
      while (true) {
        // ---- each warp waits for the chunk's S (or the item's end).  A wait that runs out is
        // told in the vote below, which every thread reaches, so all leave together.
        bool bad = !warp_wait(bar_tok + (token & 3), (token >> 2) & 1);
        const int word = bad ? 0 : meta[token & 3];
        if (!bad && word >= 0) bad = !warp_wait(bar_s, chunk & 1);
        ++token;
        tc_fence_after();
        float sv[HW];
        tmem_load_cols<HW>(ta + kColS + hb, sv);
        const bool rvalid = r < (word & (kLastChunk - 1));
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
        if (any_of(bad || word < 0 || over > kSlack, kBarCompute4, kComputeThreads)) {
          alive = !any_of(bad, kBarCompute4, kComputeThreads);
          if (!alive || word < 0) break;
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
        if ((word & kLastChunk) != 0) {  // the item's end follows: no need to wait for its token
          ++token;
          break;
        }
      }
      if (!alive) break;
      {                                  // per-head sums over the rows
        const float l = TransposeReduce<HW>::run(lsum, lane, 16u, OpAdd());
        constexpr int kRep = 32 / HW;
        if ((lane & (kRep - 1)) == 0) red[(hb + lane / kRep) * 4 + g] = l;
      }
      if (!waited) {                     // outputs are written after the previous kernels completed
        griddep_wait();
        waited = true;
      }
      named_barrier_sync(kBarCompute4, kComputeThreads);
      if (CS > 1) cluster_wait();        // every CTA's barriers are initialised
      float m_mine = -1e30f, l_mine = 0.f, M = 0.f, L = 0.f;
      if (tid < HN) {
        m_mine = m_used[tid];
        const float4 q = *reinterpret_cast<const float4*>(red + tid * 4);
        l_mine = (q.x + q.y) + (q.z + q.w);
        if (CS > 1) {
#pragma unroll 1
          for (int o = 0; o < CS; ++o) {
            if (o == crank) continue;
            st_async_v2f32(cluster_map(smem_u32(mlr + crank * HN + tid), static_cast<uint32_t>(o)), m_mine, l_mine,
                           cluster_map(smem_u32(bar_ml), static_cast<uint32_t>(o)));
          }
        }
      }
      if (CS > 1) {
        __syncwarp();
        cluster_arrive();                // see the merge below
        arrived = true;
      }
      if (tid < HN) {
        if (CS > 1) ok = bar_wait(bar_ml, 0) && ok;
        auto ml_of = [&](int c) { return c == crank ? make_float2(m_mine, l_mine) : mlr[c * HN + tid]; };
        const float sink2 = sink * kLog2e;
        M = sink2;
#pragma unroll 1
        for (int c = 0; c < CS; ++c) {
          const float2 ml = ml_of(c);
          if (!(ml.y == 0.f)) M = fmaxf(M, ml.x);
        }
        L = sink2 > -INFINITY ? ex2_approx(sink2 - M) : 0.f;    // a sink of -inf adds nothing
#pragma unroll 1
        for (int c = 0; c < CS; ++c) {
          const float2 ml = ml_of(c);
          if (!(ml.y == 0.f)) L += ml.y * ex2_approx(ml.x - M);
        }
        const float inv = L == 0.f ? 0.f : __fdividef(1.f, L);  // an empty denominator gives zeros
#pragma unroll 1
        for (int c = 0; c < CS; ++c) {
          const float2 ml = ml_of(c);
          fac[c * HN + tid] = ml.y == 0.f ? 0.f : ex2_approx(ml.x - M) * inv;
        }
      }
      auto write_lse = [&]() {           // after the output, which waits for the factors only
        if (p.lse && crank == 0 && tid < hreal)
          p.lse[static_cast<int64_t>(t) * p.H + h0 + tid] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      };
      if (CS > 1) {
        write_lse();
        break;                           // merged below, by all warps of the cluster
      }
      bool bad = false;
      if (tid == 0) bad = !bar_wait(bar_o, n_item & 1);
      alive = !any_of(bad, kBarCompute4, kComputeThreads);      // also publishes the factors
      tc_fence_after();
      if (!alive) break;
      if (tid == 0) mbar_arrive(bar_item);                      // the MMA warp has read the end's token, too
      // ---- output, 8 or 16 heads at a time: thread = dim, staged in the P buffer as words of
      // (head, head + 1), [4 or 8][512], read back eight dims a thread and stored 16 bytes a head
      const float4* rrow = rope_row(p, t);
      uint32_t* stage = reinterpret_cast<uint32_t*>(ps);
      constexpr int kStage = S::kStage;
#pragma unroll 1
      for (int j0 = 0; j0 < hreal; j0 += kStage) {
        float f[kStage];
#pragma unroll
        for (int x = 0; x < kStage; x += 4) {
          const float4 q = *reinterpret_cast<const float4*>(fac + j0 + x);
          f[x] = q.x, f[x + 1] = q.y, f[x + 2] = q.z, f[x + 3] = q.w;
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float v[kStage];
          if (have_o) {
            tmem_load_cols<kStage>(ta + kColO + (hh * 2 + b) * HN + j0, v);
          } else {
#pragma unroll
            for (int x = 0; x < kStage; ++x) v[x] = 0.f;
          }
          const int d = (static_cast<int>(hh) * 2 + b) * 128 + r;
#pragma unroll
          for (int x = 0; x < kStage; ++x) v[x] *= f[x];
          if (rrow != nullptr && d >= 512 - 64) {               // warp-uniform: dims (d, d ^ 1) are a pair, lanes (l, l ^ 1)
            const float2 cs = __ldg(reinterpret_cast<const float2*>(rrow) + ((d - (512 - 64)) >> 1));
#pragma unroll
            for (int x = 0; x < kStage; ++x) {
              const float other = __shfl_xor_sync(0xffffffffu, v[x], 1);
              v[x] = (lane & 1) ? fmaf(v[x], cs.x, -(other * cs.y)) : fmaf(v[x], cs.x, other * cs.y);
            }
          }
#pragma unroll
          for (int x = 0; x < kStage / 2; ++x) stage[x * 512 + dim_of(d)] = pack_bf16x2(v[2 * x], v[2 * x + 1]);
        }
        named_barrier_sync(kBarCompute4, kComputeThreads);
#pragma unroll
        for (int i = 0; i < kStage / 8; ++i) {
          const int hp = (tid >> 6) + 4 * i, h = j0 + 2 * hp;   // heads h, h + 1; dims 8 (tid & 63) ..
          const uint4 a = *reinterpret_cast<const uint4*>(stage + hp * 512 + (tid & 63) * 8);
          const uint4 c = *reinterpret_cast<const uint4*>(stage + hp * 512 + (tid & 63) * 8 + 4);
          uint16_t* dst = p.out + (static_cast<int64_t>(t) * p.H + h0 + h) * 512 + (tid & 63) * 8;
          if (h < hreal)
            *reinterpret_cast<uint4*>(dst) = make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                                        __byte_perm(c.x, c.y, 0x5410), __byte_perm(c.z, c.w, 0x5410));
          if (h + 1 < hreal)
            *reinterpret_cast<uint4*>(dst + 512) = make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                                              __byte_perm(c.x, c.y, 0x7632), __byte_perm(c.z, c.w, 0x7632));
        }
        named_barrier_sync(kBarCompute4, kComputeThreads);      // the buffer has been read out
      }
      write_lse();
      if (tid < HN) m_used[tid] = -1e30f;                       // read above by the same thread
      tc_fence_before();                 // O has been read; the next item's PV follows its bar_p
      named_barrier_sync(kBarCompute4, kComputeThreads);        // m_used, red, fac and the P buffers are free again
    }
    ok = ok && alive;
    if (CS > 1 && !arrived) {
      cluster_wait();
      cluster_arrive();
    }
  }

  if (CS > 1) {
    // =========================== cluster merge ===========================
    // Every thread has arrived at the cluster's second barrier, the gather warps once
    // their CTA's MMAs were complete: when it completes, every CTA's tiles are idle.
    // Receive slots of the other CS - 1 splits at [0, R), this CTA's outgoing ones
    // at [R, 2 R), R = (CS - 1) slot_bytes, inside the idle tiles.  A slot is
    // [dim][HN] fp32; its 16-byte units are permuted within 128 bytes by the dim, so
    // that the lanes of a warp (neighbouring dims) hit every bank.  The 16 gather
    // warps move the data, each a quarter of the heads of 32 dims at a time, while the
    // softmax warps wait for the others' (m, l) and form the factors.
    constexpr int HQ = HN / 4;
    const int R = (CS - 1) * slot_bytes;
    const int t = item0 / groups, h0 = (item0 - t * groups) * HN;
    const int hreal = min(HN, p.H - h0);
    const bool mover = warp >= 8 && warp < kMmaWarp;
    const uint32_t g = warp & 3u;
    const int hq = (static_cast<int>(warp) - 8) / 4 * HQ;       // a mover's first head
    const uint32_t ta = tmem + ((g * 32u) << 16);
    auto unit_at = [](uint8_t* slot, int dl, int u) {
      const int s = HN >= 32 ? (u ^ (dl & 7)) : (u ^ ((dl >> 1) & 3));
      return reinterpret_cast<float4*>(slot + dl * (HN * 4)) + s;
    };
    // fac is zero where this split attended to nothing; its O may then hold anything
    if (mover) {
#pragma unroll 1
      for (int blk = 0; blk < 4; ++blk) {
        const int d = blk * 128 + static_cast<int>(g * 32 + lane);
        const int owner = d / slice;     // warp-uniform: a slice is at least 64 aligned dims
        if (owner == crank) continue;
        uint8_t* slot = smem + R + (owner < crank ? owner : owner - 1) * slot_bytes;
        float v[HQ];
        tmem_load_cols<HQ>(ta + kColO + blk * HN + hq, v);
#pragma unroll
        for (int x = 0; x < HQ; x += 4)
          *unit_at(slot, d - owner * slice, (hq + x) / 4) = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
      }
      fence_proxy_async_smem();          // the staged slots are read by the bulk-copy engine
      named_barrier_sync(kBarGather4, kGatherThreads);
    }
    cluster_wait();                      // every CTA's tiles are idle
    if (tid == kComputeThreads) {
      for (int o = 0; o < CS; ++o) {
        if (o == crank) continue;
        const int at = crank < o ? crank : crank - 1;
        bulk_copy_to_cluster(cluster_map(smem_u32(smem + at * slot_bytes), static_cast<uint32_t>(o)),
                             smem + R + (o < crank ? o : o - 1) * slot_bytes, static_cast<uint32_t>(slot_bytes),
                             cluster_map(smem_u32(bar_recv), static_cast<uint32_t>(o)));
      }
    }
    __syncthreads();                     // the factors are there
    if (mover) ok = ok && warp_wait(bar_recv, 0);   // the other splits' slots have landed here
    cluster_arrive();                    // ... so their copies out of the senders are complete
    if (mover) {
      const float4* rrow = rope_row_of(p, t, tid == kComputeThreads);
#pragma unroll 1
      for (int blk = crank * slice / 128; blk < (crank * slice + slice + 127) / 128; ++blk) {
        const int d = blk * 128 + static_cast<int>(g * 32 + lane), dl = d - crank * slice;
        if (d / slice != crank) continue;                       // warp-uniform (half a block when slice is 64)
        // neighbouring dims lie two lanes apart in the nope part, one in the rope part (warp-uniform)
        const uint32_t apart = d < DSV4SA_NOPE_DIM ? 2u : 1u;
        const bool odd = (lane & apart) != 0;
        uint16_t* orow = p.out + (static_cast<int64_t>(t) * p.H + h0) * 512 + (dim_of(d) & ~1);
        const bool rot = rrow != nullptr && d >= 512 - 64;
        const float2 cs = rot ? __ldg(reinterpret_cast<const float2*>(rrow) + ((d - (512 - 64)) >> 1)) : make_float2(1.f, 0.f);
        // four heads at a time, not unrolled: code that runs once a launch is fetched from
        // L2 as it runs, so short loops beat straight lines
#pragma unroll 1
        for (int j0 = hq; j0 < hq + HQ; j0 += 4) {
          float v[4];
          tmem_load_cols<4>(ta + kColO + blk * HN + j0, v);
          const float4 fm = *reinterpret_cast<const float4*>(fac + crank * HN + j0);
          v[0] = fm.x == 0.f ? 0.f : v[0] * fm.x;
          v[1] = fm.y == 0.f ? 0.f : v[1] * fm.y;
          v[2] = fm.z == 0.f ? 0.f : v[2] * fm.z;
          v[3] = fm.w == 0.f ? 0.f : v[3] * fm.w;
#pragma unroll 1
          for (int c = 0; c < CS; ++c) {
            if (c == crank) continue;
            const float4 u = *unit_at(smem + (c < crank ? c : c - 1) * slot_bytes, dl, j0 / 4);
            const float4 f = *reinterpret_cast<const float4*>(fac + c * HN + j0);
            if (f.x != 0.f) v[0] = fmaf(u.x, f.x, v[0]);
            if (f.y != 0.f) v[1] = fmaf(u.y, f.y, v[1]);
            if (f.z != 0.f) v[2] = fmaf(u.z, f.z, v[2]);
            if (f.w != 0.f) v[3] = fmaf(u.w, f.w, v[3]);
          }
          // the lanes of dims (2 i, 2 i + 1) pair up: one takes head x, the other head x + 1, of both dims
#pragma unroll
          for (int x = 0; x < 4; x += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? v[x] : v[x + 1], apart);
            float lo = odd ? got : v[x], hi = odd ? v[x + 1] : got;
            if (rot) {
              const float2 z = rotate_back(lo, hi, cs.x, cs.y);
              lo = z.x;
              hi = z.y;
            }
            const int h = j0 + x + (odd ? 1 : 0);
            if (h < hreal && ok) *reinterpret_cast<uint32_t*>(orow + h * 512) = pack_bf16x2(lo, hi);
          }
        }
      }
    }
    cluster_wait();                      // no copy reads this CTA's staging any more
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int HN>
constexpr int smem_bytes4() {
  return Smem4<HN>::kBytes + 1024;       // + alignment slack
}
static_assert(smem_bytes4<16>() <= 227 * 1024 && smem_bytes4<64>() <= 227 * 1024, "shared memory of one CTA");

template <int HN>
bool prepare4(int dev) {
  return smem_attr_once(dev, 5 + HN / 32, reinterpret_cast<const void*>(sparse_attn_fp4_kernel<HN>), smem_bytes4<HN>());
}

// How many clusters of cs CTAs the device runs at once (their CTAs have to be on SMs that
// are wired together, so fewer than the SMs would suggest: of eight CTAs eight clusters ran
// at once, sixteen took twice as long).  Asked once for each device.
template <int HN>
int cluster_slots(int dev, int cs) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][4];
  const int at = cs == 2 ? 1 : (cs == 4 ? 2 : 3);
  if (dev < 0 || dev >= kDevices) return 0;
  const int have = known[dev][at].load(std::memory_order_relaxed);
  if (have > 0) return have - 1;
  if ((cs - 1) * (512 / cs) * HN * 8 > Smem4<HN>::kTiles || !prepare4<HN>(dev)) return 0;   // the merge's slots, in and out
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cs));
  cfg.blockDim = dim3(kThreads4);
  cfg.dynamicSmemBytes = smem_bytes4<HN>();
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, sparse_attn_fp4_kernel<HN>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[dev][at].store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int HN>
int launch_hn4(const AttnParams& p, int groups, int dev, int sms, cudaStream_t stream) {
  if (!prepare4<HN>(dev)) return DSV4SA_ERR_CUDA;
  const int64_t items = static_cast<int64_t>(p.T) * groups;
  if (items * p.nsplit > INT32_MAX) return DSV4SA_ERR_UNSUPPORTED;
  cudaError_t e;
  if (p.nsplit == 1) {
    e = launch_pdl(sparse_attn_fp4_kernel<HN>, dim3(static_cast<unsigned>(items < sms ? items : sms)), dim3(kThreads4),
                   smem_bytes4<HN>(), stream, p, groups);
  } else {
    e = launch_cluster_pdl(sparse_attn_fp4_kernel<HN>, dim3(static_cast<unsigned>(items * p.nsplit)), dim3(kThreads4),
                           smem_bytes4<HN>(), p.nsplit, stream, p, groups);
  }
  return e == cudaSuccess ? DSV4SA_OK : DSV4SA_ERR_CUDA;
}

// Heads of an item and CTAs that share it, by the time they should take: the fixed part of
// a call, a chunk of 128 rows, the step from one item to the next and a cluster's merge, in
// us, as measured for each size of item (calls of 128 to 2176 rows, 1 to 128 queries, 16 to
// 128 heads; the estimates are within a tenth of the times).  Few heads an item cost less
// each -- S, P and O shrink with them, and the merge moves less -- but every item widens its
// rows anew.  So few queries run as many small items, e.g. one query of 64 heads over 640
// rows: 4 items x 8 CTAs 10.5 us, 1 x 4 19.7; 32 of them: 2 x 2 18.5, 1 x 4 21.5, 4 x 1 20.4;
// and many queries as large ones, 128 of them: 1 x 1 27.6 us, 4 x 1 69.
struct Cost4 {
  float fixed, chunk, next, merge;
};
constexpr Cost4 kCost4[3] = {{4.9f, 2.95f, 1.7f, 2.5f}, {5.5f, 3.2f, 3.1f, 3.2f}, {7.7f, 3.7f, 4.4f, 4.2f}};
constexpr int kHeads4[3] = {16, 32, 64};

struct Plan4 {
  int hn, groups, cs;
};
Plan4 plan4(int32_t mode, const AttnParams& p, int dev, int sms) {
  Plan4 best{64, (p.H + 63) / 64, 1};
  float least = 3.4e38f;
  for (int i = 0; i < 3; ++i) {
    if (i > 0 && p.H <= kHeads4[i - 1]) break;               // the smaller item holds all heads
    const int hn = kHeads4[i], groups = (p.H + hn - 1) / hn;
    const int64_t items = static_cast<int64_t>(p.T) * groups;
    for (int cs = 1; cs <= kMaxClusterSplits; cs *= 2) {
      const int rows = share_of(p.kw, 0, cs) + share_of(p.kc, 0, cs), chunks = (rows + kRows - 1) / kRows;
      int slots = sms;
      if (cs > 1) {
        if (mode != DSV4SA_ATTN_DECODE || p.kw + p.kc <= kRows || items > sms / cs) break;
        slots = i == 0 ? cluster_slots<16>(dev, cs) : (i == 1 ? cluster_slots<32>(dev, cs) : cluster_slots<64>(dev, cs));
        if (items > slots) break;
      }
      const Cost4& c = kCost4[i];
      const float rounds = static_cast<float>((items + slots - 1) / slots);
      const float us = c.fixed + rounds * static_cast<float>(chunks) * c.chunk + (rounds - 1.f) * c.next + (cs > 1 ? c.merge : 0.f);
      if (us < least) {
        least = us;
        best = Plan4{hn, groups, cs};
      }
    }
  }
  return best;
}

}  // namespace

namespace attn {

int launch_fp4(int32_t mode, AttnParams& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  const Plan4 plan = plan4(mode, p, dev, sms);
  p.nsplit = plan.cs;
  switch (plan.hn) {
    case 16: return launch_hn4<16>(p, plan.groups, dev, sms, stream);
    case 32: return launch_hn4<32>(p, plan.groups, dev, sms, stream);
    default: return launch_hn4<64>(p, plan.groups, dev, sms, stream);
  }
}

}  // namespace attn

uint32_t* error_word_attn_fp4() { return error_word(); }

}  // namespace dsv4sa
