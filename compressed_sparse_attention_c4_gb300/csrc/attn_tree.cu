// attn_tree.cu -- attention of drafted tokens (nodes of a tree, or a chain) over a paged cache:
// every visible compressed entry of their sequence, the committed window and the drafted
// ancestors.
//
// For node t of sequence b and head h, over the rows
//   J(t) = { entry e of the compressed pool : e < n_vis[t] }
//        u { committed raw token p : pos[t] - window < p <= pos[t], p < ctx[b] }
//        u { drafted row j of the sequence : bit j of anc[t] }
//   o[t, h] = sum_j e^{a_j} kv_j / (sum_j e^{a_j} + e^{sink_h}),  a_j = scale * q[t, h] . kv_j
// ("DeepSeek-V4 全面解读" §3.7 sparse_attn_kernel with get_compress_topk_idxs' list, all visible
// entries, §2.8; "DeepSeek-V4 in SGLang" MQALayer: one kv tensor is both K and V.)
//
// Work.  The queries of a sequence are one matrix of nodes x heads rows; an item is 64 of them,
// for which its rows are read and widened once: eight nodes of 8 heads share them, a node of 64
// heads reads the sequence's rows for itself.  An item's rows -- the entries that any of its nodes
// sees, then the union of their windows, then drafted rows -- are cut into chunks of 128.  All
// chunks of all items are dealt out to the CTAs in equal contiguous runs, by a scan that every
// CTA makes over the batch's lengths, so long and short sequences fill the GPU alike.  A run's
// first and last item may be cut: their sums go to the workspace and a second kernel joins them.
//
// Pipeline of a CTA (as for the 4-bit cache, attn_fp4.cu):
//   scheduler warp: the next item's rows, masks and limits, two items ahead of the slowest; with
//     two more warps it fetches the item's Q when the last S of the item before is complete.
//   gather warps (16): four threads a row; a row's bytes are loaded while the chunk before is
//     worked on, and become BF16 in the 128 x 512 tile (128-byte swizzle), half by half, when
//     the PV of that chunk has read the half.
//   MMA warp: S^T = KV . Q^T (M = 128 rows, N = 64, K = 512), then O^T += V^T . P^T (M = 128
//     dims x 4, N = 64, K = 128).
//   softmax warps (8): thread = row, 32 of the item's columns.  P is BF16 against a max that is
//     only moved (and O rescaled) when a score passes it by 2^8.
// What bounds it: shared memory and the hand-overs from warp to warp.  A chunk takes about 6800
// cycles (trees of 16 nodes, 64 heads, 8336 rows; clock stamps of an instrumented copy): 2700 to
// widen its two halves, of which the first half's 1270 nothing else can hide, 1200 for the second
// half of S, 1320 for the softmax, 1090 until PV has read the first half; the matrix instructions
// read 384 KB of shared memory (3070 cycles at 128 bytes a clock) and the tile's stores are 128 KB
// more.  By the counters nothing is full: tensor pipe 28 % (20 for FP4 rows and 8 heads), L1 and
// shared memory 50, issue slots 43, DRAM 3; a warp waits 9.1 of 14 cycles between instructions
// for TMEM and global loads, 1.5 at barriers.  72 registers a thread; 212 bytes of spill stores a
// thread (180 for FP4 rows), most of them the scheduler's, whose warpgroup has 40 registers.
// 8 sequences x 16 nodes x 64 heads at 8192 entries: 225 us, 621 TFLOP/s, 0.33 of the measured
// matrix rate; 32 x 4 nodes at 512 entries 30.8 us; one token of 16 heads at 512 entries 17.8 to
// 18.9 (scan of the lengths, the item's description, Q, a chunk, its sums, the joining kernel);
// 64 FP4 sequences of 8 heads 78.7.
// Tried and not kept: sixteen warps that load, widen and do the softmax in turn (so that widening
// overlaps PV), 255 to 268 us for the first of these, 236 then with warps of one kind each; loads
// that leave L1 out, 311.
// Only chunks that hold a row that some node does not see look at masks.  A row that holds an
// infinity or a NaN shows in its scores, which then are no numbers for any column: it is taken
// out of the tile (0 times it would be a NaN for nodes that do not see it), and the nodes that
// see it get NaN.
// P is the one operand rounded (BF16); S, O, maxima, sums and the partial sums in the workspace
// are fp32.
#include "attn_common.cuh"
#include "attn_pipe.cuh"
#include "fp4.cuh"

namespace dsv4sa {
namespace {

using namespace attn;

constexpr int kN = 64;                   // columns of an item
constexpr int kComputeThreads = 256;     // warps 0-7: softmax, output
constexpr int kGatherThreads = 512;      // warps 8-23
constexpr int kMmaWarp = 24;
constexpr int kSchedWarp = 25;
constexpr int kThreadsT = kComputeThreads + kGatherThreads + 128;   // the last warpgroup: MMA warp, then
constexpr int kQThreads = 96;            // the scheduler and two more, which fetch Q
constexpr int kHalf = 4 * kKvBlock;      // bytes of a half of the tile: 128 rows x 256 dims
constexpr int kHW = kN / 2;              // columns of a softmax thread
constexpr int kStage = 16;               // columns of an output step
constexpr float kSlack = 8.f;            // log2 units a score may pass the max in use by
constexpr int kFp4RopeOff = 14336;       // KV_FP4 page layout (see dsv4sa.h)
constexpr int kFp4ScaleOff = 22528;
// Registers per thread (setmaxnreg): the launch gives 896 x 72 = 64512.
constexpr int kRegsCompute = 104, kRegsGather = 64, kRegsMma = 40;
static_assert(kComputeThreads * kRegsCompute + kGatherThreads * kRegsGather + 128 * kRegsMma <= kThreadsT * 72,
              "the register shares fit in the launch's");
constexpr uint32_t kBarCompute = 1;      // named barrier
// What is dealt out to the CTAs are an item's chunks and the step to the next item, which takes
// about as long as a chunk.
constexpr int kItemStep = 1;
// Chunks that a CTA may have more than its share when items are left whole: cutting costs the
// writing and joining of partial sums.
constexpr int kWholeSlack = 2;

struct TreeParams {
  const uint16_t* q;
  const float* sink;
  const int32_t* node_start;
  const int32_t* seq_row;    // null: sequence b's row is b
  const int32_t* ctx;
  const int32_t* pos;
  const uint64_t* anc;       // null: a chain
  const int32_t* n_vis;
  const uint8_t* comp_base;
  const int32_t* comp_pt;
  const uint8_t* win_base;
  const int32_t* win_pt;
  const float4* rope_cs;
  const int32_t* rope_pos;
  uint16_t* out;
  float* lse;
  float* ws_o;               // [CTAs][2][64][512]
  float2* ws_ml;             // [CTAs][2][64]
  int4* ws_cut;              // [CTAs]: (first row of q, columns, last CTA) of the item that CTA cuts first
  int64_t comp_page_stride, comp_num_pages, win_page_stride, win_num_pages;
  int32_t comp_pt_stride, win_pt_stride;
  int32_t comp_pt_rows, win_pt_rows;    // of the tables; INT32_MAX where the caller did not say
  int32_t n_max, window, win_ring, draft_entry;
  int32_t B, T, H, max_nodes, blocks;   // blocks: items of a sequence at most
  int32_t rope_rows;
  float scale_log2;
};

// An item in shared memory.
struct alignas(16) Item {
  int32_t c0, c1;            // chunks of it that this CTA works on; c0 = c1: no item is left
  int32_t whole;             // bit 0: its first chunk is among them, bit 1: its last
  int32_t row0;              // first row of the [T H] x 512 queries
  int32_t cols;
  int32_t col0;              // first row of its sequence's queries
  int32_t nv_max, nv_min;    // entries that any, that every node sees
  uint32_t win_rows, rows;   // rows of the windows; all rows
  int32_t runs;              // of consecutive positions that the windows' rows are
  int32_t seq_comp, seq_win; // its row of each page table, -1: not a row of it
  int32_t last_cta;          // the CTA that has the item's last chunk
  int32_t nv[kN], lo[kN], hi[kN];   // by column: entries, first and last position of the window
  uint64_t anc[kN];
  uint64_t any;              // drafted rows that some node sees
  int32_t rope[kN];          // row of the rotation table, -1: none
  uint32_t run_row[kN];      // a run's first row among the windows', and its first position less that
  int32_t run_shift[kN];
};

struct SmemT {
  static constexpr int kKv = 0;
  static constexpr int kQ = 2 * kHalf;
  static constexpr int kP = kQ + kN * 1024;
  static constexpr int kItem = kP + kRows * 128;
  static constexpr int kRed = kItem + 2 * static_cast<int>(sizeof(Item));   // float [64][4]
  static constexpr int kM = kRed + kN * 16;              // float [64] each
  static constexpr int kAlpha = kM + kN * 4;
  static constexpr int kFac = kAlpha + kN * 4;
  static constexpr int kBad = kFac + kN * 4;             // uint32 [16]: rows whose page is out of range, by gather warp
  static constexpr int kLost = kBad + 64;                // uint8 [2][128]: rows without a finite score
  static constexpr int kFirst = kLost + 256;             // int64 [5]: the scan's results
  static constexpr int kBar = kFirst + 48;
  static constexpr int kTmem = kBar + 16 * 8;
  static constexpr int kBytes = kTmem + 16;
};
static_assert(SmemT::kBytes + 1024 <= 227 * 1024, "shared memory of one CTA");

// Nodes of sequence b (0 where its bounds are no range of the call's nodes), its first in s0.
__device__ __forceinline__ int nodes_of(const TreeParams& p, int b, int& s0, bool report) {
  s0 = __ldg(p.node_start + b);
  const int64_t n = static_cast<int64_t>(__ldg(p.node_start + b + 1)) - s0;
  if (s0 < 0 || n < 0 || n > p.max_nodes || s0 + n > p.T) {
    if (report) raise_error(kErrIndex);
    return 0;
  }
  return static_cast<int>(n);
}
__device__ __forceinline__ uint64_t ancestors_of(const TreeParams& p, int s0, int node, int nodes) {
  if (p.draft_entry < 0) return 0;
  const uint64_t a = p.anc ? __ldg(p.anc + s0 + node) : (uint64_t(2) << node) - 1;
  return a & (nodes == 64 ? ~uint64_t(0) : (uint64_t(1) << nodes) - 1);
}
// The committed rows that an item's nodes see are the union of their windows, usually one run of
// consecutive positions; where nodes lie further apart than a window there are more runs.
// lo and hi are the lowest and the highest position, of those that are not negative (hi < 0: there is none).
// Of positions this close the windows leave no gap.
__device__ __forceinline__ bool one_run(uint32_t lo, int hi, int window) { return hi - static_cast<int>(lo) <= window; }
__device__ __forceinline__ int run_start(int pos, int window) { return max(pos - window + 1, 0); }
// Rows of the windows of n nodes: exact for one run; else no fewer, for dealing out chunks.
__device__ __forceinline__ uint32_t run_rows(uint32_t lo, int hi, int n, int window, int ctx) {
  if (hi < 0 || window == 0) return 0;
  const uint32_t range = static_cast<uint32_t>(max(min(hi + 1, max(ctx, 0)) - run_start(static_cast<int>(lo), window), 0));
  return one_run(lo, hi, window) ? range : min(range, static_cast<uint32_t>(n) * static_cast<uint32_t>(window));
}
__device__ __forceinline__ uint32_t rows_of(int nv_max, uint32_t win_rows, uint64_t anc) {
  return static_cast<uint32_t>(nv_max) + win_rows + static_cast<uint32_t>(64 - __clzll(static_cast<long long>(anc)));
}
// Position of row e of an item's windows.
__device__ __forceinline__ uint32_t position_of(const Item* it, uint32_t e) {
  int s = it->runs - 1;
  if (s > 0) {
#pragma unroll 1
    while (e < it->run_row[s]) --s;
  }
  return e + static_cast<uint32_t>(it->run_shift[s]);
}
__device__ __forceinline__ int chunks_of(uint32_t rows) { return rows == 0 ? 1 : static_cast<int>((rows + kRows - 1) / kRows); }
// A position as the masks use it: below 2^31 - 1, -1 for any that is negative.
__device__ __forceinline__ int pos_of(int pos) { return min(max(pos, -1), 0x7FFFFFFE); }

// Chunks of item (b, k), by one thread: eight nodes' values are on the way at a time.
__device__ __forceinline__ int chunks_of_item(const TreeParams& p, int s0, int nodes, int ctx, int k) {
  uint32_t lo = ~0u;         // a position of -1 is above all others
  int nv = 0, hi = -1;
  uint64_t anc = 0;
  const int first = k * kN / p.H, last = min(nodes - 1, ((k + 1) * kN - 1) / p.H);
  for (int n0 = first; n0 <= last; n0 += 8) {
    int v[8], pos[8];
    uint64_t a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = min(n0 + i, last);       // the last again, where there are fewer
      v[i] = __ldg(p.n_vis + s0 + n);
      pos[i] = __ldg(p.pos + s0 + n);
      a[i] = ancestors_of(p, s0, n, nodes);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = pos_of(pos[i]);
      nv = max(nv, min(v[i], p.n_max));
      lo = min(lo, static_cast<uint32_t>(at));
      hi = max(hi, at);
      anc |= a[i];
    }
  }
  return chunks_of(rows_of(nv, run_rows(lo, hi, last - first + 1, p.window, ctx), anc));
}

// a b / c, all below 2^63 c; without a 64-bit division where that is possible
__device__ __forceinline__ int64_t scaled(int64_t a, int64_t b, int64_t c) {
  const int64_t x = a * b;
  return x >> 32 == 0 ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(c)) : x / c;
}

template <bool kFp4>
__global__ void __launch_bounds__(kThreadsT, 1) tree_attn_kernel(const TreeParams p) {
  using S = SmemT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* kv = smem + S::kKv;
  uint8_t* qs = smem + S::kQ;
  uint8_t* ps = smem + S::kP;
  Item* items = reinterpret_cast<Item*>(smem + S::kItem);
  float* red = reinterpret_cast<float*>(smem + S::kRed);
  float* m_used = reinterpret_cast<float*>(smem + S::kM);
  float* alpha = reinterpret_cast<float*>(smem + S::kAlpha);
  float* fac = reinterpret_cast<float*>(smem + S::kFac);
  uint32_t* bad_rows = reinterpret_cast<uint32_t*>(smem + S::kBad);
  uint8_t* lost = smem + S::kLost;
  int64_t* first = reinterpret_cast<int64_t*>(smem + S::kFirst);
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + S::kBar);   // [2]: half of a chunk's dims is in place
  uint64_t* bar_free = bar_full + 2;       // [2]: ... has been read by PV
  uint64_t* bar_item = bar_full + 4;       // [2]: an item is described
  uint64_t* bar_done = bar_full + 6;       // [2]: ... and no longer needed
  uint64_t* bar_s = bar_full + 8;          // S is complete
  uint64_t* bar_p = bar_full + 9;          // P is written
  uint64_t* bar_o = bar_full + 10;         // every PV of the item is complete
  uint64_t* bar_q = bar_full + 11;         // the item's Q is there
  uint64_t* bar_qfree = bar_full + 12;     // every S of the item is complete
  uint64_t* bar_q0 = bar_full + 13;        // the first item's Q is there
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + S::kTmem);

  constexpr uint32_t kColS = 0, kColO = kN;
  const int tid = static_cast<int>(threadIdx.x);
  const uint32_t warp = warp_id(), lane = lane_id();

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_full + i, kGatherThreads / 32);
      mbar_init(bar_free + i, 1);
      mbar_init(bar_item + i, 1);
      mbar_init(bar_done + i, (kComputeThreads + kGatherThreads) / 32 + 1);
    }
    mbar_init(bar_s, 1);
    mbar_init(bar_p, kComputeThreads / 32);
    mbar_init(bar_o, 1);
    mbar_init(bar_q, kQThreads / 32);
    mbar_init(bar_qfree, 1);
    mbar_init(bar_q0, kComputeThreads / 32);
    fence_mbar_init();
    first[0] = -1;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  griddep_launch();
  griddep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  // ---- this CTA's run of chunks (and steps): each thread counts a run of items, a scan over the threads
  {
    int64_t* part = reinterpret_cast<int64_t*>(kv);
    int2* part_items = reinterpret_cast<int2*>(kv + 512);   // items, the longest one's chunks
    const int n_items = p.B * p.blocks, per = (n_items + kThreadsT - 1) / kThreadsT;
    const int i0 = min(static_cast<int64_t>(tid) * per, static_cast<int64_t>(n_items)), i1 = min(i0 + per, n_items);
    // adds up items from i0 on, until the one that has chunk `until`, or is number `until_item` of this run
    int seen = 0, longest = 0, size = 0;
    auto walk = [&](int64_t until, int until_item, int& item, int64_t at) {
      int b_of = -1, s0 = 0, nodes = 0, ctx = 0;
      seen = 0;
      for (item = i0; item < i1; ++item) {
        const int b = item / p.blocks, k = item - b * p.blocks;
        if (b != b_of) {
          nodes = nodes_of(p, b, s0, blockIdx.x == 0);
          ctx = __ldg(p.ctx + b);
          b_of = b;
        }
        if (k * kN >= nodes * p.H) continue;
        size = chunks_of_item(p, s0, nodes, ctx, k) + kItemStep;
        longest = max(longest, size);
        if (at + size > until || seen == until_item) return at;
        at += size;
        ++seen;
      }
      return at;
    };
    int item;
    const int64_t mine = walk(INT64_MAX, -1, item, 0);
    const int mine_items = seen;
    int64_t sum = mine;
    int sum_items = mine_items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
      const int up_items = __shfl_up_sync(0xffffffffu, sum_items, o);
      if (lane >= static_cast<uint32_t>(o)) sum += up, sum_items += up_items;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 31) part[warp] = sum, part_items[warp] = make_int2(sum_items, longest);
    __syncthreads();
    int64_t before = sum - mine, total = 0;
    int before_items = sum_items - mine_items, all_items = 0;
    for (int w = 0; w < kThreadsT / 32; ++w) {
      const int2 q = part_items[w];
      if (w < static_cast<int>(warp)) before += part[w], before_items += q.x;
      total += part[w];
      all_items += q.x;
      longest = max(longest, q.y);
    }
    // no more CTAs than there is to deal out, so that every CTA between an item's first and last has a piece of it
    const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total), g = blockIdx.x;
    // its item is this thread's where the thread counted it: number g of all items, left whole, or the one that has
    // chunk w0 of all; none where no sequence has a node
    const bool whole = total > 0 && all_items <= ctas && longest <= (total + ctas - 1) / ctas + kWholeSlack;
    int64_t w0 = total, w1 = total;
    if (!whole && g < ctas) w0 = scaled(total, g, ctas), w1 = scaled(total, g + 1, ctas);
    if (whole ? before_items <= g && g < before_items + mine_items : w0 < w1 && before <= w0 && w0 < before + mine) {
      item = i0;
      const int64_t at = per > 1 ? walk(whole ? INT64_MAX : w0, whole ? static_cast<int>(g) - before_items : -1, item, before) : before;
      if (whole) w0 = at, w1 = at + size;
      const bool step = w0 - at >= size - kItemStep;        // only its last step: that is another CTA's
      first[0] = step ? item + 1 : item;
      first[1] = step ? at + size : at;
      first[2] = step ? at + size : w0;
      first[3] = w1;
    }
    if (tid == 0) first[4] = total;
    __syncthreads();
  }
  bool ok = true;                            // no wait of this thread has run out

  // Q of an item: swizzled K-major tile; rows past the item's are zero.
  auto load_q = [&](int row0, int cols, int from, int step) {
    const uint4* src = reinterpret_cast<const uint4*>(p.q) + static_cast<int64_t>(row0) * 64;
#pragma unroll 4
    for (int u = from; u < kN * 64; u += step) {
      const int h = u >> 6, v = u & 63;
      cp_async16(qs + (v >> 3) * (kN * 128) + sw128_offset(h, v & 7), src + min(h, cols - 1) * 64 + v, h < cols ? 16u : 0u);
    }
    cp_async_wait();
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (warp >= 8 && warp < kMmaWarp) {
    // =========================== gather warps ===========================
    // A wait that runs out is not repeated: the loop goes on without waiting.
    regs_dec<kRegsGather>();
    const int gt = tid - kComputeThreads;
    const int row = gt >> 2, piece = gt & 3;
    int chunk = 0;
#pragma unroll 1
    for (int n_item = 0;; ++n_item) {
      const Item* it = items + (n_item & 1);
      ok = ok && warp_wait(bar_item + (n_item & 1), (n_item >> 1) & 1);
      if (!ok) break;
      const int c1 = it->c1;
      int c = it->c0;
      if (c == c1) break;
      const uint32_t nv_max = static_cast<uint32_t>(it->nv_max), rows = it->rows;
      // the row's page (1024-byte aligned) and its slot; 0: no row, or its page is out of range
      auto locate = [&](int ch) -> uint64_t {
        const uint32_t rr = static_cast<uint32_t>(ch) * kRows + row;
        if (rr >= rows) return 0;
        if (rr < nv_max) {
          const int seq = it->seq_comp;
          const int page = seq >= 0 ? __ldg(p.comp_pt + static_cast<int64_t>(seq) * p.comp_pt_stride + (rr >> 6)) : -1;
          if (page < 0 || page >= p.comp_num_pages) return 0;
          return reinterpret_cast<uint64_t>(p.comp_base + page * p.comp_page_stride) | (rr & 63u);
        }
        uint32_t e = rr - nv_max;
        if (e < it->win_rows) {
          const uint32_t at = position_of(it, e);
          e = p.win_ring > 0 ? at % static_cast<uint32_t>(p.win_ring) : at;
        } else {
          e = static_cast<uint32_t>(p.draft_entry) + (e - it->win_rows);
        }
        const int seq = it->seq_win;
        const int page = seq >= 0 && static_cast<int>(e >> 6) < p.win_pt_stride
                             ? __ldg(p.win_pt + static_cast<int64_t>(seq) * p.win_pt_stride + (e >> 6)) : -1;
        if (page < 0 || page >= p.win_num_pages) return 0;
        return reinterpret_cast<uint64_t>(p.win_base + page * p.win_page_stride) | (e & 63u);
      };
      uint64_t rp = locate(c);
#pragma unroll 1
      for (; c < c1; ++c) {
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        const uint8_t* page = reinterpret_cast<const uint8_t*>(rp & ~uint64_t(63));
        const int rs = static_cast<int>(rp & 63);
        const bool there = rp != 0;
        const bool bad = !there && static_cast<uint32_t>(c) * kRows + row < rows;   // its page is out of range
        uint4 code[7], rope[2], scl;
        uint2 code3;
        if constexpr (kFp4) {
          // 16-byte pieces 4 b + piece (32 values, a scale block each), then 8 bytes of the last two
          const uint8_t* cp = page + rs * 224;
          scl = there ? __ldg(reinterpret_cast<const uint4*>(page + kFp4ScaleOff + rs * 16)) : zero;
#pragma unroll
          for (int b = 0; b < 3; ++b) code[b] = there ? __ldg(reinterpret_cast<const uint4*>(cp) + 4 * b + piece) : zero;
          code3 = there ? __ldg(reinterpret_cast<const uint2*>(cp + 192) + piece) : make_uint2(0u, 0u);
        } else {
          // 16-byte pieces 4 b + piece: a quarter of the 64 values of scale block b; of the
          // scales this thread holds two, for its row's four threads
          const uint4* cp = reinterpret_cast<const uint4*>(page + rs * 448) + piece;
          const uint32_t* sp = reinterpret_cast<const uint32_t*>(page + kPageScaleOff + rs * 32);
          scl.x = there ? __ldg(sp + piece) : 0u;
          scl.y = there ? __ldg(sp + 4 + min(piece, 2)) : 0u;
#pragma unroll
          for (int b = 0; b < 7; ++b) code[b] = there ? __ldg(cp + 4 * b) : zero;
        }
        const uint4* rpp = reinterpret_cast<const uint4*>(page + (kFp4 ? kFp4RopeOff : kPageRopeOff) + rs * 128) + 2 * piece;
        rope[0] = there ? __ldg(rpp) : zero;
        rope[1] = there ? __ldg(rpp + 1) : zero;
        rp = c + 1 < c1 ? locate(c + 1) : 0;      // the next chunk's, in flight together
        uint32_t sb = 0;
        if constexpr (kFp4)
          sb = __byte_perm(__byte_perm(scl.x, scl.y, piece * 0x11 + 0x40), __byte_perm(scl.z, scl.w, piece + ((piece >> 1) + 4) * 0x10),
                           0x5410);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (chunk > 0 && ok) ok = warp_wait(bar_free + h, (chunk - 1) & 1);
          uint8_t* half = kv + h * kHalf;
          if (h == 0) {
            const uint32_t bits = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) bad_rows[warp - 8] = bits;
            if (bits != 0) {               // of a drafted row that no node sees it does not matter
              const uint32_t draft = static_cast<uint32_t>(c) * kRows + row - nv_max - it->win_rows;
              if (bad && (draft >= 64 || (it->any >> draft & 1) != 0)) raise_error(kErrIndex);
            }
          }
          if constexpr (kFp4) {
#pragma unroll
            for (int b = 2 * h; b < 3 && b < 2 * h + 2; ++b) {
              // units 4 (piece & 1) + x of column block 2 b + (piece >> 1); the upper two pieces take
              // x in the order 2, 3, 0, 1: the eight lanes of two rows hit eight bank groups
              const BlockScale bs = block_scale((sb >> (8 * b)) & 0xFFu);
              uint8_t* blk = half + (2 * (b & 1) + (piece >> 1)) * kKvBlock;
              const uint32_t c4[4] = {code[b].x, code[b].y, code[b].z, code[b].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t w = piece >= 2 ? c4[i ^ 2] : c4[i];
                const uint32_t x = static_cast<uint32_t>(i) ^ (piece & 2);
                uint4 v = widen8(w, bs.first);
                if (bs.more) v = scale_up(v, bs.more);
                *reinterpret_cast<uint4*>(blk + sw128_offset(row, static_cast<uint32_t>(4 * (piece & 1)) + x)) = v;
              }
            }
            if (h == 1) {
              const BlockScale bs = block_scale(sb >> 24);
              uint4 v0 = widen8(code3.x, bs.first), v1 = widen8(code3.y, bs.first);
              if (bs.more) {
                v0 = scale_up(v0, bs.more);
                v1 = scale_up(v1, bs.more);
              }
              *reinterpret_cast<uint4*>(half + 2 * kKvBlock + sw128_offset(row, static_cast<uint32_t>(2 * piece))) = v0;
              *reinterpret_cast<uint4*>(half + 2 * kKvBlock + sw128_offset(row, static_cast<uint32_t>(2 * piece + 1))) = v1;
            }
          } else {
#pragma unroll
            for (int b = 4 * h; b < 7 && b < 4 * h + 4; ++b) {
              const float scale = __uint_as_float(__shfl_sync(0xffffffffu, b < 4 ? scl.x : scl.y, static_cast<int>(lane & ~3u) + (b & 3)));
              uint4 v0, v1;
              dequant16(code[b], scale, v0, v1);
              uint8_t* blk = half + (b - 4 * h) * kKvBlock;
              *reinterpret_cast<uint4*>(blk + sw128_offset(row, static_cast<uint32_t>(2 * piece))) = v0;
              *reinterpret_cast<uint4*>(blk + sw128_offset(row, static_cast<uint32_t>(2 * piece + 1))) = v1;
            }
          }
          if (h == 1) {
            *reinterpret_cast<uint4*>(half + 3 * kKvBlock + sw128_offset(row, static_cast<uint32_t>(2 * piece))) = rope[0];
            *reinterpret_cast<uint4*>(half + 3 * kKvBlock + sw128_offset(row, static_cast<uint32_t>(2 * piece + 1))) = rope[1];
          }
          fence_proxy_async_smem();        // the tile is read by the tensor core
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_full + h);
        }
        __syncwarp();
        ++chunk;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_done + (n_item & 1));
    }
  } else if (warp >= kMmaWarp) {
    regs_dec<kRegsMma>();
    if (warp == kMmaWarp) {
      // =========================== MMA warp ===========================
      const uint32_t idesc_s = make_idesc(kFmtBF16, kFmtBF16, 0, 0, 128, kN);
      const uint32_t idesc_o = make_idesc(kFmtBF16, kFmtBF16, 1, 1, 128, kN);
      const uint32_t hi = static_cast<uint32_t>(smem_desc_sw128(0, 16, 1024) >> 32);   // stride, version, swizzle
      const uint32_t kvk = static_cast<uint32_t>(smem_desc_sw128(smem_u32(kv), 16, 1024));
      const uint32_t qk = static_cast<uint32_t>(smem_desc_sw128(smem_u32(qs), 16, 1024));
      const uint32_t kvm = static_cast<uint32_t>(smem_desc_sw128(smem_u32(kv), kKvBlock, 1024));
      const uint32_t pd = static_cast<uint32_t>(smem_desc_sw128(smem_u32(ps), kRows * 128, 1024));   // [row][64 columns]
      int chunk = 0;
#pragma unroll 1
      for (int n_item = 0; ok; ++n_item) {
        ok = warp_wait(bar_item + (n_item & 1), (n_item >> 1) & 1);
        if (!ok) break;
        const int n = items[n_item & 1].c1 - items[n_item & 1].c0;
        __syncwarp();
        if (n == 0) break;
        if (lane == 0) mbar_arrive(bar_done + (n_item & 1));
        __syncwarp();
        ok = n_item == 0 ? warp_wait(bar_q0, 0) : warp_wait(bar_q, (n_item - 1) & 1);
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && warp_wait(bar_full + h, chunk & 1);
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {  // not unrolled: the descriptors would not fit in registers
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_f16_elect(tmem + kColS, kvk + ((h * kHalf + b * kKvBlock + kk * 32) >> 4), qk + (((4 * h + b) * kN * 128 + kk * 32) >> 4),
                              hi, idesc_s, h > 0 || b > 0 || kk > 0 ? 1u : 0u);
            }
          }
          mma_commit_elect(bar_s);
          if (i + 1 == n) mma_commit_elect(bar_qfree);
          ok = ok && warp_wait(bar_p, chunk & 1);
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll 1
            for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_f16_elect(tmem + kColO + (2 * h + mb) * kN, kvm + ((h * kHalf + 2 * mb * kKvBlock + kk * 2048) >> 4), pd + (kk * 2048 >> 4),
                              hi, idesc_o, (i > 0 || kk > 0) ? 1u : 0u);
            }
            mma_commit_elect(bar_free + h);
          }
          ++chunk;
        }
        mma_commit_elect(bar_o);
      }
    } else {
      // =========================== scheduler and Q ===========================
      const int qt = tid - kSchedWarp * 32;
      int item = static_cast<int>(first[0]);
      int64_t base = first[1], at = first[2];    // what lies before the item; where this CTA goes on
      const int64_t w1 = first[3], total = first[4], ctas = min(static_cast<int64_t>(gridDim.x), total);
      if (item < 0) at = w1;                     // nothing for this CTA
      // Every one of the three warps walks the items (Q's place follows from the walk); the first writes them down.
#pragma unroll 1
      for (int n_item = 0;; ++n_item) {
        int b = 0, k = 0, s0 = 0, nodes = 0;
        while (at < w1) {                        // the next item with columns
          b = item / p.blocks;
          k = item - b * p.blocks;
          nodes = nodes_of(p, b, s0, false);
          if (k * kN < nodes * p.H) break;
          // none left in this sequence: look at the next 32
          int nb = b + 1;
          while (nb < p.B) {
            int s = 0;
            const bool has = nb + static_cast<int>(lane) < p.B && nodes_of(p, nb + static_cast<int>(lane), s, false) > 0;
            const uint32_t any = __ballot_sync(0xffffffffu, has);
            if (any != 0) {
              nb += __ffs(any) - 1;
              break;
            }
            nb += 32;
          }
          if (nb >= p.B) at = w1;                // cannot be: the chunks were counted
          else item = nb * p.blocks;
        }
        const bool more = at < w1;
        const int cols = more ? min(kN, nodes * p.H - k * kN) : 0;
        const int row0 = more ? s0 * p.H + k * kN : 0;
        int chunks = 0;
        if (more) {
          const int ctx = __ldg(p.ctx + b), seq = p.seq_row ? __ldg(p.seq_row + b) : b;
          uint32_t lo = ~0u;
          int nv_max = 0, nv_min = INT32_MAX, hi = -1, nvc[2], posc[2], nodec[2];
          uint64_t ancc[2], anc = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int col = static_cast<int>(lane) + 32 * j;
            const int node = (k * kN + min(col, cols - 1)) / p.H;
            nodec[j] = s0 + node;
            nvc[j] = max(min(__ldg(p.n_vis + s0 + node), p.n_max), 0);
            posc[j] = pos_of(__ldg(p.pos + s0 + node));
            ancc[j] = ancestors_of(p, s0, node, nodes);
            nv_max = max(nv_max, nvc[j]);
            nv_min = min(nv_min, nvc[j]);
            lo = min(lo, static_cast<uint32_t>(posc[j]));
            hi = max(hi, posc[j]);
            anc |= ancc[j];
          }
          nv_max = __reduce_max_sync(0xffffffffu, nv_max);
          nv_min = __reduce_min_sync(0xffffffffu, nv_min);
          lo = __reduce_min_sync(0xffffffffu, lo);
          hi = __reduce_max_sync(0xffffffffu, hi);
          anc = static_cast<uint64_t>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(anc >> 32))) << 32 |
                __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(anc));
          uint32_t win_rows = run_rows(lo, hi, (k * kN + cols - 1) / p.H - k * kN / p.H + 1, p.window, ctx);
          chunks = chunks_of(rows_of(nv_max, win_rows, anc));
          if (warp == kSchedWarp) {
            if (n_item >= 2 && ok) ok = warp_wait(bar_done + (n_item & 1), ((n_item >> 1) - 1) & 1);
            Item* it = items + (n_item & 1);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int col = static_cast<int>(lane) + 32 * j;
              it->nv[col] = nvc[j];
              it->lo[col] = posc[j] - p.window + 1;
              it->hi[col] = posc[j];
              it->anc[col] = ancc[j];
              int r = -1;
              if (p.rope_cs) {
                r = __ldg(p.rope_pos + nodec[j]);
                if (r < 0 || r >= p.rope_rows) {
                  if (col < cols) raise_error(kErrIndex);
                  r = -1;
                }
              }
              it->rope[col] = r;
            }
            int runs = 1;
            if (lane == 0) it->run_shift[0] = run_start(static_cast<int>(lo), p.window);
            if (win_rows > 0 && !one_run(lo, hi, p.window)) {
              // the union, position by position: `end` is behind the last run
              int end = 0;
              runs = 0;
              win_rows = 0;
#pragma unroll 1
              for (int x = -1;;) {
                int next = INT32_MAX;              // the lowest position above x
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  if (posc[j] > x) next = min(next, posc[j]);
                x = __reduce_min_sync(0xffffffffu, next);
                if (x == INT32_MAX) break;
                const int from = run_start(x, p.window), to = min(x + 1, ctx);
                if (to <= max(from, end)) continue;
                if (runs == 0 || from > end) {
                  if (lane == 0) it->run_row[runs] = win_rows, it->run_shift[runs] = from - static_cast<int>(win_rows);
                  ++runs;
                  end = from;
                }
                win_rows += static_cast<uint32_t>(to - end);
                end = to;
              }
            }
            if (lane == 0) {
              const int64_t end = min(base + chunks, w1);
              it->c0 = static_cast<int>(at - base);
              it->c1 = static_cast<int>(end - base);
              it->whole = (at == base ? 1 : 0) | (end == base + chunks ? 2 : 0);
              it->row0 = row0;
              it->cols = cols;
              it->col0 = k * kN;
              it->nv_max = nv_max;
              it->nv_min = nv_min;
              it->win_rows = win_rows;
              it->rows = rows_of(nv_max, win_rows, anc);
              it->any = anc;
              it->runs = runs;
              it->seq_comp = seq < p.comp_pt_rows ? seq : -1;
              it->seq_win = seq < p.win_pt_rows ? seq : -1;
              const int64_t x = (base + chunks) * ctas - 1;   // the CTA that has the item's last chunk
              it->last_cta = static_cast<int>(scaled(x, 1, total));
            }
          }
        } else if (warp == kSchedWarp) {
          if (n_item >= 2 && ok) ok = warp_wait(bar_done + (n_item & 1), ((n_item >> 1) - 1) & 1);
          if (lane == 0) items[n_item & 1].c0 = items[n_item & 1].c1 = 0;
        }
        if (warp == kSchedWarp) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_item + (n_item & 1));
        }
        if (!more || !ok) break;
        // ---- Q, when the S of the item before are complete (the first item's: by the softmax warps)
        if (n_item > 0) {
          if (qt == 0) prefetch_l2(p.q + static_cast<int64_t>(row0) * 512, static_cast<uint32_t>(cols) * 1024u);
          ok = warp_wait(bar_qfree, (n_item - 1) & 1);
          if (!ok) break;
          load_q(row0, cols, qt, kQThreads);
          if (lane == 0) mbar_arrive(bar_q);
        }
        base += chunks + kItemStep;
        at = base;
        ++item;
      }
    }
    __syncwarp();
  } else {
    // =========================== softmax warps ===========================
    regs_inc<kRegsCompute>();
    const uint32_t g = warp & 3u, hh = warp >> 2;
    const int r = static_cast<int>(g * 32 + lane);          // row of the chunk, and TMEM lane
    const int hb = static_cast<int>(hh) * kHW;              // first column of this thread
    const uint32_t ta = tmem + ((g * 32u) << 16);
    if (tid < kN) m_used[tid] = -1e30f;
    if (tid == 0) p.ws_cut[blockIdx.x] = make_int4(0, 0, 0, 0);
    named_barrier_sync(kBarCompute, kComputeThreads);
    if (warp_wait(bar_item, 0) && items[0].c0 < items[0].c1) {
      load_q(items[0].row0, items[0].cols, tid, kComputeThreads);
      if (lane == 0) mbar_arrive(bar_q0);
    }
    int chunk = 0;
    bool alive = true;                                      // the same in all compute threads
#pragma unroll 1
    for (int n_item = 0;; ++n_item) {
      const Item* it = items + (n_item & 1);
      bool bad = !warp_wait(bar_item + (n_item & 1), (n_item >> 1) & 1);
      alive = !any_of(bad, kBarCompute, kComputeThreads);
      if (!alive) break;
      const int c1 = it->c1;
      if (it->c0 == c1) break;
      float lsum[kHW];
#pragma unroll
      for (int i = 0; i < kHW; ++i) lsum[i] = 0.f;
      bool have_o = false;
#pragma unroll 1
      for (int c = it->c0; c < c1; ++c) {
        // ---- which columns see this thread's row
        uint32_t seen = ~0u;
        const uint32_t rr = static_cast<uint32_t>(c) * kRows + r;
        if (static_cast<uint32_t>(c + 1) * kRows > static_cast<uint32_t>(it->nv_min)) {
          seen = 0;
          const uint32_t nv_max = static_cast<uint32_t>(it->nv_max), win_end = nv_max + it->win_rows;
          if (rr < nv_max) {
#pragma unroll 4
            for (int i = 0; i < kHW; ++i) seen |= (rr < static_cast<uint32_t>(it->nv[hb + i]) ? 1u : 0u) << i;
          } else if (rr < win_end) {
            const int at = static_cast<int>(position_of(it, rr - nv_max));
#pragma unroll 4
            for (int i = 0; i < kHW; ++i) seen |= (at >= it->lo[hb + i] && at <= it->hi[hb + i] ? 1u : 0u) << i;
          } else if (rr < it->rows) {
            const int j = static_cast<int>(rr - win_end);
#pragma unroll 4
            for (int i = 0; i < kHW; ++i) seen |= static_cast<uint32_t>(it->anc[hb + i] >> j & 1) << i;
          }
        }
        // ---- each warp waits for the chunk's S.  A wait that runs out is told in the vote below,
        // which every thread reaches, so all leave together.
        bad = !warp_wait(bar_full, chunk & 1) || !warp_wait(bar_s, chunk & 1);
        tc_fence_after();
        if (bad_rows[r >> 3] >> ((r & 7) * 4) & 1u) seen = 0;
        float sv[kHW];
        tmem_load_cols<kHW>(ta + kColS + hb, sv);
        float over = -INFINITY, least = INFINITY;
#pragma unroll
        for (int i = 0; i < kHW; i += 4) {
          const float4 m = *reinterpret_cast<const float4*>(m_used + hb + i);
          const float mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            least = fminf(least, fabsf(sv[i + x]));
            sv[i + x] = (seen >> (i + x) & 1u) != 0u ? sv[i + x] * p.scale_log2 : -INFINITY;
            over = fmaxf(over, sv[i + x] - mm[x]);
          }
        }
        const bool none = !(least < INFINITY);              // no column has a number here
        if (any_of(bad || none || over > kSlack, kBarCompute, kComputeThreads)) {
          alive = !any_of(bad, kBarCompute, kComputeThreads);
          if (!alive) break;
          if (any_of(none, kBarCompute, kComputeThreads)) {
            // a row that is no row of numbers: out of the tile; its nodes get NaN
            lost[hh * kRows + r] = none ? 1 : 0;
            named_barrier_sync(kBarCompute, kComputeThreads);
            if (lost[r] && lost[kRows + r]) {
#pragma unroll 1
              for (int u = 0; u < 32; ++u)
                *reinterpret_cast<uint4*>(kv + hh * kHalf + (u >> 3) * kKvBlock + sw128_offset(r, u & 7)) = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
              for (int i = 0; i < kHW; ++i) sv[i] = (seen >> i & 1u) != 0u ? __uint_as_float(0x7FC00000u) : -INFINITY;
            }
            named_barrier_sync(kBarCompute, kComputeThreads);
          }
          // a score passes the max in use: take the chunk's max of those columns, rescale
          float tmp[kHW];
#pragma unroll
          for (int i = 0; i < kHW; ++i) tmp[i] = sv[i];
          const float m = TransposeReduce<kHW>::run(tmp, lane, 16u, OpMax());
          red[(hb + lane) * 4 + g] = m;
          named_barrier_sync(kBarCompute, kComputeThreads);
          if (tid < kN) {
            const float4 q = *reinterpret_cast<const float4*>(red + tid * 4);
            const float mc = fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)), mo = m_used[tid];
            const float mn = mc > mo + kSlack ? mc : mo;
            alpha[tid] = ex2_approx(mo - mn);
            m_used[tid] = mn;
          }
          named_barrier_sync(kBarCompute, kComputeThreads);
          if (have_o) {                  // S being complete, so is the PV before it
#pragma unroll
            for (int i = 0; i < kHW; ++i) lsum[i] *= alpha[hb + i];
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
              const uint32_t to = ta + kColO + (hh * 2 + b) * kN;
#pragma unroll 1
              for (int j0 = 0; j0 < kN; j0 += 16) {
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
        for (int i = 0; i < kHW; i += 8) {
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
          *reinterpret_cast<uint4*>(ps + sw128_offset(r, static_cast<uint32_t>((hb + i) >> 3))) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        have_o = true;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p);
        ++chunk;
      }
      if (!alive) break;
      // ---- the item's end: sums over the rows
      red[(hb + lane) * 4 + g] = TransposeReduce<kHW>::run(lsum, lane, 16u, OpAdd());
      named_barrier_sync(kBarCompute, kComputeThreads);
      const int cols = it->cols, row0 = it->row0;
      const bool whole = it->whole == 3;
      const int piece = (it->whole & 1) != 0 ? 1 : 0;       // the item's first piece is this CTA's last
      if (tid < kN) {
        const float m = m_used[tid];
        const float4 q = *reinterpret_cast<const float4*>(red + tid * 4);
        const float l = (q.x + q.y) + (q.z + q.w);
        if (whole) {
          const float sink2 = tid < cols ? __ldg(p.sink + (it->col0 + tid) % p.H) * kLog2e : -INFINITY;
          const float M = l == 0.f ? sink2 : fmaxf(sink2, m);
          float L = sink2 > -INFINITY ? ex2_approx(sink2 - M) : 0.f;    // a sink of -inf adds nothing
          if (!(l == 0.f)) L += l * ex2_approx(m - M);
          fac[tid] = L == 0.f || l == 0.f ? 0.f : ex2_approx(m - M) * __fdividef(1.f, L);   // an empty denominator gives zeros
          if (p.lse && tid < cols) p.lse[static_cast<int64_t>(row0) + tid] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        } else {
          p.ws_ml[(static_cast<int64_t>(blockIdx.x) * 2 + piece) * kN + tid] = make_float2(m, l);
          if (tid == 0 && piece == 1) p.ws_cut[blockIdx.x] = make_int4(row0, cols, it->last_cta, 0);
        }
        m_used[tid] = -1e30f;
      }
      bad = false;
      if (tid == 0) bad = !bar_wait(bar_o, n_item & 1);
      alive = !any_of(bad, kBarCompute, kComputeThreads);      // also publishes the factors
      tc_fence_after();
      if (!alive) break;
      if (!whole) {
        float* dst = p.ws_o + (static_cast<int64_t>(blockIdx.x) * 2 + piece) * (kN * 512) + hh * 256 + r;
#pragma unroll 1
        for (int j0 = 0; j0 < cols; j0 += kStage) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float v[kStage];
            tmem_load_cols<kStage>(ta + kColO + (hh * 2 + b) * kN + j0, v);
#pragma unroll
            for (int x = 0; x < kStage; ++x) dst[(j0 + x) * 512 + b * 128] = v[x];
          }
        }
      } else {
        // ---- output, 16 columns at a time: thread = dim, staged in the P buffer as words of
        // (column, column + 1), [8][512], read back eight dims a thread and stored 16 bytes a column
        uint32_t* stage = reinterpret_cast<uint32_t*>(ps);
#pragma unroll 1
        for (int j0 = 0; j0 < cols; j0 += kStage) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float v[kStage];
            tmem_load_cols<kStage>(ta + kColO + (hh * 2 + b) * kN + j0, v);
            const int d = (static_cast<int>(hh) * 2 + b) * 128 + r;
#pragma unroll
            for (int x = 0; x < kStage; ++x) v[x] *= fac[j0 + x];
            if (p.rope_cs != nullptr && d >= 512 - 64) {        // warp-uniform: dims (d, d ^ 1) are a pair, lanes (l, l ^ 1)
#pragma unroll
              for (int x = 0; x < kStage; ++x) {
                const float other = __shfl_xor_sync(0xffffffffu, v[x], 1);
                const int rr = it->rope[j0 + x];
                if (rr < 0) continue;
                const float2 cs = __ldg(reinterpret_cast<const float2*>(p.rope_cs) + static_cast<int64_t>(rr) * 32 + ((d - (512 - 64)) >> 1));
                v[x] = (lane & 1) ? fmaf(v[x], cs.x, -(other * cs.y)) : fmaf(v[x], cs.x, other * cs.y);
              }
            }
#pragma unroll
            for (int x = 0; x < kStage / 2; ++x) stage[x * 512 + d] = pack_bf16x2(v[2 * x], v[2 * x + 1]);
          }
          named_barrier_sync(kBarCompute, kComputeThreads);
#pragma unroll
          for (int i = 0; i < kStage / 8; ++i) {
            const int hp = (tid >> 6) + 4 * i, col = j0 + 2 * hp;   // columns col, col + 1; dims 8 (tid & 63) ..
            const uint4 a = *reinterpret_cast<const uint4*>(stage + hp * 512 + (tid & 63) * 8);
            const uint4 e = *reinterpret_cast<const uint4*>(stage + hp * 512 + (tid & 63) * 8 + 4);
            uint16_t* dst = p.out + (static_cast<int64_t>(row0) + col) * 512 + (tid & 63) * 8;
            if (col < cols)
              *reinterpret_cast<uint4*>(dst) = make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                                          __byte_perm(e.x, e.y, 0x5410), __byte_perm(e.z, e.w, 0x5410));
            if (col + 1 < cols)
              *reinterpret_cast<uint4*>(dst + 512) = make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                                                __byte_perm(e.x, e.y, 0x7632), __byte_perm(e.z, e.w, 0x7632));
          }
          named_barrier_sync(kBarCompute, kComputeThreads);      // the buffer has been read out
        }
      }
      tc_fence_before();                 // O has been read; the next item's PV follows its bar_p
      named_barrier_sync(kBarCompute, kComputeThreads);          // m_used, red and fac are free again
      if (lane == 0) mbar_arrive(bar_done + (n_item & 1));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of cut items (bound by the partial sums, 2 KB a column and piece, which are in
// L2, and for few items by its launch, 2 us).  Two columns a unit whatever the pieces, and every
// item cut, took 68.7 us for 128 items of six chunks; 33.8 with eight columns a unit and items left whole.
// A column's pieces are added up by one warp (lane l holding dims
// 4 l + 128 i) or, where there are many, by four: a unit is eight columns, or two.  The CTAs share
// out the units of all cut items.
constexpr int kMaxCtas = 160;
constexpr int kFewPieces = 8;
static_assert(kMaxCtas <= 256, "a thread of the joining kernel looks at one CTA's record");
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeParams p, int ctas) {
  __shared__ int32_t cut[kMaxCtas], units_to[kMaxCtas];   // CTA that cuts, units up to and with its item's
  __shared__ int32_t n_cut;
  __shared__ int2 sums[8];
  __shared__ float4 acc[8][128];
  griddep_launch();
  griddep_wait();
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  {
    const int4 rec = tid < ctas ? p.ws_cut[tid] : make_int4(0, 0, 0, 0);
    const bool has = rec.y > 0;
    const uint32_t bits = __ballot_sync(0xffffffffu, has);
    int u = has ? (rec.z - tid < kFewPieces ? (rec.y + 7) / 8 : (rec.y + 1) / 2) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, u, o);
      if (lane >= o) u += up;
    }
    if (lane == 31) sums[warp] = make_int2(__popc(bits), u);
    __syncthreads();
    int n = 0, units = 0, all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < warp) n += sums[i].x, units += sums[i].y;
      all += sums[i].x;
    }
    if (has) {
      const int at = n + __popc(bits & ((1u << lane) - 1u));
      cut[at] = tid;
      units_to[at] = units + u;
    }
    if (tid == 0) n_cut = all;
  }
  __syncthreads();
  const int n_units = n_cut > 0 ? units_to[n_cut - 1] : 0;
  int which = 0;
  for (int unit = blockIdx.x; unit < n_units; unit += gridDim.x) {
    while (units_to[which] <= unit) ++which;
    const int g0 = cut[which], in_item = unit - (which > 0 ? units_to[which - 1] : 0);
    const int4 rec = p.ws_cut[g0];
    const int last = rec.z, pieces = last - g0 + 1;
    const bool few = pieces <= kFewPieces;
    const int share = few ? 1 : 4;                         // warps of a column
    const int col = few ? in_item * 8 + warp : in_item * 2 + (warp >> 2);
    const int64_t row = static_cast<int64_t>(rec.x) + col;
    const bool live = col < rec.y;
    const int head = static_cast<int>(row % p.H), node = static_cast<int>(row / p.H);
    // piece i: the first lies in its CTA's second place, the others in the first place
    auto slot = [&](int i) { return (static_cast<int64_t>(g0 + i) * 2 + (i == 0 ? 1 : 0)) * kN + col; };
    float m = -1e30f;
    for (int i = lane; i < pieces; i += 32) {
      const float2 ml = p.ws_ml[slot(i)];
      if (!(ml.y == 0.f)) m = fmaxf(m, ml.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float sink2 = live ? __ldg(p.sink + head) * kLog2e : -INFINITY;
    const bool some = m > -1e30f;
    const float M = some ? fmaxf(m, sink2) : sink2;
    float l = 0.f;
    for (int i = lane; i < pieces; i += 32) {
      const float2 ml = p.ws_ml[slot(i)];
      if (!(ml.y == 0.f)) l += ml.y * ex2_approx(ml.x - M);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float L = l + (sink2 > -INFINITY ? ex2_approx(sink2 - M) : 0.f);
    float4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = few ? 0 : warp & 3; i < pieces; i += share) {
      const float2 ml = p.ws_ml[slot(i)];
      const float4* src = reinterpret_cast<const float4*>(p.ws_o + slot(i) * 512) + lane;
      float4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = __ldcs(src + 32 * j);
      if (ml.y == 0.f) continue;         // it has attended to nothing; its sums are zero
      const float f = ex2_approx(ml.x - M);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j].x = fmaf(x[j].x, f, v[j].x), v[j].y = fmaf(x[j].y, f, v[j].y);
        v[j].z = fmaf(x[j].z, f, v[j].z), v[j].w = fmaf(x[j].w, f, v[j].w);
      }
    }
    const float inv = L == 0.f ? 0.f : __fdividef(1.f, L);
    // four dims from 4 q on of this column
    auto put = [&](float4 s, int q) {
      s.x *= inv, s.y *= inv, s.z *= inv, s.w *= inv;
      if (p.rope_cs != nullptr && q >= 112) {
        const int rr = __ldg(p.rope_pos + node);
        if (rr >= 0 && rr < p.rope_rows) {                 // else flagged by the first kernel
          const float4 cs = __ldg(p.rope_cs + static_cast<int64_t>(rr) * 16 + (q - 112));
          const float2 a = rotate_back(s.x, s.y, cs.x, cs.y), b = rotate_back(s.z, s.w, cs.z, cs.w);
          s = make_float4(a.x, a.y, b.x, b.y);
        }
      }
      *reinterpret_cast<uint2*>(p.out + row * 512 + q * 4) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
      if (p.lse && q == 0) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    };
    if (few) {
      if (live)
#pragma unroll
        for (int j = 0; j < 4; ++j) put(v[j], lane + 32 * j);
      continue;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[warp][lane + 32 * j] = v[j];
    __syncthreads();
    // 128 threads a column: four dims each
    const int q = tid & 127;                               // tid >> 7 = warp >> 2, this thread's column as above
    float4 s = acc[warp & 4][q];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float4 x = acc[(warp & 4) + w][q];
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    if (live) put(s, q);
    __syncthreads();
  }
}

// idx[t][j < window] = slot of committed position pos - window + 1 + j, -1 outside [0, ctx);
// idx[t][window + j] = draft_entry + j for the drafted rows j that node t sees, else -1.
__global__ void tree_window_kernel(const TreeParams p, int32_t* __restrict__ idx, int64_t stride) {
  griddep_launch();
  griddep_wait();
  int s0;
  const int nodes = nodes_of(p, static_cast<int>(blockIdx.x), s0, threadIdx.x == 0 && blockIdx.y == 0);
  const int ctx = __ldg(p.ctx + blockIdx.x);
  for (int node = static_cast<int>(blockIdx.y); node < nodes; node += gridDim.y) {
    const int64_t pos = __ldg(p.pos + s0 + node);
    const uint64_t anc = ancestors_of(p, s0, node, nodes);
    int32_t* row = idx + static_cast<int64_t>(s0 + node) * stride;
    for (int j = static_cast<int>(threadIdx.x); j < p.window + p.max_nodes; j += static_cast<int>(blockDim.x)) {
      int32_t e;
      if (j < p.window) {
        const int64_t at = pos - p.window + 1 + j;
        e = at < 0 || at >= ctx ? -1 : static_cast<int32_t>(p.win_ring > 0 ? at % p.win_ring : at);
      } else {
        e = anc >> (j - p.window) & 1 ? p.draft_entry + (j - p.window) : -1;
      }
      row[j] = e;
    }
  }
}

// CTAs of a call at most: one for each chunk that sequences of n_max entries, a window and all
// nodes would have, and no more than the device (or the workspace) holds.
int64_t ctas_for(int64_t n_seqs, int64_t max_nodes, int64_t H, int64_t n_max, int64_t window) {
  const int64_t blocks = (max_nodes * H + kN - 1) / kN, chunks = (n_max + window + max_nodes + kRows - 1) / kRows;
  const int64_t all = n_seqs * blocks * (chunks > 0 ? chunks : 1);
  return all < kMaxCtas ? all : kMaxCtas;
}
constexpr size_t kCtaBytes = 2 * kN * (512 * 4 + 8) + 16;

}  // namespace

size_t tree_attn_workspace(int32_t n_seqs, int32_t max_nodes, int32_t H, int32_t n_max, int32_t window) {
  return static_cast<size_t>(ctas_for(n_seqs, max_nodes, H, n_max, window)) * kCtaBytes;
}

int launch_tree_attn(const dsv4sa_tree_args* a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  TreeParams p{};
  p.q = static_cast<const uint16_t*>(a->q);
  p.sink = a->attn_sink;
  p.node_start = a->node_start;
  p.seq_row = a->seq_row;
  p.ctx = a->ctx;
  p.pos = a->pos;
  p.anc = a->anc;
  p.n_vis = a->n_vis;
  bool fp4 = false;
  if (a->n_max > 0) {
    fp4 = a->comp->kind == DSV4SA_POOL_KV_FP4;
    p.comp_base = static_cast<const uint8_t*>(a->comp->base);
    p.comp_page_stride = a->comp->page_stride;
    p.comp_num_pages = a->comp->num_pages;
    p.comp_pt = a->comp_pt;
    p.comp_pt_stride = a->comp_pt_stride;
    p.comp_pt_rows = a->comp_pt_rows > 0 ? a->comp_pt_rows : INT32_MAX;
  }
  if (a->window > 0 || a->draft_entry >= 0) {
    fp4 = a->win->kind == DSV4SA_POOL_KV_FP4;
    p.win_base = static_cast<const uint8_t*>(a->win->base);
    p.win_page_stride = a->win->page_stride;
    p.win_num_pages = a->win->num_pages;
    p.win_pt = a->win_pt;
    p.win_pt_stride = a->win_pt_stride;
    p.win_pt_rows = a->win_pt_rows > 0 ? a->win_pt_rows : INT32_MAX;
  }
  p.rope_cs = reinterpret_cast<const float4*>(a->rope_cs);
  p.rope_pos = a->rope_pos;
  p.rope_rows = a->rope_rows;
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  const int64_t most = ctas_for(a->n_seqs, a->max_nodes, a->H, a->n_max, a->window);
  const int ctas = static_cast<int>(most < sms ? most : sms);
  uint8_t* ws = static_cast<uint8_t*>(a->ws);
  p.ws_o = reinterpret_cast<float*>(ws);
  p.ws_ml = reinterpret_cast<float2*>(ws + static_cast<size_t>(ctas) * 2 * kN * 512 * 4);
  p.ws_cut = reinterpret_cast<int4*>(ws + static_cast<size_t>(ctas) * 2 * kN * (512 * 4 + 8));
  p.n_max = a->n_max;
  p.window = a->window;
  p.win_ring = a->win_ring;
  p.draft_entry = a->draft_entry;
  p.B = a->n_seqs;
  p.T = a->T;
  p.H = a->H;
  p.max_nodes = a->max_nodes;
  p.blocks = (a->max_nodes * a->H + kN - 1) / kN;
  p.scale_log2 = a->softmax_scale * kLog2e;
  const auto kernel = fp4 ? tree_attn_kernel<true> : tree_attn_kernel<false>;
  if (!smem_attr_once(dev, fp4 ? 17 : 16, reinterpret_cast<const void*>(kernel), SmemT::kBytes + 1024)) return DSV4SA_ERR_CUDA;
  if (launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreadsT), SmemT::kBytes + 1024, stream, p) != cudaSuccess)
    return DSV4SA_ERR_CUDA;
  if (ctas == 1) return DSV4SA_OK;       // nothing can be cut
  return launch_pdl(tree_merge_kernel, dim3(static_cast<unsigned>(4 * sms)), dim3(256), 0, stream, p, ctas) == cudaSuccess ? DSV4SA_OK
                                                                                                                          : DSV4SA_ERR_CUDA;
}

int launch_tree_window_indices(const int32_t* node_start, const int32_t* ctx, const int32_t* pos, const uint64_t* anc, int32_t n_seqs,
                               int32_t T, int32_t max_nodes, int32_t window, int32_t ring, int32_t draft_entry, int32_t* idx_w,
                               int64_t idx_stride, cudaStream_t stream) {
  TreeParams p{};
  p.node_start = node_start;
  p.ctx = ctx;
  p.pos = pos;
  p.anc = anc;
  p.B = n_seqs;
  p.T = T;
  p.max_nodes = max_nodes;
  p.window = window;
  p.win_ring = ring;
  p.draft_entry = draft_entry;
  const unsigned y = static_cast<unsigned>(max_nodes < 1 ? 1 : max_nodes);
  return launch_pdl(tree_window_kernel, dim3(static_cast<unsigned>(n_seqs), y), dim3(128), 0, stream, p, idx_w, idx_stride) == cudaSuccess
             ? DSV4SA_OK
             : DSV4SA_ERR_CUDA;
}

uint32_t* error_word_attn_tree() { return error_word(); }

}  // namespace dsv4sa
