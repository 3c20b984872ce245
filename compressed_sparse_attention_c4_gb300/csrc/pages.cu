// pages.cu -- the pages of a cache: copied, shared by forks, released, compacted.
//
// A cache is up to four pools that share page ids ("DeepSeek-V4 in SGLang" 概念5
// DeepSeekV4TokenToKVPool: a paged pool; a sequence's KV rows and its indexer
// keys lie in the same page of two pools), one page table and one use count per
// page: how many table entries hold it, 0 for a free page.  All of it lives on
// the device, so a beam step or a clean-up costs the host no round trip.
//
// Everything here moves bytes: the bound is HBM for whole pages (compacting 29490 pages of
// 27904 bytes takes 244 us, the measured copy bandwidth; copying 16000 of them by a list
// 139, 6.4 TB/s) and latency for a few table rows (four forks of one sequence, released
// before, 8.0 us in two kernels; 256 forks of 64 sequences 13.6, their bytes 2).  Two plans
// are one CTA's walk over the use counts and grow with the pool: the search for free pages
// takes 155 us for each million pages in use below the first free one, the plan of a compaction
// in place 1.0 ms for each million pages.  Counts are 32-bit integers changed by atomic additions,
// whose order does not change the result; page ids are handed out by scans in
// id order, so a call gives the same ids every time.
#include "common.cuh"
#include "dsv4sa_internal.h"

namespace dsv4sa {
namespace {

constexpr int kPage = DSV4SA_PAGE_SIZE;
constexpr int kMaxPools = DSV4SA_MAX_POOLS;
constexpr int kCopyThreads = 256;
constexpr int kForkBatch = 4;      // 16-byte units a thread has in flight in a fork's copy

struct PoolBytes {
  uint8_t* base;
  int64_t stride;        // bytes of a page (a multiple of 256)
  int32_t off[3];        // the page's blocks: byte offset, bytes per slot
  int32_t row[3];
};

struct CacheParams {
  PoolBytes pool[kMaxPools];
  int32_t n_pools;
  int32_t rows;
  int32_t pt_stride;
  int32_t num_pages;
  int32_t* pt;
  int32_t* use;
};

// Copy `units` 16-byte units, up to eight loads in flight per thread (a page is five
// to ten units a thread, so a loop of whole batches alone would run one at a time).
__device__ __forceinline__ void copy_units(uint4* dst, const uint4* src, int units, int tid, int threads) {
  for (int u0 = tid; u0 < units; u0 += 8 * threads) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (u0 + i * threads < units) v[i] = __ldcs(src + u0 + i * threads);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (u0 + i * threads < units) __stcs(dst + u0 + i * threads, v[i]);
  }
}

// Page `to` of every pool of d = page `from` of s's, by a CTA: one list of 16-byte
// units over the pools, eight in flight a thread (a compaction that took 370 us with one
// in flight took 294 so, before the grid of launch_cache_compact).
__device__ __forceinline__ void copy_page(const CacheParams& d, int64_t to, const CacheParams& s, int64_t from, int tid) {
  int total = 0;
  for (int k = 0; k < s.n_pools; ++k) total += static_cast<int>(s.pool[k].stride / 16);
  for (int u0 = tid; u0 < total; u0 += 8 * kCopyThreads) {
    uint4 v[8];
    uint4* dst[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int at = u0 + i * kCopyThreads;
      if (at >= total) continue;
      int k = 0;
      for (; at >= static_cast<int>(s.pool[k].stride / 16); ++k) at -= static_cast<int>(s.pool[k].stride / 16);
      dst[i] = reinterpret_cast<uint4*>(d.pool[k].base + to * d.pool[k].stride) + at;
      v[i] = __ldcs(reinterpret_cast<const uint4*>(s.pool[k].base + from * s.pool[k].stride) + at);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (u0 + i * kCopyThreads < total) __stcs(dst[i], v[i]);
  }
}

// Exclusive scan over the 1024 threads of a CTA; returns the total.
__device__ __forceinline__ int scan1024(int v, int* buf, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  const int w = buf[lane];
  int wx = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, wx, o);
    if (lane >= o) wx += y;
  }
  total = __shfl_sync(0xffffffffu, wx, 31);
  const int before = __shfl_sync(0xffffffffu, wx - w, warp);
  __syncthreads();
  return before + x - v;
}

// Eight use counts, from page q0 on (a multiple of four): a bit for each page in use.
__device__ __forceinline__ uint32_t used_bits(const CacheParams& p, int q0) {
  uint32_t bits = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int q = q0 + 4 * h;
    int4 c = make_int4(0, 0, 0, 0);
    if (q + 3 < p.num_pages) {
      c = *reinterpret_cast<const int4*>(p.use + q);
    } else {
      if (q < p.num_pages) c.x = p.use[q];
      if (q + 1 < p.num_pages) c.y = p.use[q + 1];
      if (q + 2 < p.num_pages) c.z = p.use[q + 2];
    }
    bits |= static_cast<uint32_t>((c.x > 0) | ((c.y > 0) << 1) | ((c.z > 0) << 2) | ((c.w > 0) << 3)) << (4 * h);
  }
  return bits;
}
// ... and for each free page that there is.
__device__ __forceinline__ uint32_t free_bits(const CacheParams& p, int q0) {
  const int in = max(0, min(8, p.num_pages - q0));
  return ~used_bits(p, q0) & ((1u << in) - 1u);
}

// ---------------------------------------------------------------- copy
// Page dst[i] = page src[i] of every pool.  grid (n, pieces): a piece is a
// contiguous share of each page.
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const CacheParams p, const int32_t* src,
                                                                  const int32_t* dst, int pieces) {
  griddep_launch();
  griddep_wait();
  const int i = blockIdx.x / pieces, piece = blockIdx.x % pieces;
  const int32_t a = __ldg(src + i), b = __ldg(dst + i);
  if (a == -1 || b == -1) return;
  if (a < 0 || b < 0 || a >= p.num_pages || b >= p.num_pages) {
    if (threadIdx.x == 0 && piece == 0) raise_error(kErrIndex);
    return;
  }
  if (a == b) return;
  for (int k = 0; k < p.n_pools; ++k) {
    const int units = static_cast<int>(p.pool[k].stride / 16);
    const int u0 = units * piece / pieces, u1 = units * (piece + 1) / pieces;
    copy_units(reinterpret_cast<uint4*>(p.pool[k].base + b * p.pool[k].stride) + u0,
               reinterpret_cast<const uint4*>(p.pool[k].base + a * p.pool[k].stride) + u0, u1 - u0, threadIdx.x,
               kCopyThreads);
  }
}

// ---------------------------------------------------------------- release
__global__ void __launch_bounds__(kCopyThreads) cache_release_kernel(const CacheParams p, const int32_t* rows, int n) {
  griddep_launch();
  griddep_wait();
  const int64_t total = static_cast<int64_t>(n) * p.pt_stride;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
    const int64_t i = e / p.pt_stride, j = e - i * p.pt_stride;
    const int32_t row = __ldg(rows + i);
    if (row < 0 || row >= p.rows) {
      if (j == 0 && row != -1) raise_error(kErrIndex);
      continue;
    }
    int32_t* at = p.pt + static_cast<int64_t>(row) * p.pt_stride + j;
    if (*at == -1) continue;
    const int32_t page = atomicExch(at, -1);   // a row named twice is released once
    if (page < 0 || page >= p.num_pages) {
      if (page != -1) raise_error(kErrIndex);
      continue;
    }
    if (atomicSub(p.use + page, 1) <= 0) {     // the page was free: keep its count
      atomicAdd(p.use + page, 1);
      raise_error(kErrIndex);
    }
  }
}

// ---------------------------------------------------------------- fork
struct ForkParams {
  const int32_t* src;
  const int32_t* dst;
  const int32_t* len;
  int32_t* new_page;      // >= 0 the copied page, -1 none needed, kRefused, kUntouched
  int32_t n;
};

constexpr int kRefused = -2;     // no page for it: its row stays empty
constexpr int kUntouched = -3;   // its arguments are refused: its row stays as it is
constexpr int kAllocThreads = 1024;
constexpr int kAllocChunk = 8 * kAllocThreads;

// Hands out pages: fork i whose length ends inside a page gets the lowest free
// page not given to an earlier fork.  One CTA walks the use counts in id order,
// 8192 at a time, and stops as soon as every fork is served.  A fork first
// claims its row: the row must be empty (first entry negative), and of two forks
// into one row the first one has it -- the claim is the fork's number, offset to
// be the smaller the earlier, put into the row's first entry by an atomic
// minimum.  A parent that is a row of this same call is thereby empty, too, and
// refused.
__device__ __forceinline__ void fork_alloc(const CacheParams& p, const ForkParams& f) {   // by a CTA of kAllocThreads
  __shared__ int buf[32];
  __shared__ int32_t free_ids[kAllocChunk];
  const int tid = static_cast<int>(threadIdx.x);
  int avail = 0, pos = 0, next = 0;            // ids listed, ids given out, next page to look at
  uint32_t ready = free_bits(p, tid * 8);      // the first chunk's free pages, while the forks are looked at
  for (int i0 = 0; i0 < f.n; i0 += kAllocThreads) {
    const int i = i0 + tid;
    int state = -1;                            // -1 nothing to copy, 1 a page wanted, or a refusal
    int32_t* claim = nullptr;
    if (i < f.n) {
      const int32_t s = __ldg(f.src + i), d = __ldg(f.dst + i), len = __ldg(f.len + i);
      bool ok = s >= 0 && s < p.rows && d >= 0 && d < p.rows && s != d && len >= 0 &&
                len <= static_cast<int64_t>(p.pt_stride) * kPage;
      if (ok && len > 0) {
        const int32_t* srow = p.pt + static_cast<int64_t>(s) * p.pt_stride;
        const int32_t last = __ldcg(srow + (len - 1) / kPage);
        ok = __ldcg(srow) >= 0 && last >= 0 && last < p.num_pages;
      }
      if (ok) {
        claim = p.pt + static_cast<int64_t>(d) * p.pt_stride;
        if (__ldcg(claim) < 0) atomicMin(claim, INT32_MIN + i);
        else ok = false;
      }
      state = !ok ? kUntouched : (len % kPage != 0 ? 1 : -1);
    }
    __syncthreads();                           // every claim of this batch is made
    if (state != kUntouched && claim != nullptr && __ldcg(claim) != INT32_MIN + i) state = kUntouched;
    if (state == kUntouched) raise_error(kErrIndex);
    int wanted;
    const int rank = scan1024(state == 1 ? 1 : 0, buf, wanted);
    int given = 0;
    int32_t mine = state == 1 ? kRefused : state;    // until a page is found for it
    while (given < wanted) {                   // uniform: every bound here is the CTA's
      if (pos == avail) {
        if (next >= p.num_pages) {
          if (tid == 0) raise_error(kErrPages);
          break;
        }
        const int q0 = next + tid * 8;
        const uint32_t bits = next == 0 ? ready : free_bits(p, q0);
        int at = scan1024(__popc(bits), buf, avail);
#pragma unroll
        for (int h = 0; h < 8; ++h)
          if (bits >> h & 1) free_ids[at++] = q0 + h;
        pos = 0;
        next += kAllocChunk;
        __syncthreads();
        continue;
      }
      const int take = min(wanted - given, avail - pos);
      if (state == 1 && rank >= given && rank < given + take) mine = free_ids[pos + rank - given];
      given += take;
      pos += take;
      __syncthreads();                         // the list is read before it is filled again
    }
    if (i < f.n) {
      f.new_page[i] = mine;
      if (mine >= 0) p.use[mine] = 1;          // never looked at again in this call: ids only go up
    }
    __syncthreads();
  }
}

// Piece `piece` of `pieces` of fork i, by a CTA of kThreads: the row of dst is the parent's
// full pages (their counts go up) and the new page, whose first len % 64 slots are copied.
template <int kThreads>
__device__ __forceinline__ void fork_rows(const CacheParams& p, const ForkParams& f, int i, int piece, int pieces) {
  const int tid = static_cast<int>(threadIdx.x);
  const int32_t d = __ldg(f.dst + i), s = __ldg(f.src + i), len = __ldg(f.len + i), page = f.new_page[i];
  if (page == kUntouched) return;              // flagged by the first kernel
  int32_t* drow = p.pt + static_cast<int64_t>(d) * p.pt_stride;
  if (page == kRefused) {                      // only the claim was written
    if (piece == 0 && tid == 0) drow[0] = -1;
    return;
  }
  const int32_t* srow = p.pt + static_cast<int64_t>(s) * p.pt_stride;
  const int full = len / kPage, slots = len % kPage;
  // The used slots of the last page, the blocks of all pools as one list of 16-byte
  // units (the last of a block may hold 4, 8 or 12 bytes more than the block: its
  // remainder is copied in words), so that one batch of loads covers a CTA's share.
  // The loads go out first, then the table is written, then the stores follow.
  int64_t from = 0;
  int total = 0;
  if (page >= 0) {
    from = srow[full];
    for (int k = 0; k < p.n_pools; ++k)
#pragma unroll
      for (int b = 0; b < 3; ++b) total += (slots * p.pool[k].row[b] + 15) / 16;
  }
  const int u_end = total * (piece + 1) / pieces;
  int u = total * piece / pieces + tid;
  bool table_done = false;
  do {
    uint4 v[kForkBatch];
    uint8_t* to[kForkBatch];
    int bytes[kForkBatch];
#pragma unroll
    for (int i = 0; i < kForkBatch; ++i) {
      bytes[i] = 0;
      int at = u + i * kThreads;
      if (at >= u_end) continue;
      for (int k = 0; k < p.n_pools && bytes[i] == 0; ++k) {
#pragma unroll
        for (int b = 0; b < 3; ++b) {
          const int n = slots * p.pool[k].row[b], units = (n + 15) / 16;
          if (bytes[i] == 0 && at < units) {
            const int64_t off = p.pool[k].off[b] + 16 * static_cast<int64_t>(at);
            const uint8_t* fr = p.pool[k].base + from * p.pool[k].stride + off;
            to[i] = p.pool[k].base + page * p.pool[k].stride + off;
            bytes[i] = min(16, n - 16 * at);
            v[i] = __ldcs(reinterpret_cast<const uint4*>(fr));   // blocks end on 16 bytes: in the page
          }
          at -= units;
        }
      }
    }
    if (!table_done) {
      for (int j = piece * kThreads + tid; j < p.pt_stride; j += pieces * kThreads) {
        int32_t e = -1;
        if (j < full) {
          e = srow[j];
          if (e < 0 || e >= p.num_pages) {
            raise_error(kErrIndex);
            e = -1;
          } else {
            atomicAdd(p.use + e, 1);
          }
        } else if (j == full && slots > 0) {
          e = page;
        }
        drow[j] = e;
      }
      table_done = true;
    }
#pragma unroll
    for (int i = 0; i < kForkBatch; ++i) {
      if (bytes[i] == 16) {
        __stcs(reinterpret_cast<uint4*>(to[i]), v[i]);
      } else if (bytes[i] > 0) {           // row sizes are multiples of 4
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int x = 0; x < 3; ++x)
          if (4 * x < bytes[i]) reinterpret_cast<uint32_t*>(to[i])[x] = w[x];
      }
    }
    u += kForkBatch * kThreads;
  } while (u - tid < u_end);               // the same for all threads
}

__global__ void __launch_bounds__(kAllocThreads) cache_fork_alloc_kernel(const CacheParams p, const ForkParams f) {
  griddep_launch();
  griddep_wait();
  fork_alloc(p, f);
}
__global__ void __launch_bounds__(kCopyThreads) cache_fork_kernel(const CacheParams p, const ForkParams f, int pieces) {
  griddep_launch();
  griddep_wait();
  fork_rows<kCopyThreads>(p, f, blockIdx.x / pieces, blockIdx.x % pieces, pieces);
}
// Both in one kernel for up to eight forks, a cluster of CTAs: the first hands the pages out,
// then all of them copy.  The device takes as long (8 forks 7.9 us, 8.2 in two kernels), the
// host 2 us less; 16 forks took 10.5 us against 8.4.
constexpr int kForkCtas = 8;
__global__ void __launch_bounds__(kAllocThreads) cache_fork_few_kernel(const CacheParams p, const ForkParams f, int pieces) {
  griddep_launch();
  griddep_wait();
  const int r = static_cast<int>(cluster_ctarank());
  if (r == 0) fork_alloc(p, f);
  cluster_sync();                              // what the first CTA wrote is seen by the others
  for (int k = r; k < f.n * pieces; k += kForkCtas) fork_rows<kAllocThreads>(p, f, k / pieces, k % pieces, pieces);
}

// ---------------------------------------------------------------- compact
struct CompactParams {
  CacheParams src;
  CacheParams dst;
  int32_t* new_id;        // [src.num_pages]
  int32_t* n_used;
  int32_t in_place;
};

// new_id of every page when they go to other pools: the rank among the pages in use
// (-1 for a free page, or one that does not fit).  A cluster of eight CTAs, each with a
// contiguous share of the counts: it counts its pages in use, learns the counts before
// it through distributed shared memory, and ranks its pages.
constexpr int kPlanCtas = 8;

__global__ void __launch_bounds__(kAllocThreads) cache_plan_kernel(const CompactParams c) {
  __shared__ int buf[32];
  __shared__ int counts[kPlanCtas];
  griddep_launch();
  griddep_wait();
  const int tid = static_cast<int>(threadIdx.x), r = static_cast<int>(cluster_ctarank());
  const int P = c.src.num_pages;
  const int share = ((P + kPlanCtas - 1) / kPlanCtas + 7) & ~7;
  const int p0 = min(P, r * share), p1 = min(P, p0 + share);   // p0 a multiple of 8, or P
  auto bits_at = [&](int q0) {                                 // of the thread's eight pages inside the share
    return q0 < p1 ? used_bits(c.src, q0) & ((1u << min(8, p1 - q0)) - 1u) : 0u;
  };
  const uint32_t first = bits_at(p0 + tid * 8);                // most shares are one chunk: read once
  int mine = __popc(first), total;
  for (int q0 = p0 + kAllocChunk + tid * 8; q0 < p1; q0 += kAllocChunk) mine += __popc(bits_at(q0));
  scan1024(mine, buf, total);
  cluster_sync();                              // every CTA runs before its shared memory is written
  if (tid < kPlanCtas) st_cluster_u32(cluster_map(smem_u32(counts + r), static_cast<uint32_t>(tid)), static_cast<uint32_t>(total));
  cluster_sync();
  int base = 0, all = 0;
#pragma unroll
  for (int k = 0; k < kPlanCtas; ++k) {
    base += k < r ? counts[k] : 0;
    all += counts[k];
  }
  for (int c0 = p0; c0 < p1; c0 += kAllocChunk) {
    const int q0 = c0 + tid * 8;
    const uint32_t bits = c0 == p0 ? first : bits_at(q0);
    int t;
    int rank = base + scan1024(__popc(bits), buf, t);
    base += t;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (q0 + k >= p1) continue;
      int id = -1;
      if (bits >> k & 1u) {
        id = rank < c.dst.num_pages ? rank : -1;
        if (id >= 0) c.dst.use[id] = q0 + k;   // until the page is moved: which one goes there
        ++rank;
      }
      c.new_id[q0 + k] = id;
    }
  }
  if (r == 0 && tid == 0) {
    *c.n_used = all;
    if (all > c.dst.num_pages) raise_error(kErrPages);
  }
}

// ... and in place, by one CTA: pages below the number in use stay, the k-th one at or
// above it goes to the k-th free page below it.  The free pages' list is kept in
// new_id[n_used ..] until its entries are replaced: the k-th page to move has an id of
// at least n_used + k, so the chunks are walked from the highest ids down and an
// entry is read before anything at or above its place is written.
__global__ void __launch_bounds__(kAllocThreads) cache_plan_in_place_kernel(const CompactParams c) {
  __shared__ int buf[32];
  griddep_launch();
  griddep_wait();
  const int tid = static_cast<int>(threadIdx.x);
  const int P = c.src.num_pages;
  int total = 0, mine = 0;
  for (int q0 = tid * 8; q0 < P; q0 += kAllocChunk) mine += __popc(used_bits(c.src, q0));
  scan1024(mine, buf, total);
  int holes = 0;
  for (int c0 = 0; c0 < total; c0 += kAllocChunk) {
    const int q0 = c0 + tid * 8;
    const uint32_t bits = used_bits(c.src, q0), mask = (1u << max(0, min(8, total - q0))) - 1u;
    int t;
    int h = holes + scan1024(__popc(~bits & mask), buf, t);
    holes += t;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (!(mask >> k & 1u)) continue;
      const bool used = bits >> k & 1u;
      c.new_id[q0 + k] = used ? q0 + k : -1;
      if (!used) c.new_id[total + h++] = q0 + k;   // as many pages in use lie above: in range
    }
  }
  __syncthreads();
  int left = holes;                            // pages at or above n_used not yet given their place
  const int n_above = P - total;
  for (int c0 = n_above > 0 ? (n_above - 1) / kAllocChunk * kAllocChunk : -1; c0 >= 0; c0 -= kAllocChunk) {
    const int q0 = total + c0 + tid * 8;       // not a multiple of four: single loads
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) bits |= (q0 + k < P && c.src.use[q0 + k] > 0 ? 1u : 0u) << k;
    int t;
    const int before = scan1024(__popc(bits), buf, t);
    int r = left - t + before;                 // rank of the thread's first page to move
    int32_t id[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) id[k] = bits >> k & 1u ? c.new_id[total + r++] : -1;
    __syncthreads();                           // this chunk's list entries are read before they are replaced
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (q0 + k < P) c.new_id[q0 + k] = id[k];
    left -= t;
  }
  if (tid == 0) *c.n_used = total;
}

// Moves the pages to their new ids and rewrites the table and the counts.
__global__ void __launch_bounds__(kCopyThreads) cache_move_kernel(const CompactParams c) {
  griddep_launch();
  griddep_wait();
  const int tid = static_cast<int>(threadIdx.x);
  const int64_t thread = static_cast<int64_t>(blockIdx.x) * kCopyThreads + tid;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * kCopyThreads;
  const int64_t entries = static_cast<int64_t>(c.src.rows) * c.src.pt_stride;
  for (int64_t e = thread; e < entries; e += threads) {
    const int32_t t = c.src.pt[e];
    int32_t id = -1;
    if (t >= 0 && t < c.src.num_pages) id = __ldg(c.new_id + t);
    else if (t != -1) raise_error(kErrIndex);
    c.dst.pt[e] = id;
  }
  if (!c.in_place) {
    // ranks, not pages, are dealt out, so that every CTA copies as much; the plan has
    // left each rank's page where its count will be
    const int used = min(*c.n_used, c.dst.num_pages);
    for (int64_t q = thread; q < c.dst.num_pages; q += threads)
      if (q >= used) c.dst.use[q] = 0;
    int id = blockIdx.x;
    int q = id < used ? c.dst.use[id] : 0;
    for (; id < used; id += gridDim.x) {
      const int ahead = id + static_cast<int>(gridDim.x);
      const int q_next = ahead < used ? c.dst.use[ahead] : 0;
      __syncthreads();                         // every thread has q, read before, when the count replaces it
      if (tid == 0) c.dst.use[id] = c.src.use[q];
      copy_page(c.dst, id, c.src, q, tid);
      q = q_next;
    }
    return;
  }
  for (int q = blockIdx.x; q < c.src.num_pages; q += gridDim.x) {
    const int32_t id = __ldg(c.new_id + q);
    if (id < 0 || id == q) continue;
    copy_page(c.dst, id, c.src, q, tid);
    if (tid == 0) {
      c.dst.use[id] = c.src.use[q];
      c.src.use[q] = 0;
    }
  }
}

void fill_pools(const dsv4sa_pool_desc* pools, int32_t n_pools, CacheParams& p) {
  p.n_pools = n_pools;
  p.num_pages = static_cast<int32_t>(pools[0].num_pages);
  for (int k = 0; k < n_pools; ++k) {
    const dsv4sa_pool_desc& d = pools[k];
    PoolBytes& b = p.pool[k];
    b.base = static_cast<uint8_t*>(d.base);
    b.stride = d.page_stride;
    b.off[0] = static_cast<int32_t>(d.nope_off), b.row[0] = d.nope_row;
    b.off[1] = static_cast<int32_t>(d.rope_off), b.row[1] = d.rope_row;
    b.off[2] = static_cast<int32_t>(d.scale_off), b.row[2] = d.scale_row;
  }
}

void fill_cache(const dsv4sa_cache_desc* c, CacheParams& p) {
  fill_pools(c->pools, c->n_pools, p);
  p.rows = c->rows;
  p.pt_stride = c->pt_stride;
  p.pt = c->page_table;
  p.use = c->use;
}

int sm_count(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSV4SA_ERR_CUDA;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? DSV4SA_OK : DSV4SA_ERR_CUDA;
}

// CTAs that share one page's copy: enough that n pages fill the GPU, at most 8
// (a share of a few kilobytes).
int copy_pieces(int64_t n, int sms) {
  int pieces = 1;
  while (pieces < 8 && n * pieces < 4 * static_cast<int64_t>(sms)) pieces *= 2;
  return pieces;
}

int done(cudaError_t e) { return e == cudaSuccess ? DSV4SA_OK : DSV4SA_ERR_CUDA; }

}  // namespace

int launch_pages_copy(const dsv4sa_pool_desc* pools, int32_t n_pools, const int32_t* src, const int32_t* dst, int32_t n,
                      cudaStream_t stream) {
  CacheParams p{};
  fill_pools(pools, n_pools, p);
  int sms = 0;
  if (const int rc = sm_count(&sms); rc != DSV4SA_OK) return rc;
  const int pieces = copy_pieces(n, sms);
  return done(launch_pdl(pages_copy_kernel, dim3(static_cast<unsigned>(static_cast<int64_t>(n) * pieces)),
                         dim3(kCopyThreads), 0, stream, p, src, dst, pieces));
}

int launch_cache_release(const dsv4sa_cache_desc* c, const int32_t* rows, int32_t n, cudaStream_t stream) {
  CacheParams p{};
  fill_cache(c, p);
  int sms = 0;
  if (const int rc = sm_count(&sms); rc != DSV4SA_OK) return rc;
  const int64_t want = (static_cast<int64_t>(n) * p.pt_stride + kCopyThreads - 1) / kCopyThreads;
  const int64_t full = static_cast<int64_t>(sms) * 8;
  return done(launch_pdl(cache_release_kernel, dim3(static_cast<unsigned>(want < full ? want : full)),
                         dim3(kCopyThreads), 0, stream, p, rows, n));
}

int launch_cache_fork(const dsv4sa_cache_desc* c, const int32_t* src, const int32_t* dst, const int32_t* len, int32_t n,
                      int32_t* new_page, cudaStream_t stream) {
  CacheParams p{};
  fill_cache(c, p);
  const ForkParams f{src, dst, len, new_page, n};
  int sms = 0;
  if (const int rc = sm_count(&sms); rc != DSV4SA_OK) return rc;
  if (n <= kForkCtas) {
    int few = 1;                               // pieces of a fork, so that every CTA has one
    while (few < kForkCtas && n * few < kForkCtas) few *= 2;
    return done(launch_cluster_pdl(cache_fork_few_kernel, dim3(kForkCtas), dim3(kAllocThreads), 0, kForkCtas, stream, p, f, few));
  }
  if (launch_pdl(cache_fork_alloc_kernel, dim3(1), dim3(kAllocThreads), 0, stream, p, f) != cudaSuccess)
    return DSV4SA_ERR_CUDA;
  const int pieces = copy_pieces(n, sms);
  return done(launch_pdl(cache_fork_kernel, dim3(static_cast<unsigned>(static_cast<int64_t>(n) * pieces)),
                         dim3(kCopyThreads), 0, stream, p, f, pieces));
}

int launch_cache_compact(const dsv4sa_cache_desc* src, const dsv4sa_cache_desc* dst, int32_t* new_id, int32_t* n_used,
                         cudaStream_t stream) {
  CompactParams c{};
  fill_cache(src, c.src);
  fill_cache(dst, c.dst);
  c.new_id = new_id;
  c.n_used = n_used;
  c.in_place = src->pools[0].base == dst->pools[0].base;
  int sms = 0;
  if (const int rc = sm_count(&sms); rc != DSV4SA_OK) return rc;
  if ((c.in_place ? launch_pdl(cache_plan_in_place_kernel, dim3(1), dim3(kAllocThreads), 0, stream, c)
                  : launch_cluster_pdl(cache_plan_kernel, dim3(kPlanCtas), dim3(kAllocThreads), 0, kPlanCtas, stream, c)) !=
      cudaSuccess)
    return DSV4SA_ERR_CUDA;
  // far more CTAs than run at once, a page or two each: those that run then differ in where
  // they are, and none is left with more to do (29490 pages: 244 us; 8 CTAs an SM, all
  // resident, 275, 32 an SM 251, one for every page 259)
  const int64_t full = static_cast<int64_t>(sms) * 128;
  const int64_t want = c.src.num_pages;
  return done(launch_pdl(cache_move_kernel, dim3(static_cast<unsigned>(want < full ? want : full)), dim3(kCopyThreads),
                         0, stream, c));
}

uint32_t read_error_word_pages(cudaStream_t stream, bool clear) {
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
