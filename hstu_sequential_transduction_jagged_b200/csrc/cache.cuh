// The paged history cache: page bookkeeping (reserve with copy on write, fork,
// release, compact) and the row movers (append, gather).
//
// A layer's K and V live in pages of `ps` events, head-major inside a page:
// kv[layer][page][K or V][head][slot][64], so that one head's slice of a page is
// one contiguous block (ps * 128 bytes in 16 bits): the unit the attention kernels
// load, and a page is one contiguous block for the page copies.  Timestamps are
// paged the same way, once for all layers.  A sequence is a row of block_table
// (page of events b * ps .. ; -1 = no page) and a length; a page belongs to
// ref_count[page] sequences, and a page is free exactly when its count is zero.
// There is no free list to keep: an allocation takes the lowest free page ids, found by
// a scan of ref_count, so what a call hands out depends on the counts alone.
//
// The bookkeeping of reserve and compact runs as one CTA (chains of scans over a few
// thousand integers: latency, not bandwidth) and leaves copy lists in the caller's
// workspace; the copies run as a second launch over all SMs.  Measured (B200, 4
// layers, 8 heads): release + fork + reserve of 256 branches of 32 users 35 us, of
// which 21 us copy 69 MB of partial pages (the copy bandwidth); compact 151 us for
// 464 MB of pages (6.1 TB/s read and written); append 5.8 and gather 6.5 TB/s.
// The scans grow with the pool: where only the last 64 pages are free, a reservation of
// 64 events takes 6 us in 4,000 pages, 15 in 40,000 and 51 in 200,000, and a compact that
// moves nothing 6, 42 and 174.
#pragma once

#include <cstdint>

#include "ptx.cuh"
#include "status.cuh"

namespace hstu {

struct CacheView {
  uint8_t* kv;            // [L, num_pages, 2, H, ps, 64] of `elt` bytes
  int64_t* ts;            // [num_pages, ps]
  int32_t* ref;           // [num_pages]
  int32_t* table;         // [num_seqs, max_blocks]
  int32_t* lengths;       // [num_seqs]
  int32_t L, num_pages, H, ps_log2, max_blocks, num_seqs, elt;

  __device__ __forceinline__ int ps() const { return 1 << ps_log2; }
  // of any n >= 0: n + ps - 1 would overflow at the top
  __device__ __forceinline__ int blocks(int n) const {
    return (n >> ps_log2) + ((n & (ps() - 1)) != 0 ? 1 : 0);
  }
  __device__ __forceinline__ int64_t page_bytes() const {  // of one layer
    return (static_cast<int64_t>(2 * H) << ps_log2) * 64 * elt;
  }
  __device__ __forceinline__ bool page_ok(int page) const {
    return static_cast<uint32_t>(page) < static_cast<uint32_t>(num_pages);
  }
  __device__ __forceinline__ uint8_t* page_ptr(int layer, int page) const {
    return kv + (static_cast<int64_t>(layer) * num_pages + page) * page_bytes();
  }
  __device__ __forceinline__ int32_t* row(int seq) const {
    return table + static_cast<int64_t>(seq) * max_blocks;
  }
};

constexpr int CACHE_META_THREADS = 1024;
constexpr int CACHE_COPY_THREADS = 256;
// Seconds between a visible event and the last one, at most: the attention kernels work
// on int32 times.
constexpr int32_t CACHE_MAX_SPAN = INT32_MAX - 2;
constexpr int CACHE_UNIT_V = 2048;  // 16-byte vectors that a block of compact moves at a time

// Exclusive prefix sum of one value per thread over a 1024-thread CTA; `total`
// receives the sum.  sWarp: 33 ints of shared memory.
__device__ __forceinline__ int block_scan(int v, int* sWarp, int& total) {
  const int lane = lane_id(), warp = warp_id();
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sWarp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int w = sWarp[lane];
    int s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sWarp[lane] = s - w;
    if (lane == 31) sWarp[32] = s;
  }
  __syncthreads();
  const int out = sWarp[warp] + x - v;
  total = sWarp[32];
  __syncthreads();
  return out;
}

// ---------------------------------------------------------------- reserve

struct ReserveWs {
  int32_t* state;   // [1]: 1 = the reservation was made
  int32_t* old_len; // [B] length before the call
  int32_t* first;   // [B] index of the user's first page in `pages`
  int32_t* cow;     // [B, 2] (source, copy) of the shared partial last page, or (-1, -1)
  int32_t* pages;   // [num_pages] ids handed out, in order
};

// What the attention of the same call (hstu_extend) will need of the sequences.
struct ReserveSeen {
  int max_context;            // the longest one it is sized for
  int window, sinks;
  const int64_t* timestamps;  // of the new events; nullptr: no attention follows
};

// One CTA: decides the whole reservation, then makes it, or changes nothing.
// Users in batch order; a user takes the copy of its shared partial last page
// first, then its new blocks in order.  A sequence named twice, one out of range,
// a block table too short and a pool without enough free pages are reported; so is,
// where attention follows, what that would report: it would run into it after the
// lengths have grown, and later layers would append what it did not compute (64 users of
// 700 .. 4096 events, one more each: 3 us of an extension's 441).
__global__ void __launch_bounds__(CACHE_META_THREADS)
hstu_cache_reserve_kernel(const CacheView c, int B, const int32_t* __restrict__ seq_ids,
                          const int64_t* __restrict__ offsets, int64_t total_new, int max_new,
                          const ReserveSeen seen, const ReserveWs ws) {
  __shared__ int sWarp[33];
  __shared__ int sBad;
  const int tid = threadIdx.x, lane = lane_id();
  if (tid == 0) sBad = 0;
  __syncthreads();
  // what each user needs; the sign bit of lengths[] marks a sequence as taken by
  // this call, so that one named twice is seen
  int base = 0;
  for (int u0 = 0; u0 < B; u0 += CACHE_META_THREADS) {
    const int u = u0 + tid;
    int need = 0;
    if (u < B) {
      const int seq = seq_ids != nullptr ? seq_ids[u] : u;
      const int64_t o0 = offsets[u], o1 = offsets[u + 1];
      int n = -1, src = -1;
      bool bad = static_cast<uint32_t>(seq) >= static_cast<uint32_t>(c.num_seqs);
      if (!bad) {
        n = atomicOr(&c.lengths[seq], INT32_MIN);
        if (n < 0) n = -1;  // named twice
        const int64_t cnt = o1 - o0;
        bad = n < 0 || o0 < 0 || cnt < 0 || cnt > max_new || o1 > total_new ||
              n + cnt > (static_cast<int64_t>(c.max_blocks) << c.ps_log2) ||
              (cnt > 0 && n + cnt > seen.max_context);
        if (!bad) {
          const int have = c.blocks(n), want = c.blocks(n + static_cast<int>(cnt));
          need = want - have;
          if (cnt > 0 && (n & (c.ps() - 1)) != 0) {
            const int last = c.row(seq)[have - 1];
            if (!c.page_ok(last)) {
              bad = true;
            } else if (c.ref[last] > 1) {
              src = last;
              ++need;
            }
          }
        }
      }
      if (bad) {
        sBad = 1;
        need = 0;
      }
      ws.old_len[u] = n;
      ws.cow[2 * u] = src;
    }
    int total;
    const int ex = block_scan(need, sWarp, total);
    if (u < B) ws.first[u] = base + ex;
    // more pages than the pool has: no need to count on (and no overflow)
    if (total > c.num_pages - base) sBad = 1;
    __syncthreads();
    base = sBad ? 0 : base + total;
  }
  const int want_pages = base;
  // the earlier events that the new rows see: their pages exist, and the earliest is not
  // too long before the last event (a warp per user)
  if (seen.timestamps != nullptr && !sBad) {
    bool missing = false;
    for (int u = warp_id(); u < B; u += CACHE_META_THREADS / 32) {
      const int64_t o0 = offsets[u], o1 = offsets[u + 1];
      if (o1 == o0) continue;
      const int n = ws.old_len[u];
      const int32_t* row = c.row(seq_ids != nullptr ? seq_ids[u] : u);
      const int lo = seen.window > 0 ? max(0, n - seen.window + 1) : 0;  // at most n
      const int sink_end = min(seen.window > 0 ? seen.sinks : 0, lo);
      const int b0 = lo >> c.ps_log2, n_sink = min(c.blocks(sink_end), b0);
      const int nb = n_sink + c.blocks(n) - b0;
#pragma unroll 4
      for (int i = lane; i < nb; i += 32) missing |= !c.page_ok(row[i < n_sink ? i : b0 + (i - n_sink)]);
      if (lane == 0) {
        const int first = sink_end > 0 ? 0 : lo;
        int64_t t = seen.timestamps[o0];
        if (first < n) {
          const int page = row[first >> c.ps_log2];
          if (c.page_ok(page)) t = c.ts[(static_cast<int64_t>(page) << c.ps_log2) + (first & (c.ps() - 1))];
        }
        missing |= seen.timestamps[o1 - 1] - t > CACHE_MAX_SPAN;
      }
    }
    __syncthreads();  // sBad has been read
    if (missing) sBad = 1;
    __syncthreads();
  }
  // the lowest free page ids
  if (!sBad) {
    int found = 0;
    for (int p0 = 0; p0 < c.num_pages && found < want_pages; p0 += 4 * CACHE_META_THREADS) {
      const int p = p0 + 4 * tid;
      int f[4], k = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = p + e < c.num_pages && c.ref[p + e] == 0;
        k += f[e];
      }
      int total;
      int at = found + block_scan(k, sWarp, total);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (f[e]) {
          if (at < want_pages) ws.pages[at] = p + e;
          ++at;
        }
      }
      found += total;
    }
    if (found < want_pages && tid == 0) sBad = 1;
  }
  __syncthreads();
  const bool bad = sBad != 0;
  if (tid == 0) {
    ws.state[0] = bad ? 0 : 1;
    if (bad) record_status(HSTU_ERR_DEVICE_CHECK);
  }
  // hand out: a thread per user for its first pages, the warp for the rest of a long one
  constexpr int OWN = 4;
  for (int u0 = 0; u0 < B; u0 += CACHE_META_THREADS) {
    const int u = u0 + tid;
    const bool in = u < B;
    const int seq = !in ? 0 : (seq_ids != nullptr ? seq_ids[u] : u);
    if (bad) {
      if (in && static_cast<uint32_t>(seq) < static_cast<uint32_t>(c.num_seqs))
        atomicAnd(&c.lengths[seq], INT32_MAX);
      continue;
    }
    int n = 0, cnt = 0, src = -1, first = 0;
    if (in) {
      n = ws.old_len[u];
      cnt = static_cast<int>(offsets[u + 1] - offsets[u]);
      src = ws.cow[2 * u];
      first = ws.first[u];
    }
    const int b0 = c.blocks(n) - (src >= 0 ? 1 : 0);  // first block that gets a page
    const int need = in ? c.blocks(n + cnt) - b0 : 0;
    int copy = -1;
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      if (k < need) {
        const int page = ws.pages[first + k];
        if (k == 0 && src >= 0) copy = page;
        c.row(seq)[b0 + k] = page;
        c.ref[page] = 1;
      }
    }
    if (in) {
      ws.cow[2 * u + 1] = copy;
      if (src >= 0) atomicSub(&c.ref[src], 1);
      c.lengths[seq] = n + cnt;
    }
    for (unsigned m = __ballot_sync(0xffffffffu, need > OWN); m != 0u; m &= m - 1u) {
      const int w = __ffs(m) - 1;
      const int need_w = __shfl_sync(0xffffffffu, need, w), first_w = __shfl_sync(0xffffffffu, first, w);
      int32_t* row = c.row(__shfl_sync(0xffffffffu, seq, w)) + __shfl_sync(0xffffffffu, b0, w);
      for (int k = OWN + lane; k < need_w; k += 32) {
        const int page = ws.pages[first_w + k];
        row[k] = page;
        c.ref[page] = 1;
      }
    }
  }
}

// The copies of shared partial last pages (their filled rows, every layer:
// blockIdx.y) and, for blockIdx.y == L, the timestamps (copied rows, new rows).
__global__ void __launch_bounds__(CACHE_COPY_THREADS)
hstu_cache_reserve_rows_kernel(const CacheView c, const int32_t* __restrict__ seq_ids,
                               const int64_t* __restrict__ offsets,
                               const int64_t* __restrict__ timestamps, const ReserveWs ws) {
  const int u = blockIdx.x, layer = blockIdx.y;
  if (ws.state[0] == 0) return;
  const int src = ws.cow[2 * u], dst = ws.cow[2 * u + 1];
  const int n = ws.old_len[u];
  const int fill = n & (c.ps() - 1);
  if (layer < c.L) {
    if (src < 0) return;
    const uint8_t* a = c.page_ptr(layer, src);
    uint8_t* b = c.page_ptr(layer, dst);
    // 2 * H blocks of ps rows; the first `fill` rows of each
    const int row_v = 64 * c.elt / 16;  // 16-byte vectors of a row
    const int per = fill * row_v, total = 2 * c.H * per;
    const int64_t blk = static_cast<int64_t>(row_v) << c.ps_log2;
    constexpr int U = 4;
    for (int i0 = threadIdx.x; i0 < total; i0 += U * CACHE_COPY_THREADS) {
      uint4 v[U];
      int64_t at[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * CACHE_COPY_THREADS;
        if (i < total) {
          at[k] = (i / per) * blk + i % per;
          v[k] = reinterpret_cast<const uint4*>(a)[at[k]];
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (i0 + k * CACHE_COPY_THREADS < total) reinterpret_cast<uint4*>(b)[at[k]] = v[k];
    }
    return;
  }
  if (src >= 0)
    for (int i = threadIdx.x; i < fill; i += CACHE_COPY_THREADS)
      c.ts[(static_cast<int64_t>(dst) << c.ps_log2) + i] = c.ts[(static_cast<int64_t>(src) << c.ps_log2) + i];
  const int seq = seq_ids != nullptr ? seq_ids[u] : u;
  const int64_t o0 = offsets[u];
  const int cnt = static_cast<int>(offsets[u + 1] - o0);
  const int32_t* row = c.row(seq);
  for (int i = threadIdx.x; i < cnt; i += CACHE_COPY_THREADS) {
    const int pos = n + i;
    const int page = row[pos >> c.ps_log2];
    c.ts[(static_cast<int64_t>(page) << c.ps_log2) + (pos & (c.ps() - 1))] = timestamps[o0 + i];
  }
}

// ---------------------------------------------------------------- fork, release

// One CTA per fork: the destination (an empty sequence) shares every page of the source.
// No sequence that is a destination is a source too, and of the forks that name one
// destination the first is made.  What is made and what is reported does not depend on the
// order in which CTAs run: every CTA looks through all destinations (256 of them in two
// loads per thread, which travel with the CTA's own).  That work grows with the square of
// their number, so past CACHE_FORK_SCAN forks (MARKED) the destinations are marked in
// lengths by a launch before and cleared by one after.  Measured, one launch and three: 4096
// forks of one user 8 us both, 16384 84 and 16, 65535 1269 and 49; 256 with one launch 2.5.
constexpr int CACHE_FORK_THREADS = 128;
constexpr int CACHE_FORK_SCAN = 4096;

// A destination's length while MARKED forks run, negative in every state: ~i when it was
// empty and fork i is the first that names it; the sign bit over its length when it was not
// empty, and once its fork has been decided.
__global__ void __launch_bounds__(CACHE_COPY_THREADS)
hstu_cache_fork_mark_kernel(const CacheView c, int count, const int32_t* __restrict__ dst_ids) {
  const int i = blockIdx.x * CACHE_COPY_THREADS + threadIdx.x;
  if (i >= count || static_cast<uint32_t>(dst_ids[i]) >= static_cast<uint32_t>(c.num_seqs)) return;
  int32_t* len = &c.lengths[dst_ids[i]];
  int cur = atomicOr(len, 0);
  for (;;) {
    // (a fork's index is below 2^30, and so is a length: the two kinds of mark do not meet;
    // a longer one is no source and no destination anyway)
    int want = cur;
    if (cur == 0) want = ~i;
    else if (cur > 0 && cur < (1 << 30)) want = cur | INT32_MIN;
    else if (cur < 0 && cur >= -(1 << 30)) want = max(cur, ~i);
    if (want == cur) return;
    const int was = atomicCAS(len, cur, want);
    if (was == cur) return;
    cur = was;
  }
}
__global__ void __launch_bounds__(CACHE_COPY_THREADS)
hstu_cache_fork_clear_kernel(const CacheView c, int count, const int32_t* __restrict__ dst_ids) {
  const int i = blockIdx.x * CACHE_COPY_THREADS + threadIdx.x;
  if (i < count && static_cast<uint32_t>(dst_ids[i]) < static_cast<uint32_t>(c.num_seqs))
    atomicAnd(&c.lengths[dst_ids[i]], INT32_MAX);
}

template <bool MARKED>
__global__ void __launch_bounds__(CACHE_FORK_THREADS)
hstu_cache_fork_kernel(const CacheView c, const int32_t* __restrict__ src_ids,
                       const int32_t* __restrict__ dst_ids) {
  const int src = src_ids[blockIdx.x], dst = dst_ids[blockIdx.x];
  const bool ids = static_cast<uint32_t>(src) < static_cast<uint32_t>(c.num_seqs) &&
                   static_cast<uint32_t>(dst) < static_cast<uint32_t>(c.num_seqs);
  const int n = ids ? c.lengths[src] : -1;  // MARKED: negative for a destination
  bool bad = n < 0 || c.blocks(n) > c.max_blocks;
  bool mine = false;
  if constexpr (MARKED) {
    mine = static_cast<uint32_t>(dst) < static_cast<uint32_t>(c.num_seqs) &&
           c.lengths[dst] == ~static_cast<int>(blockIdx.x);
    bad |= !mine;
  } else {
    bad = bad || c.lengths[dst] != 0;
#pragma unroll 4
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += CACHE_FORK_THREADS) {
      const int d = dst_ids[i];
      bad |= d == src || (d == dst && i < blockIdx.x);
    }
  }
  // (every thread has read the destination's length)
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      record_status(HSTU_ERR_DEVICE_CHECK);
      if (MARKED && mine) c.lengths[dst] = INT32_MIN;
    }
    return;
  }
  const int nb = c.blocks(n);
  const int32_t* a = c.row(src);
  int32_t* b = c.row(dst);
  for (int i = threadIdx.x; i < nb; i += CACHE_FORK_THREADS) {
    const int page = a[i];
    b[i] = page;
    if (c.page_ok(page)) atomicAdd(&c.ref[page], 1);
  }
  if (threadIdx.x == 0) c.lengths[dst] = MARKED ? n | INT32_MIN : n;
}

// One CTA per listed sequence.  window < 0: the whole sequence; else the blocks
// none of whose events an event after the last one sees (window, sinks).  Each
// table entry is given up by whoever exchanges it for -1, so a sequence listed
// twice is released once.
__global__ void __launch_bounds__(128)
hstu_cache_release_kernel(const CacheView c, const int32_t* __restrict__ seq_ids, int window,
                          int sinks) {
  const int seq = seq_ids[blockIdx.x];
  if (static_cast<uint32_t>(seq) >= static_cast<uint32_t>(c.num_seqs)) {
    if (threadIdx.x == 0) record_status(HSTU_ERR_DEVICE_CHECK);
    return;
  }
  const int n = *reinterpret_cast<volatile int32_t*>(&c.lengths[seq]);
  if (n < 0 || c.blocks(n) > c.max_blocks) {
    if (threadIdx.x == 0) record_status(HSTU_ERR_DEVICE_CHECK);
    return;
  }
  int b0 = 0, b1 = c.blocks(n);
  if (window >= 0) {
    // an event at n sees j < sinks and j > n - window
    b0 = c.blocks(sinks < n ? sinks : n);
    const int lo = n + 1 > window ? n + 1 - window : 0;
    b1 = min(b1, lo >> c.ps_log2);
  }
  int32_t* row = c.row(seq);
  for (int i = b0 + threadIdx.x; i < b1; i += blockDim.x) {
    const int page = atomicExch(&row[i], -1);
    if (!c.page_ok(page)) continue;
    if (atomicSub(&c.ref[page], 1) <= 0) {
      atomicAdd(&c.ref[page], 1);
      record_status(HSTU_ERR_DEVICE_CHECK);
    }
  }
  __syncthreads();
  if (window < 0 && threadIdx.x == 0) c.lengths[seq] = 0;
}

// ---------------------------------------------------------------- compact

struct CompactWs {
  int32_t* count;  // [1] pages to move
  int32_t* src;    // [num_pages]
  int32_t* dst;    // [num_pages]
  int32_t* map;    // [num_pages] new id of a moved page
};

// One CTA: the k-th live page at or past the number of live pages moves to the
// k-th free page below it.
__global__ void __launch_bounds__(CACHE_META_THREADS)
hstu_cache_compact_kernel(const CacheView c, const CompactWs ws, int32_t* __restrict__ live_out) {
  __shared__ int sWarp[33];
  const int tid = threadIdx.x;
  int live = 0;
  for (int p0 = 0; p0 < c.num_pages; p0 += CACHE_META_THREADS) {
    const int p = p0 + tid;
    live += __syncthreads_count(p < c.num_pages && c.ref[p] > 0);
  }
  int holes = 0, moves = 0;
  for (int p0 = 0; p0 < c.num_pages; p0 += CACHE_META_THREADS) {
    const int p = p0 + tid;
    const bool in = p < c.num_pages;
    const int r = in ? c.ref[p] : 0;
    const bool hole = in && p < live && r <= 0, move = in && p >= live && r > 0;
    // holes lie below `live` and moves at or past it; both counts fit 16 bits per step
    int total;
    const int ex = block_scan((hole ? 1 : 0) | (move ? 1 << 16 : 0), sWarp, total);
    if (hole) ws.dst[holes + (ex & 0xffff)] = p;
    if (move) ws.src[moves + (ex >> 16)] = p;
    holes += total & 0xffff;
    moves += total >> 16;
  }
  __syncthreads();
  for (int k = tid; k < moves; k += CACHE_META_THREADS) {
    const int a = ws.src[k], b = ws.dst[k];
    ws.map[a] = b;
    c.ref[b] = c.ref[a];
    c.ref[a] = 0;
  }
  if (tid == 0) {
    ws.count[0] = moves;
    if (live_out != nullptr) live_out[0] = live;
  }
}

// Block-table entries of moved pages (one CTA per sequence), then, over the whole
// grid, the page copies: every layer's K and V and the timestamps.
__global__ void __launch_bounds__(CACHE_COPY_THREADS)
hstu_cache_compact_rows_kernel(const CacheView c, const CompactWs ws) {
  const int moves = ws.count[0];
  if (moves == 0) return;
  for (int seq = blockIdx.x; seq < c.num_seqs; seq += gridDim.x) {
    const int n = c.lengths[seq];
    const int nb = n > 0 ? min(c.blocks(n), c.max_blocks) : 0;
    int32_t* row = c.row(seq);
    for (int i = threadIdx.x; i < nb; i += CACHE_COPY_THREADS) {
      const int page = row[i];
      // a page whose count is zero now and that a sequence names has moved
      if (c.page_ok(page) && c.ref[page] == 0) row[i] = ws.map[page];
    }
  }
  // units of 32 KB of one page of one layer: eight 16-byte loads in flight per thread
  constexpr int UNIT_V = CACHE_UNIT_V;
  const int64_t page_v = c.page_bytes() / 16;
  const int64_t per_page = (page_v + UNIT_V - 1) / UNIT_V;
  const int64_t units = per_page * c.L * moves;
  constexpr int U = UNIT_V / CACHE_COPY_THREADS;
  for (int64_t w = blockIdx.x; w < units; w += gridDim.x) {
    const int64_t part = w % per_page, rest = w / per_page;
    const int layer = static_cast<int>(rest % c.L), k = static_cast<int>(rest / c.L);
    const uint4* a = reinterpret_cast<const uint4*>(c.page_ptr(layer, ws.src[k])) + part * UNIT_V;
    uint4* b = reinterpret_cast<uint4*>(c.page_ptr(layer, ws.dst[k])) + part * UNIT_V;
    const int64_t left = page_v - part * UNIT_V;
    uint4 v[U];
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int i = threadIdx.x + e * CACHE_COPY_THREADS;
      if (i < left) v[e] = __ldcs(a + i);
    }
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int i = threadIdx.x + e * CACHE_COPY_THREADS;
      if (i < left) __stcs(b + i, v[e]);
    }
  }
  const int64_t stamps = static_cast<int64_t>(moves) << c.ps_log2;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * CACHE_COPY_THREADS + threadIdx.x; i < stamps;
       i += static_cast<int64_t>(gridDim.x) * CACHE_COPY_THREADS) {
    const int k = static_cast<int>(i >> c.ps_log2), s = static_cast<int>(i & (c.ps() - 1));
    c.ts[(static_cast<int64_t>(ws.dst[k]) << c.ps_log2) + s] =
        c.ts[(static_cast<int64_t>(ws.src[k]) << c.ps_log2) + s];
  }
}

// ---------------------------------------------------------------- append, gather

// A warp per row: the new event's K and V of every head into its page.  The grid
// is (row groups, users), so no row has to look its user up.
__global__ void __launch_bounds__(CACHE_COPY_THREADS)
hstu_cache_append_kernel(const CacheView c, int layer, const int32_t* __restrict__ seq_ids,
                         const int64_t* __restrict__ offsets, int64_t total_new, int max_new,
                         const uint8_t* __restrict__ k, int64_t ldk, const uint8_t* __restrict__ v,
                         int64_t ldv, const int32_t* __restrict__ go) {
  // `go`: the reservation of the same call (0: refused, the chunk has no rows)
  if (go != nullptr && *go == 0) return;
  const int u = blockIdx.y;
  const int64_t o0 = offsets[u], o1 = offsets[u + 1];
  const int seq = seq_ids != nullptr ? seq_ids[u] : u;
  const int64_t cnt = o1 - o0;
  if (cnt == 0) return;
  const bool seq_ok = static_cast<uint32_t>(seq) < static_cast<uint32_t>(c.num_seqs);
  const int n = seq_ok ? c.lengths[seq] : -1;
  if (cnt < 0 || cnt > max_new || o0 < 0 || o1 > total_new || n < cnt ||
      c.blocks(n) > c.max_blocks) {
    if (threadIdx.x == 0 && blockIdx.x == 0) record_status(HSTU_ERR_DEVICE_CHECK);
    return;
  }
  const int32_t* row = c.row(seq);
  const int lane = lane_id();
  const int cph = 64 * c.elt / 16;         // 16-byte vectors per head
  const int per = c.H * cph;               // per K or V row
  constexpr int WARPS = CACHE_COPY_THREADS / 32;
  for (int r = blockIdx.x * WARPS + warp_id(); r < cnt; r += gridDim.x * WARPS) {
    const int pos = n - static_cast<int>(cnt) + r;
    const int page = row[pos >> c.ps_log2];
    // a page that is no page, or that another sequence shares, is not written
    if (!c.page_ok(page) || (c.ref != nullptr && c.ref[page] != 1)) {
      if (lane == 0) record_status(HSTU_ERR_DEVICE_CHECK);
      continue;
    }
    const int slot = pos & (c.ps() - 1);
    uint4* dst = reinterpret_cast<uint4*>(c.page_ptr(layer, page));
    const uint4* ks = reinterpret_cast<const uint4*>(k + (o0 + r) * ldk * c.elt);
    const uint4* vs = reinterpret_cast<const uint4*>(v + (o0 + r) * ldv * c.elt);
    constexpr int U = 4;
    for (int i0 = lane; i0 < 2 * per; i0 += 32 * U) {
      uint4 x[U];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int i = i0 + 32 * e;
        if (i < 2 * per) x[e] = i < per ? ks[i] : vs[i - per];
      }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int i = i0 + 32 * e;
        if (i < 2 * per) {
          const int hb = i / cph;  // K heads, then V heads: the page's block order
          dst[((static_cast<int64_t>(hb) << c.ps_log2) + slot) * cph + i % cph] = x[e];
        }
      }
    }
  }
}

// A warp per row and layer: a user's whole history out of its pages, dense rows
// [K of every head, V of every head] in the layout hstu_forward writes its cache
// in.  Rows without a page (released by the window) are zeros, and are reported.
__global__ void __launch_bounds__(CACHE_COPY_THREADS)
hstu_cache_gather_kernel(const CacheView c, const int32_t* __restrict__ seq_ids,
                         const int64_t* __restrict__ offsets, int64_t total, uint8_t* __restrict__ out,
                         int64_t* __restrict__ ts_out) {
  const int u = blockIdx.y;
  const int64_t o0 = offsets[u], o1 = offsets[u + 1];
  const int seq = seq_ids != nullptr ? seq_ids[u] : u;
  const int64_t cnt = o1 - o0;
  if (cnt == 0) return;
  const bool seq_ok = static_cast<uint32_t>(seq) < static_cast<uint32_t>(c.num_seqs);
  const int n = seq_ok ? c.lengths[seq] : -1;
  if (cnt < 0 || cnt != n || o0 < 0 || o1 > total || c.blocks(n) > c.max_blocks) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.z == 0) record_status(HSTU_ERR_DEVICE_CHECK);
    return;
  }
  const int32_t* row = c.row(seq);
  const int lane = lane_id(), layer = blockIdx.z;
  const int cph = 64 * c.elt / 16, per = c.H * cph;
  constexpr int WARPS = CACHE_COPY_THREADS / 32;
  for (int r = blockIdx.x * WARPS + warp_id(); r < n; r += gridDim.x * WARPS) {
    const int page = row[r >> c.ps_log2], slot = r & (c.ps() - 1);
    const bool ok = c.page_ok(page);
    if (!ok && lane == 0) record_status(HSTU_ERR_DEVICE_CHECK);
    const uint4* src = reinterpret_cast<const uint4*>(c.page_ptr(layer, ok ? page : 0));
    uint4* dst = reinterpret_cast<uint4*>(out) + (layer * total + o0 + r) * (2 * per);
    constexpr int U = 4;
    for (int i0 = lane; i0 < 2 * per; i0 += 32 * U) {
      uint4 x[U];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int i = i0 + 32 * e;
        x[e] = make_uint4(0u, 0u, 0u, 0u);
        if (i < 2 * per && ok)
          x[e] = src[((static_cast<int64_t>(i / cph) << c.ps_log2) + slot) * cph + i % cph];
      }
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const int i = i0 + 32 * e;
        if (i < 2 * per) dst[i] = x[e];
      }
    }
    if (layer == 0 && lane == 0 && ts_out != nullptr)
      ts_out[o0 + r] = ok ? c.ts[(static_cast<int64_t>(page) << c.ps_log2) + slot] : 0;
  }
}

}  // namespace hstu
