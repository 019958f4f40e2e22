// Attention of a chunk of new events over the paged history cache (cache.cuh):
// Eq. 2 of the review of "Actions Speak Louder than Words" (section 三 核心公式)
// for the last c events of a sequence of n, which attend to all n cached events up
// to themselves:
//   AV_i = sum_j phi2(q_i.k_j + rab_pos[h, min(i-j, P-1)] + rab_time[h, bt(t_i-t_j)]) v_j / n
// with a window W (0: none) only over j > i - W and the first `sinks` events;
// phi2 = softmax replaces phi2 and 1/n by a softmax over the visible keys.
//
// What bounds it: every visible K and V row is read once per group of query rows
// (256 bytes per key and head in 16 bits), so few rows are bound by the cache
// bandwidth and many rows by the element work per (row, key) pair.  One row over n
// keys is one row of CTAs, so the keys are split over the CTAs of a thread-block
// cluster; the partial sums meet in distributed shared memory, in rank order:
// one launch, no workspace, and the same bits every run.
//
// Positions and times: position biases of a key tile are a band of
// rab_pos (i - j runs over keys + rows - 1 values), loaded per tile, so neither
// the sequence length nor the table has to fit shared memory.  Times are int32
// seconds relative to the last event (offset so that they stay non-negative); a
// visible key more than 2^31 - 3 seconds before it is reported.
#pragma once

#include <cooperative_groups.h>

#include "attn.cuh"
#include "cache.cuh"

namespace hstu {

struct PagedParams {
  const uint8_t* kv;         // the layer's [num_pages, 2, H, ps, 64]
  const int64_t* ts;         // [num_pages, ps]
  const int32_t* table;      // [num_seqs, max_blocks]
  const int32_t* lengths;    // [num_seqs]
  const int32_t* seq_ids;    // [B] or nullptr (identity)
  const int64_t* q_offsets;  // [B + 1]
  const int64_t* q_ts;       // [T] timestamps of the new events
  const void* q;             // [T, ldq] operand type
  int64_t ldq;
  const float* rab_pos;      // [H, P]
  const float* rab_time;     // [H, Tb]
  void* av;                  // [T, H * 64] operand type, or
  float* av_f32;             // [T, H * 64] fp32
  float* ln_part;            // [T, H, 2] (sum, centred sum of squares) or nullptr
  int64_t T;
  int32_t B, H, P, Tb, num_pages, num_seqs, max_blocks, ps_log2;
  int32_t max_new, max_context, window, sinks;
  int32_t groups;            // row groups per sequence
  int32_t nsplit;            // CTAs of a cluster
  int32_t sorted;            // longest sequences first (at most 128 of them)
  uint64_t timeout_ns;
  int32_t thr[MAX_TIME_BUCKETS];  // time-bucket thresholds clamped to int32
  int4 oct[32];
};

// One sequence's part of a launch, the same for every CTA of its clusters; tiles of
// KEYS keys.
template <int KEYS>
struct PagedSeq {
  int seq, n, c;       // table row, events, new events
  int64_t q0;          // first query row
  int lo;              // keys [0, sink_end) and [lo, n) are visible to some row
  int sink_end;
  int n_sink, first;   // key tiles 0 .. n_sink-1, then first .. first + n_main - 1
  int n_tiles;

  __device__ __forceinline__ int tile(int k) const { return k < n_sink ? k : first + (k - n_sink); }
  // whether some row of the chunk sees position j
  __device__ __forceinline__ bool seen(int j) const {
    return (j < sink_end || j >= lo) && j < n;
  }
};

// Reads and checks sequence u; r0 / r1: the query rows [r0, r1) of this row group.
// Returns 1 to go on, 0 when the group has no rows, -1 when the input is bad.
template <int KEYS>
__device__ __forceinline__ int paged_seq(const PagedParams& p, int u, int r0, int rows, PagedSeq<KEYS>& s) {
  const int64_t o0 = p.q_offsets[u], o1 = p.q_offsets[u + 1];
  const int64_t cnt = o1 - o0;
  if (cnt == 0) return 0;
  s.seq = p.seq_ids != nullptr ? p.seq_ids[u] : u;
  if (static_cast<uint32_t>(s.seq) >= static_cast<uint32_t>(p.num_seqs)) return -1;
  s.n = p.lengths[s.seq];
  if (cnt < 0 || cnt > p.max_new || o0 < 0 || o1 > p.T || s.n < cnt || s.n > p.max_context) return -1;
  s.c = static_cast<int>(cnt);
  s.q0 = o0;
  if (r0 >= s.c) return 0;
  const int i0 = s.n - s.c + r0;                   // first row's position
  const int i1 = s.n - s.c + min(r0 + rows, s.c);  // one past the last row's
  s.lo = p.window > 0 ? max(0, i0 - p.window + 1) : 0;
  s.sink_end = min(p.sinks, s.lo);
  s.first = s.lo / KEYS;
  s.n_sink = min((s.sink_end + KEYS - 1) / KEYS, s.first);
  s.n_tiles = s.n_sink + (i1 + KEYS - 1) / KEYS - s.first;
  s.n = i1;  // keys past the group's last row are seen by none of its rows
  return 1;
}

// The sequence of the u-th longest context (ties: the lower index).  The grid starts
// CTAs in order, so with a few waves of ragged contexts the short ones fill the gaps
// that the long ones leave.  sLen: 128 ints; every thread of the CTA takes part.
__device__ __forceinline__ int paged_nth_longest(const PagedParams& p, int u, int32_t* sLen, int* sU) {
  const int t = threadIdx.x;
  if (t < p.B) {
    const int seq = p.seq_ids != nullptr ? p.seq_ids[t] : t;
    const bool live = static_cast<uint32_t>(seq) < static_cast<uint32_t>(p.num_seqs) &&
                      p.q_offsets[t + 1] > p.q_offsets[t];
    sLen[t] = live ? p.lengths[seq] : -1;
  }
  __syncthreads();
  if (t < p.B) {
    const int mine = sLen[t];
    int rank = 0;
    for (int v = 0; v < p.B; ++v) rank += sLen[v] > mine || (sLen[v] == mine && v < t);
    if (rank == u) *sU = t;
  }
  __syncthreads();
  return *sU;
}

// Seconds relative to the last event, shifted into [0, 2^31 - 3].
constexpr int32_t PG_T0 = CACHE_MAX_SPAN;
__device__ __forceinline__ int32_t paged_rel(int64_t t, int64_t t_last) {
  const int64_t d = t - t_last + PG_T0;
  return d < 0 ? 0 : (d > PG_T0 ? PG_T0 : static_cast<int32_t>(d));
}

// ---------------------------------------------------------------- fp32

// fp32 layers are small (tens to hundreds of events, one or two heads): FFMA over
// 64-key tiles in shared memory, 16 query rows per CTA, four rows and one key (or
// one column of V) per thread, 16-byte shared loads; the next tile's rows are read
// into registers meanwhile.  Exact exponentials (expf), so the result holds fp32
// accuracy.  Softmax keeps a running maximum and sum per row.  Measured: 12 users, 2
// heads, up to 50 events over up to 700 18 us (4-byte shared loads, no read-ahead: 28);
// bound by the barriers between the steps of a tile.
constexpr int PG32_KEYS = 64;
constexpr int PG32_ROWS = 16;
constexpr int PG32_THREADS = 256;

struct Paged32Smem {
  float q[PG32_ROWS][64];
  float k[PG32_KEYS][68];       // rows 4 banks apart: 16-byte loads of 8 lanes do not collide
  float v[PG32_KEYS][64];       // after the last tile, rows 0 .. 15: this CTA's partial sums
  float s[PG32_ROWS][PG32_KEYS];
  float2 ml[PG32_ROWS];         // softmax: (max, sum) of this CTA's keys
  float scale[PG32_ROWS];       // softmax: factor of the running sums
  int32_t kt[PG32_KEYS];
  int32_t qt[PG32_ROWS];
  float rt[MAX_TIME_BUCKETS];
};

__global__ void __launch_bounds__(PG32_THREADS)
hstu_paged_f32_kernel(const __grid_constant__ PagedParams p, int phi2) {
  __shared__ __align__(16) Paged32Smem sm;
  namespace cg = cooperative_groups;
  const int split = static_cast<int>(blockIdx.x % p.nsplit);
  const int64_t id = blockIdx.x / p.nsplit;
  const int h = static_cast<int>(id % p.H);
  const int g = static_cast<int>((id / p.H) % p.groups), u = static_cast<int>(id / p.H / p.groups);
  const int tid = threadIdx.x;
  PagedSeq<PG32_KEYS> s;
  const int r0 = g * PG32_ROWS;
  const int go = paged_seq(p, u, r0, PG32_ROWS, s);
  if (go <= 0) {  // the same for the whole cluster
    if (go < 0 && tid == 0) record_status(HSTU_ERR_DEVICE_CHECK);
    return;
  }
  const bool softmax = phi2 == HSTU_ACT_SOFTMAX;
  const int rows = min(PG32_ROWS, s.c - r0);
  const int n_all = p.lengths[s.seq];
  const int i0 = n_all - s.c + r0;
  const int64_t t_last = p.q_ts[s.q0 + s.c - 1];
  const int32_t* tab = p.table + static_cast<int64_t>(s.seq) * p.max_blocks;
  const int ps = 1 << p.ps_log2;
  const int k_begin = static_cast<int>(static_cast<int64_t>(s.n_tiles) * split / p.nsplit);
  const int k_end = static_cast<int>(static_cast<int64_t>(s.n_tiles) * (split + 1) / p.nsplit);
  // A tile's rows, 16 bytes per thread and step (step e: K for e < 4, V after; row
  // tid / 16 + 16 (e % 4)), and a time per thread of the first 64; keys that no row
  // sees are zeros
  float4 x[8];
  int32_t t_new = 0;
  auto load_tile = [&](int kk) {
    const int j0 = s.tile(kk) * PG32_KEYS;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + (tid >> 4) + 16 * e;
      x[e] = x[e + 4] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (s.seen(j)) {
        const int page = tab[j >> p.ps_log2];
        if (static_cast<uint32_t>(page) < static_cast<uint32_t>(p.num_pages)) {
          const float4* row = reinterpret_cast<const float4*>(p.kv) +
                              ((static_cast<int64_t>(page) * 2 * p.H + h) * ps + (j & (ps - 1))) * 16 + (tid & 15);
          x[e] = __ldg(row);
          x[e + 4] = __ldg(row + static_cast<int64_t>(p.H) * ps * 16);
        } else if ((tid & 15) == 0) {
          record_status(HSTU_ERR_DEVICE_CHECK);
        }
      }
    }
    if (tid < PG32_KEYS) {
      const int j = j0 + tid;
      t_new = 0;
      if (s.seen(j)) {
        const int page = tab[j >> p.ps_log2];
        if (static_cast<uint32_t>(page) < static_cast<uint32_t>(p.num_pages)) {
          const int64_t tj = p.ts[static_cast<int64_t>(page) * ps + (j & (ps - 1))];
          if (t_last - tj > PG_T0) record_status(HSTU_ERR_DEVICE_CHECK);
          t_new = paged_rel(tj, t_last);
        }
      }
    }
  };
  if (k_begin < k_end) load_tile(k_begin);
  {
    const int r = tid >> 4, c4 = tid & 15;
    float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (r < rows)
      q = *(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + (s.q0 + r0 + r) * p.ldq + h * 64) + c4);
    *reinterpret_cast<float4*>(&sm.q[r][4 * c4]) = q;
  }
  for (int e = tid; e < p.Tb; e += PG32_THREADS) sm.rt[e] = p.rab_time[static_cast<int64_t>(h) * p.Tb + e];
  if (tid < PG32_ROWS) {
    sm.qt[tid] = tid < rows ? paged_rel(p.q_ts[s.q0 + r0 + tid], t_last) : 0;
    sm.ml[tid] = make_float2(-INFINITY, 0.0f);
  }
  const int col = tid & 63, rg = tid >> 6;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* rp = p.rab_pos + static_cast<int64_t>(h) * p.P;
  for (int kk = k_begin; kk < k_end; ++kk) {
    const int j0 = s.tile(kk) * PG32_KEYS;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = (tid >> 4) + 16 * e;
      *reinterpret_cast<float4*>(&sm.k[r][4 * (tid & 15)]) = x[e];
      *reinterpret_cast<float4*>(&sm.v[r][4 * (tid & 15)]) = x[e + 4];
    }
    if (tid < PG32_KEYS) sm.kt[tid] = t_new;
    __syncthreads();
    if (kk + 1 < k_end) load_tile(kk + 1);
    const int j = j0 + col;
    float dot[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < 64; c += 4) {
      const float4 kx = *reinterpret_cast<const float4*>(&sm.k[col][c]);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float4 qx = *reinterpret_cast<const float4*>(&sm.q[rg + 4 * a][c]);
        dot[a] = fmaf(qx.x, kx.x, fmaf(qx.y, kx.y, fmaf(qx.z, kx.z, fmaf(qx.w, kx.w, dot[a]))));
      }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int r = rg + 4 * a, i = i0 + r;
      const bool vis = r < rows && j <= i && (p.window == 0 || j > i - p.window || j < p.sinks);
      float y = dot[a];
      if (vis) y += __ldg(rp + min(i - j, p.P - 1)) + sm.rt[time_bucket_octave(sm.qt[r] - sm.kt[col], p.oct)];
      sm.s[r][col] = softmax ? (vis ? y : -INFINITY) : (vis ? phi_runtime(y, phi2) : 0.0f);
    }
    __syncthreads();
    if (softmax) {
      // 16 lanes a row, four keys each
      const int r = tid >> 4, c4 = tid & 15;
      float4 y = *reinterpret_cast<const float4*>(&sm.s[r][4 * c4]);
      float m = fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w));
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      const float2 old = sm.ml[r];
      m = fmaxf(m, old.x);
      // (the maximum passes a NaN over: it stays one in its weight and in the sum)
      const bool any = m > -INFINITY;
      const float mm = any ? m : 0.0f;
      y.x = expf(y.x - mm);
      y.y = expf(y.y - mm);
      y.z = expf(y.z - mm);
      y.w = expf(y.w - mm);
      *reinterpret_cast<float4*>(&sm.s[r][4 * c4]) = y;
      float l = (y.x + y.y) + (y.z + y.w);
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      if (c4 == 0) {
        const float f = any ? expf(old.x - m) : 1.0f;
        sm.scale[r] = f;
        sm.ml[r] = make_float2(m, fmaf(old.y, f, l));
      }
      __syncthreads();
#pragma unroll
      for (int a = 0; a < 4; ++a) acc[a] *= sm.scale[rg + 4 * a];
    }
    // each tile's sum apart, then added: the rounding grows with the tiles, not the keys
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int c = 0; c < PG32_KEYS; c += 4) {
      const float v0 = sm.v[c][col], v1 = sm.v[c + 1][col], v2 = sm.v[c + 2][col], v3 = sm.v[c + 3][col];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const float4 w = *reinterpret_cast<const float4*>(&sm.s[rg + 4 * a][c]);
        part[a] = fmaf(w.x, v0, fmaf(w.y, v1, fmaf(w.z, v2, fmaf(w.w, v3, part[a]))));
      }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) acc[a] += part[a];
  }
  __syncthreads();
#pragma unroll
  for (int a = 0; a < 4; ++a) sm.v[rg + 4 * a][col] = acc[a];
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  // rank `split` writes rows 4 split .., 4 (split + nsplit) ..: 64 threads per row
  for (int r = split * 4 + rg; r < rows; r += 4 * p.nsplit) {
    float o = 0.0f;
    if (softmax) {
      float m = -INFINITY, l = 0.0f;
      for (int k = 0; k < p.nsplit; ++k) m = fmaxf(m, cluster.map_shared_rank(&sm, k)->ml[r].x);
      for (int k = 0; k < p.nsplit; ++k) {
        const Paged32Smem* o_sm = cluster.map_shared_rank(&sm, k);
        const float f = o_sm->ml[r].x > -INFINITY ? expf(o_sm->ml[r].x - m) : 0.0f;
        l += o_sm->ml[r].y * f;
        o += o_sm->v[r][col] * f;
      }
      o = l == 0.0f ? 0.0f : o / l;  // a NaN stays one
    } else {
      for (int k = 0; k < p.nsplit; ++k) o += cluster.map_shared_rank(&sm, k)->v[r][col];
      o /= static_cast<float>(n_all);
    }
    p.av_f32[((s.q0 + r0 + r) * p.H + h) * 64 + col] = o;
  }
  cluster.sync();  // no CTA leaves while another reads its partial sums
}

// ---------------------------------------------------------------- few rows

// 16-bit operands, 8 * MH query rows per CTA (one or both halves of a 16-row MMA tile),
// keys split over a cluster.  Bound
// by the cache bandwidth, so the tensor work runs on warp-level MMAs (m16n8k16)
// whose operands and results stay in registers: a 128-row tcgen05 tile would do
// the element work of 128 rows for the 1..16 that exist.  Warp w of 4 owns keys
// 16 w .. 16 w + 15 of every 64-key tile for all the rows: S = Q K^T, the element
// work and O += P V need no exchange between warps until the end.  A fifth warp
// streams K, V (TMA, one box per page part, 128B swizzle), key times and the
// position band (cp.async) through a ring of stages, and never waits for a value it
// loads: block-table entries come 32 boxes at a time, a batch ahead.
// Measured (B200, 8 heads, fp16): one event of each of 64 users over 700 .. 4096
// cached ones 55 us, 5.7 TB/s of K and V (87% of the copy bandwidth); 55 users over 4096,
// one full round of CTAs, 6.3 TB/s.  One event of one user over 301: 6.5 us, all
// latency (four dependent loads, then the first tile).  Per-lane copies of times and
// bands instead of bulk ones, with the producer waiting for its loads: 134 us.
// Eight warps and 128-key tiles at 2 CTAs per SM: 66 us; 32 rows per CTA (more
// registers, 2 CTAs per SM): 16 users x 16 events 49 us, with 16 rows 34 us.
constexpr int PGS_KEYS = 64;  // keys per tile, 16 per warp
constexpr int PGS_WARPS = 4;
constexpr int PGS_THREADS = (PGS_WARPS + 1) * 32;
constexpr int PGS_STAGES = 4;
constexpr uint32_t PGS_TILE_BYTES = PGS_KEYS * 128;
constexpr int PGS_OLD = 68;  // row stride (floats) of the partial sums: 16-byte rows, no bank conflicts

struct PgsSmem {
  static constexpr uint32_t kK = 0;
  static constexpr uint32_t kV = kK + PGS_STAGES * PGS_TILE_BYTES;
  static constexpr uint32_t kSide = kV + PGS_STAGES * PGS_TILE_BYTES;  // per stage: times, biases
  static constexpr uint32_t kSideBytes = PGS_KEYS * 8 + (PGS_KEYS + 16 + 4) * 4;
  static constexpr uint32_t kTime = kSide + PGS_STAGES * kSideBytes;
  static constexpr uint32_t kThr = kTime + MAX_TIME_BUCKETS * 4;
  static constexpr uint32_t kOct = kThr + MAX_TIME_BUCKETS * 4;
  static constexpr uint32_t kOrt = kOct + 32 * 16;
  static constexpr uint32_t kMl = kOrt + 32 * 16;                  // warps x 16 rows float2
  static constexpr uint32_t kMlC = kMl + PGS_WARPS * 16 * 8;       // 16 rows float2 of the CTA
  static constexpr uint32_t kBars = kMlC + 16 * 8;
  static constexpr uint32_t kAbort = kBars + 2 * PGS_STAGES * 8;
  static constexpr uint32_t kBytes = kAbort + 16 + 1024;           // + align slack
  static_assert(kMlC - kMl >= 128 * 4, "the lengths that are sorted fit over the maxima");
  static_assert(kSide % 16 == 0 && kSideBytes % 16 == 0, "bulk copies");
  static_assert(PGS_WARPS * 16 * PGS_OLD * 4 <= kSide, "the partial sums fit over the stages");
};

// Copy of `bytes` contiguous bytes (16-byte aligned, a multiple of 16) completing on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// tma_load_2d to a shared-memory address.
__device__ __forceinline__ void tma_load_2d_to(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                               int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
// One arrival on the barrier (counted in its expected arrivals) when this
// thread's asynchronous copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// First offset i - j of a tile's position band: the last key's for the first row, down
// to a multiple of 4 (16 bytes); d = i0 - j0.
__device__ __forceinline__ int paged_band0(int d, int keys) { return (d - (keys - 1)) & ~3; }

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), 16-bit operands.
template <bool F16>
__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A B: the first step of a chain.
template <bool F16>
__device__ __forceinline__ void mma_m16n8k16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                   uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack_16(float lo, float hi) {
  if constexpr (F16) return pack_h2(lo, hi);
  else return pack_bf16x2(lo, hi);
}

// A row's result: 16-bit or fp32, with the row's LayerNorm partial sums on
// request; the 16 lanes of a half warp hold the row's 64 columns (4 each).
template <bool F16>
__device__ __forceinline__ void paged_store(const PagedParams& p, int64_t row, int h, int c4, float4 o,
                                            bool live) {
  const int64_t at = (row * p.H + h) * 64 + 4 * c4;
  if (live) {
    if (p.av_f32 != nullptr)
      *reinterpret_cast<float4*>(p.av_f32 + at) = o;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.av) + at) =
          make_uint2(pack_16<F16>(o.x, o.y), pack_16<F16>(o.z, o.w));
  }
  if (p.ln_part != nullptr) {  // uniform; every lane of the warp takes part
    float sum = o.x + o.y + o.z + o.w;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const float m = sum * (1.0f / 64.0f);
    float sq = (o.x - m) * (o.x - m) + (o.y - m) * (o.y - m) + (o.z - m) * (o.z - m) + (o.w - m) * (o.w - m);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
    if (live && c4 == 0)
      reinterpret_cast<float2*>(p.ln_part)[row * p.H + h] = make_float2(sum, sq);
  }
}

template <int PHI, bool F16, int MH>
__global__ void __launch_bounds__(PGS_THREADS, 3)
hstu_paged_rows_kernel(const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ PagedParams p) {
  constexpr int R = 8 * MH;
  constexpr bool kSoftmax = PHI == HSTU_ACT_SOFTMAX;
  constexpr float kScale = phi_scale<PHI>();
  constexpr int kBand = PGS_KEYS + R + 4;  // biases of a tile, from a multiple of 4 down
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  namespace cg = cooperative_groups;
  // the same offset in every CTA of a cluster: shared memory is read across it
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int split = static_cast<int>(blockIdx.x % p.nsplit);
  const int64_t id = blockIdx.x / p.nsplit;
  const int h = static_cast<int>(id % p.H);
  const int g = static_cast<int>((id / p.H) % p.groups);
  int u = static_cast<int>(id / p.H / p.groups);
  if (p.sorted)
    u = paged_nth_longest(p, u, reinterpret_cast<int32_t*>(smem + PgsSmem::kMl),
                          reinterpret_cast<int*>(smem + PgsSmem::kMlC));
  const int warp = warp_id(), lane = lane_id(), tid = threadIdx.x;
  PagedSeq<PGS_KEYS> s;
  const int r0 = g * R;
  const int go = paged_seq(p, u, r0, R, s);
  if (go <= 0) {  // the same for the whole cluster, before any barrier
    if (go < 0 && tid == 0) record_status(HSTU_ERR_DEVICE_CHECK);
    return;
  }
  const int rows = min(R, s.c - r0);
  const int n_all = p.lengths[s.seq];
  const int i0 = n_all - s.c + r0;  // position of the group's first row
  const int64_t t_last = p.q_ts[s.q0 + s.c - 1];
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + PgsSmem::kBars);
  uint64_t* bar_empty = bar_full + PGS_STAGES;
  volatile int* sAbort = reinterpret_cast<volatile int*>(smem + PgsSmem::kAbort);
  float* sTime = reinterpret_cast<float*>(smem + PgsSmem::kTime);
  int32_t* sThr = reinterpret_cast<int32_t*>(smem + PgsSmem::kThr);
  int4* sOct = reinterpret_cast<int4*>(smem + PgsSmem::kOct);
  float4* sOrt = reinterpret_cast<float4*>(smem + PgsSmem::kOrt);
  float2* sMl = reinterpret_cast<float2*>(smem + PgsSmem::kMl);
  float2* sMlC = reinterpret_cast<float2*>(smem + PgsSmem::kMlC);
  if (tid == 0) {
    for (int k = 0; k < PGS_STAGES; ++k) {
      mbar_init(&bar_full[k], 1 + 32);  // the expect-tx arrival, the producer lanes' copies
      mbar_init(&bar_empty[k], PGS_WARPS);
    }
    *sAbort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtl ctl{sAbort, p.timeout_ns};
  const int k_begin = static_cast<int>(static_cast<int64_t>(s.n_tiles) * split / p.nsplit);
  const int k_end = static_cast<int>(static_cast<int64_t>(s.n_tiles) * (split + 1) / p.nsplit);

  if (warp == PGS_WARPS) {
    // ---------------- producer
    const int32_t* tab = p.table + static_cast<int64_t>(s.seq) * p.max_blocks;
    const float* rp = p.rab_pos + static_cast<int64_t>(h) * p.P;
    const int psl = p.ps_log2, ps = 1 << psl;
    const int boxl = min(psl, 6), box = 1 << boxl;  // rows of a box: a page or 64 rows of one
    const int nbl = 6 - boxl;                       // log2 of the boxes of a tile
    const int32_t oob = static_cast<int32_t>((static_cast<int64_t>(p.num_pages) * 2 * p.H) << psl);
    const int per = 32 >> nbl;  // tiles per batch of block-table entries
    const int bx = lane & ((1 << nbl) - 1);
    // One lane's box of a batch: the page of box bx of tile k0 + lane / boxes
    struct Box {
      int page;  // -1: no row sees it
      int j;     // its first position
    };
    auto load_box = [&](int k0) -> Box {
      Box b{-1, 0};
      const int kk = k0 + (lane >> nbl);
      if (kk >= k_end) return b;
      b.j = s.tile(kk) * PGS_KEYS + (bx << boxl);
      if (b.j < s.n && (b.j < s.sink_end || b.j + box > s.lo)) {
        b.page = tab[b.j >> psl];
        if (b.page < 0) b.page = INT32_MAX;  // seen, and no page
      }
      return b;
    };
    Box cur = load_box(k_begin);
    int st = 0, issued = 0;
    uint32_t ph = 1;
    bool ok_all = true;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t box_dst = sbase + PgsSmem::kK + (bx << boxl) * 128;
    const uint32_t side0 = sbase + PgsSmem::kSide;
    const bool rp16 = (reinterpret_cast<uintptr_t>(rp) & 15u) == 0;
    for (int kb = k_begin; kb < k_end && ok_all; kb += per) {
      const Box next = load_box(kb + per);
      // tensor-map rows of the lane's box (rows past the tensor read as zeros) and
      // the index of its first timestamp, -1 where there is none
      int32_t row_k = oob, row_v = oob, ts0 = -1;
      if (cur.page >= 0) {
        if (cur.page < p.num_pages) {
          const int32_t slot = cur.j & (ps - 1);
          row_k = ((cur.page * 2 * p.H + h) << psl) + slot;
          row_v = row_k + (p.H << psl);
          ts0 = (cur.page << psl) + slot;
        } else {
          record_status(HSTU_ERR_DEVICE_CHECK);
        }
      }
      const unsigned with_ts = __ballot_sync(0xffffffffu, ts0 >= 0);
      const int n_here = min(per, k_end - kb);
      for (int t = 0; t < n_here; ++t) {
        // Biases by position, ascending from entry 0 at offset d4: row r and column c
        // are at y = (i0 + r) - (j0 + c) - d4.  One copy inside the table, lane by
        // lane where the offsets leave it and clamp.
        const int j0 = s.tile(kb + t) * PGS_KEYS;
        const int d4 = paged_band0(i0 - j0, PGS_KEYS);
        const bool bulk = rp16 && d4 >= 0 && d4 + kBand <= p.P;
        int ok = 0;
        if (lane == 0) {
          ok = mbar_wait(&bar_empty[st], ph, ctl) ? 1 : 0;
          if (ok) {
            const unsigned mine = (with_ts >> (t << nbl)) & ((1u << (1 << nbl)) - 1u);
            mbar_arrive_expect_tx(&bar_full[st], 2 * PGS_TILE_BYTES + (__popc(mine) << (boxl + 3)) +
                                                     (bulk ? kBand * 4 : 0));
          }
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
          ok_all = false;
          break;
        }
        const uint32_t side = side0 + st * PgsSmem::kSideBytes;
        if ((lane >> nbl) == t) {
          const uint32_t dst = box_dst + st * PGS_TILE_BYTES;
          tma_load_2d_to(dst, &tm_kv, &bar_full[st], 0, row_k);
          tma_load_2d_to(dst + (PgsSmem::kV - PgsSmem::kK), &tm_kv, &bar_full[st], 0, row_v);
          // a part's times, unwritten slots and all: only those of seen keys are used
          if (ts0 >= 0) bulk_load(side + (bx << (boxl + 3)), p.ts + ts0, 8u << boxl, &bar_full[st]);
        }
        const uint32_t band = side + PGS_KEYS * 8;
        if (bulk) {
          if (lane == 0) bulk_load(band, rp + d4, kBand * 4, &bar_full[st]);
        } else {
          for (int y = lane; y < kBand; y += 32) cp_async4(band + 4 * y, rp + min(max(d4 + y, 0), p.P - 1));
        }
        cp_async_arrive(&bar_full[st]);
        ++issued;
        if (++st == PGS_STAGES) {
          st = 0;
          ph ^= 1u;
        }
      }
      cur = next;
    }
    // every issued load lands before shared memory is reused or released
    if (lane == 0)
      for (int k = max(0, issued - PGS_STAGES); k < issued; ++k)
        mbar_wait_drain(&bar_full[k % PGS_STAGES], (k / PGS_STAGES) & 1, p.timeout_ns);
    __syncwarp();
  }

  // ---------------- compute warps
  float o[8][4];
  float m_run[MH], l_run[MH];
#pragma unroll
  for (int b = 0; b < 8; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[b][e] = 0.0f;
#pragma unroll
  for (int a = 0; a < MH; ++a) {
    m_run[a] = -INFINITY;
    l_run[a] = 0.0f;
  }
  const int gr = lane >> 2, tq = lane & 3;  // row and column pair of the MMA fragments
  if (warp < PGS_WARPS) {
    // bias tables, while the first tiles are on their way
    const float* rt_g = p.rab_time + static_cast<int64_t>(h) * p.Tb;
    for (int k = tid; k < p.Tb; k += PGS_WARPS * 32) {
      sTime[k] = kScale * __ldg(rt_g + k);
      sThr[k] = p.thr[k];
    }
    if (tid < 32) {
      const int4 o4 = p.oct[tid];
      auto tb = [&](int b) { return kScale * __ldg(rt_g + min(max(b, 0), p.Tb - 1)); };
      sOct[tid] = o4;
      sOrt[tid] = make_float4(tb(o4.w), tb(o4.w + 1), tb(o4.w + 2), tb(o4.w + 3));
    }
    named_barrier_sync(1, PGS_WARPS * 32);
    uint32_t qf[4][4];
    int32_t ti[MH];
    int64_t bound[MH];  // latest time still in the row's current bucket
    float rt[MH];       // and its bias
#pragma unroll
    for (int a = 0; a < 2; ++a) {  // rows gr + 8 a
      const int r = gr + 8 * a;
      const bool in = r < rows;
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + (s.q0 + r0 + (in ? r : 0)) * p.ldq + h * 64;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qf[k][a + 2 * e] = in ? __ldg(reinterpret_cast<const uint32_t*>(q + 16 * k + 8 * e + 2 * tq)) : 0u;
      if (a < MH) {
        ti[a] = in ? paged_rel(p.q_ts[s.q0 + r0 + r], t_last) : PG_T0;
        bound[a] = INT64_MIN;  // the first chunk looks its buckets up
        rt[a] = 0.0f;
      }
    }
    const uint32_t sbase = smem_u32(smem);
    const int wk = warp * 16;  // this warp's keys of a tile
    // ldmatrix rows of this lane: K (keys, then the two k halves), V (key halves, then columns)
    const int krow = wk + ((lane >> 4) << 3) + (lane & 7), kch = (lane >> 3) & 1;
    const int vrow = wk + (((lane >> 3) & 1) << 3) + (lane & 7), vch = lane >> 4;
    const uint32_t kaddr = sbase + PgsSmem::kK + krow * 128, vaddr = sbase + PgsSmem::kV + vrow * 128;
    const int i_last = i0 + rows - 1;
    // the tiles [f_lo, f_hi) of the list that every row sees whole
    const int f_lo = p.window == 0 ? 0 : s.n_sink + max(0, (i_last - p.window + PGS_KEYS) / PGS_KEYS - s.first);
    const int f_hi = s.n_sink + (i0 + 1) / PGS_KEYS - s.first;
    int st = 0;
    uint32_t ph = 0;
    for (int kk = k_begin; kk < k_end; ++kk) {
      const bool ok = mbar_wait(&bar_full[st], ph, ctl);
      const int j_tile = s.tile(kk) * PGS_KEYS, j0 = j_tile + wk;  // this warp's first key
      const uint32_t soff = st * PGS_TILE_BYTES;
      const int64_t* times = reinterpret_cast<const int64_t*>(smem + PgsSmem::kSide + st * PgsSmem::kSideBytes);
      // every row sees every key of this warp; some key is seen by no row
      bool full = true, ragged = false;
      if (kk < f_lo || kk >= f_hi) {
        full = j0 + 15 <= i0 && (p.window == 0 || j0 > i_last - p.window || j0 + 16 <= p.sinks);
        ragged = j0 + 16 > s.n || (j0 < s.lo && j0 + 16 > s.sink_end);
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      // rows of V that no row sees may hold anything (a page's unwritten slots): P = 0
      // times a NaN is a NaN, so they are cleared
      if (ragged) {
        for (int e = lane; e < 16 * 8; e += 32)
          if (!s.seen(j0 + (e >> 3)))
            *reinterpret_cast<uint4*>(smem + PgsSmem::kV + soff + (wk + (e >> 3)) * 128 + (e & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
      }
      float sc[2][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t kf[4];
        ldsm_x4(kaddr + soff + (((2 * k + kch) ^ (krow & 7)) << 4), kf);
        if (k == 0) {
          mma_m16n8k16_first<F16>(sc[0], qf[k], kf[0], kf[1]);
          mma_m16n8k16_first<F16>(sc[1], qf[k], kf[2], kf[3]);
        } else {
          mma_m16n8k16<F16>(sc[0], qf[k], kf[0], kf[1]);
          mma_m16n8k16<F16>(sc[1], qf[k], kf[2], kf[3]);
        }
      }
      // ---- element work: columns wk + 8 b + 2 tq + {0, 1}, rows gr + 8 a
      // bias of row 0, this warp's column 0
      const float* band =
          reinterpret_cast<const float*>(times + PGS_KEYS) + (i0 - j0) - paged_band0(i0 - j_tile, PGS_KEYS);
      // Time bucket of a row: it only falls along the keys, so while the chunk's last key
      // has not passed the row's edge (`bound`) the row's one bias holds.  Keys that
      // no row sees have no time: such chunks look every bucket up, and leave no bound.
      const int64_t t_end = times[wk + 15];
      bool steady = !ragged;
#pragma unroll
      for (int a = 0; a < MH; ++a) steady = steady && t_end <= bound[a];
      steady = __all_sync(0xffffffffu, steady);
      float rtv[MH][4];
      if (steady) {
#pragma unroll
        for (int a = 0; a < MH; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) rtv[a][e] = rt[a];
      } else {
        // the earliest visible event is among the CTA's first keys
        if (kk == k_begin && lane < 16 && s.seen(j0 + lane) && t_last - times[wk + lane] > PG_T0)
          record_status(HSTU_ERR_DEVICE_CHECK);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int32_t kt = paged_rel(times[wk + 8 * (e >> 1) + 2 * tq + (e & 1)], t_last);
#pragma unroll
          for (int a = 0; a < MH; ++a) rtv[a][e] = time_bias_octave(ti[a] - kt, sOct, sOrt);
        }
#pragma unroll
        for (int a = 0; a < MH; ++a) {
          // the bucket of the chunk's last key holds until a key passes its edge
          const int bk = time_bucket_octave(ti[a] - paged_rel(t_end, t_last), sOct);
          rt[a] = sTime[bk];
          bound[a] = ragged ? INT64_MIN : (bk == 0 ? INT64_MAX : t_last - PG_T0 + (ti[a] - sThr[bk]));
        }
      }
      uint32_t pf[4];
#pragma unroll
      for (int a = 0; a < MH; ++a) {
        const int r = gr + 8 * a, i = i0 + r;
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = fmaf(sc[e >> 1][2 * a + (e & 1)] + band[r - (8 * (e >> 1) + 2 * tq + (e & 1))], kScale, rtv[a][e]);
        auto vis = [&](int e) {
          const int j = j0 + 8 * (e >> 1) + 2 * tq + (e & 1);
          return j <= i && (p.window == 0 || j > i - p.window || j < p.sinks);
        };
        if constexpr (kSoftmax) {
          // P = 2^(x - m) with a running m that follows the rows' maxima only when one of them
          // is more than 8 above it: P stays below 2^8, no sum loses anything, and most
          // tiles need neither the quad's maximum nor a rescaled O
          float cm = -INFINITY;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!full) x[e] = vis(e) ? x[e] : -INFINITY;
            cm = fmaxf(cm, x[e]);
          }
          if (__any_sync(0xffffffffu, cm > m_run[a] + 8.0f)) {
            cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 1));
            cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 2));
            const float mn = fmaxf(m_run[a], cm);
            const float f = mn > -INFINITY ? ex2_approx(m_run[a] - mn) : 1.0f;
            m_run[a] = mn;
            l_run[a] *= f;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              o[b][2 * a] *= f;
              o[b][2 * a + 1] *= f;
            }
          }
          const float mm = m_run[a] > -INFINITY ? m_run[a] : 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = ex2_approx(x[e] - mm);
            l_run[a] += x[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (PHI == HSTU_ACT_SILU) x[e] = fmaf(x[e], tanh_approx(x[e]), x[e]);
            else if constexpr (PHI == HSTU_ACT_RELU) x[e] = fmaxf(x[e], 0.0f);
            if (!full) x[e] = vis(e) ? x[e] : 0.0f;
          }
        }
        // P in the operand type: the MMA takes both operands in one type
        pf[a] = pack_16<F16>(x[0], x[1]);
        pf[a + 2] = pack_16<F16>(x[2], x[3]);
      }
      if constexpr (MH == 1) pf[1] = pf[3] = 0u;  // rows 8 .. 15 do not exist
      // ---- O += P V
#pragma unroll
      for (int b = 0; b < 8; b += 2) {
        uint32_t vf[4];
        ldsm_x4_t(vaddr + soff + (((b + vch) ^ (vrow & 7)) << 4), vf);
        mma_m16n8k16<F16>(o[b], pf, vf[0], vf[1]);
        mma_m16n8k16<F16>(o[b + 1], pf, vf[2], vf[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_empty[st]);
      if (++st == PGS_STAGES) {
        st = 0;
        ph ^= 1u;
      }
    }
  }
  __syncthreads();  // the stages are idle: the partial sums go over them
  float* sO = reinterpret_cast<float*>(smem);
  if (warp < PGS_WARPS) {
#pragma unroll
    for (int a = 0; a < MH; ++a) {
      const int r = gr + 8 * a;
#pragma unroll
      for (int b = 0; b < 8; ++b)
        *reinterpret_cast<float2*>(sO + (warp * R + r) * PGS_OLD + 8 * b + 2 * tq) =
            make_float2(o[b][2 * a], o[b][2 * a + 1]);
      if constexpr (kSoftmax) {
        float l = l_run[a];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (tq == 0) sMl[warp * R + r] = make_float2(m_run[a], l);
      }
    }
  }
  __syncthreads();
  // the CTA's sums over its warps, in place of warp 0's (8 rows x 16 lanes a step)
  const bool alone = p.nsplit == 1;
  const int c4 = tid & 15;
  const float inv_n = kSoftmax ? 1.0f : 1.0f / static_cast<float>(n_all);
  if (warp < PGS_WARPS) {
    for (int r = tid >> 4; r < 8 * MH; r += 8) {
      float f[PGS_WARPS], m = -INFINITY, l = 0.0f;
#pragma unroll
      for (int w = 0; w < PGS_WARPS; ++w) f[w] = 1.0f;
      if constexpr (kSoftmax) {
#pragma unroll
        for (int w = 0; w < PGS_WARPS; ++w) m = fmaxf(m, sMl[w * R + r].x);
#pragma unroll
        for (int w = 0; w < PGS_WARPS; ++w) {
          const float2 v = sMl[w * R + r];
          f[w] = v.x > -INFINITY ? ex2_approx(v.x - m) : 0.0f;
          l = fmaf(v.y, f[w], l);
        }
      }
      float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < PGS_WARPS; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(sO + (w * R + r) * PGS_OLD + 4 * c4);
        t.x = fmaf(v.x, f[w], t.x);
        t.y = fmaf(v.y, f[w], t.y);
        t.z = fmaf(v.z, f[w], t.z);
        t.w = fmaf(v.w, f[w], t.w);
      }
      if (alone) {
        const float k = kSoftmax ? (l > 0.0f ? 1.0f / l : 0.0f) : inv_n;
        paged_store<F16>(p, s.q0 + r0 + r, h, c4, make_float4(t.x * k, t.y * k, t.z * k, t.w * k), r < rows);
      } else {
        *reinterpret_cast<float4*>(sO + r * PGS_OLD + 4 * c4) = t;  // read by this thread alone before
        if (kSoftmax && c4 == 0) sMlC[r] = make_float2(m, l);
      }
    }
  }
  if (alone) return;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  if (warp < PGS_WARPS) {
    // rank `split` takes rows split, split + nsplit, .. (16 lanes a row; every lane of a
    // warp goes through the same steps)
    for (int base = 0; base < 8 * MH; base += 8 * p.nsplit) {
      const int r_of = base + split + p.nsplit * (tid >> 4);
      const int r = min(r_of, 8 * MH - 1);
      float m = -INFINITY, l = 0.0f;
      if constexpr (kSoftmax)
        for (int k = 0; k < p.nsplit; ++k) m = fmaxf(m, cluster.map_shared_rank(sMlC, k)[r].x);
      float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int k = 0; k < p.nsplit; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(sO, k) + r * PGS_OLD + 4 * c4);
        float f = 1.0f;
        if constexpr (kSoftmax) {
          const float2 ml = cluster.map_shared_rank(sMlC, k)[r];
          f = ml.x > -INFINITY ? ex2_approx(ml.x - m) : 0.0f;
          l = fmaf(ml.y, f, l);
        }
        t.x = fmaf(v.x, f, t.x);
        t.y = fmaf(v.y, f, t.y);
        t.z = fmaf(v.z, f, t.z);
        t.w = fmaf(v.w, f, t.w);
      }
      const float k = kSoftmax ? (l > 0.0f ? 1.0f / l : 0.0f) : inv_n;
      paged_store<F16>(p, s.q0 + r0 + r, h, c4, make_float4(t.x * k, t.y * k, t.z * k, t.w * k), r_of < rows);
    }
  }
  cluster.sync();  // no CTA leaves while another reads its partial sums
}

// ---------------------------------------------------------------- many rows

// 16-bit operands, 256 query rows per CTA (two 128-row tcgen05 tiles), keys split
// over a cluster.  Bound by the element work, one pre-activation, bias and phi2 per
// (row, key): the layout is hstu_attn_kernel's (16 element warps in two groups of
// two warpgroups, a producer warp, one MMA issuer per query tile; S in three
// tensor-memory buffers per tile, P written back over S, O += P V from tensor
// memory), fed from pages: K and V by TMA boxes, key times and the tile's band of
// position biases by bulk copies, so that one stage carries all that its 64 keys
// need and no per-sequence table is staged.  Both tiles walk the whole list of key
// tiles (the earlier rows waste at most the two that only later rows see).  A group of
// at most 128 rows has no second tile: then both halves of the machinery take the
// same rows and every other key tile each, and their results are added at the end.
// Softmax takes two passes, the first for each row's maximum and sum.
// Measured (B200, 8 heads, bf16): 512 events of each of 8 users over 8192 162 us,
// 411 TFLOP/s (25% of the measured matmul peak; the tensor pipe is 23% active, the
// schedulers issue in 63% of the cycles, about 11 thread instructions per element).
// With every event at the same time, so that no time bucket has to be looked up, it
// takes 141 us.  16 columns at a time (no register spills, twice the loads and votes): 177 us.
constexpr int PGT_KEYS = 64;
constexpr int PGT_ROWS = 256;
constexpr int PGT_STAGES = 6;
constexpr int PGT_SBUF = 3;
constexpr int PGT_THREADS = 608;
constexpr int PGT_PRODUCER = 16;
constexpr int PGT_MMA = 17;  // + query tile
constexpr uint32_t PGT_TILE_BYTES = PGT_KEYS * 128;
constexpr int PGT_BAND = PGT_KEYS + PGT_ROWS + 4;
constexpr int PGT_OLD = 68;

struct PgtSmem {
  static constexpr uint32_t kQ = 0;                                   // 2 x 16 KB
  static constexpr uint32_t kK = kQ + 2 * 128 * 128;
  static constexpr uint32_t kV = kK + PGT_STAGES * PGT_TILE_BYTES;
  static constexpr uint32_t kSide = kV + PGT_STAGES * PGT_TILE_BYTES;  // per stage: times, biases
  static constexpr uint32_t kSideBytes = PGT_KEYS * 8 + PGT_BAND * 4;
  static constexpr uint32_t kTime = kSide + PGT_STAGES * kSideBytes;
  static constexpr uint32_t kThr = kTime + MAX_TIME_BUCKETS * 4;
  static constexpr uint32_t kOct = kThr + MAX_TIME_BUCKETS * 4;
  static constexpr uint32_t kOrt = kOct + 32 * 16;
  static constexpr uint32_t kMl = kOrt + 32 * 16;                      // 2 halves x 256 rows float2
  static constexpr uint32_t kMlC = kMl + 2 * PGT_ROWS * 8;             // 256 rows float2
  static constexpr uint32_t kBars = kMlC + PGT_ROWS * 8;
  static constexpr uint32_t kMisc = kBars + 48 * 8;
  static constexpr uint32_t kBytes = kMisc + 64 + 1024;                // + align slack
  static_assert(kSideBytes % 16 == 0 && kSide % 16 == 0, "bulk copies");
  static_assert(PGT_ROWS * PGT_OLD * 4 <= kSide, "the partial sums fit over Q, K and V");
};

enum : int {
  PGB_Q = 0,
  PGB_FULL = 1,                             // + stage
  PGB_EMPTY = PGB_FULL + PGT_STAGES,        // + stage
  PGB_S = PGB_EMPTY + PGT_STAGES,           // + PGT_SBUF * tile + buffer
  PGB_P = PGB_S + 2 * PGT_SBUF,             // + PGT_SBUF * tile + buffer
  PGB_DONE = PGB_P + 2 * PGT_SBUF,          // + tile: every MMA of the tile completed
  PGB_TAIL = PGB_DONE + 2,                  // the loads of a tile that is cleaned before use
  PGB_COUNT = PGB_TAIL + 1
};
static_assert(PGB_COUNT <= 48, "barrier slots");

// Pre-activations h = scale * (s + rab_pos) + scale * rab_time of one row and 32
// keys, handed to sink(c, h2) in pairs (c even).  bp[-c]: the bias of column c; kts:
// the keys' times.  `w`: the row's bucket and the latest time still in it.
struct PagedWalk {
  int32_t ti;      // the row's time, paged_rel
  int b;           // bucket of the last key looked up
  int64_t bound;   // keys up to this time are still in it
  float rt;
};
template <class Sink>
__device__ __forceinline__ void paged_chunk(const uint32_t (&sv)[32], Sink&& sink, const float* bp,
                                            const int64_t* kts, bool ragged, bool live, PagedWalk& w,
                                            int64_t t_last, const float* sTime, const int32_t* sThr,
                                            const int4* sOct, const float4* sOrt, uint64_t scale2) {
  const unsigned all = 0xffffffffu;
  auto pre = [&](int c, uint64_t rt2) -> uint64_t {
    const uint64_t s2 = f2_pack(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
    return f2_fma(f2_add(s2, f2_pack(bp[-c], bp[-c - 1])), scale2, rt2);
  };
  const int64_t t_end = kts[31];
  // every row's bucket holds to the last key
  if (!ragged && __all_sync(all, !live || t_end <= w.bound)) {
    if (live) {
      const uint64_t rt2 = f2_pack(w.rt, w.rt);
#pragma unroll
      for (int c = 0; c < 32; c += 2) sink(c, pre(c, rt2));
    }
    return;
  }
  const int64_t t0 = kts[0];
  const int b0 = t0 <= w.bound ? w.b : time_bucket_octave(w.ti - paged_rel(t0, t_last), sOct);
  const int b1 = t_end <= w.bound ? w.b : time_bucket_octave(w.ti - paged_rel(t_end, t_last), sOct);
  auto edge_of = [&](int b) -> int64_t { return b == 0 ? INT64_MAX : t_last - PG_T0 + (w.ti - sThr[b]); };
  if (!ragged && __all_sync(all, !live || b0 - b1 <= 1)) {
    // at most two buckets in a row: keys up to the first one's edge, and the others
    if (live) {
      const float hi = sTime[b0], lo = sTime[b1];
      const int64_t edge = b0 == b1 ? INT64_MAX : edge_of(b0);
#pragma unroll
      for (int c = 0; c < 32; c += 2)
        sink(c, pre(c, f2_pack(kts[c] <= edge ? hi : lo, kts[c + 1] <= edge ? hi : lo)));
    }
  } else if (live) {
#pragma unroll
    for (int c = 0; c < 32; c += 2)
      sink(c, pre(c, f2_pack(time_bias_octave(w.ti - paged_rel(kts[c], t_last), sOct, sOrt),
                             time_bias_octave(w.ti - paged_rel(kts[c + 1], t_last), sOct, sOrt))));
  }
  // keys that no row sees have no time: the next chunk looks its buckets up
  w.b = b1;
  w.rt = sTime[b1];
  w.bound = ragged ? INT64_MIN : edge_of(b1);
}

template <int PHI, bool F16>
__global__ void __launch_bounds__(PGT_THREADS, 1)
hstu_paged_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                       const __grid_constant__ PagedParams p) {
  constexpr bool kSoftmax = PHI == HSTU_ACT_SOFTMAX;
  constexpr int kPasses = kSoftmax ? 2 : 1;
  constexpr float kScale = phi_scale<PHI>();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  namespace cg = cooperative_groups;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int split = static_cast<int>(blockIdx.x % p.nsplit);
  const int64_t id = blockIdx.x / p.nsplit;
  const int h = static_cast<int>(id % p.H);
  // later rows see more keys: first
  const int g = p.groups - 1 - static_cast<int>((id / p.H) % p.groups);
  const int u = static_cast<int>(id / p.H / p.groups);
  const int warp = warp_id(), lane = lane_id(), tid = threadIdx.x;
  PagedSeq<PGT_KEYS> s;
  const int r0 = g * PGT_ROWS;
  const int go = paged_seq(p, u, r0, PGT_ROWS, s);
  if (go <= 0) {  // the same for the whole cluster, before any barrier or allocation
    if (go < 0 && tid == 0) record_status(HSTU_ERR_DEVICE_CHECK);
    return;
  }
  const int rows = min(PGT_ROWS, s.c - r0);
  const bool dual = rows <= 128;  // one query tile: key tiles alternate between the groups
  const int n_all = p.lengths[s.seq];
  const int i0 = n_all - s.c + r0;
  const int64_t t_last = p.q_ts[s.q0 + s.c - 1];
  const int k_begin = static_cast<int>(static_cast<int64_t>(s.n_tiles) * split / p.nsplit);
  const int k_end = static_cast<int>(static_cast<int64_t>(s.n_tiles) * (split + 1) / p.nsplit);
  const int n_k = k_end - k_begin;      // key tiles of this CTA
  const int n_items = kPasses * n_k;    // stages it goes through
  // key tile k of the CTA is group t's; each of its passes has own_k of them
  auto mine = [&](int k, int t) { return !dual || (k & 1) == t; };
  auto own_k = [&](int t) { return dual ? (n_k + 1 - t) >> 1 : n_k; };
  // stage of the gi-th item of group t (its tiles, once per pass)
  auto stage_of = [&](int gi, int t) {
    const int nk = own_k(t), pass = gi >= nk ? 1 : 0, k = gi - pass * nk;
    return pass * n_k + (dual ? 2 * k + t : k);
  };

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + PgtSmem::kBars);
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(smem + PgtSmem::kMisc);
  volatile int* sAbort = reinterpret_cast<volatile int*>(smem + PgtSmem::kMisc + 4);
  float* sTime = reinterpret_cast<float*>(smem + PgtSmem::kTime);
  int32_t* sThr = reinterpret_cast<int32_t*>(smem + PgtSmem::kThr);
  int4* sOct = reinterpret_cast<int4*>(smem + PgtSmem::kOct);
  float4* sOrt = reinterpret_cast<float4*>(smem + PgtSmem::kOrt);
  float2* sMl = reinterpret_cast<float2*>(smem + PgtSmem::kMl);
  float2* sMlC = reinterpret_cast<float2*>(smem + PgtSmem::kMlC);
  if (tid == 0) {
    mbar_init(&bars[PGB_Q], 1);
    for (int k = 0; k < PGT_STAGES; ++k) {
      mbar_init(&bars[PGB_FULL + k], 1 + 32);  // the expect-tx arrival, the producer lanes' copies
      mbar_init(&bars[PGB_EMPTY + k], 2);      // one commit per issuer
    }
    for (int k = 0; k < 2 * PGT_SBUF; ++k) {
      mbar_init(&bars[PGB_S + k], 1);
      mbar_init(&bars[PGB_P + k], 256);
    }
    mbar_init(&bars[PGB_DONE], 1);
    mbar_init(&bars[PGB_DONE + 1], 1);
    mbar_init(&bars[PGB_TAIL], 1);
    *sAbort = 0;
    fence_mbar_init();
  }
  if (warp == PGT_MMA) {
    tmem_alloc(sTmem, 512);
    tmem_relinquish();
  }
  const float* rt_g = p.rab_time + static_cast<int64_t>(h) * p.Tb;
  for (int k = tid; k < p.Tb; k += PGT_THREADS) {
    sTime[k] = kScale * __ldg(rt_g + k);
    sThr[k] = p.thr[k];
  }
  if (tid < 32) {
    const int4 o4 = p.oct[tid];
    auto tb = [&](int b) { return kScale * __ldg(rt_g + min(max(b, 0), p.Tb - 1)); };
    sOct[tid] = o4;
    sOrt[tid] = make_float4(tb(o4.w), tb(o4.w + 1), tb(o4.w + 2), tb(o4.w + 3));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sTmem;
  const WaitCtl ctl{sAbort, p.timeout_ns};

  if (warp == PGT_PRODUCER) {
    // ---------------- producer (the few-rows kernel's, with two more cares: pass 0 of the
    // softmax leaves V out, and V rows that no row sees are cleared before the MMAs read them)
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[PGB_Q], (dual ? 1 : 2) * 128 * 128);
      const int32_t qrow = static_cast<int32_t>(s.q0 + r0);
      tma_load_2d(smem + PgtSmem::kQ, &tm_q, &bars[PGB_Q], h * 64, qrow);
      if (!dual) tma_load_2d(smem + PgtSmem::kQ + 128 * 128, &tm_q, &bars[PGB_Q], h * 64, qrow + 128);
    }
    const int32_t* tab = p.table + static_cast<int64_t>(s.seq) * p.max_blocks;
    const float* rp = p.rab_pos + static_cast<int64_t>(h) * p.P;
    const int psl = p.ps_log2, ps = 1 << psl;
    const int boxl = min(psl, 6), box = 1 << boxl, nbl = 6 - boxl;
    const int32_t oob = static_cast<int32_t>((static_cast<int64_t>(p.num_pages) * 2 * p.H) << psl);
    const int per = 32 >> nbl, bx = lane & ((1 << nbl) - 1);
    const bool rp16 = (reinterpret_cast<uintptr_t>(rp) & 15u) == 0;
    const uint32_t sbase = smem_u32(smem);
    int st = 0, issued = 0, tails = 0;
    uint32_t ph = 1;
    bool ok_all = true;
    for (int pass = 0; pass < kPasses && ok_all; ++pass) {
      const bool with_v = pass == kPasses - 1;
      auto load_page = [&](int k0, int& j) -> int {
        const int kk = k0 + (lane >> nbl);
        if (kk >= k_end) return -1;
        j = s.tile(kk) * PGT_KEYS + (bx << boxl);
        if (j >= s.n || (j >= s.sink_end && j + box <= s.lo)) return -1;
        const int page = tab[j >> psl];
        return page < 0 ? INT32_MAX : page;  // seen, and no page
      };
      int j_cur = 0, j_next = 0;
      int cur = load_page(k_begin, j_cur);
      for (int kb = k_begin; kb < k_end && ok_all; kb += per) {
        const int next = load_page(kb + per, j_next);
        int32_t row_k = oob, row_v = oob, ts0 = -1;
        if (cur >= 0) {
          if (cur < p.num_pages) {
            const int32_t slot = j_cur & (ps - 1);
            row_k = ((cur * 2 * p.H + h) << psl) + slot;
            row_v = row_k + (p.H << psl);
            ts0 = (cur << psl) + slot;
          } else {
            record_status(HSTU_ERR_DEVICE_CHECK);
          }
        }
        const unsigned with_ts = __ballot_sync(0xffffffffu, ts0 >= 0);
        const int n_here = min(per, k_end - kb);
        for (int t = 0; t < n_here; ++t) {
          const int j0 = s.tile(kb + t) * PGT_KEYS;
          const int d4 = paged_band0(i0 - j0, PGT_KEYS);
          const bool bulk = rp16 && d4 >= 0 && d4 + PGT_BAND <= p.P;
          // keys that no row sees: their slots may hold anything, and 0 times a NaN is a NaN
          const bool clean = with_v && (j0 + PGT_KEYS > s.n || (j0 < s.lo && j0 + PGT_KEYS > s.sink_end));
          uint64_t* full = &bars[PGB_FULL + st];
          uint64_t* land = clean ? &bars[PGB_TAIL] : full;
          int ok = 0;
          if (lane == 0) {
            ok = mbar_wait(&bars[PGB_EMPTY + st], ph, ctl) ? 1 : 0;
            if (ok) {
              const unsigned mine = (with_ts >> (t << nbl)) & ((1u << (1 << nbl)) - 1u);
              mbar_arrive_expect_tx(land, (with_v ? 2 : 1) * PGT_TILE_BYTES + (__popc(mine) << (boxl + 3)) +
                                              (bulk ? PGT_BAND * 4 : 0));
            }
          }
          if (!__shfl_sync(0xffffffffu, ok, 0)) {
            ok_all = false;
            break;
          }
          const uint32_t side = sbase + PgtSmem::kSide + st * PgtSmem::kSideBytes;
          if ((lane >> nbl) == t) {
            const uint32_t dst = sbase + PgtSmem::kK + st * PGT_TILE_BYTES + (bx << boxl) * 128;
            tma_load_2d_to(dst, &tm_kv, land, 0, row_k);
            if (with_v) tma_load_2d_to(dst + (PgtSmem::kV - PgtSmem::kK), &tm_kv, land, 0, row_v);
            if (ts0 >= 0) bulk_load(side + (bx << (boxl + 3)), p.ts + ts0, 8u << boxl, land);
          }
          const uint32_t band = side + PGT_KEYS * 8;
          if (bulk) {
            if (lane == 0) bulk_load(band, rp + d4, PGT_BAND * 4, land);
          } else {
            for (int y = lane; y < PGT_BAND; y += 32) cp_async4(band + 4 * y, rp + min(max(d4 + y, 0), p.P - 1));
          }
          if (clean) {
            // (a failed wait has raised the abort flag, which ends the other warps' waits)
            const bool landed = mbar_wait(&bars[PGB_TAIL], static_cast<uint32_t>(tails) & 1u, ctl);
            ++tails;
            if (__all_sync(0xffffffffu, landed)) {
              uint8_t* v = smem + PgtSmem::kV + st * PGT_TILE_BYTES;
              for (int e = lane; e < PGT_KEYS * 8; e += 32)
                if (!s.seen(j0 + (e >> 3)))
                  *reinterpret_cast<uint4*>(v + (e >> 3) * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
          }
          cp_async_arrive(full);
          ++issued;
          if (++st == PGT_STAGES) {
            st = 0;
            ph ^= 1u;
          }
        }
        cur = next;
        j_cur = j_next;
      }
    }
    // every issued load lands before shared memory is reused or released
    if (lane == 0) {
      mbar_wait_drain(&bars[PGB_Q], 0, p.timeout_ns);
      for (int k = max(0, issued - PGT_STAGES); k < issued; ++k)
        mbar_wait_drain(&bars[PGB_FULL + k % PGT_STAGES], (k / PGT_STAGES) & 1, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp >= PGT_MMA) {
    // ---------------- MMA issuers
    const int t = warp - PGT_MMA;
    const bool leader = elect_one();
    constexpr uint32_t idesc_qk = idesc_16_f32(128, PGT_KEYS, false, false, F16);
    constexpr uint32_t idesc_pv = idesc_16_f32(128, 64, false, true, F16);
    const uint32_t tS = tmem + static_cast<uint32_t>(t * PGT_SBUF * 64);
    const uint32_t tO = tmem + static_cast<uint32_t>(2 * PGT_SBUF * 64 + t * 64);
    const uint64_t dQ = smem_desc_sw128(smem_u32(smem + PgtSmem::kQ + (dual ? 0 : t * 128 * 128)), 16, 1024);
    const uint64_t dK0 = smem_desc_sw128(smem_u32(smem + PgtSmem::kK), 16, 1024);
    const uint64_t dV0 = smem_desc_sw128(smem_u32(smem + PgtSmem::kV), 8192, 1024);
    constexpr uint64_t kStageDesc = PGT_TILE_BYTES >> 4;
    auto wait_all = [&](uint64_t* bar, uint32_t par) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, par, ctl));
    };
    bool ok = wait_all(&bars[PGB_Q], 0);
    tc_fence_after();
    int ready = 0;  // stages this warp has seen land
    auto await_kv = [&](int it) -> bool {
      while (ready <= it) {
        if (!wait_all(&bars[PGB_FULL + ready % PGT_STAGES], static_cast<uint32_t>(ready / PGT_STAGES) & 1u))
          return false;
        tc_fence_after();
        ++ready;
      }
      return true;
    };
    auto issue_s = [&](int it, int b) {
      const uint64_t dk = dK0 + static_cast<uint64_t>(it % PGT_STAGES) * kStageDesc;
      if (leader) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16_ss(tS + static_cast<uint32_t>(b * 64), dQ + 2 * k, dk + 2 * k, idesc_qk, k > 0 ? 1u : 0u);
        mma_commit(&bars[PGB_S + PGT_SBUF * t + b]);
      }
      __syncwarp();
    };
    // S of the next items is issued ahead of their turn, as far as the ring of stages
    // reaches when every other one of them is this group's
    const int ahead = dual ? 2 : PGT_SBUF;
    const int own_items = kPasses * own_k(t), first = (kPasses - 1) * own_k(t);  // O: the last pass
    for (int gi = 0; ok && gi < ahead && gi < own_items; ++gi) {
      ok = await_kv(stage_of(gi, t));
      if (ok) issue_s(stage_of(gi, t), gi);
    }
    int b = 0, b_next = ahead % PGT_SBUF, gi = 0;
    uint32_t ph = 0;
    for (int it = 0; ok && it < n_items; ++it) {
      if (mine(it >= n_k ? it - n_k : it, t)) {
        ok = wait_all(&bars[PGB_P + PGT_SBUF * t + b], ph);
        if (!ok) break;
        tc_fence_after();
        if (gi >= first && leader) {
          const uint64_t dv = dV0 + static_cast<uint64_t>(it % PGT_STAGES) * kStageDesc;
          const uint32_t a = tS + static_cast<uint32_t>(b * 64);
          // P of keys 0-31 sits at columns 0-15 of the buffer, of keys 32-63 at 32-47
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16_ts(tO, a + (k >> 1) * 32 + (k & 1) * 8, dv + 128 * k, idesc_pv, gi > first || k > 0 ? 1u : 0u);
        }
        __syncwarp();
        if (gi + ahead < own_items) {
          const int nx = stage_of(gi + ahead, t);
          ok = await_kv(nx);
          if (!ok) break;
          issue_s(nx, b_next);  // over a P that the MMAs so far read
        }
        ++gi;
        if (++b_next == PGT_SBUF) b_next = 0;
        if (++b == PGT_SBUF) {
          b = 0;
          ph ^= 1u;
        }
      } else {
        ok = await_kv(it);  // the other group's: only keeps the stage's count
        if (!ok) break;
      }
      if (leader) mma_commit(&bars[PGB_EMPTY + it % PGT_STAGES]);
      __syncwarp();
    }
    if (leader) mma_commit(&bars[PGB_DONE + t]);
    __syncwarp();
    mbar_wait_drain(&bars[PGB_DONE + t], 0, p.timeout_ns);
    __syncwarp();
  } else {
    // ---------------- element groups: rows 128 t .. of the group, key columns 32 half ..
    const int t = warp >> 3, half = (warp >> 2) & 1, r = (dual ? 0 : t * 128) + (tid & 127);
    const int slot = t * 128 + (tid & 127);  // where this group's results of the row go
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS0 = tmem + lane_off + static_cast<uint32_t>(t * PGT_SBUF * 64 + half * 32);
    const uint32_t tO = tmem + lane_off + static_cast<uint32_t>(2 * PGT_SBUF * 64 + t * 64 + half * 32);
    const bool valid = r < rows;
    const int i = i0 + r;
    const uint64_t scale2 = f2_pack(kScale, kScale);
    PagedWalk w;
    w.ti = valid ? paged_rel(p.q_ts[s.q0 + r0 + r], t_last) : PG_T0;
    // the CTA's tiles [f_lo, f_hi) that every row of this group's tile sees whole
    const int t_i0 = i0 + (dual ? 0 : t * 128), t_i1 = i0 + min(rows, (dual ? 0 : t * 128) + 128) - 1;
    const int f_lo = (p.window == 0 ? 0 : s.n_sink + max(0, (t_i1 - p.window + PGT_KEYS) / PGT_KEYS - s.first)) - k_begin;
    const int f_hi = s.n_sink + (t_i0 + 1) / PGT_KEYS - s.first - k_begin;
    auto walk_reset = [&]() {
      w.b = 0;
      w.bound = INT64_MIN;
      w.rt = 0.0f;
    };
    walk_reset();
    bool ok = true;
    float m = -INFINITY, l = 0.0f;  // softmax: this half's maximum and sum
    int buf = 0;
    uint32_t ph = 0;
    auto run_pass = [&](int pass) {
      for (int k = dual ? t : 0; k < n_k; k += dual ? 2 : 1) {
        const int it = pass * n_k + k, st = it % PGT_STAGES;
        ok = mbar_wait(&bars[PGB_S + PGT_SBUF * t + buf], ph, ctl);
        if (ok) ok = mbar_wait(&bars[PGB_FULL + st], static_cast<uint32_t>(it / PGT_STAGES) & 1u, ctl);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        tc_fence_after();
        const int j_tile = s.tile(k_begin + k) * PGT_KEYS, j0 = j_tile + half * 32;
        const int64_t* kts =
            reinterpret_cast<const int64_t*>(smem + PgtSmem::kSide + st * PgtSmem::kSideBytes) + half * 32;
        const float* bp = reinterpret_cast<const float*>(smem + PgtSmem::kSide + st * PgtSmem::kSideBytes + PGT_KEYS * 8) +
                          (i - j0) - paged_band0(i0 - j_tile, PGT_KEYS);
        const bool ragged = (k < f_lo || k >= f_hi) && (j0 + 32 > s.n || (j0 < s.lo && j0 + 32 > s.sink_end));
        if (it == 0 && t == 0 && (warp & 3) == 0 && s.seen(j0 + lane) && t_last - kts[lane] > PG_T0)
          record_status(HSTU_ERR_DEVICE_CHECK);
        // visible columns of the row, one bit each (inside [f_lo, f_hi) all of them)
        uint32_t vis = valid ? 0xffffffffu : 0u;
        if (k < f_lo || k >= f_hi) vis = 0u;
        if (vis == 0u && valid && i >= j0) {
          vis = i - j0 >= 31 ? 0xffffffffu : (2u << (i - j0)) - 1u;
          if (p.window > 0) {
            const int lo = i - p.window + 1 - j0, sk = p.sinks - j0;
            uint32_t in = lo <= 0 ? 0xffffffffu : (lo >= 32 ? 0u : 0xffffffffu << lo);
            in |= sk >= 32 ? 0xffffffffu : (sk <= 0 ? 0u : (1u << sk) - 1u);
            vis &= in;
          }
        }
        // (rows that do not exist are nobody's: their P may be anything)
        const bool whole = __all_sync(0xffffffffu, vis == 0xffffffffu || !valid);
        const bool row_live = vis != 0u;
        uint32_t sv[32];
        const uint32_t tS = tS0 + static_cast<uint32_t>(buf * 64);
        tmem_ld32(tS, sv);
        tmem_ld_wait(sv);
        uint32_t pk[16];
        if constexpr (!kSoftmax) {
          paged_chunk(sv, [&](int c, uint64_t h2) { pk[c >> 1] = phi_pair<PHI, F16>(h2); }, bp, kts, ragged,
                      row_live, w, t_last, sTime, sThr, sOct, sOrt, scale2);
        } else {
          float x[32];
          paged_chunk(sv, [&](int c, uint64_t h2) { f2_unpack(h2, x[c], x[c + 1]); }, bp, kts, ragged, row_live, w,
                      t_last, sTime, sThr, sOct, sOrt, scale2);
          if (!whole) {
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = (vis >> c) & 1u ? x[c] : -INFINITY;
          }
          if (pass == 0) {
            float cm = x[0];
#pragma unroll
            for (int c = 1; c < 32; ++c) cm = fmaxf(cm, x[c]);
            if (row_live && cm > m) {
              l *= ex2_approx(m - cm);
              m = cm;
            }
            float a0 = 0.0f, a1 = 0.0f;
            const float mm = m > -INFINITY ? m : 0.0f;
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              a0 += ex2_approx(x[c] - mm);
              a1 += ex2_approx(x[c + 1] - mm);
            }
            if (row_live) l += a0 + a1;
          } else {
#pragma unroll
            for (int c = 0; c < 32; c += 2) pk[c >> 1] = pack_16<F16>(ex2_approx(x[c] - m), ex2_approx(x[c + 1] - m));
          }
        }
        if (!kSoftmax || pass == 1) {
          if (!whole) {
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const uint32_t keep = ((vis >> c) & 1u ? 0xffffu : 0u) | ((vis >> (c + 1)) & 1u ? 0xffff0000u : 0u);
              pk[c >> 1] = row_live ? pk[c >> 1] & keep : 0u;
            }
          }
          __syncwarp();
          tmem_st16(tS, pk);
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(&bars[PGB_P + PGT_SBUF * t + buf]);
        if (++buf == PGT_SBUF) {
          buf = 0;
          ph ^= 1u;
        }
      }
    };
    run_pass(0);
    if constexpr (kSoftmax) {
      // P = 2^(x - m) with the row's maximum over both halves; the sum goes with O
      sMl[half * PGT_ROWS + slot] = make_float2(m, l);
      named_barrier_sync(1 + t, 256);
      const float2 other = sMl[(half ^ 1) * PGT_ROWS + slot];
      const float mm = fmaxf(m, other.x);
      if (mm > -INFINITY) l = l * ex2_approx(m - mm) + other.y * ex2_approx(other.x - mm);
      m = mm > -INFINITY ? mm : 0.0f;
      if (half == 0) sMlC[slot] = make_float2(mm, l);
      walk_reset();
      if (ok) run_pass(1);
    }
    // O to shared memory, once every MMA and load of the CTA is done with it
    // (with no key tile too: the issuers have then seen Q land)
    if (ok) ok = mbar_wait(&bars[PGB_DONE], 0, ctl) && mbar_wait(&bars[PGB_DONE + 1], 0, ctl);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    named_barrier_sync(3, 512);
    float* sO = reinterpret_cast<float*>(smem);
    uint32_t ov[32];
    if (ok && own_k(t) > 0) {
      tmem_ld32(tO, ov);
      tmem_ld_wait(ov);
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c) ov[c] = 0u;
    }
#pragma unroll
    for (int c = 0; c < 32; c += 4)
      *reinterpret_cast<uint4*>(sO + slot * PGT_OLD + half * 32 + c) =
          make_uint4(ov[c], ov[c + 1], ov[c + 2], ov[c + 3]);
    tc_fence_before();
  }
  __syncthreads();
  if (warp == PGT_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // ---------------- the sums over the cluster, 16 lanes a row
  float* sO = reinterpret_cast<float*>(smem);
  const float inv_n = kSoftmax ? 1.0f : 1.0f / static_cast<float>(n_all);
  cg::cluster_group cluster = cg::this_cluster();
  if (p.nsplit > 1) cluster.sync();
  if (warp < 16) {
    const int c4 = tid & 15, rr = dual ? 128 : PGT_ROWS;
    const int parts = dual ? 2 * p.nsplit : p.nsplit;  // partial results of a row
    for (int base = 0; base < rr; base += 32 * p.nsplit) {
      const int r_of = base + split + p.nsplit * (tid >> 4);
      const int r = min(r_of, rr - 1);
      auto part_o = [&](int k) {
        const int rank = dual ? k >> 1 : k, row = r + (dual ? (k & 1) * 128 : 0);
        return (p.nsplit > 1 ? cluster.map_shared_rank(sO, rank) : sO) + row * PGT_OLD + 4 * c4;
      };
      auto part_ml = [&](int k) {
        const int rank = dual ? k >> 1 : k, row = r + (dual ? (k & 1) * 128 : 0);
        return (p.nsplit > 1 ? cluster.map_shared_rank(sMlC, rank) : sMlC)[row];
      };
      float m = -INFINITY, l = 0.0f;
      if constexpr (kSoftmax)
        for (int k = 0; k < parts; ++k) m = fmaxf(m, part_ml(k).x);
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int k = 0; k < parts; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(part_o(k));
        float f = 1.0f;
        if constexpr (kSoftmax) {
          const float2 ml = part_ml(k);
          f = ml.x > -INFINITY ? ex2_approx(ml.x - m) : 0.0f;
          l = fmaf(ml.y, f, l);
        }
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z);
        o.w = fmaf(v.w, f, o.w);
      }
      const float k = kSoftmax ? (l > 0.0f ? 1.0f / l : 0.0f) : inv_n;
      paged_store<F16>(p, s.q0 + r0 + r, h, c4, make_float4(o.x * k, o.y * k, o.z * k, o.w * k), r_of < rows);
    }
  }
  if (p.nsplit > 1) cluster.sync();  // no CTA leaves while another reads its partial sums
}

}  // namespace hstu
