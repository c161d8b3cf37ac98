// What the two kernels of kda_cache_attend share: how the work is cut, and the
// producer that feeds a ring of stages with the tiles of a CTA's stretch.
#pragma once

#include <cstdint>

#include "kda_internal.h"
#include "kda_types.cuh"
#include "umma.cuh"

namespace kda {

// Of a tile: a unit's first or last one here, the CTA's last one, seen by all rows; and of its unit: whether
// its first and last tile are here (CLOSES: known at the last one; UNIT_CLOSES, UNIT_STOPS: at the first).
enum : uint32_t { FIRST = 1, LAST = 2, STOP = 4, FULL = 8, OPENS = 16, CLOSES = 32, UNIT_CLOSES = 64, UNIT_STOPS = 128 };

struct alignas(16) Meta {  // what the consumers need to know of a stage's tile
  int n, hk, row0, pos0, len, count, end;
  uint32_t flags;
  uint32_t valid[4];  // bit j: position pos0 + j lies in a page that exists
  int tiles;          // of the unit, from this one on, in this CTA
};

struct Record {  // a unit that several CTAs hold parts of
  int unit, first, more;  // parts: slot 2 first + 1, then slots 2 (first + team), ... `more` of them
  int pad;
};

struct Params {
  AttendProblem p;
  int groups;        // row groups per (sequence, key head)
  int rows;          // query rows of a key head: K H_q / H_kv
  int group_heads;   // H_q / H_kv
  int rows_per;      // rows of a unit: 16, 32 or 48
  int box_rows;      // rows of one TMA box
  bool use_tma;      // else the producer copies rows itself, 16 bytes at a time
  bool token_first;  // the tensor map's second dimension is the token, not the head
  bool whole;        // whole units per CTA: nothing is joined
  bool by_unit;      // records are indexed by unit, else by CTA
  int min_tiles;     // tiles that a CTA takes at least
  int team;          // CTAs that walk the same positions, each for a key head of its own
  Record* records;
  float2* part_ml;   // [2 CTAs][ROWS]
  float* part_o;     // [2 CTAs][ROWS][D]
};

template <typename A> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return __is_same(A, __nv_bfloat16) ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}
// four e4m3 values to fp16 (exact)
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}"
      : "=r"(lo), "=r"(hi) : "r"(v));
}
// 2^x for x <= 0 (and NaN): results below 2^-126 are 0
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// A sequence's visible range over all its real tokens, in whole tiles.
struct Range {
  int len, count, end, tile0, tiles;
};
template <int TILE> __device__ __forceinline__ Range range_from(const Params& s, int len, int count) {
  Range r;
  const AttendProblem& p = s.p;
  r.len = min(max(len, -(1 << 30)), 1 << 30);
  r.count = min(max(count, 0), p.K);
  const int cap = p.cache.table_width * p.cache.page_size;  // at most 2^30
  r.end = r.count ? max(0, min(r.len + r.count, cap)) : 0;
  const int start = p.window && r.len >= p.window ? r.len - p.window + 1 : 0;
  r.tile0 = start / TILE;
  // one tile also where nothing is seen: the zeros are written by it
  r.tiles = max(1, (r.end + TILE - 1) / TILE - r.tile0);
  return r;
}
template <int TILE> __device__ __forceinline__ Range range_of(const Params& s, int n) {
  return range_from<TILE>(s, s.p.cache.lens[n], s.p.counts ? s.p.counts[n] : s.p.K);
}

// The maximum of a row all of whose scores are -infinity: not -infinity, which is that of a row that sees
// nothing.  Its weights are 0, and 0 / 0 is the result.
constexpr float LOWEST = -3.402823466e38f;

// Whether token i of sequence n sees a position from `begin` to before `end` that lies in a page that
// exists.  Asked only of rows without a weight: the tiles' loops need not keep track of it.
__device__ __forceinline__ bool sees_any(const Params& s, int n, int i, int begin, int end) {
  const AttendProblem& p = s.p;
  const Range r = range_of<64>(s, n);
  if (i >= r.count) return false;
  const int first = p.window && r.len + i >= p.window ? r.len + i - p.window + 1 : 0;
  const int a = max(first, begin), b = min(min(r.len + i, r.end - 1), end - 1);
  if (a > b) return false;
  for (int x = a / p.cache.page_size; x <= b / p.cache.page_size; ++x) {
    const int page = p.cache.block_table[n * p.cache.table_stride + x];
    if (page >= 0 && page < p.cache.num_pages) return true;
  }
  return false;
}

// Byte of 16-byte chunk `c` of row `row` in a [TILE][ROW_BYTES] region, as TMA's swizzle lays it
template <int ROW_BYTES, int TILE> __device__ __forceinline__ uint32_t kv_offset(int row, int c) {
  if (ROW_BYTES >= 128)
    return (uint32_t)((c >> 3) * (TILE * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
  return (uint32_t)(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
}

// A CTA's stretch of tiles, or of whole units.
struct Stretch {
  int n0, sub0;       // first unit: sequence, and unit in it
  int tile_in, left;  // tile in that unit; tiles (or, for whole units, units) to do
  int a0, live;       // first tile; teams that have any
  int each, extra;    // tiles of a team; the first `extra` have one more
  Range range;        // of the first sequence
};

// Called by all threads of a CTA; starts with every sequence's lens and counts.
template <int TILE, int THREADS> __device__ __forceinline__ Stretch find_stretch(const Params& s) {
  __shared__ int s_sum[THREADS / 32];
  __shared__ int s_before;
  __shared__ int s_n;
  __shared__ Range s_range;
  const AttendProblem& p = s.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int all_heads = p.cache.H_kv * s.groups;  // units of one sequence
  const int heads = all_heads / s.team;           // of them, a team member's
  const int c = blockIdx.x, N = p.cache.n_seq;
  const int G = gridDim.x / s.team, team = c / s.team;
  int n0, sub0;         // first unit: sequence, and unit in it
  int tile_in, left;    // tile in that unit; tiles (or, for whole units, units) to do
  int a0 = 0, live = G; // first tile; CTAs that have any
  int each = 0, extra = 0;  // tiles of a CTA; the first `extra` have one more
  if (s.whole) {
    const int units = N * heads;
    each = units / G, extra = units - each * G;
    const int u0 = team * each + min(team, extra);
    n0 = u0 / heads;
    sub0 = u0 - n0 * heads;
    tile_in = 0;
    left = each + (team < extra ? 1 : 0);
    if (tid == 0) s_range = range_of<TILE>(s, n0);
    __syncthreads();
  } else {
    // tiles of all sequences before each thread's share of them
    const int per = (N + THREADS - 1) / THREADS;
    const int b0 = min(N, tid * per), b1 = min(N, b0 + per);
    int mine = 0;
    Range r{};
    for (int n = b0; n < b1; ++n) {
      r = range_of<TILE>(s, n);
      mine += r.tiles;
    }
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += y;
    }
    if (lane == 31) s_sum[warp] = scan;
    __syncthreads();
    int before = scan - mine, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += s_sum[w];
      total += s_sum[w];
    }
    total *= heads;
    before *= heads;
    live = min(G, max(1, total / s.min_tiles));
    each = total / live, extra = total - each * live;
    a0 = team < live ? team * each + min(team, extra) : 0;
    left = team < live ? each + (team < extra ? 1 : 0) : 0;
    if (a0 >= before && a0 < before + mine * heads) {
      int n = b0;
      if (per > 1) {
        for (;; ++n) {
          r = range_of<TILE>(s, n);
          const int t = r.tiles * heads;
          if (a0 < before + t) break;
          before += t;
        }
      }
      s_n = n;
      s_before = before;
      s_range = r;
    }
    __syncthreads();
    n0 = s_n;
    const int in = a0 - s_before;
    sub0 = in / s_range.tiles;
    tile_in = in - sub0 * s_range.tiles;
    if (!s.by_unit && tid == 0 && left == 0) s.records[c].more = 0;
  }
  return Stretch{n0, sub0, tile_in, left, a0, live, each, extra, s_range};
}

// The ring: a stage's keys and values lie stage_bytes apart from `base` on.
struct Ring {
  uint32_t base;
  uint64_t *full, *empty, *told;  // barriers of each stage; told: its Meta is written
  Meta* meta;
};

// A producer warp's work: page look-ups, each stage's Meta, and the copies.  Of PRODUCERS warps, this
// one (`which`) takes every PRODUCERS-th tile.  Where a wait runs out it copies nothing more, but still
// writes the records of all its units, which the joining kernel forms addresses from; it returns when
// its copies have landed.
template <int D, bool E8, int TILE, int STAGES, int PRODUCERS = 1>
__device__ __forceinline__ void produce(const Params& s, const Stretch& st, const Ring& ring, const CUtensorMap& map_k,
                                        const CUtensorMap& map_v, int which = 0, uint64_t limit_ns = WAIT_NS) {
  constexpr int ROW_BYTES = D * (E8 ? 1 : 2), BOX_BYTES = ROW_BYTES < 128 ? ROW_BYTES : 128;
  constexpr int HALVES = ROW_BYTES / BOX_BYTES, KV_BYTES = TILE * ROW_BYTES, STAGE_BYTES = 2 * KV_BYTES;
  const AttendProblem& p = s.p;
  const int lane = threadIdx.x & 31;
  const int all_heads = p.cache.H_kv * s.groups, heads = all_heads / s.team;
  const int c = blockIdx.x, N = p.cache.n_seq, team = c / s.team, member = c - team * s.team;
  const int a0 = st.a0, each = st.each, extra = st.extra;
  int left = st.left;
  uint64_t *full = ring.full, *empty = ring.empty, *told = ring.told;
  Meta* meta = ring.meta;
  const uint32_t base = ring.base;
  const bool use_tma = s.use_tma;
  // Page numbers are looked up for as many tiles at once as 32 lanes hold, one such batch ahead
  // of the copies, and lens and counts one sequence ahead: neither latency is waited for.
  const int rows_per = s.box_rows;
  constexpr int PL = TILE / 32;  // pages of a lane, where each row of a tile is looked up
  const int boxes = TILE / rows_per, batch = boxes < 32 ? 32 / boxes : 1;
  struct Batch {
    int n, sub, j;     // tiles j .. of a unit
    Range r;
    int page[PL];       // as loaded: nothing waits for it here
    int at[PL];         // the box's first row in its page
    uint32_t need[PL];  // lanes whose page is needed
  };
  auto look_up = [&](Batch& b) {
    const int first_seen = p.window && b.r.len >= p.window ? b.r.len - p.window + 1 : 0;
#pragma unroll
    for (int x = 0; x < PL; ++x) {
      const int pos = (b.r.tile0 + b.j) * TILE + (lane + 32 * x) * rows_per;
      const bool need = (x == 0 || 32 * x < boxes) && b.j + (lane + 32 * x) / boxes < b.r.tiles &&
                        pos < b.r.end && pos + rows_per > first_seen;
      b.need[x] = __ballot_sync(0xffffffffu, need);
      if (need) {
        const int entry = pos / p.cache.page_size;
        b.page[x] = p.cache.block_table[b.n * p.cache.table_stride + entry];
        b.at[x] = pos - entry * p.cache.page_size;
      }
    }
  };
  Batch cur{st.n0, st.sub0, st.tile_in, st.range, {}, {}, {}};
  look_up(cur);
  int ahead_len = 0, ahead_count = p.K;
  auto read_ahead = [&](int n) {
    if (n >= N) return;
    ahead_len = p.cache.lens[n];
    if (p.counts) ahead_count = p.counts[n];
  };
  read_ahead(st.n0 + 1);
  bool opened_here = false, recorded = false, stop = false;
  int it = 0, sent = -1;  // sent: tiles copied when a wait ran out
  while (!stop) {
    Batch next = cur;
    next.j += batch;
    if (next.j >= cur.r.tiles) {
      next.j = 0;
      if (++next.sub == heads) {
        next.sub = 0;
        if (++next.n < N) {
          next.r = range_from<TILE>(s, ahead_len, ahead_count);
          read_ahead(next.n + 1);
        }
      }
    }
    if (next.n < N) look_up(next);
    const int n = cur.n, sub = cur.sub * s.team + member, tiles_here = min(batch, cur.r.tiles - cur.j);
    const Range& r = cur.r;
    // of the unit: its key head, first row, and first and last token
    const int hk = sub / s.groups, row0 = (sub - hk * s.groups) * s.rows_per;
    const int i0 = row0 / s.group_heads, i1 = min(s.rows - 1, row0 + s.rows_per - 1) / s.group_heads;
    const bool over = r.count && r.len + r.count > r.end && r.len + r.count > 0;
    for (int x = 0; x < tiles_here && !stop; ++x, ++it) {
    const int j = cur.j + x;
    const int stage = it % STAGES;
    const int pos0 = (r.tile0 + j) * TILE;
    const bool first = it == 0 || j == 0;
    if (first) opened_here = j == 0;
    const bool closes = j == r.tiles - 1;
    const int unit_tiles = s.whole ? r.tiles - j : min(r.tiles - j, left);
    const bool unit_stops = s.whole ? left == 1 : left == unit_tiles;
    if (!s.whole) --left; else if (closes) --left;
    stop = left == 0;
    if (!s.whole && first && opened_here && lane == 0 && which == 0) {
      // parts of this unit that other CTAs will hold
      const int last = a0 + it + r.tiles - 1, longer = extra * (each + 1);  // its last tile
      const int last_team = last < longer ? last / (each + 1) : extra + (last - longer) / each;
      if (s.by_unit) {
        Record& rec = s.records[n * all_heads + sub];
        rec.unit = n * all_heads + sub;
        rec.first = c;
        rec.more = last_team - team;
      } else if (last_team > team) {
        s.records[c].unit = n * all_heads + sub;
        s.records[c].first = c;
        s.records[c].more = last_team - team;
        recorded = true;
      }
    }
    if (sent >= 0 || (PRODUCERS > 1 && it % PRODUCERS != which)) continue;
    // lane b: the page of rows [b rows_per, (b + 1) rows_per) of the tile; of single rows b, b + 32, ...
    const int from = (x * boxes + lane) & 31;
    int page[PL], at[PL];
    uint32_t good[PL];
    uint32_t wrong = 0;
#pragma unroll
    for (int y = 0; y < PL; ++y) {
      page[y] = -1;
      good[y] = 0;
      if (32 * y >= boxes) continue;  // the same for all lanes
      page[y] = y == 0 ? __shfl_sync(0xffffffffu, cur.page[0], from) : cur.page[y];
      at[y] = y == 0 ? __shfl_sync(0xffffffffu, cur.at[0], from) : cur.at[y];
      const bool need = y == 0 ? lane < boxes && ((cur.need[0] >> from) & 1) : (cur.need[y] >> lane) & 1;
      const bool ok = need && page[y] >= 0 && page[y] < p.cache.num_pages;
      if (!ok) page[y] = -1;
      good[y] = __ballot_sync(0xffffffffu, ok);
      wrong |= __ballot_sync(0xffffffffu, need) & ~good[y];
    }
    const bool bad = wrong != 0;
    if (lane == 0 && (bad || (over && first))) *p.status = 1;
    if (it >= STAGES && !mbar_wait(&empty[stage], ((it / STAGES) - 1) & 1, limit_ns)) {
      *p.status = 6;
      sent = it;
      continue;
    }
    const uint32_t k_s = base + stage * STAGE_BYTES, v_s = k_s + KV_BYTES;
    if (lane == 0) {
      Meta& m = meta[stage];
      m.n = n;
      m.hk = hk;
      m.row0 = row0;
      m.pos0 = pos0;
      m.len = r.len;
      m.count = r.count;
      m.end = r.end;
      for (int y = 0; y < 4; ++y) m.valid[y] = ~0u;
      if (bad) {
        for (int y = 0; y < 4; ++y) m.valid[y] = 0;
        for (int y = 0; y < TILE; ++y) {
          const int b = y / rows_per;
          if ((good[b >> 5] >> (b & 31)) & 1) m.valid[y >> 5] |= 1u << (y & 31);
        }
      }
      const bool all = !bad && pos0 + TILE <= r.end && i1 < r.count && pos0 + TILE - 1 <= r.len + i0 &&
                       !(p.window && r.len + i1 >= p.window && pos0 < r.len + i1 - p.window + 1);
      m.flags = (first ? FIRST : 0) | (closes || stop ? LAST : 0) | (stop ? STOP : 0) | (all ? FULL : 0) |
                (opened_here ? OPENS : 0) | (closes ? CLOSES : 0) |
                (j + unit_tiles == r.tiles ? UNIT_CLOSES : 0) | (unit_stops ? UNIT_STOPS : 0);
      m.tiles = unit_tiles;
      mbar_arrive(&told[stage]);
    }
    if (use_tma) {
      if (lane == 0) {
        uint32_t boxes_here = 0;
#pragma unroll
        for (int y = 0; y < PL; ++y) boxes_here += __popc(good[y]);
        const uint32_t bytes = boxes_here * rows_per * ROW_BYTES * 2;
        if (bytes) mbar_arrive_expect_tx(&full[stage], bytes); else mbar_arrive(&full[stage]);
      }
      __syncwarp();
#pragma unroll
      for (int y = 0; y < PL; ++y) {
        if (page[y] < 0) continue;
        const int row = (lane + 32 * y) * rows_per;
        const int c1 = s.token_first ? at[y] : hk, c2 = s.token_first ? hk : at[y];
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          const uint32_t off = h * TILE * BOX_BYTES + row * BOX_BYTES;
          const int c0 = h * (BOX_BYTES / (E8 ? 1 : 2));
          tma_load_4d(k_s + off, &map_k, &full[stage], c0, c1, c2, page[y]);
          tma_load_4d(v_s + off, &map_v, &full[stage], c0, c1, c2, page[y]);
        }
      }
    } else {
      // 8-bit heads of 64 in pages of odd size: a box would be one row of 64 bytes, half of TMA's
      // 128-byte step in shared memory
      constexpr int CH = ROW_BYTES / 16;
      for (int x = lane; x < TILE * CH; x += 32) {
        const int row = x / CH, ch = x % CH;
        int page_of = -1;
#pragma unroll
        for (int y = 0; y < PL; ++y) {
          const int of = __shfl_sync(0xffffffffu, page[y], row & 31);
          if (y == row >> 5) page_of = of;
        }
        if (page_of < 0) continue;
        const long long at = (page_of * p.cache.page_stride +
                              (long long)((pos0 + row) % p.cache.page_size) * p.cache.token_stride +
                              hk * p.cache.head_stride) * (E8 ? 1 : 2) + ch * 16;
        const uint32_t off = kv_offset<ROW_BYTES, TILE>(row, ch);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(k_s + off),
                     "l"(static_cast<const uint8_t*>(p.cache.k) + at) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(v_s + off),
                     "l"(static_cast<const uint8_t*>(p.cache.v) + at) : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(&full[stage])) : "memory");
      if (lane == 0) mbar_arrive(&full[stage]);
    }
    }
    cur = next;
  }
  if (!s.whole && !s.by_unit && !recorded && lane == 0 && which == 0) s.records[c].more = 0;
  if (sent < 0) sent = it;
  for (int t = max(0, sent - STAGES); t < sent; ++t)
    if (t % PRODUCERS == which && !mbar_wait(&full[t % STAGES], (t / STAGES) & 1, limit_ns)) *p.status = 6;
}

// More than 16 query rows to a key head (kda_attend_wide.cu).
cudaError_t launch_attend_wide(const Params& s, const CUtensorMap& map_k, const CUtensorMap& map_v, int grid,
                               cudaStream_t stream);

}  // namespace kda
