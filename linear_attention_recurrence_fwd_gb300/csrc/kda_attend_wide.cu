// kda_cache_attend where 17 to 48 query rows share a key head (several tokens,
// many heads to a key head): both products on the tcgen05 tensor cores, with
// positions and output channels on their lanes.
//
//     S^T [128 positions x N rows] = K Q^T      (A: keys as TMA lays them, B: Q)
//     O^T [d channels x N rows]   += V^T P^T    (A: values, read transposed, B: P)
//
// N is 32 or 48: with the rows on the 128 lanes most would be padding.  A
// thread of the softmax warps has one position: it turns that position's
// scores into weights with no exchange between lanes, since the rows' maxima
// are kept from earlier tiles as long as no score passes one by 2^8 (2^3 for
// an 8-bit cache), and the sums of the weights are kept by thread until the
// unit ends.  When a score does pass (and at a unit's start), the maxima are
// found across the lanes and O and the sums are rescaled.  What runs once a
// unit is written as loops, not unrolled: its time is that of fetching
// instructions.
//
// An 8-bit cache's keys and values are operands as they are (kind::f8f6f4): no
// byte is converted.  The other operand comes in 8-bit pieces instead.  A query
// q is q_1 + q_2 / 16 (+ q_3 / 256), e4m3 numbers of 4 bits each, their scores
// side by side in N; a weight is the sum of 3 (fp16 queries: 4) e5m2 numbers of
// 3 bits each, whose products lie side by side in O and are added at the
// unit's end.  The accumulators are fp32.  The weights are 2^(s - m + 12), so
// that their pieces are normal numbers down to 2^-26 of the largest.  (e4m3
// pieces of the weights would leave absolute errors of 2^-18 of the largest,
// which a million small weights add up.)
//
// Against warp-level instructions, which run at an eighth of tcgen05's rate (64
// requests of 8192 positions, 4 key heads of 128, 40 rows): 347 us there and
// 177 us here, 6.1 TB/s.  8-bit: 277 us there (each group of 16 rows converts
// all keys and values), 258 us here with keys and values converted through
// shared and tensor memory, 133 us in pieces (4.0 TB/s; a tile takes 1620
// clocks, of which its bytes need 1400, and a unit's end and start 14000).
//
// Warps: 0-7 softmax, 8 and 11 load, 9 and 10 issue the scores and the values.
// The softmax warps are one group of which each half has half of the rows; or,
// over an 8-bit cache, two groups that take tiles in turn, each with maxima,
// sums, weights and an O of its own (as one group 146 us: the latencies of one
// tile's steps add up to 2100 clocks).  One loading warp spends 2000 clocks on
// a tile, more than its bytes take.  One CTA on an SM.
#include <atomic>

#include "kda_attend.cuh"

namespace kda {
namespace {

constexpr int TILE = 128;
constexpr float UNSEEN = 3e38f;  // takes any score of a row without a maximum past the limit

// E8: an 8-bit cache.  QP and WP: the 8-bit pieces that a query and a weight are written as.
template <typename A, int D, bool E8> struct Wide {
  // Softmax warps: two groups that take tiles in turn, or one of which each half has half of the rows
  static constexpr int GROUPS = E8 ? 2 : 1;
  // The launch's registers are split anew where a thread has all rows; the sum stays what it was.
  static constexpr int THREADS = 384;
  static constexpr int LAUNCH_REGS = 168, SOFTMAX_REGS = 192, OTHER_REGS = 120;
  static_assert(!E8 || 8 * SOFTMAX_REGS + 4 * OTHER_REGS <= 12 * LAUNCH_REGS, "registers");
  static constexpr int ES = E8 ? 1 : 2;                  // bytes of a cached element
  static constexpr int QP = E8 ? (__is_same(A, __nv_bfloat16) ? 2 : 3) : 1, WP = E8 ? QP + 1 : 1;
  // Of a weight's pieces, WN lie side by side in one product (each with columns of its own in O; the
  // values, whose reading bounds a product this narrow, are read once), in WP / WN products.
  static constexpr int WN = WP == 4 ? 2 : WP;
  static constexpr int ROW_BYTES = D * ES;
  static constexpr int KV_BYTES = TILE * ROW_BYTES;      // keys or values of a stage
  static constexpr int STAGE_BYTES = 2 * KV_BYTES;
  static constexpr int Q_BYTES = 48 * D * QP * ES, P_BYTES = 48 * TILE * WP * ES;  // P: of a group
  static constexpr int MISC_BYTES = 7680;
  static constexpr int FIT = (227 * 1024 - 1280 - Q_BYTES - GROUPS * P_BYTES - MISC_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr int SMEM = STAGES * STAGE_BYTES + Q_BYTES + GROUPS * P_BYTES + MISC_BYTES + 1024;
  // Columns of tensor memory: two tiles' scores, then each group's output
  static constexpr uint32_t T_S = 0, S_COLS = E8 ? QP * 48 : 64, T_O = 2 * S_COLS, O_COLS = 48 * WN, T_COLS = E8 ? 512 : 256;
  static_assert(T_O + GROUPS * O_COLS <= T_COLS, "tensor memory");
  // Weights are 2^(f s - m + BIAS) and reach 2^(BIAS + SLACK) before the maximum is moved.  (In fp16 the
  // bias keeps small ones to 2^-32 of the largest; its least step is 2^-24.)
  static constexpr float BIAS = E8 ? 12.f : __is_same(A, __nv_bfloat16) ? 0.f : 7.f, SLACK = E8 ? 3.f : 8.f;
};

// kind::f8f6f4 with 8-bit operands, each e4m3 or e5m2, and an fp32 accumulator; K = 32 per MMA.
enum F8 : uint32_t { F8_E4M3 = 0, F8_E5M2 = 1 };
__host__ __device__ constexpr uint32_t make_idesc_f8(int M, int N, bool a_mn_major, bool b_mn_major, F8 a, F8 b) {
  return (1u << 4) | ((uint32_t)a << 7) | ((uint32_t)b << 10) | ((a_mn_major ? 1u : 0u) << 15) |
         ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void st_u16(uint32_t at, uint32_t v) {
  asm volatile("{.reg .b16 l, h; mov.b32 {l, h}, %1; st.shared.b16 [%0], l;}" ::"r"(at), "r"(v) : "memory");
}

// 8 consecutive columns: thread i of the warp gets lane (base lane + i).
__device__ __forceinline__ void tmem_ld8(uint32_t at, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(at));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(__float_as_uint(v[0])),
               "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])),
               "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])) : "memory");
}

// op over the warp's lanes of each of 8 values, by halves: 9 exchanges.  Lane l gets value l >> 2;
// the values are lost.
template <typename Op> __device__ __forceinline__ float across(float (&v)[8], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = 4; half > 0; half >>= 1) {
    const bool upper = lane & (4 * half);
#pragma unroll
    for (int x = 0; x < half; ++x) {
      const float give = upper ? v[x] : v[x + half], take = upper ? v[x + half] : v[x];
      v[x] = op(take, __shfl_xor_sync(0xffffffffu, give, 4 * half));
    }
  }
  const float y = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 2));
  return op(y, __shfl_xor_sync(0xffffffffu, y, 1));
}

// NC: rows of a unit, in sixteens
template <typename A, int D, int NC, bool E8>
__global__ void __launch_bounds__(Wide<A, D, E8>::THREADS, 1)
    attend_wide_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const __grid_constant__ Params s) {
  using W = Wide<A, D, E8>;
  constexpr int STAGES = W::STAGES, QP = W::QP, WP = W::WP, WN = W::WN, GROUPS = W::GROUPS;
  constexpr uint32_t T_S = W::T_S, T_O = W::T_O;
  constexpr bool BF = __is_same(A, __nv_bfloat16);
  extern __shared__ uint8_t smem_raw[];
  const AttendProblem& p = s.p;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const aligned = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t q_s = base + STAGES * W::STAGE_BYTES, p_s = q_s + W::Q_BYTES;
  uint8_t* misc = aligned + STAGES * W::STAGE_BYTES + W::Q_BYTES + GROUPS * W::P_BYTES;
  // tables of the unit's rows, for two units in turn
  float* row_m = reinterpret_cast<float*>(misc);    // [group][2][48] maximum (of scores in log2 units)
  float* row_neg = row_m + 192;                     // [group][2][48] BIAS minus the maximum; UNSEEN while nothing is seen
  float* row_f = row_neg + 192;                     // [2][48] what its scores are multiplied with (8-bit)
  int* row_tok = reinterpret_cast<int*>(row_f + 96);  // [2][48] the row's token
  float* warp_top = reinterpret_cast<float*>(row_tok + 96);  // [group][4][48] maxima over a warp's positions; a unit's sums
  float* keep = warp_top + 384;                     // [group][48] what O and the sums are rescaled with; what O is multiplied with
  int* rows_lo = reinterpret_cast<int*>(keep + 96);  // [4][48] first and last position that a row sees,
  int* rows_hi = rows_lo + 192;                      // [4][48] for four tiles in turn
  long long* row_to = reinterpret_cast<long long*>(rows_hi + 192);  // [48] where a row's output goes
  int* mark = reinterpret_cast<int*>(row_to + 48);  // [4]: the tile whose values are multiplied by hand, four in turn
  int* give_up = mark + 4;                          // [group] a softmax warp met a limit
  uint64_t* bars = reinterpret_cast<uint64_t*>(give_up + 4);
  uint64_t *full = bars, *empty = bars + 6, *told = bars + 12;
  uint64_t *s_full = bars + 18, *s_empty = bars + 20, *p_full = bars + 22, *p_empty = bars + 24, *q_full = bars + 26, *joint = bars + 27;
  Meta* meta = reinterpret_cast<Meta*>(bars + 28);  // [6]
  __shared__ uint32_t s_tmem;
  __shared__ int unit_pos0[2];  // the first position of the unit's tiles here, for two units in turn

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int N = 16 * NC;  // query rows of a unit
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid < STAGES) {
    mbar_init(&full[tid], s.use_tma ? 1 : 33);
    mbar_init(&empty[tid], 2);  // the two products
    mbar_init(&told[tid], 1);
  }
  if (tid == 32) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&s_empty[x], 8 / GROUPS);
      mbar_init(&p_full[x], 8 / GROUPS);
      mbar_init(&p_empty[x], 1);
      give_up[x] = 0;
    }
    mbar_init(q_full, 8);
    mbar_init(joint, 8);
    for (int x = 0; x < 4; ++x) mark[x] = -1;
  }
  mbar_fence_init();
  if (tid == 256 && s.use_tma && p.cache.num_pages > 0) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  const Stretch st = find_stretch<TILE, W::THREADS>(s);
  if (st.left == 0) return;
  if (warp == 9) {
    tmem_alloc(&s_tmem, W::T_COLS);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;
  const int c = blockIdx.x;

  // a tile's values: [d / 64][position][128 bytes], chunks of 16 bytes XORed with the position
  auto values_of = [&](int stage) { return base + stage * W::STAGE_BYTES + W::KV_BYTES; };
  auto last_seen = [&](const Meta& t, int i) { return i < t.count ? min(t.len + i, t.end - 1) : -1; };
  auto first_seen = [&](const Meta& t, int i) { return p.window && t.len + i >= p.window ? t.len + i - p.window + 1 : 0; };
  // whether any row of the unit sees position `at`
  auto any_sees = [&](const Meta& t, int at) {
    const int i0 = t.row0 / s.group_heads, i1 = min((min(t.row0 + N, s.rows) - 1) / s.group_heads, t.count - 1);
    const int x = at - t.pos0;
    return i1 >= i0 && at <= last_seen(t, i1) && at >= first_seen(t, i0) && ((t.valid[x >> 5] >> (x & 31)) & 1);
  };

  // ---------------------------------------------------------------- softmax
  auto softmax = [&]() -> bool {
    // Group grp takes the tiles it with it % GROUPS == grp.  A thread has position `pos` of them, and the
    // 8 CH rows from r0 on.
    constexpr int HALVES = 2 / GROUPS, CH = 2 * NC / HALVES, GROUP = 256 / GROUPS;
    const int pos = tid & 127, quarter = warp & 3, upper = warp >> 2;
    const int grp = GROUPS == 2 ? upper : 0, half = GROUPS == 2 ? 0 : upper, r0 = half * (8 * CH), gt = tid - grp * GROUP;
    const uint32_t my_lane = tmem_addr(tmem, quarter * 32, 0);
    const uint32_t my_p = p_s + grp * W::P_BYTES, my_o = my_lane + T_O + grp * W::O_COLS;
    // A group's barrier, with a vote.  A warp that meets a limit marks it and comes to one more barrier
    // of its group, after which the others see the mark and leave as well: no barrier waits for a warp
    // that has left.
    auto vote = [&](bool mine, bool& any) {
      uint32_t r;
      asm volatile("{.reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, %2, %3, p; selp.u32 %0, 1, 0, q;}"
                   : "=r"(r) : "r"((uint32_t)mine), "r"(1 + grp), "n"(GROUP) : "memory");
      any = r != 0;
      return *reinterpret_cast<volatile int*>(&give_up[grp]) == 0;
    };
    auto sync = [&]() {
      bool any;
      return vote(false, any);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (__all_sync(0xffffffffu, mbar_wait(bar, parity))) return true;
      give_up[grp] = 1;
      sync();
      return false;
    };
    // all softmax warps
    uint32_t joints = 0;
    auto sync_all = [&]() {
      if (GROUPS == 1) return sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(joint);
      return wait(joint, joints++ & 1);
    };
    // this position's place in the weights: rows of 128 bytes, 64 positions each
    uint32_t at_p[8];
#pragma unroll
    for (int x = 0; x < 8; ++x)
      at_p[x] = my_p + (pos >> 6) * (N * 128) + r0 * 128 + ((((pos & 63) >> 3) ^ x) << 4) + (pos & 7) * 2;

    // Eight channels of a query in 8-bit pieces: the row is scaled by a power of two that brings its
    // largest entry to [2^7, 2^8), a piece has 4 bits of an entry, and the next one 2^4 times what is
    // left.  The 8 bits of a bf16 entry (11 of an fp16 one) fit exactly, down to 2^-14 of the largest
    // (2^-18); what is below is off by 2^-21 of it (2^-25) at most.  Infinities become NaN.
    auto write_pieces = [&](const uint4& v, int row, int ch, int odd) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      float x[8], big = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (BF) {
          x[2 * e] = __uint_as_float(w[e] << 16);
          x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        } else {
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
          x[2 * e] = y.x;
          x[2 * e + 1] = y.y;
        }
        big = fmaxf(big, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
      }
#pragma unroll
      for (int o = 1; o < D / 8; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      const int power = min(max(134 - (int)(__float_as_uint(big) >> 23), -120), 120);
      const float by = __uint_as_float((uint32_t)(127 + power) << 23);
      if (ch == 0) row_f[odd * 48 + row] = p.scale * p.cache.k_scale * 1.44269504088896340736f * __uint_as_float((uint32_t)(127 - power) << 23);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fabsf(x[e]) < INFINITY ? x[e] * by : __uint_as_float(0x7fffffffu);
#pragma unroll
      for (int pc = 0; pc < QP; ++pc) {
        uint32_t out[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          asm("{.reg .b16 l, h; cvt.rn.satfinite.e4m3x2.f32 l, %2, %1; cvt.rn.satfinite.e4m3x2.f32 h, %4, %3; mov.b32 %0, {l, h};}"
              : "=r"(out[e]) : "f"(x[4 * e]), "f"(x[4 * e + 1]), "f"(x[4 * e + 2]), "f"(x[4 * e + 3]));
          uint32_t lo, hi;
          e4m3x4_to_f16(out[e], lo, hi);
          const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
          x[4 * e] = (x[4 * e] - a.x) * 16.f;
          x[4 * e + 1] = (x[4 * e + 1] - a.y) * 16.f;
          x[4 * e + 2] = (x[4 * e + 2] - b.x) * 16.f;
          x[4 * e + 3] = (x[4 * e + 3] - b.y) * 16.f;
        }
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(q_s + pc * (N * D) + kv_offset<D, TILE>(row, ch >> 1) + (ch & 1) * 8),
                     "r"(out[0]), "r"(out[1]) : "memory");
      }
    };

    // A unit, from its first tile's stage, and its queries on their way: a thread's chunks of 8 channels.
    int u_n, u_hk, u_row0, u_tiles, u_pos0;
    uint32_t u_flags;
    constexpr int ALL = N * (D / 8), EACH = (ALL + 255) / 256;
    uint4 q[EACH];
    auto fetch_queries = [&](int stage, int turn) {
      if (!wait(&told[stage], turn)) return false;
      const Meta& t = meta[stage];
      u_n = t.n, u_hk = t.hk, u_row0 = t.row0, u_tiles = t.tiles, u_flags = t.flags, u_pos0 = t.pos0;
#pragma unroll
      for (int z = 0; z < EACH; ++z) {
        q[z] = make_uint4(0, 0, 0, 0);
        const int gr = u_row0 + (tid + z * 256) / (D / 8), i = gr / s.group_heads;
        if (gr < s.rows && tid + z * 256 < ALL)
          q[z] = *reinterpret_cast<const uint4*>(static_cast<const A*>(p.q) + ((long long)u_n * p.K + i) * p.q_stride +
                                                 (u_hk * s.group_heads + gr - i * s.group_heads) * D + tid % (D / 8) * 8);
      }
      return true;
    };
    // Its rows' tables, then its queries to shared memory: as they are, or in pieces.
    auto place_queries = [&](int odd) {
      if (tid < N) {
        const int gr = u_row0 + tid;
        for (int x = 0; x < GROUPS; ++x) {
          row_m[x * 96 + odd * 48 + tid] = -INFINITY;
          row_neg[x * 96 + odd * 48 + tid] = UNSEEN;
        }
        row_tok[odd * 48 + tid] = gr < s.rows ? gr / s.group_heads : 0x3fffffff;
        if (tid == 0) unit_pos0[odd] = u_pos0;
      }
      const int ch = tid % (D / 8);
      if constexpr (E8) {
#pragma unroll 1
        for (int z = 0; z < EACH; ++z) {
          if (ALL % 256 && tid + z * 256 >= ALL) break;  // (whole warps)
          write_pieces(q[0], (tid + z * 256) / (D / 8), ch, odd);
#pragma unroll
          for (int y = 0; y + 1 < EACH; ++y) q[y] = q[y + 1];
        }
      } else {
#pragma unroll
        for (int z = 0; z < EACH; ++z) {
          if (ALL % 256 && tid + z * 256 >= ALL) break;
          const int row = (tid + z * 256) / (D / 8);
          st_shared_v4(q_s + (ch >> 3) * (N * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), q[z].x, q[z].y, q[z].z, q[z].w);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    };

    float sums[CH][8];  // of this position's weights of each row, over the unit's tiles
    int odd = 0;
    int it = 0, stage = 0, turn = 0;
    auto advance = [&]() {
      ++it;
      if (++stage == STAGES) stage = 0, turn ^= 1;
    };
    if (!fetch_queries(0, 0)) return false;
    place_queries(0);
    if (!sync_all()) return false;
    while (true) {
    const int n = u_n, hk = u_hk, row0 = u_row0, tiles = u_tiles;
    const uint32_t unit = u_flags;
    const float *neg = row_neg + grp * 96 + odd * 48 + r0, *fs = row_f + odd * 48 + r0;  // of this thread's rows
    const int* tok = row_tok + odd * 48;
#pragma unroll
    for (int y = 0; y < CH; ++y)
#pragma unroll
      for (int x = 0; x < 8; ++x) sums[y][x] = 0.f;
    // ---- the unit's tiles, or every second of them
    for (int z = 0; z < tiles; ++z, advance()) {
      if (GROUPS == 2 && (it & 1) != grp) continue;
      if (!wait(&s_full[it & 1], (it >> 1) & 1)) return false;
      if (!wait(&told[stage], turn)) return false;
      tc_fence_after_sync();
      const Meta& t = meta[stage];  // the stage is given back after this tile's last look at it
      const bool first = z < GROUPS, all = t.flags & FULL;
      const int done_before = it / GROUPS;  // the group's tiles before this one
      uint64_t* const o_done = &p_empty[GROUPS == 2 ? grp : 0];
      const float f = p.scale * p.cache.k_scale * 1.44269504088896340736f;
      const uint32_t scores = my_lane + T_S + (it & 1) * W::S_COLS + r0;
      int at = 0;
      bool exists = true;
      if (!all) {
        at = t.pos0 + pos;
        exists = (t.valid[quarter] >> lane) & 1;
      }
      int *row_lo = rows_lo + (it & 3) * 48, *row_hi = rows_hi + (it & 3) * 48;
      auto sees = [&](int row) { return exists & (at <= row_hi[r0 + row]) & (at >= row_lo[r0 + row]); };  // (no branches)

      // ---- values that no row sees are set to zero (0 times an infinite or NaN value is NaN), and
      // values that are none but only some rows see have their product formed by hand
      bool by_hand = false;
      if (!all) {
        const uint32_t v_s = values_of(stage);
        if (!wait(&full[stage], turn)) return false;
        const bool seen = any_sees(t, at);
        if (!seen) {
          for (int x = half; x < W::ROW_BYTES / 16; x += HALVES) st_shared_v4(v_s + kv_offset<W::ROW_BYTES, TILE>(pos, x), 0, 0, 0, 0);
        }
        bool none = false;
        const int i0 = t.row0 / s.group_heads, i1 = (min(t.row0 + N, s.rows) - 1) / s.group_heads;
        if (seen && i0 != i1 && !(i1 < t.count && at <= last_seen(t, i0) && at >= first_seen(t, i1))) {
          constexpr uint32_t EXP = BF ? 0x7f80u : 0x7c00u;  // of an infinite or NaN value
#pragma unroll
          for (int x2 = 0; x2 < W::ROW_BYTES / 16 / HALVES; ++x2) {
            const int x = HALVES * x2 + half;
            uint32_t v[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(v_s + kv_offset<W::ROW_BYTES, TILE>(pos, x)) : "memory");
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              if (E8) none |= (((v[y] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;  // 0x7f: NaN
              else none |= (v[y] & EXP) == EXP || (v[y] & (EXP << 16)) == EXP << 16;
            }
          }
        }
        if (gt < N) {
          const int hi = last_seen(t, tok[gt]);
          row_hi[gt] = hi;
          row_lo[gt] = hi >= 0 ? first_seen(t, tok[gt]) : 0;
        }
        if (!vote(none, by_hand)) return false;
        if (by_hand && gt == 0) mark[it & 3] = it;
      }
      // ---- whether a score passes its row's maximum
      float v[CH][8];
      auto join_pieces = [](float (&a)[8], const float (&more)[QP][8]) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          if (QP == 2) a[x] = fmaf(more[1][x], 0.0625f, a[x]);
          if (QP == 3) a[x] = fmaf(fmaf(more[QP - 1][x], 0.0625f, more[QP > 1 ? 1 : 0][x]), 0.0625f, a[x]);
        }
      };
      auto scale = [&]() {  // f s - m; -infinity where not seen
#pragma unroll
        for (int y = 0; y < CH; ++y) {
#pragma unroll
          for (int x = 0; x < 8; x += 4) {
            const float4 nn = *reinterpret_cast<const float4*>(neg + y * 8 + x);
            const float4 ff = E8 ? *reinterpret_cast<const float4*>(fs + y * 8 + x) : make_float4(f, f, f, f);
            v[y][x] = fmaf(v[y][x], ff.x, nn.x), v[y][x + 1] = fmaf(v[y][x + 1], ff.y, nn.y);
            v[y][x + 2] = fmaf(v[y][x + 2], ff.z, nn.z), v[y][x + 3] = fmaf(v[y][x + 3], ff.w, nn.w);
          }
          if (!all) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              v[y][x] = sees(y * 8 + x) ? v[y][x] : -INFINITY;
          }
        }
      };
      bool raise = first, raised = false, done = done_before == 0;  // done: the previous weights' product has been waited for
      while (true) {
        if (raise) {
          // ---- new maxima: over the warp's positions, then over the warps
          if (!done && !wait(o_done, (done_before - 1) & 1)) return false;
          tc_fence_after_sync();
#pragma unroll (E8 ? 2 : 1)
          for (int y = 0; y < CH; ++y) {
            float w[8], more[QP][8];
            tmem_ld8(scores + y * 8, w);
#pragma unroll
            for (int z = 1; z < QP; ++z) tmem_ld8(scores + z * N + y * 8, more[z]);
            tmem_ld_wait();
            join_pieces(w, more);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              w[x] *= E8 ? fs[y * 8 + x] : f;
              if (!all) w[x] = sees(y * 8 + x) ? w[x] : -INFINITY;
            }
            const float top = across(w, [](float a, float b) { return fmaxf(a, b); });
            if (!(lane & 3)) warp_top[grp * 192 + quarter * 48 + r0 + y * 8 + (lane >> 2)] = top;
          }
          if (!sync()) return false;
          if (gt < N) {
            const int at_m = grp * 96 + odd * 48 + gt;
            const float* tops = warp_top + grp * 192 + gt;
            const float old = row_m[at_m];
            const float now = fmaxf(fmaxf(fmaxf(tops[0], tops[48]), fmaxf(tops[96], tops[144])), old);
            keep[grp * 48 + gt] = now == -INFINITY || old == -INFINITY ? 1.f : exp2_fast(old - now);
            row_m[at_m] = now;
            row_neg[at_m] = now == -INFINITY ? UNSEEN : W::BIAS - now;
          }
          if (!sync()) return false;
          if (!first) {
#pragma unroll
            for (int y = 0; y < CH; ++y)
#pragma unroll
              for (int x = 0; x < 8; ++x) sums[y][x] *= keep[grp * 48 + r0 + y * 8 + x];
#pragma unroll 1
            for (int y = 0; y < CH * WN; ++y) {
              float a[8];
              const int row = r0 + y % CH * 8;
              tmem_ld8(my_o + y / CH * N + row, a);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 8; ++x) a[x] *= keep[grp * 48 + row + x];
              tmem_st8(my_o + y / CH * N + row, a);
            }
            tmem_st_wait();
          }
          raised = done = true;
        }
        if (QP < 3) {
          float more[CH][QP][8];
#pragma unroll
          for (int y = 0; y < CH; ++y) {
            tmem_ld8(scores + y * 8, v[y]);
            if (QP == 2) tmem_ld8(scores + N + y * 8, more[y][QP - 1]);
          }
          tmem_ld_wait();
#pragma unroll
          for (int y = 0; y < CH; ++y) join_pieces(v[y], more[y]);
        } else {
#pragma unroll
          for (int y = 0; y < CH; ++y) {
            float more[QP][8];
            tmem_ld8(scores + y * 8, v[y]);
#pragma unroll
            for (int z = 1; z < QP; ++z) tmem_ld8(scores + z * N + y * 8, more[z]);
            tmem_ld_wait();
            join_pieces(v[y], more);
          }
        }
        scale();
        if (raised) break;
        float top = -INFINITY;
#pragma unroll
        for (int y = 0; y < CH; ++y)
#pragma unroll
          for (int x = 0; x < 8; ++x) top = fmaxf(top, v[y][x]);
        if (!vote(top > W::BIAS + W::SLACK, raise)) return false;
        if (!raise) break;
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[it & 1]);
      // the previous weights have been read, and O is complete up to the previous tile
      if (!done && !wait(o_done, (done_before - 1) & 1)) return false;
      tc_fence_after_sync();

      // ---- weights 2^(f s - m): in 16 bits for the product (half a step of the type each), or in
      // pieces of 8; their sums are fp32.  A piece is the upper byte of an fp16 number, an e5m2 number of
      // 3 bits: what it leaves is exact.  Three pieces hold 9 bits of a weight (the last is rounded),
      // four the 11 of fp16.
#pragma unroll
      for (int y = 0; y < CH; ++y) {
        if constexpr (E8) {
          uint32_t pieces[WP][2];
#pragma unroll
          for (int x = 0; x < 8; x += 4) {
            float a[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              a[z] = exp2_fast(v[y][x + z]);
              sums[y][x + z] += a[z];
            }
            uint32_t lo = pack_f16x2(a[0], a[1]), hi = pack_f16x2(a[2], a[3]);
#pragma unroll
            for (int z = 0; z < WP; ++z) {
              if (z == WP - 1) lo += 0x00800080u, hi += 0x00800080u;
              pieces[z][x / 4] = __byte_perm(lo, hi, 0x7531);
              if (z < WP - 1) {
                const uint32_t tl = lo & 0xff00ff00u, th = hi & 0xff00ff00u;
                const __half2 rl = __hsub2(*reinterpret_cast<const __half2*>(&lo), *reinterpret_cast<const __half2*>(&tl));
                const __half2 rh = __hsub2(*reinterpret_cast<const __half2*>(&hi), *reinterpret_cast<const __half2*>(&th));
                lo = *reinterpret_cast<const uint32_t*>(&rl);
                hi = *reinterpret_cast<const uint32_t*>(&rh);
              }
            }
          }
#pragma unroll
          for (int z = 0; z < WP; ++z)
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(my_p + (z * NC + ((r0 + y * 8) >> 4)) * (TILE * 16) + pos * 16 + ((r0 + y * 8) & 8)),
                         "r"(pieces[z][0]), "r"(pieces[z][1]) : "memory");
        } else {
#pragma unroll
          for (int x = 0; x < 8; x += 2) {
            const float a = exp2_fast(v[y][x]), b = exp2_fast(v[y][x + 1]);
            sums[y][x] += a;
            sums[y][x + 1] += b;
            const uint32_t w = BF ? pack_bf16x2(a, b) : pack_f16x2(a, b);
            st_u16(at_p[x] + (y * 8 + x) * 128, w);
            st_u16(at_p[x + 1] + (y * 8 + x + 1) * 128, w >> 16);
          }
        }
      }
      if (by_hand) {
        // O^T += V^T P^T over the rows that see a position, one channel to a thread
        if (!sync()) return false;
        const int d = D == 128 ? pos : quarter * 16 + (lane & 15);
        const uint32_t v_s = values_of(stage);
        auto value_of = [&](int y) -> float {
          const uint32_t v_at = v_s + kv_offset<W::ROW_BYTES, TILE>(y, d * W::ES / 16) + d * W::ES % 16;
          if (E8) {
            uint32_t lo, hi;
            e4m3x4_to_f16(ld_shared_u8(v_at), lo, hi);
            return __half2float(__ushort_as_half((unsigned short)lo));
          }
          const uint16_t v = ld_shared_u16(v_at);
          return BF ? to_f32(__ushort_as_bfloat16(v)) : to_f32(__ushort_as_half(v));
        };
        auto weight_of = [&](int row, int y) -> float {
          if (E8) {
            float sum = 0.f;
            for (int z = WP - 1; z >= 0; --z)
              sum += __half2float(__ushort_as_half((unsigned short)(ld_shared_u8(my_p + (z * NC + row / 16) * (TILE * 16) + y * 16 + row % 16) << 8)));
            return sum;
          }
          const uint16_t w = ld_shared_u16(my_p + (y >> 6) * (N * 128) + row * 128 + ((((y & 63) >> 3) ^ (row & 7)) << 4) + (y & 7) * 2);
          return BF ? to_f32(__ushort_as_bfloat16(w)) : to_f32(__ushort_as_half(w));
        };
        for (int c0 = r0; c0 < r0 + 8 * CH; c0 += 8) {
          float o[8];
          tmem_ld8(my_o + c0, o);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            float sum = first ? 0.f : o[x];
            const int hi = row_hi[c0 + x], lo = row_lo[c0 + x];
            for (int y = max(0, lo - t.pos0); y < TILE && t.pos0 + y <= hi; ++y)
              if ((t.valid[y >> 5] >> (y & 31)) & 1) sum += value_of(y) * weight_of(c0 + x, y);
            o[x] = sum;
          }
          tmem_st8(my_o + c0, o);
          if (first) {  // the other pieces' sums
#pragma unroll
            for (int x = 0; x < 8; ++x) o[x] = 0.f;
            for (int z = 1; z < WN; ++z) tmem_st8(my_o + z * N + c0, o);
          }
        }
        tmem_st_wait();
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[GROUPS == 2 ? grp : 0]);
    }
    // ---- the unit's end.  The next unit's queries first: its first product need not wait for what follows
    const bool stop = unit & UNIT_STOPS;
    if (!stop && !fetch_queries(stage, turn)) return false;
    if (!sync_all()) return false;  // all scores have been formed
    if (!stop) place_queries(odd ^ 1);
    // the rows' sums: over the warp's positions, then the warps
#pragma unroll
    for (int y = 0; y < CH; ++y) {
      const float sum = across(sums[y], [](float a, float b) { return a + b; });
      if (!(lane & 3)) warp_top[grp * 192 + quarter * 48 + r0 + y * 8 + (lane >> 2)] = sum;
    }
    if (!sync_all()) return false;
    const bool whole_unit = (unit & OPENS) && (unit & UNIT_CLOSES);
    const long long slot = 2LL * c + ((unit & OPENS) ? 1 : 0);
    const int unit_rows = min(N, s.rows - row0);
    if (tid < unit_rows) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int x = 0; x < GROUPS; ++x) top = fmaxf(top, row_m[x * 96 + odd * 48 + tid]);
#pragma unroll
      for (int x = 0; x < GROUPS; ++x) {
        const float m = row_m[x * 96 + odd * 48 + tid], by = m == -INFINITY ? 0.f : exp2_fast(m - top);
        const float* of = warp_top + x * 192 + tid;
        const float l = (of[0] + of[48]) + (of[96] + of[144]);
        sum += m == -INFINITY ? l : by * l;  // (nothing, or NaN, without a maximum)
        keep[x * 48 + tid] = by;
      }
      bool none = top == -INFINITY && sum == 0.f;
      const int i = tok[tid], gh = row0 + tid - i * s.group_heads;
      if (none && sees_any(s, n, i, unit_pos0[odd], unit_pos0[odd] + tiles * TILE)) none = false, top = LOWEST;
      const long long to = whole_unit ? ((long long)n * p.K + i) * p.H_q + hk * s.group_heads + gh : slot * N + tid;
      row_to[tid] = to;
      if (whole_unit) {
        const float mul = none ? 0.f : p.cache.v_scale / sum;
#pragma unroll
        for (int x = 0; x < GROUPS; ++x) keep[x * 48 + tid] *= mul;
      }
      top -= W::BIAS;
      if (!whole_unit) s.part_ml[to] = make_float2(top, sum);
      else if (p.lse) p.lse[to] = none ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
    }
    if (!sync_all()) return false;
    // every group's last product
#pragma unroll
    for (int x = 0; x < GROUPS; ++x) {
      const int products = (it + GROUPS - 1 - x) / GROUPS;
      if (products > 0 && !wait(&p_empty[x], (products - 1) & 1)) return false;
    }
    tc_fence_after_sync();
    const bool mine = D == 128 || lane < 16;
    const int d = D == 128 ? pos : quarter * 16 + (lane & 15);
#pragma unroll 1
    for (int y = 0; y < NC; ++y) {
      const int c0 = upper * (8 * NC) + y * 8;
      float o[GROUPS * WN][8];
#pragma unroll
      for (int x = 0; x < GROUPS * WN; ++x) tmem_ld8(my_lane + T_O + x / WN * W::O_COLS + x % WN * N + c0, o[x]);
      tmem_ld_wait();
      const int have = mine ? unit_rows - c0 : 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        if (x >= have) break;
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          const float by = keep[g * 48 + c0 + x];  // 0: the group has seen nothing
          float all = o[g * WN][x];
#pragma unroll
          for (int z = 1; z < WN; ++z) all += o[g * WN + z][x];
          if (by != 0.f) sum += all * by;
        }
        if (whole_unit) static_cast<A*>(p.out)[row_to[c0 + x] * D + d] = from_f32<A>(sum);
        else s.part_o[row_to[c0 + x] * D + d] = sum;
      }
    }
    tc_fence_before_sync();
    odd ^= 1;
    if (stop) return sync_all();
    // the other group's next product writes over what this one has read
    if (GROUPS == 2 && !sync_all()) return false;
    }
  };

  // ---------------------------------------------------------------- products, each issued by one thread
  // Operands' descriptors; 32 bytes of a product's depth are a step.  Keys, queries and values lie in
  // swizzled rows; the weights of an 8-bit cache in atoms of 8 positions by 16 rows.
  constexpr uint32_t SW = W::ROW_BYTES < 128 ? SW_64 : SW_128, EIGHT = W::ROW_BYTES < 128 ? 512 : 1024;
  auto product = [](uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add) {
    if (E8) umma_f8(d, a, b, id, add); else umma_bf16(d, a, b, id, add);
  };
  auto issue_scores = [&]() -> bool {
    constexpr uint32_t id = E8 ? make_idesc_f8(128, N * QP, false, false, F8_E4M3, F8_E4M3) : make_idesc(128, N, false, false, false, !BF);
    const uint64_t dq = make_sdesc(q_s, 16, EIGHT, SW), dk = make_sdesc(base, 16, EIGHT, SW);
    int units = 0;
    for (int it = 0, stage = 0, turn = 0;; ++it) {
      if (!mbar_wait(&full[stage], turn)) return false;
      if (E8 && !s.use_tma) fence_proxy_async_smem();  // (the producer's own copies)
      const uint32_t flags = meta[stage].flags;
      if ((flags & FIRST) && !mbar_wait(q_full, units++ & 1)) return false;
      if (it >= 2 && !mbar_wait(&s_empty[it & 1], ((it >> 1) - 1) & 1)) return false;
      tc_fence_after_sync();
      const uint64_t a = dk + stage * (W::STAGE_BYTES >> 4);
#pragma unroll
      for (int ks = 0; ks < W::ROW_BYTES / 32; ++ks)
        product(tmem + T_S + (it & 1) * W::S_COLS, a + ((ks >> 2) * (TILE * 128) + (ks & 3) * 32) / 16,
                dq + ((ks >> 2) * (N * 128) + (ks & 3) * 32) / 16, id, ks > 0);
      umma_commit(&s_full[it & 1]);
      if (flags & STOP) return mbar_wait(&s_full[it & 1], (it >> 1) & 1);  // nothing in flight is left behind
      umma_commit(&empty[stage]);
      if (++stage == STAGES) stage = 0, turn ^= 1;
    }
  };
  auto issue_values = [&]() -> bool {
    constexpr uint32_t id = E8 ? make_idesc_f8(D, N * WN, true, true, F8_E4M3, F8_E5M2) : make_idesc(D, N, true, false, false, !BF);
    const uint64_t dv = make_sdesc(base + W::KV_BYTES, TILE * 128, EIGHT, SW);
    const uint64_t dp = E8 ? make_sdesc(p_s, 128, TILE * 16, SW_NONE) : make_sdesc(p_s, 16, 1024, SW_128);
    int of_unit = 0;  // the unit's tiles so far
    for (int it = 0, stage = 0;; ++it) {
      const int g = GROUPS == 2 ? it & 1 : 0;
      if (!mbar_wait(&p_full[g], (it / GROUPS) & 1)) return false;
      if (E8 && !s.use_tma) fence_proxy_async_smem();
      const uint32_t flags = meta[stage].flags;
      tc_fence_after_sync();
      if (flags & FIRST) of_unit = 0;
      const bool fresh = of_unit++ < GROUPS;  // the group's first tile of a unit
      if (*reinterpret_cast<volatile int*>(&mark[it & 3]) != it) {  // else it was done by hand
        const uint64_t a = dv + stage * (W::STAGE_BYTES >> 4), b = dp + g * (W::P_BYTES >> 4);
#pragma unroll
        for (int z = 0; z < WP / WN; ++z)
#pragma unroll
          for (int ks = 0; ks < TILE * W::ES / 32; ++ks)
            product(tmem + T_O + g * W::O_COLS, a + ks * (E8 ? 2 * D : 128),
                    b + (E8 ? z * (WN * NC * TILE) + ks * 32 : ((ks >> 2) * (N * 128) + (ks & 3) * 32) / 16), id,
                    ks > 0 || z > 0 || !fresh);
      }
      umma_commit(&p_empty[g]);
      if (flags & STOP) return mbar_wait(&p_empty[g], (it / GROUPS) & 1);
      umma_commit(&empty[stage]);
      if (++stage == STAGES) stage = 0;
    }
  };

  bool ok = true;
  if (E8) {
    if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(W::SOFTMAX_REGS));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(W::OTHER_REGS));
  }
  if (warp < 8) {
    ok = softmax();
  } else if (warp == 8 || warp == 11) {
    produce<D, E8, TILE, STAGES, 2>(s, st, Ring{base, full, empty, told, meta}, map_k, map_v, warp == 11);
  } else if (warp < 11) {
    if (lane == 0) ok = warp == 9 ? issue_scores() : issue_values();
    __syncwarp();
  }
  if (!ok) *p.status = 6;
  // every wait above has a limit, so all warps come here
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 9) tmem_dealloc(tmem, W::T_COLS);
}

template <typename A, int D, int NC, bool E8>
cudaError_t launch_shape(const Params& s, const CUtensorMap& mk, const CUtensorMap& mv, int grid, cudaStream_t stream) {
  using W = Wide<A, D, E8>;
  auto kernel = attend_wide_kernel<A, D, NC, E8>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, W::SMEM);
  if (e != cudaSuccess) return e;
  if (E8) {
    // the new split of the registers waits for registers that a launch with fewer would not have
    static std::atomic<bool> enough{false};
    if (!enough.load(std::memory_order_relaxed)) {
      cudaFuncAttributes a;
      if ((e = cudaFuncGetAttributes(&a, kernel)) != cudaSuccess) return e;
      if (a.numRegs < W::LAUNCH_REGS) return cudaErrorLaunchOutOfResources;
      enough.store(true, std::memory_order_relaxed);
    }
  }
  kernel<<<grid, W::THREADS, W::SMEM, stream>>>(mk, mv, s);
  return cudaGetLastError();
}

template <typename A, int D, bool E8>
cudaError_t launch_rows(const Params& s, const CUtensorMap& mk, const CUtensorMap& mv, int grid, cudaStream_t stream) {
  return s.rows_per == 32 ? launch_shape<A, D, 2, E8>(s, mk, mv, grid, stream) : launch_shape<A, D, 3, E8>(s, mk, mv, grid, stream);
}

template <typename A>
cudaError_t launch_typed(const Params& s, const CUtensorMap& mk, const CUtensorMap& mv, int grid, cudaStream_t stream) {
  const bool e8 = s.p.cache.dtype == KDA_E4M3;
  if (s.p.cache.d == 128)
    return e8 ? launch_rows<A, 128, true>(s, mk, mv, grid, stream) : launch_rows<A, 128, false>(s, mk, mv, grid, stream);
  return e8 ? launch_rows<A, 64, true>(s, mk, mv, grid, stream) : launch_rows<A, 64, false>(s, mk, mv, grid, stream);
}

}  // namespace

cudaError_t launch_attend_wide(const Params& s, const CUtensorMap& map_k, const CUtensorMap& map_v, int grid,
                               cudaStream_t stream) {
  return s.p.dtype == KDA_BF16 ? launch_typed<__nv_bfloat16>(s, map_k, map_v, grid, stream)
                               : launch_typed<__half>(s, map_k, map_v, grid, stream);
}

}  // namespace kda
