// kda_cache_attend where 17 to 48 query rows share a key head (several tokens,
// many heads to a key head) over a 16-bit cache: both products on the tcgen05
// tensor cores, with positions and output channels on their lanes.
//
//     S^T [128 positions x N rows] = K Q^T      (A: keys as TMA lays them, B: Q)
//     O^T [d channels x N rows]   += V^T P^T    (A: values, read transposed, B: P)
//
// N is 32 or 48: with the rows on the 128 lanes most would be padding.  A
// thread of the four softmax warps has one position: it turns that position's
// N scores into weights with no exchange between lanes, since the rows' maxima
// are kept from earlier tiles as long as no score passes one by 2^8, and the
// sums of the weights are kept by thread until the unit ends.  When a score
// does pass (and at a unit's start), the maxima are found across the lanes and
// O and the sums are rescaled.  What runs once a unit is written as loops, not
// unrolled: its time is that of fetching instructions.
//
// Against warp-level instructions (kda_attend.cu, 16 rows to a group of warps),
// which run at an eighth of tcgen05's rate: 64 requests of 8192 positions with
// 40 rows, 347 us there and 203 us here.  An 8-bit cache stays there: here its
// keys and values would have to be converted through shared memory, whose
// bandwidth the products' operands take already (295 us against 278 us).
//
// Warps: 0-3 softmax, 4 producer, 5 issues the products.  One CTA on an SM.
#include "kda_attend.cuh"

namespace kda {
namespace {

constexpr int TILE = 128;
constexpr float UNSEEN = 3e38f;  // takes any score of a row without a maximum past the limit

template <int D> struct Wide {
  static constexpr int THREADS = 192;
  static constexpr int KV_BYTES = TILE * D * 2;          // keys or values of a stage
  static constexpr int STAGE_BYTES = 2 * KV_BYTES;
  static constexpr int Q_BYTES = 48 * D * 2, P_BYTES = 48 * TILE * 2;
  static constexpr int MISC_BYTES = 5120;
  static constexpr int FIT = (224 * 1024 - Q_BYTES - P_BYTES - MISC_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr int SMEM = STAGES * STAGE_BYTES + Q_BYTES + P_BYTES + MISC_BYTES + 1024;
};

// Columns of tensor memory
constexpr uint32_t T_S = 0, T_O = 128, T_COLS = 256;

__device__ __forceinline__ void st_u16(uint32_t at, uint32_t v) {
  asm volatile("{.reg .b16 l, h; mov.b32 {l, h}, %1; st.shared.b16 [%0], l;}" ::"r"(at), "r"(v) : "memory");
}

// op over the warp's lanes of each of 16 values, by halves: 16 exchanges.  Lane l gets value l >> 1;
// the values are lost.
template <typename Op> __device__ __forceinline__ float across(float (&v)[16], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = 8; half > 0; half >>= 1) {
    const bool upper = lane & (2 * half);
#pragma unroll
    for (int x = 0; x < half; ++x) {
      const float give = upper ? v[x] : v[x + half], take = upper ? v[x + half] : v[x];
      v[x] = op(take, __shfl_xor_sync(0xffffffffu, give, 2 * half));
    }
  }
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// NC: rows of a unit, in sixteens
template <typename A, int D, int NC>
__global__ void __launch_bounds__(Wide<D>::THREADS, 1)
    attend_wide_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const __grid_constant__ Params s) {
  using W = Wide<D>;
  constexpr int STAGES = W::STAGES;
  constexpr bool BF = __is_same(A, __nv_bfloat16);
  extern __shared__ uint8_t smem_raw[];
  const AttendProblem& p = s.p;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const aligned = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t q_s = base + STAGES * W::STAGE_BYTES, p_s = q_s + W::Q_BYTES;
  uint8_t* misc = aligned + STAGES * W::STAGE_BYTES + W::Q_BYTES + W::P_BYTES;
  // tables of the unit's rows, for two units in turn
  float* row_m = reinterpret_cast<float*>(misc);    // [2][48] maximum (of scores in log2 units)
  float* row_neg = row_m + 96;                      // [2][48] minus the maximum; UNSEEN while nothing is seen
  int* row_tok = reinterpret_cast<int*>(row_neg + 96);  // [2][48] the row's token
  float* warp_top = reinterpret_cast<float*>(row_tok + 96);  // [4][48]
  float* warp_sum = warp_top + 192;                 // [4][48]
  float* keep = warp_sum + 192;                     // [48] what O and the sums are rescaled with; 1 / sum at the end
  int* rows_lo = reinterpret_cast<int*>(keep + 48);  // [2][48] first and last position that a row sees,
  int* rows_hi = rows_lo + 96;                       // [2][48] for two tiles in turn
  long long* row_to = reinterpret_cast<long long*>(rows_hi + 96);  // [48] where a row's output goes
  long long* row_from = row_to + 48;                // [48] where its query is, or -1
  int* mark = reinterpret_cast<int*>(row_from + 48);  // [2]: the tile whose values are multiplied by hand, two in turn
  int* give_up = mark + 2;                          // a softmax warp met a limit
  uint64_t* bars = reinterpret_cast<uint64_t*>(mark + 4);
  uint64_t *full = bars, *empty = bars + 6, *told = bars + 12;
  uint64_t *s_full = bars + 18, *s_empty = bars + 20, *p_full = bars + 22, *p_empty = bars + 23, *q_full = bars + 24;
  Meta* meta = reinterpret_cast<Meta*>(bars + 25);  // [6]
  __shared__ uint32_t s_tmem;

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
      mbar_init(&s_empty[x], 4);
    }
    mbar_init(p_full, 4);
    mbar_init(p_empty, 1);
    mbar_init(q_full, 4);
    mark[0] = mark[1] = -1;
    *give_up = 0;
  }
  mbar_fence_init();
  if (tid == 128 && s.use_tma && p.cache.num_pages > 0) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  const Stretch st = find_stretch<TILE, W::THREADS>(s);
  if (st.left == 0) return;
  if (warp == 5) {
    tmem_alloc(&s_tmem, T_COLS);
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
    const uint32_t my_lane = tmem_addr(tmem, warp * 32, 0);
    // The four warps' barrier, with a vote.  A warp that meets a limit marks it and comes to one more
    // barrier, after which the others see the mark and leave as well: no barrier waits for a warp that
    // has left.
    auto vote = [&](bool mine, bool& any) {
      uint32_t r;
      asm volatile("{.reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, 1, 128, p; selp.u32 %0, 1, 0, q;}"
                   : "=r"(r) : "r"((uint32_t)mine) : "memory");
      any = r != 0;
      return *reinterpret_cast<volatile int*>(give_up) == 0;
    };
    auto sync = [&]() {
      bool any;
      return vote(false, any);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (__all_sync(0xffffffffu, mbar_wait(bar, parity))) return true;
      *give_up = 1;
      sync();
      return false;
    };
    // this position's place in the weights: rows of 128 bytes, 64 positions each
    uint32_t at_p[8];
#pragma unroll
    for (int x = 0; x < 8; ++x)
      at_p[x] = p_s + (tid >> 6) * (N * 128) + ((((tid & 63) >> 3) ^ x) << 4) + (tid & 7) * 2;

    // A unit's rows' tables, then its queries as they are.
    auto load_queries = [&](int stage, int turn, int odd) {
      if (!wait(&told[stage], turn)) return false;
      const Meta& t = meta[stage];
      const int n = t.n, hk = t.hk, row0 = t.row0;
      if (tid < N) {
        const int gr = row0 + tid, i = gr / s.group_heads;
        const bool real = gr < s.rows;
        row_m[odd * 48 + tid] = -INFINITY;
        row_neg[odd * 48 + tid] = UNSEEN;
        row_tok[odd * 48 + tid] = real ? i : 0x3fffffff;
        row_from[tid] = real ? ((long long)n * p.K + i) * p.q_stride + (hk * s.group_heads + gr - i * s.group_heads) * D : -1;
      }
      if (!sync()) return false;
      constexpr int EACH = N * (D / 8) / 128;  // chunks of 8 channels of a thread: all on their way together
      uint4 q[EACH];
      const int ch = tid % (D / 8);
#pragma unroll
      for (int z = 0; z < EACH; ++z) {
        const long long from = row_from[(tid + z * 128) / (D / 8)];
        q[z] = from < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(static_cast<const A*>(p.q) + from + ch * 8);
      }
#pragma unroll
      for (int z = 0; z < EACH; ++z) {
        const int row = (tid + z * 128) / (D / 8);
        st_shared_v4(q_s + (ch >> 3) * (N * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), q[z].x, q[z].y, q[z].z, q[z].w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      return true;
    };

    float sums[NC][16];  // of this position's weights of each row, over the unit's tiles
    int odd = 0;
    if (!load_queries(0, 0, odd)) return false;
    for (int it = 0, stage = 0, turn = 0;; ++it) {
      if (!wait(&s_full[it & 1], (it >> 1) & 1)) return false;
      if (!wait(&told[stage], turn)) return false;
      tc_fence_after_sync();
      const Meta& t = meta[stage];  // the stage is given back after this tile's last look at it
      const uint32_t flags = t.flags;
      const bool first = flags & FIRST, all = flags & FULL;
      const float f = p.scale * p.cache.k_scale * 1.44269504088896340736f;
      const float* neg = row_neg + odd * 48;
      const int* tok = row_tok + odd * 48;
      const uint32_t scores = my_lane + T_S + (it & 1) * 64;
      int at = 0;
      bool exists = true;
      if (!all) {
        at = t.pos0 + tid;
        exists = (t.valid[tid >> 5] >> lane) & 1;
      }
      int *row_lo = rows_lo + (it & 1) * 48, *row_hi = rows_hi + (it & 1) * 48;
      auto sees = [&](int row) { return exists & (at <= row_hi[row]) & (at >= row_lo[row]); };  // (no branches)

      // ---- values that no row sees are set to zero (0 times an infinite or NaN value is NaN), and
      // values that are none but only some rows see have their product formed by hand
      bool by_hand = false;
      if (!all) {
        const uint32_t v_s = values_of(stage);
        if (!wait(&full[stage], turn)) return false;
        const bool seen = any_sees(t, at);
        if (!seen) {
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            for (int x = 0; x < 8; ++x) st_shared_v4(v_s + h * (TILE * 128) + tid * 128 + ((x ^ (tid & 7)) << 4), 0, 0, 0, 0);
        }
        bool none = false;
        const int i0 = t.row0 / s.group_heads, i1 = (min(t.row0 + N, s.rows) - 1) / s.group_heads;
        if (seen && i0 != i1 && !(i1 < t.count && at <= last_seen(t, i0) && at >= first_seen(t, i1))) {
          constexpr uint32_t EXP = BF ? 0x7f80u : 0x7c00u;  // of an infinite or NaN value
#pragma unroll
          for (int x = 0; x < D / 8; ++x) {
            uint32_t v[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(v_s + (x >> 3) * (TILE * 128) + tid * 128 + (((x & 7) ^ (tid & 7)) << 4)) : "memory");
#pragma unroll
            for (int y = 0; y < 4; ++y) none |= (v[y] & EXP) == EXP || (v[y] & (EXP << 16)) == EXP << 16;
          }
        }
        if (tid < N) {
          const int hi = last_seen(t, tok[tid]);
          row_hi[tid] = hi;
          row_lo[tid] = hi >= 0 ? first_seen(t, tok[tid]) : 0;
        }
        if (!vote(none, by_hand)) return false;
        if (by_hand && tid == 0) mark[it & 1] = it;
      }
      // ---- whether a score passes its row's maximum
      float v[NC][16];
      auto scale = [&]() {  // f s - m; -infinity where not seen
#pragma unroll
        for (int y = 0; y < NC; ++y) {
#pragma unroll
          for (int x = 0; x < 16; x += 4) {
            const float4 nn = *reinterpret_cast<const float4*>(neg + y * 16 + x);
            v[y][x] = fmaf(v[y][x], f, nn.x), v[y][x + 1] = fmaf(v[y][x + 1], f, nn.y);
            v[y][x + 2] = fmaf(v[y][x + 2], f, nn.z), v[y][x + 3] = fmaf(v[y][x + 3], f, nn.w);
          }
          if (!all) {
#pragma unroll
            for (int x = 0; x < 16; ++x)
              v[y][x] = sees(y * 16 + x) ? v[y][x] : -INFINITY;
          }
        }
      };
      if (first) {
#pragma unroll
        for (int y = 0; y < NC; ++y)
#pragma unroll
          for (int x = 0; x < 16; ++x) sums[y][x] = 0.f;
      }
      bool raise = first, done = false;  // done: the previous tile's product has been waited for
      while (true) {
        if (raise) {
          // ---- new maxima: over the warp's positions, then over the warps
          if (it > 0 && !done && !wait(p_empty, (it - 1) & 1)) return false;
          tc_fence_after_sync();
#pragma unroll 1
          for (int y = 0; y < NC; ++y) {
            float w[16];
            tmem_ld16(scores + y * 16, w);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              w[x] *= f;
              if (!all) w[x] = sees(y * 16 + x) ? w[x] : -INFINITY;
            }
            const float top = across(w, [](float a, float b) { return fmaxf(a, b); });
            if (!(lane & 1)) warp_top[warp * 48 + y * 16 + (lane >> 1)] = top;
          }
          if (!sync()) return false;
          if (tid < N) {
            const float old = row_m[odd * 48 + tid];
            const float now = fmaxf(fmaxf(fmaxf(warp_top[tid], warp_top[48 + tid]), fmaxf(warp_top[96 + tid], warp_top[144 + tid])), old);
            keep[tid] = now == -INFINITY || old == -INFINITY ? 1.f : exp2_fast(old - now);
            row_m[odd * 48 + tid] = now;
            row_neg[odd * 48 + tid] = now == -INFINITY ? UNSEEN : -now;
          }
          if (!sync()) return false;
          if (!first) {
#pragma unroll
            for (int y = 0; y < NC; ++y)
#pragma unroll
              for (int x = 0; x < 16; ++x) sums[y][x] *= keep[y * 16 + x];
#pragma unroll 1
            for (int y = 0; y < NC; ++y) {
              float a[16];
              tmem_ld16(my_lane + T_O + y * 16, a);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x) a[x] *= keep[y * 16 + x];
              tmem_st16(my_lane + T_O + y * 16, a);
            }
            tmem_st_wait();
          }
          done = true;
        }
#pragma unroll
        for (int y = 0; y < NC; ++y) tmem_ld16(scores + y * 16, v[y]);
        tmem_ld_wait();
        scale();
        if (done) break;
        float top = -INFINITY;
#pragma unroll
        for (int y = 0; y < NC; ++y)
#pragma unroll
          for (int x = 0; x < 16; ++x) top = fmaxf(top, v[y][x]);
        if (!vote(top > 8.f, raise)) return false;
        if (!raise) break;
      }
      // the previous weights have been read, and O is complete up to the previous tile
      if (it > 0 && !done && !wait(p_empty, (it - 1) & 1)) return false;
      tc_fence_after_sync();

      // ---- weights 2^(f s - m), in 16 bits for the product (half a step of the type each); their sums
      // are fp32
#pragma unroll
      for (int y = 0; y < NC; ++y)
#pragma unroll
        for (int x = 0; x < 16; x += 2) {
          const float a = exp2_fast(v[y][x]), b = exp2_fast(v[y][x + 1]);
          sums[y][x] += a;
          sums[y][x + 1] += b;
          const uint32_t w = BF ? pack_bf16x2(a, b) : pack_f16x2(a, b);
          st_u16(at_p[x & 7] + (y * 16 + x) * 128, w);
          st_u16(at_p[(x + 1) & 7] + (y * 16 + x + 1) * 128, w >> 16);
        }
      if (by_hand) {
        // O^T += V^T P^T over the rows that see a position, one channel to a thread
        if (!sync()) return false;
        const int d = D == 128 ? tid : warp * 16 + (lane & 15);
        const uint32_t v_at = values_of(stage) + (d >> 6) * (TILE * 128) + (d & 7) * 2;
        for (int c0 = 0; c0 < N; c0 += 16) {
          float o[16];
          tmem_ld16(my_lane + T_O + c0, o);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float sum = first ? 0.f : o[x];
            const int hi = row_hi[c0 + x], lo = row_lo[c0 + x];
            for (int y = max(0, lo - t.pos0); y < TILE && t.pos0 + y <= hi; ++y) {
              if (!((t.valid[y >> 5] >> (y & 31)) & 1)) continue;
              const uint16_t v = ld_shared_u16(v_at + y * 128 + ((((d & 63) >> 3) ^ (y & 7)) << 4));
              const uint16_t w = ld_shared_u16(p_s + (y >> 6) * (N * 128) + (c0 + x) * 128 + ((((y & 63) >> 3) ^ (x & 7)) << 4) + (y & 7) * 2);
              sum += BF ? to_f32(__ushort_as_bfloat16(v)) * to_f32(__ushort_as_bfloat16(w))
                        : to_f32(__ushort_as_half(v)) * to_f32(__ushort_as_half(w));
            }
            o[x] = sum;
          }
          tmem_st16(my_lane + T_O + c0, o);
        }
        tmem_st_wait();
      }
      const int t_n = t.n, t_hk = t.hk, t_row0 = t.row0;
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s_empty[it & 1]);
        mbar_arrive(p_full);
      }

      if (flags & LAST) {
        // the next unit's queries first: its first product need not wait for what follows
        const bool stop = flags & STOP;
        int next_stage = stage + 1, next_turn = turn;
        if (next_stage == STAGES) next_stage = 0, next_turn ^= 1;
        if (!stop && !load_queries(next_stage, next_turn, odd ^ 1)) return false;
        // the rows' sums: over the warp's positions, then the warps
        const int rows = odd * 48;
#pragma unroll
        for (int y = 0; y < NC; ++y) {
          const float sum = across(sums[y], [](float a, float b) { return a + b; });
          if (!(lane & 1)) warp_sum[warp * 48 + y * 16 + (lane >> 1)] = sum;
        }
        if (!sync()) return false;
        const bool whole_unit = (flags & OPENS) && (flags & CLOSES);
        const long long slot = 2LL * c + ((flags & OPENS) ? 1 : 0);
        const int unit_rows = min(N, s.rows - t_row0);
        if (tid < unit_rows) {
          const float m = row_m[rows + tid];
          const float sum = (warp_sum[tid] + warp_sum[48 + tid]) + (warp_sum[96 + tid] + warp_sum[144 + tid]);
          const bool none = m == -INFINITY;
          const int i = tok[tid], gh = t_row0 + tid - i * s.group_heads;
          const long long to = whole_unit ? ((long long)t_n * p.K + i) * p.H_q + t_hk * s.group_heads + gh : slot * N + tid;
          row_to[tid] = to;
          keep[tid] = none ? 0.f : whole_unit ? p.cache.v_scale / sum : 1.f;
          if (!whole_unit) s.part_ml[to] = make_float2(m, sum);
          else if (p.lse) p.lse[to] = none ? -INFINITY : (m + log2f(sum)) * 0.69314718055994530942f;
        }
        if (!sync()) return false;
        if (!wait(p_empty, it & 1)) return false;
        tc_fence_after_sync();
        const bool mine = D == 128 || lane < 16;
        const int d = D == 128 ? tid : warp * 16 + (lane & 15);
#pragma unroll 1
        for (int y = 0; y < NC; ++y) {
          float o[16];
          tmem_ld16(my_lane + T_O + y * 16, o);
          tmem_ld_wait();
          const int have = mine ? unit_rows - y * 16 : 0;
          if (whole_unit) {
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float by = keep[y * 16 + x];  // 0: nothing was seen
              if (x < have) static_cast<A*>(p.out)[row_to[y * 16 + x] * D + d] = from_f32<A>(by == 0.f ? 0.f : o[x] * by);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x)
              if (x < have) s.part_o[row_to[y * 16 + x] * D + d] = keep[y * 16 + x] == 0.f ? 0.f : o[x];
          }
        }
        tc_fence_before_sync();
        odd ^= 1;
        if (stop) return sync();
      }
      if (++stage == STAGES) stage = 0, turn ^= 1;
    }
  };

  // ---------------------------------------------------------------- products, issued by one thread
  auto issue = [&]() -> bool {
    constexpr uint32_t id_s = make_idesc(128, N, false, false, false, !BF), id_o = make_idesc(D, N, true, false, false, !BF);
    // operands' descriptors; a step of 16 along a product adds a constant (in units of 16 bytes)
    const uint64_t dq = make_sdesc(q_s, 16, 1024, SW_128), dp = make_sdesc(p_s, 16, 1024, SW_128);
    const uint64_t dk = make_sdesc(base, 16, 1024, SW_128);
    const uint64_t dv = make_sdesc(base + W::KV_BYTES, TILE * 128, 1024, SW_128);
    int units = 0;
    auto values = [&](int it, int stage, uint32_t flags) {
      if (!mbar_wait(p_full, it & 1)) return false;
      tc_fence_after_sync();
      if (*reinterpret_cast<volatile int*>(&mark[it & 1]) != it) {  // else it was done by hand
        const uint64_t a = dv + stage * (W::STAGE_BYTES >> 4);
#pragma unroll
        for (int ks = 0; ks < TILE / 16; ++ks)
          umma_bf16(tmem + T_O, a + ks * 128, dp + ((ks >> 2) * (N * 128) + (ks & 3) * 32) / 16, id_o, ks > 0 || !(flags & FIRST));
      }
      umma_commit(p_empty);
      umma_commit(&empty[stage]);
      return true;
    };
    int before_stage = 0;
    uint32_t before_flags = 0;
    for (int it = 0, stage = 0, turn = 0;; ++it) {
      if (!mbar_wait(&full[stage], turn)) return false;
      const uint32_t flags = meta[stage].flags;
      if ((flags & FIRST) && !mbar_wait(q_full, units++ & 1)) return false;
      if (it >= 2 && !mbar_wait(&s_empty[it & 1], ((it >> 1) - 1) & 1)) return false;
      tc_fence_after_sync();
      const uint64_t a = dk + stage * (W::STAGE_BYTES >> 4);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        umma_bf16(tmem + T_S + (it & 1) * 64, a + ((ks >> 2) * (TILE * 128) + (ks & 3) * 32) / 16,
                  dq + ((ks >> 2) * (N * 128) + (ks & 3) * 32) / 16, id_s, ks > 0);
      umma_commit(&s_full[it & 1]);
      umma_commit(&empty[stage]);
      if (it > 0 && !values(it - 1, before_stage, before_flags)) return false;
      if (flags & STOP) return values(it, stage, flags);
      before_stage = stage;
      before_flags = flags;
      if (++stage == STAGES) stage = 0, turn ^= 1;
    }
  };

  bool ok = true;
  if (warp < 4) {
    ok = softmax();
  } else if (warp == 4) {
    produce<D, false, TILE, STAGES>(s, st, Ring{base, full, empty, told, meta}, map_k, map_v);
  } else {
    if (lane == 0) ok = issue();
    __syncwarp();
  }
  if (!ok) *p.status = 6;
  // every wait above has a limit, so all warps come here
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 5) tmem_dealloc(tmem, T_COLS);
}

template <typename A, int D, int NC>
cudaError_t launch_rows(const Params& s, const CUtensorMap& mk, const CUtensorMap& mv, int grid, cudaStream_t stream) {
  using W = Wide<D>;
  auto kernel = attend_wide_kernel<A, D, NC>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, W::SMEM);
  if (e != cudaSuccess) return e;
  kernel<<<grid, W::THREADS, W::SMEM, stream>>>(mk, mv, s);
  return cudaGetLastError();
}

template <typename A>
cudaError_t launch_typed(const Params& s, const CUtensorMap& mk, const CUtensorMap& mv, int grid, cudaStream_t stream) {
  if (s.p.cache.d == 128)
    return s.rows_per == 32 ? launch_rows<A, 128, 2>(s, mk, mv, grid, stream) : launch_rows<A, 128, 3>(s, mk, mv, grid, stream);
  return s.rows_per == 32 ? launch_rows<A, 64, 2>(s, mk, mv, grid, stream) : launch_rows<A, 64, 3>(s, mk, mv, grid, stream);
}

}  // namespace

cudaError_t launch_attend_wide(const Params& s, const CUtensorMap& map_k, const CUtensorMap& map_v, int grid,
                               cudaStream_t stream) {
  return s.p.dtype == KDA_BF16 ? launch_typed<__nv_bfloat16>(s, map_k, map_v, grid, stream)
                               : launch_typed<__half>(s, map_k, map_v, grid, stream);
}

}  // namespace kda
