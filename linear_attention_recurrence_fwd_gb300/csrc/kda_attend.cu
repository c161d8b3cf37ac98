// Attention of each sequence's newest tokens over its pages.
//
//     s_j = scale q . k_j,   o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),
//     m = max_j s_j,         lse = m + ln sum_j e^(s_j - m)
//
// over the positions j that the token sees, in one pass: m and the two sums
// are carried and rescaled when m grows.  The query rows of one key head (K
// tokens times H_q / H_kv heads, in groups of up to 48) share one read of its
// keys and values, so the call is bound by HBM: 2 flop per row and byte of a
// 16-bit cache.
//
// This file: up to 16 rows.  17 to 48 rows are kda_attend_wide.cu; how the work
// is cut is kda_attend.cuh.
//
// Work.  A unit is (sequence, key head, row group); its positions are cut into
// tiles of 64 or 128.  The tiles of all units, one after the other, are cut
// into equal stretches, whatever the lengths are; a unit that ends up in
// several CTAs is joined from their unnormalised parts by a second small
// kernel.  Where units are short, each CTA takes whole units instead and
// nothing is joined.  CTAs walk the heads of the same positions in teams of up
// to 8, since a token's heads lie side by side: DRAM is then read in longer
// runs (64 requests of 8192 positions, 8 key heads of 64: 195 us without
// teams, 163 us with).
//
// A CTA is one producer warp and 4 consumer warps around a ring of stages (a
// tile's keys and values).  The producer looks up pages and issues TMA
// boxes of the rows that lie in one page.  Each consumer warp takes 16 or 32
// positions of every tile through scores, softmax and values by itself, with
// a running maximum, sum and output of its own: no barrier between warps
// until a unit ends, when they are joined through shared memory.  (Warps that
// share a tile's softmax and split the output's columns need three barriers a
// tile; measured, 1.0 us for a tile of 64 positions against 0.74 us for its
// share of the HBM bandwidth at two CTAs on an SM.)  The products are
// warp-level tensor core instructions (m16n8k16): 16 rows are what one token
// of most layouts fills.
//
// Measured (32 query heads of 128): 256 requests of 7 to 8191 positions on 8
// key heads 630 us, 6.8 TB/s, the copy bandwidth; one request of 2^20
// positions, 16 heads on 2, 167 us (6.4 TB/s); 64 requests of 8192, 8 key heads,
// 316 us (6.8 TB/s), and 8-bit 189 us (5.7 TB/s: converting 8-bit fragments to
// fp16 is what bounds it).
#include <cstdint>

#include "kda_internal.h"
#include "kda_attend.cuh"
#include "kda_types.cuh"
#include "tma_host.h"

namespace kda {
namespace {

constexpr int KW = 4;  // consumer warps that share a tile's positions

// A consumer warp's share of a tile is KT positions, 4 KB of keys and as much of values (8-bit heads of
// 64: 2 KB).  Two CTAs on an SM.
template <int D, bool E8> struct Shape {
  static constexpr int ROW_BYTES = D * (E8 ? 1 : 2);       // of a key or value
  static constexpr int KT = ROW_BYTES > 128 ? 16 : 32;
  static constexpr int TILE = KT * KW;
  static constexpr int THREADS = 32 * KW + 32;
  static constexpr int ROWS = 16;
  static constexpr int BOX_BYTES = ROW_BYTES < 128 ? ROW_BYTES : 128;
  static constexpr int KV_BYTES = TILE * ROW_BYTES;
  static constexpr int STAGE_BYTES = 2 * KV_BYTES;
  static constexpr int MISC_BYTES = 5120;
  static constexpr int FIT = (112 * 1024 - MISC_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM = STAGES * STAGE_BYTES + MISC_BYTES + 1024;
  // At a unit's end a stage holds every warp's output of SETS times 8 rows and JC columns.
  static constexpr int JC = KW * 8 * D * 4 <= STAGE_BYTES ? D : D / 2;
  static constexpr int SETS = KW * 16 * JC * 4 <= STAGE_BYTES ? 2 : 1;
  static_assert(KW * SETS * 8 * JC * 4 <= STAGE_BYTES, "the join's buffer is a stage");
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// c += a b, 16 x 8 x 16, both operands bf16 or both fp16
template <bool BF>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename A, bool E8, int D>
__global__ void __launch_bounds__(Shape<D, E8>::THREADS, 2)
    attend_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                  const __grid_constant__ Params s) {
  using S = Shape<D, E8>;
  constexpr int KT = S::KT, TILE = S::TILE, THREADS = S::THREADS, STAGES = S::STAGES;
  constexpr bool BF = !E8 && __is_same(A, __nv_bfloat16);
  extern __shared__ uint8_t smem_raw[];
  const AttendProblem& p = s.p;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* const aligned = smem_raw + (base - smem_u32(smem_raw));
  uint8_t* misc = aligned + STAGES * S::STAGE_BYTES;
  float2* red = reinterpret_cast<float2*>(misc);          // [2][16][KW]: maximum and sum
  uint64_t* full = reinterpret_cast<uint64_t*>(red + 2 * 16 * KW);
  uint64_t* empty = full + 8;
  uint64_t* told = empty + 8;                              // a stage's Meta is written
  uint64_t* joined = told + 8;                             // the consumer warps' own barrier
  Meta* meta = reinterpret_cast<Meta*>(joined + 2);       // [8]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid < STAGES) {
    mbar_init(&full[tid], s.use_tma ? 1 : 33);
    mbar_init(&empty[tid], KW);
    mbar_init(&told[tid], 1);
  }
  if (tid == 0) mbar_init(joined, KW);
  mbar_fence_init();
  if (tid == 32 * KW && s.use_tma && p.cache.num_pages > 0) {
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }

  const Stretch st = find_stretch<TILE, THREADS>(s);
  if (st.left == 0) return;
  const int c = blockIdx.x;

  if (warp >= KW) {
    produce<D, E8, TILE, STAGES>(s, st, Ring{base, full, empty, told, meta}, map_k, map_v);
    return;
  }

  // -------------------------------------------------------------- consumers
  const int kw = warp;  // the warp's share of a tile's positions
  const int g = lane >> 2, tq = lane & 3;  // a fragment's row (and row + 8) and column pair
  constexpr int NS = KT / 8;               // n-tiles of 8 positions
  constexpr int NT = D / 8;                // n-tiles of output columns
  constexpr int KP = D / (E8 ? 32 : 16);   // fragment loads over a row's channels
  constexpr int PITCH = S::BOX_BYTES;      // of a row of keys or values in shared memory
  // Weights are 2^(f s - m), m the running maximum less BIAS, and reach 2^(BIAS + SLACK) before m is
  // moved.  In fp16 the bias keeps small ones to 2^-32 of the largest (its least step is 2^-24).
  constexpr float BIAS = BF ? 0.f : 7.f, SLACK = 8.f;
  float o[NT][4], m[2], l[2], f[2];
  int ri[2];                               // the token of each of the thread's two rows
  uint32_t qf[D / 16][4];
  const int mat = lane >> 3, mr = lane & 7;  // ldmatrix: this lane's matrix and row in it

  // Shared-memory offsets that do not change.  Chunks of 16 bytes are XORed with the row, so a step
  // of the inner loops is one of four offsets plus a constant.
  uint32_t k_off[4], v_off[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    constexpr int CH = S::ROW_BYTES / 16;
    k_off[x] = E8 ? kv_offset<S::ROW_BYTES, TILE>(kw * KT + (mat & 1) * 8 + mr, (x * 2 + (mat >> 1)) % CH)
                  : kv_offset<S::ROW_BYTES, TILE>(kw * KT + (mat >> 1) * 8 + mr, x * 2 + (mat & 1));
    v_off[x] = kv_offset<S::ROW_BYTES, TILE>(kw * KT + (mat & 1) * 8 + mr, (x * 2 + (mat >> 1)) % CH);
  }

  // A barrier of the consumer warps with a limit to its wait; false: given up.
  uint32_t joins = 0;
  auto sync = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(joined);
    const bool ok = mbar_wait(joined, joins++ & 1);
    if (!ok) *p.status = 6;
    return ok;
  };

  bool fresh = true;  // the next tile is a unit's first
  uint32_t odd = 0;   // the unit's parity
  for (int it = 0, stage = 0, turn = 0;; ++it) {
    const Meta& t = meta[stage];
    const uint32_t k_s = base + stage * S::STAGE_BYTES, v_s = k_s + S::KV_BYTES;
    if (fresh) {
      // ---- the unit's queries, straight into fragments while the tile is on its way.  For an 8-bit
      // cache they become fp16, each row scaled by a power of two so that its range fits, its channels
      // in the order of the 8-bit fragments: of 16 channels, 4 c + {0, 1} in places 2 c + {0, 1}, and
      // 4 c + {2, 3} in places 8 + 2 c + {0, 1}.
      if (!mbar_wait(&told[stage], turn)) {
        *p.status = 6;  // the other warps meet a limit too, here or at their barrier
        return;
      }
      const int n = t.n, hk = t.hk, row0 = t.row0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int gr = row0 + h * 8 + g;
        const bool real = gr < s.rows;
        m[h] = -INFINITY;
        l[h] = 0.f;
        f[h] = p.scale * p.cache.k_scale * 1.44269504088896340736f;
        ri[h] = real ? gr / s.group_heads : 0x3fffffff;
        const A* src = static_cast<const A*>(p.q);
        if (real) src += ((long long)n * p.K + ri[h]) * p.q_stride + (hk * s.group_heads + gr - ri[h] * s.group_heads) * D;
        if (E8) {
          uint2 v[D / 16];
          float big = 0.f;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            v[ks] = real ? *reinterpret_cast<const uint2*>(src + ks * 16 + tq * 4) : make_uint2(0, 0);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int z = 0; z < 4; ++z) big = fmaxf(big, fabsf(to_f32(reinterpret_cast<const A*>(&v[ks])[z])));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          // 2^floor(log2 big), within the powers whose inverse is an fp32 number
          const int ex = min(max((int)((__float_as_uint(big) >> 23) & 255u), 1), 253);
          f[h] *= __uint_as_float((uint32_t)ex << 23);
          const float inv = __uint_as_float((uint32_t)(254 - ex) << 23);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const A* e = reinterpret_cast<const A*>(&v[ks]);
            qf[ks][h] = pack_f16x2(to_f32(e[0]) * inv, to_f32(e[1]) * inv);
            qf[ks][2 + h] = pack_f16x2(to_f32(e[2]) * inv, to_f32(e[3]) * inv);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int z = 0; z < 2; ++z)
              qf[ks][z * 2 + h] = real ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + z * 8 + tq * 2) : 0u;
        }
      }
    }
    if (!mbar_wait(&full[stage], turn)) {
      *p.status = 6;
      return;
    }
    const uint32_t flags = t.flags;

    // ---- what this group's rows see of this warp's positions: everything, nothing or a part
    bool all = flags & FULL, some = true;
    int t_pos0 = 0, t_len = 0, t_count = 0, t_end = 0;  // t_pos0: of this warp's positions
    int i0 = 0, i1 = 0;                                 // tokens of the group's rows
    uint32_t valid = ~0u;
    auto last_seen = [&](int i) { return i < t_count ? min(t_len + i, t_end - 1) : -1; };
    auto first_seen = [&](int i) { return p.window && t_len + i >= p.window ? t_len + i - p.window + 1 : 0; };
    if (!all) {
      t_pos0 = t.pos0 + kw * KT, t_len = t.len, t_count = t.count, t_end = t.end;
      valid = t.valid[(kw * KT) >> 5] >> ((kw * KT) & 31);
      const uint32_t every = KT == 32 ? ~0u : 0xffffu;
      const int ra = t.row0, rb = min(ra + 16, s.rows) - 1;
      i0 = ra / s.group_heads, i1 = rb / s.group_heads;
      const int newest = min(i1, t_count - 1);
      some = ra < s.rows && newest >= i0 && t_pos0 <= last_seen(newest) && t_pos0 + KT > first_seen(i0) && (valid & every);
      all = some && i1 < t_count && t_pos0 + KT - 1 <= last_seen(i0) && t_pos0 >= first_seen(i1) && (valid & every) == every;
    }
    if (some) {
      // ---- scores
      constexpr int SPLIT = NS < 4 ? 2 : 1;  // sums side by side, to hide an instruction's latency
      float sc[SPLIT][NS][4];
#pragma unroll
      for (int x = 0; x < SPLIT; ++x)
#pragma unroll
        for (int nt = 0; nt < NS; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[x][nt][e] = 0.f;
      constexpr int BATCH = KP / 2;  // loads ahead of their products
      uint32_t kr[2 * BATCH][NS / 2][4];           // two batches: one in use, one on its way
      auto load_keys = [&](int kp) {
#pragma unroll
        for (int kb = 0; kb < NS / 2; ++kb)
          ldmatrix_x4(k_s + k_off[kp & 3] + (kp >> 2) * (TILE * 128) + kb * 16 * PITCH, kr[kp % (2 * BATCH)][kb]);
      };
#pragma unroll
      for (int x = 0; x < BATCH; ++x) load_keys(x);
#pragma unroll
      for (int kp = 0; kp < KP; ++kp) {
        if (kp % BATCH == 0) {
#pragma unroll
          for (int x = kp + BATCH; x < kp + 2 * BATCH; ++x)
            if (x < KP) load_keys(x);
        }
#pragma unroll
        for (int kb = 0; kb < NS / 2; ++kb) {
          // 16-bit: the four parts are n-tile 0 b0 b1, n-tile 1 b0 b1.  8-bit: each is b0 and b1 of
          // 8 positions, for 16 channels; parts 0, 1 of the first 16 and 2, 3 of the second.
          const uint32_t(&r)[4] = kr[kp % (2 * BATCH)][kb];
#pragma unroll
          for (int sub = 0; sub < (E8 ? 2 : 1); ++sub) {
            uint32_t b[4] = {r[0], r[1], r[2], r[3]};
            if (E8) {
              e4m3x4_to_f16(r[sub * 2], b[0], b[1]);
              e4m3x4_to_f16(r[sub * 2 + 1], b[2], b[3]);
            }
            const int ks = E8 ? kp * 2 + sub : kp;
            mma<BF>(sc[ks % SPLIT][kb * 2], qf[ks], b[0], b[1]);
            mma<BF>(sc[ks % SPLIT][kb * 2 + 1], qf[ks], b[2], b[3]);
          }
        }
      }
      // the values' fragments are on their way while the weights are formed
      uint32_t vr[NS / 2][KP][4];
#pragma unroll
      for (int ks = 0; ks < NS / 2; ++ks)
#pragma unroll
        for (int cp = 0; cp < KP; ++cp)
          ldmatrix_x4_t(v_s + v_off[cp & 3] + (cp >> 2) * (TILE * 128) + ks * 16 * PITCH, vr[ks][cp]);

      // ---- scale, mask, row maxima
      float top[2];
      bool move = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int nt = 0; nt < NS; ++nt)
#pragma unroll
          for (int e = h * 2; e < h * 2 + 2; ++e) {
            if (SPLIT > 1) sc[0][nt][e] += sc[SPLIT - 1][nt][e];
            sc[0][nt][e] *= f[h];
          }
        if (!all) {
          const int hi = last_seen(ri[h]), lo = hi >= 0 ? first_seen(ri[h]) : 0;
#pragma unroll
          for (int nt = 0; nt < NS; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = nt * 8 + tq * 2 + e;
              if (t_pos0 + key < lo || t_pos0 + key > hi || !((valid >> key) & 1)) sc[0][nt][h * 2 + e] = -INFINITY;
            }
        }
        float x = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NS; ++nt) x = fmaxf(x, fmaxf(sc[0][nt][h * 2], sc[0][nt][h * 2 + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        top[h] = x - BIAS;
        move |= top[h] > m[h] + SLACK;
      }
      // The output and the sum are rescaled only where a row's maximum has grown by more than 2^8:
      // until then the weights are just larger, which costs no precision.
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = fmaxf(m[h], top[h]);
          const float keep = mn == -INFINITY ? 1.f : exp2_fast(m[h] - mn);
          m[h] = mn;
          l[h] *= keep;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            o[nt][h * 2] *= keep;
            o[nt][h * 2 + 1] *= keep;
          }
        }
      }

      // ---- weights, in 16 bits for the product (half a step of the type each; their sum is fp32).
      // The scores' fragments are the weights' fragments.
      uint32_t pf[NS / 2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float use = m[h] == -INFINITY ? 0.f : m[h];  // nothing seen yet: weights 2^-inf = 0
        float sum = 0.f;
#pragma unroll
        for (int nt = 0; nt < NS; ++nt) {
          const float x = exp2_fast(sc[0][nt][h * 2] - use), y = exp2_fast(sc[0][nt][h * 2 + 1] - use);
          sum += x + y;
          pf[nt >> 1][(nt & 1) * 2 + h] = BF ? pack_bf16x2(x, y) : pack_f16x2(x, y);
        }
        l[h] += sum;
      }

      // ---- values
#pragma unroll
      for (int ks = 0; ks < NS / 2; ++ks) {
        uint32_t(&raw)[KP][4] = vr[ks];
        bool apart = false;
        if (!all) {
          // 0 times an infinite or NaN value is NaN: values that none of the rows' tokens sees are set
          // to zero.  If a value that only some of them see is none, they take turns below.
          const int lo = first_seen(i0), hi = last_seen(min(i1, t_count - 1));
          bool odd_value = false;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t mask = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = ks * 16 + z * 8 + tq * 2 + e, at = t_pos0 + key;
              if (at >= lo && at <= hi && ((valid >> key) & 1)) mask |= 0xffffu << (16 * e);
            }
#pragma unroll
            for (int cp = 0; cp < KP; ++cp)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t& v = raw[cp][y * 2 + z];
                v &= mask;  // two positions of one column, or of two (8-bit)
                if (E8) odd_value |= (v & 0x7fu) == 0x7fu || (v & 0x7f00u) == 0x7f00u ||
                                     (v & 0x7f0000u) == 0x7f0000u || (v & 0x7f000000u) == 0x7f000000u;
                else odd_value |= (v & (BF ? 0x7f80u : 0x7c00u)) == (BF ? 0x7f80u : 0x7c00u) ||
                                  (v & (BF ? 0x7f800000u : 0x7c000000u)) == (BF ? 0x7f800000u : 0x7c000000u);
              }
          }
          apart = i0 != i1 && __any_sync(0xffffffffu, odd_value);
        }
        constexpr int NB = E8 ? 4 : 2;  // n-tiles of a fragment load: 16 columns, or 2 x 16 (8-bit: even, odd)
        auto columns = [&](int cp, uint32_t (&b)[2 * NB]) {
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            // 8-bit, z: 16 columns z >> 1, positions 8 (z & 1) ..; bytes in the order position, column
            if (E8) e4m3x4_to_f16(__byte_perm(raw[cp][z], 0, 0x3120), b[E8 ? (z >> 1) * 4 + (z & 1) : 0], b[E8 ? (z >> 1) * 4 + 2 + (z & 1) : 0]);
            else b[z] = raw[cp][z];
          }
        };
        if (!apart) {
#pragma unroll
          for (int cp = 0; cp < KP; ++cp) {
            uint32_t b[2 * NB];
            columns(cp, b);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma<BF>(o[cp * NB + nb], pf[ks], b[nb * 2], b[nb * 2 + 1]);
          }
        } else {
#pragma unroll 1
          for (int i = i0; i <= i1; ++i) {
            const int hi = last_seen(i), lo = hi >= 0 ? first_seen(i) : 0;
            uint32_t mask[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int at = t_pos0 + ks * 16 + z * 8 + tq * 2;
              mask[z] = (at >= lo && at <= hi ? 0xffffu : 0u) | (at + 1 >= lo && at + 1 <= hi ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int cp = 0; cp < KP; ++cp) {
              uint32_t b[2 * NB];
              columns(cp, b);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                float part[4] = {0.f, 0.f, 0.f, 0.f};
                mma<BF>(part, pf[ks], b[nb * 2] & mask[0], b[nb * 2 + 1] & mask[1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (ri[e >> 1] == i) o[cp * NB + nb][e] += part[e];
              }
            }
          }
        }
      }
    }

    fresh = flags & LAST;
    if (fresh) {
      // ---- the warps' shares of the positions are joined through this stage's shared memory: first
      // their rows' maxima and sums, then their outputs, SETS times 8 rows by JC columns at a time
      const int n = t.n, hk = t.hk, unit_row0 = t.row0;
      float2* rd = red + odd * (16 * KW);
      odd ^= 1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = l[h];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (tq == 0) rd[(h * 8 + g) * KW + kw] = make_float2(m[h], x);
      }
      if (!sync()) return;  // and no warp reads this stage's keys and values any more
      const bool whole_unit = (flags & OPENS) && (flags & CLOSES);
      const long long slot = 2LL * c + ((flags & OPENS) ? 1 : 0);
      float* buf = reinterpret_cast<float*>(aligned + stage * S::STAGE_BYTES);  // [warp][SETS * 8 rows][JC]
      constexpr int SETS = S::SETS, JC = S::JC, PART = SETS * 8 * JC;
      float mul[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float big = -INFINITY;
#pragma unroll
        for (int y = 0; y < KW; ++y) big = fmaxf(big, rd[(h * 8 + g) * KW + y].x);
        mul[h] = m[h] == -INFINITY ? 0.f : exp2_fast(m[h] - big);
      }
#pragma unroll
      for (int pass = 0; pass < 2 / SETS * (D / JC); ++pass) {
        const int s0 = pass / (D / JC) * SETS, c0 = pass % (D / JC) * JC;
        if (unit_row0 + s0 * 8 >= s.rows) break;  // the first row group's rows: the same for all warps
        if (pass && !sync()) return;
#pragma unroll
        for (int h = s0; h < s0 + SETS; ++h) {
          // a row's groups of 8 columns are XORed with the row, against bank conflicts
          float* to = buf + warp * PART + ((h - s0) * 8 + g) * JC;
          const int flip = (g << 3) & (JC - 1);
#pragma unroll
          for (int cg = 0; cg < JC / 16; ++cg) {
            // 16 columns: two n-tiles, side by side, or (8-bit) the even and the odd columns
            const int nt = c0 / 8 + cg * 2;
            if (E8) {
              *reinterpret_cast<float4*>(to + ((cg * 16 + tq * 4) ^ flip)) =
                  make_float4(o[nt][h * 2] * mul[h], o[nt + 1][h * 2] * mul[h], o[nt][h * 2 + 1] * mul[h], o[nt + 1][h * 2 + 1] * mul[h]);
            } else {
              *reinterpret_cast<float2*>(to + ((cg * 16 + tq * 2) ^ flip)) = make_float2(o[nt][h * 2] * mul[h], o[nt][h * 2 + 1] * mul[h]);
              *reinterpret_cast<float2*>(to + ((cg * 16 + 8 + tq * 2) ^ flip)) = make_float2(o[nt + 1][h * 2] * mul[h], o[nt + 1][h * 2 + 1] * mul[h]);
            }
          }
        }
        if (!sync()) return;
        for (int x = tid; x < PART / 4; x += 32 * KW) {
          const int jr = x / (JC / 4), jc = x % (JC / 4) * 4;
          const int orow = s0 * 8 + jr, gr = unit_row0 + orow;
          if (gr >= s.rows) break;
          float big = -INFINITY, sum = 0.f;
#pragma unroll
          for (int y = 0; y < KW; ++y) big = fmaxf(big, rd[orow * KW + y].x);
#pragma unroll
          for (int y = 0; y < KW; ++y) {
            const float2 ml = rd[orow * KW + y];
            sum += ml.x == -INFINITY ? ml.y : ml.y * exp2_fast(ml.x - big);  // (without a maximum: 0, or NaN)
          }
          const float* from = buf + jr * JC + (jc ^ (((jr & 7) << 3) & (JC - 1)));
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int y = 0; y < KW; ++y) {
            const float4 z = *reinterpret_cast<const float4*>(from + y * PART);
            v.x += z.x, v.y += z.y, v.z += z.z, v.w += z.w;
          }
          bool none = big == -INFINITY && sum == 0.f;
          const int i = gr / s.group_heads, gh = gr - i * s.group_heads;
          if (none && sees_any(s, n, i, flags & OPENS ? 0 : t.pos0 - it * TILE, t.pos0 + TILE)) none = false, big = LOWEST;
          if (whole_unit) {
            const long long at = ((long long)n * p.K + i) * p.H_q + hk * s.group_heads + gh;
            const float by = p.cache.v_scale / sum;
            uint2 w = make_uint2(pack2<A>(v.x * by, v.y * by), pack2<A>(v.z * by, v.w * by));
            if (none) w = make_uint2(0u, 0u);
            *reinterpret_cast<uint2*>(static_cast<A*>(p.out) + at * D + c0 + jc) = w;
            if (p.lse && c0 + jc == 0) p.lse[at] = none ? -INFINITY : (big + log2f(sum)) * 0.69314718055994530942f;
          } else {
            *reinterpret_cast<float4*>(s.part_o + (slot * S::ROWS + orow) * D + c0 + jc) = v;
            if (c0 + jc == 0) s.part_ml[slot * S::ROWS + orow] = make_float2(big, sum);
          }
        }
      }
      fence_proxy_async_smem();  // this stage's next bytes come by TMA
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[stage]);
    if (flags & STOP) break;
    if (++stage == STAGES) stage = 0, turn ^= 1;
  }
}

// Joins the parts of the units that several CTAs worked on: for one row,
// M = max m_p, out = sum 2^(m_p - M) o_p / sum 2^(m_p - M) l_p.
template <typename A, int D, int THREADS>
__global__ void __launch_bounds__(THREADS) join_kernel(const __grid_constant__ Params s) {
  constexpr int LANES = D / 4, GROUPS = THREADS / LANES;
  __shared__ float4 s_o[GROUPS][LANES];
  __shared__ float2 s_ml[GROUPS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const AttendProblem& p = s.p;
  const Record rec = s.records[blockIdx.x];
  if (rec.more == 0) return;
  const int row = blockIdx.y, tid = threadIdx.x;
  const int heads = p.cache.H_kv * s.groups;
  const int n = rec.unit / heads, sub = rec.unit - n * heads, hk = sub / s.groups;
  const int gr = (sub - hk * s.groups) * s.rows_per + row;
  if (gr >= s.rows) return;
  const int parts = rec.more + 1;
  // Each of GROUPS thread groups joins every GROUPS-th part with its own running maximum, then the
  // groups are joined: a part's maximum and its output are loaded side by side.
  const int col = tid % LANES, grp = tid / LANES;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float top = -INFINITY, sum = 0.f;
#pragma unroll 4
  for (int x = grp; x < parts; x += GROUPS) {
    const long long slot = (x == 0 ? 2LL * rec.first + 1 : 2LL * (rec.first + x * s.team)) * s.rows_per + row;
    const float2 ml = s.part_ml[slot];
    const float4 y = *reinterpret_cast<const float4*>(s.part_o + slot * D + col * 4);
    if (ml.x == -INFINITY && ml.y == 0.f) continue;  // nothing seen in this part
    const float mn = fmaxf(top, ml.x);
    const float keep = exp2_fast(top - mn), w = exp2_fast(ml.x - mn);
    o.x = o.x * keep + w * y.x;
    o.y = o.y * keep + w * y.y;
    o.z = o.z * keep + w * y.z;
    o.w = o.w * keep + w * y.w;
    sum = sum * keep + w * ml.y;
    top = mn;
  }
  s_o[grp][col] = o;
  if (col == 0) s_ml[grp] = make_float2(top, sum);
  __syncthreads();
  if (grp != 0) return;
  for (int x = 1; x < GROUPS; ++x) {
    const float2 ml = s_ml[x];
    const float4 y = s_o[x][col];
    if (ml.x == -INFINITY && ml.y == 0.f) continue;
    const float mn = fmaxf(top, ml.x);
    const float keep = exp2_fast(top - mn), w = exp2_fast(ml.x - mn);
    o.x = o.x * keep + w * y.x;
    o.y = o.y * keep + w * y.y;
    o.z = o.z * keep + w * y.z;
    o.w = o.w * keep + w * y.w;
    sum = sum * keep + w * ml.y;
    top = mn;
  }
  const int i = gr / s.group_heads, gh = gr - i * s.group_heads;
  const long long at = ((long long)n * p.K + i) * p.H_q + hk * s.group_heads + gh;
  const bool none = top == -INFINITY && sum == 0.f;
  const float mul = p.cache.v_scale / sum;
  uint2 y = make_uint2(pack2<A>(o.x * mul, o.y * mul), pack2<A>(o.z * mul, o.w * mul));
  if (none) y = make_uint2(0u, 0u);
  *reinterpret_cast<uint2*>(static_cast<A*>(p.out) + at * D + col * 4) = y;
  if (p.lse && col == 0) p.lse[at] = none ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
}

// ---------------------------------------------------------------- host

struct Plan {
  int rows, per, groups, grid, team;  // query rows of a key head, in groups of at most per
  bool wide, whole, by_unit;
  long long units;
  size_t ml_at, o_at, bytes;
};

// The launch for a bound of max_len positions (0: no work).
Plan plan_for(int n_seq, int K, int H_q, int H_kv, int d, int max_len) {
  constexpr int TILE = 64;  // the smallest
  Plan a{};
  a.rows = K * (H_q / H_kv);
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess) return a;
  // at most 48 rows to a unit; more are split evenly (their units run side by side, in one team).  Few
  // and short ones are sooner done 16 rows at a time, by two CTAs on an SM (40 rows on each of 4 key
  // heads of 128): one request of 250 positions 10.9 us against 11.6, 500 positions 11.5 against 14.1,
  // 8-bit 11.2 against 13.6 and 13.1 against 16.0; but 64 requests of 250, 26.5 against 19.2.
  const int by16 = (a.rows + 15) / 16;
  const int most = max_len <= 512 && (long long)n_seq * H_kv * by16 <= 2 * sms ? 16 : 48;
  a.groups = (a.rows + most - 1) / most;
  a.per = ((a.rows + a.groups - 1) / a.groups + 15) / 16 * 16;
  a.units = (long long)n_seq * H_kv * a.groups;
  const long long unit_tiles = ((long long)max_len + TILE - 1) / TILE;
  const long long tiles = a.units * (unit_tiles > 1 ? unit_tiles : 1);
  // 64 requests of 8192 positions, 4 key heads of 128, on tcgen05 against the warp-level products with as
  // many row groups as it takes: 16-bit, 32 rows 175 us against 218, 40 rows 180 against 347; 8-bit, 32
  // rows 113 against 167, 40 rows 139 against 277.
  a.wide = a.per > 16;
  const int resident = (a.per > 16 ? 1 : 2) * sms;
  // Short units are read faster by one CTA than they are joined, the more so where there are enough of
  // them for all CTAs (8 key heads of 128; whole units against parts): 250 positions, 1 request 9.0
  // against 10.5 us; 500, 1 request 12.2 against 10.3, 16 requests 12.8 against 14.4, 64 requests 29.2
  // against 32.5; 1000, 16 requests 18.8 against 17.1, 64 requests 49.1 against 51.7.
  a.whole = max_len <= 256 || (max_len <= 512 && 4 * a.units >= resident) || (max_len <= 1024 && a.units >= resident);
  const long long want = a.whole ? a.units : tiles;
  // Where a token's heads lie side by side, CTAs that read them at the same time read DRAM in longer
  // runs: teams of up to 8 heads.
  a.team = 1;
  while (a.team < 8 && H_kv * a.groups % (2 * a.team) == 0 && resident % (2 * a.team) == 0) a.team *= 2;
  a.grid = (int)(want < resident ? want : resident) / a.team * a.team;
  a.by_unit = a.units <= a.grid;
  if (!a.whole) {
    a.ml_at = ((size_t)a.grid * sizeof(Record) + 255) / 256 * 256;
    a.o_at = a.ml_at + (size_t)2 * a.grid * a.per * sizeof(float2);
    a.bytes = a.o_at + (size_t)2 * a.grid * a.per * d * sizeof(float);
  }
  return a;
}

bool make_map(CUtensorMap* map, const kda_paged_cache_t& c, const void* base, bool token_first, int box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const int es = c.dtype == KDA_E4M3 ? 1 : 2;
  const cuuint32_t inner = c.d * es < 128 ? c.d : 128 / es;
  const cuuint64_t tok = (cuuint64_t)c.page_size, head = (cuuint64_t)c.H_kv;
  const cuuint64_t ts = c.token_stride * es, hs = c.head_stride * es;
  cuuint64_t dims[4] = {(cuuint64_t)c.d, token_first ? tok : head, token_first ? head : tok, (cuuint64_t)c.num_pages};
  cuuint64_t strides[3] = {token_first ? ts : hs, token_first ? hs : ts, (cuuint64_t)c.page_stride * es};
  cuuint32_t box[4] = {inner, token_first ? (cuuint32_t)box_rows : 1u, token_first ? 1u : (cuuint32_t)box_rows, 1u};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            c.d * es < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the second kernel, where units may be in parts
template <typename A, int D>
cudaError_t launch_join(const Plan& a, const Params& s, cudaStream_t stream) {
  if (a.whole) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.by_unit ? (unsigned)a.units : (unsigned)a.grid, (unsigned)(s.rows < a.per ? s.rows : a.per));
  // units in 32 or more parts on average: more threads, which read more parts at a time
  const bool many = a.grid >= 32 * a.units;
  cfg.blockDim = dim3(many ? 512 : 128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, join_kernel<A, D, 512>, s) : cudaLaunchKernelEx(&cfg, join_kernel<A, D, 128>, s);
}

template <typename A, bool E8, int D>
cudaError_t launch_shape(const Plan& a, const Params& s, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  using S = Shape<D, E8>;
  auto kernel = attend_kernel<A, E8, D>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
  if (e != cudaSuccess) return e;
  kernel<<<a.grid, S::THREADS, S::SMEM, stream>>>(mk, mv, s);
  return cudaGetLastError();
}

template <typename A, int D>
cudaError_t launch_both(const Plan& a, const Params& s, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  const cudaError_t e = a.wide                             ? launch_attend_wide(s, mk, mv, a.grid, stream)
                        : s.p.cache.dtype == KDA_E4M3 ? launch_shape<A, true, D>(a, s, mk, mv, stream)
                                                      : launch_shape<A, false, D>(a, s, mk, mv, stream);
  return e == cudaSuccess ? launch_join<A, D>(a, s, stream) : e;
}

template <typename A>
cudaError_t launch_typed(const Plan& a, const Params& s, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t stream) {
  return s.p.cache.d == 128 ? launch_both<A, 128>(a, s, mk, mv, stream) : launch_both<A, 64>(a, s, mk, mv, stream);
}

}  // namespace

bool attend_tiles_fit(int n_seq, int K, int H_q, int H_kv, int capacity) {
  const long long groups = ((long long)K * (H_q / H_kv) + 15) / 16;
  return (capacity / 64 + 2LL) * n_seq * H_kv * groups < (1LL << 31);
}

size_t attend_workspace_bytes(int n_seq, int K, int H_q, int H_kv, int d, int max_len) {
  return plan_for(n_seq, K, H_q, H_kv, d, max_len).bytes;
}

cudaError_t launch_cache_attend(const AttendProblem& p, void* workspace, cudaStream_t stream) {
  const kda_paged_cache_t& c = p.cache;
  const Plan a = plan_for(c.n_seq, p.K, p.H_q, c.H_kv, c.d, p.max_len);
  if (a.grid <= 0) return cudaErrorInvalidDevice;
  Params s{};
  s.p = p;
  s.groups = a.groups;
  s.rows = a.rows;
  s.group_heads = p.H_q / c.H_kv;
  s.rows_per = a.per;
  s.whole = a.whole;
  s.by_unit = a.by_unit;
  s.min_tiles = 2;
  s.team = a.team;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  s.records = reinterpret_cast<Record*>(ws);
  s.part_ml = reinterpret_cast<float2*>(ws + a.ml_at);
  s.part_o = reinterpret_cast<float*>(ws + a.o_at);
  // rows of a tile that lie in one page: the greatest power of two that divides the page size
  s.box_rows = 64;
  while (c.page_size % s.box_rows) s.box_rows >>= 1;
  s.token_first = c.token_stride <= c.head_stride;
  CUtensorMap mk{}, mv{};
  // a box starts on 128 bytes of shared memory
  s.use_tma = s.box_rows * c.d * (c.dtype == KDA_E4M3 ? 1 : 2) >= 128;
  if (s.use_tma && c.num_pages > 0) {
    if (!make_map(&mk, c, c.k, s.token_first, s.box_rows) || !make_map(&mv, c, c.v, s.token_first, s.box_rows))
      return cudaErrorInvalidValue;
  }
  return p.dtype == KDA_BF16 ? launch_typed<__nv_bfloat16>(a, s, mk, mv, stream)
                             : launch_typed<__half>(a, s, mk, mv, stream);
}

}  // namespace kda
