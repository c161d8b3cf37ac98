// The chunked walk of the linear attention's state, on the tcgen05 tensor cores.
//
// A chunk is 128 tokens.  With g the running sum of log2 of the decays in it,
// G = g at its end and S the state that enters it,
//
//     O  = scale (2^{g_i} Q S + P V),   P_ij = (q_i . k_j) 2^{g_i - g_j} for j <= i
//     S <- 2^G S + K^T V',              v'_j = 2^{G - g_j} v_j
//
// Four products of 128 x 128 x d, with tokens (or the state's rows) on the 128
// lanes: Q, K and V as TMA lays them (keys as rows and, read transposed, as
// columns), P from tensor memory, where it takes the place of the scores, the
// state in tensor memory in fp32 and, as an operand, in shared memory.
// Differences of g are never positive, so no exponential overflows whatever
// the decays are.  V' is two bf16 numbers (16 bits), since the state that the
// caller gets is fp32; so are, for fp32 outputs, P and the operand S.
//
// A sequence is cut into segments of seg_len tokens where there are fewer
// (sequence, head) pairs than SMs.  ENDS finds each segment's contribution to
// the state at its end, linear_scan_kernel joins them into the states at the
// segments' starts, and OUTPUTS walks every segment from there.  ENDS goes
// through a segment backwards with weights that reach to the segment's end, so
// the sum stays where it is in tensor memory.
//
// BACK runs against time, for gradients: the state is the gradient that
// arrives, K the queries, V the outputs' gradients, v'_i = scale 2^{g_i} v_i.
// IMAGES leaves each chunk's entering state in memory, as the bf16 operand
// image that the gradient kernel copies into its shared memory.
//
// Warps: 0-7 compute (two to each quarter of the lanes; each has half of the
// columns), 8 loads, 9 issues.  They meet at mbarriers only, with bounded
// waits.  Shared memory holds seven tiles: V' and the operand S (whose place
// the lower half of V' takes when its product is done), and five for the
// inputs, which follow one another into whichever tile is free first.  One CTA
// on an SM.
#pragma once

#include "kda_linear.cuh"
#include "tma_host.h"
#include "umma.cuh"

namespace kda {
namespace linear {

constexpr int CHUNK = 128;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LEAST = -104.f;  // its exponential is 0 in fp32

enum Mode { ENDS, OUTPUTS, IMAGES };

struct Walk {
  LinearProblem p;
  int seg_len, segs, slots;  // tokens to a segment; segments to a sequence (fixed lengths), and of all sequences
  float* carry;              // [slots][H][d][d]: ENDS writes contributions, the other modes read states
  float* decay;              // [slots][H]: log2 of each segment's decay
  uint8_t* images;           // IMAGES: [chunks][H][d x d bf16]
};

// What slot w holds: the sequence, its rows, and which of them.  n < 0: nothing.
struct Segment {
  int n, len, tokens, index, count;  // len: rows of the sequence, tokens: of the segment
  long long row0;                    // of the sequence
};

// Sequence n of a packed call has slots row0 / seg_len + n and on, enough for its length; a warp looks for
// the one that holds slot w.  (Offsets that overlap may give a slot twice; then the first sequence has it.)
__device__ __forceinline__ Segment find_segment(const LinearProblem& p, int seg_len, int segs, int w) {
  Segment s{-1, 0, 0, 0, 0, 0};
  if (!p.cu_seqlens) {
    s.n = w / segs;
    s.index = w % segs;
    s.len = p.len;
    s.row0 = (long long)s.n * p.len;
  } else {
    const int lane = threadIdx.x & 31;
    for (int n0 = 0; n0 < p.n_seq; n0 += 32) {
      const int n = n0 + lane;
      long long row0 = 0;
      int len = 0, first = 0;
      if (n < p.n_seq) {
        len = sequence_rows(p, n, &row0);
        first = (int)(row0 / seg_len) + n;
      }
      const unsigned has = __ballot_sync(~0u, n < p.n_seq && w >= first && w < first + max((len + seg_len - 1) / seg_len, 1));
      if (has) {
        const int from = __ffs(has) - 1;
        s.n = n0 + from;
        s.len = __shfl_sync(~0u, len, from);
        s.index = w - __shfl_sync(~0u, first, from);
        s.row0 = __shfl_sync(~0u, row0, from);
        break;
      }
    }
  }
  s.count = max((s.len + seg_len - 1) / seg_len, 1);
  if (s.n >= 0 && s.index >= s.count) s.n = -1;
  s.tokens = min(seg_len, s.len - s.index * seg_len);
  return s;
}

// The chunks of sequence n come one after the other from here on (packed: with at most one left out).
__device__ __forceinline__ long long first_chunk(const LinearProblem& p, const Segment& s) {
  return p.cu_seqlens ? s.row0 / CHUNK + s.n : (long long)s.n * ((p.len + CHUNK - 1) / CHUNK);
}
inline long long most_chunks(int n_seq, int T, bool packed) {
  return packed ? (long long)T / CHUNK + n_seq : (long long)n_seq * ((T / n_seq + CHUNK - 1) / CHUNK);
}

template <int D> struct Shape {
  static constexpr uint32_t TILE = CHUNK * D * 2, BLOCK = CHUNK * 128;  // a tile of tokens; 64 channels of it
  static constexpr uint32_t IMAGE = D * D * 2, IMAGE_BLOCK = D * 128;   // the state as an operand
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void lds_v4(uint32_t at, uint32_t (&u)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ float lds_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float lo_f32(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f32(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// x as two bf16 numbers, two x to a word; what the first leaves is exact.
__device__ __forceinline__ uint32_t split_bf16x2(float a, float b, uint32_t* rest) {
  const uint32_t u = pack_bf16x2(a, b);
  *rest = pack_bf16x2(a - lo_f32(u), b - hi_f32(u));
  return u;
}
__device__ __forceinline__ void tmem_st16u(uint32_t at, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
      "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
      "r"(v[14]), "r"(v[15]) : "memory");
}

// Descriptors of 128-byte-swizzled operands: rows along K (a tile's channels), or rows along the other
// dimension (a tile's tokens as K), `block` bytes between its blocks of 64 columns.
__device__ __forceinline__ uint64_t desc_k(uint32_t at) { return make_sdesc(at, 16u, 1024u, SW_128); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t at, uint32_t block) { return make_sdesc(at, block, 1024u, SW_128); }

// log2 of the decays of a chunk's tokens, summed up to each: lane l of the warp has tokens 4 l .. 4 l + 3.
struct Decays {
  float raw[4];  // log_alpha of the next chunk
  __device__ __forceinline__ void load(const LinearProblem& p, long long row, int rows, int h) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = 4 * lane + i < rows ? load_decay(p, row + 4 * lane + i, h) : 0.f;
  }
  __device__ __forceinline__ float4 sum() const {
    const int lane = threadIdx.x & 31;
    float g[4], run = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = raw[i] < LEAST ? LEAST : raw[i];  // (a NaN stays)
      run += x * LOG2E;
      g[i] = run;
    }
    float before = run;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const float x = __shfl_up_sync(~0u, before, o);
      if (lane >= o) before += x;
    }
    before = __shfl_up_sync(~0u, before, 1);
    if (lane == 0) before = 0.f;
    return make_float4(g[0] + before, g[1] + before, g[2] + before, g[3] + before);
  }
};

template <int D, Mode MODE, bool BACK, bool FINE> struct WalkShape : Shape<D> {
  using Shape<D>::TILE;
  static constexpr int IN = MODE == OUTPUTS ? 5 : 4;  // input tiles
  static constexpr uint32_t X = IN * TILE, Y = X + TILE, MISC = Y + TILE, SMEM_USED = MISC + 3072;
  // one CTA on an SM: each takes all of tensor memory
  static constexpr uint32_t SMEM = SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024;
  static constexpr uint32_t T_A = 0, T_O1 = 128, T_O2 = 128 + D, T_S = 128 + 2 * D;
};

constexpr int WALK_THREADS = 320;

// FINE: fp32 outputs, P and S as two bf16 numbers each.
template <int D, Mode MODE, bool BACK, bool FINE>
__global__ void __launch_bounds__(WALK_THREADS, 1)
    linear_walk_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, Walk w) {
  using W = WalkShape<D, MODE, BACK, FINE>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const LinearProblem& p = w.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t sb = smem_u32(smem);
  const int slot = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const Segment seg = find_segment(p, w.seg_len, w.segs, slot);
  if (seg.n < 0) return;
  if (sb & 1023u) {  // the tiles' swizzle goes by address
    if (tid == 0) atomicExch(p.status, (int)KDA_ERR_ALIGNMENT);
    return;
  }
  const bool last_seg = BACK ? seg.index == 0 : seg.index == seg.count - 1;  // in the order of the walk
  const bool first_seg = BACK ? seg.index == seg.count - 1 : seg.index == 0;
  if (MODE == ENDS && last_seg) return;  // what it would find nobody asks for
  const int nch = max((seg.tokens + CHUNK - 1) / CHUNK, 0);
  constexpr bool UP = MODE == ENDS ? BACK : !BACK;  // from the segment's first chunk to its last
  const long long row0 = seg.row0 + (long long)seg.index * w.seg_len;
  auto chunk_of = [&](int c) { return UP ? c : nch - 1 - c; };
  auto rows_of = [&](int ci) { return min(CHUNK, seg.tokens - ci * CHUNK); };

  float* s_g = reinterpret_cast<float*>(smem + W::MISC);              // [2][128]
  int* s_first = reinterpret_cast<int*>(smem + W::MISC + 1024);       // [3][128]: the first token of a channel that is not finite
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + W::MISC + 2560);  // [5] an input tile has landed
  uint64_t *s_ready = full + 5, *v_ready = full + 6, *p_ready = full + 7, *l_ready = full + 8, *f_ready = full + 9;
  uint64_t *a_done = full + 10, *qs_done = full + 11, *pv_done = full + 12, *kv_done = full + 13, *f_done = full + 14;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(full + 15);
  int* s_bad = reinterpret_cast<int*>(full + 16);                     // [3] some value of the chunk is not finite

  if (tid == 0) {
    for (int i = 0; i < 5; ++i) mbar_init(full + i, 1);
    for (uint64_t* b : {s_ready, v_ready, p_ready, l_ready, f_ready}) mbar_init(b, 8);
    for (uint64_t* b : {a_done, qs_done, pv_done, kv_done, f_done}) mbar_init(b, 1);
    mbar_fence_init();
    for (int i = 0; i < 3; ++i) s_bad[i] = 0;
  }
  for (int i = tid; i < 3 * 128; i += WALK_THREADS) s_first[i] = 0x7fffffff;
  if (warp == 0) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tb = *s_tmem;
  bool ok = true;

  // The tiles of a chunk's inputs.  Where there are queries: those of the next chunk's keys and queries are
  // already on their way; its values take the queries' place, and the chunk after it those of the values
  // and the keys.  `phase` has a bit for each tile.
  struct Tiles {
    int k = 0, q = 1, v = 2, k2 = 3, q2 = 4;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int c) {
      if constexpr (MODE == OUTPUTS) {
        phase ^= 1u << k | 1u << q | 1u << v;
        const int k0 = k, q0 = q, v0 = v;
        k = k2;
        q = q2;
        v = q0;
        k2 = v0;
        q2 = k0;
      } else {
        phase ^= 1u << k | 1u << v;
        k = (c + 1) & 1;
        v = 2 + ((c + 1) & 1);
      }
    }
  };

  if (warp == 8) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      auto load = [&](const CUtensorMap* map, int tile, int c) {
        const int row = (int)(row0 + chunk_of(c) * CHUNK);
        mbar_arrive_expect_tx(full + tile, W::TILE);
        for (int b = 0; b < D / 64; ++b)
          tma_load_3d(smem + tile * W::TILE + b * W::BLOCK, map, full + tile, 64 * b, h, row);
      };
      Tiles t;
      uint32_t loads = 0, landed = 0;  // parity of each tile's number of loads
      if constexpr (MODE != OUTPUTS) { t.q = 0; t.v = 2; }
      for (int c = -2; c < nch && ok; ++c) {
        // before chunk 0: what the first two chunks find on their way
        if constexpr (MODE == OUTPUTS) {
          if (c == -2) {
            if (nch > 0) { load(&map_k, 0, 0); load(&map_q, 1, 0); load(&map_v, 2, 0); loads ^= 7; }
          } else if (c == -1) {
            if (nch > 1) { load(&map_k, 3, 1); load(&map_q, 4, 1); loads ^= 24; }
          } else {
            const uint32_t par = c & 1;
            if (c + 1 < nch) {
              ok = mbar_wait(FINE ? f_done : qs_done, par);
              if (ok) { load(&map_v, t.q, c + 1); loads ^= 1u << t.q; }
            }
            if (ok && c + 2 < nch) {
              ok = mbar_wait(pv_done, par);
              if (ok) { load(&map_k, t.v, c + 2); loads ^= 1u << t.v; }
              ok = ok && mbar_wait(kv_done, par);
              if (ok) { load(&map_q, t.k, c + 2); loads ^= 1u << t.k; }
            }
            t.next(c);
          }
        } else {
          if (c >= 0 && c + 2 < nch) ok = mbar_wait(kv_done, c & 1);
          if (ok && c + 2 < nch) {
            load(&map_k, c & 1, c + 2);
            load(&map_v, 2 + (c & 1), c + 2);
            loads ^= 5u << (c & 1);
          }
        }
      }
      (void)landed;
      // no copy is in flight when the CTA ends: the last one into each tile has landed
      for (int i = 0; i < W::IN; ++i) {
        const uint32_t odd = loads >> i & 1;  // loads so far are odd: phases 0, 1, .. the last is even
        const bool any = MODE == OUTPUTS ? nch > (i < 3 ? 0 : 1) : nch > (i & 1);
        if (any) ok = mbar_wait(full + i, odd ^ 1) && ok;
      }
      if (!ok) atomicExch(p.status, (int)KDA_ERR_TIMEOUT);
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- products
    if (lane == 0) {
      constexpr uint32_t ID_A = make_idesc_bf16(128, 128, false, false), ID_O = make_idesc_bf16(128, D, false, true),
                         ID_S = make_idesc_bf16(D, D, true, true);
      Tiles t;
      if constexpr (MODE != OUTPUTS) t.v = 2;
      auto state_update = [&](uint32_t k_at, uint32_t v_at, bool add) {
        const uint64_t a = desc_mn(k_at, W::BLOCK), b = desc_mn(v_at, W::BLOCK);
#pragma unroll
        for (int i = 0; i < 128; i += 16)
          umma_bf16(tb + W::T_S, desc_adv(a, i, true), desc_adv(b, i, true), ID_S, add || i ? 1u : 0u);
      };
      auto from_state = [&](uint32_t q_at, bool add) {
        const uint64_t a = desc_k(q_at), b = desc_mn(sb + W::Y, W::IMAGE_BLOCK);
#pragma unroll
        for (int i = 0; i < D; i += 16)
          umma_bf16(tb + W::T_O1, desc_adv(a, i, false, W::BLOCK), desc_adv(b, i, true), ID_O, add || i ? 1u : 0u);
      };
      for (int c = 0; c < nch && ok; ++c) {
        const uint32_t par = c & 1;
        const uint32_t k_at = sb + t.k * W::TILE, v_at = sb + t.v * W::TILE, q_at = sb + t.q * W::TILE;
        ok = mbar_wait(full + t.k, t.phase >> t.k & 1);
        if constexpr (MODE == OUTPUTS) {
          ok = ok && mbar_wait(full + t.q, t.phase >> t.q & 1);
          if (!ok) break;
          const uint64_t a = desc_k(q_at), b = desc_k(k_at);
#pragma unroll
          for (int i = 0; i < D; i += 16)
            umma_bf16(tb + W::T_A, desc_adv(a, i, false, W::BLOCK), desc_adv(b, i, false, W::BLOCK), ID_A, i ? 1u : 0u);
          umma_commit(a_done);
          if (!(ok = mbar_wait(s_ready, par))) break;
          tc_fence_after_sync();
          from_state(q_at, false);
          umma_commit(qs_done);
          if (FINE) {
            if (!(ok = mbar_wait(f_ready, par))) break;
            tc_fence_after_sync();
            from_state(q_at, true);
            umma_commit(f_done);
          }
        }
        if (!ok || !(ok = mbar_wait(v_ready, par))) break;
        tc_fence_after_sync();
        state_update(k_at, sb + W::X, MODE != ENDS || c > 0);
        if constexpr (MODE == OUTPUTS) {
          if (!(ok = mbar_wait(p_ready, par))) break;
          tc_fence_after_sync();
          const uint64_t b = desc_mn(v_at, W::BLOCK);
#pragma unroll
          for (int x = 0; x <= (FINE ? 1 : 0); ++x)
#pragma unroll
            for (int i = 0; i < 128; i += 16)
              umma_f16_ta(tb + W::T_O2, tb + W::T_A + (i >= 64 ? 64 : 0) + (i % 64) / 2 + 32 * x, desc_adv(b, i, true), ID_O,
                          x || i ? 1u : 0u);
          umma_commit(pv_done);
          if (!(ok = mbar_wait(l_ready, par))) break;
          tc_fence_after_sync();
        }
        state_update(k_at, sb + W::Y, true);
        umma_commit(kv_done);
        t.next(c);
      }
      if (!ok) {  // what has been issued ends before the CTA does
        atomicExch(p.status, (int)KDA_ERR_TIMEOUT);
        umma_commit(kv_done);
        umma_commit(kv_done);
        (void)mbar_wait(kv_done, 0);
        (void)mbar_wait(kv_done, 1);
      }
    }
  } else {
    // ---------------------------------------------------------------- weights, states, outputs
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t my = tb + ((uint32_t)(32 * quarter) << 16);
    // the state: a lane has one of its rows, a warp half of its columns
    const int srow = D == 128 ? 32 * quarter + lane : 16 * quarter + (lane & 15);
    const bool has_srow = D == 128 || lane < 16;
    constexpr int SC = D / 2;
    const size_t state_at = ((size_t)seg.n * p.H + h) * D * D + (size_t)srow * D + half * SC;
    const size_t carry_at = ((size_t)slot * p.H + h) * D * D + (size_t)srow * D + half * SC;
    const int trow = tid & 127;  // this thread's token where V' is formed, and of P and O
    const uint32_t sw = (uint32_t)(trow & 7);
    const float gain = BACK ? p.scale : 1.f;
    Tiles t;
    if constexpr (MODE != OUTPUTS) t.v = 2;
    Decays la;
    float reach = 0.f;  // ENDS: log2 of the decay from the chunk to the segment's end (start)
    if (nch > 0) la.load(p, row0 + chunk_of(0) * CHUNK, rows_of(chunk_of(0)), h);
    int c = 0;
    for (; c < nch && ok; ++c) {
      const uint32_t par = c & 1;
      const int ci = chunk_of(c), rows = rows_of(ci);
      const long long row = row0 + (long long)ci * CHUNK;
      const uint32_t v_at = sb + t.v * W::TILE, k_at = sb + t.k * W::TILE;
      // every warp sums the decays for itself; all write the same numbers
      float* g = s_g + par * 128;
      const float4 g4 = la.sum();
      *reinterpret_cast<float4*>(g + 4 * lane) = g4;
      const float end = __shfl_sync(~0u, g4.w, 31);
      if (c + 1 < nch) la.load(p, row0 + chunk_of(c + 1) * CHUNK, rows_of(chunk_of(c + 1)), h);
      __syncwarp();
      const float g_mine = g[trow];
      if (MODE == OUTPUTS) {
        if (tid < 128) s_first[(c + 1) % 3 * 128 + tid] = 0x7fffffff;
        if (tid == 0) s_bad[(c + 1) % 3] = 0;
      }

      // ---- the state as an operand, and what is left of it after the chunk
      if (c > 0) {
        if (!(ok = mbar_wait(kv_done, par ^ 1))) break;
        tc_fence_after_sync();
      }
      uint32_t s_rest[FINE ? SC / 2 : 1];
      if constexpr (MODE != ENDS) {
        const float keep = ex2(end);
        const float* from = !first_seg ? w.carry + carry_at : p.s_in ? p.s_in + state_at : nullptr;
#pragma unroll
        for (int b = 0; b < SC; b += 32) {
          float s[2][16];
          if (c > 0) {
            tmem_ld16(my + W::T_S + half * SC + b, s[0]);
            tmem_ld16(my + W::T_S + half * SC + b + 16, s[1]);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 x = from && has_srow ? *reinterpret_cast<const float4*>(from + b + i) : make_float4(0.f, 0.f, 0.f, 0.f);
              s[i / 16][i % 16] = x.x;
              s[i / 16][i % 16 + 1] = x.y;
              s[i / 16][i % 16 + 2] = x.z;
              s[i / 16][i % 16 + 3] = x.w;
            }
          }
          uint32_t u[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = s[i / 8][2 * i % 16], y = s[i / 8][2 * i % 16 + 1];
            if constexpr (FINE) u[i] = split_bf16x2(x, y, &s_rest[b / 2 + i]);
            else u[i] = pack_bf16x2(x, y);
          }
          const int col = half * SC + b;
          const uint32_t line = (uint32_t)(col / 64) * W::IMAGE_BLOCK + (uint32_t)srow * 128;
          if (has_srow) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t at = line + ((((uint32_t)(col % 64) / 8 + i) ^ (uint32_t)(srow & 7)) << 4);
              if constexpr (MODE == OUTPUTS) {
                st_shared_v4(sb + W::Y + at, u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
              } else {
                uint8_t* to = w.images + ((first_chunk(p, seg) + (row - seg.row0) / CHUNK) * p.H + h) * W::IMAGE;
                *reinterpret_cast<uint4*>(to + at) = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i / 16][i % 16] *= keep;
          tmem_st16(my + W::T_S + half * SC + b, s[0]);
          tmem_st16(my + W::T_S + half * SC + b + 16, s[1]);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        if constexpr (MODE == OUTPUTS) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_ready);
        }
      }

      // ---- the weighted values
      if (!(ok = mbar_wait(full + t.v, t.phase >> t.v & 1))) break;
      const bool tail = rows < CHUNK;
      if (tail && !(ok = mbar_wait(full + t.k, t.phase >> t.k & 1))) break;
      constexpr int PIECES = D == 128 ? 8 : 4;  // of 16 bytes, to a thread
      uint32_t v_rest[4 * PIECES];
      {
        const bool real = trow < rows;
        const float weight = gain * ex2(MODE == ENDS ? reach + (BACK ? g_mine : end - g_mine) : BACK ? g_mine : end - g_mine);
        const uint32_t block = D == 128 ? half * W::BLOCK : 0;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          const uint32_t at = block + trow * 128 + (((uint32_t)(D == 128 ? i : 4 * half + i) ^ sw) << 4);
          uint32_t u[4], o[4];
          lds_v4(v_at + at, u);
          if (MODE == OUTPUTS && real) {
            bool odd = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) odd |= (u[j] & 0x7f80u) == 0x7f80u || (u[j] & 0x7f800000u) == 0x7f800000u;
            if (odd) {  // such a value is taken out of the product with the weights, where zeros would meet it
              uint32_t z[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                z[j] = u[j];
                const int ch = half * (D / 2) + 8 * i + 2 * j;
                if ((u[j] & 0x7f80u) == 0x7f80u) {
                  z[j] &= 0xffff0000u;
                  atomicMin(s_first + c % 3 * 128 + ch, trow);
                }
                if ((u[j] & 0x7f800000u) == 0x7f800000u) {
                  z[j] &= 0xffffu;
                  atomicMin(s_first + c % 3 * 128 + ch + 1, trow);
                }
              }
              st_shared_v4(v_at + at, z[0], z[1], z[2], z[3]);
              s_bad[c % 3] = 1;
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = real ? split_bf16x2(lo_f32(u[j]) * weight, hi_f32(u[j]) * weight, &v_rest[4 * i + j]) : (v_rest[4 * i + j] = 0u);
          st_shared_v4(sb + W::X + at, o[0], o[1], o[2], o[3]);
          if constexpr (MODE != OUTPUTS)
            st_shared_v4(sb + W::Y + at, v_rest[4 * i], v_rest[4 * i + 1], v_rest[4 * i + 2], v_rest[4 * i + 3]);
          if (tail && !real) {  // rows of other sequences
            st_shared_v4(v_at + at, 0u, 0u, 0u, 0u);
            st_shared_v4(k_at + at, 0u, 0u, 0u, 0u);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_ready);
      if constexpr (MODE == ENDS) reach += end;

      if constexpr (MODE == OUTPUTS) {
        // ---- the weights, in place of the scores
        if (!(ok = mbar_wait(a_done, par))) break;
        tc_fence_after_sync();
        uint32_t u[32], rest[32];
#pragma unroll
        for (int b = 0; b < 64; b += 16) {
          const int j0 = 64 * half + b;
          if (j0 <= 32 * quarter + 31) {
            float a[16];
            tmem_ld16(my + W::T_A + j0, a);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 gj = *reinterpret_cast<const float4*>(g + j0 + j);
              a[j] = j0 + j <= trow ? a[j] * p.scale * ex2(g_mine - gj.x) : 0.f;
              a[j + 1] = j0 + j + 1 <= trow ? a[j + 1] * p.scale * ex2(g_mine - gj.y) : 0.f;
              a[j + 2] = j0 + j + 2 <= trow ? a[j + 2] * p.scale * ex2(g_mine - gj.z) : 0.f;
              a[j + 3] = j0 + j + 3 <= trow ? a[j + 3] * p.scale * ex2(g_mine - gj.w) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) u[b / 2 + j] = split_bf16x2(a[2 * j], a[2 * j + 1], &rest[b / 2 + j]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) u[b / 2 + j] = rest[b / 2 + j] = 0u;
          }
        }
        // (a half's pieces lie where its own scores were, all of which it has read)
        tmem_st16u(my + W::T_A + 64 * half, u);
        tmem_st16u(my + W::T_A + 64 * half + 16, u + 16);
        if (FINE) {
          tmem_st16u(my + W::T_A + 64 * half + 32, rest);
          tmem_st16u(my + W::T_A + 64 * half + 48, rest + 16);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);

        // ---- what the operands' first numbers left takes the state's place
        if (!(ok = mbar_wait(qs_done, par))) break;
        if constexpr (FINE) {
#pragma unroll
          for (int i = 0; i < SC / 8; ++i) {
            const int col = half * SC + 8 * i;
            if (has_srow)
              st_shared_v4(sb + W::Y + (uint32_t)(col / 64) * W::IMAGE_BLOCK + (uint32_t)srow * 128 +
                               ((((uint32_t)(col % 64) / 8) ^ (uint32_t)(srow & 7)) << 4),
                           s_rest[4 * i], s_rest[4 * i + 1], s_rest[4 * i + 2], s_rest[4 * i + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(f_ready);
          if (!(ok = mbar_wait(f_done, par))) break;
        }
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          const uint32_t at = (D == 128 ? half * W::BLOCK : 0) + trow * 128 + (((uint32_t)(D == 128 ? i : 4 * half + i) ^ sw) << 4);
          st_shared_v4(sb + W::Y + at, v_rest[4 * i], v_rest[4 * i + 1], v_rest[4 * i + 2], v_rest[4 * i + 3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(l_ready);

        // ---- the outputs
        if (!(ok = mbar_wait(pv_done, par))) break;
        tc_fence_after_sync();
        const float lead = p.scale * ex2(g_mine);
        const bool bad = s_bad[c % 3] != 0;
        const size_t out_at = ((size_t)(row + trow) * p.H + h) * D + half * SC;
#pragma unroll
        for (int b = 0; b < SC; b += 16) {
          float x[16], y[16];
          tmem_ld16(my + W::T_O1 + half * SC + b, x);
          tmem_ld16(my + W::T_O2 + half * SC + b, y);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] += lead * x[i];
          if (bad) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (s_first[c % 3 * 128 + half * SC + b + i] <= trow) y[i] = NAN;
          }
          if (trow < rows) {
            if constexpr (FINE) {
              float* to = static_cast<float*>(p.out) + out_at + b;
#pragma unroll
              for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            } else {
              __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + out_at + b;
#pragma unroll
              for (int i = 0; i < 16; i += 8)
                *reinterpret_cast<uint4*>(to + i) = make_uint4(pack_bf16x2(y[i], y[i + 1]), pack_bf16x2(y[i + 2], y[i + 3]),
                                                               pack_bf16x2(y[i + 4], y[i + 5]), pack_bf16x2(y[i + 6], y[i + 7]));
            }
          }
        }
        tc_fence_before_sync();
      }
      t.next(c);
    }
    // ---- the state behind the segment
    if (ok && nch > 0) ok = mbar_wait(kv_done, (nch - 1) & 1);
    if (!ok) {
      if (lane == 0) atomicExch(p.status, (int)KDA_ERR_TIMEOUT);
    } else if (MODE == ENDS || (last_seg && p.s_out)) {
      tc_fence_after_sync();
      float* to = MODE == ENDS ? w.carry + carry_at : p.s_out + state_at;
      if (nch > 0) {
#pragma unroll
        for (int b = 0; b < SC; b += 16) {
          float s[16];
          tmem_ld16(my + W::T_S + half * SC + b, s);
          tmem_ld_wait();
          if (has_srow) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4*>(to + b + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
          }
        }
      } else if (has_srow) {  // an empty sequence
        for (int i = 0; i < SC; i += 4)
          *reinterpret_cast<float4*>(to + i) = p.s_in ? *reinterpret_cast<const float4*>(p.s_in + state_at + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (MODE == ENDS && tid == 0) w.decay[(size_t)slot * p.H + h] = reach;
    }
    tc_fence_before_sync();
  }
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tb, 512);
}

// The states at the segments' starts (BACK: the gradients at their ends) from the segments' contributions,
// which they replace: E = 2^decay E + Z, one after the other, 1024 entries of a state to a CTA.
template <bool BACK> __global__ void __launch_bounds__(256) linear_scan_kernel(Walk w) {
  const LinearProblem& p = w.p;
  const int parts = p.d * p.d / 1024;
  const int part = blockIdx.x % parts, nh = blockIdx.x / parts, n = nh / p.H, h = nh % p.H;
  long long row0 = (long long)n * p.len;
  int len = p.len;
  if (p.cu_seqlens) len = sequence_rows(p, n, &row0);
  const int count = max((len + w.seg_len - 1) / w.seg_len, 1);
  const long long first = p.cu_seqlens ? row0 / w.seg_len + n : (long long)n * w.segs;
  const size_t at = (size_t)part * 1024 + threadIdx.x * 4, size = (size_t)p.d * p.d;
  float4 e = p.s_in ? *reinterpret_cast<const float4*>(p.s_in + (size_t)nh * size + at) : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < count; ++i) {
    const size_t slot = (size_t)(first + (BACK ? count - 1 - i : i)) * p.H + h;
    float4* here = reinterpret_cast<float4*>(w.carry + slot * size + at);
    if (i + 1 < count) {
      const float4 z = *here;
      const float keep = ex2(w.decay[slot]);
      *here = e;
      e = make_float4(keep * e.x + z.x, keep * e.y + z.y, keep * e.z + z.z, keep * e.w + z.w);
    } else {
      *here = e;
    }
  }
}

// ---------------------------------------------------------------- host

inline bool make_rows_map(CUtensorMap* map, const void* base, long long stride, const LinearProblem& p) {
  return make_map_3d_bf16(map, base, (uint64_t)p.d, (uint64_t)p.H, (uint64_t)p.T, (uint64_t)p.d, (uint64_t)stride, 64, 1, CHUNK,
                          CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, Mode MODE, bool BACK, bool FINE>
cudaError_t launch_walk(const Walk& w, const void* k, long long k_stride, const void* v, long long v_stride, cudaStream_t stream) {
  using W = WalkShape<D, MODE, BACK, FINE>;
  CUtensorMap mq, mk, mv;
  const LinearProblem& p = w.p;
  if (p.T > 0 && (!make_rows_map(&mk, k, k_stride, p) || !make_rows_map(&mv, v, v_stride, p) ||
                  !make_rows_map(&mq, MODE == OUTPUTS ? p.q : k, MODE == OUTPUTS ? p.q_stride : k_stride, p)))
    return cudaErrorInvalidValue;
  auto kernel = linear_walk_kernel<D, MODE, BACK, FINE>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)W::SMEM);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)((long long)w.slots * p.H), WALK_THREADS, W::SMEM, stream>>>(mq, mk, mv, w);
  return cudaGetLastError();
}

template <bool BACK> cudaError_t launch_scan(const Walk& w, cudaStream_t stream) {
  const LinearProblem& p = w.p;
  linear_scan_kernel<BACK><<<(unsigned)((long long)p.n_seq * p.H * (p.d * p.d / 1024)), 256, 0, stream>>>(w);
  return cudaGetLastError();
}

// Tokens to a segment: whole chunks, such that the walk (and, where it is cut, the half as long one before
// it) takes the fewest steps of the machine.  Cut in more than one, a segment has at least 4 chunks.
inline int segment_tokens(int n_seq, int T, int H, bool packed, int sms) {
  const long long len = packed ? T : T / n_seq, chunks = std::max((len + CHUNK - 1) / CHUNK, 1LL);
  long long best = chunks, best_cost = -1;
  for (long long segs = 1; segs <= 256 && segs * 4 <= std::max(chunks, 4LL); ++segs) {
    const long long of = (chunks + segs - 1) / segs;
    const long long items = (packed ? chunks / of + n_seq : n_seq * ((chunks + of - 1) / of)) * H;
    const long long cost = (items + sms - 1) / sms * of * (segs > 1 ? 3 : 2);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = of;
    }
  }
  return (int)(best * CHUNK);
}
inline int segment_slots(int n_seq, int T, int seg_len, bool packed) {
  return packed ? T / seg_len + n_seq : n_seq * std::max((T / n_seq + seg_len - 1) / seg_len, 1);
}

}  // namespace linear
}  // namespace kda
