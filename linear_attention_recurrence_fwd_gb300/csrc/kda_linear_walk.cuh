// The chunked walk of the linear attention's state, on the tcgen05 tensor cores.
//
// A chunk is 128 tokens.  With g the running sum of log2 of the decays in it,
// G = g at its end and S the state that enters it,
//
//     O  = scale (2^{g_i} Q S + P V),   P_ij = (q_i . k_j) 2^{g_i - g_j} for j <= i
//     S <- 2^G S + K^T V',              v'_j = 2^{G - g_j} v_j
//
// Products of 128 x 128 x d, with tokens (or the state's rows) on the 128
// lanes: Q, K and V as TMA lays them (keys as rows and, read transposed, as
// columns), P from tensor memory, where it takes the place of the scores.  The
// state stays in registers in fp32: K^T V' comes to it from tensor memory, and
// a bf16 copy goes to shared memory as an operand, so nothing but four warps'
// arithmetic joins one chunk to the next.  Differences of g are never
// positive, so no exponential overflows whatever the decays are.
//
// V' is two bf16 numbers (16 bits) where the state is a result (what the
// caller gets, segments' ends, all of a call with fp32 outputs) and one where
// only bf16 outputs see it; for fp32 outputs so are P and the operand S.
//
// A sequence is cut into segments of seg_len tokens where that takes the
// machine fewer steps (segment_tokens).  How long packed sequences are only the
// device knows, so such a call goes the cut way as soon as it has rows for a
// segment: where no sequence is longer than one, ENDS does nothing and the scan
// copies states.  ENDS finds each segment's contribution to the state at its end, linear_scan_kernel joins them into the states at the
// segments' starts, and OUTPUTS walks every segment from there.  ENDS goes
// through a segment backwards with weights that reach to the segment's end, so
// the sum stays where it is in tensor memory.
//
// BACK runs against time, for gradients: the state is the gradient that
// arrives, K the queries, V the outputs' gradients, v'_i = scale 2^{g_i} v_i.
// IMAGES leaves each chunk's entering state in memory, as the bf16 operand
// image that the gradient kernel copies into its shared memory.
//
// Warps: 0-3 keep the state, 4-11 turn scores into weights, 12-19 form V',
// 20-27 write the outputs, 28 loads, 29 issues, 30 sums up the decays (a token's lie a row apart: 32 sectors to a load, too many
// for every warp to read them by itself, which held up all others).  They meet
// at mbarriers only, with bounded waits.  Shared memory holds seven tiles: V',
// the operand S, and five for the inputs, which follow one another into
// whichever tile is free first; outputs pass through the values' tile, so that
// they leave in whole lines.  One CTA on an SM.
//
// Measured (32 heads of 128): 8192 tokens 98 us (floor 40; ENDS 31, scan 5, OUTPUTS 66; with fp32 outputs 133, floor 50:
// the weights' warps spill second numbers), 65536 packed ones 593 us (floor 318; 196, 21, 378), of which the keys and
// values come twice: 3.2 GB in all, 5.4 TB/s.  OUTPUTS at 8192 tokens:
// DRAM 48 %, tensor pipe 23 %, issue slots 30 %: what bounds it is the chain of a chunk, from the values to the state
// and on to its operand, with 128 of 152 SMs at work.  A product of 128 x 128 x 128 takes 937 clocks with A's channels
// along K, 561 with its tokens, 602 from tensor memory.  Code size matters most: loops that unrolled to 94 KB took 831
// us for the packed tokens where rolled ones of 56 KB took 619.
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
  float* decay;              // [slots][H]: log2 of each segment's decay; null where no sequence is cut
  uint8_t* images;           // IMAGES: [chunks][H][d x d bf16]
};

// What slot w holds: the sequence, its rows, and which of them.  n < 0: nothing.
struct Segment {
  int n, len, tokens, index, count;  // len: rows of the sequence, tokens: of the segment
  long long row0;                    // of the sequence
};

// Sequence n of a packed call has slots row0 / seg_len + n and on, enough for its length; a warp looks for
// the one that holds slot w, 32 sequences at a time from the first on, so that a CTA's start takes longer the more there
// are (65536 rows of 32 heads: 4 sequences 0.62 ms, 512 of them, a chunk each, 3.45).  (Offsets that overlap may give a
// slot twice; then the first sequence has it.)
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
__device__ __forceinline__ float lo_f32(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f32(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// x as two bf16 numbers, two x to a word; what the first leaves is exact.
__device__ __forceinline__ uint32_t split_bf16x2(float a, float b, uint32_t* rest) {
  const uint32_t u = pack_bf16x2(a, b);
  *rest = pack_bf16x2(a - lo_f32(u), b - hi_f32(u));
  return u;
}
__device__ __forceinline__ void tmem_ld8(uint32_t at, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(at));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st4u(uint32_t at, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ void tmem_st8u(uint32_t at, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t at, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
      "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
      "r"(v[14]), "r"(v[15]) : "memory");
}

__device__ __forceinline__ __nv_bfloat162 as_bf16x2(uint32_t u) {
  __nv_bfloat162 v;
  memcpy(&v, &u, 4);
  return v;
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) {
  uint32_t u;
  memcpy(&u, &v, 4);
  return u;
}

// Waits for a phase; a try waits a while by itself (a microsecond or so), so this ends after a second or a few.
// Short, as everything in the walk's loops: their instructions come around once a chunk, and what does not stay
// in the instruction cache takes longer to fetch than to run.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 1 << 20; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}

// Descriptors of 128-byte-swizzled operands: rows along K (a tile's channels), or rows along the other
// dimension (a tile's tokens as K), `block` bytes between its blocks of 64 columns.
__device__ __forceinline__ uint64_t desc_k(uint32_t at) { return make_sdesc(at, 16u, 1024u, SW_128); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t at, uint32_t block) { return make_sdesc(at, block, 1024u, SW_128); }

// log2 of the decays of a chunk's tokens, summed up to each: lane l of the warp has tokens 4 l .. 4 l + 3.
struct Decays {
  uint32_t raw[4];  // log_alpha of the next chunk
  __device__ __forceinline__ void load(const LinearProblem& p, long long row, int rows, int h) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = 4 * lane + i < rows ? load_decay_bits(p, row + 4 * lane + i, h) : 0u;
  }
  __device__ __forceinline__ float4 sum(const LinearProblem& p) const {
    const int lane = threadIdx.x & 31;
    float g[4], run = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = decay_of_bits(p, raw[i]);
      run += (x < LEAST ? LEAST : x) * LOG2E;  // (a NaN stays)
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

// A launch may start while the one before it in its stream runs, up to the point where it needs what that one
// leaves: every launch lets the next one start at once, and none ends without having waited.
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Where a warp turns its rows of a state, 32 columns at a time, between memory, where 8 lanes take a row's 128
// bytes, and registers, where a lane has its own row.
__device__ __forceinline__ uint32_t turned(uint32_t region, int row, int piece) {
  return region + row * 128 + ((uint32_t)(piece ^ (row & 7)) << 4);
}

template <int D, Mode MODE, bool BACK, bool FINE> struct WalkShape : Shape<D> {
  using Shape<D>::TILE;
  static constexpr int IN = MODE == OUTPUTS ? 5 : 4;  // input tiles
  static constexpr uint32_t X = IN * TILE, Y = X + TILE, LEAVING = Y + TILE, MISC = LEAVING + (MODE == IMAGES ? TILE : 0), SMEM_USED = MISC + 3 * 1024;
  // one CTA on an SM: each takes all of tensor memory
  static constexpr uint32_t SMEM = SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024;
  // scores and weights; what the state gives; what the weights give; the chunk's part of the state
  static constexpr uint32_t T_A = 0, T_O1 = 128, T_O2 = 128 + D, T_Z = 128 + 2 * D;
};

constexpr int WALK_THREADS = 1024;
// The launch's registers, split anew by warpgroup (in every mode: one group waits for what others give back).
constexpr int LAUNCH_REGS = 64, STATE_REGS = 152, WEIGHT_REGS = 56, VALUE_REGS = 48, OUTPUT_REGS = 56, OTHER_REGS = 40;
static_assert(4 * STATE_REGS + 8 * (WEIGHT_REGS + VALUE_REGS + OUTPUT_REGS) + 4 * OTHER_REGS <= 32 * LAUNCH_REGS, "registers");

// The input tiles are a ring that keys, queries and values (keys and values) go through in this order, chunk
// after chunk: so a chunk's values take the place of the keys of the one before, which are free first, and the
// next keys and queries that of its queries and values.
template <Mode MODE> struct Ring {
  static constexpr int KINDS = MODE == OUTPUTS ? 3 : 2, TILES = MODE == OUTPUTS ? 5 : 4;
  int tile = 0;        // of a chunk's keys
  uint32_t turn = 0;   // how often the ring has been gone through, odd or even
  __device__ __forceinline__ int at(int kind) const { return tile + kind < TILES ? tile + kind : tile + kind - TILES; }
  __device__ __forceinline__ uint32_t phase(int kind) const { return turn ^ (tile + kind >= TILES ? 1u : 0u); }
  __device__ __forceinline__ void move(int kinds) {
    tile += kinds;
    if (tile >= TILES) {
      tile -= TILES;
      turn ^= 1;
    }
  }
};

// FINE: fp32 outputs, P and S as two bf16 numbers each.
template <int D, Mode MODE, bool BACK, bool FINE>
__device__ __forceinline__ void walk(const CUtensorMap& map_q, const CUtensorMap& map_k, const CUtensorMap& map_v, const Walk& w) {
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
  if (MODE == ENDS && last_seg) return;  // what it would find nobody asks for
  const bool exact = MODE != OUTPUTS || FINE || (last_seg && p.s_out);  // V' as two numbers
  const int nch = max((seg.tokens + CHUNK - 1) / CHUNK, 0);
  constexpr bool UP = MODE == ENDS ? BACK : !BACK;  // from the segment's first chunk to its last
  const int row0 = (int)(seg.row0 + (long long)seg.index * w.seg_len);
  auto chunk_of = [&](int c) { return UP ? c : nch - 1 - c; };
  auto rows_of = [&](int ci) { return min(CHUNK, seg.tokens - ci * CHUNK); };

  float* s_g = reinterpret_cast<float*>(smem + W::MISC);              // [2][128]: -g
  int* s_first = reinterpret_cast<int*>(smem + W::MISC + 1024);       // [3][128]: the first token of a channel that is not finite
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + W::MISC + 2560);  // [5] an input tile has landed
  uint64_t *s_ready = full + 5, *v_ready = full + 6, *p_ready = full + 7, *l_ready = full + 8, *f_ready = full + 9;
  uint64_t *z_free = full + 10, *o_read = full + 11, *a_done = full + 12, *pv_done = full + 13, *zh_done = full + 14;
  // for odd and even chunks: a wait tells a phase from the next one, not from the one after that, and
  // those who wait for these may be a chunk behind
  uint64_t *qs_done = full + 15, *z_done = full + 17, *f_done = full + 19, *o_done = full + 21, *g_ready = full + 23, *g_free = full + 25,
           *n_ready = full + 27;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(full + 29);
  int* s_bad = reinterpret_cast<int*>(full + 30);                     // [3] some value of the chunk is not finite

  if (tid == 0) {
    for (int i = 0; i < 5; ++i) mbar_init(full + i, 1);
    mbar_init(s_ready, 4);
    mbar_init(v_ready, 8);
    mbar_init(l_ready, 8);
    mbar_init(p_ready, 8);
    mbar_init(f_ready, 4);
    mbar_init(z_free, 4);
    mbar_init(o_read, 8);
    mbar_init(a_done, 1);
    mbar_init(pv_done, 1);
    mbar_init(zh_done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(qs_done + i, 1);
      mbar_init(z_done + i, 1);
      mbar_init(f_done + i, 1);
      mbar_init(o_done + i, 8);
      mbar_init(g_ready + i, 1);
      mbar_init(n_ready + i, 8);
      mbar_init(g_free + i, MODE == ENDS ? 8 : MODE == IMAGES ? 12 : 28);
    }
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
  const int quarter = warp & 3;
  const uint32_t my = tb + ((uint32_t)(32 * quarter) << 16);
  bool ok = true;

  if (warp < 4) {
    // ---------------------------------------------------------------- the state: a lane has one of its rows
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(STATE_REGS));
    if constexpr (MODE != ENDS) {
      const int srow = D == 128 ? 32 * quarter + lane : 16 * quarter + (lane & 15);
      const bool has_row = D == 128 || lane < 16;
      constexpr int ROWS = D / 4;  // of a warp
      const size_t warp_rows = (size_t)quarter * ROWS * D, state_at = ((size_t)seg.n * p.H + h) * D * D + warp_rows;
      uint64_t s[D / 2];  // two columns each
      // turned where this warp's part of the operand (of the leaving image) lies
      const uint32_t region = sb + (MODE == IMAGES ? W::LEAVING : W::Y) + quarter * ROWS * 128;
      dependency_wait();  // the joined states
      {
        // (a call that is cut takes all of them from there: where the caller's states are one buffer, a CTA may
        // have written its own before another has started)
        const float* from = w.decay ? w.carry + ((size_t)slot * p.H + h) * D * D + warp_rows : p.s_in ? p.s_in + state_at : nullptr;
        // all of its loads are on their way together
        float4 raw[D / 32][ROWS / 4];
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
          for (int i = 0; i < ROWS / 4; ++i)
            raw[b][i] = from ? *reinterpret_cast<const float4*>(from + (4 * i + lane / 8) * D + 32 * b + 4 * (lane % 8)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < ROWS / 4; ++i)
            st_shared_v4(turned(region, 4 * i + lane / 8, lane % 8), __float_as_uint(raw[b][i].x), __float_as_uint(raw[b][i].y),
                         __float_as_uint(raw[b][i].z), __float_as_uint(raw[b][i].w));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t u[4];
            lds_v4(turned(region, lane & (ROWS - 1), i), u);
            s[16 * b + 2 * i] = pair(__uint_as_float(u[0]), __uint_as_float(u[1]));
            s[16 * b + 2 * i + 1] = pair(__uint_as_float(u[2]), __uint_as_float(u[3]));
          }
        }
      }
      // eight columns to their place in the operand, as the first (second) of their two numbers
      auto place = [&](int i, bool second, auto to) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x, y;
          unpair(s[4 * i + j], &x, &y);
          u[j] = pack_bf16x2(x, y);
          if (second) u[j] = pack_bf16x2(x - lo_f32(u[j]), y - hi_f32(u[j]));
        }
        to((uint32_t)(i / 8) * W::IMAGE_BLOCK + (uint32_t)srow * 128 + (((uint32_t)(i % 8) ^ (uint32_t)(srow & 7)) << 4), u);
      };
      auto to_tile = [&](uint32_t at, const uint32_t (&u)[4]) {
        if (has_row) st_shared_v4(sb + W::Y + at, u[0], u[1], u[2], u[3]);
      };
      for (int c = 0; c < nch && ok; ++c) {
        const uint32_t par = c & 1;
        if (!(ok = wait_for(g_ready + par, c >> 1 & 1))) break;
        const float keep = ex2(-s_g[par * 128 + 127]);
        __syncwarp();
        if (lane == 0) mbar_arrive(g_free + par);
        if constexpr (MODE == OUTPUTS) {
          if (c > 0 && !(ok = wait_for((FINE ? f_done : qs_done) + (par ^ 1), c - 1 >> 1 & 1))) break;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) place(i, false, to_tile);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_ready);
          if constexpr (FINE) {
            if (!(ok = wait_for(qs_done + par, c >> 1 & 1))) break;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) place(i, true, to_tile);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(f_ready);
          }
        } else {
          // the image leaves by way of shared memory, each warp's rows by themselves
          if (lane == 0) bulk_wait_reads();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            place(i, false, [&](uint32_t at, const uint32_t (&u)[4]) {
              if (has_row) st_shared_v4(sb + W::LEAVING + at, u[0], u[1], u[2], u[3]);
            });
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            constexpr uint32_t ROWS = D / 4 * 128;  // bytes of a warp's rows in a block
            uint8_t* image = w.images + ((first_chunk(p, seg) + seg.index * (w.seg_len / CHUNK) + chunk_of(c)) * p.H + h) * W::IMAGE;
            for (uint32_t at = quarter * ROWS; at < W::IMAGE; at += W::IMAGE_BLOCK) bulk_s2g(image + at, sb + W::LEAVING + at, ROWS);
            bulk_commit();
          }
        }
        if (!(ok = wait_for(z_done + par, c >> 1 & 1))) break;
        tc_fence_after_sync();
#pragma unroll
        for (int b = 0; b < D; b += 16) {
          float z[16];
          tmem_ld16(my + W::T_Z + b, z);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; i += 2) s[(b + i) / 2] = fma2(s[(b + i) / 2], pair(keep, keep), pair(z[i], z[i + 1]));
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(z_free);
      }
      if (MODE == IMAGES && lane == 0) bulk_wait_all();
      if (ok && last_seg && p.s_out) {
        // (the operand's tile: its last product is done, or waited for here)
        if (MODE == OUTPUTS && nch > 0) ok = wait_for((FINE ? f_done : qs_done) + ((nch - 1) & 1), nch - 1 >> 1 & 1);
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float4 x;
            unpair(s[16 * b + 2 * i], &x.x, &x.y);
            unpair(s[16 * b + 2 * i + 1], &x.z, &x.w);
            if (has_row)
              st_shared_v4(turned(region, lane, i), __float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z), __float_as_uint(x.w));
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < ROWS / 4; ++i) {
            const int r = 4 * i + lane / 8;
            uint32_t u[4];
            lds_v4(turned(region, r, lane % 8), u);
            if (ok) *reinterpret_cast<uint4*>(p.s_out + state_at + r * D + 32 * b + 4 * (lane % 8)) = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
      }
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(WEIGHT_REGS));
    if constexpr (MODE == OUTPUTS) {
      const int half = warp >> 2 & 1, trow = 32 * quarter + lane;
      for (int c = 0; c < nch && ok; ++c) {
        // -------------------------------------------------------------- the weights, in place of the scores
        const uint32_t par = c & 1;
        const float* minus_g = s_g + par * 128;
        if (!(ok = wait_for(g_ready + par, c >> 1 & 1))) break;
        const float g_mine = -minus_g[trow];
        if (!(ok = wait_for(a_done, par))) break;
        tc_fence_after_sync();
        // 16 columns at a time; a piece's place is that of scores already read (FINE: its second numbers', 32
        // columns on, is not, so they wait)
        const uint32_t at = my + W::T_A + 64 * half;
        uint32_t held[FINE ? 32 : 1];
#pragma unroll(FINE ? 4 : 1)
        for (int b = 0; b < 4; ++b) {
          const int j0 = 64 * half + 16 * b;
          uint32_t u[8], rest[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = rest[j] = 0u;
          if (j0 <= 32 * quarter + 31) {
            float x[16];
            tmem_ld16(at + 16 * b, x);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const uint64_t to = add2(pair(g_mine, g_mine), *reinterpret_cast<const uint64_t*>(minus_g + j0 + j));
              float y, z;
              unpair(to, &y, &z);
              unpair(mul2(pair(x[j], x[j + 1]), pair(ex2(y), ex2(z))), &x[j], &x[j + 1]);
            }
            if (j0 + 15 > 32 * quarter) {  // what comes after some of the warp's tokens
#pragma unroll
              for (int j = 0; j < 16; ++j) x[j] = j0 + j <= trow ? x[j] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if constexpr (FINE) u[j] = split_bf16x2(x[2 * j], x[2 * j + 1], &rest[j]);
              else u[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
            }
          }
          tmem_st8u(at + 8 * b, u);
          if constexpr (FINE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) held[8 * b + j] = rest[j];
          }
        }
        if constexpr (FINE) {
          tmem_st16u(at + 32, held);
          tmem_st16u(at + 48, held + 16);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(p_ready);
          mbar_arrive(g_free + par);
        }
      }
    }
  } else if (warp < 20) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(VALUE_REGS));
    // a thread has a token and half of its channels
    const int half = warp >> 2 & 1, trow = 32 * quarter + lane;
    constexpr int PIECES = D / 16;  // of 16 bytes, to a thread
    auto piece = [&](int i) {
      const int x = half * PIECES + i;
      return (uint32_t)(x / 8) * W::BLOCK + trow * 128 + (((uint32_t)(x % 8) ^ (uint32_t)(trow & 7)) << 4);
    };
    float reach = 0.f;  // ENDS: log2 of the decay from the chunk to the segment's end (start)
    Ring<MODE> t;
    constexpr int VALUES = MODE == OUTPUTS ? 2 : 1;

    // ---------------------------------------------------------------- the weighted values
    // The weight is two bf16 numbers, w1 + w2: the first number of v w is v w1 rounded, what that leaves of
    // v w1 is exact, and v w2 is added to it (16 bits together).
    auto values = [&](int c) {
      const uint32_t par = c & 1;
      const int rows = rows_of(chunk_of(c));
      const uint32_t v_at = sb + t.at(VALUES) * W::TILE, k_at = sb + t.tile * W::TILE;
      if (!wait_for(g_ready + par, c >> 1 & 1)) return false;
      const float g_mine = -s_g[par * 128 + trow], end = -s_g[par * 128 + 127];
      if (MODE == OUTPUTS) {
        if (c > 1 && !wait_for(o_done + par, (c >> 1 & 1) ^ 1)) return false;
        if (half == 0) s_first[(c + 1) % 3 * 128 + trow] = 0x7fffffff;
        if (half == 0 && trow == 0) s_bad[(c + 1) % 3] = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(g_free + par);
      const bool real = trow < rows;
      const float gain = BACK ? p.scale : 1.f;
      const float weight = gain * ex2(MODE == ENDS ? reach + (BACK ? g_mine : end - g_mine) : BACK ? g_mine : end - g_mine);
      const __nv_bfloat162 w1 = __float2bfloat162_rn(weight), w2 = __float2bfloat162_rn(weight - __low2float(w1));
      const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
      if constexpr (MODE == ENDS) reach += end;
      if (!wait_for(full + t.at(VALUES), t.phase(VALUES))) return false;
      if (rows < CHUNK && !wait_for(full + t.tile, t.turn)) return false;
      if (c > 0 && !wait_for(z_done + (par ^ 1), c - 1 >> 1 & 1)) return false;
      // (what comes before the first products goes without anything that they do not wait for)
#pragma unroll 1
      for (int i = 0; i < PIECES; i += 4) {
        uint32_t u[4][4];
#pragma unroll
        for (int z = 0; z < 4; ++z) lds_v4(v_at + piece(i + z), u[z]);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          uint32_t y[4], rest[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 x = as_bf16x2(u[z][j]), first = __hmul2_rn(x, w1);
            y[j] = as_u32(first);
            if constexpr (MODE != OUTPUTS) rest[j] = as_u32(__hfma2(x, w2, __hfma2(x, w1, __hneg2(first))));
          }
          st_shared_v4(sb + W::X + piece(i + z), y[0], y[1], y[2], y[3]);
          if constexpr (MODE != OUTPUTS) st_shared_v4(sb + W::Y + piece(i + z), rest[0], rest[1], rest[2], rest[3]);
        }
      }
      if (!real) {  // rows of other sequences
#pragma unroll 1
        for (int i = 0; i < PIECES; ++i) {
          st_shared_v4(sb + W::X + piece(i), 0u, 0u, 0u, 0u);
          if (MODE != OUTPUTS) st_shared_v4(sb + W::Y + piece(i), 0u, 0u, 0u, 0u);
          st_shared_v4(v_at + piece(i), 0u, 0u, 0u, 0u);
          st_shared_v4(k_at + piece(i), 0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_ready);
      if constexpr (MODE == OUTPUTS) {
        // a value that is not finite is taken out of the product with the weights, where zeros would meet it
        __nv_bfloat162 odd = zero;
#pragma unroll 1
        for (int i = 0; i < PIECES; i += 4) {
          uint32_t u[4][4];
#pragma unroll
          for (int z = 0; z < 4; ++z) lds_v4(v_at + piece(i + z), u[z]);
#pragma unroll
          for (int j = 0; j < 16; ++j) odd = __hfma2(as_bf16x2(u[j / 4][j % 4]), zero, odd);  // NaN if one of them is not finite
        }
        if (!__hbeq2(odd, zero)) {
#pragma unroll 1
          for (int i = 0; i < PIECES; ++i) {
            uint32_t u[4];
            lds_v4(v_at + piece(i), u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int ch = 8 * (half * PIECES + i) + 2 * j;
              if ((u[j] & 0x7f80u) == 0x7f80u) {
                u[j] &= 0xffff0000u;
                atomicMin(s_first + c % 3 * 128 + ch, trow);
              }
              if ((u[j] & 0x7f800000u) == 0x7f800000u) {
                u[j] &= 0xffffu;
                atomicMin(s_first + c % 3 * 128 + ch + 1, trow);
              }
            }
            st_shared_v4(v_at + piece(i), u[0], u[1], u[2], u[3]);
          }
          s_bad[c % 3] = 1;
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(n_ready + par);
        if (exact) {  // the second numbers take the place of the first ones
          if (!wait_for(zh_done, par)) return false;
#pragma unroll 1
          for (int i = 0; i < PIECES; i += 4) {
            uint32_t u[4][4];
#pragma unroll
            for (int z = 0; z < 4; ++z) lds_v4(v_at + piece(i + z), u[z]);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 x = as_bf16x2(u[z][j]);
                u[z][j] = as_u32(__hfma2(x, w2, __hfma2(x, w1, __hneg2(__hmul2_rn(x, w1)))));
              }
              st_shared_v4(sb + W::X + piece(i + z), u[z][0], u[z][1], u[z][2], u[z][3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(l_ready);
        }
      }
      t.move(Ring<MODE>::KINDS);
      return true;
    };

    {
#pragma unroll 1
      for (int c = 0; c < nch && ok; ++c) ok = values(c);
      if constexpr (MODE == ENDS) {  // the segment's contribution
        if (ok && nch > 0) ok = wait_for(z_done + ((nch - 1) & 1), nch - 1 >> 1 & 1);
        if (ok) {
          tc_fence_after_sync();
          // (through the tiles of V', whose products are done)
          const uint32_t region = sb + W::X + (half * 4 + quarter) * (64 * D);
          float* to = w.carry + ((size_t)slot * p.H + h) * D * D + (size_t)quarter * (D / 4) * D + half * (D / 2);
          constexpr int ROW = D * 2;  // bytes of half a row
#pragma unroll 1
          for (int b = 0; b < D / 2; b += 16) {
            float s[16];
            tmem_ld16(my + W::T_Z + half * (D / 2) + b, s);
            tmem_ld_wait();
            if (D == 128 || lane < 16) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                st_shared_v4(region + lane * ROW + ((uint32_t)((b / 4 + i) ^ (lane & (ROW / 16 - 1))) << 4), __float_as_uint(s[4 * i]),
                             __float_as_uint(s[4 * i + 1]), __float_as_uint(s[4 * i + 2]), __float_as_uint(s[4 * i + 3]));
            }
          }
          __syncwarp();
          constexpr int LANES = ROW / 16;  // to a row
#pragma unroll 4
          for (int i = 0; i < D / 4 * LANES / 32; ++i) {
            const int r = i * (32 / LANES) + lane / LANES, x = lane % LANES;
            uint32_t u[4];
            lds_v4(region + r * ROW + ((uint32_t)(x ^ (r & (LANES - 1))) << 4), u);
            *reinterpret_cast<uint4*>(to + (size_t)r * D + 4 * x) = make_uint4(u[0], u[1], u[2], u[3]);
          }
          if (half == 0 && trow == 0) w.decay[(size_t)slot * p.H + h] = reach;
        }
      }
    }
  } else if (warp < 28) {
    // ---------------------------------------------------------------- the outputs: 32 rows and 128 bytes
    // (d = 64: 64) of each at a time, turned in this warp's part of the values' tile so that 8 lanes write a
    // row's piece
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OUTPUT_REGS));
    if constexpr (MODE == OUTPUTS) {
      constexpr int SC = D / 2, ES = FINE ? 4 : 2, TURN = W::TILE / 256 / ES, LANES = W::TILE / 256 / 16;  // columns; lanes to a row's piece
      const int half = warp >> 2 & 1, trow = 32 * quarter + lane;
      const size_t row_bytes = (size_t)p.H * D * ES;
      Ring<MODE> t;
      for (int c = 0; c < nch && ok; ++c) {
        const uint32_t par = c & 1;
        const int rows = rows_of(chunk_of(c));
        const uint32_t turn = sb + t.at(2) * W::TILE + (warp - 20) * (W::TILE / 8);
        if (!(ok = wait_for(g_ready + par, c >> 1 & 1))) break;
        const float lead = p.scale * ex2(-s_g[par * 128 + trow]);
        __syncwarp();
        if (lane == 0) mbar_arrive(g_free + par);
        if (!(ok = wait_for(pv_done, par))) break;
        tc_fence_after_sync();
        const bool bad = s_bad[c % 3] != 0;
        uint8_t* to = static_cast<uint8_t*>(p.out) + (size_t)(row0 + chunk_of(c) * CHUNK + 32 * quarter) * row_bytes + (h * D + half * SC) * ES;
        const uint32_t my_row = turn + lane * (LANES * 16), my_turn = (lane * LANES / 8 % LANES) << 4;
#pragma unroll 1
        for (int b = 0; b < SC; b += TURN) {
          constexpr int COLS = 16 / ES;  // to a piece of 16 bytes
#pragma unroll 1
          for (int z = 0; z < LANES; z += 2) {
            float x[2][8], y[2][8];
            uint32_t u[2][4];
            const uint32_t at = my + half * SC + b + z * COLS;
            tmem_ld8(at + W::T_O1, x[0]);
            tmem_ld8(at + W::T_O2, y[0]);
            if constexpr (!FINE) {
              tmem_ld8(at + W::T_O1 + 8, x[1]);
              tmem_ld8(at + W::T_O2 + 8, y[1]);
            }
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < (FINE ? 1 : 2); ++i)
#pragma unroll
              for (int j = 0; j < 8; j += 2) {
                float m, n;
                unpair(fma2(pair(lead, lead), pair(x[i][j], x[i][j + 1]), mul2(pair(p.scale, p.scale), pair(y[i][j], y[i][j + 1]))), &m, &n);
                if constexpr (FINE) {
                  u[j / 4][j % 4] = __float_as_uint(m);
                  u[j / 4][j % 4 + 1] = __float_as_uint(n);
                } else {
                  u[i][j / 2] = pack_bf16x2(m, n);
                }
              }
#pragma unroll
            for (int i = 0; i < 2; ++i) st_shared_v4(my_row + (((z + i) << 4) ^ my_turn), u[i][0], u[i][1], u[i][2], u[i][3]);
          }
          if (bad) {  // in place, column by column
#pragma unroll 1
            for (int i = 0; i < TURN; ++i)
              if (s_first[c % 3 * 128 + half * SC + b + i] <= trow) {
                const uint32_t at = my_row + (((i * ES >> 4) << 4) ^ my_turn) + (i * ES & 15);
                if (FINE) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(0x7fffffffu) : "memory");
                else st_shared_u16(at, 0x7fff);
              }
          }
          if (b + TURN == SC) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_read);
          } else {
            __syncwarp();
          }
          uint32_t o[LANES][4];
#pragma unroll
          for (int i = 0; i < LANES; ++i) {
            const int r = i * (32 / LANES) + lane / LANES, at = lane % LANES;
            lds_v4(turn + r * (LANES * 16) + ((at ^ (r * LANES / 8 % LANES)) << 4), o[i]);
          }
          if (b + TURN == SC) {
            fence_proxy_async_smem();  // the tile's next content comes by TMA
            __syncwarp();
            if (lane == 0) mbar_arrive(o_done + par);
          } else {
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < LANES; ++i) {
            const int r = i * (32 / LANES) + lane / LANES, at = lane % LANES;
            if (32 * quarter + r < rows)
              *reinterpret_cast<uint4*>(to + r * row_bytes + b * ES + at * 16) = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
          }
        }
        t.move(3);
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
    if (warp == 28 && lane == 0) {
      // -------------------------------------------------------------- loads
      constexpr int KINDS = Ring<MODE>::KINDS, TILES = Ring<MODE>::TILES;
      const int items = KINDS * nch;
      Ring<MODE> t;
      int kind = 0, c = 0, used = 0, used_c = 0;  // of the item, and of the one whose place it takes
#pragma unroll 1
      for (int i = 0; i < items && ok; ++i) {
        if (i >= TILES) {
          uint64_t* free = used == 0 ? z_done : MODE != OUTPUTS ? z_done : used == 1 ? (FINE ? f_done : qs_done) : o_done;
          if (!(ok = wait_for(free + (used_c & 1), used_c >> 1 & 1))) break;
          if (++used == KINDS) {
            used = 0;
            ++used_c;
          }
        }
        const CUtensorMap* map = kind == 0 ? &map_k : MODE == OUTPUTS && kind == 1 ? &map_q : &map_v;
        mbar_arrive_expect_tx(full + t.tile, W::TILE);
#pragma unroll 1
        for (int b = 0; b < D / 64; ++b)
          tma_load_3d(smem + t.tile * W::TILE + b * W::BLOCK, map, full + t.tile, 64 * b, h, row0 + chunk_of(c) * CHUNK);
        t.move(1);
        if (++kind == KINDS) {
          kind = 0;
          ++c;
        }
      }
      // no copy is in flight when the CTA ends: the last one into each tile has landed (after a wait that ran
      // out, fewer may be on their way than are waited for)
      Ring<MODE> last;
      for (int i = 0; i < items; ++i) {
        if (i + TILES >= items) ok = wait_for(full + last.tile, last.turn) && ok;
        last.move(1);
      }
    } else if (warp == 29 && lane == 0) {
      // -------------------------------------------------------------- products
      constexpr uint32_t ID_A = make_idesc_bf16(128, 128, false, false), ID_O = make_idesc_bf16(128, D, false, true),
                         ID_Z = make_idesc_bf16(D, D, true, true);
      Ring<MODE> t;
      constexpr int VALUES = MODE == OUTPUTS ? 2 : 1;
      // D = (D +) A B over K = 64 n; descriptors advance by `in` for each 16 of K and `out` for each 64
      constexpr uint32_t K_IN = 2, K_OUT = W::BLOCK >> 4, MN_IN = 128, MN_OUT = 512;
      auto product = [&](uint32_t to, uint64_t a, uint32_t a_in, uint32_t a_out, uint64_t b, uint32_t b_in, uint32_t b_out, uint32_t id,
                         int n, uint32_t add) {
#pragma unroll 1
        for (int o = 0; o < n; ++o)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            umma_bf16(to, a + o * a_out + i * a_in, b + o * b_out + i * b_in, id, add);
            add = 1;
          }
      };
      auto state_part = [&](uint32_t k_at, uint32_t v_at, bool add) {
        product(tb + W::T_Z, desc_mn(k_at, W::BLOCK), MN_IN, MN_OUT, desc_mn(v_at, W::BLOCK), MN_IN, MN_OUT, ID_Z, 2, add);
      };
      auto from_state = [&](uint32_t q_at, bool add) {
        product(tb + W::T_O1, desc_k(q_at), K_IN, K_OUT, desc_mn(sb + W::Y, W::IMAGE_BLOCK), MN_IN, MN_OUT, ID_O, D / 64, add);
      };
#pragma unroll 1
      for (int c = 0; c < nch && ok; ++c) {
        const uint32_t par = c & 1;
        const uint32_t k_at = sb + t.tile * W::TILE, v_at = sb + t.at(VALUES) * W::TILE, q_at = sb + t.at(1) * W::TILE;
        if (!(ok = wait_for(full + t.tile, t.turn))) break;
        if constexpr (MODE == OUTPUTS) {
          if (!(ok = wait_for(full + t.at(1), t.phase(1)))) break;
          product(tb + W::T_A, desc_k(q_at), K_IN, K_OUT, desc_k(k_at), K_IN, K_OUT, ID_A, D / 64, 0);
          umma_commit(a_done);
        }
        if (!(ok = wait_for(v_ready, par))) break;
        if (MODE != ENDS && c > 0 && !(ok = wait_for(z_free, par ^ 1))) break;
        tc_fence_after_sync();
        state_part(k_at, sb + W::X, MODE == ENDS && c > 0);
        if constexpr (MODE == OUTPUTS) {
          if (exact) {
            umma_commit(zh_done);
            if (!(ok = wait_for(l_ready, par))) break;
            state_part(k_at, sb + W::X, true);
          }
          umma_commit(z_done + par);
          if (!(ok = wait_for(s_ready, par))) break;
          if (c > 0 && !(ok = wait_for(o_read, par ^ 1))) break;
          tc_fence_after_sync();
          from_state(q_at, false);
          umma_commit(qs_done + par);
          if (FINE) {
            if (!(ok = wait_for(f_ready, par))) break;
            from_state(q_at, true);
            umma_commit(f_done + par);
          }
          if (!(ok = wait_for(p_ready, par) && wait_for(n_ready + par, c >> 1 & 1))) break;
          tc_fence_after_sync();
          const uint64_t b = desc_mn(v_at, W::BLOCK);
#pragma unroll 1
          for (int o = 0; o < (FINE ? 4 : 2); ++o)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              umma_f16_ta(tb + W::T_O2, tb + W::T_A + 64 * (o & 1) + 16 * (o & 2) + 8 * i, b + (o & 1) * MN_OUT + i * MN_IN, ID_O, o || i ? 1u : 0u);
          umma_commit(pv_done);
        } else {
          state_part(k_at, sb + W::Y, true);
          umma_commit(z_done + par);
        }
        t.move(Ring<MODE>::KINDS);
      }
      if (!ok) {  // what has been issued ends before the CTA does
        umma_commit(pv_done);
        umma_commit(pv_done);
        (void)wait_for(pv_done, 0);
        (void)wait_for(pv_done, 1);
      }
    } else if (warp == 30) {
      // -------------------------------------------------------------- decays
      Decays la = {};
#pragma unroll 1
      for (int c = -1; c < nch; ++c) {
        const float4 g4 = la.sum(p);
        if (c + 1 < nch) la.load(p, row0 + chunk_of(c + 1) * CHUNK, rows_of(chunk_of(c + 1)), h);
        if (c < 0) continue;
        if (c > 1 && !(ok = wait_for(g_free + (c & 1), (c >> 1 & 1) ^ 1))) break;
        *reinterpret_cast<float4*>(s_g + (c & 1) * 128 + 4 * lane) = make_float4(-g4.x, -g4.y, -g4.z, -g4.w);
        __syncwarp();
        if (lane == 0) mbar_arrive(g_ready + (c & 1));
      }
    }
  }
  if (!ok && lane == 0) atomicExch(p.status, (int)KDA_ERR_TIMEOUT);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tb, 512);
}

template <int D, Mode MODE, bool FINE>
__global__ void __launch_bounds__(WALK_THREADS, 1)
    linear_walk_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Walk w) {
  dependents_may_start();
  walk<D, MODE, false, FINE>(map_q, map_k, map_v, w);
}

// Both directions: keys and values ahead, queries and the outputs' gradients back.
template <int D, Mode MODE>
__global__ void __launch_bounds__(WALK_THREADS, 1)
    linear_walks_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
                        const __grid_constant__ Walk ahead, const __grid_constant__ Walk back) {
  dependents_may_start();
  if (blockIdx.y == 0) walk<D, MODE, false, false>(map_k, map_k, map_v, ahead);
  else walk<D, MODE, true, false>(map_q, map_q, map_do, back);
}

// The states at the segments' starts (BACK: the gradients at their ends) from the segments' contributions,
// which they replace: E = 2^decay E + Z, one after the other, 1024 entries of a state to a CTA.
template <bool BACK> __device__ __forceinline__ void scan(const Walk& w) {
  const LinearProblem& p = w.p;
  const int parts = p.d * p.d / 1024;
  const int part = blockIdx.x % parts, nh = blockIdx.x / parts, n = nh / p.H, h = nh % p.H;
  long long row0 = (long long)n * p.len;
  int len = p.len;
  if (p.cu_seqlens) len = sequence_rows(p, n, &row0);
  const int count = max((len + w.seg_len - 1) / w.seg_len, 1);
  const long long first = p.cu_seqlens ? row0 / w.seg_len + n : (long long)n * w.segs;
  const size_t at = (size_t)part * 1024 + threadIdx.x * 4, size = (size_t)p.d * p.d;
  dependency_wait();
  float4 e = p.s_in ? *reinterpret_cast<const float4*>(p.s_in + (size_t)nh * size + at) : make_float4(0.f, 0.f, 0.f, 0.f);
  // the contributions of AHEAD segments are on their way together
  constexpr int AHEAD = 8;
  for (int i0 = 0; i0 < count; i0 += AHEAD) {
    float4 z[AHEAD];
    float keep[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const size_t slot = (size_t)(first + (BACK ? count - 1 - i0 - i : i0 + i)) * p.H + h;
      if (i0 + i + 1 < count) {
        z[i] = *reinterpret_cast<const float4*>(w.carry + slot * size + at);
        keep[i] = w.decay[slot];
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const size_t slot = (size_t)(first + (BACK ? count - 1 - i0 - i : i0 + i)) * p.H + h;
      if (i0 + i < count) *reinterpret_cast<float4*>(w.carry + slot * size + at) = e;
      if (i0 + i + 1 < count) {
        const float k = ex2(keep[i]);
        e = make_float4(k * e.x + z[i].x, k * e.y + z[i].y, k * e.z + z[i].z, k * e.w + z[i].w);
      }
    }
  }
}

static __global__ void __launch_bounds__(256) linear_scan_kernel(const __grid_constant__ Walk ahead, const __grid_constant__ Walk back) {
  dependents_may_start();
  if (blockIdx.y == 0) scan<false>(ahead);
  else scan<true>(back);
}

// ---------------------------------------------------------------- host

inline bool make_rows_map(CUtensorMap* map, const void* base, long long stride, const LinearProblem& p) {
  return make_map_3d_bf16(map, base, (uint64_t)p.d, (uint64_t)p.H, (uint64_t)p.T, (uint64_t)p.d, (uint64_t)stride, 64, 1, CHUNK,
                          CU_TENSOR_MAP_SWIZZLE_128B);
}

// A launch; `after`: it may start while the one before it in the stream runs, which this call made.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, bool after, cudaStream_t stream, A... args) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline unsigned walk_ctas(const Walk& w) { return (unsigned)((long long)w.slots * w.p.H); }
inline cudaError_t launch_scan(const Walk& ahead, const Walk& back, int directions, cudaStream_t stream) {
  const LinearProblem& p = ahead.p;
  return launch(linear_scan_kernel, dim3((unsigned)((long long)p.n_seq * p.H * (p.d * p.d / 1024)), directions), 256, 0, true, stream,
                ahead, back);
}

// Tokens to a segment: whole chunks, such that the walk (and, where it is cut, the half as long one before
// it) takes the fewest steps of the machine.  Cut in more than one, a segment has at least 4 chunks.
inline int segment_tokens(int n_seq, int T, int H, bool packed, int sms) {
  const long long len = packed ? T : T / n_seq, chunks = std::max((len + CHUNK - 1) / CHUNK, 1LL);
  long long best = chunks, best_cost = -1;
  for (long long segs = 1; segs <= 256 && segs * 4 <= std::max(chunks, 4LL); ++segs) {
    const long long of = (chunks + segs - 1) / segs;
    const long long items = (packed ? chunks / of + n_seq : n_seq * ((chunks + of - 1) / of)) * H;
    const long long cost = (items + sms - 1) / sms * (of + 3) * (segs > 1 ? 3 : 2);
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
