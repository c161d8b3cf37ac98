// Gradients of the linear attention, chunk by chunk.  With the notation of
// kda_linear_walk.cuh, do scaled, dS the gradient that arrives at a chunk's
// end, D_ij = 2^{g_i - g_j} for j <= i, A = Q K^T and B = dO V^T:
//
//     R = B . D,  P = A . D
//     dQ = R K   + 2^{g_i} dO S^T
//     dK = R^T Q + 2^{G - g_j} V dS^T
//     dV = P^T dO + 2^{G - g_j} K dS
//     dS <- 2^G dS + (2^{g_i} Q)^T dO       (to the chunk before)
//
// Two walks leave S and dS at every chunk as bf16 operand images (the second
// runs against time); then every chunk is a CTA of its own.  Nine products of
// 128 x 128 x d: three scores (B with either side on the lanes, and A^T), three
// from the states, three from the weights, which lie in tensor memory where
// the scores were.
//
// A decay's gradient is the sum over all pairs of tokens on either side of it,
//
//     D_t = sum_{j < t <= i} w_ij + sum_{i >= t} q_i^T x_i + sum_{j < t} k_j^T y_j + 2^G <S, dS>,
//     w = A . B . D,  x_i = 2^{g_i} S do_i,  y_j = 2^{G - g_j} dS v_j,
//
// the sums of chunk-crossing pairs being those of the states.  From one token
// to the next D changes by what token t takes out (as i) and brings in (as j):
// an exclusive running sum in the chunk, of fp32 numbers that no operand's
// rounding has touched but the states'.  (The shorter way, q . dq - k . dk
// summed from the sequence's end, cancels: after a few thousand tokens the
// rounding of dq and dk is all that is left of it.)
//
// Warps: 0-15 compute (four to each quarter of the lanes, with a quarter of the
// columns each), 16 loads and issues.  One CTA on an SM; six tiles of shared
// memory (Q, K, V, dO, S, dS), through which the gradients leave once their
// content has been used.
//
// Measured (8192 tokens, 32 heads of 128): 308 us, of which the segments' ends
// take 50, their join 8, the images 70 and this kernel 177 to 190 (573 MB, 38 %
// of DRAM's throughput, tensor pipe 17 %, issue slots 31 %).  What bounds it is
// the chain within a chunk, 13 us of products and the arithmetic between them:
// a CTA that stays, with the next chunk's tiles on their way from the moment
// theirs are free, took 177 instead of 188 us by itself and as long in the call
// (302 to 307 us).  Two chunks at once do not fit the tensor memory as it is
// used: while scores are in it, one has three times 128 columns of them and 128
// of sums.  Later on the weights leave half of the scores' columns free, but in
// pieces of 16, one beside each 16 of weights, where no sum fits; weights laid
// out together would make room.  The code that a chunk of
// finite values runs is kept within 32 KB, as the instruction cache holds it
// (313 -> 306 us).
#include <algorithm>
#include <cstddef>

#include "kda_linear_walk.cuh"

namespace kda {
namespace {

using namespace linear;

struct Grad {
  LinearProblem p;
  const uint8_t *s_images, *ds_images;
  void *dq, *dk, *dv, *dla;
  float* sums;  // [chunks][H]: a chunk's part of the sum over all tokens, or null
};

template <int D> struct GradShape : Shape<D> {
  using Shape<D>::TILE;
  static constexpr uint32_t Q = 0, K = TILE, V = 2 * TILE, DO = 3 * TILE, S = 4 * TILE, DS = 5 * TILE, MISC = 6 * TILE;
  static constexpr uint32_t ODD = MISC + 8192;
  static constexpr uint32_t SMEM_USED = ODD + 2048, SMEM = SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024;
  static constexpr uint32_t T0 = 0, T1 = 128, T2 = 256, T3 = 384;  // tensor memory
};

__device__ __forceinline__ uint32_t to_bf16x2(uint64_t v) {
  float a, b;
  unpair(v, &a, &b);
  return pack_bf16x2(a, b);
}

// Sums over the warp's lanes of 8 numbers each; lane l gets that of number l >> 2.
__device__ __forceinline__ float sum_lanes(float (&x)[8]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 4; k; k /= 2) {
    const bool up = lane & (4 * k);
#pragma unroll
    for (int i = 0; i < k; ++i) {
      const float keep = up ? x[i + k] : x[i], give = up ? x[i] : x[i + k];
      x[i] = keep + __shfl_xor_sync(~0u, give, 4 * k);
    }
  }
  x[0] += __shfl_xor_sync(~0u, x[0], 2);
  return x[0] + __shfl_xor_sync(~0u, x[0], 1);
}

constexpr int GRAD_WARPS = 16, GRAD_THREADS = 32 * GRAD_WARPS + 32;

// Values that are not finite.  One reaches the gradients that the formulas put it into, and no others: in a query or an
// output's gradient those of its own token and earlier ones, in a key or a value those of its own and later ones.  Weights
// that are 0 would carry it further, into a whole chunk.  It shows in the sums over a chunk's pairs (0 times it is not
// finite, either), so that other chunks pay nothing but a look at those: all that follows is in functions of their own, out
// of the way of the code that every chunk runs (8192 tokens 307 -> 309 us; in the loops themselves 318 to 323).
struct Odd {
  static constexpr int NEVER = 0x7fffffff;
  int edge[3][128];  // of channels of Q, K and dO: 127 less the last token (K: the first token) with such a value
  int queries, keys; // 127 less the last token with one in Q or dO; the first token with one in K or V
  int any;           // whether the chunk may have some
};

// In a chunk that may have some, before the weights' products: takes them out of Q, K and dO, of which the scores have been
// formed (this thread's token's, in its part of the channels); makes the weights of pairs in the wrong order 0, which only
// products with 0 have made so; and forms the decays' sums again of the pairs that some finite gradient of a decay needs:
// a later token after the last odd one of the queries' side with an earlier one before the first odd one of the keys'.
template <int D>
__device__ __noinline__ bool without_odd(uint8_t* smem, uint32_t tb, uint64_t* cleared, const float* s_g, float* s_out, float* s_in, float scale) {
  using W = GradShape<D>;
  Odd* odd = reinterpret_cast<Odd*>(smem + W::ODD);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quarter = warp & 3, part = warp >> 2, trow = 32 * quarter + lane;
  auto at = [&](uint32_t tile, int row, int ch) {
    return smem + tile + ch / 64 * W::BLOCK + row * 128 + (((uint32_t)(ch / 8 % 8) ^ (uint32_t)(row & 7)) << 4) + ch % 8 * 2;
  };
  if (threadIdx.x < offsetof(Odd, any) / 4) odd->edge[0][threadIdx.x] = Odd::NEVER;  // (and the two after the edges)
  __syncwarp();
  if (lane == 0) mbar_arrive(cleared);
  if (!wait_for(cleared, 0)) return false;
#pragma unroll 1
  for (int tile = 0; tile < 4; ++tile) {
    const bool keys = tile == 1 || tile == 2;
    const int when = keys ? trow : 127 - trow;
#pragma unroll 1
    for (int ch = part * (D / 4); ch < (part + 1) * (D / 4); ++ch) {
      uint16_t* x = reinterpret_cast<uint16_t*>(at(tile * W::TILE, trow, ch));
      if ((*x & 0x7f80) != 0x7f80) continue;
      atomicMin(keys ? &odd->keys : &odd->queries, when);
      if (tile == 2) continue;  // (the values' side meets no weights)
      atomicMin(&odd->edge[tile == 3 ? 2 : tile][ch], when);
      *x = 0;
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(cleared);
  if (!wait_for(cleared, 1)) return false;
  const uint32_t weights = tb + ((uint32_t)(32 * quarter) << 16) + 32 * part;
#pragma unroll 1
  for (int c = 0; c < 12; ++c) {  // four pairs of later tokens (T0: earlier ones) at a time
    uint32_t u[4];
    const uint32_t from = weights + c / 4 * 128 + c % 4 * 4;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(from));
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int other = 32 * part + c % 4 * 8 + 2 * i;
      if (c < 4 ? other > trow : other < trow) u[i] &= 0xffff0000u;
      if (c < 4 ? other + 1 > trow : other + 1 < trow) u[i] &= 0xffffu;
    }
    tmem_st4u(from, u);
  }
  tmem_st_wait();
  const int after = 127 - min(odd->queries, 128), before = odd->keys;
  float later = 0.f;
#pragma unroll 1
  for (int i = 32 * part; i < 32 * part + 32; ++i) {
    float w = 0.f;
    if (i > trow && i > after && trow < before) {
      float a = 0.f, b = 0.f;
#pragma unroll 1
      for (int ch = 0; ch < D; ++ch) {
        auto get = [&](uint32_t tile, int row) { return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(at(tile, row, ch))); };
        a = fmaf(get(W::Q, i), get(W::K, trow), a);
        b = fmaf(get(W::DO, i), get(W::V, trow), b);
      }
      w = scale * ex2(-(s_g[i] - s_g[trow])) * a * b;
    }
    later += w;
#pragma unroll
    for (int o = 16; o; o /= 2) w += __shfl_xor_sync(~0u, w, o);
    if (lane == 0) s_in[quarter * 128 + i] = w;
  }
  s_out[part * 128 + trow] = later;
  return true;
}

// Afterwards: the channels that they reach, in gradients that have been written.
template <int D> __device__ __noinline__ void mark_odd(const uint8_t* smem, const Grad& a, int row0, int rows, int h) {
  const Odd* odd = reinterpret_cast<const Odd*>(smem + GradShape<D>::ODD);
  const int warp = threadIdx.x >> 5, part = warp >> 2, trow = 32 * (warp & 3) + (threadIdx.x & 31);
  __syncwarp();
  if (trow >= rows) return;
  const size_t at = ((size_t)(row0 + trow) * a.p.H + h) * D;
#pragma unroll 1
  for (int ch = part * (D / 4); ch < (part + 1) * (D / 4); ++ch) {
    if (odd->edge[0][ch] <= 127 - trow) static_cast<uint16_t*>(a.dk)[at + ch] = 0x7fff;
    if (odd->edge[1][ch] <= trow) static_cast<uint16_t*>(a.dq)[at + ch] = 0x7fff;
    if (odd->edge[2][ch] <= 127 - trow) static_cast<uint16_t*>(a.dv)[at + ch] = 0x7fff;
  }
}

// A warp, before the decays' gradients are formed: tokens' parts that only those take which are not finite.
__device__ __noinline__ void drop_odd(const Odd* odd, float* s_out, float* s_x) {
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < 512; i += 32) {
    if (127 - i % 128 >= odd->queries) s_x[i] = 0.f;
    if (i % 128 >= odd->keys) s_out[i] = 0.f;
  }
  __syncwarp();
}
// And afterwards those.
__device__ __noinline__ void mark_odd_decays(const Odd* odd, const Grad& a, int row0, int rows, int slot, int h) {
  __syncwarp();
#pragma unroll 1
  for (int t = threadIdx.x & 31; t < rows; t += 32) {
    if (t <= odd->keys && 127 - t < odd->queries) continue;
    const size_t at = (size_t)(row0 + t) * a.p.H + h;
    if (a.sums) a.sums[(size_t)slot * a.p.H + h] = NAN;
    else if (a.p.la_f32) static_cast<float*>(a.dla)[at] = NAN;
    else static_cast<uint16_t*>(a.dla)[at] = 0x7fff;
  }
}

template <int D>
__global__ void __launch_bounds__(GRAD_THREADS, 1)
    linear_grad_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                       const __grid_constant__ Grad a) {
  using W = GradShape<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const LinearProblem& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t sb = smem_u32(smem);
  const int slot = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const Segment seg = find_segment(p, CHUNK, (p.len + CHUNK - 1) / CHUNK, slot);
  if (seg.n < 0 || seg.tokens <= 0) {
    if (a.sums && tid == 0) a.sums[(size_t)slot * p.H + h] = 0.f;
    // one CTA waits even if offsets leave no rows to any: what follows this launch relies on the ones before it
    if (blockIdx.x == 0) dependency_wait();
    return;
  }
  if (sb & 1023u) {  // the tiles' swizzle goes by address
    if (tid == 0) atomicExch(p.status, (int)KDA_ERR_ALIGNMENT);
    return;
  }
  const int rows = seg.tokens, row0 = (int)(seg.row0 + (long long)seg.index * CHUNK);

  float* s_g = reinterpret_cast<float*>(smem + W::MISC);  // [128]: -g
  float* s_out = s_g + 128;                               // [4][128]: sums over later tokens, and of k . y, by part of the columns
  float* s_in = s_out + 512;                              // [4][128]: sums over earlier tokens, by quarter of the lanes
  float* s_x = s_in + 512;                                // [4][128]: q . x, by part of the columns
  float* s_dot = s_x + 512;                               // [16]: <S, dS>, by warp
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + W::MISC + 7168);
  uint64_t* done = bars;  // [9] the products, in their order
  uint64_t *bt_done = done, *at_done = done + 1, *b_done = done + 2, *x_done = done + 3, *dq_done = done + 4, *y_done = done + 5,
           *z_done = done + 6, *dk_done = done + 7, *dv_done = done + 8;
  uint64_t *landed = bars + 9, *images = bars + 10;
  uint64_t *clean = bars + 11, *r_ready = bars + 12, *w_ready = bars + 13, *x_ready = bars + 14, *dq_read = bars + 15,
           *y_ready = bars + 16, *z_ready = bars + 17, *sums_ready = bars + 18;  // by all warps
  uint64_t* cleared = bars + 19;  // by all warps, of a chunk with values that are not finite
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 20);
  Odd* s_odd = reinterpret_cast<Odd*>(smem + W::ODD);

  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (warp == GRAD_WARPS && lane == 0) {
#pragma unroll 1
    for (int i = 0; i < 20; ++i) mbar_init(bars + i, i < 11 ? 1 : GRAD_WARPS);
    s_odd->any = 0;
    mbar_fence_init();
    fence_proxy_async_smem();
    // on their way while the rest of the CTA is made ready
    mbar_arrive_expect_tx(landed, 4 * W::TILE);
    for (int b = 0; b < D / 64; ++b) {
      tma_load_3d(smem + W::V + b * W::BLOCK, &map_v, landed, 64 * b, h, row0);
      tma_load_3d(smem + W::DO + b * W::BLOCK, &map_do, landed, 64 * b, h, row0);
      tma_load_3d(smem + W::K + b * W::BLOCK, &map_k, landed, 64 * b, h, row0);
      tma_load_3d(smem + W::Q + b * W::BLOCK, &map_q, landed, 64 * b, h, row0);
    }
  }
  if (warp == 0) {
    Decays la;
    la.load(p, row0, rows, h);
    const float4 g4 = la.sum(p);
    *reinterpret_cast<float4*>(s_g + 4 * lane) = make_float4(-g4.x, -g4.y, -g4.z, -g4.w);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tb = *s_tmem;
  bool ok = true;

  if (warp == GRAD_WARPS) {
    if (lane == 0) {
      // -------------------------------------------------------------- the states, then products in the order of their needs
      dependency_wait();
      const size_t image = ((size_t)slot * p.H + h) * W::IMAGE;
      mbar_arrive_expect_tx(images, 2 * W::IMAGE);
      bulk_g2s(smem + W::S, a.s_images + image, W::IMAGE, images);
      bulk_g2s(smem + W::DS, a.ds_images + image, W::IMAGE, images);
      // As steps of one loop, so that the issuing of a product comes once in the code.  A step's tiles, tensor
      // memory and so on are hexadecimal digits, the first step's the last one: tiles Q 0, K 1, V 2, dO 3, S 4,
      // dS 5; scores over channels (0), sums from the states over channels as they lie (1) or read transposed
      // (2), sums over tokens with weights from tensor memory, added to what is there (3).
      constexpr uint64_t TO = 0x303033021, A = 0x211203312, B = 0x305514203, KIND = 0x332131000;
      static_assert(W::T1 == 128 && W::T2 == 256 && W::T3 == 384, "their digits");
      constexpr uint32_t ID_SCORE = make_idesc_bf16(128, 128, false, false), ID_ROWS = make_idesc_bf16(128, D, false, false),
                         ID_COLS = make_idesc_bf16(128, D, false, true);
#pragma unroll 1
      for (int step = 0; step < 9 && ok; ++step) {
        auto digit = [&](uint64_t digits) { return (uint32_t)(digits >> (4 * step)) & 15u; };
        if (step == 0) ok = wait_for(landed, 0) && wait_for(clean, 0);
        if (step == 3) ok = wait_for(images, 0);
        if (step == 4) ok = wait_for(r_ready, 0) && wait_for(x_ready, 0);
        if (step == 6) ok = wait_for(dq_read, 0);
        if (step == 7) ok = wait_for(w_ready, 0) && wait_for(y_ready, 0);
        if (step == 8) ok = wait_for(z_ready, 0);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t kind = digit(KIND), to = tb + 128 * digit(TO), b_at = sb + digit(B) * W::TILE;
        const bool rows_k = kind < 2;  // B's rows lie along K
        const uint32_t id = kind == 0 ? ID_SCORE : kind == 1 ? ID_ROWS : ID_COLS, block = kind == 0 || kind == 3 ? W::BLOCK : W::IMAGE_BLOCK;
        const uint64_t b = rows_k ? desc_k(b_at) : desc_mn(b_at, block), a = desc_k(sb + digit(A) * W::TILE);
        const uint32_t b_in = rows_k ? 2 : 128, b_out = rows_k ? block >> 4 : 512, weights = tb + 128 * digit(A);
        if (kind == 3) {
#pragma unroll 1
          for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              umma_f16_ta(to, weights + 64 * o + 32 * (i >> 1) + 8 * (i & 1), b + o * 512 + i * 128, ID_COLS, 1u);
        } else {
#pragma unroll 1
          for (int o = 0; o < D / 64; ++o)
#pragma unroll
            for (int i = 0; i < 4; ++i) umma_bf16(to, a + o * (W::BLOCK >> 4) + i * 2, b + o * b_out + i * b_in, id, o || i ? 1u : 0u);
        }
        umma_commit(done + step);
      }
      if (!ok) {  // what has been issued ends before the CTA does
        umma_commit(dv_done);
        (void)wait_for(dv_done, 0);
      }
    }
  } else {
    const int quarter = warp & 3, part = warp >> 2, trow = 32 * quarter + lane;
    const uint32_t my = tb + ((uint32_t)(32 * quarter) << 16);
    const float g_mine = -s_g[trow], lead = p.scale * ex2(g_mine), trail = ex2(-s_g[127] - g_mine), keep = ex2(-s_g[127]);
    constexpr int SC = D / 4;
    const uint32_t row_at = (uint32_t)trow * 128;
    bool odd = false;
    auto piece = [&](int x) { return (uint32_t)(x / 8) * W::BLOCK + row_at + (((uint32_t)(x % 8) ^ (uint32_t)(trow & 7)) << 4); };

    ok = wait_for(landed, 0);
    if (ok) {
      if (rows < CHUNK && trow >= rows) {  // rows of other sequences
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i)
          for (uint32_t tile : {W::Q, W::K, W::V, W::DO}) st_shared_v4(sb + tile + piece(part * (D / 32) + i), 0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(clean);
      ok = wait_for(images, 0);
    }
    if (ok) {
      // <S, dS>: 16 bytes of either at a time, wherever they belong
      float dot = 0.f;
#pragma unroll 1
      for (uint32_t i = tid * 16; i < W::IMAGE; i += 32 * GRAD_WARPS * 16) {
        uint32_t u[4], v[4];
        lds_v4(sb + W::S + i, u);
        lds_v4(sb + W::DS + i, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) dot = fmaf(lo_f32(u[j]), lo_f32(v[j]), fmaf(hi_f32(u[j]), hi_f32(v[j]), dot));
      }
#pragma unroll
      for (int o = 16; o; o /= 2) dot += __shfl_xor_sync(~0u, dot, o);
      if (lane == 0) s_dot[warp] = dot;
      ok = wait_for(bt_done, 0) && wait_for(at_done, 0);
    }
    if (ok) {
      // ---- R^T and P^T, earlier tokens on the lanes, 8 later ones at a time, and what a pair gives to the decays
      tc_fence_after_sync();
      uint64_t later = pair(0.f, 0.f);
#pragma unroll 1
      for (int i0 = 32 * part; i0 < 32 * part + 32; i0 += 8) {
        uint32_t u[4] = {0u, 0u, 0u, 0u}, v[4] = {0u, 0u, 0u, 0u};
        float earlier = 0.f;
        if (i0 + 7 >= 32 * quarter) {
          float x[8], y[8], w[8], e[8];  // e: log2 of the decays between, with the other sign
          tmem_ld8(my + W::T1 + i0, x);
          tmem_ld8(my + W::T2 + i0, y);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            unpair(add2(*reinterpret_cast<const uint64_t*>(s_g + i0 + i), pair(g_mine, g_mine)), &e[i], &e[i + 1]);
          if (i0 < 32 * quarter + 31) {  // some of the warp's tokens are not before all of these
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = i0 + i >= trow ? e[i] : INFINITY;
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const uint64_t decay = mul2(pair(ex2(-e[i]), ex2(-e[i + 1])), pair(p.scale, p.scale)), z = mul2(decay, pair(x[i], x[i + 1]));
            u[i / 2] = to_bf16x2(z);
            v[i / 2] = to_bf16x2(mul2(decay, pair(y[i], y[i + 1])));
            unpair(mul2(z, pair(y[i], y[i + 1])), &w[i], &w[i + 1]);
          }
          if (i0 <= 32 * quarter + 31) {  // a token's pair with itself straddles no decay
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = i0 + i == trow ? 0.f : w[i];
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2) later = add2(later, pair(w[i], w[i + 1]));
          earlier = sum_lanes(w);
        }
        const int at = 32 * part + (i0 - 32 * part) / 2;
        tmem_st4u(my + W::T1 + at, u);
        tmem_st4u(my + W::T2 + at, v);
        if (lane % 4 == 0) s_in[quarter * 128 + i0 + lane / 4] = earlier;
      }
      float later_0, later_1;
      unpair(later, &later_0, &later_1);
      s_out[part * 128 + trow] = later_0 + later_1;
      if (!(fabsf(later_0 + later_1) < INFINITY)) s_odd->any = 1;
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(w_ready);
      ok = wait_for(b_done, 0);
    }
    if (ok) {
      // ---- R, later tokens on the lanes
      tc_fence_after_sync();
#pragma unroll 1
      for (int j0 = 32 * part; j0 < 32 * part + 32; j0 += 8) {
        uint32_t u[4] = {0u, 0u, 0u, 0u};
        if (j0 <= 32 * quarter + 31) {
          float x[8], e[8];
          tmem_ld8(my + W::T0 + j0, x);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; j += 2)
            unpair(add2(*reinterpret_cast<const uint64_t*>(s_g + j0 + j), pair(g_mine, g_mine)), &e[j], &e[j + 1]);
          if (j0 + 7 > 32 * quarter) {  // some come after some of the warp's tokens
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = j0 + j <= trow ? e[j] : -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const uint64_t decay = mul2(pair(ex2(e[j]), ex2(e[j + 1])), pair(p.scale, p.scale));
            u[j / 2] = to_bf16x2(mul2(decay, pair(x[j], x[j + 1])));
          }
        }
        tmem_st4u(my + W::T0 + 32 * part + (j0 - 32 * part) / 2, u);
      }
      tmem_st_wait();
      ok = wait_for(w_ready, 0);
      odd = s_odd->any != 0;
      if (ok && odd) ok = without_odd<D>(smem, tb, cleared, s_g, s_out, s_in, p.scale);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(r_ready);
    }
    // ---- accumulators scaled and written back (0, 2 and 3, of dQ, dK and dV), then, the other products added,
    // written out (1, 4 and 5): as steps of one loop, so that either comes once in the code
#pragma unroll 1
    for (int step = 0; step < 6 && ok; ++step) {
      const uint32_t t = step == 2 || step == 4 ? W::T0 : W::T3;
      ok = wait_for(step == 0 ? x_done : step == 1 ? dq_done : step == 2 ? y_done : step == 3 ? z_done : step == 4 ? dk_done : dv_done, 0);
      if (!ok) break;
      tc_fence_after_sync();
      if (step == 0 || step == 2 || step == 3) {
        const float by = step == 0 ? lead : trail;
        const uint32_t tile = step == 0 ? W::Q : W::K;  // its rows' products with the accumulator's are the decays' part
        uint64_t sum = pair(0.f, 0.f);
#pragma unroll 1
        for (int b = 0; b < SC; b += 16) {
          float x[16];
          uint32_t u[2][4];
          tmem_ld16(my + t + part * SC + b, x);
          lds_v4(sb + tile + piece((part * SC + b) / 8), u[0]);
          lds_v4(sb + tile + piece((part * SC + b) / 8 + 1), u[1]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const uint32_t w = u[i / 8][i % 8 / 2];
            const uint64_t y = mul2(pair(x[i], x[i + 1]), pair(by, by));
            sum = fma2(y, pair(lo_f32(w), hi_f32(w)), sum);
            unpair(y, &x[i], &x[i + 1]);
          }
          tmem_st16(my + t + part * SC + b, x);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        float s, z;
        unpair(sum, &s, &z);
        if (step == 0) s_x[part * 128 + trow] = s + z;
        if (step == 2) s_out[part * 128 + trow] += s + z;
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(step == 0 ? x_ready : step == 2 ? y_ready : z_ready);
          if (step == 2) mbar_arrive(sums_ready);
        }
      } else {
        // through this warp's part of a tile whose content has been used, so that whole lines are written
        constexpr int LANES = W::TILE / 512 / 16;  // to a row's piece of SC channels
        const uint32_t turn = sb + (step == 1 ? W::S : step == 4 ? W::V : W::K) + warp * (W::TILE / 16), mine = turn + lane * (LANES * 16);
#pragma unroll 1
        for (int z = 0; z < LANES; z += 2) {
          float x[16];
          tmem_ld16(my + t + part * SC + 8 * z, x);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 2; ++i)
            st_shared_v4(mine + (((z + i) ^ (lane * LANES / 8 & (LANES - 1))) << 4), pack_bf16x2(x[8 * i], x[8 * i + 1]),
                         pack_bf16x2(x[8 * i + 2], x[8 * i + 3]), pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
        }
        tc_fence_before_sync();
        __syncwarp();
        if (step == 1 && lane == 0) mbar_arrive(dq_read);
        uint32_t o[LANES][4];
#pragma unroll
        for (int i = 0; i < LANES; ++i) {
          const int r = i * (32 / LANES) + lane / LANES, at = lane % LANES;
          lds_v4(turn + r * (LANES * 16) + ((at ^ (r * LANES / 8 & (LANES - 1))) << 4), o[i]);
        }
        uint8_t* to = static_cast<uint8_t*>(step == 1 ? a.dq : step == 4 ? a.dk : a.dv) + ((size_t)(row0 + 32 * quarter) * p.H + h) * D * 2 + part * SC * 2;
#pragma unroll
        for (int i = 0; i < LANES; ++i) {
          const int r = i * (32 / LANES) + lane / LANES, at = lane % LANES;
          if (32 * quarter + r < rows) *reinterpret_cast<uint4*>(to + (size_t)r * p.H * D * 2 + at * 16) = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
        }
      }
    }
    if (ok && odd) mark_odd<D>(smem, a, row0, rows, h);
    // ---- the decays' gradients
    if (ok && warp == 0 && (a.dla || a.sums) && (ok = wait_for(sums_ready, 0))) {
      if (odd) drop_odd(s_odd, s_out, s_x);
      float total = lane < GRAD_WARPS ? keep * s_dot[lane] : 0.f;
#pragma unroll 1
      for (int t = lane; t < 128; t += 32) {  // (what has been added up takes the place of its first part)
        float in = 0.f, out = 0.f, x = 0.f;
#pragma unroll
        for (int i = 0; i < 512; i += 128) {
          in += s_in[i + t];
          out += s_out[i + t];
          x += s_x[i + t];
        }
        total += t < rows ? x : 0.f;
        s_out[t] = t < rows ? out - in - x : 0.f;
      }
#pragma unroll
      for (int o = 16; o; o /= 2) total += __shfl_xor_sync(~0u, total, o);
      __syncwarp();
      const float4 e = *reinterpret_cast<const float4*>(s_out + 4 * lane);
      const float run = (e.x + e.y) + (e.z + e.w);
      float before = run;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const float x = __shfl_up_sync(~0u, before, o);
        if (lane >= o) before += x;
      }
      before = __shfl_up_sync(~0u, before, 1);
      if (lane == 0) before = 0.f;
      *reinterpret_cast<float4*>(s_x + 4 * lane) = make_float4(before, before + e.x, before + (e.x + e.y), before + (e.x + e.y + e.z));
      __syncwarp();
      float sum = 0.f;
#pragma unroll 1
      for (int t = lane; t < rows; t += 32) {
        const float x = total + s_x[t];
        sum += x;
        const size_t at = (size_t)(row0 + t) * p.H + h;
        if (!a.sums) {
          if (p.la_f32) static_cast<float*>(a.dla)[at] = x;
          else static_cast<__nv_bfloat16*>(a.dla)[at] = __float2bfloat16_rn(x);
        }
      }
      if (a.sums) {
#pragma unroll
        for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == 0) a.sums[(size_t)slot * p.H + h] = sum;
      }
      if (odd) mark_odd_decays(s_odd, a, row0, rows, slot, h);
    }
  }
  if (!ok && lane == 0) atomicExch(p.status, (int)KDA_ERR_TIMEOUT);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc(tb, 512);
}

// The sum over all tokens of a head's decay gradients, chunk by chunk in a fixed order.
__global__ void __launch_bounds__(256) decay_sum_kernel(LinearProblem p, const float* sums, long long slots, void* dla) {
  __shared__ float s[256];
  const int h = blockIdx.x, tid = threadIdx.x;
  float sum = 0.f;
  for (long long i = tid; i < slots; i += 256) sum += sums[i * p.H + h];
  s[tid] = sum;
  __syncthreads();
  for (int o = 128; o; o /= 2) {
    if (tid < o) s[tid] += s[tid + o];
    __syncthreads();
  }
  if (tid) return;
  if (p.la_f32) static_cast<float*>(dla)[h] = s[0];
  else static_cast<__nv_bfloat16*>(dla)[h] = __float2bfloat16_rn(s[0]);
}

struct Plan {
  int seg_len, slots;
  long long chunks;
  bool cut;
  size_t carry, decay, images, at_back, at_images, at_sums, bytes;
};

Plan plan_for(int n_seq, int T, int H, int d, bool packed) {
  Plan a{};
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess) sms = 152;
  auto whole = [](size_t x) { return (x + 255) / 256 * 256; };
  a.seg_len = segment_tokens(n_seq, T, 2 * H, packed, sms);  // both directions in one launch
  a.slots = segment_slots(n_seq, T, a.seg_len, packed);
  a.chunks = most_chunks(n_seq, T, packed);
  a.cut = a.slots > n_seq;
  a.carry = a.cut ? (size_t)a.slots * H * d * d * 4 : 0;
  a.decay = a.cut ? whole((size_t)a.slots * H * 4) : 0;
  a.images = (size_t)a.chunks * H * d * d * 2;
  a.at_back = a.carry + a.decay;
  a.at_images = 2 * a.at_back;
  a.at_sums = a.at_images + 2 * a.images;
  a.bytes = a.at_sums + whole((size_t)a.chunks * H * 4);
  return a;
}

template <int D> cudaError_t run(const LinearProblem& p, const LinearGrads& g, void* workspace, cudaStream_t stream) {
  const Plan a = plan_for(p.n_seq, p.T, p.H, D, p.cu_seqlens != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int segs = std::max((p.len + a.seg_len - 1) / a.seg_len, 1);
  Walk ahead{p, a.seg_len, segs, a.slots, reinterpret_cast<float*>(ws),
             a.cut ? reinterpret_cast<float*>(ws + a.carry) : nullptr, ws + a.at_images};
  ahead.p.s_out = nullptr;
  Walk back = ahead;
  back.p.s_in = g.d_final;
  back.p.s_out = g.ds0;
  back.carry = reinterpret_cast<float*>(ws + a.at_back);
  if (a.cut) back.decay = reinterpret_cast<float*>(ws + a.at_back + a.carry);
  back.images = ahead.images + a.images;
  CUtensorMap mq, mk, mv, mo;
  if (p.T > 0 && (!make_rows_map(&mq, p.q, p.q_stride, p) || !make_rows_map(&mk, p.k, p.k_stride, p) ||
                  !make_rows_map(&mv, p.v, p.v_stride, p) || !make_rows_map(&mo, g.d_out, g.d_out_stride, p)))
    return cudaErrorInvalidValue;
  const dim3 both(walk_ctas(ahead), 2);
  cudaError_t e = cudaSuccess;
  if (a.cut) {
    e = launch(linear_walks_kernel<D, ENDS>, both, WALK_THREADS, WalkShape<D, ENDS, false, false>::SMEM, false, stream, mk, mv, mq, mo, ahead,
               back);
    if (e == cudaSuccess) e = launch_scan(ahead, back, 2, stream);
  }
  if (e == cudaSuccess)
    e = launch(linear_walks_kernel<D, IMAGES>, both, WALK_THREADS, WalkShape<D, IMAGES, false, false>::SMEM, a.cut, stream, mk, mv, mq, mo,
               ahead, back);
  if (e != cudaSuccess) return e;
  const Grad x{p, ahead.images, back.images, g.dq, g.dk, g.dv, g.dla,
               g.dla && g.sum_la ? reinterpret_cast<float*>(ws + a.at_sums) : nullptr};
  if (p.T > 0) {
    e = launch(linear_grad_kernel<D>, dim3((unsigned)(a.chunks * p.H)), GRAD_THREADS, GradShape<D>::SMEM, true, stream, mq, mk, mv, mo, x);
    if (e != cudaSuccess) return e;
  }
  if (g.dla && g.sum_la) decay_sum_kernel<<<p.H, 256, 0, stream>>>(p, reinterpret_cast<float*>(ws + a.at_sums), p.T > 0 ? a.chunks : 0, g.dla);
  return cudaGetLastError();
}

}  // namespace

size_t linear_bwd_workspace_bytes(int n_seq, int T, int H, int d, bool packed) { return plan_for(n_seq, T, H, d, packed).bytes; }

cudaError_t launch_linear_bwd(const LinearProblem& p, const LinearGrads& g, void* workspace, cudaStream_t stream) {
  if (p.cu_seqlens) check_offsets_kernel<<<1, 256, 0, stream>>>(p);
  return p.d == 128 ? run<128>(p, g, workspace, stream) : run<64>(p, g, workspace, stream);
}

}  // namespace kda
