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
// Warps: 0-7 compute (two to each quarter of the lanes, with half of the
// columns each), 8 loads and issues.  One CTA on an SM; six tiles of shared
// memory (Q, K, V, dO, S, dS), through which the gradients leave once their
// content has been used.
#include <algorithm>

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
  static constexpr uint32_t SMEM_USED = MISC + 6144, SMEM = SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024;
  static constexpr uint32_t T0 = 0, T1 = 128, T2 = 256, T3 = 384;  // tensor memory
};

// Sums over the warp's lanes of 16 numbers each; lane l gets that of number l >> 1.
__device__ __forceinline__ float sum_lanes(float (&x)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 8; k; k /= 2) {
    const bool up = lane & (2 * k);
#pragma unroll
    for (int i = 0; i < k; ++i) {
      const float keep = up ? x[i + k] : x[i], give = up ? x[i] : x[i + k];
      x[i] = keep + __shfl_xor_sync(~0u, give, 2 * k);
    }
  }
  return x[0] + __shfl_xor_sync(~0u, x[0], 1);
}

constexpr int GRAD_THREADS = 288;

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
    return;
  }
  if (sb & 1023u) {  // the tiles' swizzle goes by address
    if (tid == 0) atomicExch(p.status, (int)KDA_ERR_ALIGNMENT);
    return;
  }
  const int rows = seg.tokens, row0 = (int)(seg.row0 + (long long)seg.index * CHUNK);

  float* s_g = reinterpret_cast<float*>(smem + W::MISC);  // [128]: -g
  float* s_out = s_g + 128;                               // [2][128]: sums over later tokens, and of k . y, by half
  float* s_in = s_out + 256;                              // [4][128]: sums over earlier tokens, by quarter
  float* s_x = s_in + 512;                                // [2][128]: q . x, by half
  float* s_dot = s_x + 256;                               // [8]: <S, dS>, by warp
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + W::MISC + 5120);
  uint64_t *landed = bars, *clean = bars + 1, *b_done = bars + 2, *bt_done = bars + 3, *at_done = bars + 4, *x_done = bars + 5,
           *r_ready = bars + 6, *w_ready = bars + 7, *x_ready = bars + 8, *dq_done = bars + 9, *y_done = bars + 10,
           *dq_read = bars + 11, *y_ready = bars + 12, *z_done = bars + 13, *z_ready = bars + 14, *dk_done = bars + 15,
           *dv_done = bars + 16, *sums_ready = bars + 17;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 18);

  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 18; ++i) mbar_init(bars + i, 1);
    for (uint64_t* b : {clean, r_ready, w_ready, x_ready, dq_read, y_ready, z_ready, sums_ready}) mbar_init(b, 8);
    mbar_fence_init();
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

  if (warp == 8) {
    if (lane == 0) {
      // -------------------------------------------------------------- loads, then products in the order of their needs
      mbar_arrive_expect_tx(landed, 4 * W::TILE + 2 * W::IMAGE);
      for (int b = 0; b < D / 64; ++b) {
        tma_load_3d(smem + W::DO + b * W::BLOCK, &map_do, landed, 64 * b, h, row0);
        tma_load_3d(smem + W::V + b * W::BLOCK, &map_v, landed, 64 * b, h, row0);
        tma_load_3d(smem + W::Q + b * W::BLOCK, &map_q, landed, 64 * b, h, row0);
        tma_load_3d(smem + W::K + b * W::BLOCK, &map_k, landed, 64 * b, h, row0);
      }
      dependency_wait();
      const size_t image = ((size_t)slot * p.H + h) * W::IMAGE;
      bulk_g2s(smem + W::S, a.s_images + image, W::IMAGE, landed);
      bulk_g2s(smem + W::DS, a.ds_images + image, W::IMAGE, landed);
      constexpr uint32_t ID_SCORE = make_idesc_bf16(128, 128, false, false), ID_ROWS = make_idesc_bf16(128, D, false, false),
                         ID_COLS = make_idesc_bf16(128, D, false, true);
      constexpr uint32_t K_IN = 2, K_OUT = W::BLOCK >> 4, I_OUT = W::IMAGE_BLOCK >> 4, MN_IN = 128, MN_OUT = 512;
      // over channels: both operands' rows along K
      auto over_channels = [&](uint32_t to, uint32_t x, uint64_t b, uint32_t b_in, uint32_t b_out, uint32_t id) {
        const uint64_t d = desc_k(sb + x);
#pragma unroll 1
        for (int o = 0; o < D / 64; ++o)
#pragma unroll
          for (int i = 0; i < 4; ++i) umma_bf16(tb + to, d + o * K_OUT + i * K_IN, b + o * b_out + i * b_in, id, o || i ? 1u : 0u);
      };
      // over tokens: weights from tensor memory, added to what is there
      auto over_tokens = [&](uint32_t to, uint32_t weights, uint32_t x) {
        const uint64_t b = desc_mn(sb + x, W::BLOCK);
#pragma unroll 1
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int i = 0; i < 4; ++i) umma_f16_ta(tb + to, tb + weights + 64 * o + 8 * i, b + o * MN_OUT + i * MN_IN, ID_COLS, 1u);
      };
      ok = mbar_wait(landed, 0) && mbar_wait(clean, 0);
      if (ok) {
        over_channels(W::T1, W::V, desc_k(sb + W::DO), K_IN, K_OUT, ID_SCORE);
        umma_commit(bt_done);
        over_channels(W::T2, W::K, desc_k(sb + W::Q), K_IN, K_OUT, ID_SCORE);
        umma_commit(at_done);
        over_channels(W::T0, W::DO, desc_k(sb + W::V), K_IN, K_OUT, ID_SCORE);
        umma_commit(b_done);
        over_channels(W::T3, W::DO, desc_k(sb + W::S), K_IN, I_OUT, ID_ROWS);
        umma_commit(x_done);
        ok = mbar_wait(r_ready, 0) && mbar_wait(x_ready, 0);
      }
      if (ok) {
        tc_fence_after_sync();
        over_tokens(W::T3, W::T0, W::K);
        umma_commit(dq_done);
        over_channels(W::T0, W::V, desc_k(sb + W::DS), K_IN, I_OUT, ID_ROWS);  // (after the product that reads T0)
        umma_commit(y_done);
        ok = mbar_wait(dq_read, 0);
      }
      if (ok) {
        tc_fence_after_sync();
        over_channels(W::T3, W::K, desc_mn(sb + W::DS, W::IMAGE_BLOCK), MN_IN, MN_OUT, ID_COLS);
        umma_commit(z_done);
        ok = mbar_wait(w_ready, 0) && mbar_wait(y_ready, 0);
      }
      if (ok) {
        tc_fence_after_sync();
        over_tokens(W::T0, W::T1, W::Q);
        umma_commit(dk_done);
        ok = mbar_wait(z_ready, 0);
      }
      if (ok) {
        tc_fence_after_sync();
        over_tokens(W::T3, W::T2, W::DO);
        umma_commit(dv_done);
      } else {  // what has been issued ends before the CTA does
        umma_commit(dv_done);
      }
      ok = mbar_wait(dv_done, 0) && ok;
    }
  } else {
    const int quarter = warp & 3, half = warp >> 2, trow = 32 * quarter + lane;
    const uint32_t my = tb + ((uint32_t)(32 * quarter) << 16);
    const float g_mine = -s_g[trow], lead = p.scale * ex2(g_mine), trail = ex2(-s_g[127] - g_mine), keep = ex2(-s_g[127]);
    constexpr int SC = D / 2;
    const uint32_t row_at = (uint32_t)trow * 128;
    auto piece = [&](int x) { return (uint32_t)(x / 8) * W::BLOCK + row_at + (((uint32_t)(x % 8) ^ (uint32_t)(trow & 7)) << 4); };

    // half a row of an accumulator times `by`, written back; returns its product with the same half of a tile's row
    auto scale_and_dot = [&](uint32_t t, float by, uint32_t tile) {
      uint64_t sum = pair(0.f, 0.f);
#pragma unroll 1
      for (int b = 0; b < SC; b += 16) {
        float x[16];
        uint32_t u[2][4];
        tmem_ld16(my + t + half * SC + b, x);
        lds_v4(sb + tile + piece((half * SC + b) / 8), u[0]);
        lds_v4(sb + tile + piece((half * SC + b) / 8 + 1), u[1]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const uint32_t w = u[i / 8][i % 8 / 2];
          const uint64_t y = mul2(pair(x[i], x[i + 1]), pair(by, by));
          sum = fma2(y, pair(lo_f32(w), hi_f32(w)), sum);
          unpair(y, &x[i], &x[i + 1]);
        }
        tmem_st16(my + t + half * SC + b, x);
      }
      tmem_st_wait();
      tc_fence_before_sync();
      float s, z;
      unpair(sum, &s, &z);
      return s + z;
    };
    // an accumulator to memory, through this warp's part of a tile so that whole lines are written
    auto write_out = [&](uint32_t t, uint32_t tile, void* out, uint64_t* read) {
      constexpr int LANES = W::TILE / 256 / 16;  // to a row's piece of SC channels
      const uint32_t turn = sb + tile + warp * (W::TILE / 8), mine = turn + lane * (LANES * 16);
#pragma unroll 1
      for (int z = 0; z < LANES; z += 2) {
        float x[16];
        tmem_ld16(my + t + half * SC + 8 * z, x);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 2; ++i)
          st_shared_v4(mine + (((z + i) ^ (lane * LANES / 8 % LANES)) << 4), pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                       pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
      }
      tc_fence_before_sync();
      __syncwarp();
      if (read && lane == 0) mbar_arrive(read);
      uint32_t o[LANES][4];
#pragma unroll
      for (int i = 0; i < LANES; ++i) {
        const int r = i * (32 / LANES) + lane / LANES, at = lane % LANES;
        lds_v4(turn + r * (LANES * 16) + ((at ^ (r * LANES / 8 % LANES)) << 4), o[i]);
      }
      uint8_t* to = static_cast<uint8_t*>(out) + ((size_t)(row0 + 32 * quarter) * p.H + h) * D * 2 + half * D;
#pragma unroll
      for (int i = 0; i < LANES; ++i) {
        const int r = i * (32 / LANES) + lane / LANES, at = lane % LANES;
        if (32 * quarter + r < rows) *reinterpret_cast<uint4*>(to + (size_t)r * p.H * D * 2 + at * 16) = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
      }
    };

    ok = mbar_wait(landed, 0);
    if (ok) {
      if (rows < CHUNK && trow >= rows) {  // rows of other sequences
#pragma unroll 1
        for (int i = 0; i < D / 16; ++i)
          for (uint32_t tile : {W::Q, W::K, W::V, W::DO}) st_shared_v4(sb + tile + piece(half * (D / 16) + i), 0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(clean);
      // <S, dS>: 16 bytes of either at a time, wherever they belong
      float dot = 0.f;
#pragma unroll 1
      for (uint32_t i = tid * 16; i < W::IMAGE; i += 256 * 16) {
        uint32_t u[4], v[4];
        lds_v4(sb + W::S + i, u);
        lds_v4(sb + W::DS + i, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) dot = fmaf(lo_f32(u[j]), lo_f32(v[j]), fmaf(hi_f32(u[j]), hi_f32(v[j]), dot));
      }
#pragma unroll
      for (int o = 16; o; o /= 2) dot += __shfl_xor_sync(~0u, dot, o);
      if (lane == 0) s_dot[warp] = dot;
      ok = mbar_wait(bt_done, 0) && mbar_wait(at_done, 0);
    }
    if (ok) {
      // ---- R^T and P^T, earlier tokens on the lanes, 16 later ones at a time, and what a pair gives to the decays
      tc_fence_after_sync();
      float later = 0.f;
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        const int i0 = 64 * half + 16 * b;
        uint32_t u[8], v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = v[i] = 0u;
        float w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = 0.f;
        if (i0 + 15 >= 32 * quarter) {
          float x[16], y[16];
          tmem_ld16(my + W::T1 + i0, x);
          tmem_ld16(my + W::T2 + i0, y);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float d = i0 + i >= trow ? p.scale * ex2(-s_g[i0 + i] - g_mine) : 0.f;
            w[i] = i0 + i > trow ? d * x[i] * y[i] : 0.f;
            later += w[i];
            x[i] = i0 + i >= trow ? d * x[i] : 0.f;
            y[i] = i0 + i >= trow ? d * y[i] : 0.f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            u[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            v[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
          }
        }
        tmem_st8u(my + W::T1 + 64 * half + 8 * b, u);
        tmem_st8u(my + W::T2 + 64 * half + 8 * b, v);
        const float earlier = sum_lanes(w);
        if (lane % 2 == 0) s_in[quarter * 128 + i0 + lane / 2] = earlier;
      }
      s_out[half * 128 + trow] = later;
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(w_ready);
      ok = mbar_wait(b_done, 0);
    }
    if (ok) {
      // ---- R, later tokens on the lanes
      tc_fence_after_sync();
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        const int j0 = 64 * half + 16 * b;
        uint32_t u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = 0u;
        if (j0 <= 32 * quarter + 31) {
          float x[16];
          tmem_ld16(my + W::T0 + j0, x);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = j0 + j <= trow ? p.scale * ex2(g_mine + s_g[j0 + j]) * x[j] : 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
        }
        tmem_st8u(my + W::T0 + 64 * half + 8 * b, u);
      }
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(r_ready);
      ok = mbar_wait(x_done, 0);
    }
    if (ok) {
      tc_fence_after_sync();
      s_x[half * 128 + trow] = scale_and_dot(W::T3, lead, W::Q);
      __syncwarp();
      if (lane == 0) mbar_arrive(x_ready);
      ok = mbar_wait(dq_done, 0);
    }
    if (ok) {
      tc_fence_after_sync();
      write_out(W::T3, W::S, a.dq, dq_read);
      ok = mbar_wait(y_done, 0);
    }
    if (ok) {
      tc_fence_after_sync();
      s_out[half * 128 + trow] += scale_and_dot(W::T0, trail, W::K);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(y_ready);
        mbar_arrive(sums_ready);
      }
      ok = mbar_wait(z_done, 0);
    }
    if (ok) {
      tc_fence_after_sync();
#pragma unroll 1
      for (int b = 0; b < SC; b += 16) {
        float x[16];
        tmem_ld16(my + W::T3 + half * SC + b, x);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= trail;
        tmem_st16(my + W::T3 + half * SC + b, x);
      }
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(z_ready);
      // ---- the decays' gradients
      if (warp == 0 && (a.dla || a.sums) && (ok = mbar_wait(sums_ready, 0))) {
        float total = 0.f, e[4], run = 0.f, x4[4];
#pragma unroll
        for (int i = 0; i < 8; ++i) total += s_dot[i];
        total *= keep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 4 * lane + i;
          const float in = s_in[t] + s_in[128 + t] + s_in[256 + t] + s_in[384 + t];
          x4[i] = t < rows ? s_x[t] + s_x[128 + t] : 0.f;
          e[i] = run;
          run += t < rows ? s_out[t] + s_out[128 + t] - in - x4[i] : 0.f;
        }
        float all = x4[0] + x4[1] + x4[2] + x4[3], before = run;
#pragma unroll
        for (int o = 16; o; o /= 2) all += __shfl_xor_sync(~0u, all, o);
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const float x = __shfl_up_sync(~0u, before, o);
          if (lane >= o) before += x;
        }
        before = __shfl_up_sync(~0u, before, 1);
        if (lane == 0) before = 0.f;
        total += all;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 4 * lane + i;
          const float x = total + (before + e[i]);
          if (t < rows) {
            sum += x;
            const size_t at = (size_t)(row0 + t) * p.H + h;
            if (!a.sums) {
              if (p.la_f32) static_cast<float*>(a.dla)[at] = x;
              else static_cast<__nv_bfloat16*>(a.dla)[at] = __float2bfloat16_rn(x);
            }
          }
        }
        if (a.sums) {
#pragma unroll
          for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(~0u, sum, o);
          if (lane == 0) a.sums[(size_t)slot * p.H + h] = sum;
        }
      }
      ok = ok && mbar_wait(dk_done, 0);
    }
    if (ok) {
      tc_fence_after_sync();
      write_out(W::T0, W::V, a.dk, nullptr);
      ok = mbar_wait(dv_done, 0);
    }
    if (ok) {
      tc_fence_after_sync();
      write_out(W::T3, W::K, a.dv, nullptr);
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
