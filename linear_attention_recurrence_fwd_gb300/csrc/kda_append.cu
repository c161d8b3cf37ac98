// New tokens into a paged cache: keys turned by their position's angles,
// values as they are, each to the row of its page; queries turned in passing.
//
// A turn of position p by frequency f (radians per position) is the fraction
// of p f / 2 pi that is left over whole turns.  f / 2 pi is held as a 64-bit
// fixed-point fraction of a turn, so the product with the integer p wraps
// exactly and a position of 2^20 loses nothing (an fp32 angle would be off by
// 2^20 * 2^-24 radians).
//
// The call moves bytes: it is bound by HBM for prompts (65536 packed tokens of
// 32 query and 8 key heads of 128, 1.61 GB: 249 us, 6.5 TB/s) and by latency
// for single tokens (256 tokens: 4.5 us).  A CTA has 256 threads and takes 1 or
// 4 tokens at a time.  A token's sines and cosines are formed once, for all its
// heads, and kept in shared memory; the heads' first bytes are on their way
// meanwhile.  A thread takes 8 channels and the 8 that they are turned with, 16
// bytes each, and loads into their registers again at once: two such pieces are
// always on their way (loaded two by two instead: 277 us; three, with spills:
// 293; three with three CTAs on an SM instead of four: 276).
#include "kda_internal.h"
#include "kda_types.cuh"

namespace kda {
namespace {

constexpr int THREADS = 256;

// f in radians per position as a fraction of a turn, in units of 2^-64.
__device__ __forceinline__ long long turn_step(double f) {
  const double turns = f * 0.15915494309189533577;  // 1 / 2 pi
  const double frac = turns - rint(turns);          // in [-1/2, 1/2]
  return __double2ll_rn(frac * 9223372036854775808.0) << 1;  // 2^63, then times 2
}

__device__ __forceinline__ float2 turn(long long step, int pos) {
  const long long phase = (long long)((unsigned long long)step * (unsigned long long)(long long)pos);
  const float half_turns = (float)(phase >> 32) * 4.656612873077392578125e-10f;  // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c, s);
}

// The sequence of packed row t, found by a whole warp: the first n with
// cu[n + 1] > t, in steps of 32 probes; -1 where no sequence has the row.
__device__ __forceinline__ int owner_of(const int* cu, int N, int t, int lane) {
  int lo = 0, hi = N;  // n is in [lo, hi), or there is none
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int last = min(lo + (lane + 1) * step, hi) - 1;
    const unsigned past = __ballot_sync(0xffffffffu, cu[last + 1] > t);
    if (!past) return -1;
    const int k = __ffs(past) - 1;
    hi = min(lo + (k + 1) * step, hi);
    lo = min(lo + k * step, hi - 1);
    if (step == 1) break;
  }
  return lo < hi && t >= cu[lo] ? lo : -1;
}

struct Place {
  int pos;
  bool owned;     // the row has a sequence
  long long row;  // element of the token's row in the pages, or -1: not stored
};

// A token's position and its row in the pages; the page is looked up where `store`.
__device__ __forceinline__ Place place_of(const AppendProblem& p, int t, int lane, bool store) {
  Place a{0, true, -1};
  int n, i;
  if (p.cu_seqlens) {
    n = owner_of(p.cu_seqlens, p.cache.n_seq, t, lane);
    if (n < 0) return Place{0, false, -1};
    i = t - p.cu_seqlens[n];
  } else {
    n = t / p.K;
    i = t - n * p.K;
  }
  a.pos = p.cache.lens[n] + i;
  if (store && (!p.counts || i < p.counts[n]) && a.pos >= 0) {
    const int entry = a.pos / p.cache.page_size;
    if (entry < p.cache.table_width) {
      const int page = p.cache.block_table[n * p.cache.table_stride + entry];
      if (page >= 0 && page < p.cache.num_pages)
        a.row = page * p.cache.page_stride + (a.pos - entry * p.cache.page_size) * p.cache.token_stride;
    }
  }
  if (store && a.row < 0 && (!p.counts || i < p.counts[n])) *p.status = 1;
  return a;
}

// The offsets as a whole: from 0 to T, none decreasing.
__device__ __forceinline__ void check_offsets(const AppendProblem& p) {
  bool bad = p.cu_seqlens[0] != 0 || p.cu_seqlens[p.cache.n_seq] != p.T;
  for (int m = threadIdx.x; m < p.cache.n_seq; m += blockDim.x) bad |= p.cu_seqlens[m] > p.cu_seqlens[m + 1];
  if (bad) *p.status = 1;
}

// Eight 16-bit channels as fp32, and back: one rounding each.
template <typename T> __device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (__is_same(T, __nv_bfloat16)) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (__is_same(T, __nv_bfloat16)) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
// to a row of the cache or of the queries, divided by `scale`
template <typename C> __device__ __forceinline__ void store8(C* dst, float (&x)[8], float scale) {
  if (scale != 1.f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] /= scale;
  }
  if constexpr (sizeof(C) == 1) {
    C y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = from_f32<C>(x[e]);
    *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(y);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<C>(x[0], x[1]), pack2<C>(x[2], x[3]), pack2<C>(x[4], x[5]), pack2<C>(x[6], x[7]));
  }
}

// jobs: of a head, the pieces that a thread takes: 8 pairs of channels (c and
// c + rot_dim / 2), then 8 channels that are not turned; or, with neighbouring
// pairs, 8 channels each.
template <typename T, typename C, int TOKENS>
__global__ void __launch_bounds__(THREADS, 4) append_kernel(const __grid_constant__ AppendProblem p, int jobs) {
  constexpr int AHEAD = 2;  // pieces of a thread whose loads are in flight together
  __shared__ __align__(16) float2 s_turn[2][TOKENS][64];
  __shared__ long long s_row[2][TOKENS];
  __shared__ int s_owned[2][TOKENS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int d = p.cache.d, half = p.rot_dim / 2, heads = p.H_q + 2 * p.cache.H_kv;

  const int slots = THREADS / jobs, j = tid % jobs, slot = tid / jobs;
  const bool pairs_apart = !p.interleaved && half > 0;
  const bool two = pairs_apart && j < half / 8;
  const int at = two || !pairs_apart ? 8 * j : p.rot_dim + 8 * (j - half / 8);
  const int tt0 = slot / heads, h0 = slot - tt0 * heads;  // a thread's first piece of a group of tokens
  const int tt_step = slots / heads, h_step = slots - tt_step * heads;

  // the turn of a position by this thread's pair
  constexpr int WARPS = THREADS / 32, PER = WARPS / TOKENS;  // warps of a token
  const int my_token = warp / PER, part = warp % PER, pair = part * 32 + lane;
  const long long step = pair < half ? turn_step(p.inv_freq[pair]) : 0;

  uint4 a[AHEAD] = {}, b[AHEAD] = {};
  int tt, h;  // the next piece to load
  auto advance = [&](int& t, int& x) {
    t += tt_step;
    x += h_step;
    if (x >= heads) x -= heads, ++t;
  };
  auto load = [&](int t0, uint4& lo, uint4& hi) {
    const long long t = t0 + tt;
    if (tt < TOKENS && t < p.T && slot < slots) {
      const T* src = h < p.H_q ? static_cast<const T*>(p.q) + t * p.q_stride + h * d
                     : h < p.H_q + p.cache.H_kv
                         ? static_cast<const T*>(p.k) + t * p.k_stride + (h - p.H_q) * d
                         : static_cast<const T*>(p.v) + t * p.v_stride + (h - p.H_q - p.cache.H_kv) * d;
      lo = *reinterpret_cast<const uint4*>(src + at);
      if (two) hi = *reinterpret_cast<const uint4*>(src + at + half);
    }
    advance(tt, h);
  };
  if (p.cu_seqlens && blockIdx.x == 0) check_offsets(p);

  int buf = 0;
  for (int t0 = blockIdx.x * TOKENS; t0 < p.T; t0 += gridDim.x * TOKENS, buf ^= 1) {
    tt = tt0, h = h0;
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) load(t0, a[x], b[x]);
    // ---- places and turns: the CTA's warps share its tokens
    if (t0 + my_token < p.T) {
      const Place pl = place_of(p, t0 + my_token, lane, part == 0);
      if (part == 0 && lane == 0) {
        s_row[buf][my_token] = pl.row;
        s_owned[buf][my_token] = pl.owned;
        if (!pl.owned) *p.status = 1;
      }
      if (pair < half) s_turn[buf][my_token][pair] = turn(step, pl.pos);
    }
    __syncthreads();

    int ct = tt0, ch = h0;  // the piece to store
    while (ct < TOKENS && t0 + ct < p.T && slot < slots) {
#pragma unroll
      for (int x = 0; x < AHEAD; ++x) {
        if (ct >= TOKENS || t0 + ct >= p.T) break;
        const bool is_q = ch < p.H_q, is_k = !is_q && ch < p.H_q + p.cache.H_kv;
        if (__is_same(T, C) && !is_q && !is_k && p.cache.v_scale == 1.f) {  // values as they are
          if (s_row[buf][ct] >= 0) {
            T* dst = static_cast<T*>(p.cache.v) + s_row[buf][ct] + (ch - p.H_q - p.cache.H_kv) * p.cache.head_stride + at;
            *reinterpret_cast<uint4*>(dst) = a[x];
            if (two) *reinterpret_cast<uint4*>(dst + half) = b[x];
          }
          advance(ct, ch);
          load(t0, a[x], b[x]);
          continue;
        }
        float lo[8], hi[8];
        unpack8<T>(a[x], lo);
        unpack8<T>(b[x], hi);  // (read only where `two`)
        load(t0, a[x], b[x]);
        if (is_q || is_k) {
          if (two) {
            const float4* cs = reinterpret_cast<const float4*>(&s_turn[buf][ct][8 * j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 z = cs[e];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float c = y ? z.z : z.x, s = y ? z.w : z.y;
                const float r = lo[2 * e + y] * c - hi[2 * e + y] * s;
                hi[2 * e + y] = lo[2 * e + y] * s + hi[2 * e + y] * c;
                lo[2 * e + y] = r;
              }
            }
          } else if (p.interleaved) {
            const float4* cs = reinterpret_cast<const float4*>(&s_turn[buf][ct][at / 2]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float4 z = cs[e];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                if (at / 2 + 2 * e + y >= half) continue;  // not turned
                const float c = y ? z.z : z.x, s = y ? z.w : z.y;
                float &f = lo[4 * e + 2 * y], &g = lo[4 * e + 2 * y + 1];
                const float r = f * c - g * s;
                g = f * s + g * c;
                f = r;
              }
            }
          }
        }
        if (is_q) {
          if (s_owned[buf][ct]) {
            T* dst = static_cast<T*>(p.q_out) + (long long)(t0 + ct) * p.q_out_stride + ch * d + at;
            store8<T>(dst, lo, 1.f);
            if (two) store8<T>(dst + half, hi, 1.f);
          }
        } else if (s_row[buf][ct] >= 0) {
          const int hk = ch - p.H_q - (is_k ? 0 : p.cache.H_kv);
          C* dst = static_cast<C*>(is_k ? p.cache.k : p.cache.v) + s_row[buf][ct] + hk * p.cache.head_stride + at;
          const float scale = is_k ? p.cache.k_scale : p.cache.v_scale;
          store8<C>(dst, lo, scale);
          if (two) store8<C>(dst + half, hi, scale);
        }
        advance(ct, ch);
      }
    }
    // The next group's places and turns go to the other buffer; its writers have all passed this
    // group's barrier, and so are done with the one before.
  }
}

// Any number of turned channels, one pair at a time (pairs rot_dim / 2 apart
// where that is no multiple of 8: their two halves cannot be read 16 bytes at
// a time).
template <typename T, typename C>
__global__ void __launch_bounds__(128) append_pairs_kernel(const __grid_constant__ AppendProblem p) {
  const int t = blockIdx.x;
  const Place pl = place_of(p, t, threadIdx.x & 31, true);
  if (p.cu_seqlens && t == 0) check_offsets(p);
  if (!pl.owned) {
    if (threadIdx.x == 0) *p.status = 1;
    return;
  }
  const int d = p.cache.d, Hkv = p.cache.H_kv, half = p.rot_dim / 2;
  const int per_head = half + (d - p.rot_dim);  // pairs first, then the channels that are not turned
  for (int w = threadIdx.x; w < (p.H_q + 2 * Hkv) * per_head; w += blockDim.x) {
    const int head = w / per_head, j = w - head * per_head;
    const bool is_q = head < p.H_q, is_k = !is_q && head < p.H_q + Hkv;
    const int h = is_q ? head : is_k ? head - p.H_q : head - p.H_q - Hkv;
    const T* src = is_q   ? static_cast<const T*>(p.q) + t * p.q_stride
                   : is_k ? static_cast<const T*>(p.k) + t * p.k_stride
                          : static_cast<const T*>(p.v) + t * p.v_stride;
    src += h * d;
    const int a = j < half ? j : j + half, b = j < half ? j + half : a;
    float x = to_f32(src[a]), y = to_f32(src[b]);
    if (j < half && (is_q || is_k)) {
      const float2 cs = turn(turn_step(p.inv_freq[j]), pl.pos);
      const float u = x * cs.x - y * cs.y;
      y = x * cs.y + y * cs.x;
      x = u;
    }
    if (is_q) {
      T* dst = static_cast<T*>(p.q_out) + t * p.q_out_stride + h * d;
      dst[a] = from_f32<T>(x);
      if (j < half) dst[b] = from_f32<T>(y);
    } else if (pl.row >= 0) {
      C* dst = static_cast<C*>(is_k ? p.cache.k : p.cache.v) + pl.row + h * p.cache.head_stride;
      const float scale = is_k ? p.cache.k_scale : p.cache.v_scale;
      dst[a] = from_f32<C>(x / scale);
      if (j < half) dst[b] = from_f32<C>(y / scale);
    }
  }
}

template <typename T, typename C> cudaError_t launch_stored(const AppendProblem& p, cudaStream_t stream) {
  const int half = p.rot_dim / 2;
  if (!p.interleaved && half % 8) {
    append_pairs_kernel<T, C><<<p.T, 128, 0, stream>>>(p);
    return cudaGetLastError();
  }
  const int jobs = p.interleaved ? p.cache.d / 8 : half / 8 + (p.cache.d - p.rot_dim) / 8;
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // A CTA to a token while all are resident together; else as many CTAs as are, four tokens at a time.
  // 48 heads of 128: 608 tokens 5.6 us one by one and 8.1 us by four, 912 tokens 9.0 and 8.2 us, 4096
  // tokens 28 and 21 us.
  const int resident = 4 * sms;
  if (p.T <= resident)
    append_kernel<T, C, 1><<<p.T, THREADS, 0, stream>>>(p, jobs);
  else
    append_kernel<T, C, 4><<<resident, THREADS, 0, stream>>>(p, jobs);
  return cudaGetLastError();
}

template <typename T> cudaError_t launch_typed(const AppendProblem& p, cudaStream_t stream) {
  return p.cache.dtype == KDA_E4M3 ? launch_stored<T, __nv_fp8_e4m3>(p, stream) : launch_stored<T, T>(p, stream);
}

}  // namespace

cudaError_t launch_cache_append(const AppendProblem& p, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  return p.dtype == KDA_BF16 ? launch_typed<__nv_bfloat16>(p, stream) : launch_typed<__half>(p, stream);
}

}  // namespace kda
