// New tokens into a paged cache: keys turned by their position's angles,
// values as they are, each to the row of its page; queries turned in passing.
//
// A turn of position p by frequency f (radians per position) is the fraction
// of p f / 2 pi that is left over whole turns.  f / 2 pi is held as a 64-bit
// fixed-point fraction of a turn, so the product with the integer p wraps
// exactly and a position of 2^20 loses nothing (an fp32 angle would be off by
// 2^20 * 2^-24 radians).
#include "kda_internal.h"
#include "kda_types.cuh"

namespace kda {
namespace {

// f in radians per position as a fraction of a turn, in units of 2^-64.
__device__ __forceinline__ long long turn_step(double f) {
  const double turns = f * 0.15915494309189533577;  // 1 / 2 pi
  const double frac = turns - rint(turns);          // in [-1/2, 1/2]
  return __double2ll_rn(frac * 9223372036854775808.0) << 1;  // 2^63, then times 2
}

__device__ __forceinline__ void turn(long long step, int pos, float* c, float* s) {
  const long long phase = (long long)((unsigned long long)step * (unsigned long long)(long long)pos);
  const float half_turns = (float)(phase >> 32) * 4.656612873077392578125e-10f;  // 2^-31
  sincospif(half_turns, s, c);
}

template <typename T, typename C>
__global__ void __launch_bounds__(128) append_kernel(AppendProblem p) {
  const int t = blockIdx.x;
  // the token's sequence n and its number i in it
  int n, i;
  bool owned = true;
  if (p.cu_seqlens) {
    if (t == 0) {  // the offsets as a whole: from 0 to T, none decreasing
      bool bad = p.cu_seqlens[0] != 0 || p.cu_seqlens[p.cache.n_seq] != p.T;
      for (int m = threadIdx.x; m < p.cache.n_seq; m += blockDim.x)
        bad |= p.cu_seqlens[m] > p.cu_seqlens[m + 1];
      if (bad) *p.status = 1;
    }
    int lo = 0, hi = p.cache.n_seq;  // the first n with cu[n + 1] > t
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.cu_seqlens[mid + 1] > t) hi = mid; else lo = mid + 1;
    }
    n = lo;
    owned = n < p.cache.n_seq && t >= p.cu_seqlens[n];
    i = owned ? t - p.cu_seqlens[n] : 0;
    if (!owned) {
      if (threadIdx.x == 0) *p.status = 1;
      return;
    }
  } else {
    n = t / p.K;
    i = t - n * p.K;
  }
  const int pos = p.cache.lens[n] + i;
  const bool real = !p.counts || i < p.counts[n];
  long long row = -1;
  if (real) {
    if (pos >= 0 && pos / p.cache.page_size < p.cache.table_width) {
      const int page = p.cache.block_table[n * p.cache.table_stride + pos / p.cache.page_size];
      if (page >= 0 && page < p.cache.num_pages)
        row = page * p.cache.page_stride + (pos % p.cache.page_size) * p.cache.token_stride;
    }
    if (row < 0 && threadIdx.x == 0) *p.status = 1;
  }
  const int d = p.cache.d, Hkv = p.cache.H_kv;
  const int half = p.rot_dim / 2, rest = d - p.rot_dim;
  // pairs first, then the channels that are not turned
  const int per_head = half + rest;
  for (int w = threadIdx.x; w < (p.H_q + 2 * Hkv) * per_head; w += blockDim.x) {
    const int head = w / per_head, j = w - head * per_head;
    const bool is_q = head < p.H_q, is_k = !is_q && head < p.H_q + Hkv;
    const int h = is_q ? head : is_k ? head - p.H_q : head - p.H_q - Hkv;
    const T* src = is_q   ? static_cast<const T*>(p.q) + t * p.q_stride
                   : is_k ? static_cast<const T*>(p.k) + t * p.k_stride
                          : static_cast<const T*>(p.v) + t * p.v_stride;
    src += h * d;
    const int a = j < half ? (p.interleaved ? 2 * j : j) : j + half;
    const int b = j < half ? (p.interleaved ? 2 * j + 1 : j + half) : a;
    float x = to_f32(src[a]), y = to_f32(src[b]);
    if (j < half && (is_q || is_k)) {
      float c, s;
      turn(turn_step(p.inv_freq[j]), pos, &c, &s);
      const float u = x * c - y * s;
      y = x * s + y * c;
      x = u;
    }
    if (is_q) {
      T* dst = static_cast<T*>(p.q_out) + t * p.q_out_stride + h * d;
      dst[a] = from_f32<T>(x);
      if (j < half) dst[b] = from_f32<T>(y);
    } else if (row >= 0) {
      C* dst = static_cast<C*>(is_k ? p.cache.k : p.cache.v) + row + h * p.cache.head_stride;
      const float scale = is_k ? p.cache.k_scale : p.cache.v_scale;
      dst[a] = from_f32<C>(x / scale);
      if (j < half) dst[b] = from_f32<C>(y / scale);
    }
  }
}

template <typename T>
cudaError_t launch_typed(const AppendProblem& p, cudaStream_t stream) {
  if (p.cache.dtype == KDA_E4M3)
    append_kernel<T, __nv_fp8_e4m3><<<p.T, 128, 0, stream>>>(p);
  else
    append_kernel<T, T><<<p.T, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const AppendProblem& p, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  return p.dtype == KDA_BF16 ? launch_typed<__nv_bfloat16>(p, stream)
                             : launch_typed<__half>(p, stream);
}

}  // namespace kda
