// Drafted tokens against the target's probabilities.
//
// Draft i is kept while u_i q_i(t_i) < p_i(t_i); the token after the kept ones
// is the first index whose running sum of weights passes u_K times their
// total, the weights being max(p_a - q_a, 0) at a draft that is not kept and
// p_a after the last.  One CTA per sequence: the total, then the 1024-wide
// stretch in which the running sum passes, then the index in it.  Sums are
// fp64: an fp32 running sum over 10^5 weights is off by about 10^-7 of the
// total, enough to change a token in every few hundred draws.
#include "kda_internal.h"
#include "kda_types.cuh"

namespace kda {
namespace {

constexpr int THREADS = 1024;

// Sum over the block; every thread gets it.  `scan` gets the inclusive sum up
// to the caller's thread.
__device__ double block_scan(double x, double* scratch, double* scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = s;
  __syncthreads();
  double before = 0., total = 0.;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) before = total;
    total += scratch[w];
  }
  *scan = before + s;
  return total;
}

template <typename T>
__global__ void __launch_bounds__(THREADS) accept_kernel(AcceptProblem p) {
  __shared__ double scratch[THREADS / 32];
  __shared__ int s_next, s_last;
  const int n = blockIdx.x, tid = threadIdx.x, K = p.K, V = p.V;
  int* tokens = p.tokens + (long long)n * (K + 1);
  const int len = p.draft_lens ? min(p.draft_lens[n], K) : K;
  if (len < 0) {
    if (tid <= K) tokens[tid] = -1;
    for (int i = THREADS + tid; i <= K; i += THREADS) tokens[i] = -1;
    if (tid == 0) p.counts[n] = 0;
    return;
  }
  const T* target = static_cast<const T*>(p.target) + n * p.target_stride_n;
  const T* draft = p.draft ? static_cast<const T*>(p.draft) + n * p.draft_stride_n : nullptr;
  const float* u = p.uniform + (long long)n * (K + 1);
  const int* toks = p.draft_tokens + (long long)n * K;
  int a = 0;
  bool bad = false;
  for (; a < len; ++a) {
    const int t = toks[a];
    bad = t < 0 || t >= V;
    if (bad) break;
    const double qt = draft ? (double)to_f32(draft[a * p.draft_stride_k + t]) : 1.;
    if (!((double)u[a] * qt < (double)to_f32(target[a * p.target_stride_k + t]))) break;
  }
  if (bad && tid == 0) *p.status = 1;
  const T* top = target + a * p.target_stride_k;
  const T* low = draft && a < len ? draft + a * p.draft_stride_k : nullptr;
  int skip = !draft && a < len ? toks[a] : -1;
  auto weight = [&](int j) -> double {
    if (j >= V || j == skip) return 0.;
    double w = (double)to_f32(top[j]);
    if (low) w -= (double)to_f32(low[j]);
    return w > 0. && w < (double)INFINITY ? w : 0.;
  };
  double total, scan;
  for (int pass = 0;; ++pass) {
    double s = 0.;
    for (int j = tid; j < V; j += THREADS) s += weight(j);
    total = block_scan(s, scratch, &scan);
    if (total > 0. || pass == 1) break;
    low = nullptr;  // no weight is positive: the target's own probabilities
    skip = -1;
  }
  if (tid == 0) s_next = V, s_last = -1;
  __syncthreads();
  const double goal = (double)u[K] * total;
  double base = 0.;
  for (int j0 = 0; j0 < V; j0 += THREADS) {
    const double w = weight(j0 + tid);
    const double sum = block_scan(w, scratch, &scan);
    if (w > 0.) {
      atomicMax(&s_last, j0 + tid);
      if (base + scan > goal) atomicMin(&s_next, j0 + tid);
    }
    __syncthreads();
    if (s_next < V) break;
    base += sum;
  }
  if (tid == 0) {
    tokens[a] = s_next < V ? s_next : s_last;
    p.counts[n] = a + 1;
  }
  for (int i = tid; i <= K; i += THREADS)
    if (i != a) tokens[i] = i < a ? toks[i] : -1;
}

}  // namespace

cudaError_t launch_draft_accept(const AcceptProblem& p, cudaStream_t stream) {
  if (p.N == 0) return cudaSuccess;
  if (p.dtype == KDA_F32)
    accept_kernel<float><<<p.N, THREADS, 0, stream>>>(p);
  else if (p.dtype == KDA_BF16)
    accept_kernel<__nv_bfloat16><<<p.N, THREADS, 0, stream>>>(p);
  else
    accept_kernel<__half><<<p.N, THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kda
