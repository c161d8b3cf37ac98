// Drafted tokens against the target's probabilities.
//
// Draft i is kept while u_i q_i(t_i) < p_i(t_i); the token after the kept ones
// is the first index whose running sum of weights passes u_K times their
// total, the weights being max(p_a - q_a, 0) at a draft that is not kept and
// p_a after the last.
//
// The call reads one row of p and, for a rejected draft, one of q: it is bound
// by HBM for many sequences and by latency for few.  A cluster of 1 to 8 CTAs
// takes a sequence and each of its warps a contiguous slice of the vocabulary.
// The slices' sums meet in every CTA's shared memory; the CTA whose slice
// holds the border sums that slice again in 256 contiguous pieces, and one
// warp looks through the piece that holds it, out of L2.  256 sequences of
// 131072 fp32 entries: 48 us, 4.5 TB/s; one of 32768: 5.8 us.
//
// Sums: an fp32 running sum over 10^5 weights is off by about 10^-7 of the
// total, enough to change a token in every few hundred draws, and fp64 runs at
// a 64th of fp32's rate here (40 such instructions in every warp were a third
// of the call).  All sums are therefore pairs of fp32 numbers (hi + lo, with
// the exact error of every difference and sum; Knuth's two-sum), which hold 48
// bits.
#include "kda_internal.h"
#include "kda_types.cuh"

namespace kda {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32, MOST = 8;  // CTAs of a cluster

struct Row {
  const void* top;  // the target's probabilities
  const void* low;  // the draft model's, or null
  int skip;         // an entry without weight, or -1
};

// A number as hi + lo, hi the sum rounded to fp32.
struct Pair {
  float hi = 0.f, lo = 0.f;
};
__device__ __forceinline__ Pair normal(float hi, float lo) {
  const float s = hi + lo;
  return Pair{s, lo - (s - hi)};
}
__device__ __forceinline__ Pair operator+(const Pair& a, const Pair& b) {
  const float s = a.hi + b.hi, z = s - a.hi;
  return normal(s, ((a.hi - (s - z)) + (b.hi - z)) + (a.lo + b.lo));
}
__device__ __forceinline__ Pair operator*(float u, const Pair& a) {
  const float x = u * a.hi;
  return normal(x, fmaf(u, a.lo, fmaf(u, a.hi, -x)));
}
__device__ __forceinline__ bool operator>(const Pair& a, const Pair& b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
__device__ __forceinline__ Pair shfl(const Pair& a, int lane) {
  return Pair{__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}
__device__ __forceinline__ Pair shfl_up(const Pair& a, int by) {
  return Pair{__shfl_up_sync(0xffffffffu, a.hi, by), __shfl_up_sync(0xffffffffu, a.lo, by)};
}
__device__ __forceinline__ Pair shfl_xor(const Pair& a, int by) {
  return Pair{__shfl_xor_sync(0xffffffffu, a.hi, by), __shfl_xor_sync(0xffffffffu, a.lo, by)};
}

// The weight of an entry: max(p - q, 0), exactly; 0 where it is not finite.
template <typename T> __device__ __forceinline__ Pair weight(const Row& r, int j) {
  const float p = to_f32(static_cast<const T*>(r.top)[j]), q = r.low ? to_f32(static_cast<const T*>(r.low)[j]) : 0.f;
  const float x = p - q, z = x - p;
  return x > 0.f && x < INFINITY && j != r.skip ? Pair{x, (p - (x - z)) - (q + z)} : Pair{};
}

// Two fp32 numbers in a register pair, and their sums and differences.
__device__ __forceinline__ uint64_t pack(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
// Two sums, each of two fp32 numbers; what is added is x + e, |e| far below |x|.
struct Sum2 {
  uint64_t hi = 0, lo = 0;
  __device__ __forceinline__ void add(uint64_t x, uint64_t e) {
    const uint64_t t = add2(hi, x), z = sub2(t, hi);
    lo = add2(lo, add2(add2(sub2(hi, sub2(t, z)), sub2(x, z)), e));
    hi = t;
  }
  // the weights max(p - q, 0) of two entries, exactly; 0 where one is not finite
  __device__ __forceinline__ void add(float p0, float p1, float q0, float q1) {
    const uint64_t p = pack(p0, p1), q = pack(q0, q1);
    const uint64_t x = sub2(p, q), z = sub2(x, p), e = sub2(sub2(p, sub2(x, z)), add2(q, z));
    float x0, x1, e0, e1;
    unpack(x, x0, x1);
    unpack(e, e0, e1);
    // positive and finite: bits 1 to 0x7f7fffff
    const bool ok0 = __float_as_uint(x0) - 1u < 0x7f7fffffu, ok1 = __float_as_uint(x1) - 1u < 0x7f7fffffu;
    add(pack(ok0 ? x0 : 0.f, ok1 ? x1 : 0.f), pack(ok0 ? e0 : 0.f, ok1 ? e1 : 0.f));
  }
  __device__ __forceinline__ Pair value() const {
    float a, b, c, d;
    unpack(hi, a, b);
    unpack(lo, c, d);
    return normal(a, c) + normal(b, d);
  }
};

// This lane's share of the weights of [j0, j1), 16 bytes at a time; the next
// bytes are on their way while these are summed.
template <typename T> __device__ __forceinline__ Pair sum_vectors(const Row& r, int j0, int j1, int lane) {
  constexpr int VE = 16 / sizeof(T), AHEAD = 2, STEP = 32 * VE * AHEAD;
  Sum2 s;
  uint4 a[2][AHEAD], b[2][AHEAD];
  const T* top = static_cast<const T*>(r.top);
  const T* low = static_cast<const T*>(r.low);
  auto load = [&](int buf, int j) {
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
      const int at = j + x * 32 * VE;
      a[buf][x] = b[buf][x] = make_uint4(0, 0, 0, 0);
      if (at < j1) {
        a[buf][x] = *reinterpret_cast<const uint4*>(top + at);
        if (low) b[buf][x] = *reinterpret_cast<const uint4*>(low + at);
      }
    }
  };
  auto sum = [&](int buf, int j) {
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
      T* p = reinterpret_cast<T*>(&a[buf][x]);
      const T* q = reinterpret_cast<const T*>(&b[buf][x]);
      const int at = j + x * 32 * VE;
      const int skip = r.skip - at;  // an entry of these without weight
#pragma unroll
      for (int e = 0; e < VE; e += 2)
        s.add(skip == e ? 0.f : to_f32(p[e]), skip == e + 1 ? 0.f : to_f32(p[e + 1]), to_f32(q[e]), to_f32(q[e + 1]));
    }
  };
  int j = j0 + lane * VE;
  if (j < j1) load(0, j);
  for (; j < j1; j += 2 * STEP) {
    load(1, j + STEP);
    sum(0, j);
    load(0, j + 2 * STEP);
    sum(1, j + STEP);
  }
  return s.value();
}

// The same, one entry at a time (rows that do not start on 16 bytes), `step` apart from j0 on; AHEAD
// loads are on their way together.
template <int AHEAD, typename T> __device__ __forceinline__ Pair sum_entries(const Row& r, int j0, int j1, int step) {
  Sum2 s;
  for (int j = j0; j < j1; j += step * AHEAD) {
    float a[AHEAD], b[AHEAD];
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) {
      const int at = j + x * step;
      a[x] = b[x] = 0.f;
      if (at < j1) {
        a[x] = to_f32(static_cast<const T*>(r.top)[at]);
        if (r.low) b[x] = to_f32(static_cast<const T*>(r.low)[at]);
        if (at == r.skip) a[x] = 0.f;
      }
    }
#pragma unroll
    for (int x = 0; x < AHEAD; x += 2) s.add(a[x], a[x + 1], b[x], b[x + 1]);
  }
  return s.value();
}

__device__ __forceinline__ Pair warp_scan(Pair s, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y = shfl_up(s, o);
    if (lane >= o) s = s + y;
  }
  return s;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// (relaxed: nothing written before is for the others)
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// stores x at the place of `local` in the shared memory of the cluster's CTA `rank`
__device__ __forceinline__ void store_remote(const Pair* local, uint32_t rank, const Pair& x) {
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(local));
  asm volatile("{.reg .u32 r; mapa.shared::cluster.u32 r, %0, %1; st.shared::cluster.v2.f32 [r], {%2, %3};}" ::"r"(at), "r"(rank),
               "f"(x.hi), "f"(x.lo) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 4) accept_kernel(const __grid_constant__ AcceptProblem p, int cluster) {
  __shared__ __align__(8) float2 s_slices[2][MOST * WARPS];  // the slices' sums, for each of two attempts
  __shared__ float2 s_warps[WARPS];
  __shared__ int s_next;
  Pair(*const s_slice)[MOST * WARPS] = reinterpret_cast<Pair(*)[MOST * WARPS]>(s_slices);
  Pair* const s_warp = reinterpret_cast<Pair*>(s_warps);
  const int rank = cluster == 1 ? 0 : (int)cluster_rank();
  // Another CTA's shared memory exists once that CTA has started: all arrive here, and wait before
  // their first store to it (the drafts' test and the sums lie in between).
  if (cluster > 1) cluster_started();
  const int n = blockIdx.x / cluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = p.K, V = p.V;
  int* tokens = p.tokens + (long long)n * (K + 1);
  const int* toks = p.draft_tokens + (long long)n * K;
  const float* u = p.uniform + (long long)n * (K + 1);
  const T* target = static_cast<const T*>(p.target) + n * p.target_stride_n;
  const T* draft = p.draft ? static_cast<const T*>(p.draft) + n * p.draft_stride_n : nullptr;
  const int len = p.draft_lens ? min(p.draft_lens[n], K) : K;
  const float u_last = u[K];

  // ---- the first draft that is not kept: every warp looks at 32 drafts at a time
  int a = 0;
  bool bad = false;
  for (int i0 = 0; i0 < K; i0 += 32) {
    const int i = i0 + lane;
    bool ok = false, outside = false;
    if (i < K) {
      const int t = toks[i];
      outside = t < 0 || t >= V;
      if (!outside) {
        const float qt = draft ? to_f32(draft[i * p.draft_stride_k + t]) : 1.f, pt = to_f32(target[i * p.target_stride_k + t]);
        // u q < p for the exact product: its rounding error is exact too, unless it falls below 2^-149
        const float uq = u[i] * qt;
        ok = uq < pt || (uq == pt && fmaf(u[i], qt, -uq) < 0.f);
        if (uq < 0x1p-100f) ok = (double)u[i] * (double)qt < (double)pt;
      }
    }
    const unsigned stop = __ballot_sync(0xffffffffu, !ok || i >= len);
    a = i0 + (stop ? __ffs(stop) - 1 : 32);
    bad = stop && __shfl_sync(0xffffffffu, outside, stop ? __ffs(stop) - 1 : 0) && a < len;
    if (stop) break;
  }
  if (len < 0) {  // an idle sequence: the same for the whole cluster
    if (cluster > 1) cluster_wait();
    if (rank == 0) {
      for (int i = tid; i <= K; i += THREADS) tokens[i] = -1;
      if (tid == 0) p.counts[n] = 0;
    }
    return;
  }
  a = min(a, len);
  if (bad && tid == 0) *p.status = 1;
  Row row;
  row.top = target + a * p.target_stride_k;
  row.low = draft && a < len ? draft + a * p.draft_stride_k : nullptr;
  row.skip = !draft && a < len ? toks[a] : -1;

  // ---- slices of 256 E entries, one for each warp of the cluster
  const int slices = cluster * WARPS, mine = rank * WARPS + warp;
  const int E = (V + slices * THREADS - 1) / (slices * THREADS);
  const int L = E * THREADS;
  const auto odd = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) != 0; };
  const bool vectors = !odd(row.top) && !(row.low && odd(row.low)) && V % (16 / sizeof(T)) == 0;
  Pair goal, before;
  int slice = -1;
  for (int attempt = 0; attempt < 2; ++attempt) {
    const int j0 = (int)min((long long)mine * L, (long long)V), j1 = (int)min((long long)j0 + L, (long long)V);
    Pair total = vectors ? sum_vectors<T>(row, j0, j1, lane) : sum_entries<8, T>(row, j0 + lane, j1, 32);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total = total + shfl_xor(total, o);
    if (cluster == 1) {
      if (lane == 0) s_slice[attempt][mine] = total;
      __syncthreads();
    } else {
      if (attempt == 0) cluster_wait();  // all of the cluster's CTAs have started
      if (lane < cluster) store_remote(&s_slice[attempt][mine], lane, total);
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    }
    // every warp finds the slice that holds the border: the first whose running sum passes the goal
    const Pair x = lane * 2 < slices ? s_slice[attempt][lane * 2] : Pair{}, y = lane * 2 + 1 < slices ? s_slice[attempt][lane * 2 + 1] : Pair{};
    const Pair end = warp_scan(x + y, lane);       // after slice 2 lane + 1
    const Pair start = shfl_up(end, 1);
    const Pair first = lane ? start : Pair{};      // before slice 2 lane
    const Pair middle = first + x;
    const Pair all = shfl(end, 31);
    if (!(all.hi > 0.f)) {
      if (!row.low && row.skip < 0) break;
      row.low = nullptr;  // no weight is positive: the target's own probabilities
      row.skip = -1;
      continue;
    }
    goal = u_last * all;
    const unsigned in_x = __ballot_sync(0xffffffffu, x.hi > 0.f && middle > goal);
    const unsigned in_y = __ballot_sync(0xffffffffu, y.hi > 0.f && end > goal);
    const int kx = in_x ? __ffs(in_x) - 1 : 32, ky = in_y ? __ffs(in_y) - 1 : 32;
    if (kx == 32 && ky == 32) {  // rounding (or u = 1): the last slice that has weight
      const unsigned has_x = __ballot_sync(0xffffffffu, x.hi > 0.f), has_y = __ballot_sync(0xffffffffu, y.hi > 0.f);
      const int lx = has_x ? 31 - __clz(has_x) : -1, ly = has_y ? 31 - __clz(has_y) : -1;
      slice = ly >= lx ? 2 * ly + 1 : 2 * lx;
    } else {
      slice = kx <= ky ? 2 * kx : 2 * ky + 1;
    }
    before = shfl(slice & 1 ? middle : first, slice >> 1);
    break;
  }
  // all of the cluster's shared memory has been written: its CTAs go on alone
  if (slice >= 0 ? slice / WARPS != rank : rank != 0) return;

  // ---- the slice in 256 contiguous pieces, then the piece
  int next = -1;
  if (slice >= 0) {
    const long long s0 = (long long)slice * L;
    const int j0 = (int)min(s0 + tid * E, (long long)V), j1 = (int)min((long long)j0 + E, (long long)V);
    // (pieces of few entries: loads past a piece's end are not free)
    const Pair mine_sum = E <= 2   ? sum_entries<2, T>(row, j0, j1, 1)
                          : E <= 4 ? sum_entries<4, T>(row, j0, j1, 1)
                                   : sum_entries<8, T>(row, j0, j1, 1);
    const Pair scan = warp_scan(mine_sum, lane);
    if (tid == 0) s_next = -1;
    if (lane == 31) s_warp[warp] = scan;
    __syncthreads();
    Pair base = before;
    for (int w = 0; w < warp; ++w) base = base + s_warp[w];
    const Pair to_here = shfl_up(scan, 1), from = lane ? base + to_here : base;  // before this piece
    // the first piece that passes the goal, or else (rounding) the last that has weight: candidates
    // are numbered so that one maximum decides
    const bool passes = mine_sum.hi > 0.f && base + scan > goal;
    if (mine_sum.hi > 0.f) atomicMax(&s_next, passes ? 2 * THREADS - tid : tid);
    __syncthreads();
    const int piece = s_next >= THREADS ? 2 * THREADS - s_next : s_next;
    if (piece >= 0 && piece / 32 == warp) {
      Pair run = shfl(from, piece & 31);
      const int p0 = (int)min(s0 + (long long)piece * E, (long long)V), p1 = (int)min((long long)p0 + E, (long long)V);
      int last = -1;
      for (int q0 = p0; q0 < p1 && next < 0; q0 += 32) {
        const Pair w = q0 + lane < p1 ? weight<T>(row, q0 + lane) : Pair{};
        const Pair sum = run + warp_scan(w, lane);
        const unsigned pass = __ballot_sync(0xffffffffu, w.hi > 0.f && sum > goal), has = __ballot_sync(0xffffffffu, w.hi > 0.f);
        if (pass) next = q0 + __ffs(pass) - 1;
        if (has) last = q0 + 31 - __clz(has);
        run = shfl(sum, 31);
      }
      if (next < 0) next = last;
      if (lane == 0) {
        tokens[a] = next;
        p.counts[n] = a + 1;
      }
    }
  } else if (tid == 0) {
    tokens[a] = -1;
    p.counts[n] = a + 1;
  }
  for (int i = tid; i <= K; i += THREADS)
    if (i != a) tokens[i] = i < a ? toks[i] : -1;
}

template <typename T> cudaError_t launch_typed(const AcceptProblem& p, cudaStream_t stream) {
  // As many CTAs to a sequence as make two rounds of the resident ones (4 on an SM), while each has
  // at least 1024 entries.  Two rounds, because a sequence that keeps all its drafts reads one row and
  // the others two: 256 sequences of 131072 fp32 entries take 65 us with 2 CTAs each (all resident),
  // 48 us with 4 and 50 us with 8.
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  int cluster = MOST;
  while (cluster > 1 && ((long long)p.N * cluster > 8LL * sms || p.V < 1024 * cluster)) cluster /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.N * cluster);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)cluster, 1u, 1u};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, accept_kernel<T>, p, cluster);
}

}  // namespace

cudaError_t launch_draft_accept(const AcceptProblem& p, cudaStream_t stream) {
  if (p.N == 0) return cudaSuccess;
  switch (p.dtype) {
    case KDA_F32: return launch_typed<float>(p, stream);
    case KDA_BF16: return launch_typed<__nv_bfloat16>(p, stream);
    default: return launch_typed<__half>(p, stream);
  }
}

}  // namespace kda
