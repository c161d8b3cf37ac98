// Probabilities from logits.  For each row, x = logit and then, in order,
//
//     said before:   x = x > 0 ? x / repetition : x * repetition
//     said in reply: x = x - frequency * count - presence
//     x = x + bias,   masked entries leave,   p = softmax(x / temperature)
//
// One pass: a row's entries are read once, wait in registers for the row's
// maximum and sum, and are written once as probabilities, so HBM bounds it
// (2 x 4 bytes an entry in fp32).  A cluster of up to 8 CTAs takes the rows of
// a request; CTA c holds entries [c slice, (c + 1) slice) of each.  Each warp
// takes its exponentials against its own maximum and leaves (maximum, sum) in
// every CTA's shared memory: one cluster barrier a row, and no other.
//
// Vectors of 16 bytes are read where memory has them, also where a row starts
// between two of them (an odd vocabulary): entry numbers are shifted by up to
// seven then, and what a vector holds of neighbours is left out.
//
// What has been said is counted once for a request, in shared memory, one
// 32-bit word an entry of the slice: 2 * (how often in the reply) + (whether
// in the prompt); where rows start between vectors, a word is left out after
// every 32 so that lanes 4 or 8 entries apart meet no bank twice.  The counts are whole numbers, so the order
// of the adding does not matter; a request's biases are kept in their order.  A
// row's drafts are added as the rows go by.
//
// Measured: 256 requests of 5 rows of 131072 (fp32, everything given) 332 us, floor 201; without rules 247, the mask
// adds 9, biases 18, penalties 55.  DRAM is at 51 %, issue slots at 46 %: 189 million warp instructions, 36 to each 32
// entries.  37 requests of 8 rows of 50021 in bf16 43 us, floor 9: 61 warp instructions to each 32 entries, for edges of
// rows, counts read one by one (48 us with each one's place worked out by itself), two groups of a request's rows that each
// count its history.  Where rows of logits and of probabilities start differently within 16 bytes (those 50021 entries in
// rows 50048 apart) every store is one of an entry: 71 us, without biases, where rows packed alike take 39.  One request 6.4
// to 8.4 us, dependent loads and two barriers.  Dropped: 16 entries to each of 1024 threads, with the next row's loads
// ahead (705 us without rules); sums and stores in one loop over tiles, so that the loads come once in the code (383
// us, spills).
#include <algorithm>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "kda_internal.h"
#include "kda_linear.cuh"
#include "kda_types.cuh"

namespace kda {
namespace {

constexpr int MOST = 8;      // CTAs to a cluster
constexpr int PER = 32;      // entries a thread holds
constexpr int LIST = 1024;   // biases held at a time
constexpr int NARROW = 512 * PER;   // entries that 512 threads hold
constexpr int MOST_SLICE = 51200;   // entries of a CTA's slice whose counts fit its shared memory
constexpr float LOG2E = 1.4426950408889634f;

struct __align__(16) Part { float top, sum; int at, unused; };  // of some entries: the largest, the sum against it, its lowest index

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Vectors of 16 bytes of the logits' type.
template <typename T> struct Vec { static constexpr int E = 16 / sizeof(T); };

template <typename T> __device__ __forceinline__ void unpack(const uint4& w, float* x) {
  if constexpr (sizeof(T) == 4) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  } else {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      T lo, hi;
      const uint16_t a = (uint16_t)u[i], b = (uint16_t)(u[i] >> 16);
      memcpy(&lo, &a, 2);
      memcpy(&hi, &b, 2);
      x[2 * i] = to_f32(lo);
      x[2 * i + 1] = to_f32(hi);
    }
  }
}

// E values to consecutive entries of the output, 16 bytes at a time.
template <typename O, int E> __device__ __forceinline__ void store_vec(O* to, const float* x) {
  if constexpr (sizeof(O) == 4) {
#pragma unroll
    for (int i = 0; i < E; i += 4) *reinterpret_cast<float4*>(to + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
    uint32_t u[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const O lo = from_f32<O>(x[2 * i]), hi = from_f32<O>(x[2 * i + 1]);
      uint16_t a, b;
      memcpy(&a, &lo, 2);
      memcpy(&b, &hi, 2);
      u[i] = a | (uint32_t)b << 16;
    }
    *reinterpret_cast<uint4*>(to) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// Words of shared memory for a slice's counts: where rows start between vectors, one is left out after every 32, and
// some on either side stay 0, for the entries of a vector that lie outside.
constexpr int BEFORE = 12;
template <bool EVEN> constexpr __host__ __device__ int said_words(int slice) { return EVEN ? slice : slice + slice / 32 + 2 * BEFORE; }
template <bool EVEN> constexpr size_t said_bytes(int slice) { return (size_t)((said_words<EVEN>(slice) + 3) / 4 * 4) * 4; }

// EVEN: every row starts with a vector.
template <typename T, typename O, int THREADS, bool EVEN>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) logits_kernel(LogitsProblem p, int cluster, int slice, int rows, int step) {
  namespace cg = cooperative_groups;
  constexpr int E = Vec<T>::E, TILE = THREADS * PER, WARPS = THREADS / 32;
  extern __shared__ __align__(16) uint32_t s_said[];  // [said_words], see said_at; only where something is counted
  __shared__ Part s_parts[2][MOST * WARPS];
  __shared__ int s_id[LIST];
  __shared__ float s_bias[LIST];
  __shared__ int s_listed, s_more;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster, item = blockIdx.x / cluster;
  const int groups = (p.R + rows - 1) / rows;
  const int n = item / groups, r0 = item % groups * rows, r1 = min(r0 + rows, p.R);
  const int lo = min(rank * slice, p.V), hi = min(lo + slice, p.V);
  const kda_logits_rules_t& u = p.rules;

  // ---- what this request has said, and its biases
  const bool counted = u.repetition || u.presence || u.frequency;
  auto said_at = [&](int t) { return EVEN ? t - lo : t - lo + ((t - lo) >> 5) + BEFORE; };
  if (counted) {
    const int L = u.tokens ? (u.lens ? min(max(u.lens[n], 0), u.L) : u.L) : 0;
    const int prompt = u.prompt_lens ? u.prompt_lens[n] : 0;
    const int* said = u.tokens + n * u.tokens_stride;
    // eight tokens a thread at a time, their loads on their way together, the first while the counts are cleared
    constexpr int AHEAD = 8;
    int t[AHEAD];
    auto read = [&](int i0) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) t[i] = i0 + i * THREADS < L ? said[i0 + i * THREADS] : -1;
    };
    read(tid);
    for (int i = 4 * tid; i < said_words<EVEN>(slice); i += 4 * THREADS)
      *reinterpret_cast<uint4*>(s_said + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int i0 = tid; i0 < L; i0 += AHEAD * THREADS) {
      if (i0 != tid) read(i0);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (t[i] < lo || t[i] >= hi) continue;
        if (i0 + i * THREADS < prompt) atomicOr(&s_said[said_at(t[i])], 1u);
        else atomicAdd(&s_said[said_at(t[i])], 2u);
      }
    }
    for (int i = tid; u.drafts && i < r0; i += THREADS) {
      const int t = u.drafts[(size_t)n * (p.R - 1) + i];
      if (t >= lo && t < hi) atomicAdd(&s_said[said_at(t)], 2u);
    }
  }
  const float repetition = u.repetition ? u.repetition[n] : 1.f, presence = u.presence ? u.presence[n] : 0.f;
  const float frequency = u.frequency ? u.frequency[n] : 0.f, temperature = u.temperature ? u.temperature[n] : 1.f;
  const bool greedy = !(temperature > 0.f);
  // (finite and not 0: the largest entry's 0 times it is 0, a masked one's -infinity stays)
  const float factor = greedy ? 1.f : fmaxf(fminf(LOG2E / temperature, 1e37f), 1e-37f), one_over_repetition = 1.f / repetition;
  // the biases of this slice in their order, as many as the list holds; the rest is looked up in memory
  if (warp == 0) {
    int have = 0, j0 = 0;
    for (; u.bias_ids && j0 < u.J && have <= LIST - 32; j0 += 32) {
      const int t = j0 + lane < u.J ? u.bias_ids[(size_t)n * u.J + j0 + lane] : -1;
      const bool in = t >= lo && t < hi;
      const unsigned who = __ballot_sync(~0u, in);
      if (in) {
        const int at = have + __popc(who & ((1u << lane) - 1));
        s_id[at] = t;
        s_bias[at] = u.bias[(size_t)n * u.J + j0 + lane];
      }
      have += __popc(who);
    }
    if (lane == 0) {
      s_listed = have;
      s_more = u.bias_ids ? min(j0, u.J) : 0;
    }
  }
  __syncthreads();

  const T* logits = static_cast<const T*>(p.logits) + n * p.stride_n;
  // the first entry that a tile's vectors hold: that of the vector in which entry `from` of row r lies
  auto first_of = [&](int r, int from) {
    return EVEN ? from : from - (int)((reinterpret_cast<uintptr_t>(logits + r * p.stride_r + from) & 15) / sizeof(T));
  };
  // adds b to the entry t where this thread holds it in x (vectors from `base` on).  (Going to one vector first, and
  // to its entries then, puts x into memory: 256 requests 563 us instead of 333.)
  auto add_bias = [&](float (&x)[PER], int base, int t, float b) {
    const unsigned at = t - base;
    if ((at / E & (THREADS - 1)) != tid || at >= (unsigned)TILE) return;
    const int mine = at / (E * THREADS) * E + at % E;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i == mine) x[i] += b;
  };
  // the entries [from, end) of the tile of vectors that starts at entry `base`, with everything but the
  // temperature; all others are -infinity, as masked ones are.  (Vectors past the row's end are its last ones
  // instead, so that no load waits for another.)
  auto load = [&](float (&x)[PER], int r, int base, int from, int end) {
    const T* row = logits + r * p.stride_r;
    const int* mask = u.mask ? u.mask + n * u.mask_stride_n + r * u.mask_stride_r : nullptr;
    const int last_word = (p.V - 1) >> 5;
    const bool whole = EVEN || base % 32 == 0;
    // where the vectors start with a word of the mask, the 32 words that cover the warp's entries, one to a
    // lane: E of them for each of its PER / E vectors
    uint32_t bits = 0;
    if (mask && whole) bits = mask[min(((base + (lane / E * THREADS + warp * 32) * E) >> 5) + lane % E, last_word)];
    uint4 raw[PER / E];
    // the first and the last vector that lie within the row
    const int least = base < 0 ? base + E : base, most = EVEN ? p.V - E : p.V - E - ((p.V - base) % E + E) % E;
    if (EVEN || most >= least) {
#pragma unroll
      for (int i = 0; i < PER / E; ++i)
        raw[i] = *reinterpret_cast<const uint4*>(row + min(EVEN ? base + (i * THREADS + tid) * E : max(base + (i * THREADS + tid) * E, least), most));
    } else {
#pragma unroll
      for (int i = 0; i < PER / E; ++i) raw[i] = make_uint4(0, 0, 0, 0);
    }
    if constexpr (!EVEN) {
      // those that hold something else, too, entry by entry: the one before the first, that behind the last
      const int v = (max(most, base - E) + E - base) / E;
      if ((base < 0 && tid == 0) || (v % THREADS == tid && v < TILE / E && base + v * E < p.V)) {
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          const int i0 = k ? v / THREADS : 0, at = base + (i0 * THREADS + tid) * E;
          if (k ? v % THREADS != tid || i0 >= PER / E || at >= p.V : base >= 0 || tid != 0) continue;
          uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (at + e < 0 || at + e >= p.V) continue;
            if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(to_f32(row[at + e]));
            else w[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[at + e] << (e % 2 * 16);
          }
#pragma unroll
          for (int i = 0; i < PER / E; ++i)
            if (i == i0) raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PER / E; ++i) unpack<T>(raw[i], x + i * E);
    if (counted) {
#pragma unroll
      for (int i = 0; i < PER; i += E) {
        const int at = base + (i / E * THREADS + tid) * E;
        uint32_t c[E], any = 0;
        if constexpr (EVEN) {
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            const uint4 w = at < end ? *reinterpret_cast<const uint4*>(s_said + at - lo + e) : make_uint4(0, 0, 0, 0);
            c[e] = w.x; c[e + 1] = w.y; c[e + 2] = w.z; c[e + 3] = w.w;
          }
        } else {
          // (counts of entries outside the tile do no harm: those leave below)
          const int o = min(at - lo, slice), turn = 32 - (o & 31);
          const uint32_t* here = s_said + o + (o >> 5) + BEFORE;
#pragma unroll
          for (int e = 0; e < E; ++e) c[e] = (e >= turn ? here + 1 : here)[e];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) any |= c[e];
        if (any) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float y = x[i + e] * (x[i + e] > 0.f ? one_over_repetition : repetition);
            x[i + e] = c[e] > 1 ? y - fmaf(frequency, (float)(c[e] >> 1), presence) : c[e] ? y : x[i + e];
          }
        }
      }
    }
    if (u.bias_ids) {
      // (of 32 listed ones, those that some lane of this warp holds, in their order)
      for (int j = 0; j < s_listed; j += 32) {
        const int id = j + lane < s_listed ? s_id[j + lane] : 0x7fffffff;  // (no tile's: tiles start from -7 on)
        const unsigned at = id - base;
        unsigned who = __ballot_sync(~0u, at < (unsigned)TILE && (int)(at / E & (THREADS - 1)) >> 5 == warp);
        for (; who; who &= who - 1) {
          const int i = __ffs(who) - 1;
          add_bias(x, base, s_id[j + i], s_bias[j + i]);
        }
      }
      for (int j = s_more; j < u.J; ++j) add_bias(x, base, u.bias_ids[(size_t)n * u.J + j], u.bias[(size_t)n * u.J + j]);
    }
#pragma unroll
    for (int i = 0; i < PER; i += E) {
      const int at = base + (i / E * THREADS + tid) * E;
      uint32_t word = ~0u;
      if (mask) {
        if (whole) {
          word = __shfl_sync(~0u, bits, i + lane * E / 32) >> (at & 31);
        } else {
          const int w = at >> 5;  // (rounded down, also below 0)
          word = __funnelshift_r((uint32_t)mask[min(max(w, 0), last_word)], (uint32_t)mask[min(w + 1, last_word)], at & 31);
        }
      }
      if (EVEN || (at >= from && at + E <= end)) {
        if (EVEN && at >= end) word = 0;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!(word >> e & 1)) x[i + e] = -INFINITY;
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (!(word >> e & 1) || at + e < from || at + e >= end) x[i + e] = -INFINITY;
      }
    }
  };
  // 2^((x - top) factor), 0 where x is -infinity
  auto weight = [&](float x, float top) { return exp2_fast((x - (top == -INFINITY ? 0.f : top)) * factor); };

  // all of a tile's, two at a time, and their sum
  auto weights = [&](float (&x)[PER], float top) {
    const uint64_t less = pair(top == -INFINITY ? -0.f : -top, top == -INFINITY ? -0.f : -top), by = pair(factor, factor);
    uint64_t sum = pair(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      float a, b;
      unpair(mul2(add2(pair(x[i], x[i + 1]), less), by), &a, &b);
      x[i] = exp2_fast(a);
      x[i + 1] = exp2_fast(b);
      sum = add2(sum, pair(x[i], x[i + 1]));
    }
    float a, b;
    unpair(sum, &a, &b);
    return a + b;
  };
  auto join = [&](const Part& a, const Part& b) {
    const float both = fmaxf(a.top, b.top);
    return Part{both, a.sum * weight(a.top, both) + b.sum * weight(b.top, both), b.top > a.top ? b.at : b.top == a.top ? min(a.at, b.at) : a.at, 0};
  };

  cg::cluster_group all = cg::this_cluster();
  all.sync();  // no CTA stores to one that has not started
  for (int r = r0; r < r1; ++r) {
    float x[PER];
    Part mine{-INFINITY, 0.f, 0x7fffffff, 0};
    for (int from = lo; from < hi || from == lo; from += step) {
      const int base = first_of(r, from);
      load(x, r, base, from, min(from + step, hi));
      float top = -INFINITY, sum = 0.f;
      int at = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < PER; ++i) top = fmaxf(top, x[i]);
      if (greedy) {
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) {
          if (x[i] == top && top > -INFINITY) at = min(at, base + (i / E * THREADS + tid) * E + i % E);
          if (!(x[i] < INFINITY)) sum = NAN;
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float t = __shfl_xor_sync(~0u, top, o);
        if (greedy) {
          const int a = __shfl_xor_sync(~0u, at, o);
          at = t > top ? a : t == top ? min(a, at) : at;
        }
        top = fmaxf(top, t);
      }
      if (!greedy) sum = weights(x, top);
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
      if (from == lo) mine = {top, sum, at, 0};
      else mine = join(mine, {top, sum, at, 0});
    }
    // ---- with the other warps' entries, in every CTA
    const int turn = r & 1, parts = cluster * WARPS;
    if (lane < cluster) *all.map_shared_rank(&s_parts[turn][rank * WARPS + warp], lane) = mine;
    all.sync();
    // the largest of all, then the sums against it; a lane has every 32nd part
    constexpr int MINE = MOST * WARPS / 32;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < MINE; ++i)
      if (lane + 32 * i < parts) top = fmaxf(top, s_parts[turn][lane + 32 * i].top);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    int at = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      if (lane + 32 * i >= parts) break;
      const Part q = s_parts[turn][lane + 32 * i];
      sum += q.sum * weight(q.top, top);
      if (q.top == top) at = min(at, q.at);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (greedy) {
#pragma unroll
      for (int o = 16; o; o >>= 1) at = min(at, __shfl_xor_sync(~0u, at, o));
    }
    O* to = static_cast<O*>(p.out) + ((size_t)n * p.R + r) * p.V;
    const float mul = greedy ? sum : sum > 0.f ? weight(mine.top, top) / sum : sum;
    for (int from = lo; from < hi; from += step) {
      const int base = first_of(r, from), end = min(from + step, hi);
      if (slice > step) {
        load(x, r, base, from, end);
        if (!greedy) (void)weights(x, mine.top);
      }
      const bool vec = EVEN || ((reinterpret_cast<uintptr_t>(to) + base * (long long)sizeof(O)) & 15) == 0;
#pragma unroll
      for (int i = 0; i < PER; i += E) {
        const int id = base + (i / E * THREADS + tid) * E;
        float y[E];
        if (greedy) {
#pragma unroll
          for (int e = 0; e < E; ++e) y[e] = id + e == at ? 1.f + mul : mul;
        } else {
#pragma unroll
          for (int e = 0; e < E; e += 2) unpair(mul2(pair(x[i + e], x[i + e + 1]), pair(mul, mul)), &y[e], &y[e + 1]);
        }
        if (EVEN ? id < end : vec && id >= from && id + E <= end) {
          store_vec<O, E>(to + id, y);
        } else if (!EVEN && id + E > from && id < end) {
          float z[E];  // in memory of the thread's own, so that a short loop can go through it
#pragma unroll
          for (int e = 0; e < E; ++e) z[e] = y[e];
#pragma unroll 1
          for (int e = max(from - id, 0); e < min(E, end - id); ++e) to[id + e] = from_f32<O>(z[e]);
        }
      }
    }
    if (counted && u.drafts && r + 1 < r1) {  // this row's draft has been said before the next row
      __syncthreads();
      const int t = u.drafts[(size_t)n * (p.R - 1) + r];
      if (tid == 0 && t >= lo && t < hi) s_said[said_at(t)] += 2;
      __syncthreads();
    }
  }
}

template <typename T, typename O, int THREADS, bool EVEN>
cudaError_t launch_kernel(const LogitsProblem& p, int cluster, int slice, int rows, int step, cudaStream_t stream) {
  const bool counted = p.rules.repetition || p.rules.presence || p.rules.frequency;
  const size_t smem = counted ? said_bytes<EVEN>(slice) : 0;
  auto kernel = logits_kernel<T, O, THREADS, EVEN>;
  if (smem > 32 * 1024) {
    // always to the most that a call may need: the limit is the function's, and another thread's call may be between
    // its own setting and its launch
    constexpr int MOST_BYTES = (int)said_bytes<EVEN>(THREADS == 1024 ? MOST_SLICE : NARROW);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST_BYTES);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p.N * ((p.R + rows - 1) / rows) * cluster));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)cluster, 1u, 1u};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, cluster, slice, rows, step);
}

template <typename T, typename O> cudaError_t launch_typed(const LogitsProblem& p, cudaStream_t stream) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // a tile of vectors holds up to 32 entries less than its size of a row that does not start with one
  auto in16 = [](const void* x, long long stride) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && (stride * (long long)sizeof(T)) % 16 == 0;
  };
  const bool even = in16(p.logits, p.N > 1 ? p.stride_n : 0) && in16(nullptr, p.R > 1 ? p.stride_r : 0) && p.V % Vec<T>::E == 0 &&
                    (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
  const int less = even ? 0 : 32;
  // the fewest CTAs that hold a row in registers, more while some SMs have none
  int cluster = 1;
  while (cluster < MOST && (p.V > cluster * (NARROW - less) ||
                            ((long long)p.N * p.R * cluster < sms && p.V >= cluster * 4096)))
    cluster *= 2;
  const int slice = ((p.V + cluster - 1) / cluster + 31) / 32 * 32;
  // a request's rows one after the other, its history counted once, or in as many groups as leave all CTAs
  // resident (2 on an SM): 37 requests of 8 rows, 4 CTAs each, in 1 / 2 / 4 / 8 groups 94 / 54 / 61 / 68 us; 256
  // requests of 5 rows, 8 CTAs each, in 1 / 2 / 3 / 5 groups 384 / 408 / 435 / 480
  const long long groups = std::min((long long)p.R, std::max(2LL * sms / ((long long)p.N * cluster), 1LL));
  const int rows = (int)((p.R + groups - 1) / groups);
  const bool narrow = slice <= NARROW - less;
  const int step = (narrow ? NARROW : 1024 * PER) - less;
  if (narrow && even) return launch_kernel<T, O, 512, true>(p, cluster, slice, rows, step, stream);
  if (narrow) return launch_kernel<T, O, 512, false>(p, cluster, slice, rows, step, stream);
  if (even) return launch_kernel<T, O, 1024, true>(p, cluster, slice, rows, step, stream);
  return launch_kernel<T, O, 1024, false>(p, cluster, slice, rows, step, stream);
}

}  // namespace

// The counts of a row fit the shared memory of a cluster up to here.
int logits_most_counted() { return MOST * MOST_SLICE; }

cudaError_t launch_logits_probs(const LogitsProblem& p, cudaStream_t stream) {
  if (p.N == 0 || p.R == 0) return cudaSuccess;
  const bool wide = p.out_dtype == KDA_F32;
  switch (p.dtype) {
    case KDA_F32: return launch_typed<float, float>(p, stream);
    case KDA_BF16:
      return wide ? launch_typed<__nv_bfloat16, float>(p, stream) : launch_typed<__nv_bfloat16, __nv_bfloat16>(p, stream);
    default: return wide ? launch_typed<__half, float>(p, stream) : launch_typed<__half, __half>(p, stream);
  }
}

}  // namespace kda
