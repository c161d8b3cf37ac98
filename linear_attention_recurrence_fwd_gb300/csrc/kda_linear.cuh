// What the linear attention's kernels share: a sequence's rows, a token's decay, packed arithmetic.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_internal.h"

namespace kda {

// The rows of packed sequence n: their number, and the first one.  Offsets are clamped to [0, T] and
// to an order, so that no row outside the tensors is touched whatever cu_seqlens holds.
__device__ __forceinline__ int sequence_rows(const LinearProblem& p, int n, long long* row0) {
  const int a = min(max(p.cu_seqlens[n], 0), p.T), b = min(max(p.cu_seqlens[n + 1], a), p.T);
  *row0 = a;
  return b - a;
}

// Whether the offsets of sequence n are ones that the interface allows.
__device__ __forceinline__ bool offsets_good(const LinearProblem& p, int n) {
  const int a = p.cu_seqlens[n], b = p.cu_seqlens[n + 1];
  return a >= 0 && b >= a && b <= p.T && (n > 0 || a == 0) && (n < p.n_seq - 1 || b == p.T);
}
// Flags a call whose offsets are not, once for all of its launches.
static __global__ void __launch_bounds__(256) check_offsets_kernel(LinearProblem p) {
  for (int n = threadIdx.x; n < p.n_seq; n += 256)
    if (!offsets_good(p, n)) atomicExch(p.status, (int)KDA_ERR_INVALID_ARG);
}

// A token's decay as it is stored, so that a load can be on its way for long, and what it stands for.
__device__ __forceinline__ uint32_t load_decay_bits(const LinearProblem& p, long long row, int h) {
  const long long at = row * p.la_token_stride + h * p.la_head_stride;
  return p.la_f32 ? static_cast<const uint32_t*>(p.log_alpha)[at] : static_cast<const uint16_t*>(p.log_alpha)[at];
}
__device__ __forceinline__ float decay_of_bits(const LinearProblem& p, uint32_t bits) {
  return __uint_as_float(p.la_f32 ? bits : bits << 16);
}

// Two fp32 numbers in a register pair, and what sm_100 does with both at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float* a, float* b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}

}  // namespace kda
