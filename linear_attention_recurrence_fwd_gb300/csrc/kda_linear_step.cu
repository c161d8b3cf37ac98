// Linear attention with one decay per head, token after token.  For each
// (sequence, head), with a = exp(log_alpha):
//
//     S = a S + k v^T,     o = scale S^T q
//
// The state stays in registers while a sequence's tokens pass, so a call
// reads it once and writes it once (or not at all, for a verification): 128 KiB
// (d = 128) against 1 KiB of activations a token.  HBM bounds it.
//
// A CTA of 128 threads takes 64 value columns of one (sequence, head): thread
// t holds columns [4 j, 4 j + 4) (j = t % 16) of the key rows [R g, R g + R)
// (g = t / 16, R = d / 8), so that a warp's load covers two 256-byte pieces of
// rows.  Unlike the delta rule's step nothing is subtracted from v, so no
// token waits for a sum over the rows of its predecessor: the row groups'
// parts of KT tokens' outputs are left in shared memory and added up together,
// one barrier for KT tokens.
//
// Measured (32 heads of 128): one token for 256 requests 158 us, 6.8 TB/s, the
// copy bandwidth; five tokens of 61 requests 38 us to verify (140 MB) and 43 to
// commit (264 MB, 6.1 TB/s); one request 4.3 us.  KT of 2, 4, 5, 6 and 8 gave
// 43, 41, 38, 39 and 43 us for the verification, a launch bound of four CTAs on
// an SM 55 us for the commit (spills).  (KT is chosen at these sizes alone; eight
// tokens, as five and three, take 58 us to verify.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int COLS = 64, GROUPS = 8;

template <int D, int KT, typename OutT>
__global__ void __launch_bounds__(128) linear_tokens_kernel(LinearProblem p) {
  constexpr int R = D / GROUPS, PARTS = D / COLS;
  __shared__ __align__(16) float s_k[KT][D], s_q[KT][D], s_v[KT][COLS];
  __shared__ __align__(16) float s_part[KT][GROUPS][COLS];
  __shared__ float s_a[KT];

  const int tid = threadIdx.x;
  const int nh = blockIdx.x / PARTS, part = blockIdx.x % PARTS;
  const int n = nh / p.H, h = nh - n * p.H;
  long long row0 = (long long)n * p.len;
  int steps = p.len;
  if (p.cu_seqlens) steps = sequence_rows(p, n, &row0);
  if (p.counts) steps = min(max(p.counts[n], 0), steps);

  const int j = tid % 16, g = tid / 16;
  const size_t off = (size_t)nh * D * D + part * COLS + 4 * j;
  ulonglong2 s[R];  // four columns of a row, as pairs
#pragma unroll
  for (int i = 0; i < R; ++i)
    s[i] = p.s_in ? *reinterpret_cast<const ulonglong2*>(p.s_in + off + (size_t)(g * R + i) * D) : make_ulonglong2(0, 0);

  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + h * D;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + h * D;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + h * D + part * COLS;
  OutT* out = static_cast<OutT*>(p.out);

  for (int t0 = 0; t0 < steps; t0 += KT) {
    const int nt = min(KT, steps - t0);
    if (t0) __syncthreads();  // the previous tokens' readers are done
    // all loads of the KT tokens together (past the last one that one again)
    __nv_bfloat16 rk[KT], rq[KT], rv[KT];
    uint32_t ra[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const long long row = row0 + t0 + min(t, nt - 1);
      if (tid < D) rk[t] = k[row * p.k_stride + tid];
      if (tid < D && out) rq[t] = q[row * p.q_stride + tid];
      if (tid < COLS) rv[t] = v[row * p.v_stride + tid];
      if (tid == 127) ra[t] = load_decay_bits(p, row, h);
    }
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      if (tid < D) s_k[t][tid] = __bfloat162float(rk[t]);
      if (tid < D && out) s_q[t][tid] = __bfloat162float(rq[t]);
      if (tid < COLS) s_v[t][tid] = __bfloat162float(rv[t]);
      if (tid == 127) s_a[t] = expf(decay_of_bits(p, ra[t]));
    }
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
      const uint64_t a = pair(s_a[t], s_a[t]);
      const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&s_v[t][4 * j]);
      ulonglong2 b = make_ulonglong2(0, 0);
#pragma unroll
      for (int i0 = 0; i0 < R; i0 += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(&s_k[t][g * R + i0]);
        const float kc[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ulonglong2& y = s[i0 + i];
          const uint64_t k2 = pair(kc[i], kc[i]);
          y.x = fma2(a, y.x, mul2(k2, x.x));
          y.y = fma2(a, y.y, mul2(k2, x.y));
        }
        if (out) {
          const float4 q4 = *reinterpret_cast<const float4*>(&s_q[t][g * R + i0]);
          const float qc[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t q2 = pair(qc[i], qc[i]);
            b.x = fma2(s[i0 + i].x, q2, b.x);
            b.y = fma2(s[i0 + i].y, q2, b.y);
          }
        }
      }
      if (out) *reinterpret_cast<ulonglong2*>(&s_part[t][g][4 * j]) = b;
    }
    if (out) {
      __syncthreads();
      for (int i = tid; i < nt * COLS; i += 128) {
        const int t = i / COLS, c = i % COLS;
        float o = 0.f;
#pragma unroll
        for (int r = 0; r < GROUPS; ++r) o += s_part[t][r][c];
        store_out(out + ((row0 + t0 + t) * p.H + h) * D + part * COLS + c, p.scale * o);
      }
    }
  }
  if (p.s_out) {
#pragma unroll
    for (int i = 0; i < R; ++i) *reinterpret_cast<ulonglong2*>(p.s_out + off + (size_t)(g * R + i) * D) = s[i];
  }
}

template <int D, int KT>
cudaError_t launch_typed(const LinearProblem& p, cudaStream_t stream) {
  const unsigned blocks = (unsigned)((long long)p.n_seq * p.H * (D / COLS));
  if (p.out && !p.out_f32) linear_tokens_kernel<D, KT, __nv_bfloat16><<<blocks, 128, 0, stream>>>(p);
  else linear_tokens_kernel<D, KT, float><<<blocks, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_tokens(const LinearProblem& p, cudaStream_t stream) {
  if (p.n_seq == 0 || p.H == 0) return cudaSuccess;
  if (p.d == 128) return p.len == 1 ? launch_typed<128, 1>(p, stream) : launch_typed<128, 5>(p, stream);
  return p.len == 1 ? launch_typed<64, 1>(p, stream) : launch_typed<64, 5>(p, stream);
}

}  // namespace kda
