// Gradients of the linear attention (simple form): each is the operator itself with its arguments in
// other places, two of them backwards in time.
#include "kda_linear.cuh"

namespace kda {
namespace {

struct Scan {
  const __nv_bfloat16 *a, *b, *c;  // out_t = sum over the tokens up to t (from t on) of decay (a_t . b_s) c_s
  long long a_stride, b_stride, c_stride;
  const float* start;
  bool start_transposed, back;
  float* out32;       // [T, H, d] or null
  __nv_bfloat16* out;
  float* last;        // or null
  bool last_decayed;  // once more by the first token's decay
  float scale_a, scale_b;
};

template <int D>
__global__ void __launch_bounds__(D) scan_kernel(LinearProblem p, Scan x) {
  __shared__ float s_a[D], s_b[D];
  const int c = threadIdx.x, nh = blockIdx.x, n = nh / p.H, h = nh % p.H;
  long long row0 = (long long)n * p.len;
  const int steps = p.cu_seqlens ? sequence_rows(p, n, &row0) : p.len;
  float s[D];
  const float* start = x.start ? x.start + (size_t)nh * D * D : nullptr;
#pragma unroll
  for (int i = 0; i < D; ++i) s[i] = !start ? 0.f : x.start_transposed ? start[c * D + i] : start[i * D + c];
  for (int i = 0; i < steps; ++i) {
    const long long row = row0 + (x.back ? steps - 1 - i : i);
    __syncthreads();
    s_a[c] = __bfloat162float(x.a[row * x.a_stride + h * D + c]) * x.scale_a;
    s_b[c] = __bfloat162float(x.b[row * x.b_stride + h * D + c]) * x.scale_b;
    const float v = __bfloat162float(x.c[row * x.c_stride + h * D + c]);
    const float decay = x.back && i == 0 ? 1.f : expf(load_decay(p, x.back ? row + 1 : row, h));
    __syncthreads();
    float o = 0.f;
#pragma unroll
    for (int r = 0; r < D; ++r) {
      s[r] = decay * s[r] + s_b[r] * v;
      o += s_a[r] * s[r];
    }
    if (x.out32) x.out32[(row * p.H + h) * D + c] = o;
    if (x.out) x.out[(row * p.H + h) * D + c] = __float2bfloat16_rn(o);
  }
  const float decay = x.last_decayed && steps ? expf(load_decay(p, row0, h)) : 1.f;
  if (x.last) {
#pragma unroll
    for (int i = 0; i < D; ++i) x.last[(size_t)nh * D * D + i * D + c] = decay * s[i];
  }
}

// dlog_alpha_t = <S_T, dS_T> + sum over s >= t of q_s . dq_s - k_s . dk_s
__global__ void __launch_bounds__(32) decay_grad_kernel(LinearProblem p, LinearGrads g, const float* dq, const float* dk,
                                                        const float* last_t, float* dla) {
  const int lane = threadIdx.x, nh = blockIdx.x, n = nh / p.H, h = nh % p.H, D = p.d;
  long long row0 = (long long)n * p.len;
  const int steps = p.cu_seqlens ? sequence_rows(p, n, &row0) : p.len;
  double sum = 0;
  if (g.d_final)
    for (int i = lane; i < D * D; i += 32) sum += (double)g.d_final[(size_t)nh * D * D + i] * last_t[(size_t)nh * D * D + (i % D) * D + i / D];
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  for (int i = steps - 1; i >= 0; --i) {
    const long long row = row0 + i;
    double part = 0;
    for (int c = lane; c < D; c += 32)
      part += (double)__bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[row * p.q_stride + h * D + c]) * dq[(row * p.H + h) * D + c] -
              (double)__bfloat162float(static_cast<const __nv_bfloat16*>(p.k)[row * p.k_stride + h * D + c]) * dk[(row * p.H + h) * D + c];
    for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(~0u, part, o);
    sum += part;
    if (lane == 0) dla[row * p.H + h] = (float)sum;
  }
}

__global__ void __launch_bounds__(256) decay_write_kernel(LinearProblem p, LinearGrads g, const float* dla) {
  if (g.sum_la) {
    __shared__ double s[256];
    double sum = 0;
    for (int t = threadIdx.x; t < p.T; t += 256) sum += dla[(size_t)t * p.H + blockIdx.x];
    s[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x) return;
    for (int i = 1; i < 256; ++i) sum += s[i];
    if (p.la_f32) static_cast<float*>(g.dla)[blockIdx.x] = (float)sum;
    else static_cast<__nv_bfloat16*>(g.dla)[blockIdx.x] = __float2bfloat16_rn((float)sum);
    return;
  }
  for (size_t t = threadIdx.x; t < (size_t)p.T; t += 256) {
    const size_t i = t * p.H + blockIdx.x;
    if (p.la_f32) static_cast<float*>(g.dla)[i] = dla[i];
    else static_cast<__nv_bfloat16*>(g.dla)[i] = __float2bfloat16_rn(dla[i]);
  }
}

template <int D> cudaError_t run(const LinearProblem& p, const LinearGrads& g, void* ws, cudaStream_t stream) {
  auto bf = [](const void* x) { return static_cast<const __nv_bfloat16*>(x); };
  float* dq = static_cast<float*>(ws);
  float* dk = dq + (size_t)p.T * p.H * D;
  float* last = dk + (size_t)p.T * p.H * D;
  float* dla = last + (size_t)p.n_seq * p.H * D * D;
  const unsigned blocks = (unsigned)(p.n_seq * p.H);
  auto go = [&](const Scan& x) { scan_kernel<D><<<blocks, D, 0, stream>>>(p, x); };
  go({bf(g.d_out), bf(p.v), bf(p.k), g.d_out_stride, p.v_stride, p.k_stride, p.s_in, true, false, dq, (__nv_bfloat16*)g.dq, last, false, p.scale, 1.f});
  go({bf(p.v), bf(g.d_out), bf(p.q), p.v_stride, g.d_out_stride, p.q_stride, g.d_final, true, true, dk, (__nv_bfloat16*)g.dk, nullptr, false, 1.f, p.scale});
  go({bf(p.k), bf(p.q), bf(g.d_out), p.k_stride, p.q_stride, g.d_out_stride, g.d_final, false, true, nullptr, (__nv_bfloat16*)g.dv, g.ds0, true, 1.f, p.scale});
  if (g.dla) {
    decay_grad_kernel<<<blocks, 32, 0, stream>>>(p, g, dq, dk, last, dla);
    decay_write_kernel<<<p.H, 256, 0, stream>>>(p, g, dla);
  }
  return cudaGetLastError();
}

}  // namespace

size_t linear_bwd_workspace_bytes(int n_seq, int T, int H, int d, bool) {
  return ((size_t)2 * T * H * d + (size_t)n_seq * H * d * d + (size_t)T * H) * 4;
}

cudaError_t launch_linear_bwd(const LinearProblem& p, const LinearGrads& g, void* workspace, cudaStream_t stream) {
  if (p.d == 128) return run<128>(p, g, workspace, stream);
  return run<64>(p, g, workspace, stream);
}

}  // namespace kda
