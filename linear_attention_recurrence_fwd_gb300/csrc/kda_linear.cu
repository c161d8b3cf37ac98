// Prompts of the linear attention: the walk in kda_linear_walk.cuh.
#include <algorithm>

#include "kda_linear_walk.cuh"

namespace kda {
namespace {

using namespace linear;

struct Plan {
  int seg_len, slots;
  bool cut;
  size_t decay_at, bytes;
};

Plan plan_for(int n_seq, int T, int H, int d, bool packed) {
  Plan a{};
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess) sms = 152;
  a.seg_len = segment_tokens(n_seq, T, H, packed, sms);
  a.slots = segment_slots(n_seq, T, a.seg_len, packed);
  a.cut = a.slots > n_seq;
  if (a.cut) {
    a.decay_at = (size_t)a.slots * H * d * d * 4;
    a.bytes = a.decay_at + ((size_t)a.slots * H * 4 + 255) / 256 * 256;
  }
  return a;
}

template <int D> cudaError_t run(const LinearProblem& p, void* workspace, cudaStream_t stream) {
  const Plan a = plan_for(p.n_seq, p.T, p.H, D, p.cu_seqlens != nullptr);
  Walk w{p, a.seg_len, std::max((p.len + a.seg_len - 1) / a.seg_len, 1), a.slots, static_cast<float*>(workspace), nullptr, nullptr};
  CUtensorMap mq, mk, mv;
  if (p.T > 0 && (!make_rows_map(&mq, p.q, p.q_stride, p) || !make_rows_map(&mk, p.k, p.k_stride, p) ||
                  !make_rows_map(&mv, p.v, p.v_stride, p)))
    return cudaErrorInvalidValue;
  if (a.cut) {
    w.decay = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + a.decay_at);
    cudaError_t e = launch(linear_walk_kernel<D, ENDS, false>, walk_ctas(w), WALK_THREADS, WalkShape<D, ENDS, false, false>::SMEM, false,
                           stream, mk, mk, mv, w);
    if (e == cudaSuccess) e = launch_scan(w, w, 1, stream);
    if (e != cudaSuccess) return e;
  }
  return p.out_f32 ? launch(linear_walk_kernel<D, OUTPUTS, true>, walk_ctas(w), WALK_THREADS, WalkShape<D, OUTPUTS, false, true>::SMEM, a.cut,
                            stream, mq, mk, mv, w)
                   : launch(linear_walk_kernel<D, OUTPUTS, false>, walk_ctas(w), WALK_THREADS, WalkShape<D, OUTPUTS, false, false>::SMEM,
                            a.cut, stream, mq, mk, mv, w);
}

}  // namespace

size_t linear_fwd_workspace_bytes(int n_seq, int T, int H, int d, bool packed) { return plan_for(n_seq, T, H, d, packed).bytes; }

cudaError_t launch_linear_fwd(const LinearProblem& p, void* workspace, cudaStream_t stream) {
  if (p.cu_seqlens) check_offsets_kernel<<<1, 256, 0, stream>>>(p);
  // Few tokens are sooner done one after the other, in one launch without tensor memory to set up.  32 heads of 128:
  // 1 sequence of 8 / 16 / 24 tokens 8.4 / 10.4 / 14.4 us against 10.3 to 11 as a chunk, 16 sequences 21 / 33 / 45
  // against 35, 128 sequences 127 / 221 / 303 against 213 to 217.  Heads of 64 have half the work in a token and more of
  // a chunk's time in its chain: 1 sequence 8.3 / 12.3 / 14.4 against 10.3, 16 sequences 10.3 / 14.4 / 18.5 against 27,
  // 128 sequences 37 / 67 / 90 (32 tokens: 120) against 168.  (Packed calls go by the rows of all sequences, as only the
  // device knows each one's: 61 sequences of 5 tokens take 137 us as a chunk each, 37 token by token.)
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  if (p.len <= (p.d == 64 && (long long)p.n_seq * p.H > 2 * sms ? 32 : 16)) return launch_linear_tokens(p, stream);
  return p.d == 128 ? run<128>(p, workspace, stream) : run<64>(p, workspace, stream);
}

}  // namespace kda
