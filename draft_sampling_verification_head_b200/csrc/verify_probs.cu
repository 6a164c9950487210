// Verification of drafted tokens from probabilities and given uniforms.
#include "head_ops.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;

// A probability's mass: 0 for NaN, infinities and negative values.
SPEC_DEV double mass_of(double p) { return p > 0.0 && p < INFINITY ? p : 0.0; }

// One CTA per batch row: the accept chain, then the draw by two passes over
// the stop row (totals per thread segment, then the segment of the token).
template <typename T, typename TD>
__global__ void __launch_bounds__(kThreads)
    k_verify_probs(spec_probs_params p, const T* __restrict__ target,
                   const TD* __restrict__ draft_probs, const int32_t* __restrict__ draft,
                   const float* __restrict__ u_accept, const float* __restrict__ u_draw,
                   const int32_t* __restrict__ verify_len, int32_t* out, int32_t* tau,
                   float* p_draft, float* q_draft, WsHeader* hdr) {
  __shared__ double part[2][kThreads];
  __shared__ int stop, kb_s;
  const int b = blockIdx.x, tid = threadIdx.x, K = p.K, V = p.V;
  const T* P = target + (int64_t)b * (K + 1) * p.target_stride;
  const TD* Q = draft_probs + (int64_t)b * K * p.draft_stride;
  if (tid == 0) {
    int kb = K;
    if (verify_len) {
      kb = verify_len[b];
      if (kb > K) {
        report_error(hdr, SPEC_ERR_INVALID_ARG, SITE_NONE, b, kb);
        kb = K;
      }
    }
    int j = 0;
    bool open = true;
    for (int i = 0; i < K && kb >= 0; ++i) {
      float pv = NAN, qv = NAN;
      if (i < kb && open) {
        const int d = draft[b * (int64_t)K + i];
        if (d < 0 || d >= V) {
          report_error(hdr, SPEC_ERR_TOKEN_RANGE, SITE_TOKEN_RANGE, b * K + i, d);
          open = false;
        } else {
          pv = load_f(P, i * p.target_stride + d);
          qv = load_f(Q, i * p.draft_stride + d);
          open = (double)u_accept[b * (int64_t)K + i] * (double)qv < (double)pv;
          j += open;
        }
      }
      if (p_draft) p_draft[b * (int64_t)K + i] = pv;
      if (q_draft) q_draft[b * (int64_t)K + i] = qv;
    }
    stop = j;
    kb_s = kb;
  }
  __syncthreads();
  if (kb_s < 0) return;
  const int j = stop;
  const bool bonus = j == kb_s;
  P += j * p.target_stride;
  Q += (bonus ? 0 : j) * p.draft_stride;
  auto residual = [&](int v) {
    return mass_of((double)load_f(P, v) - (double)load_f(Q, v));
  };
  // contiguous segments, one per thread
  const int seg = (V + kThreads - 1) / kThreads;
  const int v0 = min(tid * seg, V), v1 = min(v0 + seg, V);
  double r = 0.0, t = 0.0;
  for (int v = v0; v < v1; ++v) {
    t += mass_of(load_f(P, v));
    if (!bonus) r += residual(v);
  }
  part[0][tid] = t;
  part[1][tid] = r;
  __syncthreads();
  if (tid != 0) return;
  double tot_r = 0.0, tot_t = 0.0;
  for (int k = 0; k < kThreads; ++k) {
    tot_t += part[0][k];
    tot_r += part[1][k];
  }
  const bool res = !bonus && tot_r > 0.0;
  const double total = res ? tot_r : tot_t, goal = (double)u_draw[b] * total;
  int tok = -1;
  double cum = 0.0;
  for (int k = 0; k < kThreads; ++k) {
    const double m = part[res][k];
    if (cum + m > goal) {
      double c = cum;
      int last = -1;
      for (int v = k * seg; v < min((k + 1) * seg, V); ++v) {
        const double w = res ? residual(v) : mass_of(load_f(P, v));
        if (w > 0.0) last = v;
        c += w;
        if (w > 0.0 && c > goal) break;
      }
      tok = last;
      break;
    }
    cum += m;
  }
  if (tok < 0 && total > 0.0)
    for (int v = V - 1; v >= 0 && tok < 0; --v)
      if ((res ? residual(v) : mass_of(load_f(P, v))) > 0.0) tok = v;
  if (tok < 0) report_error(hdr, SPEC_ERR_INVALID_ARG, SITE_NONE, b, j);
  for (int i = 0; i <= K; ++i)
    out[b * (int64_t)(K + 1) + i] = i < j ? draft[b * (int64_t)K + i] : i == j ? tok : -1;
  tau[b] = j + (tok >= 0);
}

}  // namespace

template <typename T, typename TD>
cudaError_t launch_verify_probs(const spec_probs_params& p, const T* target, const TD* draft_probs,
                                const int32_t* draft, const float* u_accept, const float* u_draw,
                                const int32_t* verify_len, int32_t* out, int32_t* tau,
                                float* p_draft, float* q_draft, WsHeader* hdr, int,
                                cudaStream_t st, int* launches) {
  k_verify_probs<T, TD><<<p.B, kThreads, 0, st>>>(p, target, draft_probs, draft, u_accept, u_draw,
                                                  verify_len, out, tau, p_draft, q_draft, hdr);
  *launches = 1;
  return cudaGetLastError();
}

#define SPEC_INST(T, TD)                                                                           \
  template cudaError_t launch_verify_probs<T, TD>(                                                 \
      const spec_probs_params&, const T*, const TD*, const int32_t*, const float*, const float*,   \
      const int32_t*, int32_t*, int32_t*, float*, float*, WsHeader*, int, cudaStream_t, int*);
SPEC_INST(float, float)
SPEC_INST(float, __nv_bfloat16)
SPEC_INST(__nv_bfloat16, float)
SPEC_INST(__nv_bfloat16, __nv_bfloat16)
#undef SPEC_INST

}  // namespace specdec
