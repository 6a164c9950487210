// C-ABI entry points of the head's operators (include/specdec.h): argument
// validation on the host, then the launch.  No allocation happens here.
#include <climits>
#include <cmath>
#include <cstdio>

#include "head_ops.cuh"
#include "specdec_debug.h"

namespace specdec {
namespace {

bool is_dtype(int32_t t) { return t == SPEC_F32 || t == SPEC_BF16; }

// Element pointers are aligned to their elements.
bool aligned_to(const void* p, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == SPEC_BF16 ? 1u : 3u)) == 0;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A stride of 0 means dense; any other covers the row.
bool good_stride(int64_t s, int64_t width) { return s == 0 || (s >= width && s <= INT_MAX); }

bool good_workspace(const void* ws) {
  return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0;
}

WsHeader* header_of(void* ws) { return reinterpret_cast<WsHeader*>(ws); }
uint8_t* body_of(void* ws) { return reinterpret_cast<uint8_t*>(ws) + sizeof(WsHeader); }

spec_status launched(cudaError_t e, int launches) {
  g_last_launches = launches;
  if (cuda_ok(e)) return SPEC_OK;
  fprintf(stderr, "specdec: launch failed: %s\n", cudaGetErrorString(e));
  return SPEC_ERR_CUDA;
}

spec_status check_embed(const spec_embed_params* p, spec_embed_params* d) {
  if (!p || p->n < 0 || p->V < 1 || p->D < 1 || p->D > 65536 || !is_dtype(p->dtype) ||
      !is_dtype(p->row_dtype) || (p->accumulate != 0 && p->accumulate != 1) ||
      !std::isfinite(p->scale) || p->reserved != 0 || !good_stride(p->table_stride, p->D) ||
      !good_stride(p->row_stride, p->D))
    return SPEC_ERR_INVALID_ARG;
  if (p->n > (1 << 30)) return SPEC_ERR_UNSUPPORTED;  // ends of pieces fit 32 bits
  *d = *p;
  if (d->table_stride == 0) d->table_stride = d->D;
  if (d->row_stride == 0) d->row_stride = d->D;
  return SPEC_OK;
}

spec_status check_scan(const spec_scan_params* p, spec_scan_params* d) {
  if (!p || p->B < 1 || p->T < 0 || p->D < 1 || !is_dtype(p->dtype) ||
      !good_stride(p->gate_stride, p->D) || !good_stride(p->x_stride, p->D) ||
      !good_stride(p->h_stride, p->D))
    return SPEC_ERR_INVALID_ARG;
  if ((int64_t)p->B * p->D > INT_MAX || p->T > INT_MAX - 65536) return SPEC_ERR_UNSUPPORTED;
  *d = *p;
  if (d->gate_stride == 0) d->gate_stride = d->D;
  if (d->x_stride == 0) d->x_stride = d->D;
  if (d->h_stride == 0) d->h_stride = d->D;
  return SPEC_OK;
}

spec_status check_w4(const spec_w4_params* p, spec_w4_params* d) {
  if (!p || p->B < 1 || p->r < 1 || p->r > 65536 || p->V < 1 || !is_dtype(p->dtype) ||
      !is_dtype(p->scale_dtype) || !is_dtype(p->base_dtype) || !is_dtype(p->out_dtype) ||
      p->reserved != 0 || !good_stride(p->x_stride, p->r) || !good_stride(p->base_stride, p->V) ||
      !good_stride(p->out_stride, p->V))
    return SPEC_ERR_INVALID_ARG;
  if (p->B > (1 << 16) || p->V > (1 << 30)) return SPEC_ERR_UNSUPPORTED;  // grid and index limits
  if ((p->group != 32 && p->group != 64 && p->group != 128) || p->r % p->group != 0) {
    fprintf(stderr, "specdec: 4-bit weights come in groups of 32, 64 or 128 features that divide "
                    "the rank\n");
    return SPEC_ERR_UNSUPPORTED;
  }
  *d = *p;
  if (d->x_stride == 0) d->x_stride = d->r;
  if (d->base_stride == 0) d->base_stride = d->V;
  if (d->out_stride == 0) d->out_stride = d->V;
  return SPEC_OK;
}

spec_status check_probs(const spec_probs_params* p, spec_probs_params* d) {
  if (!p || p->B < 1 || p->K < 1 || p->K > 1024 || p->V < 1 || !is_dtype(p->dtype) ||
      !is_dtype(p->draft_dtype) || p->reserved != 0 || !good_stride(p->target_stride, p->V) ||
      !good_stride(p->draft_stride, p->V))
    return SPEC_ERR_INVALID_ARG;
  if (p->V > (1 << 30)) return SPEC_ERR_UNSUPPORTED;  // token indices of a tile fit 32 bits
  *d = *p;
  if (d->target_stride == 0) d->target_stride = d->V;
  if (d->draft_stride == 0) d->draft_stride = d->V;
  return SPEC_OK;
}

template <typename F>
cudaError_t by_dtypes(int32_t a, int32_t b, F f) {
  const float* f32 = nullptr;
  const __nv_bfloat16* b16 = nullptr;
  if (a == SPEC_BF16) return b == SPEC_BF16 ? f(b16, b16) : f(b16, f32);
  return b == SPEC_BF16 ? f(f32, b16) : f(f32, f32);
}
template <typename P>
using Elem = std::remove_const_t<std::remove_pointer_t<P>>;

}  // namespace
}  // namespace specdec

using namespace specdec;

extern "C" {

size_t spec_embed_workspace_size(const spec_embed_params* p) {
  spec_embed_params d;
  if (check_embed(p, &d) != SPEC_OK) return 0;
  return (sizeof(WsHeader) + embed_grad_ws_bytes(d) + 255) & ~size_t(255);
}

spec_status spec_embed(const spec_embed_params* p, const void* table, const int32_t* ids,
                       void* rows, void* ws, spec_stream_t stream) {
  g_last_launches = 0;
  spec_embed_params d;
  const spec_status s = check_embed(p, &d);
  if (s != SPEC_OK) return s;
  if (!good_workspace(ws)) return SPEC_ERR_WORKSPACE;
  if (d.n == 0) return SPEC_OK;
  if (!table || !ids || !rows || !aligned_to(table, d.dtype) || !aligned_to(rows, d.row_dtype) ||
      !aligned4(ids))
    return SPEC_ERR_INVALID_ARG;
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  int launches = 0;
  const cudaError_t e = by_dtypes(d.dtype, d.row_dtype, [&](auto tt, auto tr) {
    using TT = Elem<decltype(tt)>;
    using TR = Elem<decltype(tr)>;
    return launch_embed<TT, TR>(d, (const TT*)table, ids, (TR*)rows, header_of(ws), sms,
                                (cudaStream_t)stream, &launches);
  });
  return launched(e, launches);
}

spec_status spec_embed_grad(const spec_embed_params* p, const int32_t* ids, const void* drows,
                            void* dtable, void* ws, spec_stream_t stream) {
  g_last_launches = 0;
  spec_embed_params d;
  const spec_status s = check_embed(p, &d);
  if (s != SPEC_OK) return s;
  if (!good_workspace(ws)) return SPEC_ERR_WORKSPACE;
  if (d.n == 0 && d.accumulate) return SPEC_OK;
  if (!dtable || !aligned_to(dtable, d.dtype)) return SPEC_ERR_INVALID_ARG;
  if (d.n > 0 && (!ids || !drows || !aligned_to(drows, d.row_dtype) || !aligned4(ids)))
    return SPEC_ERR_INVALID_ARG;
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  int launches = 0;
  const cudaError_t e = by_dtypes(d.dtype, d.row_dtype, [&](auto tt, auto tr) {
    using TT = Elem<decltype(tt)>;
    using TR = Elem<decltype(tr)>;
    return launch_embed_grad<TT, TR>(d, ids, (const TR*)drows, (TT*)dtable, body_of(ws),
                                     header_of(ws), sms, (cudaStream_t)stream, &launches);
  });
  return launched(e, launches);
}

size_t spec_scan_workspace_size(const spec_scan_params* p) {
  spec_scan_params d;
  if (check_scan(p, &d) != SPEC_OK) return 0;
  const int sms = num_sms();
  if (sms <= 0) return 0;
  return (sizeof(WsHeader) + scan_ws_bytes(d, sms) + 255) & ~size_t(255);
}

spec_status spec_gated_scan(const spec_scan_params* p, const void* gate, const void* x,
                            const float* h0, const int32_t* len, void* h, float* h_last,
                            float* states, void* ws, spec_stream_t stream) {
  g_last_launches = 0;
  spec_scan_params d;
  const spec_status s = check_scan(p, &d);
  if (s != SPEC_OK) return s;
  if (!good_workspace(ws)) return SPEC_ERR_WORKSPACE;
  // no steps: h and states have no element, so their pointers may be NULL
  if (d.T > 0 && (!gate || !x || (!h && !h_last && !states))) return SPEC_ERR_INVALID_ARG;
  if (!aligned_to(gate, d.dtype) || !aligned_to(x, d.dtype) || !aligned_to(h, d.dtype) ||
      !aligned4(h0) || !aligned4(h_last) || !aligned4(states) || !aligned4(len))
    return SPEC_ERR_INVALID_ARG;
  if (d.T == 0 && !h_last) return SPEC_OK;
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  int launches = 0;
  const cudaError_t e =
      d.dtype == SPEC_BF16
          ? launch_scan(d, (const __nv_bfloat16*)gate, (const __nv_bfloat16*)x, h0, len,
                        (__nv_bfloat16*)h, h_last, states, body_of(ws), header_of(ws), sms,
                        (cudaStream_t)stream, &launches)
          : launch_scan(d, (const float*)gate, (const float*)x, h0, len, (float*)h, h_last, states,
                        body_of(ws), header_of(ws), sms, (cudaStream_t)stream, &launches);
  return launched(e, launches);
}

spec_status spec_gated_scan_grad(const spec_scan_params* p, const void* gate, const void* x,
                                 const float* h0, const int32_t* len, const float* states,
                                 const void* dh, const float* dh_last, void* dgate, void* dx,
                                 float* dh0, void* ws, spec_stream_t stream) {
  g_last_launches = 0;
  spec_scan_params d;
  const spec_status s = check_scan(p, &d);
  if (s != SPEC_OK) return s;
  if (!good_workspace(ws)) return SPEC_ERR_WORKSPACE;
  if (d.T > 0 && (!gate || !x || !states || !dh || !dgate || !dx)) return SPEC_ERR_INVALID_ARG;
  if (!aligned_to(gate, d.dtype) || !aligned_to(x, d.dtype) || !aligned_to(dh, d.dtype) ||
      !aligned_to(dgate, d.dtype) || !aligned_to(dx, d.dtype) || !aligned4(h0) ||
      !aligned4(dh_last) || !aligned4(dh0) || !aligned4(states) || !aligned4(len))
    return SPEC_ERR_INVALID_ARG;
  if (d.T == 0 && !dh0) return SPEC_OK;
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  int launches = 0;
  const cudaError_t e =
      d.dtype == SPEC_BF16
          ? launch_scan_grad(d, (const __nv_bfloat16*)gate, (const __nv_bfloat16*)x, h0, len,
                             states, (const __nv_bfloat16*)dh, dh_last, (__nv_bfloat16*)dgate,
                             (__nv_bfloat16*)dx, dh0, body_of(ws), header_of(ws), sms, (cudaStream_t)stream,
                             &launches)
          : launch_scan_grad(d, (const float*)gate, (const float*)x, h0, len, states,
                             (const float*)dh, dh_last, (float*)dgate, (float*)dx, dh0,
                             body_of(ws), header_of(ws), sms, (cudaStream_t)stream, &launches);
  return launched(e, launches);
}

spec_status spec_debug_scan_polls(int64_t polls) {
  set_scan_polls(polls);
  return SPEC_OK;
}

size_t spec_w4_workspace_size(const spec_w4_params* p) {
  spec_w4_params d;
  if (check_w4(p, &d) != SPEC_OK) return 0;
  return (sizeof(WsHeader) + w4_ws_bytes(d) + 255) & ~size_t(255);
}

spec_status spec_bias_w4(const spec_w4_params* p, const void* x, const int32_t* prev,
                         const void* wq, const void* wscale, const void* base, void* out, void* ws,
                         spec_stream_t stream) {
  g_last_launches = 0;
  spec_w4_params d;
  const spec_status s = check_w4(p, &d);
  if (s != SPEC_OK) return s;
  if (!x || !wq || !wscale || !out || (prev && d.x_rows < 1)) return SPEC_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(wq) & 15u) || !aligned_to(x, d.dtype) ||
      !aligned_to(wscale, d.scale_dtype) || !aligned_to(base, d.base_dtype) ||
      !aligned_to(out, d.out_dtype) || !aligned4(prev))
    return SPEC_ERR_INVALID_ARG;
  if (!good_workspace(ws)) return SPEC_ERR_WORKSPACE;
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  int launches = 0;
  const cudaError_t e =
      d.dtype == SPEC_BF16
          ? launch_bias_w4(d, (const __nv_bfloat16*)x, prev, (const uint8_t*)wq, wscale, base, out,
                           body_of(ws), header_of(ws), sms, (cudaStream_t)stream, &launches)
          : launch_bias_w4(d, (const float*)x, prev, (const uint8_t*)wq, wscale, base, out,
                           body_of(ws), header_of(ws), sms, (cudaStream_t)stream, &launches);
  return launched(e, launches);
}

spec_status spec_w4_quantize(const spec_w4_params* p, const void* W, int32_t w_dtype, void* wq,
                             void* wscale, spec_stream_t stream) {
  g_last_launches = 0;
  spec_w4_params d;
  const spec_status s = check_w4(p, &d);
  if (s != SPEC_OK) return s;
  if (!W || !wq || !wscale || !is_dtype(w_dtype) || !aligned_to(W, w_dtype) ||
      (reinterpret_cast<uintptr_t>(wq) & 15u) || !aligned_to(wscale, d.scale_dtype))
    return SPEC_ERR_INVALID_ARG;
  const cudaError_t e =
      w_dtype == SPEC_BF16
          ? launch_w4_quantize(d, (const __nv_bfloat16*)W, (uint8_t*)wq, wscale,
                               (cudaStream_t)stream)
          : launch_w4_quantize(d, (const float*)W, (uint8_t*)wq, wscale, (cudaStream_t)stream);
  return launched(e, 1);
}

spec_status spec_verify_probs(const spec_probs_params* p, const void* target,
                              const void* draft_probs, const int32_t* draft,
                              const float* u_accept, const float* u_draw,
                              const int32_t* verify_len, int32_t* out, int32_t* tau,
                              float* p_draft, float* q_draft, void* ws, spec_stream_t stream) {
  g_last_launches = 0;
  spec_probs_params d;
  const spec_status s = check_probs(p, &d);
  if (s != SPEC_OK) return s;
  if (!target || !draft_probs || !draft || !u_accept || !u_draw || !out || !tau)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned_to(target, d.dtype) || !aligned_to(draft_probs, d.draft_dtype) ||
      !aligned4(draft) || !aligned4(u_accept) || !aligned4(u_draw) || !aligned4(verify_len) ||
      !aligned4(out) || !aligned4(tau) || !aligned4(p_draft) || !aligned4(q_draft))
    return SPEC_ERR_INVALID_ARG;
  if (!good_workspace(ws)) return SPEC_ERR_WORKSPACE;
  const int sms = num_sms();
  if (sms <= 0) return SPEC_ERR_CUDA;
  int launches = 0;
  const cudaError_t e = by_dtypes(d.dtype, d.draft_dtype, [&](auto tp, auto tq) {
    using T = Elem<decltype(tp)>;
    using TD = Elem<decltype(tq)>;
    return launch_verify_probs<T, TD>(d, (const T*)target, (const TD*)draft_probs, draft, u_accept,
                                      u_draw, verify_len, out, tau, p_draft, q_draft,
                                      header_of(ws), sms, (cudaStream_t)stream, &launches);
  });
  return launched(e, launches);
}

}  // extern "C"
