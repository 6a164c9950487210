// Interfaces between the entry points of the head's operators (head_api.cu)
// and their kernels, and the device helpers those share.
#pragma once

#include "common.cuh"

namespace specdec {

// ---- Shared by the entry points (api.cu) ------------------------------------------
extern thread_local int32_t g_last_launches;  // kernel launches of the thread's last call
int num_sms();                                // SMs of the current device, 0 on an error
// Whether a runtime call succeeded.  An error is taken off the runtime's last one:
// the call that met it reports it, and no later launch must.
bool cuda_ok(cudaError_t e);

// Record a device-side error of an operator: the first one stays.  Unlike
// record_error this leaves the abort flag alone, which ends the waits of the
// launches that have barriers of the grid (the cycle's, the gradient's sort).
SPEC_DEV void report_error(WsHeader* h, int32_t code, int32_t site, int32_t a, int32_t b) {
  if (atomicCAS(&h->status, 0, code) == 0) {
    h->err_where = site;
    h->err_a = a;
    h->err_b = b;
  }
}

// Element stores: fp32 as it is, bf16 rounded to nearest even.
SPEC_DEV void store_f(float* p, int64_t i, float v) { p[i] = v; }
SPEC_DEV void store_f(__nv_bfloat16* p, int64_t i, float v) { p[i] = __float2bfloat16_rn(v); }

// A launch that was allowed to start early waits here for the one before it;
// a kernel lets the launch after it start early.
SPEC_DEV void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
SPEC_DEV void grid_dependency_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launch a kernel and return that launch's own error: the runtime's last one may
// be an earlier call's.
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem,
                          cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// The same for a kernel that calls grid_dependency_wait before it touches anything
// the launch before it writes: its CTAs may be set up while that one ends.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem,
                         cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// ---- Scaled lookup and its gradient -------------------------------------------
size_t embed_grad_ws_bytes(const spec_embed_params& p);
template <typename TT, typename TR>
cudaError_t launch_embed(const spec_embed_params& p, const TT* table, const int32_t* ids, TR* rows,
                         WsHeader* hdr, int num_sms, cudaStream_t st, int* launches);
template <typename TT, typename TR>
cudaError_t launch_embed_grad(const spec_embed_params& p, const int32_t* ids, const TR* drows,
                              TT* dtable, uint8_t* body, WsHeader* hdr, int num_sms,
                              cudaStream_t st, int* launches);

// ---- Gated linear recurrence and its gradient -------------------------------------
size_t scan_ws_bytes(const spec_scan_params& p, int num_sms);
void set_scan_polls(int64_t polls);
template <typename T>
cudaError_t launch_scan(const spec_scan_params& p, const T* gate, const T* x, const float* h0,
                        const int32_t* len, T* h, float* h_last, float* states, uint8_t* body,
                        WsHeader* hdr, int num_sms, cudaStream_t st, int* launches);
template <typename T>
cudaError_t launch_scan_grad(const spec_scan_params& p, const T* gate, const T* x, const float* h0,
                             const int32_t* len, const float* states, const T* dh,
                             const float* dh_last, T* dgate, T* dx, float* dh0, uint8_t* body,
                             WsHeader* hdr, int num_sms, cudaStream_t st, int* launches);

// ---- Vocabulary product with 4-bit weights ------------------------------------------
size_t w4_ws_bytes(const spec_w4_params& p);
template <typename T>
cudaError_t launch_bias_w4(const spec_w4_params& p, const T* x, const int32_t* prev,
                           const uint8_t* wq, const void* wscale, const void* base, void* out,
                           uint8_t* body, WsHeader* hdr, int num_sms, cudaStream_t st,
                           int* launches);
template <typename T>
cudaError_t launch_w4_quantize(const spec_w4_params& p, const T* W, uint8_t* wq, void* wscale,
                               cudaStream_t st);

// ---- Verification from probabilities ---------------------------------------------------
template <typename T, typename TD>
cudaError_t launch_verify_probs(const spec_probs_params& p, const T* target, const TD* draft_probs,
                                const int32_t* draft, const float* u_accept, const float* u_draw,
                                const int32_t* verify_len, int32_t* out, int32_t* tau,
                                float* p_draft, float* q_draft, WsHeader* hdr, int num_sms,
                                cudaStream_t st, int* launches);

}  // namespace specdec
