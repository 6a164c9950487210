// Gated linear recurrence over sequences, h_t = f_t h_{t-1} + (1 - f_t) x_t
// with f = sigmoid(gate), and its gradient.
#include "head_ops.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 128;
constexpr int kChunk = SPEC_SCAN_CHUNK;

// f = sigmoid(g) and i = 1 - f = sigmoid(-g), each to fp32 accuracy.
SPEC_DEV void gate_of(float g, float& f, float& i) {
  const float e = expf(-fabsf(g));  // in (0, 1]
  const float big = 1.f / (1.f + e), small = e * big;
  f = g >= 0.f ? big : small;
  i = g >= 0.f ? small : big;
}

SPEC_DEV int len_of(const int32_t* len, int b, int T, WsHeader* hdr, bool say) {
  if (!len) return T;
  const int n = len[b];
  if (n >= 0 && n <= T) return n;
  if (say) report_error(hdr, SPEC_ERR_INVALID_ARG, SITE_NONE, b, n);
  return n < 0 ? 0 : T;
}

// One thread per channel, step by step.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_scan(spec_scan_params p, const T* __restrict__ gate, const T* __restrict__ x,
           const float* h0, const int32_t* __restrict__ len, T* h, float* h_last, float* states,
           WsHeader* hdr) {
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (e >= (int64_t)p.B * p.D) return;
  const int b = (int)(e / p.D), c = (int)(e % p.D);
  const int n = len_of(len, b, p.T, hdr, c == 0);
  const int nch = (p.T + kChunk - 1) / kChunk;
  float s = h0 ? h0[e] : 0.f;
  for (int t = 0; t < p.T; ++t) {
    if (states && t % kChunk == 0) states[((int64_t)b * nch + t / kChunk) * p.D + c] = s;
    if (t >= n) continue;
    const int64_t row = (int64_t)b * p.T + t;
    float f, i;
    gate_of(load_f(gate, row * p.gate_stride + c), f, i);
    s = fmaf(f, s, i * load_f(x, row * p.x_stride + c));
    if (h) store_f(h, row * p.h_stride + c, s);
  }
  if (h_last) h_last[e] = s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_scan_grad(spec_scan_params p, const T* __restrict__ gate, const T* __restrict__ x,
                const int32_t* __restrict__ len, const float* __restrict__ states,
                const T* __restrict__ dh, const float* dh_last, T* dgate, T* dx, float* dh0,
                WsHeader* hdr) {
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (e >= (int64_t)p.B * p.D) return;
  const int b = (int)(e / p.D), c = (int)(e % p.D);
  const int n = len_of(len, b, p.T, hdr, c == 0);
  const int nch = (p.T + kChunk - 1) / kChunk;
  float carry = dh_last ? dh_last[e] : 0.f;
  for (int ch = nch - 1; ch >= 0; --ch) {
    const int t0 = ch * kChunk;
    float s = states[((int64_t)b * nch + ch) * p.D + c];
    float f[kChunk], i[kChunk], u[kChunk];
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      if (t0 + k < n) {
        const int64_t row = (int64_t)b * p.T + t0 + k;
        gate_of(load_f(gate, row * p.gate_stride + c), f[k], i[k]);
        const float xv = load_f(x, row * p.x_stride + c);
        u[k] = s - xv;
        s = fmaf(f[k], s, i[k] * xv);
      }
    }
#pragma unroll
    for (int k = kChunk - 1; k >= 0; --k) {
      if (t0 + k >= p.T) continue;
      const int64_t row = (int64_t)b * p.T + t0 + k;
      float dg = 0.f, dxv = 0.f;
      if (t0 + k < n) {
        const float delta = carry + load_f(dh, row * p.h_stride + c);
        dxv = delta * i[k];
        dg = dxv * u[k] * f[k];
        carry = delta * f[k];
      }
      store_f(dgate, row * p.gate_stride + c, dg);
      store_f(dx, row * p.x_stride + c, dxv);
    }
  }
  if (dh0) dh0[e] = carry;
}

int grid_of(const spec_scan_params& p) {
  return (int)(((int64_t)p.B * p.D + kThreads - 1) / kThreads);
}

}  // namespace

template <typename T>
cudaError_t launch_scan(const spec_scan_params& p, const T* gate, const T* x, const float* h0,
                        const int32_t* len, T* h, float* h_last, float* states, WsHeader* hdr, int,
                        cudaStream_t st, int* launches) {
  k_scan<T><<<grid_of(p), kThreads, 0, st>>>(p, gate, x, h0, len, h, h_last, states, hdr);
  *launches = 1;
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_scan_grad(const spec_scan_params& p, const T* gate, const T* x, const float*,
                             const int32_t* len, const float* states, const T* dh,
                             const float* dh_last, T* dgate, T* dx, float* dh0, WsHeader* hdr, int,
                             cudaStream_t st, int* launches) {
  k_scan_grad<T><<<grid_of(p), kThreads, 0, st>>>(p, gate, x, len, states, dh, dh_last, dgate, dx,
                                                  dh0, hdr);
  *launches = 1;
  return cudaGetLastError();
}

#define SPEC_INST(T)                                                                               \
  template cudaError_t launch_scan<T>(const spec_scan_params&, const T*, const T*, const float*,   \
                                      const int32_t*, T*, float*, float*, WsHeader*, int,          \
                                      cudaStream_t, int*);                                         \
  template cudaError_t launch_scan_grad<T>(const spec_scan_params&, const T*, const T*,            \
                                           const float*, const int32_t*, const float*, const T*,   \
                                           const float*, T*, T*, float*, WsHeader*, int,           \
                                           cudaStream_t, int*);
SPEC_INST(float)
SPEC_INST(__nv_bfloat16)
#undef SPEC_INST

}  // namespace specdec
