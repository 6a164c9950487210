// Vocabulary product with 4-bit weights and group scales, and the quantiser
// that lays a factor out for it.
#include "head_ops.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;

SPEC_DEV float load_any(const void* p, int32_t dtype, int64_t i) {
  return dtype == SPEC_BF16 ? load_f((const __nv_bfloat16*)p, i) : load_f((const float*)p, i);
}
SPEC_DEV void store_any(void* p, int32_t dtype, int64_t i, float v) {
  if (dtype == SPEC_BF16)
    store_f((__nv_bfloat16*)p, i, v);
  else
    store_f((float*)p, i, v);
}

// Byte of features k, k + 1 (k even) inside a packed row.
__host__ __device__ __forceinline__ int packed_byte(int k) {
  const int w = (k & 127) >> 3;  // word of eight features
  return (k >> 7) * 64 + (4 * (w & 3) + (w >> 2)) * 4 + ((k & 7) >> 1);
}

// One thread per output.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_bias_w4(spec_w4_params p, const T* __restrict__ x, const int32_t* __restrict__ prev,
              const uint8_t* __restrict__ wq, const void* __restrict__ wscale, const void* base,
              void* out, WsHeader* hdr) {
  const int v = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
  int row = b;
  if (prev) {
    row = prev[b];
    if (row < 0 || row >= p.x_rows) {
      if (v == 0) report_error(hdr, SPEC_ERR_TOKEN_RANGE, SITE_TOKEN_RANGE, b, row);
      row = row < 0 ? 0 : p.x_rows - 1;
    }
  }
  if (v >= p.V) return;
  const T* xr = x + (int64_t)row * p.x_stride;
  const uint8_t* wr = wq + (int64_t)v * ((p.r + 127) / 128 * 64);
  const int ng = p.r / p.group;
  float acc = 0.f;
  for (int g = 0; g < ng; ++g) {
    float part = 0.f;
    for (int k = g * p.group; k < (g + 1) * p.group; k += 2) {
      const int by = wr[packed_byte(k)];
      part = fmaf(load_f(xr, k), (float)((by & 15) - 8), part);
      part = fmaf(load_f(xr, k + 1), (float)((by >> 4) - 8), part);
    }
    acc = fmaf(part, load_any(wscale, p.scale_dtype, (int64_t)v * ng + g), acc);
  }
  if (base) acc += load_any(base, p.base_dtype, (int64_t)b * p.base_stride + v);
  store_any(out, p.out_dtype, (int64_t)b * p.out_stride + v, acc);
}

// One thread per token and 128 features, reading W's columns.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_w4_quantize(spec_w4_params p, const T* __restrict__ W, uint8_t* wq, void* wscale) {
  const int v = blockIdx.x * kThreads + threadIdx.x, blk = blockIdx.y;
  if (v >= p.V) return;
  uint32_t words[16];
  const int ng = p.r / p.group;
  auto at = [&](int k) {
    const float w = load_f(W, (int64_t)k * p.V + v);
    return w == w ? w : 0.f;
  };
  float scale = 0.f;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    const int k0 = blk * 128 + 8 * w;
    uint32_t word = 0x88888888u;
    if (k0 < p.r) {
      if (k0 % p.group == 0) {
        float m = 0.f;
        for (int k = k0; k < k0 + p.group; ++k) m = fmaxf(m, fabsf(at(k)));
        scale = m / 7.f;
        const int64_t si = (int64_t)v * ng + k0 / p.group;
        store_any(wscale, p.scale_dtype, si, scale);
        if (p.scale_dtype == SPEC_BF16) scale = __bfloat162float(__float2bfloat16_rn(scale));
      }
      word = 0;
      for (int j = 0; j < 8; ++j) {
        // the clamp on the quotient also takes the infinities
        const float q = scale > 0.f ? rintf(fminf(fmaxf(at(k0 + j) / scale, -8.f), 7.f)) : 0.f;
        word |= (uint32_t)((int)q + 8) << (4 * j);
      }
    }
    words[4 * (w & 3) + (w >> 2)] = word;
  }
  uint4* dst = reinterpret_cast<uint4*>(wq + (int64_t)v * ((p.r + 127) / 128 * 64) + blk * 64);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    dst[q] = make_uint4(words[4 * q], words[4 * q + 1], words[4 * q + 2], words[4 * q + 3]);
}

}  // namespace

template <typename T>
cudaError_t launch_bias_w4(const spec_w4_params& p, const T* x, const int32_t* prev,
                           const uint8_t* wq, const void* wscale, const void* base, void* out,
                           WsHeader* hdr, int, cudaStream_t st, int* launches) {
  if (p.B > 65535) return cudaErrorInvalidValue;
  k_bias_w4<T><<<dim3((p.V + kThreads - 1) / kThreads, p.B), kThreads, 0, st>>>(
      p, x, prev, wq, wscale, base, out, hdr);
  *launches = 1;
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_w4_quantize(const spec_w4_params& p, const T* W, uint8_t* wq, void* wscale,
                               cudaStream_t st) {
  k_w4_quantize<T><<<dim3((p.V + kThreads - 1) / kThreads, (p.r + 127) / 128), kThreads, 0, st>>>(
      p, W, wq, wscale);
  return cudaGetLastError();
}

#define SPEC_INST(T)                                                                               \
  template cudaError_t launch_bias_w4<T>(const spec_w4_params&, const T*, const int32_t*,          \
                                         const uint8_t*, const void*, const void*, void*,          \
                                         WsHeader*, int, cudaStream_t, int*);                      \
  template cudaError_t launch_w4_quantize<T>(const spec_w4_params&, const T*, uint8_t*, void*,     \
                                             cudaStream_t);
SPEC_INST(float)
SPEC_INST(__nv_bfloat16)
#undef SPEC_INST

}  // namespace specdec
