// Vocabulary product with 4-bit weights and group scales, and the quantiser
// that lays a factor out for it.
#include <algorithm>

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

// ----------------------------------------------------------------------------
// The product.  A warp multiplies MT tiles of 16 tokens by up to 8 NT columns of
// X on the tensor cores (m16n8k16, bf16 in, fp32 out).  Codes become bf16
// exactly (0x4300 | code is 128 + code, less 136); a lane's 16 bytes of a row
// hold one word of each 32 features, so the multiply of a group needs no other
// lane's bytes, and the order of the features inside a word is given to X instead
// (a nibble and the one 16 bits above it make a pair).  The sum of a group stays
// in the accumulator, is scaled in fp32 and added to the row's.  fp32 X is cut
// into three bf16 parts, which together hold all its 24 bits, as columns of
// their own, so its products are exact as well.
//
// Bytes bound it: the codes pass through once.  The features are split over up
// to 8 warps of a CTA, which keeps its tail short, and joined in order in shared
// memory.
// ----------------------------------------------------------------------------
constexpr int kWarps = kThreads / 32;

SPEC_DEV void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight codes as four pairs (k, k + 4) of bf16.
SPEC_DEV void codes_to_bf16(uint32_t w, uint32_t* p) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t u = ((w >> (4 * k)) & 0x000F000Fu) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p[k]) : "r"(u), "r"(0x43084308u));  // 136
  }
}

SPEC_DEV uint4 load_once(const uint8_t* p) {
  uint4 w;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p));
  return w;
}
SPEC_DEV uint32_t part_of(const uint4& w, int i) {
  return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
}

// Eight features of one row of X, as pairs (k, k + 4): bf16, or part s (0 the
// leading one) of an fp32.
SPEC_DEV void x_pairs(const __nv_bfloat16* x, bool wide, int, uint32_t* b) {
  uint32_t u[4];
  if (wide) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(x));
    u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
  } else {
    const unsigned short* h = reinterpret_cast<const unsigned short*>(x);
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = (uint32_t)__ldg(h + 2 * k) | (uint32_t)__ldg(h + 2 * k + 1) << 16;
  }
  b[0] = __byte_perm(u[0], u[2], 0x5410);
  b[1] = __byte_perm(u[0], u[2], 0x7632);
  b[2] = __byte_perm(u[1], u[3], 0x5410);
  b[3] = __byte_perm(u[1], u[3], 0x7632);
}
SPEC_DEV void x_pairs(const float* x, bool wide, int s, uint32_t* b) {
  float v[8];
  if (wide) {
    const float4 lo = __ldg(reinterpret_cast<const float4*>(x));
    const float4 hi = __ldg(reinterpret_cast<const float4*>(x) + 1);
    v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
    v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __ldg(x + k);
  }
  uint32_t part[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t bits = __float_as_uint(v[k]);
    const bool finite = (bits & 0x7F800000u) != 0x7F800000u;
    // cutting keeps the leading 8 bits; the rest is exact, and so is its rest
    const float r1 = v[k] - __uint_as_float(bits & 0xFFFF0000u);
    const float r2 = r1 - __uint_as_float(__float_as_uint(r1) & 0xFFFF0000u);
    const uint32_t head = finite || (bits & 0x007FFFFFu) == 0 ? bits : 0x7FC00000u;
    const uint32_t tail = __float_as_uint(s == 1 ? r1 : r2);
    part[k] = s == 0 ? head : finite ? tail : 0u;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) b[k] = __byte_perm(part[k], part[k + 4], 0x7632);
}

template <typename T, int NT, int MT>
__global__ void __launch_bounds__(kThreads, MT == 4 ? 1 : 2)
    k_bias_w4(spec_w4_params p, const T* __restrict__ x, const int32_t* __restrict__ prev,
              const uint8_t* __restrict__ wq, const void* __restrict__ wscale, const void* base,
              void* out, int split, int wide, WsHeader* hdr) {
  constexpr int kParts = sizeof(T) == 4 ? 3 : 1;    // columns per row of X
  constexpr int kRows = 8 * NT / kParts < 16 ? 8 * NT / kParts : 16;
  constexpr int kTokens = 16 * MT, kPitch = kTokens + 4;
  extern __shared__ float red[];  // [warp][column][kPitch]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int ks = warp % split, rg = warp / split;
  const int64_t v0 = ((int64_t)blockIdx.x * (kWarps / split) + rg) * kTokens;
  const int b0 = blockIdx.y * kRows, nb = min(kRows, p.B - b0);
  const int nkb = (p.r + 127) / 128, kb0 = nkb * ks / split, kb1 = nkb * (ks + 1) / split;
  const int rowb = nkb * 64, ng = p.r / p.group;

  // this lane's columns of X
  const T* xr[NT];
  bool has[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int b = (nt * 8 + g) / kParts;
    has[nt] = b < nb;
    int row = has[nt] ? b0 + b : b0;
    if (prev) {
      row = __ldg(prev + row);
      if (row < 0 || row >= p.x_rows) {
        if (blockIdx.x == 0 && warp == 0 && has[nt])
          report_error(hdr, SPEC_ERR_TOKEN_RANGE, SITE_TOKEN_RANGE, b0 + b, row);
        row = row < 0 ? 0 : p.x_rows - 1;
      }
    }
    xr[nt] = x + (int64_t)row * p.x_stride + 8 * t4;
  }

  float total[MT][NT][4] = {};
  if (v0 < p.V) {
    const int last = (int)min((int64_t)kTokens, p.V - v0) - 1;
    const uint8_t* w0 = wq + v0 * rowb + t4 * 16;
    int at[MT][2];  // rows of the tile, the ones past the vocabulary read its last
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      at[mt][0] = min(mt * 16 + g, last);
      at[mt][1] = min(mt * 16 + g + 8, last);
    }
    uint4 cur[MT][2], nxt[MT][2];
    float sc[MT][2], sn[MT][2];
    const int per = 128 / p.group;  // groups per block; lane t4 holds the scale of group t4 % per
    auto request = [&](int kb, uint4 (&w)[MT][2], float (&s)[MT][2]) {
      const int gi = min(kb * per + t4 % per, ng - 1);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[mt][h] = load_once(w0 + (int64_t)at[mt][h] * rowb + kb * 64);
          s[mt][h] = load_any(wscale, p.scale_dtype, (v0 + at[mt][h]) * ng + gi);
        }
    };
    if (kb0 < kb1) request(kb0, cur, sc);
    for (int kb = kb0; kb < kb1; ++kb) {
      if (kb + 1 < kb1) request(kb + 1, nxt, sn);
      float acc[MT][NT][4] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = kb * 128 + 32 * i;
        if (k < p.r) {
          uint32_t xb[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (has[nt])
              x_pairs(xr[nt] + k, wide, (nt * 8 + g) % kParts, xb[nt]);
            else
              xb[nt][0] = xb[nt][1] = xb[nt][2] = xb[nt][3] = 0u;
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t lo[4], hi[4];
            codes_to_bf16(part_of(cur[mt][0], i), lo);
            codes_to_bf16(part_of(cur[mt][1], i), hi);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_bf16(acc[mt][nt], lo[0], hi[0], lo[1], hi[1], xb[nt][0], xb[nt][1]);
              mma_bf16(acc[mt][nt], lo[2], hi[2], lo[3], hi[3], xb[nt][2], xb[nt][3]);
            }
          }
          if ((32 * (i + 1)) % p.group == 0) {  // a group ends
            const int from = (lane & ~3) + 32 * i / p.group;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const float s0 = __shfl_sync(0xffffffffu, sc[mt][0], from);
              const float s1 = __shfl_sync(0xffffffffu, sc[mt][1], from);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                total[mt][nt][0] = fmaf(s0, acc[mt][nt][0], total[mt][nt][0]);
                total[mt][nt][1] = fmaf(s0, acc[mt][nt][1], total[mt][nt][1]);
                total[mt][nt][2] = fmaf(s1, acc[mt][nt][2], total[mt][nt][2]);
                total[mt][nt][3] = fmaf(s1, acc[mt][nt][3], total[mt][nt][3]);
                acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.f;
              }
            }
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          cur[mt][h] = nxt[mt][h];
          sc[mt][h] = sn[mt][h];
        }
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[(warp * 8 * NT + nt * 8 + 2 * t4 + (q & 1)) * kPitch + mt * 16 + g + 8 * (q >> 1)] =
            total[mt][nt][q];
  __syncthreads();
  // a row group's outputs by its warps, tokens fastest
  for (int e = ks * 32 + lane; e < nb * kTokens; e += split * 32) {
    const int b = e / kTokens, t = e % kTokens;
    if (v0 + t >= p.V) continue;
    float z = 0.f;
    for (int w = 0; w < split; ++w) {
      const float* r = red + ((rg * split + w) * 8 * NT + b * kParts) * kPitch + t;
      z += kParts == 3 ? (r[2 * kPitch] + r[kPitch]) + r[0] : r[0];
    }
    if (base) z += load_any(base, p.base_dtype, (int64_t)(b0 + b) * p.base_stride + v0 + t);
    store_any(out, p.out_dtype, (int64_t)(b0 + b) * p.out_stride + v0 + t, z);
  }
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

template <typename T, int NT, int MT>
static cudaError_t product(const spec_w4_params& p, const T* x, const int32_t* prev,
                           const uint8_t* wq, const void* wscale, const void* base, void* out,
                           WsHeader* hdr, cudaStream_t st) {
  constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
  constexpr int kRows = 8 * NT / kParts < 16 ? 8 * NT / kParts : 16;
  const int nkb = (p.r + 127) / 128;
  int split = 1;
  while (split < kWarps && 2 * split <= nkb) split *= 2;
  const int64_t per = (int64_t)16 * MT * (kWarps / split);
  const int wide = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && p.x_stride * sizeof(T) % 16 == 0;
  constexpr size_t smem = sizeof(float) * kWarps * 8 * NT * (16 * MT + 4);
  auto kernel = k_bias_w4<T, NT, MT>;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<dim3((unsigned)((p.V + per - 1) / per), (p.B + kRows - 1) / kRows), kThreads, smem, st>>>(
      p, x, prev, wq, wscale, base, out, split, wide, hdr);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bias_w4(const spec_w4_params& p, const T* x, const int32_t* prev,
                           const uint8_t* wq, const void* wscale, const void* base, void* out,
                           WsHeader* hdr, int, cudaStream_t st, int* launches) {
  if (p.B > 65535) return cudaErrorInvalidValue;
  *launches = 1;
  const int rows = std::min(p.B, 16);
#define SPEC_W4(NT, MT) return product<T, NT, MT>(p, x, prev, wq, wscale, base, out, hdr, st)
  if constexpr (sizeof(T) == 2) {
    if (rows <= 8) SPEC_W4(1, 4);
    SPEC_W4(2, 4);
  } else {  // three columns a row
    if (rows <= 2) SPEC_W4(1, 4);
    if (rows <= 5) SPEC_W4(2, 4);
    if (rows <= 8) SPEC_W4(3, 2);
    if (rows <= 10) SPEC_W4(4, 2);
    SPEC_W4(6, 2);
  }
#undef SPEC_W4
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
