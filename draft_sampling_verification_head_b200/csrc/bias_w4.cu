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
// Bytes bound it: the codes pass through once, two blocks of 128 features ahead
// of the products in registers.  The block of X that a CTA's warps multiply by is
// laid out in shared memory as the fragments they read, one block ahead.  Where
// the vocabulary gives too few CTAs, the warps split the features and join their
// sums in order.
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

template <typename T>
struct XWord {  // eight features of one row of X as they lie in memory
  static constexpr int kParts = sizeof(T) == 4 ? 3 : 1;  // columns per row of X
  uint4 v[sizeof(T) / 2];
  SPEC_DEV void clear() {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) v[k] = make_uint4(0, 0, 0, 0);
  }
  SPEC_DEV void load(const T* x, bool wide) {
    if (wide) {
#pragma unroll
      for (int k = 0; k < (int)sizeof(T) / 2; ++k) v[k] = __ldg(reinterpret_cast<const uint4*>(x) + k);
    } else if constexpr (sizeof(T) == 4) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(x);
      v[0] = make_uint4(__ldg(w), __ldg(w + 1), __ldg(w + 2), __ldg(w + 3));
      v[1] = make_uint4(__ldg(w + 4), __ldg(w + 5), __ldg(w + 6), __ldg(w + 7));
    } else {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(x);
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        u[k] = (uint32_t)__ldg(h + 2 * k) | (uint32_t)__ldg(h + 2 * k + 1) << 16;
      v[0] = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
  // the pairs (k, k + 4) of column `part` (0 holds the leading bits)
  SPEC_DEV uint4 pairs(int part) const {
    if constexpr (sizeof(T) == 2) {
      return make_uint4(__byte_perm(v[0].x, v[0].z, 0x5410), __byte_perm(v[0].x, v[0].z, 0x7632),
                        __byte_perm(v[0].y, v[0].w, 0x5410), __byte_perm(v[0].y, v[0].w, 0x7632));
    } else {
      const uint32_t b[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
      uint32_t c[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const bool finite = (b[k] & 0x7F800000u) != 0x7F800000u;
        // cutting keeps the leading 8 bits; the rest is exact, and so is its rest
        const float r1 = __uint_as_float(b[k]) - __uint_as_float(b[k] & 0xFFFF0000u);
        const float r2 = r1 - __uint_as_float(__float_as_uint(r1) & 0xFFFF0000u);
        const uint32_t head = finite || (b[k] & 0x007FFFFFu) == 0 ? b[k] : 0x7FC00000u;
        c[k] = part == 0 ? head : finite ? __float_as_uint(part == 1 ? r1 : r2) : 0u;
      }
      return make_uint4(__byte_perm(c[0], c[4], 0x7632), __byte_perm(c[1], c[5], 0x7632),
                        __byte_perm(c[2], c[6], 0x7632), __byte_perm(c[3], c[7], 0x7632));
    }
  }
};

template <typename T, int NT>
__host__ __device__ constexpr int rows_of() {  // rows of X that 8 NT columns hold, 16 at most
  return 8 * NT / XWord<T>::kParts < 16 ? 8 * NT / XWord<T>::kParts : 16;
}
constexpr int kTiles = 2;                       // tiles of 16 tokens per warp
constexpr int kTokens = 16 * kTiles, kPitch = kTokens + 4;
template <int NT>
__host__ __device__ constexpr int block_bytes() { return 4 * NT * 32 * 16; }  // one block of X as fragments

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, NT <= 3 ? 2 : 1)
    k_bias_w4(spec_w4_params p, const T* __restrict__ x, const int32_t* __restrict__ prev,
              const uint8_t* __restrict__ wq, const void* __restrict__ wscale, const void* base,
              void* out, int split, int wide, WsHeader* hdr) {
  constexpr int kParts = XWord<T>::kParts, kRows = rows_of<T, NT>();
  // [2][split] blocks of X; at the end [warp][column][kPitch] sums
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t row_at[kRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int ks = warp % split, rg = warp / split;
  const int64_t v0 = ((int64_t)blockIdx.x * (kWarps / split) + rg) * kTokens;
  const int b0 = blockIdx.y * kRows, nb = min(kRows, p.B - b0);
  const int nkb = (p.r + 127) / 128, steps = (nkb + split - 1) / split;
  const int rowb = nkb * 64, ng = p.r / p.group;
  if (tid < nb) {
    int row = b0 + tid;
    if (prev) {
      row = __ldg(prev + row);
      if (row < 0 || row >= p.x_rows) {
        if (blockIdx.x == 0)
          report_error(hdr, SPEC_ERR_TOKEN_RANGE, SITE_TOKEN_RANGE, b0 + tid, row);
        row = row < 0 ? 0 : p.x_rows - 1;
      }
    }
    row_at[tid] = row * p.x_stride;
  }

  // codes and scales: a warp reads block step * split + ks, two steps ahead
  const int last = (int)min((int64_t)kTokens, p.V - v0) - 1;  // < 0: no tokens here
  const uint8_t* w0 = wq + v0 * rowb + t4 * 16;
  const int per = 128 / p.group;  // groups per block; lane t4 holds the scale of group t4 % per
  struct Codes {
    uint4 w[kTiles][2];
    float s[kTiles][2];
  };
  Codes c0, c1, c2;
  auto request = [&](int step, Codes& c) {
    const int kb = step * split + ks;
    if (kb >= nkb || last < 0) return;
    const int gi = min(kb * per + t4 % per, ng - 1);
#pragma unroll
    for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = min(mt * 16 + g + 8 * h, last);  // past the vocabulary: its last row
        c.w[mt][h] = load_once(w0 + (int64_t)at * rowb + kb * 64);
        c.s[mt][h] = load_any(wscale, p.scale_dtype, (v0 + at) * ng + gi);
      }
  };
  request(0, c0);
  request(1, c1);

  // X: word (row, w) of a step's blocks, one per thread and round
  const int words = split * 16;
  auto x_at = [&](int step, int e, XWord<T>& q) {
    const int row = e / words, k = (step * words + e % words) * 8;
    if (row < nb && k < p.r)
      q.load(x + row_at[row] + k, wide);
    else
      q.clear();
  };
  auto x_put = [&](int step, int e, const XWord<T>& q) {
    const int row = e / words, w = e % words, blk = w >> 4, i = (w >> 2) & 3, j = w & 3;
    uint4* to = reinterpret_cast<uint4*>(smem) + ((step & 1) * split + blk) * (block_bytes<NT>() / 16);
#pragma unroll
    for (int s = 0; s < kParts; ++s) {
      const int col = row * kParts + s;
      to[(i * NT + (col >> 3)) * 32 + (col & 7) * 4 + j] = q.pairs(s);
    }
  };
  // columns beyond the rows of X stay zero
  for (int k = tid; k < 2 * split * block_bytes<NT>() / 16; k += kThreads)
    reinterpret_cast<uint4*>(smem)[k] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  const int items = kRows * words;
  for (int e = tid; e < items; e += kThreads) {
    XWord<T> q;
    x_at(0, e, q);
    if (e / words < nb) x_put(0, e, q);
  }
  __syncthreads();

  float total[kTiles][NT][4] = {};
  for (int step = 0; step < steps; ++step) {
    request(step + 2, c2);
    XWord<T> held;  // the next step's first word, stored when this step is done
    if (step + 1 < steps) x_at(step + 1, tid, held);
    const int kb = step * split + ks;
    if (kb < nkb && last >= 0) {
      const uint4* xs = reinterpret_cast<const uint4*>(smem) +
                        ((step & 1) * split + ks) * (block_bytes<NT>() / 16) + lane;
      float acc[kTiles][NT][4] = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (kb * 128 + 32 * i >= p.r) break;
        uint32_t a[kTiles][2][4];
#pragma unroll
        for (int mt = 0; mt < kTiles; ++mt) {
          codes_to_bf16(part_of(c0.w[mt][0], i), a[mt][0]);
          codes_to_bf16(part_of(c0.w[mt][1], i), a[mt][1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 xb = xs[(i * NT + nt) * 32];
#pragma unroll
          for (int mt = 0; mt < kTiles; ++mt) {
            mma_bf16(acc[mt][nt], a[mt][0][0], a[mt][1][0], a[mt][0][1], a[mt][1][1], xb.x, xb.y);
            mma_bf16(acc[mt][nt], a[mt][0][2], a[mt][1][2], a[mt][0][3], a[mt][1][3], xb.z, xb.w);
          }
        }
        if ((32 * (i + 1)) % p.group == 0) {  // a group ends
          const int from = (lane & ~3) + 32 * i / p.group;
#pragma unroll
          for (int mt = 0; mt < kTiles; ++mt) {
            const float s0 = __shfl_sync(0xffffffffu, c0.s[mt][0], from);
            const float s1 = __shfl_sync(0xffffffffu, c0.s[mt][1], from);
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
    if (step + 1 < steps) {
      if (tid < items && tid / words < nb) x_put(step + 1, tid, held);
      for (int e = tid + kThreads; e < items; e += kThreads) {
        XWord<T> q;
        x_at(step + 1, e, q);
        if (e / words < nb) x_put(step + 1, e, q);
      }
    }
    c0 = c1;
    c1 = c2;
    __syncthreads();
  }

  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[(warp * 8 * NT + nt * 8 + 2 * t4 + (q & 1)) * kPitch + mt * 16 + g + 8 * (q >> 1)] =
            total[mt][nt][q];
  __syncthreads();
  // a row group's outputs by its warps, tokens fastest
  for (int b = ks; b < nb; b += split) {
    if (lane > last) break;  // kTokens = 32: a lane per token
    float z = 0.f;
    for (int w = 0; w < split; ++w) {
      const float* r = red + ((rg * split + w) * 8 * NT + b * kParts) * kPitch + lane;
      z += kParts == 3 ? (r[2 * kPitch] + r[kPitch]) + r[0] : r[0];
    }
    const int64_t v = v0 + lane;
    if (base) z += load_any(base, p.base_dtype, (int64_t)(b0 + b) * p.base_stride + v);
    store_any(out, p.out_dtype, (int64_t)(b0 + b) * p.out_stride + v, z);
  }
}
static_assert(kTokens == 32, "the epilogue gives every lane a token");

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

template <typename T, int NT>
static cudaError_t product(const spec_w4_params& p, const T* x, const int32_t* prev,
                           const uint8_t* wq, const void* wscale, const void* base, void* out,
                           WsHeader* hdr, int num_sms, cudaStream_t st) {
  constexpr int kRows = rows_of<T, NT>();
  const int nkb = (p.r + 127) / 128;
  // warps split the features while the tokens give fewer than two CTAs per SM
  int split = 1;
  while (split < kWarps && 2 * split <= nkb &&
         ((int64_t)p.V + kTokens * kWarps / split - 1) / (kTokens * kWarps / split) < 2 * num_sms)
    split *= 2;
  const int64_t per = (int64_t)kTokens * kWarps / split;
  const int wide = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && p.x_stride * sizeof(T) % 16 == 0;
  const size_t smem = std::max(sizeof(float) * kWarps * 8 * NT * kPitch,
                               (size_t)2 * split * block_bytes<NT>());
  auto kernel = k_bias_w4<T, NT>;
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
                           WsHeader* hdr, int num_sms, cudaStream_t st, int* launches) {
  if (p.B > 65535) return cudaErrorInvalidValue;
  *launches = 1;
  const int rows = std::min(p.B, 16);
#define SPEC_W4(NT) return product<T, NT>(p, x, prev, wq, wscale, base, out, hdr, num_sms, st)
  if constexpr (sizeof(T) == 2) {
    if (rows <= 8) SPEC_W4(1);
    SPEC_W4(2);
  } else {  // three columns a row
    if (rows <= 2) SPEC_W4(1);
    if (rows <= 5) SPEC_W4(2);
    if (rows <= 8) SPEC_W4(3);
    if (rows <= 10) SPEC_W4(4);
    SPEC_W4(6);
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
