// Vocabulary product with 4-bit weights and group scales, and the quantiser
// that lays a factor out for it.
#include <algorithm>
#include <cfloat>

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

// Eight codes as four pairs (k, k + 4) of bf16.  A bf16 has 7 fraction bits, so from
// 128 to 256 its steps are 1: 0x4300 is 128, 0x4300 | code is 128 + code, and taking
// 136 (0x4308) off is exact and leaves code - 8.
SPEC_DEV void codes_to_bf16(uint32_t w, uint32_t* p) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t u;  // (w >> 4 k) & 0x000F000F | 0x43004300
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(u)
        : "r"(w >> (4 * k)), "r"(0x000F000Fu), "r"(0x43004300u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p[k]) : "r"(u), "r"(0x43084308u));  // 136
  }
}

SPEC_DEV uint32_t part_of(const uint4& w, int i) {
  return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
}

// Row of X that row b reads (prev or itself), out-of-range tokens clamped and
// reported once.
SPEC_DEV int x_row(const spec_w4_params& p, const int32_t* prev, int b, bool say, WsHeader* hdr) {
  if (!prev) return b;
  const int row = __ldg(prev + b);
  if (row >= 0 && row < p.x_rows) return row;
  if (say) report_error(hdr, SPEC_ERR_TOKEN_RANGE, SITE_TOKEN_RANGE, b, row);
  return row < 0 ? 0 : p.x_rows - 1;
}

// Eight features of one row of X as they lie in memory.
template <typename T>
struct XWord {
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

// Rows of X on 16-byte boundaries.
template <typename T>
bool x_wide(const spec_w4_params& p, const T* x) {
  return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && p.x_stride * sizeof(T) % 16 == 0;
}

// ----------------------------------------------------------------------------
// The product.  A warp multiplies kTiles tiles of 16 tokens by up to 8 NT columns
// of X on the tensor cores (m16n8k16, bf16 in, fp32 out).  Codes become bf16
// exactly; a lane's 16 bytes of a row hold one word of each 32 features, so the
// multiply of a group needs no other lane's bytes, and the order of the features
// inside a word is given to X instead (a nibble and the one 16 bits above it make
// a pair).  The sum of a group stays in the accumulator, is scaled in fp32 and
// added to the row's.  fp32 X is cut into three bf16 parts, which together hold
// all its 24 bits, as columns of their own, so its products are exact as well.
//
// The codes pass through once, two blocks of 128 features ahead of the products
// in registers; that is their floor in bytes.  X is laid out beforehand (k_w4_x) as the
// fragments the warps read, and stays in the SMs' first-level caches, so the
// warps of a CTA need not wait for one another.  Where the vocabulary gives few
// CTAs, or much work to each, the warps split the features and join their sums
// in order.
//
// What bounds it: one row is bound by the codes' latency and the launches (r 256,
// V 129280: 12.3 us); 16 rows by unpacking and multiplying, which the loads
// overlap only in part (r 4096, V 151936: 123 us, 2.7 TB/s, 160 TFLOP/s.  Without
// the products 90 us, without the weights' loads 84, without any loads 76, without
// the sums' way out 108).  Registers allow 16 warps an SM.  Slower were: a tile of
// tokens per warp or three CTAs an SM (150 to 175), a block's X or the codes staged
// in shared memory (210, 126), persistent CTAs (140), and the fifth-generation
// tensor cores with the codes unpacked into tensor memory, where the unpacking
// threads' chain of waits costs more than the products save (166).
// ----------------------------------------------------------------------------
constexpr int kWarps = kThreads / 32;

SPEC_DEV void mma_bf16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

SPEC_DEV void mma_bf16_zero(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                            uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

SPEC_DEV uint4 load_once(const uint8_t* p) {
  uint4 w;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p));
  return w;
}
template <typename T>
int rows_of(int NT) { return std::min(8 * NT / XWord<T>::kParts, 16); }  // that 8 NT columns hold
constexpr int kTiles = 2;  // tiles of 16 tokens per warp
constexpr int kTokens = 16 * kTiles, kPitch = kTokens + 4;

// X as fragments: [row group][block of 128 features][32 features][NT][lane] of
// 16 bytes, the lane's four pairs of features of its column.  Features past r are
// zero; columns without a row hold anything, no output is taken from them.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_w4_x(spec_w4_params p, const T* __restrict__ x, const int32_t* __restrict__ prev, uint4* xf,
           int NT, int rows, int wide, WsHeader* hdr) {
  grid_dependency_release();
  const int words = (p.r + 127) / 128 * 16;  // of eight features
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int b = (int)(e / words), w = (int)(e % words);
  if (b >= p.B) return;
  const int row = x_row(p, prev, b, w == 0, hdr);
  XWord<T> q;
  q.clear();
  if (8 * w < p.r) q.load(x + (int64_t)row * p.x_stride + 8 * w, wide);
  // word w of the row is word w % 4 of 32 features w / 4
  uint4* to = xf + ((int64_t)(b / rows) * (words / 4) + w / 4) * NT * 32;
#pragma unroll
  for (int s = 0; s < XWord<T>::kParts; ++s) {
    const int col = b % rows * XWord<T>::kParts + s;
    to[(col >> 3) * 32 + (col & 7) * 4 + (w & 3)] = q.pairs(s);
  }
}

template <int NT, int G>
__global__ void __launch_bounds__(kThreads, NT <= 3 ? 2 : 1)
    k_bias_w4(spec_w4_params p, const uint4* xf, const uint8_t* __restrict__ wq,
              const void* __restrict__ wscale, const void* base, void* out, int split, int parts,
              int rows) {
  constexpr int kPer = 128 / G;  // groups per block; lane t4 holds the scale of group t4 % kPer
  extern __shared__ __align__(16) float red[];  // [warp][column][kPitch]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int ks = warp % split, rg = warp / split;
  const int64_t v0 = ((int64_t)blockIdx.x * (kWarps / split) + rg) * kTokens;
  const int b0 = blockIdx.y * rows, nb = min(rows, p.B - b0);
  const int nkb = (p.r + 127) / 128, rowb = nkb * 64, ng = p.r / G;
  const int kb0 = nkb * ks / split, kb1 = nkb * (ks + 1) / split;
  const int last = (int)min((int64_t)kTokens, p.V - v0) - 1;  // < 0: no tokens here

  struct Codes {
    uint4 w[kTiles][2];
    uint32_t s[kTiles][2];  // as they lie in memory: converted when used, not waited for here
  };
  const uint8_t* wp = wq + v0 * rowb + t4 * 16;
  int w_at[kTiles][2], s_at[kTiles][2];  // past the vocabulary: its last row
#pragma unroll
  for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = max(min(mt * 16 + g + 8 * h, last), 0);
      w_at[mt][h] = at * rowb;
      s_at[mt][h] = at * ng;
    }
  const bool bf16_scales = p.scale_dtype == SPEC_BF16;
  auto scale_of = [&](uint32_t raw) { return __uint_as_float(bf16_scales ? raw << 16 : raw); };
  auto request = [&](int kb, Codes& c) {
    if (kb >= kb1 || last < 0) return;
    const uint8_t* w = wp + (int64_t)kb * 64;
    const int64_t s = v0 * ng + min(kb * kPer + t4 % kPer, ng - 1);
#pragma unroll
    for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) c.w[mt][h] = load_once(w + w_at[mt][h]);
    if (bf16_scales) {
#pragma unroll
      for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          c.s[mt][h] = __ldg((const unsigned short*)wscale + s + s_at[mt][h]);
    } else {
#pragma unroll
      for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) c.s[mt][h] = __ldg((const uint32_t*)wscale + s + s_at[mt][h]);
    }
  };
  if (base && ks == 0 && lane < nb && last >= 0)  // what the outputs are added to, for the end
    asm volatile("prefetch.global.L2 [%0];" ::"l"(
        (const char*)base + ((int64_t)(b0 + lane) * p.base_stride + v0) * (p.base_dtype == SPEC_BF16 ? 2 : 4)));
  Codes c0, c1;
  request(kb0, c0);
  request(kb0 + 1, c1);
  grid_dependency_wait();  // X's fragments

  const uint4* xs = xf + (int64_t)blockIdx.y * nkb * (4 * NT * 32) + lane;
  float total[kTiles][NT][4] = {};
  auto multiply = [&](int kb, const Codes& c) {
    const uint4* xk = xs + kb * (4 * NT * 32);
    float acc[kTiles][NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 xb[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) xb[nt] = xk[(i * NT + nt) * 32];
      const bool first = 32 * i % G == 0, ends = 32 * (i + 1) % G == 0;
#pragma unroll
      for (int mt = 0; mt < kTiles; ++mt) {
        uint32_t lo[4], hi[4];
        codes_to_bf16(part_of(c.w[mt][0], i), lo);
        codes_to_bf16(part_of(c.w[mt][1], i), hi);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (first)
            mma_bf16_zero(acc[mt][nt], lo[0], hi[0], lo[1], hi[1], xb[nt].x, xb[nt].y);
          else
            mma_bf16(acc[mt][nt], lo[0], hi[0], lo[1], hi[1], xb[nt].x, xb[nt].y);
          mma_bf16(acc[mt][nt], lo[2], hi[2], lo[3], hi[3], xb[nt].z, xb[nt].w);
        }
      }
      if (ends) {
        const int from = (lane & ~3) + 32 * i / G;
#pragma unroll
        for (int mt = 0; mt < kTiles; ++mt) {
          const float s0 = scale_of(kPer == 1 ? c.s[mt][0] : __shfl_sync(0xffffffffu, c.s[mt][0], from));
          const float s1 = scale_of(kPer == 1 ? c.s[mt][1] : __shfl_sync(0xffffffffu, c.s[mt][1], from));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            total[mt][nt][0] = fmaf(s0, acc[mt][nt][0], total[mt][nt][0]);
            total[mt][nt][1] = fmaf(s0, acc[mt][nt][1], total[mt][nt][1]);
            total[mt][nt][2] = fmaf(s1, acc[mt][nt][2], total[mt][nt][2]);
            total[mt][nt][3] = fmaf(s1, acc[mt][nt][3], total[mt][nt][3]);
          }
        }
      }
    }
  };
  if (last >= 0) {
    for (int kb = kb0; kb < kb1; kb += 2) {
      multiply(kb, c0);
      request(kb + 2, c0);
      if (kb + 1 < kb1) multiply(kb + 1, c1);
      request(kb + 3, c1);
    }
  }

#pragma unroll
  for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[(warp * 8 * NT + nt * 8 + 2 * t4 + (q & 1)) * kPitch + mt * 16 + g + 8 * (q >> 1)] =
            total[mt][nt][q];
  __syncthreads();
  // a row group's outputs by its warps, a lane per token; base is read for all of
  // them first, since the stores (out may be base) hold later reads back
  if (lane > last) return;
  const int64_t v = v0 + lane;
  float z[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int b = ks + q * split;
    z[q] = base && b < nb ? load_any(base, p.base_dtype, (int64_t)(b0 + b) * p.base_stride + v) : 0.f;
  }
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int b = ks + q * split;
    if (b >= nb) break;
    float sum = 0.f;
    for (int w = 0; w < split; ++w) {
      const float* r = red + ((rg * split + w) * 8 * NT + b * parts) * kPitch + lane;
      sum += parts == 3 ? (r[2 * kPitch] + r[kPitch]) + r[0] : r[0];
    }
    store_any(out, p.out_dtype, (int64_t)(b0 + b) * p.out_stride + v, z[q] + sum);
  }
}
static_assert(kTokens == 32, "the epilogue gives every lane a token");

// One thread per token and 128 features, reading W's columns: neighbouring threads
// read neighbouring tokens.  Run once per factor, so its time is not on any path.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_w4_quantize(spec_w4_params p, const T* __restrict__ W, uint8_t* wq, void* wscale) {
  const int v = blockIdx.x * kThreads + threadIdx.x, blk = blockIdx.y;
  if (v >= p.V) return;
  uint32_t words[16];
  const int ng = p.r / p.group;
  auto at = [&](int k) {
    // an infinity counts as the largest number of its sign: the scale stays finite,
    // where inf / inf would give NaN and a finite weight's code no meaning
    const float w = load_f(W, (int64_t)k * p.V + v);
    return w == w ? fminf(fmaxf(w, -FLT_MAX), FLT_MAX) : 0.f;
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
        // a scale rounded down can leave the largest weights past the codes' ends
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

constexpr int kSteps = 16;  // blocks of 128 features a warp goes through, at most

// Tiles of eight columns for up to 16 rows of X.
static int column_tiles(const spec_w4_params& p) {
  const int rows = std::min(p.B, 16);
  if (p.dtype == SPEC_BF16) return rows <= 8 ? 1 : 2;
  return rows <= 2 ? 1 : rows <= 5 ? 2 : rows <= 8 ? 3 : rows <= 10 ? 4 : 6;  // three a row
}

size_t w4_ws_bytes(const spec_w4_params& p) {
  const int NT = column_tiles(p);
  const int rows = p.dtype == SPEC_BF16 ? rows_of<__nv_bfloat16>(NT) : rows_of<float>(NT);
  return sizeof(uint4) * 32 * 4 * NT * (size_t)((p.r + 127) / 128) * ((p.B + rows - 1) / rows);
}

template <int NT, int G>
static cudaError_t product(const spec_w4_params& p, const uint4* xf, const uint8_t* wq,
                           const void* wscale, const void* base, void* out, int rows, int parts,
                           int num_sms, cudaStream_t st) {
  const int nkb = (p.r + 127) / 128;
  // warps split the features while the tokens give fewer than two CTAs per SM
  // (4 rows, r 4096, V 8000: 15 us, unsplit 25), and until a CTA's work is short,
  // so that the last ones to run end together (16 rows, r 4096, V 151936, groups of
  // 64: 152 us, unsplit 169)
  int split = 1;
  while (split < kWarps && 2 * split <= nkb &&
         (nkb / split > kSteps ||
          ((int64_t)p.V + kTokens * kWarps / split - 1) / (kTokens * kWarps / split) < 2 * num_sms))
    split *= 2;
  const int64_t per = (int64_t)kTokens * kWarps / split;
  constexpr size_t smem = sizeof(float) * kWarps * 8 * NT * kPitch;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        k_bias_w4<NT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_after(k_bias_w4<NT, G>,
                      dim3((unsigned)((p.V + per - 1) / per), (p.B + rows - 1) / rows), kThreads,
                      smem, st, p, xf, wq, wscale, base, out, split, parts, rows);
}

template <typename T>
cudaError_t launch_bias_w4(const spec_w4_params& p, const T* x, const int32_t* prev,
                           const uint8_t* wq, const void* wscale, const void* base, void* out,
                           uint8_t* body, WsHeader* hdr, int num_sms, cudaStream_t st,
                           int* launches) {
  const int NT = column_tiles(p), rows = rows_of<T>(NT), parts = XWord<T>::kParts;
  if ((p.B + rows - 1) / rows > 65535) return cudaErrorInvalidValue;
  uint4* xf = reinterpret_cast<uint4*>(body);
  const int wide = x_wide(p, x);
  const int64_t words = (int64_t)p.B * ((p.r + 127) / 128 * 16);
  const cudaError_t e = launch_kernel(k_w4_x<T>, (unsigned)((words + kThreads - 1) / kThreads),
                                      kThreads, 0, st, p, x, prev, xf, NT, rows, wide, hdr);
  if (e != cudaSuccess) return e;
  *launches = 2;
#define SPEC_W4(NT, G) return product<NT, G>(p, xf, wq, wscale, base, out, rows, parts, num_sms, st)
#define SPEC_W4_G(NT)                                                                              \
  if (p.group == 32) SPEC_W4(NT, 32);                                                              \
  if (p.group == 64) SPEC_W4(NT, 64);                                                              \
  SPEC_W4(NT, 128)
  switch (NT) {
    case 1: SPEC_W4_G(1);
    case 2: SPEC_W4_G(2);
    case 3: SPEC_W4_G(3);
    case 4: SPEC_W4_G(4);
    default: SPEC_W4_G(6);
  }
#undef SPEC_W4_G
#undef SPEC_W4
}

template <typename T>
cudaError_t launch_w4_quantize(const spec_w4_params& p, const T* W, uint8_t* wq, void* wscale,
                               cudaStream_t st) {
  return launch_kernel(k_w4_quantize<T>, dim3((p.V + kThreads - 1) / kThreads, (p.r + 127) / 128),
                       kThreads, 0, st, p, W, wq, wscale);
}

#define SPEC_INST(T)                                                                               \
  template cudaError_t launch_bias_w4<T>(const spec_w4_params&, const T*, const int32_t*,          \
                                         const uint8_t*, const void*, const void*, void*,          \
                                         uint8_t*, WsHeader*, int, cudaStream_t, int*);            \
  template cudaError_t launch_w4_quantize<T>(const spec_w4_params&, const T*, uint8_t*, void*,     \
                                             cudaStream_t);
SPEC_INST(float)
SPEC_INST(__nv_bfloat16)
#undef SPEC_INST

}  // namespace specdec
