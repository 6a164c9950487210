// Device helpers of the two 4-bit vocabulary products (bias_w4.cu on warp-level
// matrix instructions, bias_w4_tc.cu on tensor memory).
#pragma once

#include "head_ops.cuh"

namespace specdec {

SPEC_DEV float load_any(const void* p, int32_t dtype, int64_t i) {
  return dtype == SPEC_BF16 ? load_f((const __nv_bfloat16*)p, i) : load_f((const float*)p, i);
}
SPEC_DEV void store_any(void* p, int32_t dtype, int64_t i, float v) {
  if (dtype == SPEC_BF16)
    store_f((__nv_bfloat16*)p, i, v);
  else
    store_f((float*)p, i, v);
}

// Eight codes as four pairs (k, k + 4) of bf16.
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

// The tensor-memory product, for vocabularies that fill the GPU.
bool w4_tc_fits(const spec_w4_params& p, int num_sms);
size_t w4_tc_ws_bytes(const spec_w4_params& p);
template <typename T>
cudaError_t launch_bias_w4_tc(const spec_w4_params& p, const T* x, const int32_t* prev,
                              const uint8_t* wq, const void* wscale, const void* base, void* out,
                              uint8_t* body, WsHeader* hdr, int num_sms, cudaStream_t st,
                              int* launches);

}  // namespace specdec
