// Vocabulary product with 4-bit weights on tcgen05, for vocabularies that fill the
// GPU: out[b, v] = base[b, v] + sum_g s[v, g] sum_{k in g} X[b, k] (code[v, k] - 8).
//
// Tokens lie on M: a tile is 128 of them, a thread of a quartet of warps each.  The
// thread turns its token's codes into bf16 (exact) and stores them as the A operand
// in tensor memory, 64 features at a time; X (as many bf16 columns as its type
// needs: one, or three whose sum is an fp32 exactly) is the B operand in shared
// memory.  The MMA of a group of features adds into an accumulator of its own;
// the thread reads it back, scales it in fp32 and adds it to its token's sums in
// registers, so no scaled weight is ever rounded.  While one half block is
// multiplied the quartet unpacks the next: two A buffers, two accumulators.
//
// A CTA per SM runs up to four quartets on tiles of their own in step, so that a
// block of X, which one warp copies through a ring, serves all of them.  Codes go
// through rings of 16-byte asynchronous copies, private to a warp.  Tiles are cut
// to equal numbers of tokens so that every SM gets as many.
#include <algorithm>

#include "w4.cuh"

namespace specdec {
namespace {

constexpr int kBStages = 4;   // blocks of X in flight
constexpr int kCStages = 4;   // blocks of codes in flight per warp
constexpr int kCodeBytes = 32 * 64;  // a warp's codes of one block of 128 features
constexpr int kACols = 32;    // tensor-memory columns of 64 features of A
constexpr uint64_t kPolls = 1ull << 22;

template <int NC, int G>
struct Plan {
  static constexpr int kPer = 128 / G;                       // groups per block
  static constexpr int kDBufs = G == 32 ? 4 : 2;             // accumulators per quartet
  static constexpr int kCols = 2 * kACols + kDBufs * NC;     // tensor memory per quartet
  // quartets that tensor memory and the register file hold
  static constexpr int kMaxQ = NC == 16 ? 4 : (NC == 32 ? (G == 32 ? 2 : 3) : (G == 32 ? 2 : 3));
  static constexpr int kBBytes = NC * 256;                   // a block of X
  static constexpr int kThreadsMax = kMaxQ * 128 + 32;
  static_assert(kMaxQ * kCols <= 512, "tensor memory");
};

struct Ctl {
  uint64_t bfull[kBStages], bempty[kBStages];
  uint64_t dfull[4][2];
  uint32_t tmem;
  uint32_t failed;
};

struct Args {
  spec_w4_params p;
  const uint8_t* xf;
  const uint8_t* wq;
  const void* wscale;
  const void* base;
  void* out;
  WsHeader* hdr;
  int quartets, rounds, tokens;  // tokens per tile
  int rows, parts;               // rows of X per launch row, columns of each
};

// X as B operands: [row group][block][64 features][NC rows of 128 bytes], 16-byte
// chunks swizzled, the features of a word in the order of its code pairs.
template <typename T>
__global__ void __launch_bounds__(256)
    k_w4_x_tc(spec_w4_params p, const T* __restrict__ x, const int32_t* __restrict__ prev,
              uint4* xf, int NC, int rows, int wide, WsHeader* hdr) {
  grid_dependency_release();
  const int nkb = (p.r + 127) / 128, words = nkb * 16;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int b = (int)(e / words), w = (int)(e % words);
  if (b >= p.B) return;
  const int row = x_row(p, prev, b, w == 0, hdr);
  XWord<T> q;
  q.clear();
  if (8 * w < p.r) q.load(x + (int64_t)row * p.x_stride + 8 * w, wide);
  uint4* to = xf + ((int64_t)(b / rows) * nkb * 2 + (w >> 3)) * (NC * 8);
#pragma unroll
  for (int s = 0; s < XWord<T>::kParts; ++s) {
    const int n = b % rows * XWord<T>::kParts + s;
    to[n * 8 + ((w & 7) ^ (n & 7))] = q.pairs(s);
  }
}

SPEC_DEV void umma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
SPEC_DEV void tmem_store32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}

// Bounded wait; once one ran out, none of the CTA's waits waits any more.
SPEC_DEV void wait_for(uint64_t* bar, uint32_t parity, Ctl* ctl, WsHeader* hdr, int site) {
  for (uint64_t it = 0; it < kPolls; ++it) {
    if (mbar_try_wait(bar, parity)) return;
    if ((it & 63) == 63 && ld_volatile_u32(&ctl->failed)) return;
  }
  *reinterpret_cast<volatile uint32_t*>(&ctl->failed) = 1u;
  report_error(hdr, SPEC_ERR_TIMEOUT, site, blockIdx.x, 0);
}

template <int NC, int G>
__global__ void __launch_bounds__(Plan<NC, G>::kThreadsMax, 1) k_bias_w4_tc(Args a) {
  using P = Plan<NC, G>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sB = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sC = sB + kBStages * P::kBBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(sC + (size_t)a.quartets * 4 * kCStages * kCodeBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, Q = a.quartets;
  const int V = a.p.V, nkb = (a.p.r + 127) / 128, steps = a.rounds * nkb;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBStages; ++i) {
      mbar_init(&ctl->bfull[i], 1);
      mbar_init(&ctl->bempty[i], Q);
    }
    for (int q = 0; q < 4; ++q)
      for (int i = 0; i < 2; ++i) mbar_init(&ctl->dfull[q][i], 1);
    ctl->failed = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;

  if (warp == 4 * Q) {
    // ---- blocks of X through the ring ----
    if (lane == 0) {
      grid_dependency_wait();
      const uint8_t* src = a.xf + (int64_t)blockIdx.y * nkb * P::kBBytes;
      const uint64_t policy = policy_evict_last();
      for (int it = 0; it < steps; ++it) {
        const int slot = it % kBStages;
        if (it >= kBStages)
          wait_for(&ctl->bempty[slot], (it / kBStages - 1) & 1, ctl, a.hdr, SITE_MBAR_BASE);
        if (ld_volatile_u32(&ctl->failed)) break;
        mbar_arrive_expect_tx(&ctl->bfull[slot], P::kBBytes);
        bulk_load(sB + slot * P::kBBytes, src + (int64_t)(it % nkb) * P::kBBytes, P::kBBytes,
                  &ctl->bfull[slot], policy);
      }
      // the last blocks' commits land before the CTA may end
      for (int it = max(steps - kBStages, 0); it < steps; ++it)
        wait_for(&ctl->bempty[it % kBStages], (it / kBStages) & 1, ctl, a.hdr, SITE_MBAR_BASE);
    }
    __syncwarp();
  } else if (warp < 4 * Q) {
    const int q = warp >> 2, w4 = warp & 3, m = w4 * 32 + lane;  // the thread's token of the tile
    uint8_t* ring = sC + (size_t)warp * kCStages * kCodeBytes;
    const int rowb = nkb * 64, ng = a.p.r / G;
    const bool bf16_scales = a.p.scale_dtype == SPEC_BF16;
    const int64_t cta0 = (int64_t)blockIdx.x * a.rounds * Q * a.tokens;
    auto tile_at = [&](int round) { return cta0 + (int64_t)(round * Q + q) * a.tokens; };
    // token m of a tile exists
    auto token_in = [&](int64_t v0, int k) { return k < a.tokens && v0 + k < V; };

    // the warp's 32 rows of a block: eight rows of 64 bytes per instruction,
    // swizzled so that a thread's later 16-byte reads of its row hit all banks
    auto request = [&](int it) {
      if (it < steps) {
        const int64_t v0 = tile_at(it / nkb);
        const int kb = it % nkb, c = lane & 3;
        uint8_t* to = ring + (it % kCStages) * kCodeBytes;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = (lane >> 2) + 8 * j;
          const bool in = token_in(v0, w4 * 32 + r);
          const uint8_t* src = in ? a.wq + (v0 + w4 * 32 + r) * rowb + kb * 64 + c * 16 : a.wq;
          asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(
                           smem_u32(to + (r >> 1) * 128 + ((r & 1) * 4 + (c ^ ((r >> 1) & 3))) * 16)),
                       "l"(src), "r"(in ? 16 : 0)
                       : "memory");
        }
      }
      cp_async_commit();
    };
    // the token's scales of a block, as they lie in memory
    auto scales = [&](int it, uint32_t (&s)[P::kPer]) {
#pragma unroll
      for (int j = 0; j < P::kPer; ++j) s[j] = 0u;
      if (it >= steps) return;
      const int64_t v0 = tile_at(it / nkb);
      if (!token_in(v0, m)) return;
      const int64_t at = (v0 + m) * ng;
#pragma unroll
      for (int j = 0; j < P::kPer; ++j) {
        const int g = min((it % nkb) * P::kPer + j, ng - 1);
        s[j] = bf16_scales ? (uint32_t)__ldg((const unsigned short*)a.wscale + at + g)
                           : __ldg((const uint32_t*)a.wscale + at + g);
      }
    };

    const uint32_t tq = tmem + q * P::kCols;                      // the quartet's columns
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    const uint32_t idesc = idesc_bf16_f32(128, NC, false, false);
    // accumulator of group j of half block s (all groups of 128: of its block)
    auto d_at = [&](int s, int j) {
      const int buf = G == 128 ? (s >> 1) & 1 : G == 64 ? s & 1 : (s & 1) * 2 + j;
      return tq + 2 * kACols + buf * NC;
    };
    float total[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) total[c] = 0.f;

    // adds what half block s (of block it) accumulated, if a group ends with it
    auto gather = [&](int s, const uint32_t (&sc)[P::kPer]) {
      wait_for(&ctl->dfull[q][s & 1], (s >> 1) & 1, ctl, a.hdr, SITE_MBAR_MMA);
      tc_fence_after();
      if (G == 128 && (s & 1) == 0) return;
      constexpr int kGroups = G == 32 ? 2 : 1;
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const uint32_t raw = G == 32 ? ((s & 1) ? sc[(2 + j) % P::kPer] : sc[j % P::kPer])
                             : G == 64 ? ((s & 1) ? sc[1 % P::kPer] : sc[0]) : sc[0];
        const float scale = __uint_as_float(bf16_scales ? raw << 16 : raw);
#pragma unroll
        for (int c = 0; c < NC; c += 16) {
          float d[16];
          tmem_ld16(d_at(s, j) + lanes + c, d);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) total[c + k] = fmaf(scale, d[k], total[c + k]);
        }
      }
    };
    // the token's outputs, and zero again
    auto put = [&](int round) {
      const int64_t v0 = tile_at(round);
      const int b0 = blockIdx.y * a.rows, nb = min(a.rows, a.p.B - b0);
      if (token_in(v0, m)) {
        const int64_t v = v0 + m;
        constexpr int kEach = 8;  // rows whose base is read together: out may be base
#pragma unroll
        for (int b = 0; b < 16; b += kEach) {
          float z[kEach];
#pragma unroll
          for (int k = 0; k < kEach; ++k)
            z[k] = a.base && b + k < nb
                       ? load_any(a.base, a.p.base_dtype, (int64_t)(b0 + b + k) * a.p.base_stride + v)
                       : 0.f;
#pragma unroll
          for (int k = 0; k < kEach; ++k) {
            float sum;
            if (a.parts == 3) {
              constexpr int kLast = NC - 1;
              const int c = 3 * (b + k);
              sum = (total[c + 2 < NC ? c + 2 : kLast] + total[c + 1 < NC ? c + 1 : kLast]) +
                    total[c < NC ? c : kLast];
            } else {
              sum = total[b + k < NC ? b + k : 0];
            }
            if (b + k < nb)
              store_any(a.out, a.p.out_dtype, (int64_t)(b0 + b + k) * a.p.out_stride + v, z[k] + sum);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) total[c] = 0.f;
    };

#pragma unroll
    for (int k = 0; k < kCStages - 1; ++k) request(k);
    uint32_t s_old[P::kPer], s_now[P::kPer], s_next[P::kPer];
    scales(0, s_next);
#pragma unroll
    for (int j = 0; j < P::kPer; ++j) s_now[j] = 0u;
    for (int it = 0; it < steps; ++it) {
      cp_async_wait<kCStages - 2>();
      __syncwarp();
      uint4 w[4];  // chunk t: word t of each 32 features
      {
        const uint8_t* from = ring + (it % kCStages) * kCodeBytes + (lane >> 1) * 128;
#pragma unroll
        for (int t = 0; t < 4; ++t)
          w[t] = *reinterpret_cast<const uint4*>(from + ((lane & 1) * 4 + (t ^ ((lane >> 1) & 3))) * 16);
      }
      __syncwarp();
      request(it + kCStages - 1);
#pragma unroll
      for (int j = 0; j < P::kPer; ++j) {
        s_old[j] = s_now[j];
        s_now[j] = s_next[j];
      }
      scales(it + 1, s_next);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int s = 2 * it + h;
        {
          uint32_t pk[32];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t pair[4];
            codes_to_bf16(part_of(w[j & 3], 2 * h + (j >> 2)), pair);
#pragma unroll
            for (int k = 0; k < 4; ++k) pk[4 * j + k] = pair[k];
          }
          tmem_store32(tq + lanes + h * kACols, pk);
          tmem_st_wait();
        }
        tc_fence_before();
        asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory");
        if (w4 == 0 && lane == 0) {
          tc_fence_after();
          const int slot = it % kBStages;
          if (h == 0) wait_for(&ctl->bfull[slot], (it / kBStages) & 1, ctl, a.hdr, SITE_MBAR_FULL);
          const uint32_t b0 = smem_u32(sB + slot * P::kBBytes + h * (NC * 128));
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const int g = G == 32 ? ks >> 1 : 0;
            const bool first = G == 32 ? (ks & 1) == 0 : G == 64 ? ks == 0 : (h == 0 && ks == 0);
            umma_ts(d_at(s, g), tq + h * kACols + ks * 8, smem_desc_sw128(b0 + ks * 32, 16, 1024),
                    idesc, first ? 0u : 1u);
          }
          umma_commit(&ctl->dfull[q][h]);
          if (h == 1) umma_commit(&ctl->bempty[slot]);
        }
        __syncwarp();
        if (s > 0) {
          if (h == 0)
            gather(s - 1, s_old);
          else
            gather(s - 1, s_now);
          if (h == 0 && it % nkb == 0) put(it / nkb - 1);  // the tile before is whole
        }
      }
    }
    gather(2 * steps - 1, s_now);
    put(a.rounds - 1);
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Columns of X's parts for up to 16 rows, and the rows they hold.
int columns_of(const spec_w4_params& p) {
  if (p.dtype == SPEC_BF16) return 16;
  const int rows = std::min(p.B, 16);
  return rows <= 5 ? 16 : rows <= 10 ? 32 : 48;
}
int rows_of(const spec_w4_params& p, int NC) {
  return std::min(p.dtype == SPEC_BF16 ? NC : NC / 3, 16);
}

template <int NC, int G>
cudaError_t product(Args& a, int num_sms, cudaStream_t st) {
  using P = Plan<NC, G>;
  // as many quartets as fit, and tiles as full as an equal share per SM allows
  double best = 0.0;
  for (int Q = P::kMaxQ; Q >= 2; --Q) {
    const int64_t per = (int64_t)128 * Q * num_sms;
    const int rounds = (int)((a.p.V + per - 1) / per);
    const double full = (double)a.p.V / ((double)per * rounds) * (Q >= 3 ? 1.0 : 0.9);
    if (full > best) {
      best = full;
      a.quartets = Q;
      a.rounds = rounds;
    }
  }
  const int64_t tiles = (int64_t)num_sms * a.quartets * a.rounds;
  a.tokens = (int)((a.p.V + tiles - 1) / tiles);
  const int64_t per_cta = (int64_t)a.quartets * a.rounds * a.tokens;
  const int grid = (int)((a.p.V + per_cta - 1) / per_cta);
  const size_t smem = 1024 + kBStages * P::kBBytes +
                      (size_t)a.quartets * 4 * kCStages * kCodeBytes + sizeof(Ctl);
  const cudaError_t e = cudaFuncSetAttribute(
      k_bias_w4_tc<NC, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_after(k_bias_w4_tc<NC, G>, dim3(grid, (a.p.B + a.rows - 1) / a.rows),
                      a.quartets * 128 + 32, smem, st, a);
}

}  // namespace

bool w4_tc_fits(const spec_w4_params& p, int num_sms) { return p.V >= 64 * num_sms; }

size_t w4_tc_ws_bytes(const spec_w4_params& p) {
  const int NC = columns_of(p), rows = rows_of(p, NC);
  return (size_t)NC * 256 * ((p.r + 127) / 128) * ((p.B + rows - 1) / rows);
}

template <typename T>
cudaError_t launch_bias_w4_tc(const spec_w4_params& p, const T* x, const int32_t* prev,
                              const uint8_t* wq, const void* wscale, const void* base, void* out,
                              uint8_t* body, WsHeader* hdr, int num_sms, cudaStream_t st,
                              int* launches) {
  const int NC = columns_of(p);
  Args a = {};
  a.p = p;
  a.xf = body;
  a.wq = wq;
  a.wscale = wscale;
  a.base = base;
  a.out = out;
  a.hdr = hdr;
  a.rows = rows_of(p, NC);
  a.parts = XWord<T>::kParts;
  if ((p.B + a.rows - 1) / a.rows > 65535) return cudaErrorInvalidValue;
  const int64_t words = (int64_t)p.B * ((p.r + 127) / 128 * 16);
  k_w4_x_tc<T><<<(unsigned)((words + 255) / 256), 256, 0, st>>>(
      p, x, prev, reinterpret_cast<uint4*>(body), NC, a.rows, x_wide(p, x), hdr);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  *launches = 2;
  if (NC == 16)
    return p.group == 32   ? product<16, 32>(a, num_sms, st)
           : p.group == 64 ? product<16, 64>(a, num_sms, st)
                           : product<16, 128>(a, num_sms, st);
  if (NC == 32)
    return p.group == 32   ? product<32, 32>(a, num_sms, st)
           : p.group == 64 ? product<32, 64>(a, num_sms, st)
                           : product<32, 128>(a, num_sms, st);
  return p.group == 32   ? product<48, 32>(a, num_sms, st)
         : p.group == 64 ? product<48, 64>(a, num_sms, st)
                         : product<48, 128>(a, num_sms, st);
}

#define SPEC_INST(T)                                                                               \
  template cudaError_t launch_bias_w4_tc<T>(const spec_w4_params&, const T*, const int32_t*,       \
                                            const uint8_t*, const void*, const void*, void*,       \
                                            uint8_t*, WsHeader*, int, cudaStream_t, int*);
SPEC_INST(float)
SPEC_INST(__nv_bfloat16)
#undef SPEC_INST

}  // namespace specdec
