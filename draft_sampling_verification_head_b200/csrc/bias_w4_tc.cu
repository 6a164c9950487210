// Vocabulary product with 4-bit weights on tcgen05, for vocabularies that fill the
// GPU: out[b, v] = base[b, v] + sum_g s[v, g] sum_{k in g} X[b, k] (code[v, k] - 8).
//
// Tokens lie on M: a tile is 128 of them, a thread of a quartet of warps each.  The
// thread turns its token's codes into bf16 (exact) and stores them as the A operand
// in tensor memory, 64 features at a time; X (as many bf16 columns as its type
// needs: one, or three whose sum is an fp32 exactly) is the B operand in shared
// memory.  The MMA of a group of features adds into an accumulator of its own;
// the thread reads it back, scales it in fp32 and adds it to its token's sums in
// registers, so no scaled weight is ever rounded.  A warp of its own issues the
// quartet's MMAs; while they run the quartet unpacks the next half blocks.
//
// A CTA per SM runs up to three quartets on tiles of their own in step, so that a
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
  static constexpr int kPer = 128 / G;  // groups per block
  // half blocks between a store of A and the reading of its products, as many as
  // tensor memory allows: an MMA's way there and back takes longer than a half block
  static constexpr int kLag = NC > 16 && G == 32 ? 1 : 2;
  static constexpr int kA = kLag + 1;   // A buffers
  static constexpr int kDBufs = G == 128 ? 2 : G == 64 ? kA : 2 * kA;  // accumulators
  static constexpr int kCols = kA * kACols + kDBufs * NC;  // tensor memory per quartet
  // quartets that tensor memory and the register file hold
  static constexpr int kMaxQ = 512 / kCols < 3 ? 512 / kCols : 3;
  static constexpr int kBBytes = NC * 256;  // a block of X
  static constexpr int kThreadsMax = kMaxQ * 160 + 32;
  static_assert(kMaxQ >= 2, "tensor memory");
};

struct Ctl {
  uint64_t bfull[kBStages], bempty[kBStages];
  uint64_t aready[4][3], dfull[4][3];
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

template <typename TS, int NC, int G>
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
      for (int i = 0; i < P::kA; ++i) {
        mbar_init(&ctl->aready[q][i], 4);
        mbar_init(&ctl->dfull[q][i], 1);
      }
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

  // accumulator of group j of half block s (all groups of 128: of its block), as
  // a column of the quartet's
  auto d_at = [&](int s, int j) {
    const int buf = G == 128 ? (s >> 1) & 1 : G == 64 ? s % P::kA : (s % P::kA) * 2 + j;
    return P::kA * kACols + buf * NC;
  };

  if (warp == 5 * Q) {
    // ---- blocks of X through the ring ----
    if (lane == 0) {
      grid_dependency_wait();
      const uint8_t* src = a.xf + (int64_t)blockIdx.y * nkb * P::kBBytes;
      const uint64_t policy = policy_evict_last();
      for (int it = 0, kb = 0; it < steps; ++it) {
        const int slot = it % kBStages;
        if (it >= kBStages)
          wait_for(&ctl->bempty[slot], (it / kBStages - 1) & 1, ctl, a.hdr, SITE_MBAR_BASE);
        if (ld_volatile_u32(&ctl->failed)) break;
        mbar_arrive_expect_tx(&ctl->bfull[slot], P::kBBytes);
        bulk_load(sB + slot * P::kBBytes, src + (int64_t)kb * P::kBBytes, P::kBBytes,
                  &ctl->bfull[slot], policy);
        if (++kb == nkb) kb = 0;
      }
      // the last blocks' commits land before the CTA may end
      for (int it = max(steps - kBStages, 0); it < steps; ++it)
        wait_for(&ctl->bempty[it % kBStages], (it / kBStages) & 1, ctl, a.hdr, SITE_MBAR_BASE);
    }
    __syncwarp();
  } else if (warp >= 4 * Q) {
    // ---- a quartet's matrix instructions, by one thread ----
    if (lane == 0) {
      const int q = warp - 4 * Q;
      const uint32_t tq = tmem + q * P::kCols;
      const uint32_t idesc = idesc_bf16_f32(128, NC, false, false);
      uint32_t buf = 0, par = 0;  // s % kA, (s / kA) & 1
      for (int s = 0; s < 2 * steps; ++s) {
        const int it = s >> 1, slot = it % kBStages;
        wait_for(&ctl->aready[q][buf], par, ctl, a.hdr, SITE_MBAR_BREADY);
        if ((s & 1) == 0) wait_for(&ctl->bfull[slot], (it / kBStages) & 1, ctl, a.hdr, SITE_MBAR_FULL);
        tc_fence_after();
        const uint32_t b0 = smem_u32(sB + slot * P::kBBytes + (s & 1) * (NC * 128));
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const int g = G == 32 ? ks >> 1 : 0;
          const bool first = G == 32 ? (ks & 1) == 0 : G == 64 ? ks == 0 : ((s & 1) == 0 && ks == 0);
          umma_ts(tq + d_at(s, g), tq + buf * kACols + ks * 8, smem_desc_sw128(b0 + ks * 32, 16, 1024),
                  idesc, first ? 0u : 1u);
        }
        umma_commit(&ctl->dfull[q][buf]);
        if (s & 1) umma_commit(&ctl->bempty[slot]);
        if (++buf == P::kA) {
          buf = 0;
          par ^= 1;
        }
      }
    }
    __syncwarp();
  } else {
    const int q = warp >> 2, w4 = warp & 3, m = w4 * 32 + lane;  // the thread's token of the tile
    uint8_t* ring = sC + (size_t)warp * kCStages * kCodeBytes;
    const int rowb = nkb * 64, ng = a.p.r / G;
    const int64_t cta0 = (int64_t)blockIdx.x * a.rounds * Q * a.tokens;
    auto tile_at = [&](int round) { return cta0 + (int64_t)(round * Q + q) * a.tokens; };
    // token m of a tile exists
    auto token_in = [&](int64_t v0, int k) { return k < a.tokens && v0 + k < V; };

    // the warp's 32 rows of a block: eight rows of 64 bytes per instruction,
    // swizzled so that a thread's later 16-byte reads of its row hit all banks.
    // Blocks are asked for in order, so places advance by addition.
    int r_round = 0, r_kb = 0, r_slot = 0;
    const uint8_t* r_src = nullptr;
    bool r_in[4];
    const uint32_t r_to = smem_u32(ring) + (lane >> 3) * 128 +
                          (((lane >> 2) & 1) * 4 + ((lane & 3) ^ ((lane >> 3) & 3))) * 16;
    const int64_t row8 = (int64_t)8 * rowb;
    auto request = [&]() {
      if (r_round < a.rounds) {
        if (r_kb == 0) {
          const int64_t v0 = tile_at(r_round);
          const int r = w4 * 32 + (lane >> 2);
          r_src = a.wq + (v0 + r) * rowb + (lane & 3) * 16;
#pragma unroll
          for (int j = 0; j < 4; ++j) r_in[j] = token_in(v0, r + 8 * j);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // row + 8 j: four lines of 128 bytes further
          const uint8_t* src = r_in[j] ? r_src + j * row8 : a.wq;
          asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(
                           r_to + r_slot * kCodeBytes + j * 512),
                       "l"(src), "r"(r_in[j] ? 16 : 0)
                       : "memory");
        }
        r_src += 64;
        if (++r_slot == kCStages) r_slot = 0;
        if (++r_kb == nkb) {
          r_kb = 0;
          ++r_round;
        }
      }
      cp_async_commit();
    };
    // the token's scales of the next block, as they lie in memory: loads without
    // a condition (rows and groups that do not exist read ones that do, and scale
    // zeros), so that nothing waits for them before they are used
    int c_round = 0, c_kb = 0;
    const TS* c_src = nullptr;
    auto scales = [&](TS (&s)[P::kPer]) {
      if (c_kb == 0)
        c_src = (const TS*)a.wscale + min(tile_at(min(c_round, a.rounds - 1)) + m, (int64_t)V - 1) * ng;
#pragma unroll
      for (int j = 0; j < P::kPer; ++j) s[j] = c_src[min(c_kb * P::kPer + j, ng - 1)];
      if (++c_kb == nkb) {
        c_kb = 0;
        ++c_round;
      }
    };

    const uint32_t tq = tmem + q * P::kCols + ((uint32_t)(w4 * 32) << 16);  // its columns, own lanes
    float total[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) total[c] = 0.f;

    // adds what half block s accumulated, if a group ends with it; half blocks are
    // gathered in order
    uint32_t g_buf = 0, g_par = 0;
    auto gather = [&](int s, int half, const TS (&sc)[P::kPer]) {
      wait_for(&ctl->dfull[q][g_buf], g_par, ctl, a.hdr, SITE_MBAR_MMA);
      if (++g_buf == P::kA) {
        g_buf = 0;
        g_par ^= 1;
      }
      tc_fence_after();
      if (G == 128 && half == 0) return;
      constexpr int kGroups = G == 32 ? 2 : 1;
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const TS raw = G == 32 ? (half ? sc[(2 + j) % P::kPer] : sc[j % P::kPer])
                       : G == 64 ? (half ? sc[1 % P::kPer] : sc[0]) : sc[0];
        const float scale = (float)raw;
#pragma unroll
        for (int c = 0; c < NC; c += 16) {
          float d[16];
          tmem_ld16(tq + d_at(s, j) + c, d);
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
    for (int k = 0; k < kCStages - 1; ++k) request();
    // Two sets of scales, of even and of odd blocks; a set is asked for again as
    // soon as its block's last group has been gathered, a block before its next
    // use, and no copy of it in between waits for it.
    TS sc[2][P::kPer];
    scales(sc[0]);
    int round = 0, kb = 0;
    uint32_t a_buf = 0;  // half block % kA
    auto block = [&](int it, TS (&s_now)[P::kPer], TS (&s_other)[P::kPer]) {
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
      request();
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
          tmem_store32(tq + a_buf * kACols, pk);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->aready[q][a_buf]);
        if (++a_buf == P::kA) a_buf = 0;
        // what lies kLag half blocks back; this store's buffer comes free with it
        if constexpr (P::kLag == 1) {
          if (h == 1) {
            gather(s - 1, 0, s_now);
          } else {
            if (it > 0) gather(s - 1, 1, s_other);
            if (kb == 0 && it > 0) put(round - 1);  // the tile before is whole
            scales(s_other);
          }
        } else {
          if (it > 0) gather(s - 2, h, s_other);
          if (h == 1) {
            if (kb == 0 && it > 0) put(round - 1);
            scales(s_other);
          }
        }
      }
      if (++kb == nkb) {
        kb = 0;
        ++round;
      }
    };
    for (int it = 0; it < steps; it += 2) {
      block(it, sc[0], sc[1]);
      if (it + 1 < steps) block(it + 1, sc[1], sc[0]);
    }
    TS(&s_last)[P::kPer] = sc[(steps & 1) ? 0 : 1];
    if constexpr (P::kLag == 2) gather(2 * steps - 2, 0, s_last);
    gather(2 * steps - 1, 1, s_last);
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

template <typename TS, int NC, int G>
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
      k_bias_w4_tc<TS, NC, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_after(k_bias_w4_tc<TS, NC, G>, dim3(grid, (a.p.B + a.rows - 1) / a.rows),
                      a.quartets * 160 + 32, smem, st, a);
}

template <typename TS>
cudaError_t by_shape(Args& a, int NC, int num_sms, cudaStream_t st) {
  const int G = a.p.group;
  if (NC == 16)
    return G == 32   ? product<TS, 16, 32>(a, num_sms, st)
           : G == 64 ? product<TS, 16, 64>(a, num_sms, st)
                     : product<TS, 16, 128>(a, num_sms, st);
  if (NC == 32)
    return G == 32   ? product<TS, 32, 32>(a, num_sms, st)
           : G == 64 ? product<TS, 32, 64>(a, num_sms, st)
                     : product<TS, 32, 128>(a, num_sms, st);
  return G == 32   ? product<TS, 48, 32>(a, num_sms, st)
         : G == 64 ? product<TS, 48, 64>(a, num_sms, st)
                   : product<TS, 48, 128>(a, num_sms, st);
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
  return p.scale_dtype == SPEC_BF16 ? by_shape<__nv_bfloat16>(a, NC, num_sms, st)
                                    : by_shape<float>(a, NC, num_sms, st);
}

#define SPEC_INST(T)                                                                               \
  template cudaError_t launch_bias_w4_tc<T>(const spec_w4_params&, const T*, const int32_t*,       \
                                            const uint8_t*, const void*, const void*, void*,       \
                                            uint8_t*, WsHeader*, int, cudaStream_t, int*);
SPEC_INST(float)
SPEC_INST(__nv_bfloat16)
#undef SPEC_INST

}  // namespace specdec
