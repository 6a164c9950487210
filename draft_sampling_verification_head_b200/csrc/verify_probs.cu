// Verification of drafted tokens from probabilities and given uniforms.
//
// A cluster of CTAs takes a batch row.  The accept chain touches two numbers per
// position; every CTA follows it by itself.  Then one row of the target (and one
// of the draft, where a draft was rejected) is read once: its tiles of 256 tokens
// are dealt to the warps in contiguous chunks, whose masses are summed in 64 bits
// and sent to all CTAs of the cluster.  Each warp sees from the chunks' sums
// whether the drawn token lies in its own; the one that holds it reads its chunk
// again (from L2) and finds the token.  The order of these 64-bit sums is fixed by
// the sizes and the device.  A sum of n terms, none negative, each rounded once, is
// off by at most n 2^-53 of itself in any order; so are the total and the mass up to
// a token, and another order can only decide otherwise where the draw lies within
// (n + 2) 2^-52 of the total of the token's border (n = 151936: 3.4e-11).
//
// What bounds it: the rows' bytes, behind a chain of dependent reads (lengths,
// drafts, their probabilities, the row, the chunk again) that a row's CTAs go
// through one after the other, so three CTAs an SM overlap their chains
// (256 x 8 x 151936 fp32, 75 us, 3.8 TB/s; two CTAs of more registers 77;
// four tiles ahead instead of two 115).
#include <cooperative_groups.h>

#include <type_traits>

#include "head_ops.cuh"

namespace cg = cooperative_groups;

namespace specdec {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kEach = 8;            // tokens per lane and tile
constexpr int kTile = 32 * kEach;   // tokens per tile of a warp

// What a token adds to the mass: p (0 for NaN, infinities and negative values), or
// max(p - q, 0) with a q that is NaN or negative counting as 0.  The difference
// of two fp32 is exact in 64 bits but for exponents 29 apart.
template <bool kRes>
SPEC_DEV void add_mass(double& sum, float p, float q) {
  if constexpr (kRes) {
    q = fmaxf(q, 0.f);
    const double d = (double)p - (double)q;
    if (q < p && p < INFINITY) sum += d;
  } else {
    const double d = (double)p;
    if (p > 0.f && p < INFINITY) sum += d;
  }
}

// A lane's tokens v .. v + 7 as they lie in memory.
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
  SPEC_DEV void load(const T* row, int v, int V, bool wide) {
    if (wide && v + kEach <= V) {
#pragma unroll
      for (int k = 0; k < (int)sizeof(T) / 2; ++k)
        w[k] = __ldg(reinterpret_cast<const uint4*>(row + v) + k);
      return;
    }
    uint32_t u[2 * sizeof(T)];
#pragma unroll
    for (int k = 0; k < (int)(2 * sizeof(T)); ++k) {
      if constexpr (sizeof(T) == 4) {
        u[k] = v + k < V ? __ldg(reinterpret_cast<const uint32_t*>(row) + v + k) : 0u;
      } else {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(row);
        const uint32_t lo = v + 2 * k < V ? __ldg(h + v + 2 * k) : 0u;
        const uint32_t hi = v + 2 * k + 1 < V ? __ldg(h + v + 2 * k + 1) : 0u;
        u[k] = lo | hi << 16;
      }
    }
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k)
      w[k] = make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
  }
  SPEC_DEV float get(int k) const {
    const int word = sizeof(T) == 4 ? k : k >> 1;
    const uint4& q = w[word >> 2];
    const uint32_t u = (word & 3) == 0 ? q.x : (word & 3) == 1 ? q.y : (word & 3) == 2 ? q.z : q.w;
    if constexpr (sizeof(T) == 4) return __uint_as_float(u);
    return __uint_as_float((k & 1) ? (u & 0xFFFF0000u) : (u << 16));
  }
};

SPEC_DEV double shfl_up(double v, int d) { return __shfl_up_sync(0xffffffffu, v, d); }

// Sum over the lanes up to the calling one.
SPEC_DEV double warp_prefix(double v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = shfl_up(v, o);
    if (lane >= o) v += y;
  }
  return v;
}

struct ProbsArgs {
  spec_probs_params p;
  const int32_t* draft;
  const float* u_accept;
  const float* u_draw;
  const int32_t* verify_len;
  int32_t* out;
  int32_t* tau;
  float* p_draft;
  float* q_draft;
  WsHeader* hdr;
  int cluster;
  int wide;  // bit 0: target rows on 16-byte boundaries, bit 1: draft rows
};

template <typename T, typename TD>
__global__ void __launch_bounds__(kThreads, 3)
    k_verify_probs(ProbsArgs a, const T* __restrict__ target, const TD* __restrict__ draft_probs) {
  __shared__ double chunk[2][kMaxCluster * kWarps];  // mass of every chunk of the row
  __shared__ int stop;
  const int C = a.cluster, rank = blockIdx.x % C, b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, K = a.p.K, V = a.p.V;
  const T* P = target + (int64_t)b * (K + 1) * a.p.target_stride;
  const TD* Q = draft_probs + (int64_t)b * K * a.p.draft_stride;
  const int64_t row = (int64_t)b * K;

  int kb = a.verify_len ? __ldg(a.verify_len + b) : K;
  if (kb < 0) return;  // a row to skip: the whole cluster leaves
  if (kb > K) {
    if (tid == 0 && rank == 0) report_error(a.hdr, SPEC_ERR_INVALID_ARG, SITE_NONE, b, kb);
    kb = K;
  }
  if (C > 1) cg::this_cluster().barrier_arrive();  // waited for before another CTA is written to
  const float u_draw = __ldg(a.u_draw + b);
  // the first position whose test fails; every position's two numbers are read,
  // all at once, those after it for nothing
  int first = kb;
  for (int i0 = 0; i0 < kb && first == kb; i0 += kThreads) {
    const int i = i0 + tid;
    bool fails = false;
    float pv = 0.f, qv = 0.f;
    int d = 0;
    if (i < kb) {
      d = __ldg(a.draft + row + i);
      const float u = __ldg(a.u_accept + row + i);
      if (d >= 0 && d < V) {
        pv = load_f(P, i * a.p.target_stride + d);
        qv = load_f(Q, i * a.p.draft_stride + d);
        fails = !((double)u * (double)qv < (double)pv);
      } else {
        fails = true;
      }
    }
    if (tid == 0) stop = kb;
    __syncthreads();
    if (fails) atomicMin(&stop, i);
    __syncthreads();
    first = stop;
    if (rank == 0 && i < kb && i <= first) {
      const bool bad = d < 0 || d >= V;
      if (bad) report_error(a.hdr, SPEC_ERR_TOKEN_RANGE, SITE_TOKEN_RANGE, (int)min(row + i, (int64_t)INT32_MAX), d);
      if (a.p_draft) a.p_draft[row + i] = bad ? NAN : pv;
      if (a.q_draft) a.q_draft[row + i] = bad ? NAN : qv;
    }
    __syncthreads();
  }
  const int j = first;
  const bool bonus = j == kb;
  if (rank == 0) {
    for (int i = tid; i < K; i += kThreads) {
      if (i > j || i >= kb) {  // no test ran here
        if (a.p_draft) a.p_draft[row + i] = NAN;
        if (a.q_draft) a.q_draft[row + i] = NAN;
      }
    }
    for (int i = tid; i <= K; i += kThreads)
      if (i != j) a.out[row + b + i] = i < j ? __ldg(a.draft + row + i) : -1;
  }
  P += j * a.p.target_stride;
  Q += (bonus ? 0 : j) * a.p.draft_stride;
  const bool wide_p = a.wide & 1, wide_q = a.wide & 2;

  const int tiles = (V + kTile - 1) / kTile, chunks = C * kWarps, mine = rank * kWarps + warp;
  const int t0 = (int)((int64_t)tiles * mine / chunks), t1 = (int)((int64_t)tiles * (mine + 1) / chunks);
  // the chunk's mass; two tiles are requested ahead of the two being added
  auto sum_chunk = [&](auto res) {
    constexpr bool kRes = decltype(res)::value;
    constexpr int kAhead = 2;
    Eight<T> pw[kAhead], pn[kAhead];
    Eight<TD> qw[kAhead], qn[kAhead];
    auto fetch = [&](int t, Eight<T>(&pe)[kAhead], Eight<TD>(&qe)[kAhead]) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int v = t + k < t1 ? (t + k) * kTile + lane * kEach : V;  // V: nothing, zeros
        pe[k].load(P, v, V, wide_p);
        if (kRes) qe[k].load(Q, v, V, wide_q);
      }
    };
    double sum[2] = {0.0, 0.0};
    if (t0 < t1) fetch(t0, pw, qw);
    for (int t = t0; t < t1; t += kAhead) {
      if (t + kAhead < t1) fetch(t + kAhead, pn, qn);
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
#pragma unroll
        for (int e = 0; e < kEach; ++e)
          add_mass<kRes>(sum[k], pw[k].get(e), kRes ? qw[k].get(e) : 0.f);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        pw[k] = pn[k];
        qw[k] = qn[k];
      }
    }
    double all = sum[0] + sum[1];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    return all;
  };
  // the chunk sums of the whole row in every CTA; round 1 only where a residual
  // has no mass at all
  auto share = [&](double mass, int round) {
    if (C > 1) {
      cg::cluster_group cl = cg::this_cluster();
      if (round == 0) cl.barrier_wait();
      if (lane < C) cl.map_shared_rank(&chunk[round][0], lane)[mine] = mass;
      cl.sync();
    } else {
      if (lane == 0) chunk[round][mine] = mass;
      __syncthreads();
    }
  };
  bool from_res = !bonus;
  int round = 0;
  share(bonus ? sum_chunk(std::false_type()) : sum_chunk(std::true_type()), 0);
  // Every warp alike: the total, and the first chunk that passes the draw (else
  // the last one with mass).  Lane l holds chunks 2 l and 2 l + 1.
  double m0, m1;
  auto look = [&]() {
    m0 = 2 * lane < chunks ? chunk[round][2 * lane] : 0.0;
    m1 = 2 * lane + 1 < chunks ? chunk[round][2 * lane + 1] : 0.0;
    return __any_sync(0xffffffffu, m0 > 0.0 || m1 > 0.0);
  };
  if (!look() && from_res) {
    from_res = false;
    round = 1;
    share(sum_chunk(std::false_type()), 1);
    look();
  }
  const double pre = warp_prefix(m0 + m1), total = __shfl_sync(0xffffffffu, pre, 31);
  const double goal = fmax((double)u_draw, 0.0) * total;
  const double up = __shfl_up_sync(0xffffffffu, pre, 1);
  const double start0 = lane == 0 ? 0.0 : up, start1 = start0 + m0;
  const uint32_t over0 = __ballot_sync(0xffffffffu, m0 > 0.0 && start1 > goal);
  const uint32_t over1 = __ballot_sync(0xffffffffu, m1 > 0.0 && pre > goal);
  const uint32_t any0 = __ballot_sync(0xffffffffu, m0 > 0.0), any1 = __ballot_sync(0xffffffffu, m1 > 0.0);
  int owner = -1;
  if (over0 | over1) {
    const int l0 = over0 ? 2 * (__ffs(over0) - 1) : 1 << 20, l1 = over1 ? 2 * (__ffs(over1) - 1) + 1 : 1 << 20;
    owner = min(l0, l1);
  } else if (any0 | any1) {
    owner = max(any0 ? 2 * (31 - __clz(any0)) : -1, any1 ? 2 * (31 - __clz(any1)) + 1 : -1);
  }
  if (rank == 0 && tid == 0) {
    a.tau[b] = j + (owner >= 0);
    if (owner < 0) {
      a.out[row + b + j] = -1;
      report_error(a.hdr, SPEC_ERR_INVALID_ARG, SITE_NONE, b, j);
    }
  }
  if (owner != mine) return;

  // this warp's chunk holds the token
  double cum = __shfl_sync(0xffffffffu, (mine & 1) ? start1 : start0, mine >> 1);
  int tok = -1;
  Eight<T> pw, pn;
  Eight<TD> qw, qn;
  auto fetch = [&](int t, Eight<T>& pe, Eight<TD>& qe) {
    const int v = t < t1 ? t * kTile + lane * kEach : V;
    pe.load(P, v, V, wide_p);
    if (from_res) qe.load(Q, v, V, wide_q);
  };
  fetch(t0, pw, qw);
  for (int t = t0; t < t1; ++t) {
    fetch(t + 1, pn, qn);
    double m[kEach], sum = 0.0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      m[e] = 0.0;
      if (from_res)
        add_mass<true>(m[e], pw.get(e), qw.get(e));
      else
        add_mass<false>(m[e], pw.get(e), 0.f);
      sum += m[e];
    }
    const double incl = warp_prefix(sum);
    const uint32_t has = __ballot_sync(0xffffffffu, sum > 0.0);
    const uint32_t over = __ballot_sync(0xffffffffu, sum > 0.0 && cum + incl > goal);
    if (has) {  // the token, or the last one with mass so far
      const int l = over ? __ffs(over) - 1 : 31 - __clz(has);
      double c = cum + (incl - sum);
      int hit = -1, last = -1;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        c += m[e];
        if (m[e] > 0.0) {
          last = e;
          if (hit < 0 && c > goal) hit = e;
        }
      }
      const int pick = over && hit >= 0 ? hit : last;
      tok = t * kTile + l * kEach + __shfl_sync(0xffffffffu, pick, l);
      if (over) break;
    }
    cum += __shfl_sync(0xffffffffu, incl, 31);
    pw = pn;
    qw = qn;
  }
  if (lane == 0) a.out[row + b + j] = tok;
}

}  // namespace

template <typename T, typename TD>
cudaError_t launch_verify_probs(const spec_probs_params& p, const T* target, const TD* draft_probs,
                                const int32_t* draft, const float* u_accept, const float* u_draw,
                                const int32_t* verify_len, int32_t* out, int32_t* tau,
                                float* p_draft, float* q_draft, WsHeader* hdr, int num_sms,
                                cudaStream_t st, int* launches) {
  ProbsArgs a = {};
  a.p = p;
  a.draft = draft;
  a.u_accept = u_accept;
  a.u_draw = u_draw;
  a.verify_len = verify_len;
  a.out = out;
  a.tau = tau;
  a.p_draft = p_draft;
  a.q_draft = q_draft;
  a.hdr = hdr;
  auto rows_wide = [](const void* x, int64_t stride, size_t es) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && stride * es % 16 == 0;
  };
  a.wide = (rows_wide(target, p.target_stride, sizeof(T)) ? 1 : 0) |
           (rows_wide(draft_probs, p.draft_stride, sizeof(TD)) ? 2 : 0);
  // CTAs per row: enough for eight on every SM (three run at a time; rows that
  // draw from one distribution end sooner than those that compare two), while
  // each warp has tiles.  From cold caches, 256 rows of 151936 take 82 us (with
  // four on every SM 85), 1024 rows of 32000 72 (74).
  const int tiles = (p.V + kTile - 1) / kTile;
  int C = 1;
  while (C < kMaxCluster && (int64_t)p.B * C < 8 * num_sms && 2 * C * kWarps <= tiles) C *= 2;
  a.cluster = C;
  if ((int64_t)p.B * C > INT32_MAX) return cudaErrorInvalidValue;
  *launches = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = C;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_verify_probs<T, TD>, a, target, draft_probs);
}

#define SPEC_INST(T, TD)                                                                           \
  template cudaError_t launch_verify_probs<T, TD>(                                                 \
      const spec_probs_params&, const T*, const TD*, const int32_t*, const float*, const float*,   \
      const int32_t*, int32_t*, int32_t*, float*, float*, WsHeader*, int, cudaStream_t, int*);
SPEC_INST(float, float)
SPEC_INST(float, __nv_bfloat16)
SPEC_INST(__nv_bfloat16, float)
SPEC_INST(__nv_bfloat16, __nv_bfloat16)
#undef SPEC_INST

}  // namespace specdec
