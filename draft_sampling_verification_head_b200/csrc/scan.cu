// Gated linear recurrence over sequences, h_t = f_t h_{t-1} + (1 - f_t) x_t
// with f = sigmoid(gate), and its gradient.
//
// A step is the affine map h -> f h + z, z = (1 - f) x, and maps compose:
// (f2, z2) after (f1, z1) is (f1 f2, f2 z1 + z2).  So a long sequence is cut
// into pieces of kChunk steps, one per warp, which are reduced to one map per
// channel each while their f and z stay in registers; the maps are joined in
// time order (warps of a CTA through shared memory, CTAs of a cluster through
// each other's shared memory), which gives every piece the state it starts
// from, and the pieces are run once more from there.  Inputs are read once and
// outputs written once, whatever the length; equal inputs give equal bits since
// the joins are taken in a fixed order.
//
// What bounds it: bytes where jobs fill the GPU (forward, 256 x 256 x 1024 bf16:
// 78 us, 5.2 TB/s), instruction issue and the joins' barriers in the gradient
// (8 x 8192 x 1024 bf16: 175 us, 3.9 TB/s; about 45 instructions a pair of
// elements, the issue slots half used), the chain of dependent steps and launches
// where work is small.  Clusters of 16, of which only part fits the GPU, took
// 96 us where 8 took 85; a cluster barrier in place of the counted stores 186
// against 172.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "head_ops.cuh"

namespace cg = cooperative_groups;

namespace specdec {
namespace {

constexpr int kChunk = SPEC_SCAN_CHUNK;  // steps per piece
constexpr int kMaxCluster = 8;           // CTAs per cluster (portable limit)
constexpr int kSoloWarps = 8;            // warps per CTA where each has a job of its own
constexpr int kSplitSteps = 5120;        // shortest sequence whose steps are split
constexpr int kMinSegment = 64;          // shortest segment
constexpr int kStages = 2;               // pieces of a warp on their way, forward

SPEC_DEV int len_of(const int32_t* len, int b, int T, WsHeader* hdr, bool say) {
  if (!len) return T;
  const int n = len[b];
  if (n >= 0 && n <= T) return n;
  if (say) report_error(hdr, SPEC_ERR_INVALID_ARG, SITE_NONE, b, n);
  return n < 0 ? 0 : T;
}

// ----------------------------------------------------------------------------
// V fp32 values of one thread: V = 2 in one 64-bit register on the packed pipe
// (each lane rounded exactly like the scalar operation), which halves the issue
// slots that bound these kernels.
// ----------------------------------------------------------------------------
template <int V>
struct Vec;
template <>
struct Vec<1> {
  float v;
  SPEC_DEV static Vec all(float a) { return {a}; }
  SPEC_DEV float get(int) const { return v; }
  SPEC_DEV friend Vec operator+(Vec a, Vec b) { return {a.v + b.v}; }
  SPEC_DEV friend Vec operator*(Vec a, Vec b) { return {a.v * b.v}; }
  SPEC_DEV friend Vec fma(Vec a, Vec b, Vec c) { return {fmaf(a.v, b.v, c.v)}; }
  template <typename F>
  SPEC_DEV Vec map(F f) const { return {f(v)}; }
};
template <>
struct Vec<2> {
  uint64_t v;
  SPEC_DEV static Vec of(float a, float b) {
    Vec r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
  }
  SPEC_DEV static Vec all(float a) { return of(a, a); }
  SPEC_DEV float get(int k) const {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    return k ? b : a;
  }
  SPEC_DEV friend Vec operator+(Vec a, Vec b) {
    Vec r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
  }
  SPEC_DEV friend Vec operator*(Vec a, Vec b) {
    Vec r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
  }
  SPEC_DEV friend Vec fma(Vec a, Vec b, Vec c) {
    Vec r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
  }
  template <typename F>
  SPEC_DEV Vec map(F f) const { return of(f(get(0)), f(get(1))); }
};

// V channels of one step as they lie in memory: a float, two bf16, or a single
// bf16 where width or alignment leave no pairs or channels are few.
template <typename T, int V>
using RawOf = std::conditional_t<std::is_same<T, float>::value || V == 2, uint32_t, uint16_t>;

template <typename T, int V>
SPEC_DEV Vec<V> raw_value(RawOf<T, V> r) {
  if constexpr (std::is_same<T, float>::value)
    return {__uint_as_float(r)};
  else if constexpr (V == 2)
    return Vec<2>::of(__uint_as_float(r << 16), __uint_as_float(r & 0xFFFF0000u));
  else
    return {__uint_as_float((uint32_t)r << 16)};
}
template <typename T, int V>
SPEC_DEV void raw_store(T* p, Vec<V> x) {
  if constexpr (std::is_same<T, float>::value)
    *p = x.get(0);
  else if constexpr (V == 2)
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x.get(0), x.get(1));
  else
    *p = __float2bfloat16_rn(x.get(0));
}

// f = sigmoid(g) = 1 / (1 + e), i = 1 - f = e f with e = exp(-g), so neither is
// found by cancellation.  g is clamped to [-87, 87], where e, f and i stay normal
// numbers above 0: nothing in fp32's range is lost by it, and an infinite state or
// input stays infinite; a NaN passes.  e = 2^t (1 + d) where t
// is -g log2(e) rounded to fp32 and d makes up for that rounding, which for
// large |g| would cost more than the rest together.
template <typename T, int V>
SPEC_DEV void gate_of(RawOf<T, V> raw, Vec<V>& f, Vec<V>& i) {
  constexpr float kLn2 = 0.69314718056f;
  Vec<V> t, d;
  if constexpr (std::is_same<T, float>::value) {
    float g = __uint_as_float(raw);
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(g) : "f"(g), "f"(-87.f));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(g) : "f"(g), "f"(87.f));
    constexpr float kL = 1.44269504089f;
    t.v = g * -kL;
    d.v = fmaf(g, -kL, -t.v) * kLn2;
  } else {
    // bf16 has 8 significant bits: with the upper 16 of log2(e) the product is
    // exact, and the lower ones give d
    constexpr float kHi = 1.44268798828125f;  // 47274 / 2^15
    constexpr float kLo = (float)(1.4426950408889634 - 47274.0 / 32768.0);
    uint32_t g2 = raw;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(g2) : "r"(g2), "r"(0xC2AEC2AEu));  // -87
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(g2) : "r"(g2), "r"(0x42AE42AEu));  // 87
    const Vec<V> g = raw_value<T, V>((RawOf<T, V>)g2);
    t = g * Vec<V>::all(-kHi);
    d = g * Vec<V>::all(-kLo * kLn2);
  }
  Vec<V> e = t.map([](float x) { return fexp2(x); });
  e = fma(e, d, e);
  f = (e + Vec<V>::all(1.f)).map([](float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
  });
  i = e * f;
}

// A product of gates is above 0, however many: where it leaves fp32's range it is
// held at the smallest normal number, so that an infinite state times it stays
// infinite.  A finite state s gains less than s 2^-126 by it.
SPEC_DEV float above_zero(float product) { return fmaxf(product, 1.17549435e-38f); }

struct ScanArgs {
  spec_scan_params p;
  const void* gate;
  const void* x;
  const float* h0;
  const int32_t* len;
  void* h;
  float* h_last;
  float* states;
  const void* dh;
  const float* dh_last;
  void* dgate;
  void* dx;
  float* dh0;
  WsHeader* hdr;
  int tiles;    // channel tiles per sequence
  int cluster;  // CTAs per cluster
  int wide;     // rows lie on 16-byte boundaries
  int jobs;     // sequences x tiles (x segments)
  int nseg;     // segments per sequence, where a warp has one of its own
  int seg;      // steps per segment, a multiple of kChunk
  uint64_t polls;  // of a join's wait, until it gives up
  float2* maps;    // [B][nseg][D] a segment's map
  float2* groups;  // [B][nseg / kSoloWarps][D] the map of a CTA's segments
  float* first;    // [B][D] h0 (or dh_last), which the last segment may write over
};

// Where a job lies: a sequence, a tile of channels and a segment of the steps
// (all of them where nothing is split).  `pos` numbers the segments in the order
// of the recurrence, which the gradient runs backwards.
struct Place {
  int b, ct, pos, t0, t1;
  SPEC_DEV int ch0() const { return t0 / kChunk; }
  SPEC_DEV int ch1() const { return t1 > t0 ? (t1 + kChunk - 1) / kChunk : ch0(); }
};
SPEC_DEV Place place_of(const ScanArgs& a, int job, int width, bool grad) {
  Place p;
  p.pos = job % a.nseg;
  job /= a.nseg;
  p.b = job / a.tiles;
  p.ct = (job % a.tiles) * width;
  const int64_t t0 = (int64_t)(grad ? a.nseg - 1 - p.pos : p.pos) * a.seg;
  p.t0 = (int)min(t0, (int64_t)a.p.T);
  p.t1 = (int)min(t0 + a.seg, (int64_t)a.p.T);
  return p;
}

// One piece of one input in shared memory, written by 16-byte asynchronous
// copies where rows allow (zero-filled behind the end), else by plain loads.
template <typename T, int V>
struct alignas(16) Piece {
  RawOf<T, V> at[kChunk][32];
};

// Steps t .. t + kChunk - 1 of the lane's tile; `left` of them exist.
template <typename T, int V>
SPEC_DEV void fetch(Piece<T, V>& dst, const T* src, int64_t stride, int left, int channels,
                    bool wide) {
  const int lane = threadIdx.x & 31;
  if (wide) {
    constexpr int kEach = 16 / sizeof(T);           // channels per copy
    constexpr int kPer = 32 * V / kEach;            // copies per step
    constexpr int kSteps = 32 / kPer;               // steps per instruction
    const int c = (lane % kPer) * kEach, k0 = lane / kPer;
#pragma unroll
    for (int k = 0; k < kChunk; k += kSteps) {
      const bool in = k + k0 < left && c < channels;
      const T* s = in ? src + (int64_t)(k + k0) * stride + c : src;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       smem_u32(&dst.at[k + k0][0]) + c * (uint32_t)sizeof(T)),
                   "l"(s), "r"(in ? 16 : 0)
                   : "memory");
    }
  } else {
    RawOf<T, V> r[kChunk];
#pragma unroll
    for (int k = 0; k < kChunk; ++k)
      r[k] = k < left && lane * V < channels
                 ? __ldg(reinterpret_cast<const RawOf<T, V>*>(src + k * stride + lane * V))
                 : RawOf<T, V>(0);
#pragma unroll
    for (int k = 0; k < kChunk; ++k) dst.at[k][lane] = r[k];
  }
}

// Joins the maps of a window's W pieces in each of `cluster` CTAs.  (a, c) is
// the calling warp's map; warps and ranks are numbered in the order of the
// recurrence.  carry holds the value before the window in every thread and
// becomes the one after it; `before` is the one before the calling warp's
// piece.  The slots alternate between windows, so a window needs one barrier of
// the CTA.  Between the CTAs of a cluster the maps travel as asynchronous
// stores that count their bytes on the receiver's mbarrier: a cluster barrier
// would also wait for the outputs' stores.  A slot is free again when it is
// written: its writer has received the window in between from the slot's owner,
// who sent that after every warp had read the slot.
template <int V, int W>
struct Joiner {
  float2 piece[2][W][32 * V];
  float2 cta[2][kMaxCluster][32 * V];
  uint64_t full[2];
  volatile int gave_up[2];  // by a window's parity: a wait of it ran out
};
template <int V>
struct Joiner<V, 1> {
  float2 part[kSoloWarps][32 * V];
};

constexpr uint64_t kJoinPolls = 1ull << 22;  // about 4 s
std::atomic<int64_t> g_join_polls{-1};       // set by a test; negative: kJoinPolls

template <int V, int W>
SPEC_DEV void join_init(Joiner<V, W>& sm, int cluster) {
  if constexpr (W > 1) {
    if (cluster == 1) return;
    if (threadIdx.x == 0) {
      mbar_init(&sm.full[0], 1);
      mbar_init(&sm.full[1], 1);
      sm.gave_up[0] = sm.gave_up[1] = 0;
      fence_mbar_init();
    }
    cg::this_cluster().sync();  // every CTA runs, its barriers ready, before another writes to it
  }
}

SPEC_DEV uint32_t at_rank(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
SPEC_DEV void send(uint32_t to, float2 v, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
          to),
      "f"(v.x), "f"(v.y), "r"(bar)
      : "memory");
}
SPEC_DEV bool cluster_wait(uint64_t* bar, uint32_t parity, uint64_t polls) {
  for (uint64_t it = 0; it < polls; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000u)
        : "memory");
    if (ok) return true;
  }
  return false;
}

// The end of a CTA in which a wait ran out: others may still send to its shared
// memory, so it stays until their threads have ended or wait here as well (which
// they do, as their own waits are bounded) and what they sent has arrived.
template <int V, int W>
SPEC_DEV void join_end(Joiner<V, W>& sm, int cluster) {
  if constexpr (W > 1) {
    if (cluster == 1 || !(sm.gave_up[0] | sm.gave_up[1])) return;
    cp_async_wait<0>();
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    __nanosleep(1000000);
  }
}

// Returns false where the CTA has to leave, all of its threads alike: a wait of one
// of them ran out in the window before.  It sends and arrives no more then, since
// its barriers' phases are no longer the others', who give up in turn.  (The flag
// in shared memory costs the gradient of 8 x 8192 x 1024 4 % against no way out; as
// the window barrier's own reduction 5 %, kept by each thread 7 %.)
template <int V, int W>
SPEC_DEV bool join(Joiner<V, W>& sm, int win, int warp, int rank, int cluster, Vec<V> a, Vec<V> c,
                   Vec<V>& carry, Vec<V>& before, uint64_t polls, WsHeader* hdr) {
  const int par = win & 1;
  if constexpr (W == 1) {
    before = carry;
    carry = fma(a, carry, c);
  } else {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int v = 0; v < V; ++v)
      sm.piece[par][warp][v * 32 + lane] = make_float2(a.get(v), c.get(v));
    __syncthreads();
    if (cluster > 1 && sm.gave_up[par ^ 1]) return false;
    float out_b[V], out_c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float ta = 1.f, tc = 0.f, pa = 1.f, pc = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (w == warp) {
          pa = ta;
          pc = tc;
        }
        const float2 m = sm.piece[par][w][v * 32 + lane];
        ta *= m.x;
        tc = fmaf(m.x, tc, m.y);
      }
      ta = above_zero(ta);
      pa = above_zero(pa);
      if (cluster > 1) {
        if (warp < cluster)  // the warps hand the CTA's map to one CTA each
          send(at_rank(smem_u32(&sm.cta[par][rank][v * 32 + lane]), warp), make_float2(ta, tc),
               at_rank(smem_u32(&sm.full[par]), warp));
        out_b[v] = pa;
        out_c[v] = pc;
      } else {
        out_b[v] = fmaf(pa, carry.get(v), pc);
        out_c[v] = fmaf(ta, carry.get(v), tc);
      }
    }
    if (cluster > 1) {
      if (threadIdx.x == 0)
        mbar_arrive_expect_tx(&sm.full[par], (uint32_t)(cluster * 32 * V * sizeof(float2)));
      if (!cluster_wait(&sm.full[par], (win >> 1) & 1, polls)) {
        sm.gave_up[par] = 1;
        report_error(hdr, SPEC_ERR_TIMEOUT, SITE_MBAR_FULL, rank, win);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float s = carry.get(v), mine = s;
        for (int r = 0; r < cluster; ++r) {
          if (r == rank) mine = s;
          const float2 m = sm.cta[par][r][v * 32 + lane];
          s = fmaf(m.x, s, m.y);
        }
        out_b[v] = fmaf(out_b[v], mine, out_c[v]);
        out_c[v] = s;
      }
    }
    if constexpr (V == 2) {
      before = Vec<2>::of(out_b[0], out_b[1]);
      carry = Vec<2>::of(out_c[0], out_c[1]);
    } else {
      before = {out_b[0]};
      carry = {out_c[0]};
    }
  }
  return true;
}

template <int V>
SPEC_DEV Vec<V> state_load(const float* p, bool on) {
  if constexpr (V == 2)
    return on ? Vec<2>::of(p[0], p[1]) : Vec<2>::all(0.f);
  else
    return {on ? p[0] : 0.f};
}
template <int V>
SPEC_DEV void state_store(float* p, Vec<V> x) {
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] = x.get(v);
}

// The value a segment of a split sequence starts from: the first one taken through
// the maps of the groups before the segment's own (a run of them per warp,
// joined in order) and of the segments before it in its group.  The CTA's warps
// hold the consecutive segments of one group.
template <int V>
SPEC_DEV Vec<V> segment_start(const ScanArgs& a, Joiner<V, 1>& sm, const Place& at, int c,
                              bool on) {
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, D = a.p.D;
  const int group = at.pos / kSoloWarps, per = (group + kSoloWarps - 1) / kSoloWarps;
  const int g0 = min(wid * per, group), g1 = min(g0 + per, group);
  const int64_t grow = (int64_t)at.b * (a.nseg / kSoloWarps) * D + c;
  const int64_t mrow = ((int64_t)at.b * a.nseg + group * kSoloWarps) * D + c;
  float s[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float2 own[kSoloWarps - 1];
#pragma unroll
    for (int w = 0; w < kSoloWarps - 1; ++w)
      own[w] = on && w < wid ? __ldcg(a.maps + mrow + (int64_t)w * D + v) : make_float2(1.f, 0.f);
    float ma = 1.f, mc = 0.f;
#pragma unroll 8
    for (int g = g0; g < g1; ++g) {
      const float2 m = on ? __ldcg(a.groups + grow + (int64_t)g * D + v) : make_float2(1.f, 0.f);
      ma *= m.x;
      mc = fmaf(m.x, mc, m.y);
    }
    sm.part[wid][v * 32 + lane] = make_float2(above_zero(ma), mc);
    __syncthreads();
    s[v] = on ? __ldcg(a.first + (int64_t)at.b * D + c + v) : 0.f;
#pragma unroll
    for (int w = 0; w < kSoloWarps; ++w) {
      const float2 m = sm.part[w][v * 32 + lane];
      s[v] = fmaf(m.x, s[v], m.y);
    }
#pragma unroll
    for (int w = 0; w < kSoloWarps - 1; ++w) s[v] = fmaf(own[w].x, s[v], own[w].y);
  }
  if constexpr (V == 2)
    return Vec<2>::of(s[0], s[1]);
  else
    return {s[0]};
}

// Forward.  W > 1: a cluster per job (a sequence's tile of 32 V channels) walks
// the steps in windows of cluster * W pieces.  W = 1: a warp per job, a window is
// one piece and nothing is joined.  Two windows' inputs are on their way while
// one is computed (one instead of two: 256 x 256 x 1024 bf16 90 us, two 78, three
// 78).
template <typename T, int V, int W>
struct ScanShared {
  Joiner<V, W> joiner;
  Piece<T, V> gate[W == 1 ? kSoloWarps : W][kStages], x[W == 1 ? kSoloWarps : W][kStages];
};

template <typename T, int V, int W>
__global__ void __launch_bounds__(32 * (W == 1 ? kSoloWarps : W), 2)
    k_scan(ScanArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  ScanShared<T, V, W>& sm = *reinterpret_cast<ScanShared<T, V, W>*>(smem_raw);
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = W == 1 ? 1 : a.cluster, rank = blockIdx.x % C, warp = W == 1 ? 0 : wid;
  const int job = W == 1 ? blockIdx.x * kSoloWarps + wid : blockIdx.x / C;
  if (job >= a.jobs) return;  // whole warps, only where no barrier follows (W = 1, unsplit)
  const Place at = place_of(a, job, 32 * V, false);
  const int b = at.b, ct = at.ct, c = ct + lane * V;
  const int D = a.p.D, Tn = a.p.T;
  const bool on = c < D;  // pairs are only taken where D is even
  const int n = len_of(a.len, b, Tn, a.hdr,
                       ct == 0 && at.pos == 0 && rank == 0 && warp == 0 && lane == 0);
  const int64_t row0 = (int64_t)b * Tn;
  const T* gp = (const T*)a.gate + row0 * a.p.gate_stride + ct;
  const T* xp = (const T*)a.x + row0 * a.p.x_stride + ct;
  T* hp = (T*)a.h + row0 * a.p.h_stride + c;
  const int nch = (Tn + kChunk - 1) / kChunk;
  Vec<V> carry = state_load<V>(a.h0 + (int64_t)b * D + c, a.h0 && on);

  const int window = C * W * kChunk;
  int t0 = at.t0 + (rank * W + warp) * kChunk;
  auto request = [&](int t, int stage) {
    if (t < min(n, at.t1)) {
      fetch(sm.gate[wid][stage], gp + (int64_t)t * a.p.gate_stride, a.p.gate_stride, n - t, D - ct, a.wide);
      fetch(sm.x[wid][stage], xp + (int64_t)t * a.p.x_stride, a.p.x_stride, n - t, D - ct, a.wide);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int q = 0; q < kStages; ++q) request(t0 + q * window, q);
  join_init<V, W>(sm.joiner, C);
  if constexpr (W == 1) {
    if (a.nseg > 1) {
      grid_dependency_wait();  // the maps; the inputs above do not depend on them
      carry = segment_start<V>(a, sm.joiner, at, c, on);
    }
  }
  const int nwin = (at.t1 - at.t0 + window - 1) / window;
  for (int win = 0, stage = 0; win < nwin; ++win, t0 += window) {
    Vec<V> f[kChunk], z[kChunk], ma = Vec<V>::all(1.f), mc = Vec<V>::all(0.f);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const int left = n - t0;  // steps of the piece that belong to the sequence
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      gate_of<T, V>(sm.gate[wid][stage].at[k][lane], f[k], z[k]);
      z[k] = z[k] * raw_value<T, V>(sm.x[wid][stage].at[k][lane]);
    }
    if (left < kChunk) {  // the others leave the state as it is
#pragma unroll
      for (int k = 0; k < kChunk; ++k)
        if (k >= left) {
          f[k] = Vec<V>::all(1.f);
          z[k] = Vec<V>::all(0.f);
        }
    }
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      ma = ma * f[k];
      mc = fma(f[k], mc, z[k]);
    }
    ma = ma.map(above_zero);
    __syncwarp();
    request(t0 + kStages * window, stage);
    stage ^= 1;
    Vec<V> s;
    if (!join<V, W>(sm.joiner, win, warp, rank, C, ma, mc, carry, s, a.polls, a.hdr)) break;
    if (on && a.states && t0 < Tn)
      state_store<V>(a.states + ((int64_t)b * nch + t0 / kChunk) * D + c, s);
    if (on && a.h && left > 0) {
      T* h = hp + (int64_t)t0 * a.p.h_stride;
      const int hs = (int)a.p.h_stride;
      if (left >= kChunk) {
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
          s = fma(f[k], s, z[k]);
          raw_store<T, V>(h + (int64_t)k * hs, s);
        }
      } else {
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
          s = fma(f[k], s, z[k]);
          if (k < left) raw_store<T, V>(h + (int64_t)k * hs, s);
        }
      }
    }
    __syncwarp();
  }
  if (a.h_last && at.pos == a.nseg - 1 && rank == 0 && warp == 0 && on)
    state_store<V>(a.h_last + (int64_t)b * D + c, carry);
  join_end<V, W>(sm.joiner, C);
}

// Gradient.  The state before each piece comes from `states`, so its h are run
// forward again inside the warp; what is joined, last piece first, are the maps
// of the reversed recurrence carry -> f (dh + carry).
template <typename T, int V, int W>
struct GradShared {
  Joiner<V, W> joiner;
  Piece<T, V> gate[W == 1 ? kSoloWarps : W], x[W == 1 ? kSoloWarps : W];
  Piece<T, V> dh[2][W == 1 ? kSoloWarps : W];  // read again after the join
};

template <typename T, int V, int W>
__global__ void __launch_bounds__(32 * (W == 1 ? kSoloWarps : W), 2)
    k_scan_grad(ScanArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  GradShared<T, V, W>& sm = *reinterpret_cast<GradShared<T, V, W>*>(smem_raw);
  // pieces are numbered from the end: piece 0 of window 0 holds the last steps
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = W == 1 ? 1 : a.cluster, rank = blockIdx.x % C, warp = W == 1 ? 0 : wid;
  const int job = W == 1 ? blockIdx.x * kSoloWarps + wid : blockIdx.x / C;
  if (job >= a.jobs) return;  // whole warps, only where no barrier follows (W = 1, unsplit)
  const Place at = place_of(a, job, 32 * V, true);
  const int b = at.b, ct = at.ct, c = ct + lane * V;
  const int D = a.p.D, Tn = a.p.T;
  const bool on = c < D;
  const int n = len_of(a.len, b, Tn, a.hdr,
                       ct == 0 && at.pos == 0 && rank == 0 && warp == 0 && lane == 0);
  const int64_t row0 = (int64_t)b * Tn;
  const T* gp = (const T*)a.gate + row0 * a.p.gate_stride + ct;
  const T* xp = (const T*)a.x + row0 * a.p.x_stride + ct;
  const T* dp = (const T*)a.dh + row0 * a.p.h_stride + ct;
  T* dgp = (T*)a.dgate + row0 * a.p.gate_stride + c;
  T* dxp = (T*)a.dx + row0 * a.p.x_stride + c;
  const int nch = (Tn + kChunk - 1) / kChunk;
  Vec<V> carry = state_load<V>(a.dh_last + (int64_t)b * D + c, a.dh_last && on);

  const int window = C * W;  // in pieces
  const int ch0 = at.ch0(), ch1 = at.ch1();
  int ch = ch1 - 1 - (rank * W + warp);
  Vec<V> s0;
  auto request = [&](int q, int par) {
    const int t = q * kChunk;
    if (q >= ch0 && t < n) {
      fetch(sm.gate[wid], gp + (int64_t)t * a.p.gate_stride, a.p.gate_stride, n - t, D - ct, a.wide);
      fetch(sm.x[wid], xp + (int64_t)t * a.p.x_stride, a.p.x_stride, n - t, D - ct, a.wide);
      fetch(sm.dh[par][wid], dp + (int64_t)t * a.p.h_stride, a.p.h_stride, n - t, D - ct, a.wide);
    }
    cp_async_commit();
    s0 = state_load<V>(a.states + ((int64_t)b * nch + q) * D + c, on && q >= ch0);
  };
  request(ch, 0);
  join_init<V, W>(sm.joiner, C);
  if constexpr (W == 1) {
    if (a.nseg > 1) {
      grid_dependency_wait();  // the maps; the inputs above do not depend on them
      carry = segment_start<V>(a, sm.joiner, at, c, on);
    }
  }
  const int nwin = (ch1 - ch0 + window - 1) / window;
  for (int win = 0; win < nwin; ++win, ch -= window) {
    const int t0 = ch * kChunk, left = ch < ch0 ? 0 : n - t0, par = win & 1;
    Vec<V> f[kChunk], i[kChunk], w[kChunk], ma = Vec<V>::all(1.f), mc = Vec<V>::all(0.f);
    cp_async_wait<0>();
    __syncwarp();
    Vec<V> s = s0;
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      gate_of<T, V>(sm.gate[wid].at[k][lane], f[k], i[k]);
      const Vec<V> x = raw_value<T, V>(sm.x[wid].at[k][lane]);
      w[k] = fma(x, Vec<V>::all(-1.f), s) * (f[k] * i[k]);
      s = fma(f[k], s, i[k] * x);
    }
    if (left < kChunk) {
#pragma unroll
      for (int k = 0; k < kChunk; ++k)
        if (k >= left) {  // not a step of the sequence: the carry passes, no gradient
          f[k] = Vec<V>::all(1.f);
          i[k] = w[k] = Vec<V>::all(0.f);
          sm.dh[par][wid].at[k][lane] = RawOf<T, V>(0);
        }
    }
#pragma unroll
    for (int k = kChunk - 1; k >= 0; --k) {
      ma = ma * f[k];
      mc = f[k] * (mc + raw_value<T, V>(sm.dh[par][wid].at[k][lane]));
    }
    ma = ma.map(above_zero);
    __syncwarp();
    request(ch - window, par ^ 1);
    if (!join<V, W>(sm.joiner, win, warp, rank, C, ma, mc, carry, s, a.polls, a.hdr)) break;
    if (on && ch >= ch0) {
      T* dg = dgp + (int64_t)t0 * a.p.gate_stride;
      T* dx = dxp + (int64_t)t0 * a.p.x_stride;
      const int gs = (int)a.p.gate_stride, xs = (int)a.p.x_stride;
      if (left >= kChunk) {
#pragma unroll
        for (int k = kChunk - 1; k >= 0; --k) {
          const Vec<V> delta = s + raw_value<T, V>(sm.dh[par][wid].at[k][lane]);
          raw_store<T, V>(dg + (int64_t)k * gs, delta * w[k]);
          raw_store<T, V>(dx + (int64_t)k * xs, delta * i[k]);
          s = delta * f[k];
        }
      } else {
        const int rows = min(kChunk, Tn - t0);
#pragma unroll
        for (int k = kChunk - 1; k >= 0; --k) {
          const Vec<V> delta = s + raw_value<T, V>(sm.dh[par][wid].at[k][lane]);
          const Vec<V> zero = Vec<V>::all(0.f);
          if (k < rows) {
            raw_store<T, V>(dg + (int64_t)k * gs, k < left ? delta * w[k] : zero);
            raw_store<T, V>(dx + (int64_t)k * xs, k < left ? delta * i[k] : zero);
          }
          s = delta * f[k];
        }
      }
    }
    __syncwarp();
  }
  if (a.dh0 && at.pos == a.nseg - 1 && rank == 0 && warp == 0 && on)
    state_store<V>(a.dh0 + (int64_t)b * D + c, carry);
  join_end<V, W>(sm.joiner, C);
}

// ----------------------------------------------------------------------------
// Long sequences of few channels: even a cluster per job leaves most of the GPU
// idle, so the steps are split into segments, a warp each.  A first pass reduces
// every segment, and every CTA's group of them, to its map; the kernels above
// then run with a warp per segment, which they start from the joined maps of
// what lies before.  The inputs of the recurrence are read twice, the second
// time mostly from L2.
// ----------------------------------------------------------------------------
template <typename T, int V>
struct MapShared {
  Piece<T, V> gate[kSoloWarps][2], other[kSoloWarps][2];
  float2 part[kSoloWarps][32 * V];
};

template <typename T, int V, bool kGrad>
__global__ void __launch_bounds__(32 * kSoloWarps, 2) k_scan_maps(ScanArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  MapShared<T, V>& sm = *reinterpret_cast<MapShared<T, V>*>(smem_raw);
  grid_dependency_release();
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Place at = place_of(a, blockIdx.x * kSoloWarps + wid, 32 * V, kGrad);
  const int b = at.b, ct = at.ct, c = ct + lane * V, D = a.p.D;
  const int n = len_of(a.len, b, a.p.T, a.hdr, false);
  const int64_t row0 = (int64_t)b * a.p.T;
  const int64_t stride = kGrad ? a.p.h_stride : a.p.x_stride;
  const T* gp = (const T*)a.gate + row0 * a.p.gate_stride + ct;
  const T* op = (const T*)(kGrad ? a.dh : a.x) + row0 * stride + ct;
  const int ch0 = at.ch0(), ch1 = at.ch1();
  // the pieces in the order of the recurrence
  auto piece = [&](int q) { return kGrad ? ch1 - 1 - q : ch0 + q; };
  auto request = [&](int q) {
    const int t = piece(q) * kChunk;
    if (q < ch1 - ch0 && t < n) {
      fetch(sm.gate[wid][q & 1], gp + (int64_t)t * a.p.gate_stride, a.p.gate_stride, n - t, D - ct, a.wide);
      fetch(sm.other[wid][q & 1], op + (int64_t)t * stride, stride, n - t, D - ct, a.wide);
    }
    cp_async_commit();
  };
  Vec<V> ma = Vec<V>::all(1.f), mc = Vec<V>::all(0.f);
  request(0);
  for (int q = 0; q < ch1 - ch0; ++q) {
    request(q + 1);
    cp_async_wait<1>();
    __syncwarp();
    const int left = n - piece(q) * kChunk;
    auto step = [&](int k) {
      Vec<V> f, i;
      gate_of<T, V>(sm.gate[wid][q & 1].at[k][lane], f, i);
      const Vec<V> o = raw_value<T, V>(sm.other[wid][q & 1].at[k][lane]);
      ma = ma * f;
      if constexpr (kGrad)
        mc = f * (mc + o);
      else
        mc = fma(f, mc, i * o);
    };
    if (left >= kChunk) {
#pragma unroll
      for (int k = 0; k < kChunk; ++k) step(kGrad ? kChunk - 1 - k : k);
    } else {
      for (int k = 0; k < left; ++k) step(kGrad ? left - 1 - k : k);
    }
    __syncwarp();
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float2 m = make_float2(above_zero(ma.get(v)), mc.get(v));
    sm.part[wid][v * 32 + lane] = m;
    if (at.pos == 0 && c < D) {
      const float* first = kGrad ? a.dh_last : a.h0;
      const int64_t e = (int64_t)b * D + c + v;
      a.first[e] = first ? first[e] : 0.f;
    }
    if (c < D) a.maps[((int64_t)b * a.nseg + at.pos) * D + c + v] = m;
  }
  __syncthreads();
  if (wid < V && ct + lane * V + wid < D) {
    float ta = 1.f, tc = 0.f;
#pragma unroll
    for (int w = 0; w < kSoloWarps; ++w) {
      const float2 m = sm.part[w][wid * 32 + lane];
      ta *= m.x;
      tc = fmaf(m.x, tc, m.y);
    }
    a.groups[((int64_t)b * (a.nseg / kSoloWarps) + at.pos / kSoloWarps) * D + c + wid] =
        make_float2(above_zero(ta), tc);
  }
}

// Rows of all inputs on 16-byte boundaries: copies of 16 bytes.
template <typename T>
bool wide_ok(const ScanArgs& a) {
  const uintptr_t all = (uintptr_t)a.gate | (uintptr_t)a.x | (uintptr_t)a.dh;
  const int64_t st = a.p.D | a.p.gate_stride | a.p.x_stride | (a.dh ? a.p.h_stride : 0);
  return (st * (int64_t)sizeof(T)) % 16 == 0 && (all & 15) == 0;
}

// Pairs of bf16: even width and strides, 4-byte aligned rows.
bool pairs_ok(const ScanArgs& a) {
  const uintptr_t all = (uintptr_t)a.gate | (uintptr_t)a.x | (uintptr_t)a.h | (uintptr_t)a.dh |
                        (uintptr_t)a.dgate | (uintptr_t)a.dx;
  return ((a.p.D | a.p.gate_stride | a.p.x_stride | a.p.h_stride) & 1) == 0 && (all & 3) == 0;
}

int64_t jobs_of(const spec_scan_params& p, int V) {
  return (int64_t)p.B * ((p.D + 32 * V - 1) / (32 * V));
}

// Steps per segment where the steps are split, 0 where they are not.  Split
// when clusters of every job would still leave SMs without a CTA and the steps
// fill five of their windows (one sequence of 256 bf16 channels, forward and
// gradient: split 17 and 23 us at 4096 steps, 19 and 24 at 8192; in clusters 15
// and 21, 25 and 36); segments then give every SM about 16 warps.
int segment_steps(const spec_scan_params& p, int64_t jobs, int num_sms) {
  if (jobs * kMaxCluster >= num_sms || p.T < kSplitSteps) return 0;
  const int64_t segs = (16 * (int64_t)num_sms + jobs - 1) / jobs;
  const int64_t steps = (p.T + segs - 1) / segs;
  return (int)std::max<int64_t>((steps + kChunk - 1) / kChunk * kChunk, kMinSegment);
}

// Dynamic shared memory beyond the default needs leave.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int V, int W>
cudaError_t launch(ScanArgs& a, bool grad, int num_sms, cudaStream_t st) {
  const int64_t jobs = jobs_of(a.p, V) * a.nseg;
  a.tiles = (a.p.D + 32 * V - 1) / (32 * V);
  a.jobs = (int)jobs;
  // Split a sequence over a cluster while there are not two CTAs for every SM
  // and its steps fill more than one window.
  int C = 1;
  if (W > 1)
    while (C < kMaxCluster && jobs * C < 2 * num_sms && (int64_t)C * W * kChunk < a.p.T) C *= 2;
  a.cluster = C;
  const int64_t grid = W == 1 ? (jobs + kSoloWarps - 1) / kSoloWarps : jobs * C;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  void (*kernel)(ScanArgs) = grad ? k_scan_grad<T, V, W> : k_scan<T, V, W>;
  const size_t smem = grad ? sizeof(GradShared<T, V, W>) : sizeof(ScanShared<T, V, W>);
  const cudaError_t e = allow_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(32 * (W == 1 ? kSoloWarps : W));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.nseg > 1 ? 2 : 1;  // behind its maps' launch it may start early
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Segments per sequence, whole groups of them (the last ones may be empty).
int segments(const spec_scan_params& p, int seg) {
  const int n = (p.T + seg - 1) / seg;
  return (n + kSoloWarps - 1) / kSoloWarps * kSoloWarps;
}

template <typename T, int V, int W>
cudaError_t by_shape(ScanArgs& a, bool grad, int num_sms, uint8_t* body, cudaStream_t st,
                     int* launches) {
  a.nseg = 1;
  a.seg = a.p.T;
  *launches = 1;
  // A warp per job where the sequence is one piece, or where jobs fill the GPU:
  // forward from six an SM (bf16, 64 x 512 x 2048: 76 us, joined 86; at 4.3 an SM
  // 82 against 61).  The gradient, whose warps hold too much for two pieces on
  // their way, only where a CTA's window would stay half empty (1024 x 64 x 512:
  // 90 us, joined 123; 512 x 128 x 1024: 169 against 158).
  const int64_t jobs = jobs_of(a.p, V);
  if (a.p.T <= kChunk || (grad ? a.p.T <= W * kChunk / 2 && jobs >= 16 * (int64_t)num_sms
                               : jobs >= 6 * (int64_t)num_sms))
    return launch<T, V, 1>(a, grad, num_sms, st);
  a.seg = segment_steps(a.p, jobs_of(a.p, V), num_sms);
  if (a.seg == 0) {
    a.seg = a.p.T;
    return launch<T, V, W>(a, grad, num_sms, st);
  }
  a.nseg = segments(a.p, a.seg);
  a.tiles = (a.p.D + 32 * V - 1) / (32 * V);
  a.maps = reinterpret_cast<float2*>(body);
  a.groups = a.maps + (size_t)a.p.B * a.nseg * a.p.D;
  a.first = reinterpret_cast<float*>(a.groups + (size_t)a.p.B * (a.nseg / kSoloWarps) * a.p.D);
  const int grid = (int)(jobs_of(a.p, V) * (a.nseg / kSoloWarps));
  void (*maps)(ScanArgs) = grad ? k_scan_maps<T, V, true> : k_scan_maps<T, V, false>;
  cudaError_t e = allow_smem(maps, sizeof(MapShared<T, V>));
  if (e != cudaSuccess) return e;
  e = launch_kernel(maps, grid, 32 * kSoloWarps, sizeof(MapShared<T, V>), st, a);
  if (e != cudaSuccess) return e;
  *launches = 2;
  return launch<T, V, 1>(a, grad, num_sms, st);
}

template <typename T>
cudaError_t dispatch(ScanArgs& a, bool grad, int num_sms, uint8_t* body, cudaStream_t st,
                     int* launches) {
  a.wide = wide_ok<T>(a);
  const int64_t polls = g_join_polls.load(std::memory_order_relaxed);
  a.polls = polls < 0 ? kJoinPolls : (uint64_t)polls;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    if (pairs_ok(a)) return by_shape<T, 2, 8>(a, grad, num_sms, body, st, launches);
  }
  return by_shape<T, 1, 8>(a, grad, num_sms, body, st, launches);
}

}  // namespace

void set_scan_polls(int64_t polls) { g_join_polls.store(polls); }

size_t scan_ws_bytes(const spec_scan_params& p, int num_sms) {
  size_t need = 0;
  for (int V = 1; V <= (p.dtype == SPEC_BF16 ? 2 : 1); ++V) {  // whichever alignment allows
    const int seg = segment_steps(p, jobs_of(p, V), num_sms);
    if (seg == 0) continue;
    const size_t nseg = segments(p, seg);
    need = std::max(need, (sizeof(float2) * (nseg + nseg / kSoloWarps) + sizeof(float)) *
                              (size_t)p.B * p.D);
  }
  return need;
}

template <typename T>
cudaError_t launch_scan(const spec_scan_params& p, const T* gate, const T* x, const float* h0,
                        const int32_t* len, T* h, float* h_last, float* states, uint8_t* body,
                        WsHeader* hdr, int num_sms, cudaStream_t st, int* launches) {
  ScanArgs a = {};
  a.p = p;
  a.gate = gate;
  a.x = x;
  a.h0 = h0;
  a.len = len;
  a.h = h;
  a.h_last = h_last;
  a.states = states;
  a.hdr = hdr;
  return dispatch<T>(a, false, num_sms, body, st, launches);
}

template <typename T>
cudaError_t launch_scan_grad(const spec_scan_params& p, const T* gate, const T* x, const float* h0,
                             const int32_t* len, const float* states, const T* dh,
                             const float* dh_last, T* dgate, T* dx, float* dh0, uint8_t* body,
                             WsHeader* hdr, int num_sms, cudaStream_t st, int* launches) {
  ScanArgs a = {};
  a.p = p;
  a.gate = gate;
  a.x = x;
  a.h0 = h0;
  a.len = len;
  a.states = const_cast<float*>(states);
  a.dh = dh;
  a.dh_last = dh_last;
  a.dgate = dgate;
  a.dx = dx;
  a.dh0 = dh0;
  a.hdr = hdr;
  return dispatch<T>(a, true, num_sms, body, st, launches);
}

#define SPEC_INST(T)                                                                               \
  template cudaError_t launch_scan<T>(const spec_scan_params&, const T*, const T*, const float*,   \
                                      const int32_t*, T*, float*, float*, uint8_t*, WsHeader*, int, \
                                      cudaStream_t, int*);                                         \
  template cudaError_t launch_scan_grad<T>(const spec_scan_params&, const T*, const T*,            \
                                           const float*, const int32_t*, const float*, const T*,   \
                                           const float*, T*, T*, float*, uint8_t*, WsHeader*, int, \
                                           cudaStream_t, int*);
SPEC_INST(float)
SPEC_INST(__nv_bfloat16)
#undef SPEC_INST

}  // namespace specdec
