// Scaled lookup of table rows by token, and its gradient.
//
// The gradient of a table row is the sum of the rows of all positions that name
// it.  Few positions (k_grad_direct): a CTA per position looks through all of
// them, which needs no order.  Many: the positions are sorted by token
// (k_grad_sort, stable, so positions ascend within a token), equal pieces of the
// sorted list are summed however the tokens are spread (k_grad_sums), and runs
// that cross pieces are joined in order (k_grad_join).  Every sum is taken in
// fp32 in an order that only the tokens fix.
#include <algorithm>
#include <type_traits>

#include "head_ops.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 8;  // columns per lane and block of columns

// The columns of one lane of `lanes` that share a block of kCols * lanes: two
// vectors of four (kWide: an instruction of the group covers neighbouring
// vectors, whole sectors of memory for either type), or eight single ones.
template <bool kWide>
struct Columns {
  static constexpr int kEach = kWide ? 4 : 1;
  int at, step, left;  // first column, distance of its vectors, columns from it to the row's end
  SPEC_DEV Columns(int block, int lane, int lanes, int D) {
    at = block * kCols * lanes + lane * kEach;
    step = kEach * lanes;
    left = D - at;
  }
  SPEC_DEV bool any() const { return left > 0; }
};

// One lane's columns of a row as they lie in memory.
template <bool kWide, typename T>
struct Raw;
template <>
struct Raw<true, __nv_bfloat16> {
  uint2 v[2];
  SPEC_DEV void load(const __nv_bfloat16* p, const Columns<true>& c) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      v[k] = k * c.step < c.left ? __ldg(reinterpret_cast<const uint2*>(p + k * c.step)) : make_uint2(0, 0);
  }
  SPEC_DEV void clear() { v[0] = v[1] = make_uint2(0, 0); }
  SPEC_DEV float get(int k) const {
    const uint32_t w = (k & 2) ? v[k >> 2].y : v[k >> 2].x;
    return __uint_as_float((k & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
};
template <>
struct Raw<true, float> {
  float4 v[2];
  SPEC_DEV void load(const float* p, const Columns<true>& c) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      v[k] = k * c.step < c.left ? __ldg(reinterpret_cast<const float4*>(p + k * c.step))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  SPEC_DEV void clear() { v[0] = v[1] = make_float4(0.f, 0.f, 0.f, 0.f); }
  SPEC_DEV float get(int k) const {
    const float4& q = v[k >> 2];
    return (k & 3) == 0 ? q.x : (k & 3) == 1 ? q.y : (k & 3) == 2 ? q.z : q.w;
  }
};
template <typename T>
struct Raw<false, T> {
  using Bits = std::conditional_t<sizeof(T) == 4, uint32_t, uint16_t>;
  Bits v[kCols];  // converted when used, so that loads do not wait for one another
  SPEC_DEV void load(const T* p, const Columns<false>& c) {
#pragma unroll
    for (int k = 0; k < kCols; ++k)
      v[k] = k * c.step < c.left ? __ldg(reinterpret_cast<const Bits*>(p) + k * c.step) : Bits(0);
  }
  SPEC_DEV void clear() {
#pragma unroll
    for (int k = 0; k < kCols; ++k) v[k] = 0;
  }
  SPEC_DEV float get(int k) const {
    return __uint_as_float(sizeof(T) == 4 ? (uint32_t)v[k] : (uint32_t)v[k] << 16);
  }
};

template <bool kWide, typename T>
SPEC_DEV void store8(T* p, const Columns<kWide>& c, const float* x) {
  if constexpr (!kWide) {
#pragma unroll
    for (int k = 0; k < kCols; ++k)
      if (k * c.step < c.left) store_f(p, k * c.step, x[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k * c.step >= c.left) continue;
      const float* q = x + 4 * k;
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p + k * c.step) = make_float4(q[0], q[1], q[2], q[3]);
      } else {
        uint2 w;
        reinterpret_cast<__nv_bfloat162*>(&w)[0] = __floats2bfloat162_rn(q[0], q[1]);
        reinterpret_cast<__nv_bfloat162*>(&w)[1] = __floats2bfloat162_rn(q[2], q[3]);
        *reinterpret_cast<uint2*>(p + k * c.step) = w;
      }
    }
  }
}

// rows[i] = scale * table[ids[i]].  `lanes` lanes take one row of four blocks of
// columns at a time, or kRows rows of 4 / kRows blocks, so that four blocks' loads
// are in flight together (single columns, which cost eight loads a block, take one
// block of each row).  Bytes bound it: the named rows of the table in, the rows out.
// Repeated rows come from the caches (65536 rows of 1024 fp32 to bf16 by Zipf's
// tokens: 39 % of what is read from L1, 42 % from L2, the rest from memory), and the
// traffic of L2, 163 MB in and 134 MB out at 8 TB/s, is then the limit: 40 us, 4.4
// TB/s of the distinct bytes.  One row at a time instead: rows of 256 bf16 in 30 us
// against 17, of 512 in 33 against 23.
template <bool kWide, int kRows, typename TT, typename TR>
__global__ void __launch_bounds__(kThreads, kWide ? 1 : 4)
    k_embed(spec_embed_params p, const TT* __restrict__ table, const int32_t* __restrict__ ids,
            TR* __restrict__ rows, int shift, WsHeader* hdr) {
  constexpr int kAhead = kWide ? 4 : kRows, kBlocks = kAhead / kRows;
  const int lanes = 1 << shift, lane = threadIdx.x & (lanes - 1);
  const int64_t i0 = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> shift) * kRows;
  int id[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) id[r] = i0 + r < p.n ? __ldg(ids + i0 + r) : -1;
  bool in[kRows];
  const TT* src[kRows];
  TR* dst[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    in[r] = id[r] >= 0 && id[r] < p.V;
    src[r] = table + (int64_t)(in[r] ? id[r] : 0) * p.table_stride;
    dst[r] = rows + (i0 + r) * p.row_stride;
    if (!in[r] && id[r] != -1 && lane == 0)
      report_error(hdr, SPEC_ERR_TOKEN_RANGE, SITE_TOKEN_RANGE, (int)(i0 + r), id[r]);
  }
  const int blocks = (p.D + kCols * lanes - 1) / (kCols * lanes);
  for (int k0 = 0; k0 < blocks; k0 += kBlocks) {
    Raw<kWide, TT> x[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int r = q / kBlocks;
      const Columns<kWide> c(k0 + q % kBlocks, lane, lanes, p.D);  // none past the last block
      x[q].load(src[r] + c.at, c);
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int r = q / kBlocks;
      const Columns<kWide> c(k0 + q % kBlocks, lane, lanes, p.D);
      float y[kCols];
#pragma unroll
      for (int k = 0; k < kCols; ++k) y[k] = in[r] ? x[q].get(k) * p.scale : 0.f;
      if (c.any() && i0 + r < p.n) store8<kWide>(dst[r] + c.at, c, y);
    }
  }
}

// ----------------------------------------------------------------------------
// Gradient
// ----------------------------------------------------------------------------
// What goes into a table row: scale * sum, added to what is there or not.
template <bool kWide, typename TT>
SPEC_DEV void put_row(const spec_embed_params& p, TT* dtable, int64_t row, const Columns<kWide>& c,
                      float* acc) {
  if (!c.any()) return;
  TT* dst = dtable + row * p.table_stride + c.at;
#pragma unroll
  for (int k = 0; k < kCols; ++k) acc[k] *= p.scale;
  if (p.accumulate) {
    Raw<kWide, TT> old;
    old.load(dst, c);
#pragma unroll
    for (int k = 0; k < kCols; ++k) acc[k] += old.get(k);
  }
  store8<kWide>(dst, c, acc);
}

// Zero a run of table rows, but for those in a bitmap.
template <bool kWide, typename TT>
SPEC_DEV void zero_rows(const spec_embed_params& p, TT* dtable, int64_t v0, int64_t v1,
                        const uint32_t* skip) {
  const float zero[kCols] = {};
  const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
  for (int64_t v = v0 + threadIdx.x / 32; v < v1; v += warps) {
    const int k = (int)(v - v0);
    if (skip && (skip[k >> 5] >> (k & 31) & 1)) continue;
    for (int block = 0; block * kCols * 32 < p.D; ++block) {
      const Columns<kWide> c(block, lane, 32, p.D);
      if (c.any()) store8<kWide>(dtable + v * p.table_stride + c.at, c, zero);
    }
  }
}

// Most positions that are not sorted: every CTA looks through all of them, so
// the direct form's time grows with their square, while the sort's launches and
// barriers are there from the first on (V 32000, D 256: 1000 positions 14 us,
// sorted 27; 2048 18 and 33; 4096 29 and 34; 6000 44 and 33).
constexpr int kDirect = 4096;
constexpr int kZeroRows = 1024;   // most table rows a CTA zeroes beside them

constexpr int kDirectWarps = 16;
constexpr int kRun = kDirect / kDirectWarps;  // most positions a warp looks through
constexpr int kIds = 4;                       // of them per lane at a time

// CTAs 0 .. n - 1: the first position of a token sums the rows of all positions
// that name it; its warps list those of a run of positions each.  The CTAs after
// them zero the rows that no position names.
template <bool kWide, typename TT, typename TR>
__global__ void __launch_bounds__(32 * kDirectWarps, 2)
    k_grad_direct(spec_embed_params p, const int32_t* __restrict__ ids,
                  const TR* __restrict__ drows, TT* dtable, int zero_per, WsHeader* hdr) {
  constexpr int kAll = 32 * kDirectWarps;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = p.n;
  if ((int)blockIdx.x >= n) {
    __shared__ uint32_t named[kZeroRows / 32];
    const int64_t v0 = (int64_t)(blockIdx.x - n) * zero_per, v1 = min(v0 + zero_per, (int64_t)p.V);
    for (int k = tid; k < kZeroRows / 32; k += kAll) named[k] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kAll) {
      const int64_t k = __ldg(ids + j) - v0;
      if (k >= 0 && k < v1 - v0) atomicOr(&named[k >> 5], 1u << (k & 31));
    }
    __syncthreads();
    zero_rows<kWide>(p, dtable, v0, v1, named);
    return;
  }
  __shared__ float part[kDirectWarps][32 * kCols];
  __shared__ uint16_t list[kDirectWarps][kRun];
  const int i = blockIdx.x, id = __ldg(ids + i);
  if (id < 0 || id >= p.V) {
    if (id != -1 && tid == 0) report_error(hdr, SPEC_ERR_TOKEN_RANGE, SITE_TOKEN_RANGE, i, id);
    return;
  }
  // the warp's run of positions: those that name the token, in order
  const int run = (n + 32 * kDirectWarps - 1) / (32 * kDirectWarps) * 32;
  int count = 0;
  bool before = false;
  for (int k0 = 0; k0 < run; k0 += 32 * kIds) {
#pragma unroll
    for (int k = 0; k < kIds; ++k) {
      const int in = k0 + k * 32 + lane, j = warp * run + in;
      const bool same = in < run && j < n && __ldg(ids + j) == id;
      before |= same && j < i;
      const uint32_t m = __ballot_sync(0xffffffffu, same);
      if (same) list[warp][count + __popc(m & ((1u << lane) - 1))] = (uint16_t)j;
      count += __popc(m);
    }
  }
  if (__syncthreads_or(before)) return;
  const bool alone = !__syncthreads_or(count > (warp == i / run));
  if (alone) {  // the common case: one row
    for (int block = warp; block * kCols * 32 < p.D; block += kDirectWarps) {
      const Columns<kWide> c(block, lane, 32, p.D);
      Raw<kWide, TR> x;
      x.load(drows + (int64_t)i * p.row_stride + c.at, c);
      float acc[kCols];
#pragma unroll
      for (int k = 0; k < kCols; ++k) acc[k] = x.get(k);
      put_row<kWide>(p, dtable, id, c, acc);
    }
    return;
  }
  constexpr int kAhead = 8;
  for (int block = 0; block * kCols * 32 < p.D; ++block) {
    const Columns<kWide> c(block, lane, 32, p.D);
    float acc[kCols] = {};
    for (int k0 = 0; k0 < count; k0 += kAhead) {
      Raw<kWide, TR> x[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        x[q].load(drows + (int64_t)list[warp][min(k0 + q, count - 1)] * p.row_stride + c.at, c);
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (k0 + q >= count) break;
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] += x[q].get(k);
      }
    }
#pragma unroll
    for (int k = 0; k < kCols; ++k) part[warp][k * 32 + lane] = acc[k];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int w = 1; w < kDirectWarps; ++w)
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] += part[w][k * 32 + lane];
      put_row<kWide>(p, dtable, id, c, acc);
    }
    __syncthreads();
  }
}

// ---- Sort ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigits = 512;                       // 9 bits a pass
constexpr int kFewRounds = 2, kManyRounds = 4;     // 32 neighbouring positions of a warp each
static_assert(kDirect <= 65536, "positions of the list fit 16 bits");
static_assert(kDigits == kSortThreads, "one thread per digit");

struct SortArgs {
  spec_embed_params p;
  const int32_t* ids;
  int32_t* keys[2];   // tokens; V for positions that name none
  int32_t* pos[2];
  int32_t* hist;      // [CTA][digit]
  int ctas;
  int per;            // positions per CTA, whole tiles
  int passes, bits;   // bits per pass
  uint64_t spin;
  WsHeader* hdr;
};

struct SortShared {
  int32_t count[kDigits];
  int32_t base[kDigits];
  uint16_t warp[kSortWarps][kDigits];
  int32_t scan[kSortWarps];
};

// Exclusive prefix sums over the CTA's threads.
SPEC_DEV int exclusive_scan(int x, int32_t* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) warps[warp] = s;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += warps[w];
  return before + s - x;
}

// Stable sort by token, 9 bits a pass from the lowest: every CTA counts the
// digits of its run of positions, and after a barrier of the CTAs knows where
// its own of each digit go; tile by tile the positions are ranked by ballots and
// written there.  Latency bounds it (131072 positions, two passes: 20 to 26 us,
// 0.3 % of the memory's bandwidth), so a run of one tile (131072 positions) stays
// in registers, and the counts of all CTAs are requested at once.  Zeroing the
// table beside it in further CTAs made its barriers slower than it saved (47 us).
// Up to 65536 positions the tiles are half as long, on as many CTAs (9000: 2 us
// less; at 131072, where that takes 128 CTAs, 2 us more).
// Cooperative launch: the CTAs wait for one another.
template <int kRounds>
__global__ void __launch_bounds__(kSortThreads) k_grad_sort(SortArgs a) {
  constexpr int kTile = kRounds * kSortThreads;  // positions ranked together
  __shared__ SortShared sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  const int64_t n = a.p.n, i0 = min((int64_t)cta * a.per, n), i1 = min(i0 + a.per, n);
  grid_dependency_release();
  uint32_t barrier = 0;
  auto grid_sync = [&]() {
    __syncthreads();
    if (a.ctas == 1) return true;
    barrier += a.ctas;
    int ok = 1;
    if (tid == 0) {
      __threadfence();
      red_release_add_u32(&a.hdr->bar, 1u);
      ok = grid_wait_count(a.hdr, &a.hdr->bar, barrier, a.spin, SITE_GRID_BARRIER);
    }
    return __syncthreads_and(ok) != 0;
  };
  int32_t key[kRounds], pos[kRounds];
  auto load = [&](int pass, int64_t t0) {
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      const int64_t i = t0 + warp * (kTile / kSortWarps) + r * 32 + lane;
      key[r] = -1;
      if (i >= i1) continue;
      if (pass == 0) {
        const int id = __ldg(a.ids + i);
        key[r] = id >= 0 && id < a.p.V ? id : a.p.V;
        pos[r] = (int32_t)i;
        if (id < -1 || id >= a.p.V)
          report_error(a.hdr, SPEC_ERR_TOKEN_RANGE, SITE_TOKEN_RANGE, (int)i, id);
      } else {
        key[r] = __ldcg(a.keys[pass & 1] + i);
        pos[r] = __ldcg(a.pos[pass & 1] + i);
      }
    }
  };
  const bool one_tile = i1 - i0 <= kTile;
  bool ok = true;
  for (int pass = 0; pass < a.passes && ok; ++pass) {
    const int shift = pass * a.bits, mask = (1 << a.bits) - 1;
    sm.count[tid] = 0;
    __syncthreads();
    for (int64_t t0 = i0; t0 < i1; t0 += kTile) {
      load(pass, t0);
#pragma unroll
      for (int r = 0; r < kRounds; ++r)
        if (key[r] >= 0) atomicAdd(&sm.count[(key[r] >> shift) & mask], 1);
    }
    __syncthreads();
    a.hist[(int64_t)cta * kDigits + tid] = sm.count[tid];
    ok = grid_sync();
    if (!ok) break;
    // thread = digit: all positions of it, and those in the CTAs before this one
    int total = 0, before = 0;
    for (int q0 = 0; q0 < a.ctas; q0 += 32) {
      int h[32];
#pragma unroll
      for (int q = 0; q < 32; ++q)
        h[q] = q0 + q < a.ctas ? __ldcg(a.hist + (int64_t)(q0 + q) * kDigits + tid) : 0;
#pragma unroll
      for (int q = 0; q < 32; ++q) {
        before += q0 + q < cta ? h[q] : 0;
        total += h[q];
      }
    }
    sm.base[tid] = before + exclusive_scan(total, sm.scan);
    __syncthreads();
    int32_t* const to_key = a.keys[(pass + 1) & 1];
    int32_t* const to_pos = a.pos[(pass + 1) & 1];
    for (int64_t t0 = i0; t0 < i1; t0 += kTile) {
      for (int k = lane; k < kDigits; k += 32) sm.warp[warp][k] = 0;
      __syncwarp();
      if (!one_tile) load(pass, t0);
      int rank[kRounds];
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const int d = key[r] < 0 ? -1 : (key[r] >> shift) & mask;
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        const int lower = __popc(same & ((1u << lane) - 1));
        rank[r] = d < 0 ? 0 : sm.warp[warp][d] + lower;
        __syncwarp();
        if (d >= 0 && lower == 0) sm.warp[warp][d] += (uint16_t)__popc(same);
        __syncwarp();
      }
      __syncthreads();
      {  // thread = digit: counts of the warps become their offsets
        int s = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
          const int c = sm.warp[w][tid];
          sm.warp[w][tid] = (uint16_t)s;
          s += c;
        }
        sm.count[tid] = s;
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        if (key[r] < 0) continue;
        const int d = (key[r] >> shift) & mask;
        const int64_t to = (int64_t)sm.base[d] + sm.warp[warp][d] + rank[r];
        to_key[to] = key[r];
        to_pos[to] = pos[r];
      }
      __syncthreads();
      sm.base[tid] += sm.count[tid];
      __syncthreads();
    }
    if (pass + 1 < a.passes) ok = grid_sync();
  }
  if (a.ctas == 1) return;
  // All CTAs are counted, those that gave up in the upper half, and the last one
  // leaves the counters as the next launch needs them.  After a wait that ran out
  // the lists are in no order and may hold anything: then no place of them names
  // a token, so that the launches behind this one read no row and add nothing.
  bool gave_up = false;
  if (tid == 0) {
    if (!ok) report_error(a.hdr, SPEC_ERR_TIMEOUT, SITE_GRID_BARRIER, cta, (int)barrier);
    __threadfence();
    const uint32_t left = atomicAdd(&a.hdr->exit_count, ok ? 1u : 0x10001u);
    if ((left & 0xFFFFu) == (uint32_t)a.ctas - 1) {
      gave_up = !ok || left >> 16;
      if (gave_up) __threadfence();  // the list is written after what the others wrote
      a.hdr->bar = 0;
      a.hdr->abort = 0;
      a.hdr->exit_count = 0;
    }
  }
  if (__syncthreads_or(gave_up))
    for (int64_t i = tid; i < n; i += kSortThreads) a.keys[a.passes & 1][i] = a.p.V;
}

// ---- Sums of the sorted list -------------------------------------------------------------
struct SumArgs {
  spec_embed_params p;
  const int32_t* keys;
  const int32_t* pos;
  float* part;  // [piece][2][width]: the sum of the run that came in, of the one that goes on
  int piece;    // positions per piece
  int pieces, lanes, blocks;
  int width;    // columns, whole blocks
  int sum_ctas;  // the CTAs after them zero zero_per table rows each
  int zero_per;
};

// First place in the sorted list whose token is not below v; a whole warp asks,
// 32 places at a time.
SPEC_DEV int lower_bound(const int32_t* keys, int n, int64_t v) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // the answer is in [lo, hi]
  while (lo < hi) {
    const int64_t step = ((int64_t)hi - lo + 32) / 33;
    const int64_t at = lo + step * (lane + 1) - 1;
    const bool below = at < hi && __ldg(keys + at) < v;
    const int k = __popc(__ballot_sync(0xffffffffu, below));  // the list ascends: the first k
    const int64_t low = lo + step * k;
    if (k < 32) hi = (int)min((int64_t)hi, low + step - 1);
    lo = (int)min((int64_t)hi, low);
  }
  return lo;
}

// CTAs after the sums': zero a run of table rows, but for those in the list.
template <bool kWide, typename TT>
SPEC_DEV void zero_unnamed(const SumArgs& a, TT* dtable, int cta) {
  __shared__ uint32_t named[kZeroRows / 32];
  __shared__ int range[2];
  const int64_t v0 = (int64_t)cta * a.zero_per, v1 = min(v0 + a.zero_per, (int64_t)a.p.V);
  const int tid = threadIdx.x, warp = tid >> 5;
  for (int k = tid; k < kZeroRows / 32; k += kThreads) named[k] = 0;
  if (warp < 2) {
    const int at = lower_bound(a.keys, a.p.n, warp ? v1 : v0);
    if ((tid & 31) == 0) range[warp] = at;
  }
  __syncthreads();
  constexpr int kAhead = 16;  // a token named often fills many places
  for (int j = range[0] + tid; j < range[1]; j += kAhead * kThreads) {
    int key[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
      key[q] = __ldg(a.keys + min(j + q * kThreads, range[1] - 1));
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int k = (int)(key[q] - v0);
      if (q == 0 || key[q] != key[q - 1]) atomicOr(&named[k >> 5], 1u << (k & 31));
    }
  }
  __syncthreads();
  zero_rows<kWide>(a.p, dtable, v0, v1, named);
}

// `lanes` lanes per piece and block of kCols * lanes columns.  Bytes bound it: the
// rows in, gathered, and the whole table out (131072 rows of 256 bf16 into 129280
// of fp32: 41 us, 4.9 TB/s of 199 MB).
template <bool kWide, typename TT, typename TR>
__global__ void __launch_bounds__(kThreads)
    k_grad_sums(SumArgs a, const TR* __restrict__ drows, TT* dtable) {
  grid_dependency_release();
  grid_dependency_wait();
  if ((int)blockIdx.x >= a.sum_ctas) {
    zero_unnamed<kWide>(a, dtable, blockIdx.x - a.sum_ctas);
    return;
  }
  const int64_t job = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / a.lanes;
  const int m = (int)(job / a.blocks);
  if (m >= a.pieces) return;
  const Columns<kWide> c((int)(job % a.blocks), threadIdx.x % a.lanes, a.lanes, a.p.D);
  const int n = a.p.n, V = a.p.V, j0 = m * a.piece, j1 = min(j0 + a.piece, n);
  int cur = __ldg(a.keys + j0);
  bool came_in = j0 > 0 && __ldg(a.keys + j0 - 1) == cur;
  const int next = j1 < n ? __ldg(a.keys + j1) : V;
  float acc[kCols] = {};
  auto part = [&](int which) {
    if (c.any()) store8<kWide>(a.part + ((int64_t)m * 2 + which) * a.width + c.at, c, acc);
  };
  // four positions at a time; while one four is added, the rows of the next are
  // on their way and the positions after those are read (lists end on 256 bytes)
  constexpr int kFour = 4;
  int4 key = __ldg(reinterpret_cast<const int4*>(a.keys + j0));
  int4 pos = __ldg(reinterpret_cast<const int4*>(a.pos + j0));
  Raw<kWide, TR> x[kFour];
  int now[kFour];
  auto fetch = [&](int j) {
    const int k[kFour] = {key.x, key.y, key.z, key.w}, at[kFour] = {pos.x, pos.y, pos.z, pos.w};
#pragma unroll
    for (int q = 0; q < kFour; ++q) {
      now[q] = j + q < j1 ? k[q] : V;
      if (now[q] < V)
        x[q].load(drows + (int64_t)at[q] * a.p.row_stride + c.at, c);
      else
        x[q].clear();
    }
    if (j + kFour < j1) {
      key = __ldg(reinterpret_cast<const int4*>(a.keys + j + kFour));
      pos = __ldg(reinterpret_cast<const int4*>(a.pos + j + kFour));
    }
  };
  fetch(j0);
  for (int j = j0; j < j1; j += kFour) {
    Raw<kWide, TR> y[kFour];
    int own[kFour];
#pragma unroll
    for (int q = 0; q < kFour; ++q) {
      y[q] = x[q];
      own[q] = now[q];
    }
    if (j + kFour < j1) fetch(j + kFour);
#pragma unroll
    for (int q = 0; q < kFour; ++q) {
      if (own[q] != cur) {  // the run ends here, or no run goes on
        if (cur < V) {
          if (came_in)
            part(0);
          else
            put_row<kWide>(a.p, dtable, cur, c, acc);
        }
        cur = own[q];
        came_in = false;
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < kCols; ++k) acc[k] += y[q].get(k);
    }
  }
  if (cur >= V) return;
  if (came_in)
    part(0);
  else if (next == cur)
    part(1);
  else
    put_row<kWide>(a.p, dtable, cur, c, acc);
}

// A warp per piece and block of columns: if a run begins in the piece that goes on
// after it, the sum of the run's parts.  A run through many pieces is summed by
// the CTA together, a stretch of the parts per warp; no two of them begin among
// the pieces of one CTA.  Latency bounds it: the keys at the borders, the keys of
// the pieces after, the parts.
constexpr int kJoinWarps = kThreads / 32;
constexpr int kManyParts = 16;
static_assert(kManyParts >= kJoinWarps && kManyParts <= 32, "one long run per CTA, seen by one look");

template <bool kWide, typename TT>
__global__ void __launch_bounds__(kThreads) k_grad_join(SumArgs a, TT* dtable) {
  __shared__ float sums[kJoinWarps][32 * kCols];
  __shared__ int long_piece;
  const int n = a.p.n, V = a.p.V, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m = blockIdx.x * kJoinWarps + warp;
  const Columns<kWide> c(blockIdx.y, lane, 32, a.p.D);
  if (threadIdx.x == 0) long_piece = -1;
  __syncthreads();
  grid_dependency_wait();
  // the parts q0 .. q1 - 1 of the run that begins in piece `from`
  auto sum = [&](int from, int q0, int q1, float* acc) {
    constexpr int kAhead = 8;
#pragma unroll
    for (int k = 0; k < kCols; ++k) acc[k] = 0.f;
    for (int q = q0; q < q1; q += kAhead) {
      Raw<kWide, float> x[kAhead];
#pragma unroll
      for (int r = 0; r < kAhead; ++r) {
        const int at = min(q + r, q1 - 1);
        x[r].load(a.part + ((int64_t)(from + at) * 2 + (at == 0)) * a.width + c.at, c);
      }
#pragma unroll
      for (int r = 0; r < kAhead; ++r) {
        if (q + r >= q1) break;
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] += x[r].get(k);
      }
    }
  };
  float acc[kCols];
  const int64_t j0 = (int64_t)m * a.piece, j1 = j0 + a.piece;
  if (j1 < n) {
    // all looks at once: the piece's borders, and where the pieces after it begin
    const int64_t ahead = (int64_t)(m + 1 + lane) * a.piece;
    const int key = __ldg(a.keys + j1), end = __ldg(a.keys + j1 - 1);
    const int before = j0 > 0 ? __ldg(a.keys + j0 - 1) : -1;
    const int more = __popc(__ballot_sync(0xffffffffu, ahead < n && __ldg(a.keys + min(ahead, (int64_t)n - 1)) == key));
    if (key < V && end == key && before != key) {
      if (more >= kManyParts) {
        if (lane == 0) long_piece = m;
      } else {
        sum(m, 0, more + 1, acc);
        put_row<kWide>(a.p, dtable, key, c, acc);
      }
    }
  }
  __syncthreads();
  const int from = long_piece;
  if (from < 0) return;
  const int key = __ldg(a.keys + (int64_t)(from + 1) * a.piece);
  int more = 0;  // pieces after it into which the run goes
  for (int q0 = from + 1;; q0 += kThreads) {
    const int64_t q = (int64_t)q0 + threadIdx.x;
    const int got = __syncthreads_count(q < a.pieces && __ldg(a.keys + q * a.piece) == key);
    more += got;
    if (got < kThreads) break;
  }
  const int per = (more + 1 + kJoinWarps - 1) / kJoinWarps;
  const int q0 = min(warp * per, more + 1), q1 = min(q0 + per, more + 1);
  sum(from, q0, q1, acc);
#pragma unroll
  for (int k = 0; k < kCols; ++k) sums[warp][k * 32 + lane] = acc[k];
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
    for (int k = 0; k < kCols; ++k) acc[k] += sums[w][k * 32 + lane];
  put_row<kWide>(a.p, dtable, key, c, acc);
}

// ---- Host ----------------------------------------------------------------------------------
constexpr int kMaxSortCtas = 64;

struct GradPlan {
  int rounds, ctas, per, passes, bits;  // sort
  int piece, pieces, lanes, blocks, width;  // sums
  size_t keys, hist, part, bytes;      // offsets after the two key and position arrays
};

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

GradPlan plan_of(const spec_embed_params& p) {
  GradPlan g = {};
  g.rounds = p.n <= kMaxSortCtas * kFewRounds * kSortThreads ? kFewRounds : kManyRounds;
  const int tile = g.rounds * kSortThreads;
  const int64_t tiles = ((int64_t)p.n + tile - 1) / tile;
  g.ctas = (int)std::min<int64_t>(tiles, kMaxSortCtas);
  g.per = (int)((tiles + g.ctas - 1) / g.ctas) * tile;
  g.ctas = (int)(((int64_t)p.n + g.per - 1) / g.per);
  int bits = 1;
  while (bits < 31 && (int64_t(1) << bits) <= p.V) ++bits;  // the largest key is V
  if ((int64_t(1) << bits) <= p.V) ++bits;
  g.passes = (bits + 8) / 9;
  g.bits = (bits + g.passes - 1) / g.passes;
  g.lanes = 1;
  while (g.lanes < 32 && g.lanes * kCols < p.D) g.lanes *= 2;
  g.blocks = (p.D + g.lanes * kCols - 1) / (g.lanes * kCols);
  g.width = g.blocks * g.lanes * kCols;
  // enough pieces to fill the GPU, long enough to be worth their parts; of a B200's
  // size on any device, so that the workspace's size is the same on all
  g.piece = 16;
  while (g.piece < 128 && (int64_t)p.n / (2 * g.piece) * g.blocks * g.lanes >= 148 * 384) g.piece *= 2;
  g.pieces = (int)(((int64_t)p.n + g.piece - 1) / g.piece);
  const size_t list = round256(sizeof(int32_t) * (size_t)p.n);
  g.keys = 4 * list;
  g.hist = g.keys;
  g.part = g.hist + round256(sizeof(int32_t) * (size_t)g.ctas * kDigits);
  g.bytes = g.part + round256(sizeof(float) * 2 * (size_t)g.pieces * g.width);
  return g;
}

// Table rows that a CTA zeroes: about four CTAs for every SM.
int zero_rows_per_cta(const spec_embed_params& p, int num_sms) {
  return (int)std::min<int64_t>(kZeroRows, ((int64_t)p.V + 4 * num_sms - 1) / (4 * num_sms));
}

template <bool kWide, typename TT, typename TR>
cudaError_t grad(const spec_embed_params& p, const int32_t* ids, const TR* drows, TT* dtable,
                 uint8_t* body, WsHeader* hdr, int num_sms, cudaStream_t st, int* launches) {
  if (p.n <= kDirect) {
    const int per = zero_rows_per_cta(p, num_sms);
    const int zero = p.accumulate ? 0 : (int)(((int64_t)p.V + per - 1) / per);
    *launches = 1;
    return launch_kernel(k_grad_direct<kWide, TT, TR>, p.n + zero, 32 * kDirectWarps, 0, st, p, ids,
                         drows, dtable, per, hdr);
  }
  const GradPlan g = plan_of(p);
  const size_t list = g.keys / 4;
  SortArgs a = {};
  a.p = p;
  a.ids = ids;
  for (int k = 0; k < 2; ++k) {
    a.keys[k] = reinterpret_cast<int32_t*>(body + k * list);
    a.pos[k] = reinterpret_cast<int32_t*>(body + (2 + k) * list);
  }
  a.hist = reinterpret_cast<int32_t*>(body + g.hist);
  a.ctas = g.ctas;
  a.per = g.per;
  a.passes = g.passes;
  a.bits = g.bits;
  a.spin = 4000000ull;
  a.hdr = hdr;
  void* args[] = {&a};
  const void* sort = g.rounds == kFewRounds ? (const void*)k_grad_sort<kFewRounds>
                                            : (const void*)k_grad_sort<kManyRounds>;
  cudaError_t e = cudaLaunchCooperativeKernel(sort, dim3(g.ctas), dim3(kSortThreads), args, 0, st);
  if (e != cudaSuccess) return e;
  SumArgs s = {};
  s.p = p;
  s.keys = a.keys[g.passes & 1];
  s.pos = a.pos[g.passes & 1];
  s.part = reinterpret_cast<float*>(body + g.part);
  s.piece = g.piece;
  s.pieces = g.pieces;
  s.lanes = g.lanes;
  s.blocks = g.blocks;
  s.width = g.width;
  const int64_t threads = (int64_t)g.pieces * g.blocks * g.lanes;
  const int64_t sum_ctas = (threads + kThreads - 1) / kThreads;
  s.zero_per = zero_rows_per_cta(p, num_sms);
  const int64_t zero = p.accumulate ? 0 : ((int64_t)p.V + s.zero_per - 1) / s.zero_per;
  if (sum_ctas + zero > INT32_MAX) return cudaErrorInvalidValue;
  s.sum_ctas = (int)sum_ctas;
  e = launch_after(k_grad_sums<kWide, TT, TR>, dim3((unsigned)(sum_ctas + zero)), kThreads, 0, st, s,
                   drows, dtable);
  if (e != cudaSuccess) return e;
  *launches = 3;
  return launch_after(k_grad_join<kWide, TT>,
                      dim3((g.pieces + kJoinWarps - 1) / kJoinWarps, (p.D + 32 * kCols - 1) / (32 * kCols)),
                      kThreads, 0, st, s, dtable);
}

}  // namespace

size_t embed_grad_ws_bytes(const spec_embed_params& p) {
  return p.n <= kDirect ? 0 : plan_of(p).bytes;
}

// Rows of whole vectors of four columns, 16-byte aligned, in both tensors.
template <typename TT, typename TR>
bool wide_ok(const spec_embed_params& p, const void* table, const void* rows) {
  return p.D % 4 == 0 && p.table_stride * sizeof(TT) % 16 == 0 &&
         p.row_stride * sizeof(TR) % 16 == 0 &&
         ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(rows)) & 15) == 0;
}

template <typename TT, typename TR>
cudaError_t launch_embed(const spec_embed_params& p, const TT* table, const int32_t* ids, TR* rows,
                         WsHeader* hdr, int, cudaStream_t st, int* launches) {
  int shift = 0;  // log2 of the lanes per row
  while (shift < 5 && (kCols << shift) < p.D) ++shift;
  const int blocks = (p.D + (kCols << shift) - 1) / (kCols << shift);
  const int per = blocks == 1 ? 4 : blocks == 2 ? 2 : 1;  // rows that lanes take together
  const int64_t groups = ((int64_t)p.n + per - 1) / per;
  const int64_t grid = ((groups << shift) + kThreads - 1) / kThreads;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  *launches = 1;
  const bool wide = wide_ok<TT, TR>(p, table, rows);
  auto run = [&](auto kernel) {
    return launch_kernel(kernel, (unsigned)grid, kThreads, 0, st, p, table, ids, rows, shift, hdr);
  };
  if (per == 4) return wide ? run(k_embed<true, 4, TT, TR>) : run(k_embed<false, 4, TT, TR>);
  if (per == 2) return wide ? run(k_embed<true, 2, TT, TR>) : run(k_embed<false, 2, TT, TR>);
  return wide ? run(k_embed<true, 1, TT, TR>) : run(k_embed<false, 1, TT, TR>);
}

template <typename TT, typename TR>
cudaError_t launch_embed_grad(const spec_embed_params& p, const int32_t* ids, const TR* drows,
                              TT* dtable, uint8_t* body, WsHeader* hdr, int num_sms,
                              cudaStream_t st, int* launches) {
  return wide_ok<TT, TR>(p, dtable, drows)
             ? grad<true, TT, TR>(p, ids, drows, dtable, body, hdr, num_sms, st, launches)
             : grad<false, TT, TR>(p, ids, drows, dtable, body, hdr, num_sms, st, launches);
}

#define SPEC_INST(TT, TR)                                                                          \
  template cudaError_t launch_embed<TT, TR>(const spec_embed_params&, const TT*, const int32_t*,   \
                                            TR*, WsHeader*, int, cudaStream_t, int*);              \
  template cudaError_t launch_embed_grad<TT, TR>(const spec_embed_params&, const int32_t*,         \
                                                 const TR*, TT*, uint8_t*, WsHeader*, int,         \
                                                 cudaStream_t, int*);
SPEC_INST(float, float)
SPEC_INST(float, __nv_bfloat16)
SPEC_INST(__nv_bfloat16, float)
SPEC_INST(__nv_bfloat16, __nv_bfloat16)
#undef SPEC_INST

}  // namespace specdec
