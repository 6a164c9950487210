// Scaled lookup of table rows by token, and its gradient.
#include "head_ops.cuh"

namespace specdec {
namespace {

constexpr int kThreads = 256;

// rows[i] = scale * table[ids[i]]: one CTA per row.
template <typename TT, typename TR>
__global__ void __launch_bounds__(kThreads)
    k_embed(spec_embed_params p, const TT* __restrict__ table, const int32_t* __restrict__ ids,
            TR* __restrict__ rows, WsHeader* hdr) {
  const int i = blockIdx.x;
  const int id = ids[i];
  const bool in = id >= 0 && id < p.V;
  if (!in && id != -1 && threadIdx.x == 0)
    report_error(hdr, SPEC_ERR_TOKEN_RANGE, SITE_TOKEN_RANGE, i, id);
  const TT* src = table + (int64_t)(in ? id : 0) * p.table_stride;
  TR* dst = rows + (int64_t)i * p.row_stride;
  for (int c = threadIdx.x; c < p.D; c += kThreads)
    store_f(dst, c, in ? load_f(src, c) * p.scale : 0.f);
}

// Zero the table's gradient.
template <typename TT>
__global__ void __launch_bounds__(kThreads) k_embed_zero(spec_embed_params p, TT* dtable) {
  TT* dst = dtable + (int64_t)blockIdx.x * p.table_stride;
  for (int c = threadIdx.x; c < p.D; c += kThreads) store_f(dst, c, 0.f);
}

// One CTA per position: the first position of each token sums the rows of all
// positions that name it, in ascending order.
template <typename TT, typename TR>
__global__ void __launch_bounds__(kThreads)
    k_embed_grad(spec_embed_params p, const int32_t* __restrict__ ids,
                 const TR* __restrict__ drows, TT* dtable, WsHeader* hdr) {
  const int i = blockIdx.x;
  const int id = ids[i];
  if (id < 0 || id >= p.V) {
    if (id != -1 && threadIdx.x == 0)
      report_error(hdr, SPEC_ERR_TOKEN_RANGE, SITE_TOKEN_RANGE, i, id);
    return;
  }
  bool seen = false;
  for (int j = threadIdx.x; j < i; j += kThreads) seen |= ids[j] == id;
  if (__syncthreads_or(seen)) return;
  TT* dst = dtable + (int64_t)id * p.table_stride;
  for (int c = threadIdx.x; c < p.D; c += kThreads) {
    float acc = 0.f;
    for (int j = i; j < p.n; ++j)
      if (ids[j] == id) acc += load_f(drows, (int64_t)j * p.row_stride + c);
    acc *= p.scale;
    if (p.accumulate) acc += load_f((const TT*)dst, c);
    store_f(dst, c, acc);
  }
}

}  // namespace

size_t embed_grad_ws_bytes(const spec_embed_params&) { return 0; }

template <typename TT, typename TR>
cudaError_t launch_embed(const spec_embed_params& p, const TT* table, const int32_t* ids, TR* rows,
                         WsHeader* hdr, int, cudaStream_t st, int* launches) {
  k_embed<TT, TR><<<p.n, kThreads, 0, st>>>(p, table, ids, rows, hdr);
  *launches = 1;
  return cudaGetLastError();
}

template <typename TT, typename TR>
cudaError_t launch_embed_grad(const spec_embed_params& p, const int32_t* ids, const TR* drows,
                              TT* dtable, uint8_t*, WsHeader* hdr, int, cudaStream_t st,
                              int* launches) {
  if (!p.accumulate) {
    k_embed_zero<TT><<<p.V, kThreads, 0, st>>>(p, dtable);
    ++*launches;
  }
  if (p.n > 0) {
    k_embed_grad<TT, TR><<<p.n, kThreads, 0, st>>>(p, ids, drows, dtable, hdr);
    ++*launches;
  }
  return cudaGetLastError();
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
