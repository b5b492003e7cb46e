// Entry points of cross attention (include/wb.h): argument checks, tensor maps and launches.
#include <cmath>
#include <mutex>

#include "../../include/wb.h"
#include "internal.h"
#include "cross_attention.cuh"
#include "cross_few.cuh"
#include "cross_backward.cuh"

namespace wb {
namespace {

constexpr int64_t MAX_T = 1 << 24;
constexpr int64_t MAX_STRIDE = 1LL << 38;      // elements: a tensor map's strides stay below 2^40 bytes

std::mutex g_mu;

// Raise a kernel's dynamic shared-memory limit once per device: launches stay free of attribute calls.
template <typename K>
cudaError_t allow_smem(K kern, int smem, uint64_t* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(g_mu);
  const uint64_t bit = 1ull << (dev & 63);
  if (*done & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) *done |= bit;
  return e;
}

// Rows of bf16 [items][T][heads * 64] with strides in elements.
struct Rows {
  const void* p;
  int64_t batch, row;
  int items;                 // 0: all items read the first one's rows
};

// A dimension of one element has no stride; a batch stride of 0 is one item for all.
bool rows_ok(Rows& r, const void* p, int64_t batch_stride, int64_t row_stride, int batch, int T, int heads) {
  if (!p || !aligned16(p)) return false;
  r.p = p;
  r.row = T == 1 ? heads * 64LL : row_stride;
  r.batch = batch == 1 ? 0 : batch_stride;
  r.items = r.batch != 0;
  return r.row >= heads * 64LL && r.row < MAX_STRIDE && r.row % 8 == 0 && r.batch >= 0 && r.batch < MAX_STRIDE && r.batch % 8 == 0;
}

bool rows_map(CUtensorMap* m, const Rows& r, int batch, int T, int heads, int box_rows) {
  const uint64_t dims[3] = {heads * 64ull, static_cast<uint64_t>(T), r.items ? static_cast<uint64_t>(batch) : 1ull};
  const uint64_t str[2] = {static_cast<uint64_t>(r.row) * 2, static_cast<uint64_t>(r.items ? r.batch : r.row) * 2};
  const uint32_t box[3] = {64u, static_cast<uint32_t>(box_rows), 1u};
  return tma_map_bf16(m, 3, r.p, dims, str, box);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Sizes that every call checks; the largest grid is one block for each 64 rows of an (item, head).
bool sizes_ok(int batch, int Tq, int Tk, int H, int Hk, float scale) {
  if (batch < 0 || Tq < 0 || Tk < 0 || Tq > MAX_T || Tk > MAX_T || Hk < 1 || H < Hk || H > 1024 || H % Hk != 0) return false;
  if (!(scale >= 0x1p-64f && scale <= 0x1p64f)) return false;
  const int64_t tiles = ((Tq > Tk ? Tq : Tk) + 127) / 128 + 1;
  return static_cast<int64_t>(batch) * H * tiles * 8 <= 0x7fffffffLL;
}

void base(CrossParams& x, int batch, int Tq, int Tk, int H, int Hk, float scale, const int32_t* q_lens, const int32_t* kv_lens,
          const Rows& q, const Rows& k) {
  x.batch = batch;
  x.Tq = Tq;
  x.Tk = Tk;
  x.H = H;
  x.Hk = Hk;
  x.group = H / Hk;
  x.splits = 1;
  x.q_items = q.items;
  x.kv_items = k.items;
  x.scale = scale;
  x.c = scale * 1.4426950408889634f;
  x.slack = 8.0f / x.c;
  x.q_lens = q_lens;
  x.kv_lens = kv_lens;
  x.out = nullptr;
  x.lse = nullptr;
  x.err = tc_err_ptr();
}

// As launch_pdl, in clusters of `splits` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_split(void (*kern)(KArgs...), unsigned grid, unsigned block, size_t smem, unsigned splits, cudaStream_t s,
                         Args... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Splits of the keys of few rows: 1, 2, 4 or 8, while there are fewer CTAs than SMs and a split has 64 keys.  Up to twice the SMs, as two fit each,
// was slower: 2 x 20 pairs over 1500 keys 9.4 us against 7.8, 5 x 20 14.6 against 11.8, 12 x 20 23.5 against 20.
int few_splits(long long pairs, int Tk) {
  int n = 1;
  while (n < FEW_MAX_SPLITS && pairs * n < sm_count() && Tk >= 2 * n * 64) n *= 2;
  return n;
}

// Splits of the keys of a tile of rows: 1, 2, 4 or 8, while `places` for CTAs stay empty and a split has two tiles of keys.
int tile_splits(long long tiles, int Tk, int places) {
  int n = 1;
  while (n < CRA_MAX_SPLITS && 2 * tiles * n <= places && Tk > 2 * n * 2 * CRA_BK - CRA_BK) n *= 2;
  return n;
}

}  // namespace
}  // namespace wb

using namespace wb;

extern "C" {

wb_status wb_cross_attention(const void* q, int64_t q_batch, int64_t q_row, const void* k, int64_t k_batch, int64_t k_row,
                             const void* v, int64_t v_batch, int64_t v_row, const int32_t* q_lens, const int32_t* kv_lens,
                             int batch, int Tq, int Tk, int n_heads, int n_kv_heads, float scale, void* out, float* lse,
                             void* stream) {
  if (!sizes_ok(batch, Tq, Tk, n_heads, n_kv_heads, scale)) return WB_EINVAL;
  if (batch == 0 || Tq == 0) return WB_OK;
  Rows rq, rk{nullptr, 0, 0, 0}, rv{nullptr, 0, 0, 0};
  if (!rows_ok(rq, q, q_batch, q_row, batch, Tq, n_heads)) return WB_EINVAL;
  if (Tk > 0 && (!rows_ok(rk, k, k_batch, k_row, batch, Tk, n_kv_heads) || !rows_ok(rv, v, v_batch, v_row, batch, Tk, n_kv_heads) ||
                 rk.items != rv.items))
    return WB_EINVAL;
  if (!out || !aligned16(out) || !lse || !aligned4(lse) || !aligned4(q_lens) || !aligned4(kv_lens)) return WB_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  FewParams p;
  base(p.x, batch, Tq, Tk, n_heads, n_kv_heads, scale, q_lens, kv_lens, rq, rk);
  if (!p.x.err) return WB_ECUDA;
  p.x.out = static_cast<__nv_bfloat16*>(out);
  p.x.lse = lse;
  Prof pr(PC_CROSS_FWD, s);
  const long long rows = static_cast<long long>(p.x.group) * Tq;
  if (rows <= FEW_ROWS) {
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.q_batch = rq.batch;
    p.q_row = rq.row;
    p.k_batch = rk.batch;
    p.k_row = rk.row;
    p.v_batch = rv.batch;
    p.v_row = rv.row;
    p.splits = few_splits(static_cast<long long>(batch) * n_kv_heads, Tk);
    static uint64_t few_done = 0;
    WB_CUDA(allow_smem(cross_few_kernel, FewSmem::TOTAL, &few_done));
    WB_CUDA(launch_split(cross_few_kernel, static_cast<unsigned>(batch) * n_kv_heads * p.splits, FEW_THREADS, FewSmem::TOTAL, p.splits, s, p));
    return WB_OK;
  }
  CUtensorMap qm, km, vm;
  if (!rows_map(&qm, rq, batch, Tq, n_heads, CRA_BQ)) return WB_ECUDA;
  km = vm = qm;                    // no keys: never read
  if (Tk > 0 && (!rows_map(&km, rk, batch, Tk, n_kv_heads, CRA_BK) || !rows_map(&vm, rv, batch, Tk, n_kv_heads, CRA_BK))) return WB_ECUDA;
  static uint64_t done = 0;
  WB_CUDA(allow_smem(cross_fwd_kernel, CrossSmem::TOTAL, &done));
  const unsigned tiles = static_cast<unsigned>(batch) * n_heads * ((Tq + CRA_BQ - 1) / CRA_BQ);
  p.x.splits = tile_splits(tiles, Tk, 2 * sm_count());
  WB_CUDA(launch_split(cross_fwd_kernel, tiles * p.x.splits, CRA_THREADS, CrossSmem::TOTAL, p.x.splits, s, qm, km, vm, p.x));
  return WB_OK;
}

size_t wb_cross_attention_backward_workspace_bytes(int batch, int Tq, int n_heads) {
  if (batch < 1 || Tq < 1 || n_heads < 1 || Tq > MAX_T || n_heads > 1024) return 0;
  return static_cast<size_t>(batch) * n_heads * ((Tq + 127) / 128 * 128) * 2 * sizeof(float);
}

wb_status wb_cross_attention_backward(const void* dout, int64_t do_batch, int64_t do_row, const void* q, int64_t q_batch,
                                      int64_t q_row, const void* k, int64_t k_batch, int64_t k_row, const void* v,
                                      int64_t v_batch, int64_t v_row, const void* out, const float* lse,
                                      const int32_t* q_lens, const int32_t* kv_lens, int batch, int Tq, int Tk, int n_heads,
                                      int n_kv_heads, float scale, void* dq, void* dk, void* dv, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  if (!sizes_ok(batch, Tq, Tk, n_heads, n_kv_heads, scale)) return WB_EINVAL;
  if (!dk != !dv || !aligned16(dq) || !aligned16(dk) || !aligned16(dv)) return WB_EINVAL;
  if (batch == 0 || (!dq && !dk)) return WB_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t q_bytes = static_cast<size_t>(batch) * Tq * n_heads * 128, kv_bytes = static_cast<size_t>(batch) * Tk * n_kv_heads * 128;
  if (Tq == 0 || Tk == 0) {
    if (dq && q_bytes) WB_CUDA(cudaMemsetAsync(dq, 0, q_bytes, s));
    if (dk && kv_bytes) {
      WB_CUDA(cudaMemsetAsync(dk, 0, kv_bytes, s));
      WB_CUDA(cudaMemsetAsync(dv, 0, kv_bytes, s));
    }
    return WB_OK;
  }
  Rows ro, rq, rk, rv;
  if (!rows_ok(ro, dout, do_batch, do_row, batch, Tq, n_heads) || !rows_ok(rq, q, q_batch, q_row, batch, Tq, n_heads) ||
      !rows_ok(rk, k, k_batch, k_row, batch, Tk, n_kv_heads) || !rows_ok(rv, v, v_batch, v_row, batch, Tk, n_kv_heads) ||
      rk.items != rv.items)
    return WB_EINVAL;
  if (!out || !aligned16(out) || !lse || !aligned4(lse) || !aligned4(q_lens) || !aligned4(kv_lens)) return WB_EINVAL;
  if (!workspace || !aligned16(workspace) || workspace_bytes < wb_cross_attention_backward_workspace_bytes(batch, Tq, n_heads))
    return WB_EWORKSPACE;
  CrossBwdParams p;
  base(p.x, batch, Tq, Tk, n_heads, n_kv_heads, scale, q_lens, kv_lens, rq, rk);
  if (!p.x.err) return WB_ECUDA;
  p.x.out = const_cast<__nv_bfloat16*>(static_cast<const __nv_bfloat16*>(out));
  p.x.lse = const_cast<float*>(lse);
  p.dout = static_cast<const __nv_bfloat16*>(dout);
  p.do_batch = ro.batch;
  p.do_row = ro.row;
  p.do_items = ro.items;
  p.stats = static_cast<float*>(workspace);
  p.stats_ld = (Tq + 127) / 128 * 128;
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.want_dq = dq != nullptr;
  Prof pr(PC_CROSS_BWD, s, dk ? 2 : 1);
  const int sms = sm_count();
  CUtensorMap qm, dm, km, vm;
  if (!rows_map(&qm, rq, batch, Tq, n_heads, CRB_M) || !rows_map(&dm, ro, batch, Tq, n_heads, CRB_M) ||
      !rows_map(&km, rk, batch, Tk, n_kv_heads, CRB_M) || !rows_map(&vm, rv, batch, Tk, n_kv_heads, CRB_M))
    return WB_ECUDA;
  static uint64_t dq_done[2] = {}, dkv_done[2] = {};
  constexpr int SMEM = CrossBwdSmem::TOTAL;
  const bool few_keys = Tk <= CRB_STEP / 2, few_rows = Tq <= CRB_STEP / 2;
  auto dq_kernel = few_keys ? cross_bwd_kernel<false, true> : cross_bwd_kernel<false, false>;
  auto dkv_kernel = few_rows ? cross_bwd_kernel<true, true> : cross_bwd_kernel<true, false>;
  WB_CUDA(allow_smem(dq_kernel, SMEM, &dq_done[few_keys]));
  if (dk) WB_CUDA(allow_smem(dkv_kernel, SMEM, &dkv_done[few_rows]));
  const long long q_items = static_cast<long long>(batch) * n_heads * ((Tq + CRB_M - 1) / CRB_M);
  const long long k_items = static_cast<long long>(batch) * n_kv_heads * ((Tk + CRB_M - 1) / CRB_M);
  p.x.splits = tile_splits(q_items, Tk, sms);
  const unsigned q_grid = p.x.splits > 1 ? static_cast<unsigned>(q_items) * p.x.splits : static_cast<unsigned>(q_items < sms ? q_items : sms);
  WB_CUDA(launch_split(dq_kernel, q_grid, CRB_THREADS, SMEM, p.x.splits, s, qm, dm, km, vm, p));
  if (dk)
    WB_CUDA(launch_pdl(dkv_kernel, dim3(static_cast<unsigned>(k_items < sms ? k_items : sms)), dim3(CRB_THREADS), SMEM, s, km, vm, qm, dm, p));
  return WB_OK;
}

}  // extern "C"
