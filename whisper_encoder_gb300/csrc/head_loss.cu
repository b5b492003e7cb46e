// Losses of a vocabulary head straight from hidden states and the projection matrix: softmax cross
// entropy and distillation from a teacher's top logits, forward and backward, without keeping the
// logits.
//
// Both are one operator with sparse targets.  Row i has target entries (v_j, P_j) (cross entropy: its
// label with weight 1 - e, and e / V everywhere), s = x w^T / T, lse_i = log sum_v exp s_iv:
//   loss_i = T^2 sum_j P_j (log P_j - s_ij + lse_i)      D_iv = exp(s_iv - lse_i) - P_iv
//   dx_i = T dloss_i sum_v D_iv w_v                      dw_v = T sum_i dloss_i D_iv x_i
// Rows without a target take no part: they are taken out first (rows_kernel), so they cost no product,
// and whatever their x holds reaches nothing.  head_gemm.cuh has the products.
//
// Precision: s, lse, losses and every sum are float32.  D is rounded to bf16 once, as a factor of the
// two gradient products: w and x are bf16 and an MMA's operands have one type.  That makes dx and dw 1.8e-3 to
// 2.4e-3 of the 2-norm off 64 bits, their own rounding alone 1.7e-3; D in two parts would be two products more on
// top of four.  |D| <= 1, and dloss stays outside of it (applied to the float32 sums of dx,
// and to x' = dloss / max|dloss| x for dw, exactly 1 where all dloss are equal), so that one rounding of
// dloss is not shared by all of a row's or all of dw's entries.
#include <cfloat>
#include <cstring>
#include <mutex>

#include "../../include/wb.h"
#include "internal.h"
#include "head_gemm.cuh"
#include "head_gemv.cuh"

namespace wb {
namespace {

constexpr int HEAD_MAX_K = 1024;
constexpr int ROWS_THREADS = 256;
constexpr int FIN_ROWS = 32, FIN_SLICES = 32;
constexpr int HEAD_SMS = 152;    // sizes of workspaces do not depend on the device that asks
constexpr int OWN_MAX_ROWS = 2048;   // up to here each block of rows_kernel finds max |dloss| itself

// ---------------------------------------------------------------------------
// Teacher entries of one row per block: softmax of the stored logits at the temperature, equal indices
// merged, sorted by index.  cnt: entries, 0 for a row without any, -2 for a row with an index >= V.
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float teacher_f32(T v);
template <>
__device__ __forceinline__ float teacher_f32(float v) { return v; }
template <>
__device__ __forceinline__ float teacher_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float teacher_f32(__half v) { return __half2float(v); }

constexpr int LIST_THREADS = 128;

__device__ __forceinline__ float block_reduce(float v, bool is_max, float* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = is_max ? fmaxf(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sm[0];
  for (int i = 1; i < LIST_THREADS / 32; ++i) v = is_max ? fmaxf(v, sm[i]) : v + sm[i];
  return v;
}

template <typename T>
__global__ void __launch_bounds__(LIST_THREADS)
    target_lists_kernel(const T* __restrict__ top, const int64_t* __restrict__ index, int M, int k, int V,
                        float inv_t, int* __restrict__ out_idx, float* __restrict__ out_p, int* __restrict__ out_cnt,
                        uint32_t* err) {
  extern __shared__ __align__(16) int sm_list[];
  const int kp = (k + 3) & ~3;                             // read four at a time
  int* id = sm_list;                                       // [kp]
  float* pr = reinterpret_cast<float*>(sm_list + kp);      // [kp]
  int* lead = sm_list + 2 * kp;                            // [kp]: the index, where the entry stands for it
  __shared__ float sm[LIST_THREADS / 32];
  __shared__ int n_bad, n_out;
  grid_dependency_wait();
  grid_dependents_launch();
  const long long n_el = static_cast<long long>(M) * k;
  const int row = blockIdx.x;
  const long long base = static_cast<long long>(row) * k;
  if (threadIdx.x == 0) n_bad = n_out = 0;
  __syncthreads();
  float mx = -INFINITY;
  for (int j = threadIdx.x; j < kp; j += LIST_THREADS) {
    id[j] = -1;
    pr[j] = 0.0f;
    if (j >= k || !in_bounds(err, base + j, 1, n_el, SITE_HEAD_LIST)) continue;
    const long long v = index[base + j];
    const float t = teacher_f32<T>(top[base + j]);
    if (v >= V) atomicAdd(&n_bad, 1);
    const bool on = v >= 0 && v < V && !(t == -INFINITY);
    id[j] = on ? static_cast<int>(v) : -1;
    pr[j] = on ? t : -INFINITY;
    if (on) mx = fmaxf(mx, t);
  }
  mx = block_reduce(mx, true, sm);
  float sum = 0.0f;
  for (int j = threadIdx.x; j < k; j += LIST_THREADS) {
    if (id[j] < 0) continue;
    pr[j] = expf((pr[j] - mx) * inv_t);          // a difference that is never positive, whatever the temperature
    sum += pr[j];
  }
  sum = block_reduce(sum, false, sm);
  // entry j stands for its index if no earlier entry has it; it then has the sum of all of them
  constexpr int NONE = 0x7fffffff;
  for (int j = threadIdx.x; j < kp; j += LIST_THREADS) {
    const int my = id[j];
    bool first = my >= 0;
    float p = 0.0f;
    for (int q = 0; first && q < kp; q += 4) {
      const int4 o = *reinterpret_cast<const int4*>(id + q);
      if (o.x != my && o.y != my && o.z != my && o.w != my) continue;
      const int e[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (e[u] == my) {
          first = first && q + u >= j;
          p += pr[q + u];
        }
    }
    // a weight of zero is no entry (log 0): the weight as it is stored, which may be zero where exp was not
    lead[j] = first && !(p / sum == 0.0f) ? my : NONE;
  }
  __syncthreads();
  for (int j = threadIdx.x; j < k; j += LIST_THREADS) {
    const int my = lead[j];
    if (my == NONE) continue;
    int rank = 0;
    float p = 0.0f;
    for (int q = 0; q < kp; q += 4) {
      const int4 o = *reinterpret_cast<const int4*>(lead + q), e = *reinterpret_cast<const int4*>(id + q);
      rank += (o.x < my) + (o.y < my) + (o.z < my) + (o.w < my);
      if (e.x == my) p += pr[q];
      if (e.y == my) p += pr[q + 1];
      if (e.z == my) p += pr[q + 2];
      if (e.w == my) p += pr[q + 3];
    }
    if (in_bounds(err, base + rank, 1, n_el, SITE_HEAD_LIST)) {
      out_idx[base + rank] = my;
      out_p[base + rank] = p / sum;
    }
    atomicAdd(&n_out, 1);
  }
  __syncthreads();
  if (threadIdx.x == 0 && in_bounds(err, row, 1, M, SITE_HEAD_LIST)) out_cnt[row] = n_bad ? -2 : n_out;
}

// ---------------------------------------------------------------------------
// Rows that take part, in order: row_src, their x (and x'), what the others get.
// ---------------------------------------------------------------------------
struct RowsArgs {
  const int64_t* labels;     // cross entropy: 0 <= label < V takes part
  const int* cnt;            // distillation: cnt > 0 takes part
  int M, V, d, rows_per_block;
  int m_pad;                 // rows of xc and xs
  const __nv_bfloat16* x;
  __nv_bfloat16* xc;         // compacted
  int* row_src;
  int* row_tgt;              // by compact row: its label (cross entropy); distillation reads row_src and row_cnt
  int* row_cnt;
  float* row_lse;            // by compact row (backward)
  int* n_rows;
  // forward: what the rows without a target get
  float* loss;
  float* lse;
  // backward
  const float* dloss;
  const float* lse_in;
  float* g_max;              // max |dloss|: found by dloss_max_kernel before, or (own_max) by each block here
  int own_max;
  __nv_bfloat16* xs;         // compacted x' (null: not wanted)
  __nv_bfloat16* dx;         // rows without a target: zeros (null: not wanted)
  uint32_t* err;
};

// 1: row i takes part, 0: it does not, -1: its target is a mistake.
__device__ __forceinline__ int target_state(const int64_t* labels, const int* cnt, int V, int i) {
  if (labels) {
    const long long v = labels[i];
    return v < 0 ? 0 : v < V ? 1 : -1;
  }
  const int c = cnt[i];
  return c > 0 ? 1 : c == 0 ? 0 : -1;
}
__device__ __forceinline__ int row_state(const RowsArgs& a, int i) { return target_state(a.labels, a.cnt, a.V, i); }

__global__ void __launch_bounds__(ROWS_THREADS) rows_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ int warp_sum[ROWS_THREADS / 32];
  __shared__ float warp_max[ROWS_THREADS / 32];
  __shared__ int at[ROWS_THREADS];           // compact index of the block's rows, or -1 / -2
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_dependents_launch();
  const int r0 = blockIdx.x * a.rows_per_block;
  const int r1 = min(r0 + a.rows_per_block, a.M);
  // this warp's first row of x is asked for before its place is known
  constexpr int PRE = 5;
  const int nv = a.d / 8;
  uint4 pre[PRE];
  const uint4* pre_src = reinterpret_cast<const uint4*>(a.x + static_cast<long long>(r0 + warp) * a.d);
#pragma unroll
  for (int q = 0; q < PRE; ++q)
    if (r0 + warp < r1 && lane + 32 * q < nv &&
        in_bounds(a.err, static_cast<long long>(r0 + warp) * a.d + 8 * (lane + 32 * q), 8,
                  static_cast<long long>(a.M) * a.d, SITE_HEAD_X))
      pre[q] = pre_src[lane + 32 * q];
  // rows that take part before this block's
  int before = 0;
  for (int i = threadIdx.x; i < r0; i += ROWS_THREADS) before += row_state(a, i) == 1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (lane == 0) warp_sum[warp] = before;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int w = 0; w < ROWS_THREADS / 32; ++w) before += warp_sum[w];
  __syncthreads();
  int all = before;                          // rows that take part up to the end of the chunk at hand
  float g = 0.0f;
  const long long n_el = static_cast<long long>(a.M) * a.d;   // xc and xs have at least as many
  // the block's own rows, a chunk of one a thread at a time (beyond 311296 rows a block has more than one chunk)
  for (int c0 = r0; c0 < r1; c0 += ROWS_THREADS) {
    const int c1 = min(c0 + ROWS_THREADS, r1);
    if (c0 != r0) __syncthreads();           // at and warp_sum have been read
    const int row = c0 + threadIdx.x;
    const int st = row < c1 ? row_state(a, row) : 0;
    const unsigned ball = __ballot_sync(0xffffffffu, st == 1);
    if (lane == 0) warp_sum[warp] = __popc(ball);
    __syncthreads();
    int off = all;
#pragma unroll
    for (int w = 0; w < ROWS_THREADS / 32; ++w) {
      if (w < warp) off += warp_sum[w];
      all += warp_sum[w];
    }
    off += __popc(ball & ((1u << lane) - 1u));
    if (row < c1) {
      at[threadIdx.x] = st == 1 ? off : -1;
      if (st == 1 && in_bounds(a.err, off, 1, a.M, SITE_HEAD_ROWS)) {
        a.row_src[off] = row;
        if (a.labels) a.row_tgt[off] = static_cast<int>(a.labels[row]);
        else a.row_cnt[off] = a.cnt[row];
        if (a.lse_in) a.row_lse[off] = a.lse_in[row];
      }
      if (st != 1 && a.loss) {
        a.loss[row] = st == 0 ? 0.0f : __int_as_float(0x7fc00000);
        a.lse[row] = 0.0f;
      }
    }
    const bool find_max = a.xs && a.own_max && c0 == r0;
    if (find_max) {
      for (int i = threadIdx.x; i < a.M; i += ROWS_THREADS)
        if (row_state(a, i) == 1) g = fmaxf(g, fabsf(a.dloss[i]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
      if (lane == 0) warp_max[warp] = g;
    }
    __syncthreads();
    if (find_max) {
#pragma unroll
      for (int w = 0; w < ROWS_THREADS / 32; ++w) g = fmaxf(g, warp_max[w]);
      if (blockIdx.x == 0 && threadIdx.x == 0) *a.g_max = g;
    } else if (a.xs && !a.own_max) {
      g = *a.g_max;
    }
    for (int i = c0 + warp; i < c1; i += ROWS_THREADS / 32) {
      const int dst = at[i - c0];
      if (dst < 0) {
        if (a.dx)
          for (int v = lane; v < nv; v += 32)
            if (in_bounds(a.err, static_cast<long long>(i) * a.d + 8 * v, 8, n_el, SITE_HEAD_DX))
              *reinterpret_cast<uint4*>(a.dx + static_cast<long long>(i) * a.d + 8 * v) = make_uint4(0, 0, 0, 0);
        continue;
      }
      const uint4* src = reinterpret_cast<const uint4*>(a.x + static_cast<long long>(i) * a.d);
      uint4* to = reinterpret_cast<uint4*>(a.xc + static_cast<long long>(dst) * a.d);
      const float r = a.xs ? (g > 0.0f ? a.dloss[i] / g : a.dloss[i]) : 0.0f;   // g = 0: all zero (or not a number)
      auto put = [&](int v, uint4 u) {
        if (!in_bounds(a.err, static_cast<long long>(dst) * a.d + 8 * v, 8, n_el, SITE_HEAD_X)) return;
        to[v] = u;
        if (a.xs) {
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          uint32_t o[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            o[q] = pack_bf16(__uint_as_float(w[q] << 16) * r, __uint_as_float(w[q] & 0xffff0000u) * r);
          *reinterpret_cast<uint4*>(a.xs + static_cast<long long>(dst) * a.d + 8 * v) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      };
      int v = lane;
      if (i == r0 + warp) {
#pragma unroll
        for (int q = 0; q < PRE; ++q, v += 32)
          if (v < nv) put(v, pre[q]);
      }
      for (; v < nv; v += 32) put(v, src[v]);
    }
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) *a.n_rows = all;
  // x' up to the next whole block of 64 rows is a factor of the sum over rows: zeros
  if (a.xs && blockIdx.x == gridDim.x - 1) {
    const int end = max((all + 63) / 64 * 64, 64);
    for (long long v = static_cast<long long>(all) * nv + threadIdx.x; v < static_cast<long long>(end) * nv;
         v += ROWS_THREADS)
      if (in_bounds(a.err, v * 8, 8, static_cast<long long>(a.m_pad) * a.d, SITE_HEAD_X))
        reinterpret_cast<uint4*>(a.xs)[v] = make_uint4(0, 0, 0, 0);
  }
}

// Largest |dloss| of the rows that take part (one block).
__global__ void __launch_bounds__(1024) dloss_max_kernel(const __grid_constant__ RowsArgs a, float* g_max) {
  __shared__ float sm[32];
  grid_dependency_wait();
  grid_dependents_launch();
  float g = 0.0f;
  for (int i = threadIdx.x; i < a.M; i += 1024)
    if (row_state(a, i) == 1) g = fmaxf(g, fabsf(a.dloss[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = g;
  __syncthreads();
  if (threadIdx.x < 32) {
    g = sm[threadIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (threadIdx.x == 0) *g_max = g;
  }
}

// ---------------------------------------------------------------------------
// Row losses from the tiles' (max, sum): 32 rows a block, 32 interleaved slices of the column tiles.
// ---------------------------------------------------------------------------
struct FinishArgs {
  const int* n_rows;         // null (with row_src): every row of the call, those without a target too
  const int* row_src;
  const int64_t* labels;     // cross entropy, where every row is there
  int M, V, n_tiles, k;
  const float2* part;
  const float* part_sum;
  long long part_ld;
  const float* tgt_s;        // by compact row
  const float* tgt_p;        // by source row; null: cross entropy
  const int* tgt_cnt;
  float inv_t, scale_log2, temperature, smoothing;
  float* loss;
  float* lse;
  uint32_t* err;
};

__global__ void __launch_bounds__(FIN_ROWS* FIN_SLICES) head_finish_kernel(const __grid_constant__ FinishArgs a) {
  __shared__ float sm[3][FIN_SLICES][FIN_ROWS + 1];
  __shared__ float row_lse[FIN_ROWS];
  const int rx = threadIdx.x & 31, sl = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_dependents_launch();
  const int n = a.n_rows ? min(max(*a.n_rows, 0), a.M) : a.M;
  for (int r0 = blockIdx.x * FIN_ROWS; r0 < n; r0 += gridDim.x * FIN_ROWS) {
    const int row = r0 + rx;
    const bool on = row < n;
    float m = -INFINITY, l = 0.0f, s = 0.0f;
    // what the row's last step needs, asked for before the tiles' values; distillation: this warp's row of it
    const int tr = r0 + sl;
    int t_src = tr, t_cnt = 0;
    if (a.tgt_p && tr < n && in_bounds(a.err, tr, 1, a.M, SITE_HEAD_ROWS)) {
      if (a.row_src) t_src = a.row_src[tr];
      if (in_bounds(a.err, t_src, 1, a.M, SITE_HEAD_ROWS)) t_cnt = a.tgt_cnt[t_src];
    }
    int src = row, state = 1;
    float sy = 0.0f;
    if (sl == 0 && on && in_bounds(a.err, row, 1, a.M, SITE_HEAD_ROWS)) {
      if (a.row_src) src = a.row_src[row];
      else state = target_state(a.labels, a.tgt_cnt, a.V, row);
      if (!a.tgt_p) sy = a.tgt_s[row];
    }
    if (on) {
#pragma unroll 8
      for (int t = sl; t < a.n_tiles; t += FIN_SLICES) {
        const long long i = static_cast<long long>(t) * a.part_ld + row;
        if (!in_bounds(a.err, i, 1, static_cast<long long>(a.n_tiles) * a.part_ld, SITE_HEAD_PART)) continue;
        const float2 q = a.part[i];
        const float mn = fmaxf(m, q.x), mo = mn == -INFINITY ? 0.0f : mn;
        l = l * exp2f((m - mo) * a.scale_log2) + q.y * exp2f((q.x - mo) * a.scale_log2);
        m = mn;
        if (a.part_sum) s += a.part_sum[i];
      }
    }
    sm[0][sl][rx] = m;
    sm[1][sl][rx] = l;
    sm[2][sl][rx] = s;
    __syncthreads();
    if (sl == 0 && on) {
#pragma unroll
      for (int q = 1; q < FIN_SLICES; ++q) m = fmaxf(m, sm[0][q][rx]);
      const float mo = m == -INFINITY ? 0.0f : m;
      l = 0.0f;
      s = 0.0f;
#pragma unroll
      for (int q = 0; q < FIN_SLICES; ++q) {
        l += sm[1][q][rx] * exp2f((sm[0][q][rx] - mo) * a.scale_log2);
        s += sm[2][q][rx];
      }
      const float lse = fmaf(mo, a.inv_t, logf(l));
      row_lse[rx] = lse;
      if (in_bounds(a.err, src, 1, a.M, SITE_HEAD_ROWS)) {
        a.lse[src] = state == 1 ? lse : 0.0f;
        if (state != 1) {
          a.loss[src] = state == 0 ? 0.0f : __int_as_float(0x7fc00000);
        } else if (!a.tgt_p) {
          a.loss[src] = a.smoothing > 0.0f
                            ? (1.0f - a.smoothing) * (lse - sy) + a.smoothing * (lse - s / static_cast<float>(a.V))
                            : lse - sy;
        }
      }
    }
    __syncthreads();
    static_assert(FIN_ROWS == FIN_SLICES, "a warp a row");
    if (a.tgt_p) {       // distillation: a warp per row over its entries
      const float lse = row_lse[sl];
      float t = 0.0f;
      for (int j = rx; j < t_cnt; j += 32) {
        const long long i = static_cast<long long>(t_src) * a.k + j, is = static_cast<long long>(tr) * a.k + j;
        if (!in_bounds(a.err, i, 1, static_cast<long long>(a.M) * a.k, SITE_HEAD_TARGET)) continue;
        const float p = a.tgt_p[i];
        t += p * (logf(p) - a.tgt_s[is] * a.inv_t + lse);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (rx == 0 && t_cnt > 0) a.loss[t_src] = t * a.temperature * a.temperature;   // T^2 alone may be out of range
      __syncthreads();
    }
  }
}

// dx of the rows that take part: the slabs' sum times T dloss, rounded once.  `lanes` (1 to 8) threads
// share a vector of 8 columns, each adding every lanes-th slab; their sums are added in order.
__global__ void __launch_bounds__(256)
    head_dx_kernel(const int* __restrict__ n_rows, const int* __restrict__ row_src, int M, int m_pad, int d, int splits, int lanes,
                   const float* __restrict__ slab, const float* __restrict__ dloss, float temperature,
                   __nv_bfloat16* __restrict__ dx, uint32_t* err) {
  __shared__ float sm[256][8];
  grid_dependency_wait();
  grid_dependents_launch();
  const int n = min(max(*n_rows, 0), M);
  const int nv = d / 8, per_block = 256 / lanes;
  const long long per_slab = static_cast<long long>(m_pad) * d;
  const long long work = static_cast<long long>(n) * nv;
  const int vx = threadIdx.x % per_block, sl = threadIdx.x / per_block;
  for (long long w0 = static_cast<long long>(blockIdx.x) * per_block; w0 < work;
       w0 += static_cast<long long>(gridDim.x) * per_block) {
    const long long w = w0 + vx;
    const bool on = w < work;
    const int row = on ? static_cast<int>(w / nv) : 0, v = on ? static_cast<int>(w % nv) : 0;
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    int src = 0;
    float f = 0.0f;
    if (on && sl == 0) {
      src = row_src[row];
      if (in_bounds(err, src, 1, M, SITE_HEAD_ROWS)) f = dloss[src] * temperature;
    }
    if (on) {
#pragma unroll 4
      for (int q = sl; q < splits; q += lanes) {
        const long long i = q * per_slab + static_cast<long long>(row) * d + 8 * v;
        if (!in_bounds(err, i, 8, splits * per_slab, SITE_HEAD_SLAB)) continue;
        const float4 a = *reinterpret_cast<const float4*>(slab + i), b = *reinterpret_cast<const float4*>(slab + i + 4);
        s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
        s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
      }
    }
    if (lanes > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) sm[threadIdx.x][j] = s[j];
      __syncthreads();
      if (sl != 0) continue;
      for (int q = 1; q < lanes; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += sm[q * per_block + vx][j];
    }
    if (!on) continue;
    const long long o = static_cast<long long>(src) * d + 8 * v;
    if (in_bounds(err, o, 8, static_cast<long long>(M) * d, SITE_HEAD_DX))
      *reinterpret_cast<uint4*>(dx + o) = make_uint4(pack_bf16(s[0] * f, s[1] * f), pack_bf16(s[2] * f, s[3] * f),
                                                     pack_bf16(s[4] * f, s[5] * f), pack_bf16(s[6] * f, s[7] * f));
  }
}

// ------------------------------ host side ------------------------------
int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

struct HeadShape {
  int M, d, V, k;              // k = 0: cross entropy
  bool pair;                   // the pair form of the products
  int entries() const { return k > 0 ? k : 1; }
  int bm() const { return head_bm(pair); }
  int slots() const { return pair ? HEAD_SMS / 2 : HEAD_SMS; }   // tiles at a time
  int row_tiles() const { return ceil_div(M, bm()); }
  // rows of the workspace's matrices: whole tiles, so that no load of theirs runs past the end (filling rows
  // that are not there is slow: 17 rows against 51866 x 1280 took 43 us with boxes of 128 rows, 33 with 24)
  int m_pad() const { return row_tiles() * bm(); }
  int a_rows() const { return M < 128 ? (M + 7) / 8 * 8 : 128; }
  // one tile of rows: taking out rows saves no product, so the forward pass reads x as it is
  bool direct() const { return row_tiles() <= 1; }
  // a few rows: w straight to registers (head_gemv.cuh)
  bool gemv() const { return M <= GEMV_MAX_M && d <= GEMV_MAX_D; }
};

// The pair form wins where there are rows for it and, forward, where a tile's k is long.  Device time of the
// pair and the single form against 51866 entries, us: forward, d = 1280: 64 rows 35 / 32, 448 rows 57 / 62,
// 14336 rows 1030 / 1128; d = 384: 448 rows 29 / 27, 14336 rows 415 / 374.  Backward, d = 1280: 64 rows
// 101 / 87, 200 rows 117 / 123, 1500 rows 387 / 451; d = 384: 64 rows 47 / 38, 448 rows 77 / 85, 14336 rows
// 1556 / 1649.
HeadShape fwd_shape(int M, int d, int V, int k) { return HeadShape{M, d, V, k, M > 128 && d >= 768}; }
HeadShape bwd_shape(int M, int d, int V, int k) { return HeadShape{M, d, V, k, M > 128}; }

bool shape_ok(int M, int d, int V) {
  return M >= 0 && M <= (1 << 24) && d >= 8 && d <= (1 << 16) && d % 8 == 0 && V >= 1 && V <= (1 << 24);
}

// Column-tile width of the products x w^T: the one whose rounds of tiles over the device end first.  A tile
// costs about 100 columns on top of its own (a stage's round trip through the ring bounds narrow tiles):
// measured at 1500 rows of 1280, 256 / 192 / 128 / 64 columns 127 / 148 / 208 / 383 us.  So 256 nearly always;
// 192 where it takes as few rounds (one tile of rows, 51866 entries: 31.5 us against 34.7).
int logits_width(const HeadShape& h, int vc) {
  int best = HEAD_BN;
  long long cost = -1;
  for (int bn = HEAD_BN; bn >= 64; bn -= 32) {
    const long long tiles = static_cast<long long>(h.row_tiles()) * ceil_div(vc, bn);
    const long long c = (tiles + h.slots() - 1) / h.slots() * (bn + 100);
    if (cost < 0 || c < cost) {
      cost = c;
      best = bn;
    }
  }
  return best;
}

// Column-tile width of the gradient products: the fewest columns past d (384 = 2 x 192).
int grad_width(int d) {
  int best = HEAD_BN;
  for (int bn = HEAD_BN; bn >= 128; bn -= 64)
    if (ceil_div(d, bn) * bn < ceil_div(d, best) * best) best = bn;
  return best;
}

// Targets and row map, shared by both passes.
struct RowsLayout {
  size_t n_rows, row_src, row_tgt, row_cnt, row_lse, idx, p, cnt, xc;
};

RowsLayout rows_layout(Carver& c, const HeadShape& h) {
  RowsLayout L;
  const size_t m = static_cast<size_t>(h.M);
  L.n_rows = c.take(256);
  L.row_src = c.take(m * sizeof(int));
  L.row_lse = c.take(m * sizeof(float));
  L.row_tgt = L.row_cnt = L.idx = L.p = L.cnt = 0;
  if (h.k > 0) {
    L.row_cnt = c.take(m * sizeof(int));
    L.idx = c.take(m * h.k * sizeof(int));
    L.p = c.take(m * h.k * sizeof(float));
    L.cnt = c.take(m * sizeof(int));
  } else {
    L.row_tgt = c.take(m * sizeof(int));
  }
  L.xc = c.take(static_cast<size_t>(h.m_pad()) * h.d * 2);
  return L;
}

struct FwdLayout {
  RowsLayout r;
  size_t part, part_sum, tgt_s, total;
  long long part_ld;
  int bn, n_tiles;
};

FwdLayout fwd_layout(const HeadShape& h) {
  Carver c;
  FwdLayout L;
  L.r = rows_layout(c, h);
  L.part_ld = (static_cast<long long>(h.M) + 31) / 32 * 32;
  L.bn = logits_width(h, h.V);
  L.n_tiles = h.gemv() ? HEAD_SMS : ceil_div(h.V, L.bn);
  L.part = c.take(static_cast<size_t>(L.n_tiles) * L.part_ld * sizeof(float2));
  L.part_sum = h.k > 0 ? 0 : c.take(static_cast<size_t>(L.n_tiles) * L.part_ld * sizeof(float));
  L.tgt_s = c.take(static_cast<size_t>(h.M) * h.entries() * sizeof(float));
  L.total = c.off;
  return L;
}

struct BwdLayout {
  RowsLayout r;
  size_t g_max, xs, dl, slab, total;
  int bn;                      // column-tile width of the logits
  int piece, splits;           // vocabulary rows per piece (a multiple of 256), slabs of dx
};

// A piece's D (whole tiles of rows) takes at most this much memory, or 256 columns: from 2^19 rows on 512 bytes a row.
constexpr long long PIECE_BYTES = 256ll << 20;

// Slabs of dx: where its tiles are too few for the device, the sum over the piece is split.
int dx_splits(const HeadShape& h, int piece) {
  const long long tiles = static_cast<long long>(h.row_tiles()) * ceil_div(h.d, grad_width(h.d));
  const int kb = piece / HEAD_BK;
  long long s = h.slots() / tiles;
  if (s > kb / 8) s = kb / 8;
  return s < 1 ? 1 : static_cast<int>(s);
}

// Time of the products of one piece of vc rows, in blocks of 64 along k of a whole tile (about a quarter
// of a microsecond): tiles go round the SMs (or pairs), so each product lasts as long as the fullest.
long long piece_cost(const HeadShape& h, int vc, int splits) {
  const int kb_d = ceil_div(h.d, HEAD_BK), kb_v = ceil_div(vc, HEAD_BK), kb_n = ceil_div(h.M, HEAD_BK);
  const long long rt = h.row_tiles(), dt = ceil_div(h.d, grad_width(h.d)), slots = h.slots();
  const long long logits = (rt * ceil_div(vc, HEAD_BN) + slots - 1) / slots * (kb_d + 4);
  const long long dw = ceil_div(vc, h.bm()) * dt, all = dw + rt * dt * splits;
  long long grads = 0;
  for (int c = 0; c < slots && c < all; ++c) {
    const long long mine = (all - 1 - c) / slots + 1, mine_dw = c < dw ? (dw - 1 - c) / slots + 1 : 0;
    const long long t = mine_dw * (kb_n + 4) + (mine - mine_dw) * (ceil_div(kb_v, splits) + 4);
    if (t > grads) grads = t;
  }
  return logits + grads + 64;                  // two launches: 16 us, measured best of 8, 16, 32 and 64
}

BwdLayout bwd_layout(const HeadShape& h) {
  Carver c;
  BwdLayout L;
  L.r = rows_layout(c, h);
  const long long v256 = (static_cast<long long>(h.V) + 255) / 256 * 256;
  long long most = PIECE_BYTES / (2ll * h.m_pad()) / 256 * 256;
  if (most < 256) most = 256;
  if (most > v256) most = v256;
  // equal pieces, as many as leave the fewest idle SMs: 14336 rows of 1280, a quarter padding, both
  // directions, 3.60 ms against 3.75 with the largest pieces
  L.piece = static_cast<int>(most);
  if (most < v256) {
    const int fewest = ceil_div(v256, most);
    long long best = -1;
    for (int pieces = fewest; pieces <= fewest + 8 && pieces * 256ll <= v256; ++pieces) {
      const int vc = ceil_div(ceil_div(h.V, pieces), 256) * 256;
      const int last = h.V - (ceil_div(h.V, vc) - 1) * vc;
      const long long t = (ceil_div(h.V, vc) - 1) * piece_cost(h, vc, 1) + piece_cost(h, last, 1);
      if (best < 0 || t < best) {
        best = t;
        L.piece = vc;
      }
    }
  }
  L.splits = dx_splits(h, L.piece);
  L.bn = logits_width(h, L.piece) / 64 * 64;     // whole staging boxes; past the piece the store is clipped
  const size_t m = static_cast<size_t>(h.m_pad());
  L.g_max = c.take(256);
  L.xs = c.take(m * h.d * 2);
  L.dl = c.take(m * static_cast<size_t>(most) * 2);
  L.slab = c.take(static_cast<size_t>(L.splits) * m * h.d * sizeof(float));
  L.total = c.off;
  return L;
}

bool map2(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint64_t ld, uint32_t bx, uint32_t by) {
  const uint64_t dims[2] = {inner, rows};
  const uint64_t str[1] = {ld * 2};
  const uint32_t box[2] = {bx, by};
  return tma_map_bf16(m, 2, base, dims, str, box);
}

std::mutex g_head_mu;

template <int KIND, bool PAIR>
cudaError_t launch_form(const HeadMaps& maps, const HeadParams& p, cudaStream_t s) {
  static uint64_t attr_done = 0;
  constexpr int SMEM = HeadSmem<KIND, PAIR>::TOTAL;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    // once per device, so that launches stay legal inside a graph capture
    std::lock_guard<std::mutex> lk(g_head_mu);
    if (dev < 0 || dev > 63) return cudaErrorInvalidDevice;
    if (!(attr_done & (1ull << dev))) {
      e = cudaFuncSetAttribute(head_gemm_kernel<KIND, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
      if (e != cudaSuccess) return e;
      attr_done |= 1ull << dev;
    }
  }
  constexpr int BM = head_bm(PAIR), CTAS = PAIR ? 2 : 1;
  const long long rows = ceil_div(p.m_cap, BM), dn = ceil_div(p.d, p.bn);
  const long long tiles = KIND != HEAD_GRADS ? rows * ceil_div(p.vc, p.bn)
                                             : (p.want_dw ? ceil_div(p.vc, BM) * dn : 0) + rows * dn * p.dx_splits;
  long long slots = sm_count() / CTAS;
  if (slots < 1) slots = 1;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(CTAS * (tiles < slots ? tiles : slots)));
  cfg.blockDim = dim3(GEMM_THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, head_gemm_kernel<KIND, PAIR>, maps, p);
}
template <int KIND>
cudaError_t launch_head(const HeadShape& h, const HeadMaps& maps, const HeadParams& p, cudaStream_t s) {
  return h.pair ? launch_form<KIND, true>(maps, p, s) : launch_form<KIND, false>(maps, p, s);
}

template <int MT>
cudaError_t launch_gemv(const GemvParams& p, int blocks, cudaStream_t s) {
  static uint64_t attr_done = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lk(g_head_mu);
    if (dev < 0 || dev > 63) return cudaErrorInvalidDevice;
    if (!(attr_done & (1ull << dev))) {
      e = cudaFuncSetAttribute(head_gemv_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               8 * MT * gemv_row_bytes(GEMV_MAX_D));
      if (e != cudaSuccess) return e;
      attr_done |= 1ull << dev;
    }
  }
  return launch_pdl(head_gemv_kernel<MT>, dim3(blocks), dim3(GEMV_WARPS * 32),
                    static_cast<size_t>(8 * MT) * gemv_row_bytes(p.d), s, p);
}

struct Targets {
  const int64_t* labels;       // cross entropy
  float smoothing;
  const void* top;             // distillation
  int top_type;
  const int64_t* index;
  float temperature;
};

cudaError_t launch_lists(const HeadShape& h, const Targets& t, int* idx, float* p, int* cnt, uint32_t* err,
                         cudaStream_t s) {
  const size_t smem = static_cast<size_t>((h.k + 3) & ~3) * 12;
  const float inv_t = 1.0f / t.temperature;
  const dim3 grid(h.M), block(LIST_THREADS);
  if (t.top_type == WB_F32)
    return launch_pdl(target_lists_kernel<float>, grid, block, smem, s, static_cast<const float*>(t.top), t.index, h.M,
                      h.k, h.V, inv_t, idx, p, cnt, err);
  if (t.top_type == WB_BF16)
    return launch_pdl(target_lists_kernel<__nv_bfloat16>, grid, block, smem, s,
                      static_cast<const __nv_bfloat16*>(t.top), t.index, h.M, h.k, h.V, inv_t, idx, p, cnt, err);
  return launch_pdl(target_lists_kernel<__half>, grid, block, smem, s, static_cast<const __half*>(t.top), t.index, h.M,
                    h.k, h.V, inv_t, idx, p, cnt, err);
}

// Fewer rows a block while there are few (the copy wants many blocks); each block counts the rows
// before its own, M / 2 labels on average, so at most 1216 of them (blocks of 256 rows, as many as it takes:
// 2^24 rows of 8 forward 226 ms against 13.4, 2^20 rows 1.17 against 0.69).
int rows_per_block(int M) {
  int r = 8;
  while (M > 1216 * r) r *= 2;
  return r;
}

struct HeadBase {
  HeadShape h;
  uint8_t* ws;
  uint32_t* err;
  const int* row_src;
  const int* n_rows;
  int* row_tgt;                // cross entropy
  int* row_cnt;                // distillation, and the lists by source row
  float* row_lse;
  int* tgt_idx;
  float* tgt_p;
  int* tgt_cnt;
  __nv_bfloat16* xc;
};

HeadParams head_params(const HeadBase& b, const Targets& t) {
  HeadParams p = {};
  p.n_rows = b.n_rows;
  p.m_cap = b.h.M;
  p.V = b.h.V;
  p.d = b.h.d;
  p.vc = b.h.V;
  p.bn = HEAD_BN;
  p.a_rows = b.h.a_rows();
  p.panel = 8;
  p.scale_log2 = 1.4426950408889634f / t.temperature;
  p.inv_t = 1.0f / t.temperature;
  p.row_tgt = b.h.k > 0 ? b.row_src : b.row_tgt;
  p.row_cnt = b.row_cnt;
  p.tgt_idx = b.tgt_idx;
  p.tgt_p = b.tgt_p;
  p.k = b.h.entries();
  p.label_p = 1.0f - t.smoothing;
  p.smooth = t.smoothing / static_cast<float>(b.h.V);
  p.err = b.err;
  return p;
}

HeadBase head_base(const HeadShape& h, uint8_t* ws, const RowsLayout& L, uint32_t* err) {
  HeadBase b;
  b.h = h;
  b.ws = ws;
  b.err = err;
  b.row_src = reinterpret_cast<int*>(ws + L.row_src);
  b.n_rows = reinterpret_cast<int*>(ws + L.n_rows);
  b.row_tgt = h.k > 0 ? nullptr : reinterpret_cast<int*>(ws + L.row_tgt);
  b.row_cnt = h.k > 0 ? reinterpret_cast<int*>(ws + L.row_cnt) : nullptr;
  b.row_lse = reinterpret_cast<float*>(ws + L.row_lse);
  b.tgt_idx = h.k > 0 ? reinterpret_cast<int*>(ws + L.idx) : nullptr;
  b.tgt_p = h.k > 0 ? reinterpret_cast<float*>(ws + L.p) : nullptr;
  b.tgt_cnt = h.k > 0 ? reinterpret_cast<int*>(ws + L.cnt) : nullptr;
  b.xc = reinterpret_cast<__nv_bfloat16*>(ws + L.xc);
  return b;
}

RowsArgs rows_args(const HeadBase& b, const Targets& t, const RowsLayout& L, const void* x) {
  RowsArgs a = {};
  a.labels = t.labels;
  a.cnt = b.tgt_cnt;
  a.M = b.h.M;
  a.V = b.h.V;
  a.d = b.h.d;
  a.rows_per_block = rows_per_block(b.h.M);
  a.m_pad = b.h.m_pad();
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.xc = b.xc;
  a.row_src = reinterpret_cast<int*>(b.ws + L.row_src);
  a.n_rows = reinterpret_cast<int*>(b.ws + L.n_rows);
  a.row_tgt = b.row_tgt;
  a.row_cnt = b.row_cnt;
  a.row_lse = b.row_lse;
  a.err = b.err;
  return a;
}

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t s) {
  return launch_pdl(rows_kernel, dim3((a.M + a.rows_per_block - 1) / a.rows_per_block), dim3(ROWS_THREADS), 0, s, a);
}

wb_status head_forward(const HeadShape& h, const Targets& t, const void* x, const void* w, float* loss, float* lse,
                       void* workspace, cudaStream_t s) {
  uint32_t* err = tc_err_ptr();
  if (!err) return WB_ECUDA;
  const FwdLayout L = fwd_layout(h);
  const HeadBase b = head_base(h, static_cast<uint8_t*>(workspace), L.r, err);
  const bool direct = h.direct();
  if (h.k > 0 || !direct) {
    Prof pr(PC_HEAD_ROWS, s, (h.k > 0) + !direct);
    if (h.k > 0) WB_CUDA(launch_lists(h, t, b.tgt_idx, b.tgt_p, b.tgt_cnt, err, s));
    if (!direct) {
      RowsArgs a = rows_args(b, t, L.r, x);
      a.loss = loss;
      a.lse = lse;
      WB_CUDA(launch_rows(a, s));
    }
  }
  int n_tiles = L.n_tiles;
  auto* part = reinterpret_cast<float2*>(b.ws + L.part);
  float* part_sum = t.smoothing > 0.0f ? reinterpret_cast<float*>(b.ws + L.part_sum) : nullptr;
  auto* tgt_s = reinterpret_cast<float*>(b.ws + L.tgt_s);
  if (h.gemv()) {
    GemvParams p = {};
    p.x = static_cast<const __nv_bfloat16*>(x);
    p.w = static_cast<const __nv_bfloat16*>(w);
    p.M = h.M;
    p.V = h.V;
    p.d = h.d;
    p.scale_log2 = 1.4426950408889634f / t.temperature;
    p.labels = t.labels;
    p.cnt = b.tgt_cnt;
    p.tgt_idx = b.tgt_idx;
    p.k = h.entries();
    p.part = part;
    p.part_sum = part_sum;
    p.part_ld = L.part_ld;
    p.tgt_s = tgt_s;
    p.err = err;
    const int groups = ceil_div(h.V, 16);
    n_tiles = groups < HEAD_SMS ? groups : HEAD_SMS;
    Prof pr(PC_HEAD_LSE, s);
    WB_CUDA(h.M <= 8 ? launch_gemv<1>(p, n_tiles, s) : launch_gemv<2>(p, n_tiles, s));
  } else {
    HeadParams p = head_params(b, t);
    if (direct) {
      p.n_rows = nullptr;
      p.labels = t.labels;
      p.row_tgt = nullptr;
      p.row_cnt = b.tgt_cnt;
    }
    p.part = part;
    p.part_sum = part_sum;
    p.part_ld = L.part_ld;
    p.tgt_s = tgt_s;
    p.bn = L.bn;
    HeadMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    if (!map2(&maps.a0, direct ? x : b.xc, h.d, direct ? h.M : h.m_pad(), h.d, HEAD_BK, h.a_rows()) ||
        !map2(&maps.b0, w, h.d, h.V, h.d, HEAD_BK, h.pair ? L.bn / 2 : L.bn))
      return WB_ECUDA;
    {
      Prof pr(PC_HEAD_LSE, s);
      WB_CUDA(launch_head<HEAD_LSE>(h, maps, p, s));
    }
  }
  FinishArgs f = {};
  f.n_rows = direct ? nullptr : b.n_rows;
  f.row_src = direct ? nullptr : b.row_src;
  f.labels = t.labels;
  f.M = h.M;
  f.V = h.V;
  f.n_tiles = n_tiles;
  f.k = h.entries();
  f.part = part;
  f.part_sum = part_sum;
  f.part_ld = L.part_ld;
  f.tgt_s = tgt_s;
  f.tgt_p = b.tgt_p;
  f.tgt_cnt = b.tgt_cnt;
  f.inv_t = 1.0f / t.temperature;
  f.scale_log2 = 1.4426950408889634f / t.temperature;
  f.temperature = t.temperature;
  f.smoothing = t.smoothing;
  f.loss = loss;
  f.lse = lse;
  f.err = err;
  {
    Prof pr(PC_HEAD_FINISH, s);
    const int blocks = (h.M + FIN_ROWS - 1) / FIN_ROWS;
    WB_CUDA(launch_pdl(head_finish_kernel, dim3(blocks < 1216 ? blocks : 1216), dim3(FIN_ROWS * FIN_SLICES), 0,
                       s, f));
  }
  return WB_OK;
}

wb_status head_backward(const HeadShape& h, const Targets& t, const float* dloss, const void* x, const void* w,
                        const float* lse, void* dx, void* dw, void* workspace, cudaStream_t s) {
  uint32_t* err = tc_err_ptr();
  if (!err) return WB_ECUDA;
  const BwdLayout L = bwd_layout(h);
  const HeadBase b = head_base(h, static_cast<uint8_t*>(workspace), L.r, err);
  auto* g_max = reinterpret_cast<float*>(b.ws + L.g_max);
  auto* xs = reinterpret_cast<__nv_bfloat16*>(b.ws + L.xs);
  auto* dl = reinterpret_cast<__nv_bfloat16*>(b.ws + L.dl);
  auto* slab = reinterpret_cast<float*>(b.ws + L.slab);
  {
    Prof pr(PC_HEAD_ROWS, s, (h.k > 0 ? 2 : 1) + (dw && h.M > OWN_MAX_ROWS ? 1 : 0));
    if (h.k > 0)
      WB_CUDA(launch_lists(h, t, b.tgt_idx, b.tgt_p, b.tgt_cnt, err, s));
    RowsArgs a = rows_args(b, t, L.r, x);
    a.dloss = dloss;
    a.lse_in = lse;
    a.g_max = g_max;
    a.own_max = h.M <= OWN_MAX_ROWS;
    a.xs = dw ? xs : nullptr;
    a.dx = static_cast<__nv_bfloat16*>(dx);
    if (dw && !a.own_max) WB_CUDA(launch_pdl(dloss_max_kernel, dim3(1), dim3(1024), 0, s, a, g_max));
    WB_CUDA(launch_rows(a, s));
  }
  HeadParams p = head_params(b, t);
  p.dl_cols = L.piece;
  p.row_lse = b.row_lse;
  p.g_scale = g_max;
  p.out_scale = t.temperature;
  p.dx_splits = dx ? L.splits : 0;
  p.want_dw = dw != nullptr;
  HeadMaps lm, gm;
  std::memset(&lm, 0, sizeof(lm));
  std::memset(&gm, 0, sizeof(gm));
  const uint64_t ld = L.piece, mp = h.m_pad();
  bool ok = map2(&lm.a0, b.xc, h.d, mp, h.d, HEAD_BK, h.a_rows()) &&
            map2(&lm.b0, w, h.d, h.V, h.d, HEAD_BK, h.pair ? L.bn / 2 : L.bn) &&
            map2(&lm.o0, dl, ld, mp, ld, 64, 32);
  if (dx) {
    const uint64_t dims[3] = {static_cast<uint64_t>(h.d), mp, static_cast<uint64_t>(L.splits)};
    const uint64_t str[2] = {static_cast<uint64_t>(h.d) * 4, static_cast<uint64_t>(h.d) * 4 * mp};
    const uint32_t box[3] = {32, 32, 1};
    ok = ok && map2(&gm.a0, dl, ld, mp, ld, HEAD_BK, h.a_rows()) && map2(&gm.b0, w, h.d, h.V, h.d, 64, HEAD_BK) &&
         tma_map_f32(&gm.o0, 3, slab, dims, str, box);
  }
  if (dw)
    ok = ok && map2(&gm.a1, dl, ld, mp, ld, 64, HEAD_BK) && map2(&gm.b1, xs, h.d, mp, h.d, 64, HEAD_BK) &&
         map2(&gm.o1, dw, h.d, h.V, h.d, 64, 32);
  if (!ok) return WB_ECUDA;
  for (int v0 = 0; v0 < h.V; v0 += L.piece) {
    p.v0 = v0;
    p.vc = h.V - v0 < L.piece ? h.V - v0 : L.piece;
    p.first_piece = v0 == 0;
    p.bn = L.bn;
    {
      Prof pr(PC_HEAD_DLOGITS, s);
      WB_CUDA(launch_head<HEAD_DLOGITS>(h, lm, p, s));
    }
    p.bn = grad_width(h.d);
    Prof pr(PC_HEAD_GRADS, s);
    WB_CUDA(launch_head<HEAD_GRADS>(h, gm, p, s));
  }
  if (dx) {
    Prof pr(PC_HEAD_FINISH, s);
    const int lanes = L.splits >= 8 ? 8 : L.splits >= 4 ? 4 : L.splits >= 2 ? 2 : 1;
    const long long work = static_cast<long long>(h.M) * (h.d / 8) * lanes;
    const long long blocks = (work + 255) / 256;
    WB_CUDA(launch_pdl(head_dx_kernel, dim3(static_cast<unsigned>(blocks < 2432 ? blocks : 2432)), dim3(256), 0, s,
                       b.n_rows, b.row_src, h.M, h.m_pad(), h.d, L.splits, lanes, static_cast<const float*>(slab), dloss,
                       t.temperature, static_cast<__nv_bfloat16*>(dx), err));
  }
  return WB_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

wb_status check_forward(const HeadShape& h, const void* x, const void* w, const float* loss, const float* lse,
                        const void* ws, size_t ws_bytes) {
  if (!x || !w || !loss || !lse || !aligned16(x) || !aligned16(w) || !aligned4(loss) || !aligned4(lse))
    return WB_EINVAL;
  if (!ws || !aligned16(ws) || ws_bytes < fwd_layout(h).total) return WB_EWORKSPACE;
  return WB_OK;
}

wb_status check_backward(const HeadShape& h, const float* dloss, const void* x, const void* w, const float* lse,
                         const void* dx, const void* dw, const void* ws, size_t ws_bytes) {
  if (!dloss || !x || !w || !lse || !aligned16(x) || !aligned16(w) || !aligned4(dloss) || !aligned4(lse) ||
      (dx && !aligned16(dx)) || (dw && !aligned16(dw)) || dx == x || dw == w)
    return WB_EINVAL;
  if (!ws || !aligned16(ws) || ws_bytes < bwd_layout(h).total) return WB_EWORKSPACE;
  return WB_OK;
}

bool top_aligned(const void* p, int type) { return (reinterpret_cast<uintptr_t>(p) & (type == WB_F32 ? 3u : 1u)) == 0; }
bool top_ok(int type) { return type == WB_BF16 || type == WB_F16 || type == WB_F32; }
// From the smallest normal value on: below, 1 / T is not finite.
bool temperature_ok(float t) { return t >= FLT_MIN && t < INFINITY; }

}  // namespace
}  // namespace wb

using namespace wb;

extern "C" {

size_t wb_linear_cross_entropy_workspace_bytes(int M, int d, int V) {
  return shape_ok(M, d, V) && M > 0 ? fwd_layout(fwd_shape(M, d, V, 0)).total : 0;
}
size_t wb_linear_cross_entropy_backward_workspace_bytes(int M, int d, int V) {
  return shape_ok(M, d, V) && M > 0 ? bwd_layout(bwd_shape(M, d, V, 0)).total : 0;
}
size_t wb_linear_distill_workspace_bytes(int M, int d, int V, int k) {
  return shape_ok(M, d, V) && M > 0 && k >= 1 && k <= HEAD_MAX_K ? fwd_layout(fwd_shape(M, d, V, k)).total : 0;
}
size_t wb_linear_distill_backward_workspace_bytes(int M, int d, int V, int k) {
  return shape_ok(M, d, V) && M > 0 && k >= 1 && k <= HEAD_MAX_K ? bwd_layout(bwd_shape(M, d, V, k)).total : 0;
}

wb_status wb_linear_cross_entropy(const void* x, const void* w, const int64_t* labels, int M, int d, int V,
                                  float label_smoothing, float* loss, float* lse, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!shape_ok(M, d, V) || !(label_smoothing >= 0.0f && label_smoothing < 1.0f)) return WB_EINVAL;
  if (M == 0) return WB_OK;
  if (!labels || !aligned8(labels)) return WB_EINVAL;
  const HeadShape h = fwd_shape(M, d, V, 0);
  const wb_status st = check_forward(h, x, w, loss, lse, workspace, workspace_bytes);
  if (st != WB_OK) return st;
  const Targets t{labels, label_smoothing, nullptr, 0, nullptr, 1.0f};
  return head_forward(h, t, x, w, loss, lse, workspace, static_cast<cudaStream_t>(stream));
}

wb_status wb_linear_cross_entropy_backward(const float* dloss, const void* x, const void* w, const int64_t* labels,
                                           const float* lse, int M, int d, int V, float label_smoothing, void* dx,
                                           void* dw, void* workspace, size_t workspace_bytes, void* stream) {
  if (!shape_ok(M, d, V) || !(label_smoothing >= 0.0f && label_smoothing < 1.0f)) return WB_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (dw && !aligned16(dw)) return WB_EINVAL;
    if (dw) WB_CUDA(cudaMemsetAsync(dw, 0, static_cast<size_t>(V) * d * 2, s));
    return WB_OK;
  }
  if (!labels || !aligned8(labels)) return WB_EINVAL;
  const HeadShape h = bwd_shape(M, d, V, 0);
  const wb_status st = check_backward(h, dloss, x, w, lse, dx, dw, workspace, workspace_bytes);
  if (st != WB_OK) return st;
  if (!dx && !dw) return WB_OK;
  const Targets t{labels, label_smoothing, nullptr, 0, nullptr, 1.0f};
  return head_backward(h, t, dloss, x, w, lse, dx, dw, workspace, s);
}

wb_status wb_linear_distill(const void* x, const void* w, const void* top, int top_dtype, const int64_t* index, int M,
                            int d, int V, int k, float temperature, float* loss, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!top_ok(top_dtype)) return WB_EUNSUPPORTED;
  if (!shape_ok(M, d, V) || k < 1 || k > HEAD_MAX_K || !temperature_ok(temperature)) return WB_EINVAL;
  if (M == 0) return WB_OK;
  if (!top || !index || !top_aligned(top, top_dtype) || !aligned8(index)) return WB_EINVAL;
  const HeadShape h = fwd_shape(M, d, V, k);
  const wb_status st = check_forward(h, x, w, loss, lse, workspace, workspace_bytes);
  if (st != WB_OK) return st;
  const Targets t{nullptr, 0.0f, top, top_dtype, index, temperature};
  return head_forward(h, t, x, w, loss, lse, workspace, static_cast<cudaStream_t>(stream));
}

wb_status wb_linear_distill_backward(const float* dloss, const void* x, const void* w, const void* top, int top_dtype,
                                     const int64_t* index, const float* lse, int M, int d, int V, int k,
                                     float temperature, void* dx, void* dw, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  if (!top_ok(top_dtype)) return WB_EUNSUPPORTED;
  if (!shape_ok(M, d, V) || k < 1 || k > HEAD_MAX_K || !temperature_ok(temperature)) return WB_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (dw && !aligned16(dw)) return WB_EINVAL;
    if (dw) WB_CUDA(cudaMemsetAsync(dw, 0, static_cast<size_t>(V) * d * 2, s));
    return WB_OK;
  }
  if (!top || !index || !top_aligned(top, top_dtype) || !aligned8(index)) return WB_EINVAL;
  const HeadShape h = bwd_shape(M, d, V, k);
  const wb_status st = check_backward(h, dloss, x, w, lse, dx, dw, workspace, workspace_bytes);
  if (st != WB_OK) return st;
  if (!dx && !dw) return WB_OK;
  const Targets t{nullptr, 0.0f, top, top_dtype, index, temperature};
  return head_backward(h, t, dloss, x, w, lse, dx, dw, workspace, s);
}

}  // extern "C"
