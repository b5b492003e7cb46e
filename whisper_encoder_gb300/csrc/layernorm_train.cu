// LayerNorm for training: the forward pass that keeps its row statistics, and the backward pass with
// the reduction of the weight's and the bias's gradient.  Any width up to 10240, bf16 / f16 / f32.
//
//   t = round(x + r), mu = mean(t), rs = 1 / sqrt(mean((t - mu)^2) + eps), y = (t - mu) rs g + b
//   h = (t - mu) rs, u = g dy:
//   dx = rs (u - mean(u) - h mean(u h)) (+ dt),  dg = sum_rows dy h,  db = sum_rows dy
//
// Both passes are bound by memory: each element is read once and written once.  A team of W warps
// (1, 2, 4 or 8, by the width) holds one row in registers, at most 40 elements a lane, so the row
// statistics take their two passes over registers; the statistics, the row sums and the sums over
// rows are fp32.  The backward pass keeps each lane's columns of dg and db in registers over all the
// rows that its team takes (team-strided), adds the teams of a block in shared memory in a fixed
// order and leaves one partial row per block, which a second kernel adds in block order: no
// atomics, the same result every time.
#include "../../include/wb.h"
#include "internal.h"
#include "ptx.cuh"

namespace wb {
namespace {

constexpr int LNT_MAX_D = 10240;
constexpr int LNT_FWD_BLOCKS = 152 * 8;   // grid caps; the partial rows of the backward pass are bounded by the second
constexpr int LNT_BWD_BLOCKS = 152 * 3;
constexpr int COL_SLICES = 16;            // column-sum kernel: slices of the partial rows per block

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }

// VEC elements of T as one load: 16 bytes, or a single element where no vector divides the width.
template <typename T, int VEC>
struct Pack {
  struct alignas(VEC * sizeof(T)) Raw {
    T e[VEC];
  };
};

// VEC consecutive gamma / beta values.
template <int VEC>
__device__ __forceinline__ void load_params(const float* p, float (&o)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p) + j);
      o[4 * j] = f.x; o[4 * j + 1] = f.y; o[4 * j + 2] = f.z; o[4 * j + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = __ldg(p + j);
  }
}

// Sum of (a, b) over the W warps of a team; every thread of the team gets it.  `slot` alternates
// between calls: between two uses of a slot lies another call's barrier, which a warp reaches only
// after it has read this one.
template <int W>
__device__ __forceinline__ float2 team_sum(float a, float b, float2 (*red)[W], int team, int warp_in_team, int lane,
                                           int slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if (W == 1) return make_float2(a, b);
  if (lane == 0) red[slot][warp_in_team] = make_float2(a, b);
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(W * 32) : "memory");
  a = b = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    a += red[slot][i].x;
    b += red[slot][i].y;
  }
  return make_float2(a, b);
}

constexpr int lnt_warps(int W) { return W < 4 ? 4 : W; }   // warps per block: one to four teams

template <typename T, int VEC, int NV, int W>
__global__ void __launch_bounds__(lnt_warps(W) * 32)
    ln_train_fwd_kernel(const T* __restrict__ x, const T* __restrict__ res, const float* __restrict__ g,
                        const float* __restrict__ bta, int rows, int d, float eps, T* __restrict__ y,
                        T* __restrict__ total, float2* __restrict__ stats, uint32_t* err) {
  constexpr int TEAMS = lnt_warps(W) / W;
  using Raw = typename Pack<T, VEC>::Raw;
  __shared__ float2 red[TEAMS][2][W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / W, wt = warp % W;
  const long long n_el = static_cast<long long>(rows) * d;
  const float inv_d = 1.0f / static_cast<float>(d);
  grid_dependency_wait();
  grid_dependents_launch();
  for (long long row = static_cast<long long>(blockIdx.x) * TEAMS + team; row < rows;
       row += static_cast<long long>(gridDim.x) * TEAMS) {
    const long long base = row * d;
    Raw u[NV], r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = ((i * W + wt) * 32 + lane) * VEC;
      if (col < d && in_bounds(err, base + col, VEC, n_el, SITE_LNT_X)) {
        u[i] = *reinterpret_cast<const Raw*>(x + base + col);
        if (res) r[i] = *reinterpret_cast<const Raw*>(res + base + col);
      }
    }
    float v[NV * VEC];
    float sm = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = ((i * W + wt) * 32 + lane) * VEC;
      const bool on = col < d;
      if (on && res) {
        // the sum is rounded to the tensor's type first: what is normalised is what is stored
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[i].e[j] = from_f32<T>(to_f32<T>(u[i].e[j]) + to_f32<T>(r[i].e[j]));
        if (total && in_bounds(err, base + col, VEC, n_el, SITE_LNT_TOTAL))
          *reinterpret_cast<Raw*>(total + base + col) = u[i];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i * VEC + j] = on ? to_f32<T>(u[i].e[j]) : 0.0f;
        sm += v[i * VEC + j];
      }
    }
    const float mean = team_sum<W>(sm, 0.0f, red[team], team, wt, lane, 0).x * inv_d;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool on = ((i * W + wt) * 32 + lane) * VEC < d;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float t = v[i * VEC + j] - mean;
        q += on ? t * t : 0.0f;
      }
    }
    const float rstd = rsqrtf(team_sum<W>(q, 0.0f, red[team], team, wt, lane, 1).x * inv_d + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = ((i * W + wt) * 32 + lane) * VEC;
      if (col >= d || !in_bounds(err, base + col, VEC, n_el, SITE_LNT_Y)) continue;
      float gg[VEC], bb[VEC];
      load_params<VEC>(g + col, gg);
      load_params<VEC>(bta + col, bb);
      Raw o;
#pragma unroll
      for (int j = 0; j < VEC; ++j) o.e[j] = from_f32<T>(fmaf((v[i * VEC + j] - mean) * rstd, gg[j], bb[j]));
      *reinterpret_cast<Raw*>(y + base + col) = o;
    }
    if (wt == 0 && lane == 0 && in_bounds(err, row, 1, rows, SITE_LNT_STATS)) stats[row] = make_float2(mean, rstd);
  }
}

// Partial rows part[block] = [dg (d) | db (d)]; null where the caller wants dx alone.
template <typename T, int VEC, int NV, int W>
__global__ void __launch_bounds__(lnt_warps(W) * 32)
    ln_train_bwd_kernel(const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ g,
                        const float2* __restrict__ stats, const T* __restrict__ dt, int rows, int d,
                        T* __restrict__ dx, float* __restrict__ part, uint32_t* err) {
  constexpr int TEAMS = lnt_warps(W) / W;
  using Raw = typename Pack<T, VEC>::Raw;
  extern __shared__ float acc_sm[];          // [2 d], where a block has several teams
  __shared__ float2 red[TEAMS][2][W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / W, wt = warp % W;
  const long long n_el = static_cast<long long>(rows) * d;
  const float inv_d = 1.0f / static_cast<float>(d);
  float ag[NV * VEC], ab[NV * VEC];          // this lane's columns of dg and db
#pragma unroll
  for (int i = 0; i < NV * VEC; ++i) ag[i] = ab[i] = 0.0f;
  grid_dependency_wait();
  grid_dependents_launch();
  int slot = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * TEAMS + team; row < rows;
       row += static_cast<long long>(gridDim.x) * TEAMS, slot ^= 1) {
    const long long base = row * d;
    Raw u[NV], w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = ((i * W + wt) * 32 + lane) * VEC;
      if (col < d && in_bounds(err, base + col, VEC, n_el, SITE_LNT_X)) {
        u[i] = *reinterpret_cast<const Raw*>(x + base + col);
        w[i] = *reinterpret_cast<const Raw*>(dy + base + col);
      }
    }
    const float2 st = in_bounds(err, row, 1, rows, SITE_LNT_STATS) ? stats[row] : make_float2(0.0f, 0.0f);
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = ((i * W + wt) * 32 + lane) * VEC;
      if (col >= d) continue;
      float gg[VEC];
      load_params<VEC>(g + col, gg);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float h = (to_f32<T>(u[i].e[j]) - st.x) * st.y, t = to_f32<T>(w[i].e[j]);
        ag[i * VEC + j] = fmaf(t, h, ag[i * VEC + j]);
        ab[i * VEC + j] += t;
        c1 = fmaf(gg[j], t, c1);
        c2 = fmaf(gg[j] * t, h, c2);
      }
    }
    const float2 c = team_sum<W>(c1, c2, red[team], team, wt, lane, slot);
    c1 = c.x * inv_d;
    c2 = c.y * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = ((i * W + wt) * 32 + lane) * VEC;
      if (col >= d || !in_bounds(err, base + col, VEC, n_el, SITE_LNT_Y)) continue;
      float gg[VEC];
      load_params<VEC>(g + col, gg);
      Raw t;
      if (dt) t = *reinterpret_cast<const Raw*>(dt + base + col);
      Raw o;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float h = (to_f32<T>(u[i].e[j]) - st.x) * st.y;
        float r = st.y * (fmaf(gg[j], to_f32<T>(w[i].e[j]), -c1) - h * c2);
        if (dt) r += to_f32<T>(t.e[j]);
        o.e[j] = from_f32<T>(r);
      }
      *reinterpret_cast<Raw*>(dx + base + col) = o;
    }
  }
  if (!part) return;
  float* dst = part + static_cast<long long>(blockIdx.x) * 2 * d;
  const long long part_el = static_cast<long long>(gridDim.x) * 2 * d;
  for (int t = 0; t < TEAMS; ++t) {          // teams in order: a fixed order of the sum
    if (team == t) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = ((i * W + wt) * 32 + lane) * VEC;
        if (col >= d) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float sg = ag[i * VEC + j], sb = ab[i * VEC + j];
          if (t > 0) {
            sg += acc_sm[col + j];
            sb += acc_sm[d + col + j];
          }
          if (t < TEAMS - 1) {
            acc_sm[col + j] = sg;
            acc_sm[d + col + j] = sb;
          } else if (in_bounds(err, (dst - part) + d + col + j, 1, part_el, SITE_LNT_PART)) {
            dst[col + j] = sg;
            dst[d + col + j] = sb;
          }
        }
      }
    }
    if (TEAMS > 1) __syncthreads();
  }
}

// dg and db: sums of the partial rows, 32 columns and COL_SLICES interleaved slices of the rows a block.
__global__ void __launch_bounds__(32 * COL_SLICES)
    ln_train_colsum_kernel(const float* __restrict__ part, int n_part, int d, float* __restrict__ dg,
                           float* __restrict__ db, uint32_t* err) {
  __shared__ float red[COL_SLICES][32];
  const int cx = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + cx;
  grid_dependency_wait();
  grid_dependents_launch();
  float s = 0.0f;
  if (col < 2 * d) {
#pragma unroll 4
    for (int p = sl; p < n_part; p += COL_SLICES) {
      const long long i = static_cast<long long>(p) * 2 * d + col;
      if (in_bounds(err, i, 1, static_cast<long long>(n_part) * 2 * d, SITE_LNT_PART)) s += part[i];
    }
  }
  red[sl][cx] = s;
  __syncthreads();
  if (sl != 0 || col >= 2 * d) return;
#pragma unroll
  for (int i = 1; i < COL_SLICES; ++i) s += red[i][cx];
  const int c = col < d ? col : col - d;
  if (!in_bounds(err, c, 1, d, SITE_LNT_GRAD)) return;
  (col < d ? dg : db)[c] = s;
}

// ------------------------------ launch ------------------------------
// Warps per row: the fewest that hold the width at 40 elements a lane.
int team_warps(int d) { return d <= 1280 ? 1 : d <= 2560 ? 2 : d <= 5120 ? 4 : 8; }
int teams_per_block(int d) {
  const int w = team_warps(d);
  return lnt_warps(w) / w;
}
int blocks_for(int rows, int d, int cap) {
  const int t = teams_per_block(d);
  const long long b = (static_cast<long long>(rows) + t - 1) / t;
  return static_cast<int>(b < cap ? b : cap);
}

template <typename T>
struct FwdArgs {
  const T *x, *res;
  const float *g, *b;
  int rows, d;
  float eps;
  T *y, *total;
  float2* stats;
  uint32_t* err;
};
template <typename T>
struct BwdArgs {
  const T *dy, *x;
  const float* g;
  const float2* stats;
  const T* dt;
  int rows, d;
  T* dx;
  float* part;
  uint32_t* err;
};

template <typename T, int VEC, int NV, int W>
cudaError_t go(const FwdArgs<T>& a, cudaStream_t s) {
  return launch_pdl(ln_train_fwd_kernel<T, VEC, NV, W>, dim3(blocks_for(a.rows, a.d, LNT_FWD_BLOCKS)),
                    dim3(lnt_warps(W) * 32), 0, s, a.x, a.res, a.g, a.b, a.rows, a.d, a.eps, a.y, a.total, a.stats,
                    a.err);
}
template <typename T, int VEC, int NV, int W>
cudaError_t go(const BwdArgs<T>& a, cudaStream_t s) {
  const size_t smem = lnt_warps(W) > W ? static_cast<size_t>(2) * a.d * sizeof(float) : 0;
  return launch_pdl(ln_train_bwd_kernel<T, VEC, NV, W>, dim3(blocks_for(a.rows, a.d, LNT_BWD_BLOCKS)),
                    dim3(lnt_warps(W) * 32), smem, s, a.dy, a.x, a.g, a.stats, a.dt, a.rows, a.d, a.dx, a.part, a.err);
}

// Elements a lane: fifths of 40 for rows of one warp (short rows keep few registers), 40 for the rest.
template <typename T, int VEC, typename Args>
cudaError_t by_width(const Args& a, cudaStream_t s) {
  constexpr int FULL = 40 / VEC;
  const int w = team_warps(a.d);
  if (w == 2) return go<T, VEC, FULL, 2>(a, s);
  if (w == 4) return go<T, VEC, FULL, 4>(a, s);
  if (w == 8) return go<T, VEC, FULL, 8>(a, s);
  if (a.d <= 256) return go<T, VEC, FULL / 5, 1>(a, s);
  if (a.d <= 512) return go<T, VEC, 2 * FULL / 5, 1>(a, s);
  if (a.d <= 768) return go<T, VEC, 3 * FULL / 5, 1>(a, s);
  if (a.d <= 1024) return go<T, VEC, 4 * FULL / 5, 1>(a, s);
  return go<T, VEC, FULL, 1>(a, s);
}

template <typename T, typename Args>
cudaError_t by_alignment(const Args& a, cudaStream_t s) {
  // a row starts on 16 bytes only where the width is a multiple of a 16-byte vector
  constexpr int VEC = 16 / sizeof(T);
  return a.d % VEC == 0 ? by_width<T, VEC>(a, s) : by_width<T, 1>(a, s);
}

bool type_ok(int dtype) { return dtype == WB_BF16 || dtype == WB_F16 || dtype == WB_F32; }

template <typename T>
cudaError_t fwd_t(const void* x, const void* res, const float* g, const float* b, int rows, int d, float eps, void* y,
                  void* total, float* stats, uint32_t* err, cudaStream_t s) {
  const FwdArgs<T> a{static_cast<const T*>(x), static_cast<const T*>(res), g, b, rows, d, eps, static_cast<T*>(y),
                     static_cast<T*>(total), reinterpret_cast<float2*>(stats), err};
  return by_alignment<T>(a, s);
}
template <typename T>
cudaError_t bwd_t(const void* dy, const void* x, const float* g, const float* stats, const void* dt, int rows, int d,
                  void* dx, float* part, uint32_t* err, cudaStream_t s) {
  const BwdArgs<T> a{static_cast<const T*>(dy), static_cast<const T*>(x), g, reinterpret_cast<const float2*>(stats),
                     static_cast<const T*>(dt), rows, d, static_cast<T*>(dx), part, err};
  return by_alignment<T>(a, s);
}

}  // namespace
}  // namespace wb

using namespace wb;

extern "C" {

wb_status wb_layernorm_forward(const void* x, const void* residual, const float* g, const float* b, int rows, int d,
                               float eps, int dtype, void* y, void* total, float* stats, void* stream) {
  if (!type_ok(dtype)) return WB_EUNSUPPORTED;
  if (rows < 0 || d < 1 || d > LNT_MAX_D || !(eps > 0.0f)) return WB_EINVAL;
  if (rows == 0) return WB_OK;
  if (!x || !g || !b || !y || !stats || !aligned16(x) || !aligned16(g) || !aligned16(b) || !aligned16(y) ||
      !aligned16(stats))
    return WB_EINVAL;
  if (residual ? !aligned16(residual) || !total || !aligned16(total) : total != nullptr) return WB_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t* err = tc_err_ptr();
  if (!err) return WB_ECUDA;
  Prof pr(PC_TRAIN_LN, s);
  if (dtype == WB_BF16) WB_CUDA(fwd_t<__nv_bfloat16>(x, residual, g, b, rows, d, eps, y, total, stats, err, s));
  else if (dtype == WB_F16) WB_CUDA(fwd_t<__half>(x, residual, g, b, rows, d, eps, y, total, stats, err, s));
  else WB_CUDA(fwd_t<float>(x, residual, g, b, rows, d, eps, y, total, stats, err, s));
  return WB_OK;
}

size_t wb_layernorm_backward_workspace_bytes(int rows, int d) {
  if (rows < 1 || d < 1 || d > LNT_MAX_D) return 0;
  return static_cast<size_t>(blocks_for(rows, d, LNT_BWD_BLOCKS)) * 2 * d * sizeof(float);
}

wb_status wb_layernorm_backward(const void* dy, const void* x, const float* g, const float* stats, const void* dtotal,
                                int rows, int d, int dtype, void* dx, float* dg, float* db, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!type_ok(dtype)) return WB_EUNSUPPORTED;
  if (rows < 0 || d < 1 || d > LNT_MAX_D || !dg != !db) return WB_EINVAL;
  if (dg && (!aligned16(dg) || !aligned16(db))) return WB_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dg) {
      WB_CUDA(cudaMemsetAsync(dg, 0, sizeof(float) * d, s));
      WB_CUDA(cudaMemsetAsync(db, 0, sizeof(float) * d, s));
    }
    return WB_OK;
  }
  if (!dy || !x || !g || !stats || !dx || !aligned16(dy) || !aligned16(x) || !aligned16(g) || !aligned16(stats) ||
      !aligned16(dx) || (dtotal && !aligned16(dtotal)))
    return WB_EINVAL;
  if (dg && (!workspace || !aligned16(workspace) ||
             workspace_bytes < wb_layernorm_backward_workspace_bytes(rows, d)))
    return WB_EWORKSPACE;
  uint32_t* err = tc_err_ptr();
  if (!err) return WB_ECUDA;
  float* part = dg ? static_cast<float*>(workspace) : nullptr;
  Prof pr(PC_TRAIN_LN, s, dg ? 2 : 1);
  if (dtype == WB_BF16) WB_CUDA(bwd_t<__nv_bfloat16>(dy, x, g, stats, dtotal, rows, d, dx, part, err, s));
  else if (dtype == WB_F16) WB_CUDA(bwd_t<__half>(dy, x, g, stats, dtotal, rows, d, dx, part, err, s));
  else WB_CUDA(bwd_t<float>(dy, x, g, stats, dtotal, rows, d, dx, part, err, s));
  if (dg)
    WB_CUDA(launch_pdl(ln_train_colsum_kernel, dim3((2 * d + 31) / 32), dim3(32 * COL_SLICES), 0, s,
                       static_cast<const float*>(part), blocks_for(rows, d, LNT_BWD_BLOCKS), d, dg, db, err));
  return WB_OK;
}

}  // extern "C"
