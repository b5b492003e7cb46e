// Statistics of the logits of a few rows (a token or some hypotheses): the same (max, sum) and target
// logits as HEAD_LSE, for M <= 16.
//
// Bound by reading w once: 51866 x 1280 bf16 are 133 MB, 19.5 us at 6.8 TB/s.  The tcgen05 tile carries that
// through a ring of shared memory and 128 rows of accumulators, and has two or three tiles a CTA.  Both kernels
// of the loss, calls back to back in a graph over four matrices in turn: with the tiles 28.1 us at one row and
// 27.8 at 16, with this form 25.7 and 27.5 (d = 384: 13.7 and 13.7 against 11.5 and 12.9).  Here w goes straight
// from global memory to registers, 16 bytes a lane, as the A operand of m16n8k16 MMAs: a warp takes 16
// vocabulary rows, lane (g, q) reads 8 k of rows g and g + 8.  A dot product does not mind the order of its k, so the lane's 8
// consecutive k fill the fragment slots of two MMAs, and x (shared memory, read the same way) fills B's
// slots in the same order.  Each lane keeps a running (max, sum) of its rows for its tokens; lanes and
// warps are joined once at the end, and a block leaves one partial per token.
#pragma once
#include "ptx.cuh"
#include "types.h"

namespace wb {

constexpr int GEMV_WARPS = 24, GEMV_MAX_M = 16, GEMV_MAX_D = 4096;
// Bytes between x rows in shared memory: 64 past a multiple of 128, so that rows g and g + 1 of a load fall on
// different banks.
__host__ __device__ constexpr int gemv_row_bytes(int d) { return (2 * d + 127) / 128 * 128 + 64; }

struct GemvParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  int M, V, d;
  float scale_log2;
  const int64_t* labels;     // cross entropy
  const int* cnt;            // distillation: entries of row m at tgt_idx[m k ..]
  const int* tgt_idx;
  int k;
  float2* part;              // [block][part_ld]
  float* part_sum;
  long long part_ld;
  float* tgt_s;              // [m][k]
  uint32_t* err;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (m, l) joined with (m2, l2): l = sum of 2^((logit - m) c).
__device__ __forceinline__ void lse_join(float& m, float& l, float m2, float l2, float c) {
  const float mn = fmaxf(m, m2), mo = mn == -INFINITY ? 0.0f : mn;
  l = l * ex2_approx((m - mo) * c) + l2 * ex2_approx((m2 - mo) * c);
  m = mn;
}

template <int MT>   // groups of 8 rows of x
__global__ void __launch_bounds__(GEMV_WARPS * 32, 1) head_gemv_kernel(const __grid_constant__ GemvParams p) {
  extern __shared__ __align__(128) uint8_t xs[];           // [8 MT][gemv_row_bytes(d)]
  __shared__ float red[3][GEMV_WARPS][8 * MT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int rb = gemv_row_bytes(p.d);
  const int d8 = p.d / 8;
  const long long x_el = static_cast<long long>(p.M) * p.d, w_el = static_cast<long long>(p.V) * p.d;
  grid_dependency_wait();
  grid_dependents_launch();
  // x, zeros behind its rows and its width (a multiple of 32)
  const int chunks = (p.d + 31) / 32 * 4;                  // 16-byte chunks a row
  for (int i = threadIdx.x; i < 8 * MT * chunks; i += GEMV_WARPS * 32) {
    const int m = i / chunks, c = i % chunks;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (m < p.M && c < d8 && in_bounds(p.err, static_cast<long long>(m) * p.d + 8 * c, 8, x_el, SITE_HEAD_X))
      v = *reinterpret_cast<const uint4*>(p.x + static_cast<long long>(m) * p.d + 8 * c);
    *reinterpret_cast<uint4*>(xs + m * rb + 16 * c) = v;
  }
  __syncthreads();

  // 16 vocabulary rows at a time; consecutive groups go to different SMs
  const int wg = blockIdx.x + warp * gridDim.x, n_warps = gridDim.x * GEMV_WARPS;
  const int groups = (p.V + 15) / 16;
  const float c2 = p.scale_log2;
  float mx[2 * MT], l[2 * MT], sum[2 * MT];                // tokens 8 mt + 2 q and + 1
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    mx[i] = -INFINITY;
    l[i] = sum[i] = 0.0f;
  }
  for (int grp = wg; grp < groups; grp += n_warps) {
    const int v0 = grp * 16 + g, v1 = v0 + 8;
    const uint4* w0 = reinterpret_cast<const uint4*>(p.w + static_cast<long long>(v0) * p.d);
    const uint4* w1 = reinterpret_cast<const uint4*>(p.w + static_cast<long long>(v1) * p.d);
    const bool on0 = v0 < p.V, on1 = v1 < p.V;
    float acc[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[mt][i] = 0.0f;
    constexpr int U = 4;                                   // blocks of 32 k whose loads are in flight together
    for (int kb = 0; kb * 4 < d8; kb += U) {
      uint4 a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = (kb + u) * 4 + q;
        a[u] = b[u] = make_uint4(0, 0, 0, 0);
        if (c < d8) {
          if (on0 && in_bounds(p.err, static_cast<long long>(v0) * p.d + 8 * c, 8, w_el, SITE_HEAD_X)) a[u] = __ldcs(w0 + c);
          if (on1 && in_bounds(p.err, static_cast<long long>(v1) * p.d + 8 * c, 8, w_el, SITE_HEAD_X)) b[u] = __ldcs(w1 + c);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = (kb + u) * 4 + q;
        if ((kb + u) * 4 >= d8) break;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint4 xv = *reinterpret_cast<const uint4*>(xs + (8 * mt + g) * rb + 16 * c);
          mma_16816(acc[mt], a[u].x, b[u].x, a[u].y, b[u].y, xv.x, xv.y);
          mma_16816(acc[mt], a[u].z, b[u].z, a[u].w, b[u].w, xv.z, xv.w);
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int i = 2 * mt + t;
        const float s0 = on0 ? acc[mt][t] : -INFINITY, s1 = on1 ? acc[mt][2 + t] : -INFINITY;
        const float mn = fmaxf(mx[i], fmaxf(s0, s1)), mo = mn == -INFINITY ? 0.0f : mn;
        l[i] = l[i] * ex2_approx((mx[i] - mo) * c2) + ex2_approx((s0 - mo) * c2) + ex2_approx((s1 - mo) * c2);
        mx[i] = mn;
        sum[i] += (on0 ? acc[mt][t] : 0.0f) + (on1 ? acc[mt][2 + t] : 0.0f);
      }
  }
  // logits at the targets: a warp each, the last warps first (they have the fewest groups)
  for (int e = n_warps - 1 - wg; e < p.M * p.k; e += n_warps) {
    const int m = e / p.k, j = e % p.k;
    long long v = -1;
    if (p.labels) v = p.labels[m];
    else if (j < p.cnt[m]) v = p.tgt_idx[e];
    if (v < 0 || v >= p.V) continue;
    float s = 0.0f;
    for (int c = lane; c < d8; c += 32) {
      if (!in_bounds(p.err, v * p.d + 8 * c, 8, w_el, SITE_HEAD_X)) continue;
      const uint4 a = *reinterpret_cast<const uint4*>(p.w + v * p.d + 8 * c);
      const uint4 b = *reinterpret_cast<const uint4*>(xs + m * rb + 16 * c);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s = fmaf(__uint_as_float(aw[i] << 16), __uint_as_float(bw[i] << 16), s);
        s = fmaf(__uint_as_float(aw[i] & 0xffff0000u), __uint_as_float(bw[i] & 0xffff0000u), s);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) p.tgt_s[e] = s;
  }
  // lanes of the same q (8 rows each), then the warps, in order
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      lse_join(mx[i], l[i], __shfl_xor_sync(0xffffffffu, mx[i], o), __shfl_xor_sync(0xffffffffu, l[i], o), c2);
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    }
    if (g == 0) {
      const int tok = 8 * (i / 2) + 2 * q + (i & 1);
      red[0][warp][tok] = mx[i];
      red[1][warp][tok] = l[i];
      red[2][warp][tok] = sum[i];
    }
  }
  __syncthreads();
  const int tok = threadIdx.x;
  if (tok < p.M) {
    float m = red[0][0][tok], s = red[1][0][tok], t = red[2][0][tok];
    for (int w = 1; w < GEMV_WARPS; ++w) {
      lse_join(m, s, red[0][w][tok], red[1][w][tok], c2);
      t += red[2][w][tok];
    }
    const long long i = blockIdx.x * p.part_ld + tok;
    if (in_bounds(p.err, i, 1, gridDim.x * p.part_ld, SITE_HEAD_PART)) {
      p.part[i] = make_float2(m, s);
      if (p.part_sum) p.part_sum[i] = t;
    }
  }
}

}  // namespace wb
