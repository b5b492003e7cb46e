// Attention of a few rows (a token, the hypotheses of a beam) to an encoder's states: the same results as
// cross_fwd_kernel where the rows that read one head's keys, 64-wide group x Tq of them, are 32 or fewer.
//
// Bound by reading K and V once (7.7 MB an item of 1500 x 20 heads, 1.1 us at 6.8 TB/s; 32 items 36 us).  They go straight from
// global memory to registers, 16 bytes a lane: S = Q K^T and O += P V as m16n8k16 products whose B fragments are
// those registers.  Lane (g, t) reads of key g the 8 elements from 8 t and from 32 + 8 t (a dot product does not mind the order
// of its k, so they fill the slots of four products, and Q fills A's slots in the same order), and of keys 2t, 2t + 1,
// 8 + 2t, 9 + 2t of V the 8 elements from 8 g: B wants pairs of keys, which byte permutations make.  P's accumulator layout is
// the A layout of the next product: no shared memory until the end.
//
// A warp takes every eighth group of 16 keys of its CTA's share and keeps its own running maximum, sum and O; warps are joined in shared
// memory, and where there are few (item, head) pairs a cluster of up to 8 CTAs splits the keys and joins through
// distributed shared memory: one launch, no workspace, a fixed order of sums.
#pragma once
#include "cross_attention.cuh"
#include "head_gemv.cuh"

namespace wb {

constexpr int FEW_WARPS = 8, FEW_THREADS = FEW_WARPS * 32;
constexpr int FEW_MAX_ROWS = 32;

struct FewParams {
  CrossParams x;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long q_batch, q_row, k_batch, k_row, v_batch, v_row;   // elements
  int splits;                // CTAs of a cluster
};

__host__ __device__ constexpr int few_smem(int mt) { return FEW_WARPS * 16 * mt * (CRA_HD + 4) * 4 + 2 * FEW_WARPS * 16 * mt * 4; }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(s));
  return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// 16 keys of a lane: K of keys 8b + g (two pieces each), V of keys 2t, 2t + 1, 8 + 2t, 9 + 2t.
struct FewTile {
  uint4 k[2][2], v[4];
};

template <int MT>
__global__ void __launch_bounds__(FEW_THREADS) cross_few_kernel(const __grid_constant__ FewParams p) {
  constexpr int ROWS = 16 * MT, LD = CRA_HD + 4;
  extern __shared__ __align__(16) float few_raw[];
  float* part_o = few_raw;                                  // [warp][row][LD]
  float* part_m = few_raw + FEW_WARPS * ROWS * LD;          // [warp][row]
  float* part_l = part_m + FEW_WARPS * ROWS;
  const CrossParams& x = p.x;
  const int lane = lane_id(), warp = warp_id();
  const int g = lane >> 2, t = lane & 3;
  const int splits = p.splits;
  const int rank = blockIdx.x % splits;
  const int pair = blockIdx.x / splits;
  const int b = pair / x.Hk, hk = pair % x.Hk;
  const int rows = x.group * x.Tq;                          // row r: head r / Tq of the group, position r % Tq

  grid_dependency_wait();
  grid_dependents_launch();
  const int q_len = cross_len(x.q_lens, b, x.batch, x.Tq, x.err);
  const int kv_len = q_len > 0 ? cross_len(x.kv_lens, b, x.batch, x.Tk, x.err) : 0;
  const int groups = (kv_len + 15) / 16;
  const int first = static_cast<int>(static_cast<long long>(groups) * rank / splits);
  const int last = static_cast<int>(static_cast<long long>(groups) * (rank + 1) / splits);

  // A fragments of Q: rows 16 i + g and + 8, elements 8t.. and 32 + 8t..
  uint32_t qf[MT][4][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int r = 16 * i + g + 8 * hi;
      uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (r < rows) {
        const long long at = static_cast<long long>(b) * p.q_batch + static_cast<long long>(r % x.Tq) * p.q_row +
                             (hk * x.group + r / x.Tq) * CRA_HD + 8 * t;
        const long long el = static_cast<long long>(x.batch - 1) * p.q_batch + (x.Tq - 1) * p.q_row + x.H * CRA_HD;
        if (in_bounds(x.err, at, 40, el, SITE_CROSS_Q)) {
          u[0] = *reinterpret_cast<const uint4*>(p.q + at);
          u[1] = *reinterpret_cast<const uint4*>(p.q + at + 32);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qf[i][2 * c][hi] = u[c].x;
        qf[i][2 * c][2 + hi] = u[c].y;
        qf[i][2 * c + 1][hi] = u[c].z;
        qf[i][2 * c + 1][2 + hi] = u[c].w;
      }
    }

  const __nv_bfloat16* kp = p.k + static_cast<long long>(b) * p.k_batch + hk * CRA_HD + 8 * t;
  const __nv_bfloat16* vp = p.v + static_cast<long long>(b) * p.v_batch + hk * CRA_HD + 8 * g;
  auto load = [&](FewTile& f, int grp) {
    const int key0 = grp * 16;
    const long long k_el = static_cast<long long>(x.Tk - 1) * p.k_row + x.Hk * CRA_HD;
    const long long v_el = static_cast<long long>(x.Tk - 1) * p.v_row + x.Hk * CRA_HD;
#pragma unroll
    for (int bl = 0; bl < 2; ++bl) {
      const int key = key0 + 8 * bl + g;
      const long long at = static_cast<long long>(key) * p.k_row;
      f.k[bl][0] = f.k[bl][1] = make_uint4(0, 0, 0, 0);
      if (key < kv_len && in_bounds(x.err, at + hk * CRA_HD + 8 * t, 40, k_el, SITE_CROSS_KV)) {
        f.k[bl][0] = *reinterpret_cast<const uint4*>(kp + at);
        f.k[bl][1] = *reinterpret_cast<const uint4*>(kp + at + 32);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = key0 + 8 * (i >> 1) + 2 * t + (i & 1);
      const long long at = static_cast<long long>(key) * p.v_row;
      f.v[i] = make_uint4(0, 0, 0, 0);
      if (key < kv_len && in_bounds(x.err, at + hk * CRA_HD + 8 * g, 8, v_el, SITE_CROSS_KV))
        f.v[i] = *reinterpret_cast<const uint4*>(vp + at);
    }
  };

  float m[MT][2], l[MT][2], o[MT][8][4];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    m[i][0] = m[i][1] = -INFINITY;
    l[i][0] = l[i][1] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][j][k] = 0.0f;
  }
  auto step = [&](const FewTile& f, int grp) {
    const int key0 = grp * 16;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      float s[2][4];
#pragma unroll
      for (int bl = 0; bl < 2; ++bl) {
        s[bl][0] = s[bl][1] = s[bl][2] = s[bl][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mma_16816(s[bl], qf[i][2 * c][0], qf[i][2 * c][1], qf[i][2 * c][2], qf[i][2 * c][3], f.k[bl][c].x, f.k[bl][c].y);
          mma_16816(s[bl], qf[i][2 * c + 1][0], qf[i][2 * c + 1][1], qf[i][2 * c + 1][2], qf[i][2 * c + 1][3], f.k[bl][c].z,
                    f.k[bl][c].w);
        }
      }
      if (key0 + 16 > kv_len) {
#pragma unroll
        for (int bl = 0; bl < 2; ++bl)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (key0 + 8 * bl + 2 * t + (k & 1) >= kv_len) s[bl][k] = -INFINITY;
      }
      float top[2];
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) top[hi] = fmaxf(fmaxf(s[0][2 * hi], s[0][2 * hi + 1]), fmaxf(s[1][2 * hi], s[1][2 * hi + 1]));
      if (__any_sync(0xffffffffu, top[0] > m[i][0] + x.slack || top[1] > m[i][1] + x.slack)) {
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          float v = fmaxf(top[hi], __shfl_xor_sync(0xffffffffu, top[hi], 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          if (v > m[i][hi] + x.slack) {
            const float a = ex2_approx((m[i][hi] - v) * x.c);
            m[i][hi] = v;
            l[i][hi] *= a;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              o[i][j][2 * hi] *= a;
              o[i][j][2 * hi + 1] *= a;
            }
          }
        }
      }
      uint32_t a[4];
#pragma unroll
      for (int bl = 0; bl < 2; ++bl)
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          const float mo = m[i][hi] == -INFINITY ? 0.0f : m[i][hi];
          const float p0 = ex2_approx((s[bl][2 * hi] - mo) * x.c), p1 = ex2_approx((s[bl][2 * hi + 1] - mo) * x.c);
          l[i][hi] += p0 + p1;
          a[2 * bl + hi] = pack_bf16(p0, p1);
        }
      const uint32_t v0[4] = {f.v[0].x, f.v[0].y, f.v[0].z, f.v[0].w}, v1[4] = {f.v[1].x, f.v[1].y, f.v[1].z, f.v[1].w};
      const uint32_t v2[4] = {f.v[2].x, f.v[2].y, f.v[2].z, f.v[2].w}, v3[4] = {f.v[3].x, f.v[3].y, f.v[3].z, f.v[3].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
        mma_16816(o[i][j], a[0], a[1], a[2], a[3], prmt(v0[j >> 1], v1[j >> 1], sel), prmt(v2[j >> 1], v3[j >> 1], sel));
      }
    }
  };

  int grp = first + warp;
  FewTile cur, next;
  if (grp < last) load(cur, grp);
  for (; grp < last; grp += FEW_WARPS) {
    if (grp + FEW_WARPS < last) load(next, grp + FEW_WARPS);
    step(cur, grp);
    cur = next;
  }

  // this warp's share: o[i][j] holds elements 16 t + j and 16 t + 8 + j of rows 16 i + g and + 8
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int r = 16 * i + g + 8 * hi;
      float sum = l[i][hi];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      float* dst = part_o + (warp * ROWS + r) * LD + 16 * t;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j = 0; j < 8; j += 4)
          *reinterpret_cast<float4*>(dst + 8 * e + j) = make_float4(o[i][j][2 * hi + e], o[i][j + 1][2 * hi + e],
                                                                   o[i][j + 2][2 * hi + e], o[i][j + 3][2 * hi + e]);
      if (t == 0) {
        part_m[warp * ROWS + r] = m[i][hi];
        part_l[warp * ROWS + r] = sum;
      }
    }
  __syncthreads();

  // join the warps: the block's (m, l, O) of a row in the first warp's place
  for (int i = threadIdx.x; i < ROWS * (CRA_HD / 4); i += FEW_THREADS) {
    const int r = i / (CRA_HD / 4), e = i % (CRA_HD / 4) * 4;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < FEW_WARPS; ++w) top = fmaxf(top, part_m[w * ROWS + r]);
    const float mo = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < FEW_WARPS; ++w) {
      const float f = ex2_approx((part_m[w * ROWS + r] - mo) * x.c);
      const float4 u = *reinterpret_cast<const float4*>(part_o + (w * ROWS + r) * LD + e);
      sum += f * part_l[w * ROWS + r];
      acc.x = fmaf(f, u.x, acc.x);
      acc.y = fmaf(f, u.y, acc.y);
      acc.z = fmaf(f, u.z, acc.z);
      acc.w = fmaf(f, u.w, acc.w);
    }
    // row r's columns e.. of the first warp are read by this thread alone; its m and l only behind the barrier below
    *reinterpret_cast<float4*>(part_o + r * LD + e) = acc;
    if (e == 0) {
      part_o[r * LD + CRA_HD] = top;
      part_o[r * LD + CRA_HD + 1] = sum;
    }
  }
  __syncthreads();
  if (splits > 1) cluster_sync();

  // a split writes its share of the rows
  const long long out_el = static_cast<long long>(x.batch) * x.Tq * x.H * CRA_HD;
  const long long lse_el = static_cast<long long>(x.batch) * x.H * x.Tq;
  for (int i = threadIdx.x + rank * FEW_THREADS; i < rows * (CRA_HD / 4); i += FEW_THREADS * splits) {
    const int r = i / (CRA_HD / 4), e = i % (CRA_HD / 4) * 4;
    const float* mine = part_o + r * LD;
    float top = mine[CRA_HD], sum = mine[CRA_HD + 1];
    float4 acc = *reinterpret_cast<const float4*>(mine + e);
    if (splits > 1) {
      top = -INFINITY;
      for (int s = 0; s < splits; ++s) top = fmaxf(top, ld_cluster_f32(cluster_addr(mine + CRA_HD, s)));
      const float mo = top == -INFINITY ? 0.0f : top;
      sum = 0.0f;
      acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int s = 0; s < splits; ++s) {
        const float f = ex2_approx((ld_cluster_f32(cluster_addr(mine + CRA_HD, s)) - mo) * x.c);
        const uint32_t a = cluster_addr(mine + e, s);
        sum += f * ld_cluster_f32(cluster_addr(mine + CRA_HD + 1, s));
        acc.x = fmaf(f, ld_cluster_f32(a), acc.x);
        acc.y = fmaf(f, ld_cluster_f32(a + 4), acc.y);
        acc.z = fmaf(f, ld_cluster_f32(a + 8), acc.z);
        acc.w = fmaf(f, ld_cluster_f32(a + 12), acc.w);
      }
    }
    const int h = hk * x.group + r / x.Tq, q = r % x.Tq;
    const bool there = kv_len > 0 && q < q_len;
    const float inv = 1.0f / sum;
    const long long at = (static_cast<long long>(b) * x.Tq + q) * x.H * CRA_HD + h * CRA_HD + e;
    if (in_bounds(x.err, at, 4, out_el, SITE_CROSS_OUT))
      *reinterpret_cast<uint2*>(x.out + at) =
          there ? make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv)) : make_uint2(0u, 0u);
    const long long li = (static_cast<long long>(b) * x.H + h) * x.Tq + q;
    if (e == 0 && in_bounds(x.err, li, 1, lse_el, SITE_CROSS_LSE)) x.lse[li] = there ? top * x.scale + logf(sum) : -INFINITY;
  }
  if (splits > 1) cluster_sync();        // the others have read this CTA's share
}

}  // namespace wb
