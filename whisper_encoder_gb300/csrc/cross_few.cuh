// Attention of a few rows (a token, the hypotheses of a beam) to an encoder's states: the same results as
// cross_fwd_kernel where the rows that read one key head, group x Tq of them, are 16 or fewer.
//
// Bound by reading K and V once (7.7 MB an item of 1500 x 20 heads, 1.1 us at 6.8 TB/s; 32 items 36 us).  S = Q K^T and
// O += P V are m16n8k16 products whose B fragments are K and V as they lie: lane (g, t) takes of key g the 8 elements from 8 t
// and from 32 + 8 t (a dot product does not mind the order of its k, so they fill the slots of four products, and Q
// fills A's slots in the same order), and of keys 2t, 2t + 1, 8 + 2t, 9 + 2t of V the 8 elements from 8 g: B wants pairs
// of keys, which byte permutations make.  P's accumulator layout is the A layout of the next product.
// A lane needs no other lane's K or V, so each has its own slots of a ring in shared memory that 16-byte asynchronous copies fill
// three groups of 16 keys ahead: 192 KB in flight an SM without a register or a barrier.
//
// A warp takes every eighth group of its CTA's share of the keys and keeps its own running maximum, sum and O.  Warps are joined in shared
// memory; where there are few (item, head) pairs a cluster of up to 8 CTAs splits the keys, and each pushes its share of a
// row to the CTA that writes the row, through distributed shared memory: one launch, no workspace, a fixed order of sums.
#pragma once
#include "cross_attention.cuh"
#include "head_gemv.cuh"

namespace wb {

constexpr int FEW_WARPS = 8, FEW_THREADS = FEW_WARPS * 32;
constexpr int FEW_ROWS = 16, FEW_KEYS = 16;
constexpr int FEW_STAGES = 3, FEW_STAGE_BYTES = 8 * 32 * 16;
constexpr int FEW_MAX_SPLITS = 8;
constexpr int FEW_LD = CRA_HD + 4;             // floats of a row's share: O, its maximum, its sum

struct FewSmem {
  static constexpr int WARP_BYTES = FEW_STAGES * FEW_STAGE_BYTES;    // a warp's ring; after the loop, its share of the rows
  static constexpr int OFF_SHARED = FEW_WARPS * WARP_BYTES;          // shares that the cluster's CTAs push here
  static constexpr int SHARED_ROWS = FEW_ROWS + FEW_MAX_SPLITS;      // splits * ceil(16 / splits) at most
  static constexpr int TOTAL = OFF_SHARED + SHARED_ROWS * FEW_LD * 4;
};
static_assert(FEW_ROWS * FEW_LD * 4 <= FewSmem::WARP_BYTES, "a warp's share fits its ring");
static_assert(2 * FewSmem::TOTAL <= 226 * 1024, "two CTAs an SM");

struct FewParams {
  CrossParams x;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long q_batch, q_row, k_batch, k_row, v_batch, v_row;   // elements
  int splits;                // CTAs of a cluster
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(s));
  return r;
}
// 16 bytes to shared memory, zeros where !there (the address is then not read).
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
  return r;
}
__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, const float4& v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

__global__ void __launch_bounds__(FEW_THREADS, 2) cross_few_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ __align__(16) uint8_t few_raw[];
  const CrossParams& x = p.x;
  const int lane = lane_id(), warp = warp_id();
  const int g = lane >> 2, t = lane & 3;
  const int splits = p.splits;
  const int rank = blockIdx.x % splits;
  const int pair = blockIdx.x / splits;
  const int b = pair / x.Hk, hk = pair % x.Hk;
  const int rows = x.group * x.Tq;                          // row r: head r / Tq of the group, position r % Tq

  if (splits > 1) cluster_arrive();                         // waited for before the first push: the others run by then
  grid_dependency_wait();
  grid_dependents_launch();
  const int q_len = cross_len(x.q_lens, b, x.batch, x.Tq, x.err);
  const int kv_len = q_len > 0 ? cross_len(x.kv_lens, b, x.batch, x.Tk, x.err) : 0;
  const int groups = (kv_len + FEW_KEYS - 1) / FEW_KEYS;
  const int first = static_cast<int>(static_cast<long long>(groups) * rank / splits);
  const int last = static_cast<int>(static_cast<long long>(groups) * (rank + 1) / splits);

  const __nv_bfloat16* kp = p.k + static_cast<long long>(b) * p.k_batch + hk * CRA_HD + 8 * t;
  const __nv_bfloat16* vp = p.v + static_cast<long long>(b) * p.v_batch + hk * CRA_HD + 8 * g;
  uint8_t* const ring = few_raw + warp * FewSmem::WARP_BYTES;
  const uint32_t slots = smem_u32(ring) + lane * 16;
  // a group's 8 pieces of this lane: K of keys g and 8 + g, two each; V of keys 2t, 2t + 1, 8 + 2t, 9 + 2t
  auto load = [&](int grp, int stage) {
    if (grp < last) {
      const int key0 = grp * FEW_KEYS;
      const long long k_el = static_cast<long long>(x.Tk - 1) * p.k_row + x.Hk * CRA_HD;
      const long long v_el = static_cast<long long>(x.Tk - 1) * p.v_row + x.Hk * CRA_HD;
      const uint32_t dst = slots + stage * FEW_STAGE_BYTES;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = key0 + 8 * i + g;
        const long long at = static_cast<long long>(key) * p.k_row;
        const bool there = key < kv_len && in_bounds(x.err, at + hk * CRA_HD + 8 * t, 40, k_el, SITE_CROSS_KV);
        const __nv_bfloat16* src = there ? kp + at : p.k;
        copy_async16(dst + (2 * i) * 512, src, there);
        copy_async16(dst + (2 * i + 1) * 512, there ? src + 32 : p.k, there);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + 8 * (i >> 1) + 2 * t + (i & 1);
        const long long at = static_cast<long long>(key) * p.v_row;
        const bool there = key < kv_len && in_bounds(x.err, at + hk * CRA_HD + 8 * g, 8, v_el, SITE_CROSS_KV);
        copy_async16(dst + (4 + i) * 512, there ? vp + at : p.v, there);
      }
    }
    copy_async_commit();
  };
#pragma unroll
  for (int s = 0; s < FEW_STAGES - 1; ++s) load(first + warp + s * FEW_WARPS, s);

  // A fragments of Q: rows g and g + 8, elements 8t.. and 32 + 8t..
  uint32_t qf[4][4];
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    const int r = g + 8 * hi;
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
      qf[2 * c][hi] = u[c].x;
      qf[2 * c][2 + hi] = u[c].y;
      qf[2 * c + 1][hi] = u[c].z;
      qf[2 * c + 1][2 + hi] = u[c].w;
    }
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, o[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;

  int stage = 0;
  for (int grp = first + warp; grp < last; grp += FEW_WARPS) {
    load(grp + (FEW_STAGES - 1) * FEW_WARPS, stage == 0 ? FEW_STAGES - 1 : stage - 1);
    copy_async_wait<FEW_STAGES - 1>();
    const uint32_t src = slots + stage * FEW_STAGE_BYTES;
    stage = stage + 1 == FEW_STAGES ? 0 : stage + 1;
    float s[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 u = ld_shared_v4(src + (2 * i + c) * 512);
        mma_16816(s[i], qf[2 * c][0], qf[2 * c][1], qf[2 * c][2], qf[2 * c][3], u.x, u.y);
        mma_16816(s[i], qf[2 * c + 1][0], qf[2 * c + 1][1], qf[2 * c + 1][2], qf[2 * c + 1][3], u.z, u.w);
      }
    }
    const int key0 = grp * FEW_KEYS;
    if (key0 + FEW_KEYS > kv_len) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (key0 + 8 * i + 2 * t + (k & 1) >= kv_len) s[i][k] = -INFINITY;
    }
    float top[2];
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) top[hi] = fmaxf(fmaxf(s[0][2 * hi], s[0][2 * hi + 1]), fmaxf(s[1][2 * hi], s[1][2 * hi + 1]));
    if (__any_sync(0xffffffffu, top[0] > m[0] + x.slack || top[1] > m[1] + x.slack)) {
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        float v = fmaxf(top[hi], __shfl_xor_sync(0xffffffffu, top[hi], 1));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
        if (v > m[hi] + x.slack) {
          const float a = ex2_approx((m[hi] - v) * x.c);
          m[hi] = v;
          l[hi] *= a;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[j][2 * hi] *= a;
            o[j][2 * hi + 1] *= a;
          }
        }
      }
    }
    uint32_t a[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const float mo = m[hi] == -INFINITY ? 0.0f : m[hi];
        const float p0 = ex2_approx((s[i][2 * hi] - mo) * x.c), p1 = ex2_approx((s[i][2 * hi + 1] - mo) * x.c);
        l[hi] += p0 + p1;
        a[2 * i + hi] = pack_bf16(p0, p1);
      }
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ld_shared_v4(src + (4 + i) * 512);
    const uint32_t v0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, v1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
    const uint32_t v2[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, v3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
      mma_16816(o[j], a[0], a[1], a[2], a[3], prmt(v0[j >> 1], v1[j >> 1], sel), prmt(v2[j >> 1], v3[j >> 1], sel));
    }
  }
  copy_async_wait<0>();
  __syncwarp();                  // every lane's copies have landed: the ring becomes the warp's share

  // o[j] holds elements 16 t + j and 16 t + 8 + j of rows g and g + 8
  float* const share = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    float sum = l[hi];
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    float* dst = share + (g + 8 * hi) * FEW_LD;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < 8; j += 4)
        *reinterpret_cast<float4*>(dst + 16 * t + 8 * e + j) =
            make_float4(o[j][2 * hi + e], o[j + 1][2 * hi + e], o[j + 2][2 * hi + e], o[j + 3][2 * hi + e]);
    if (t == 0) {
      dst[CRA_HD] = m[hi];
      dst[CRA_HD + 1] = sum;
    }
  }
  __syncthreads();
  if (splits > 1) cluster_wait();

  // n shares of a row, `step` floats apart, joined: elements e.. of O and (maximum, sum)
  auto join = [&](const float* from, int step, int n, int e, float& top, float& sum) -> float4 {
    top = -INFINITY;
#pragma unroll
    for (int w = 0; w < 8; ++w)
      if (w < n) top = fmaxf(top, from[w * step + CRA_HD]);
    const float mo = top == -INFINITY ? 0.0f : top;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w >= n) continue;
      const float f = ex2_approx((from[w * step + CRA_HD] - mo) * x.c);
      const float4 u = *reinterpret_cast<const float4*>(from + w * step + e);
      sum = fmaf(f, from[w * step + CRA_HD + 1], sum);
      acc.x = fmaf(f, u.x, acc.x);
      acc.y = fmaf(f, u.y, acc.y);
      acc.z = fmaf(f, u.z, acc.z);
      acc.w = fmaf(f, u.w, acc.w);
    }
    return acc;
  };
  const long long out_el = static_cast<long long>(x.batch) * x.Tq * x.H * CRA_HD;
  const long long lse_el = static_cast<long long>(x.batch) * x.H * x.Tq;
  auto write = [&](int r, int e, const float4& acc, float top, float sum) {
    const int h = hk * x.group + r / x.Tq, q = r % x.Tq;
    const bool there = kv_len > 0 && q < q_len;
    const float inv = 1.0f / sum;
    const long long at = (static_cast<long long>(b) * x.Tq + q) * x.H * CRA_HD + h * CRA_HD + e;
    if (in_bounds(x.err, at, 4, out_el, SITE_CROSS_OUT))
      *reinterpret_cast<uint2*>(x.out + at) =
          there ? make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv)) : make_uint2(0u, 0u);
    const long long li = (static_cast<long long>(b) * x.H + h) * x.Tq + q;
    if (e == 0 && in_bounds(x.err, li, 1, lse_el, SITE_CROSS_LSE)) x.lse[li] = there ? top * x.scale + logf(sum) : -INFINITY;
  };
  const int r = threadIdx.x >> 4, e = (threadIdx.x & 15) * 4;        // 16 threads a row
  float top, sum;
  if (r < rows) {
    const float4 acc = join(reinterpret_cast<float*>(few_raw) + r * FEW_LD, FewSmem::WARP_BYTES / 4, FEW_WARPS, e, top, sum);
    if (splits == 1) {
      write(r, e, acc, top, sum);
    } else {
      // row r is written by CTA r % splits, which has a place for each CTA's share of its r / splits-th row
      const uint32_t dst = cluster_addr(few_raw + FewSmem::OFF_SHARED, r % splits) + ((r / splits) * splits + rank) * FEW_LD * 4;
      st_cluster_f32x4(dst + e * 4, acc);
      if (e == 0) st_cluster_f32x4(dst + CRA_HD * 4, make_float4(top, sum, 0.0f, 0.0f));
    }
  }
  if (splits == 1) return;
  cluster_arrive();
  cluster_wait();
  if (r * splits + rank < rows) {
    const float* from = reinterpret_cast<const float*>(few_raw + FewSmem::OFF_SHARED) + r * splits * FEW_LD;
    const float4 acc = join(from, FEW_LD, splits, e, top, sum);
    write(r * splits + rank, e, acc, top, sum);
  }
}

}  // namespace wb
