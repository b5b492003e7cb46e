// Backward pass of cross_fwd_kernel on tcgen05 (head dim 64).
//
// With P = exp(s - lse), dP = dout v^T, delta = sum_e dout out and dS = P (dP - delta):
//   dv = P^T dout,  dk = scale dS^T q   (over the rows of all heads of a group),   dq = scale dS k
// No scores are stored: two kernels form P and dP again, each from the side whose sums it keeps, so that every sum runs inside one
// CTA in a fixed order and nothing is added through memory (one kernel for all three would save two of seven products
// and add dq of every key tile to float32 memory, in an order that changes).
//   cross_dkv_kernel  128 keys a CTA, 64 query rows a step: S^T = K Q^T and dP^T = V dO^T (lane = key) -> P^T and dS^T as
//                     packed bf16 over the columns they came from -> dV += P^T dO, dK += dS^T Q
//   cross_dq_kernel   128 query rows a CTA, 64 keys a step: S = Q K^T, dP = dO V^T -> dS -> dQ += dS K
// P^T and dS^T are A operands read from TMEM; Q, dO and K are read both as K-major and as MN-major B tiles of the
// same shared memory, so nothing is transposed.  256 TMEM columns a CTA, two CTAs an SM: one's softmax under the other's products.
// cross_stats_kernel prepares (lse / scale, delta) of every row, (infinity, 0) for rows that take no part: their P is 0.
//
// Numbers.  Sums are float32; P and dS are rounded to bf16 once each, as operands beside bf16 q, k and dout.
// Rows past their item's lengths may hold anything: they are cleared in shared memory where a zero would multiply them.
#pragma once
#include "cross_attention.cuh"

namespace wb {

constexpr int CRB_M = 128, CRB_STEP = 64;      // accumulator rows of a CTA, rows of the other side a step
constexpr int CRB_STAGES = 3;
constexpr uint32_t CRB_TM_S = 0, CRB_TM_D = 64, CRB_TM_ACC0 = 128, CRB_TM_ACC1 = 192, CRB_TM_COLS = 256;

struct CrossBwdSmem {
  static constexpr int M_BYTES = CRB_M * 128;               // K and V (dkv) or Q and dO (dq)
  static constexpr int STEP_BYTES = CRB_STEP * 128;         // Q and dO (dkv) or K and V (dq)
  static constexpr int STATS_BYTES = CRB_STEP * 8;          // dkv: (lse / scale, delta) of the step's rows
  static constexpr int OFF_M0 = 0;
  static constexpr int OFF_M1 = OFF_M0 + M_BYTES;
  static constexpr int OFF_STEP = OFF_M1 + M_BYTES;
  static constexpr int OFF_STATS = OFF_STEP + CRB_STAGES * 2 * STEP_BYTES;
  static constexpr int OFF_BAR = OFF_STATS + CRB_STAGES * STATS_BYTES;
  static constexpr int TOTAL = 1024 + OFF_BAR + 256;
};
static_assert(2 * CrossBwdSmem::TOTAL <= 227 * 1024, "two CTAs an SM");

struct CrossBwdParams {
  CrossParams x;             // out and lse unused here
  int do_items;              // as q_items, for dout
  const float2* stats;       // [batch][H][stats_ld]
  int stats_ld;              // Tq rounded up to 128
  __nv_bfloat16* dq;         // [batch][Tq][H 64]
  __nv_bfloat16* dk;         // [batch][Tk][Hk 64]
  __nv_bfloat16* dv;
};

struct CrossStatsParams {
  CrossParams x;             // lse, out: the forward pass's
  const __nv_bfloat16* dout;
  long long do_batch, do_row;
  float2* stats;
  int stats_ld;
};

// 8 lanes a row of 64 elements, 16 bytes each.
__global__ void __launch_bounds__(256) cross_stats_kernel(const __grid_constant__ CrossStatsParams p) {
  const CrossParams& x = p.x;
  grid_dependency_wait();
  grid_dependents_launch();
  const long long rows = static_cast<long long>(x.batch) * x.H * p.stats_ld;
  const int e = (threadIdx.x & 7) * 8;
  const float inv_scale = 1.0f / x.scale;
  for (long long r0 = static_cast<long long>(blockIdx.x) * 32; r0 < rows; r0 += static_cast<long long>(gridDim.x) * 32) {
    const long long r = r0 + (threadIdx.x >> 3);
    const bool in = r < rows;
    // heads fastest: the rows of a position lie side by side in memory
    const int h = static_cast<int>(r % x.H);
    const long long bt = r / x.H;
    const int t = static_cast<int>(bt % p.stats_ld), b = static_cast<int>(bt / p.stats_ld);
    const bool there = in && t < cross_len(x.q_lens, b, x.batch, x.Tq, x.err);
    float d = 0.0f;
    if (there) {
      const long long oi = (static_cast<long long>(b) * x.Tq + t) * x.H * CRA_HD + h * CRA_HD + e;
      const long long di = static_cast<long long>(b) * p.do_batch + static_cast<long long>(t) * p.do_row + h * CRA_HD + e;
      if (in_bounds(x.err, oi, 8, static_cast<long long>(x.batch) * x.Tq * x.H * CRA_HD, SITE_CROSS_OUT) &&
          in_bounds(x.err, di, 8, (x.batch - 1) * p.do_batch + (x.Tq - 1) * p.do_row + x.H * CRA_HD, SITE_CROSS_Q)) {
        const uint4 a = *reinterpret_cast<const uint4*>(x.out + oi), c = *reinterpret_cast<const uint4*>(p.dout + di);
        const uint32_t au[4] = {a.x, a.y, a.z, a.w}, cu[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d = fmaf(__uint_as_float(au[i] << 16), __uint_as_float(cu[i] << 16), d);
          d = fmaf(__uint_as_float(au[i] & 0xffff0000u), __uint_as_float(cu[i] & 0xffff0000u), d);
        }
      }
    }
    d += __shfl_xor_sync(0xffffffffu, d, 1);
    d += __shfl_xor_sync(0xffffffffu, d, 2);
    d += __shfl_xor_sync(0xffffffffu, d, 4);
    if (in && e == 0) {
      const long long si = (static_cast<long long>(b) * x.H + h) * p.stats_ld + t;
      const long long li = (static_cast<long long>(b) * x.H + h) * x.Tq + t;
      float2 v = make_float2(INFINITY, 0.0f);
      if (there && in_bounds(x.err, li, 1, static_cast<long long>(x.batch) * x.H * x.Tq, SITE_CROSS_LSE))
        v = make_float2(x.lse[li] * inv_scale, d);
      if (in_bounds(x.err, si, 1, rows, SITE_CROSS_STATS)) p.stats[si] = v;
    }
  }
}

// What both kernels share: barriers, TMEM, and the 64-column exchange between products and softmax warps.
struct CrossBwdBars {
  uint64_t* m_full;
  uint64_t* full;            // [CRB_STAGES]
  uint64_t* empty;           // [CRB_STAGES]
  uint64_t* s_full;          // S and dP hold a step
  uint64_t* p_full;          // P and dS written over them
  uint64_t* fixed;           // dkv: the step's rows that take no part are cleared
  uint64_t* acc_done;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
};
__device__ __forceinline__ CrossBwdBars cross_bwd_bars(uint8_t* smem) {
  CrossBwdBars b;
  b.m_full = reinterpret_cast<uint64_t*>(smem + CrossBwdSmem::OFF_BAR);
  b.full = b.m_full + 1;
  b.empty = b.full + CRB_STAGES;
  b.s_full = b.empty + CRB_STAGES;
  b.p_full = b.s_full + 1;
  b.fixed = b.p_full + 1;
  b.acc_done = b.fixed + 1;
  b.tmem_slot = reinterpret_cast<uint32_t*>(b.acc_done + 1);
  b.abort_flag = reinterpret_cast<volatile int*>(b.tmem_slot + 1);
  return b;
}
__device__ __forceinline__ void cross_bwd_init(const CrossBwdBars& b) {
  mbar_init(b.m_full, 1);
  for (int s = 0; s < CRB_STAGES; ++s) {
    mbar_init(&b.full[s], 1);
    mbar_init(&b.empty[s], 1);
  }
  mbar_init(b.s_full, 1);
  mbar_init(b.p_full, CRA_SOFTMAX_WARPS);
  mbar_init(b.fixed, CRA_SOFTMAX_WARPS);
  mbar_init(b.acc_done, 1);
  *b.abort_flag = 0;
  fence_mbar_init();
}

// Rows [valid, CRB_STEP) of a step's tile become zeros: the softmax warps' 256 threads, a row being 128 bytes.
__device__ __forceinline__ void cross_clear_rows(uint8_t* tile, int valid) {
  uint4* rows = reinterpret_cast<uint4*>(tile);
  for (int i = valid * 8 + static_cast<int>(threadIdx.x) - 64; i < CRB_STEP * 8; i += 32 * CRA_SOFTMAX_WARPS)
    rows[i] = make_uint4(0, 0, 0, 0);
}

// An accumulator's rows lane_base + lane / 4 and + 8, scaled, as bf16; zeros for rows at or past `there`.
__device__ __forceinline__ void cross_store_acc(uint32_t tm, float scale, __nv_bfloat16* dst, long long at, long long row_ld,
                                                long long extent, int row, int there, int rows, int cq, bool any, uint32_t* err) {
  uint32_t v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0;
  if (any) {
    tmem_ld_16x256b_x8(tm, v);
    tmem_ld_wait();
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = row + 8 * half;
    if (r >= rows) continue;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const long long o = at + 8 * half * row_ld + 8 * kk + cq;
      const float x0 = __uint_as_float(v[4 * kk + 2 * half]) * scale, x1 = __uint_as_float(v[4 * kk + 2 * half + 1]) * scale;
      if (in_bounds(err, o, 2, extent, SITE_CROSS_OUT))
        *reinterpret_cast<uint32_t*>(dst + o) = any && r < there ? pack_bf16(x0, x1) : 0u;
    }
  }
}

// q, do maps: boxes of 64 x 64 rows; k, v maps: boxes of 64 x 128 rows.
__global__ void __launch_bounds__(CRA_THREADS, 2)
    cross_dkv_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap do_map,
                     const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                     const __grid_constant__ CrossBwdParams p) {
  using S = CrossBwdSmem;
  constexpr uint32_t IDESC_S = make_idesc(128, CRB_STEP, 1u);
  constexpr uint32_t IDESC_ACC = make_idesc(128, CRA_HD, 1u) | IDESC_B_MN;
  const CrossParams& x = p.x;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base_u32 - smem_u32(smem_raw));
  const CrossBwdBars bar = cross_bwd_bars(smem);
  const int warp = warp_id();
  const int lane = lane_id();
  const int n_kt = (x.Tk + CRB_M - 1) / CRB_M;
  const int kt = blockIdx.x % n_kt;
  const int bh = blockIdx.x / n_kt;
  const int b = bh / x.Hk, hk = bh % x.Hk;
  const int k0 = kt * CRB_M;

  if (threadIdx.x == 0) cross_bwd_init(bar);
  if (warp == 1) tmem_alloc(bar.tmem_slot, CRB_TM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *bar.tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();

  const int q_len = cross_len(x.q_lens, b, x.batch, x.Tq, x.err);
  const int kv_len = cross_len(x.kv_lens, b, x.batch, x.Tk, x.err);
  const int per_head = (q_len + CRB_STEP - 1) / CRB_STEP;
  const int steps = k0 < kv_len ? per_head * x.group : 0;      // the rows of the group's heads, one head after another

  if (warp == 0) {
    if (lane == 0 && steps > 0) {
      const int qb = b * x.q_items, db = b * p.do_items, kb = b * x.kv_items;
      mbar_arrive_expect_tx(bar.m_full, 2 * S::M_BYTES);
      tma_load_3d(smem + S::OFF_M0, &k_map, bar.m_full, hk * CRA_HD, k0, kb);
      tma_load_3d(smem + S::OFF_M1, &v_map, bar.m_full, hk * CRA_HD, k0, kb);
      uint32_t issued = 0, par = 0;
      bool ok = true;
      for (int j = 0; j < steps; ++j) {
        const int st = j % CRB_STAGES;
        const uint32_t ph = (j / CRB_STAGES) & 1;
        if (!mbar_wait(&bar.empty[st], ph ^ 1u, x.err, bar.abort_flag, 43)) { ok = false; break; }
        mbar_arrive_expect_tx(&bar.full[st], 2 * S::STEP_BYTES + S::STATS_BYTES);
        const int h = hk * x.group + j / per_head, t0 = (j % per_head) * CRB_STEP;
        uint8_t* dst = smem + S::OFF_STEP + st * 2 * S::STEP_BYTES;
        tma_load_3d(dst, &q_map, &bar.full[st], h * CRA_HD, t0, qb);
        tma_load_3d(dst + S::STEP_BYTES, &do_map, &bar.full[st], h * CRA_HD, t0, db);
        bulk_load(smem + S::OFF_STATS + st * S::STATS_BYTES, p.stats + (static_cast<long long>(b) * x.H + h) * p.stats_ld + t0,
                  S::STATS_BYTES, &bar.full[st]);
        issued |= 1u << st;
        par = (par & ~(1u << st)) | (ph << st);
      }
      if (!ok) {
        mbar_drain(bar.m_full, 0);
        for (int s = 0; s < CRB_STAGES; ++s)
          if (issued & (1u << s)) mbar_drain(&bar.full[s], (par >> s) & 1u);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && steps > 0) {
      const uint64_t k_desc = sw128_desc(smem_u32(smem + S::OFF_M0)), v_desc = sw128_desc(smem_u32(smem + S::OFF_M1));
      const uint32_t step0 = smem_u32(smem + S::OFF_STEP);
      bool ok = mbar_wait(bar.m_full, 0, x.err, bar.abort_flag, 44);
      int fixes = 0;
      for (int j = 0; j < steps && ok; ++j) {
        const int st = j % CRB_STAGES;
        ok = mbar_wait(&bar.full[st], (j / CRB_STAGES) & 1, x.err, bar.abort_flag, 45);
        const int t0 = (j % per_head) * CRB_STEP;
        if (ok && t0 + CRB_STEP > q_len && q_len < x.Tq) ok = mbar_wait(bar.fixed, fixes++ & 1, x.err, bar.abort_flag, 46);
        if (!ok) break;
        tc_fence_after();
        const uint32_t q_at = step0 + st * 2 * S::STEP_BYTES, do_at = q_at + S::STEP_BYTES;
        const uint64_t qd = sw128_desc(q_at), dd = sw128_desc(do_at);
        // the step before is read: its products were issued before these and run before them
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16(tmem + CRB_TM_S, k_desc + 2 * k, qd + 2 * k, IDESC_S, k != 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16(tmem + CRB_TM_D, v_desc + 2 * k, dd + 2 * k, IDESC_S, k != 0);
        mma_commit(bar.s_full);
        if (!mbar_wait(bar.p_full, j & 1, x.err, bar.abort_flag, 47)) { ok = false; break; }
        tc_fence_after();
        const uint64_t qn = sw128_mn_desc(q_at, S::STEP_BYTES), dn = sw128_mn_desc(do_at, S::STEP_BYTES);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_tmem_a(tmem + CRB_TM_ACC0, tmem + CRB_TM_S + k * 8, dn + k * (2048 >> 4), IDESC_ACC, (j > 0 || k != 0) ? 1u : 0u);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_tmem_a(tmem + CRB_TM_ACC1, tmem + CRB_TM_D + k * 8, qn + k * (2048 >> 4), IDESC_ACC, (j > 0 || k != 0) ? 1u : 0u);
        mma_commit(&bar.empty[st]);
      }
      mma_commit(bar.acc_done);
      mbar_drain(bar.acc_done, 0);
    }
  } else {
    const int quarter = warp & 3;
    const int sub = ((warp - 2) >> 2) & 1;
    const int lane_base = quarter * 32 + sub * 16;
    const uint32_t lane_off = static_cast<uint32_t>(lane_base) << 16;
    const uint32_t s_tm = tmem + lane_off + CRB_TM_S, d_tm = tmem + lane_off + CRB_TM_D;
    const int cq = 2 * (lane & 3);
    const uint64_t c2 = f32x2_pack(x.c, x.c);
    bool ok = true;
    for (int j = 0; j < steps && ok; ++j) {
      const int st = j % CRB_STAGES;
      const int t0 = (j % per_head) * CRB_STEP;
      if (t0 + CRB_STEP > q_len && q_len < x.Tq) {
        if (!__all_sync(0xffffffffu, mbar_wait(&bar.full[st], (j / CRB_STAGES) & 1, x.err, bar.abort_flag, 48))) { ok = false; break; }
        uint8_t* tile = smem + S::OFF_STEP + st * 2 * S::STEP_BYTES;
        cross_clear_rows(tile, q_len - t0);
        cross_clear_rows(tile + S::STEP_BYTES, q_len - t0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar.fixed);
      }
      // the statistics came with the step's tiles; the products that follow need them too
      if (!__all_sync(0xffffffffu, mbar_wait(&bar.full[st], (j / CRB_STAGES) & 1, x.err, bar.abort_flag, 48) &&
                                       mbar_wait(bar.s_full, j & 1, x.err, bar.abort_flag, 49))) { ok = false; break; }
      tc_fence_after();
      // s[4k], s[4k+1]: key ra, rows 8k + cq, + 1; s[4k+2], s[4k+3]: key ra + 8, the same rows
      uint32_t s[32], d[32];
      tmem_ld_16x256b_x8(s_tm, s);
      tmem_ld_16x256b_x8(d_tm, d);
      tmem_ld_wait();
      const float4* stats = reinterpret_cast<const float4*>(smem + S::OFF_STATS + st * S::STATS_BYTES);
      uint32_t pw[16], dw[16];
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const float4 z = stats[4 * kk + (lane & 3)];       // (lse, delta) of rows 8k + cq and + 1
        const uint64_t nl = f32x2_pack(-z.x, -z.z), nd = f32x2_pack(-z.y, -z.w);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint64_t sv = f32x2_pack(__uint_as_float(s[4 * kk + 2 * half]), __uint_as_float(s[4 * kk + 2 * half + 1]));
          const uint64_t dv = f32x2_pack(__uint_as_float(d[4 * kk + 2 * half]), __uint_as_float(d[4 * kk + 2 * half + 1]));
          float a, e;
          f32x2_unpack(f32x2_mul(f32x2_add(sv, nl), c2), a, e);
          a = ex2_approx(a);
          e = ex2_approx(e);
          pw[2 * kk + half] = pack_bf16(a, e);
          f32x2_unpack(f32x2_mul(f32x2_add(dv, nd), f32x2_pack(a, e)), a, e);
          dw[2 * kk + half] = pack_bf16(a, e);
        }
      }
      tmem_st_16x128b_x8(s_tm, pw);
      tmem_st_16x128b_x8(d_tm, dw);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.p_full);
    }
    if (ok && steps > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar.acc_done, 0, x.err, bar.abort_flag, 50));
      tc_fence_after();
    }
    if (ok) {
      const int row = k0 + lane_base + (lane >> 2);
      const long long ld = static_cast<long long>(x.Hk) * CRA_HD;
      const long long at = (static_cast<long long>(b) * x.Tk + row) * ld + hk * CRA_HD;
      const long long extent = static_cast<long long>(x.batch) * x.Tk * ld;
      cross_store_acc(tmem + lane_off + CRB_TM_ACC0, 1.0f, p.dv, at, ld, extent, row, kv_len, x.Tk, cq, steps > 0, x.err);
      cross_store_acc(tmem + lane_off + CRB_TM_ACC1, x.scale, p.dk, at, ld, extent, row, kv_len, x.Tk, cq, steps > 0, x.err);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, CRB_TM_COLS);
}

// q, do maps: boxes of 64 x 128 rows; k, v maps: boxes of 64 x 64 rows.
__global__ void __launch_bounds__(CRA_THREADS, 2)
    cross_dq_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap do_map,
                    const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                    const __grid_constant__ CrossBwdParams p) {
  using S = CrossBwdSmem;
  constexpr uint32_t IDESC_S = make_idesc(128, CRB_STEP, 1u);
  constexpr uint32_t IDESC_ACC = make_idesc(128, CRA_HD, 1u) | IDESC_B_MN;
  const CrossParams& x = p.x;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base_u32 - smem_u32(smem_raw));
  const CrossBwdBars bar = cross_bwd_bars(smem);
  const int warp = warp_id();
  const int lane = lane_id();
  const int n_qt = (x.Tq + CRB_M - 1) / CRB_M;
  const int qt = blockIdx.x % n_qt;
  const int bh = blockIdx.x / n_qt;
  const int b = bh / x.H, h = bh % x.H;
  const int q0 = qt * CRB_M;

  if (threadIdx.x == 0) cross_bwd_init(bar);
  if (warp == 1) tmem_alloc(bar.tmem_slot, CRB_TM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *bar.tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();

  const int q_len = cross_len(x.q_lens, b, x.batch, x.Tq, x.err);
  const int kv_len = cross_len(x.kv_lens, b, x.batch, x.Tk, x.err);
  const int steps = q0 < q_len ? (kv_len + CRB_STEP - 1) / CRB_STEP : 0;

  if (warp == 0) {
    if (lane == 0 && steps > 0) {
      const int hk = h / x.group, qb = b * x.q_items, db = b * p.do_items, kb = b * x.kv_items;
      mbar_arrive_expect_tx(bar.m_full, 2 * S::M_BYTES);
      tma_load_3d(smem + S::OFF_M0, &q_map, bar.m_full, h * CRA_HD, q0, qb);
      tma_load_3d(smem + S::OFF_M1, &do_map, bar.m_full, h * CRA_HD, q0, db);
      uint32_t issued = 0, par = 0;
      bool ok = true;
      for (int j = 0; j < steps; ++j) {
        const int st = j % CRB_STAGES;
        const uint32_t ph = (j / CRB_STAGES) & 1;
        if (!mbar_wait(&bar.empty[st], ph ^ 1u, x.err, bar.abort_flag, 51)) { ok = false; break; }
        mbar_arrive_expect_tx(&bar.full[st], 2 * S::STEP_BYTES);
        uint8_t* dst = smem + S::OFF_STEP + st * 2 * S::STEP_BYTES;
        tma_load_3d(dst, &k_map, &bar.full[st], hk * CRA_HD, j * CRB_STEP, kb);
        tma_load_3d(dst + S::STEP_BYTES, &v_map, &bar.full[st], hk * CRA_HD, j * CRB_STEP, kb);
        issued |= 1u << st;
        par = (par & ~(1u << st)) | (ph << st);
      }
      if (!ok) {
        mbar_drain(bar.m_full, 0);
        for (int s = 0; s < CRB_STAGES; ++s)
          if (issued & (1u << s)) mbar_drain(&bar.full[s], (par >> s) & 1u);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && steps > 0) {
      const uint64_t q_desc = sw128_desc(smem_u32(smem + S::OFF_M0)), do_desc = sw128_desc(smem_u32(smem + S::OFF_M1));
      const uint32_t step0 = smem_u32(smem + S::OFF_STEP);
      bool ok = mbar_wait(bar.m_full, 0, x.err, bar.abort_flag, 52);
      for (int j = 0; j < steps && ok; ++j) {
        const int st = j % CRB_STAGES;
        if (!mbar_wait(&bar.full[st], (j / CRB_STAGES) & 1, x.err, bar.abort_flag, 53)) { ok = false; break; }
        tc_fence_after();
        const uint32_t k_at = step0 + st * 2 * S::STEP_BYTES;
        const uint64_t kd = sw128_desc(k_at), vd = sw128_desc(k_at + S::STEP_BYTES), kn = sw128_mn_desc(k_at, S::STEP_BYTES);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16(tmem + CRB_TM_S, q_desc + 2 * k, kd + 2 * k, IDESC_S, k != 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16(tmem + CRB_TM_D, do_desc + 2 * k, vd + 2 * k, IDESC_S, k != 0);
        mma_commit(bar.s_full);
        if (!mbar_wait(bar.p_full, j & 1, x.err, bar.abort_flag, 54)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_tmem_a(tmem + CRB_TM_ACC0, tmem + CRB_TM_D + k * 8, kn + k * (2048 >> 4), IDESC_ACC, (j > 0 || k != 0) ? 1u : 0u);
        mma_commit(&bar.empty[st]);
      }
      mma_commit(bar.acc_done);
      mbar_drain(bar.acc_done, 0);
    }
  } else {
    const int quarter = warp & 3;
    const int sub = ((warp - 2) >> 2) & 1;
    const int lane_base = quarter * 32 + sub * 16;
    const uint32_t lane_off = static_cast<uint32_t>(lane_base) << 16;
    const uint32_t s_tm = tmem + lane_off + CRB_TM_S, d_tm = tmem + lane_off + CRB_TM_D;
    const int cq = 2 * (lane & 3);
    const int row = q0 + lane_base + (lane >> 2);
    const uint64_t c2 = f32x2_pack(x.c, x.c);
    const long long si = (static_cast<long long>(b) * x.H + h) * p.stats_ld + row;   // rows up to the next 128 have an entry
    float2 za = make_float2(INFINITY, 0.0f), zb = za;
    if (steps > 0 && in_bounds(x.err, si, 9, static_cast<long long>(x.batch) * x.H * p.stats_ld, SITE_CROSS_STATS)) {
      za = p.stats[si];
      zb = p.stats[si + 8];
    }
    bool ok = true;
    for (int j = 0; j < steps && ok; ++j) {
      const int st = j % CRB_STAGES;
      if (!__all_sync(0xffffffffu, mbar_wait(bar.s_full, j & 1, x.err, bar.abort_flag, 55))) { ok = false; break; }
      tc_fence_after();
      uint32_t s[32], d[32];
      tmem_ld_16x256b_x8(s_tm, s);
      tmem_ld_16x256b_x8(d_tm, d);
      tmem_ld_wait();
      uint32_t dw[16];
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float2 z = half ? zb : za;
          const uint64_t sv = f32x2_pack(__uint_as_float(s[4 * kk + 2 * half]), __uint_as_float(s[4 * kk + 2 * half + 1]));
          const uint64_t dv = f32x2_pack(__uint_as_float(d[4 * kk + 2 * half]), __uint_as_float(d[4 * kk + 2 * half + 1]));
          float a, e;
          f32x2_unpack(f32x2_mul(f32x2_add(sv, f32x2_pack(-z.x, -z.x)), c2), a, e);
          a = ex2_approx(a);
          e = ex2_approx(e);
          f32x2_unpack(f32x2_mul(f32x2_add(dv, f32x2_pack(-z.y, -z.y)), f32x2_pack(a, e)), a, e);
          dw[2 * kk + half] = pack_bf16(a, e);
        }
      }
      const int valid = kv_len - j * CRB_STEP;
      if (valid < CRB_STEP) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t keep = (8 * kk + cq < valid ? 0xffffu : 0u) | (8 * kk + cq + 1 < valid ? 0xffff0000u : 0u);
          dw[2 * kk] &= keep;
          dw[2 * kk + 1] &= keep;
        }
        if (j * CRB_STEP + valid < x.Tk) {       // K's rows behind the length: factors of those zeros
          cross_clear_rows(smem + S::OFF_STEP + st * 2 * S::STEP_BYTES, valid);
          fence_proxy_async_smem();
        }
      }
      tmem_st_16x128b_x8(d_tm, dw);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.p_full);
    }
    if (ok && steps > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar.acc_done, 0, x.err, bar.abort_flag, 56));
      tc_fence_after();
    }
    if (ok) {
      const long long ld = static_cast<long long>(x.H) * CRA_HD;
      const long long at = (static_cast<long long>(b) * x.Tq + row) * ld + h * CRA_HD;
      cross_store_acc(tmem + lane_off + CRB_TM_ACC0, x.scale, p.dq, at, ld, static_cast<long long>(x.batch) * x.Tq * ld, row, q_len,
                      x.Tq, cq, steps > 0, x.err);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, CRB_TM_COLS);
}

}  // namespace wb
