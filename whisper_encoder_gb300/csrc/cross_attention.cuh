// Attention of a decoder's rows to an encoder's states of another length (head dim 64), forward, on tcgen05.
//
//   s = scale q k^T,  p = softmax of s over the state's kv_len keys,  out = p v,  lse = ln sum exp s
//
// A CTA has 128 query rows of one (item, head) and walks its keys 128 at a time:
//   S = Q K_j^T           -> TMEM, fp32, 128 columns
//   P = 2^((S - m) c)     -> bf16 in TMEM, 64 columns; the PV product reads its A operand from there
//   l += row sums of the unrounded P, float32
//   O += P V_j            -> TMEM, fp32, 64 columns; V is read where it lies, as an MN-major B tile
// Two CTAs share an SM (256 TMEM columns each), so that one's softmax runs under the other's products.  Where there are too few
// tiles of rows for the SMs, a cluster of up to 8 CTAs splits a tile's keys; each leaves its O, maxima and sums in
// shared memory and joins a share of the rows of all of them, in order (224 rows of 16 heads over 13501 keys: 92 us in
// 32 CTAs, 24 in 256).
// One lane of warp 0 loads with TMA, one of warp 1 issues the MMAs, warps 2-9 run the softmax: each owns 16 query
// rows through the 16-lane TMEM shapes, four threads a row.
//
// Numbers.  Scores stay float32, and so do the exponent's argument and the exponential: lse is a float32 result
// that the backward pass takes its softmax from.  The difference s - m comes before the scale: in one
// fused step, what the rounding leaves of a large score is an exponent.  The running maximum moves only when
// a new one is above it by 2^8.  P is rounded to bf16 once, because one MMA takes one type and V is bf16.
// Rows and keys past their item's lengths may hold anything: keys are masked by selection, the tail's rows of V (which the
// zeros of P would multiply) are cleared in shared memory before the product, and rows of Q reach only their own row.
#pragma once
#include "ptx.cuh"
#include "types.h"

namespace wb {

constexpr int CRA_BQ = 128, CRA_BK = 128, CRA_HD = 64;
constexpr int CRA_KSTAGES = 3, CRA_VSTAGES = 2;
constexpr int CRA_SOFTMAX_WARPS = 8;
constexpr int CRA_THREADS = 64 + 32 * CRA_SOFTMAX_WARPS;
constexpr uint32_t CRA_TM_S = 0, CRA_TM_O = 128, CRA_TM_P = 192, CRA_TM_COLS = 256;

struct CrossSmem {
  static constexpr int Q_BYTES = CRA_BQ * 128;
  static constexpr int KV_BYTES = CRA_BK * 128;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + Q_BYTES;
  static constexpr int OFF_V = OFF_K + CRA_KSTAGES * KV_BYTES;
  static constexpr int OFF_BAR = OFF_V + CRA_VSTAGES * KV_BYTES;
  static constexpr int TOTAL = 1024 + OFF_BAR + 256;
  // a split's share, over the rings when they are done: rows of 64 floats of O, its maximum and its sum
  static constexpr int SHARE_LD = CRA_HD + 4;
};
static_assert(2 * CrossSmem::TOTAL <= 227 * 1024, "two CTAs an SM");
static_assert(CRA_BQ * CrossSmem::SHARE_LD * 4 <= CrossSmem::OFF_BAR, "a share fits the rings");
constexpr int CRA_MAX_SPLITS = 8;

struct CrossParams {
  int batch, Tq, Tk, H, Hk;
  int group;                 // H / Hk
  int splits;                // cross_fwd_kernel: CTAs of a cluster, for the keys of a tile
  int q_items, kv_items;     // 0: every item reads the first one's rows (a batch stride of 0), else 1
  float scale;
  float c;                   // scale log2(e)
  float slack;               // 8 / c: how far a score may pass the running maximum
  const int* q_lens;         // [batch] or null
  const int* kv_lens;
  __nv_bfloat16* out;        // [batch][Tq][H 64]
  float* lse;                // [batch][H][Tq]
  uint32_t* err;
};

__device__ __forceinline__ int cross_len(const int* lens, int i, int batch, int most, uint32_t* err) {
  if (!lens || !in_bounds(err, i, 1, batch, SITE_CROSS_LENS)) return most;
  return min(max(lens[i], 0), most);
}

// Four lanes t hold words (columns 8k + 2t and + 1) of k = 0..3; lane t gets all four words of k = t: 16 bytes in a row.
__device__ __forceinline__ uint4 quad_transpose(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, int t) {
  const bool odd = t & 1, high = t & 2;
  uint32_t a = __shfl_xor_sync(0xffffffffu, odd ? w0 : w1, 1), b = __shfl_xor_sync(0xffffffffu, odd ? w2 : w3, 1);
  if (odd) { w0 = a; w2 = b; } else { w1 = a; w3 = b; }
  a = __shfl_xor_sync(0xffffffffu, high ? w0 : w2, 2);
  b = __shfl_xor_sync(0xffffffffu, high ? w1 : w3, 2);
  if (high) { w0 = a; w1 = b; } else { w2 = a; w3 = b; }
  return make_uint4(w0, w1, w2, w3);
}

// q, k, v maps: (64 heads, T, items) of bf16 rows, boxes of 64 x 128 x 1.
__global__ void __launch_bounds__(CRA_THREADS, 2)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CrossParams p) {
  using S = CrossSmem;
  constexpr uint32_t IDESC_S = make_idesc(128, CRA_BK, 1u);
  constexpr uint32_t IDESC_O = make_idesc(128, CRA_HD, 1u) | IDESC_B_MN;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base_u32 - smem_u32(smem_raw));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* k_full = q_full + 1;
  uint64_t* k_empty = k_full + CRA_KSTAGES;
  uint64_t* v_full = k_empty + CRA_KSTAGES;
  uint64_t* v_empty = v_full + CRA_VSTAGES;
  uint64_t* s_full = v_empty + CRA_VSTAGES;
  uint64_t* s_free = s_full + 1;
  uint64_t* p_full = s_free + 1;
  uint64_t* pv_done = p_full + 1;
  uint64_t* mma_done = pv_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = warp_id();
  const int lane = lane_id();
  const int n_qt = (p.Tq + CRA_BQ - 1) / CRA_BQ;
  const int splits = p.splits, rank = blockIdx.x % splits;
  const int qt = blockIdx.x / splits % n_qt;
  const int bh = blockIdx.x / splits / n_qt;
  const int b = bh / p.H, h = bh % p.H;
  const int q0 = qt * CRA_BQ;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < CRA_KSTAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < CRA_VSTAGES; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, CRA_SOFTMAX_WARPS);
    mbar_init(p_full, CRA_SOFTMAX_WARPS);
    mbar_init(pv_done, 1);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  const long long out_el = static_cast<long long>(p.batch) * p.Tq * p.H * CRA_HD;
  const long long lse_el = static_cast<long long>(p.batch) * p.H * p.Tq;
  if (warp == 1) tmem_alloc(tmem_slot, CRA_TM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();

  const int q_len = cross_len(p.q_lens, b, p.batch, p.Tq, p.err);
  const int kv_len = cross_len(p.kv_lens, b, p.batch, p.Tk, p.err);
  // rows that take part, and the tiles of their keys, of which this CTA has [j0, j0 + nkv); without any, zeros are written below
  const int all_kv = q0 < q_len ? (kv_len + CRA_BK - 1) / CRA_BK : 0;
  const int j0 = static_cast<int>(static_cast<long long>(all_kv) * rank / splits);
  const int nkv = static_cast<int>(static_cast<long long>(all_kv) * (rank + 1) / splits) - j0;

  if (warp == 0) {
    if (nkv > 0 && elect_one()) {
      tma_prefetch_desc(&q_map);
      tma_prefetch_desc(&k_map);
      tma_prefetch_desc(&v_map);
      const int hk = h / p.group, qb = b * p.q_items, kb = b * p.kv_items;
      mbar_arrive_expect_tx(q_full, S::Q_BYTES);
      tma_load_3d(smem + S::OFF_Q, &q_map, q_full, h * CRA_HD, q0, qb);
      uint32_t k_issued = 0, k_par = 0, v_issued = 0, v_par = 0;
      auto load_k = [&](int jj) -> bool {
        const int st = jj % CRA_KSTAGES;
        const uint32_t ph = (jj / CRA_KSTAGES) & 1;
        if (!mbar_wait(&k_empty[st], ph ^ 1u, p.err, abort_flag, 32)) return false;
        mbar_arrive_expect_tx(&k_full[st], S::KV_BYTES);
        tma_load_3d(smem + S::OFF_K + st * S::KV_BYTES, &k_map, &k_full[st], hk * CRA_HD, (j0 + jj) * CRA_BK, kb);
        k_issued |= 1u << st;
        k_par = (k_par & ~(1u << st)) | (ph << st);
        return true;
      };
      auto load_v = [&](int jj) -> bool {
        const int st = jj % CRA_VSTAGES;
        const uint32_t ph = (jj / CRA_VSTAGES) & 1;
        if (!mbar_wait(&v_empty[st], ph ^ 1u, p.err, abort_flag, 33)) return false;
        mbar_arrive_expect_tx(&v_full[st], S::KV_BYTES);
        tma_load_3d(smem + S::OFF_V + st * S::KV_BYTES, &v_map, &v_full[st], hk * CRA_HD, (j0 + jj) * CRA_BK, kb);
        v_issued |= 1u << st;
        v_par = (v_par & ~(1u << st)) | (ph << st);
        return true;
      };
      bool ok = load_k(0);
      for (int i = 0; i < nkv && ok; ++i) {
        if (i + 1 < nkv) ok = load_k(i + 1);
        ok = ok && load_v(i);
      }
      if (!ok) {
        // copies already issued still land in shared memory: wait for them before the CTA exits
        mbar_drain(q_full, 0);
        for (int s = 0; s < CRA_KSTAGES; ++s)
          if (k_issued & (1u << s)) mbar_drain(&k_full[s], (k_par >> s) & 1u);
        for (int s = 0; s < CRA_VSTAGES; ++s)
          if (v_issued & (1u << s)) mbar_drain(&v_full[s], (v_par >> s) & 1u);
      }
    }
  } else if (warp == 1) {
    if (nkv > 0 && elect_one()) {
      const uint64_t q_desc = sw128_desc(smem_u32(smem + S::OFF_Q));
      const uint64_t k_desc0 = sw128_desc(smem_u32(smem + S::OFF_K));
      const uint64_t v_desc0 = sw128_mn_desc(smem_u32(smem + S::OFF_V), S::KV_BYTES);
      auto qk = [&](int jj) -> bool {
        const int st = jj % CRA_KSTAGES;
        if (!mbar_wait(&k_full[st], (jj / CRA_KSTAGES) & 1, p.err, abort_flag, 34)) return false;
        if (jj > 0 && !mbar_wait(s_free, (jj - 1) & 1, p.err, abort_flag, 35)) return false;
        tc_fence_after();
        const uint64_t kd = k_desc0 + static_cast<uint64_t>(st * (S::KV_BYTES >> 4));
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_bf16(tmem + CRA_TM_S, q_desc + 2 * k, kd + 2 * k, IDESC_S, k != 0);
        mma_commit(s_full);
        mma_commit(&k_empty[st]);
        return true;
      };
      auto pv = [&](int jj) -> bool {
        // P holds 128 keys as 64 packed columns, 8 per K16 step; V advances 16 rows of 128 bytes
        const int st = jj % CRA_VSTAGES;
        if (!mbar_wait(&v_full[st], (jj / CRA_VSTAGES) & 1, p.err, abort_flag, 36)) return false;
        if (!mbar_wait(p_full, jj & 1, p.err, abort_flag, 37)) return false;
        tc_fence_after();
        const uint64_t vd = v_desc0 + static_cast<uint64_t>(st * (S::KV_BYTES >> 4));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_f16_tmem_a(tmem + CRA_TM_O, tmem + CRA_TM_P + k * 8, vd + k * (2048 >> 4), IDESC_O, (jj > 0 || k != 0) ? 1u : 0u);
        mma_commit(pv_done);
        mma_commit(&v_empty[st]);
        return true;
      };
      bool ok = mbar_wait(q_full, 0, p.err, abort_flag, 38) && qk(0);
      for (int j = 0; j < nkv && ok; ++j) {
        if (j + 1 < nkv) ok = qk(j + 1);
        ok = ok && pv(j);
      }
      mma_commit(mma_done);
      mbar_drain(mma_done, 0);
    }
  } else {
    // 16 rows a warp; thread t holds rows ra = t/4 and ra + 8 of them and of each the columns 8k + 2 (t % 4) and + 1
    const int quarter = warp & 3;
    const int sub = ((warp - 2) >> 2) & 1;
    const int lane_base = quarter * 32 + sub * 16;
    const uint32_t lane_off = static_cast<uint32_t>(lane_base) << 16;
    const uint32_t s_tm = tmem + lane_off + CRA_TM_S;
    const uint32_t o_tm = tmem + lane_off + CRA_TM_O;
    const uint32_t p_tm = tmem + lane_off + CRA_TM_P;
    const int ra = lane_base + (lane >> 2);
    const int cq = 2 * (lane & 3);
    const float c = p.c;
    float m_a = -INFINITY, m_b = -INFINITY;        // running maxima of the scores of rows ra and ra + 8
    float l_a = 0.0f, l_b = 0.0f;                  // this thread's share of the two row sums
    bool ok = true;

    for (int j = 0; j < nkv && ok; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(s_full, j & 1, p.err, abort_flag, 39))) { ok = false; break; }
      tc_fence_after();
      float s[64];
      {
        uint32_t v[32];
        tmem_ld_16x256b_x8(s_tm, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(v[i]);
        tmem_ld_16x256b_x8(s_tm + 64, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) s[32 + i] = __uint_as_float(v[i]);
      }
      tmem_ld_wait();
      tc_fence_before();           // S is in registers: QK of the next key tile may overwrite it
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free);
      const int valid = kv_len - (j0 + j) * CRA_BK;   // keys of this tile that take part
      if (valid < CRA_BK) {
#pragma unroll
        for (int kk = 0; kk < 16; ++kk) {
          const int col = 8 * kk + cq;
          if (col >= valid) s[4 * kk] = s[4 * kk + 2] = -INFINITY;
          if (col + 1 >= valid) s[4 * kk + 1] = s[4 * kk + 3] = -INFINITY;
        }
        // past the last row TMA has filled in zeros; before it V's rows may hold anything
        if (kv_len < p.Tk) {
          const int st = j % CRA_VSTAGES;
          if (!__all_sync(0xffffffffu, mbar_wait(&v_full[st], (j / CRA_VSTAGES) & 1, p.err, abort_flag, 40))) { ok = false; break; }
          uint4* rows = reinterpret_cast<uint4*>(smem + S::OFF_V + st * S::KV_BYTES);
          for (int i = valid * 8 + static_cast<int>(threadIdx.x) - 64; i < CRA_BK * 8; i += 32 * CRA_SOFTMAX_WARPS)
            rows[i] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
      }
      float xa0 = fmaxf(s[0], s[1]), xa1 = fmaxf(s[4], s[5]);
      float xb0 = fmaxf(s[2], s[3]), xb1 = fmaxf(s[6], s[7]);
#pragma unroll
      for (int kk = 2; kk < 16; kk += 2) {
        xa0 = fmax3(xa0, s[4 * kk], s[4 * kk + 1]);
        xa1 = fmax3(xa1, s[4 * kk + 4], s[4 * kk + 5]);
        xb0 = fmax3(xb0, s[4 * kk + 2], s[4 * kk + 3]);
        xb1 = fmax3(xb1, s[4 * kk + 6], s[4 * kk + 7]);
      }
      float xa = fmaxf(xa0, xa1), xb = fmaxf(xb0, xb1);
      float alpha_a = 1.0f, alpha_b = 1.0f;
      bool rescale = false;
      // a vote on the threads' own maxima finds the (rare) tiles in which a row's maximum moves
      if (j == 0 || __any_sync(0xffffffffu, xa > m_a + p.slack || xb > m_b + p.slack)) {
        xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
        xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
        xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2));
        xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2));
        if (j == 0) {
          m_a = xa;
          m_b = xb;
        } else {
          if (xa > m_a + p.slack) {
            alpha_a = ex2_approx((m_a - xa) * c);
            m_a = xa;
            l_a *= alpha_a;
            rescale = true;
          }
          if (xb > m_b + p.slack) {
            alpha_b = ex2_approx((m_b - xb) * c);
            m_b = xb;
            l_b *= alpha_b;
            rescale = true;
          }
        }
      }
      // scores of -infinity alone: their differences are -infinity and not NaN
      const float ma = m_a == -INFINITY ? 0.0f : m_a, mb = m_b == -INFINITY ? 0.0f : m_b;
      const uint64_t c2 = f32x2_pack(c, c), na2 = f32x2_pack(-ma, -ma), nb2 = f32x2_pack(-mb, -mb);
      uint32_t pw[32];             // pw[2k]: row ra, P column 4k + t % 4; pw[2k+1]: row ra + 8
      uint64_t la2 = 0, lb2 = 0;
#pragma unroll
      for (int kk = 0; kk < 16; ++kk) {
        float x0, x1, x2, x3;
        f32x2_unpack(f32x2_mul(f32x2_add(f32x2_pack(s[4 * kk], s[4 * kk + 1]), na2), c2), x0, x1);
        f32x2_unpack(f32x2_mul(f32x2_add(f32x2_pack(s[4 * kk + 2], s[4 * kk + 3]), nb2), c2), x2, x3);
        x0 = ex2_approx(x0);
        x1 = ex2_approx(x1);
        x2 = ex2_approx(x2);
        x3 = ex2_approx(x3);
        la2 = f32x2_add(la2, f32x2_pack(x0, x1));
        lb2 = f32x2_add(lb2, f32x2_pack(x2, x3));
        pw[2 * kk] = pack_bf16(x0, x1);
        pw[2 * kk + 1] = pack_bf16(x2, x3);
      }
      {
        float x0, x1;
        f32x2_unpack(la2, x0, x1);
        l_a += x0 + x1;
        f32x2_unpack(lb2, x0, x1);
        l_b += x0 + x1;
      }
      // PV of key tile j-1 is done: P may be overwritten, and O is stable until PV of tile j is issued
      if (j > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(pv_done, (j - 1) & 1, p.err, abort_flag, 41))) { ok = false; break; }
        tc_fence_after();
      }
      tmem_st_16x128b_x16(p_tm, pw);
      if (j > 0 && __any_sync(0xffffffffu, rescale)) {
        uint32_t v[32];
        tmem_ld_16x256b_x8(o_tm, v);
        tmem_ld_wait();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          v[4 * kk] = __float_as_uint(__uint_as_float(v[4 * kk]) * alpha_a);
          v[4 * kk + 1] = __float_as_uint(__uint_as_float(v[4 * kk + 1]) * alpha_a);
          v[4 * kk + 2] = __float_as_uint(__uint_as_float(v[4 * kk + 2]) * alpha_b);
          v[4 * kk + 3] = __float_as_uint(__uint_as_float(v[4 * kk + 3]) * alpha_b);
        }
        tmem_st_16x256b_x8(o_tm, v);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
    }
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
    l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
    l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
    if (ok && nkv > 0) ok = __all_sync(0xffffffffu, mbar_wait(pv_done, (nkv - 1) & 1, p.err, abort_flag, 42));
    if (ok) {
      uint32_t v[32];                              // [4k..4k+3]: rows ra / ra + 8, columns 8k + cq, + 1
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0;
      if (nkv > 0) {
        tc_fence_after();
        tmem_ld_16x256b_x8(o_tm, v);
        tmem_ld_wait();
      }
      if (splits > 1 && all_kv > 0) {
        float* share = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float* row = share + (ra + 8 * half) * S::SHARE_LD;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            *reinterpret_cast<float2*>(row + 8 * kk + cq) =
                make_float2(__uint_as_float(v[4 * kk + 2 * half]), __uint_as_float(v[4 * kk + 2 * half + 1]));
          if ((lane & 3) == 0) *reinterpret_cast<float2*>(row + CRA_HD) = half ? make_float2(m_b, l_b) : make_float2(m_a, l_a);
        }
      } else if (rank == 0) {
        const int t = lane & 3;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int q = q0 + ra + 8 * half;
          const bool there = nkv > 0 && q < q_len;
          const float l = half ? l_b : l_a, inv = 1.0f / l;
          uint32_t w[8];
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            w[kk] = there ? pack_bf16(__uint_as_float(v[4 * kk + 2 * half]) * inv, __uint_as_float(v[4 * kk + 2 * half + 1]) * inv) : 0u;
          const uint4 u0 = quad_transpose(w[0], w[1], w[2], w[3], t), u1 = quad_transpose(w[4], w[5], w[6], w[7], t);
          if (q >= p.Tq) continue;
          const long long o = (static_cast<long long>(b) * p.Tq + q) * p.H * CRA_HD + h * CRA_HD + 8 * t;
          if (in_bounds(p.err, o, 40, out_el, SITE_CROSS_OUT)) {
            *reinterpret_cast<uint4*>(p.out + o) = u0;
            *reinterpret_cast<uint4*>(p.out + o + 32) = u1;
          }
          const long long li = (static_cast<long long>(b) * p.H + h) * p.Tq + q;
          if (t == 0 && in_bounds(p.err, li, 1, lse_el, SITE_CROSS_LSE))
            p.lse[li] = there ? (half ? m_b : m_a) * p.scale + logf(l) : -INFINITY;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, CRA_TM_COLS);
  if (splits == 1 || all_kv == 0) return;          // the same in all CTAs of a cluster
  cluster_sync();                                  // everyone's share is written
  const int r0 = CRA_BQ * rank / splits, r1 = CRA_BQ * (rank + 1) / splits;
  for (int i = threadIdx.x; i < (r1 - r0) * (CRA_HD / 4); i += CRA_THREADS) {
    const int r = r0 + i / (CRA_HD / 4), e = i % (CRA_HD / 4) * 4, q = q0 + r;
    if (q >= p.Tq) break;
    const uint32_t at = smem_u32(smem) + r * S::SHARE_LD * 4;
    float4 o[CRA_MAX_SPLITS], ml[CRA_MAX_SPLITS];
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < CRA_MAX_SPLITS; ++k) {
      if (k >= splits) continue;
      const uint32_t from = cluster_map(at, k);
      o[k] = ld_cluster_f32x4(from + e * 4);
      ml[k] = ld_cluster_f32x4(from + CRA_HD * 4);
      top = fmaxf(top, ml[k].x);
    }
    const float mo = top == -INFINITY ? 0.0f : top;
    float l = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < CRA_MAX_SPLITS; ++k) {
      if (k >= splits) continue;
      const float f = ex2_approx((ml[k].x - mo) * p.c);
      l = fmaf(f, ml[k].y, l);
      acc.x = fmaf(f, o[k].x, acc.x);
      acc.y = fmaf(f, o[k].y, acc.y);
      acc.z = fmaf(f, o[k].z, acc.z);
      acc.w = fmaf(f, o[k].w, acc.w);
    }
    const bool there = q < q_len;
    const float inv = 1.0f / l;
    const long long at_o = (static_cast<long long>(b) * p.Tq + q) * p.H * CRA_HD + h * CRA_HD + e;
    if (in_bounds(p.err, at_o, 4, out_el, SITE_CROSS_OUT))
      *reinterpret_cast<uint2*>(p.out + at_o) =
          there ? make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv)) : make_uint2(0u, 0u);
    const long long li = (static_cast<long long>(b) * p.H + h) * p.Tq + q;
    if (e == 0 && in_bounds(p.err, li, 1, lse_el, SITE_CROSS_LSE)) p.lse[li] = there ? top * p.scale + logf(l) : -INFINITY;
  }
  cluster_sync();                                  // the others have read this CTA's share
}

}  // namespace wb
