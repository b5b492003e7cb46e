// Backward pass of cross_fwd_kernel on tcgen05 (head dim 64).
//
// With P = exp(s - lse), dP = dout v^T, delta = sum_k P dP and dS = P (dP - delta):
//   dv = P^T dout,  dk = scale dS^T q   (over the rows of all heads of a group),   dq = scale dS k
// No scores are stored: two kernels form P and dP again, each from the side whose sums it keeps, so that every sum runs inside one
// CTA in a fixed order and nothing is added through memory (one kernel for all three would save two of seven products
// and add dq of every key tile to float32 memory, in an order that changes).
//   cross_bwd_kernel<false,.> 128 query rows an item, 128 keys a step: S = Q K^T, dP = dO V^T -> dQ += dS K, M += P K
//   cross_bwd_kernel<true,.>  128 keys an item, 128 query rows a step: S^T = K Q^T, dP^T = V dO^T (lane = key) ->
//                             dV += P^T dO, dK += dS^T Q
// P and dS go as packed bf16 over the TMEM columns S came from and are read there as A operands; the step's tiles are read both as
// K-major and as MN-major B tiles of the same shared memory, so nothing is transposed.
//
// Persistent, one CTA an SM over its items in turn.  Bound by the chain of a step (scores, 16 warps read them, the softmax, P and dS back to
// TMEM, sums).  Its 24 products, 8 of 128 x 128 x 16 (S and dP) and 16 of 128 x 64 x 16 (the two sums), take 1230 cycles at the rates
// they have alone (64 and 45 each), a step about 2500 (8 x 448 x 1500 x 20 heads; tensor pipe active 36 to 40 %).
// What overlaps: S is double, dP is given back as soon as the softmax holds it in registers, so the scores of step n + 1 are formed under the
// softmax of step n, and its sums under the softmax of step n + 1; an item's sums are stored after the next item's first softmax.
// Where there are fewer tiles of query rows than SMs, clusters of up to 8 CTAs split their keys and join dQ, M and b through
// distributed shared memory (dq of 224 rows of 16 heads over 13501 keys 106 -> 37 us).
// 128 columns a step: with 64, two buffers of both and a group of warps for each, a product took 48 cycles for half the work and a step
// 2000 (dk and dv of 32 x 448 x 1500 x 20 heads 526 us; one item a CTA, two CTAs an SM, 419).
// The dq kernel takes lse and delta of its rows at the start of an item and leaves them for the dkv kernel, -infinity and 0 for rows that
// take no part, whose P is then 0 (a kernel of their own before both: 514 us against 518 for 32 x 448 x 1500 x 20 heads, but 22.2
// against 20.2 for 3 x 77 x 1371 x 6).
// One lane of warp 0 loads, one of warp 1 issues, warps 2-17 run the softmax: 16 rows of half of the columns each.  All 16 rows of a warp
// are computed, also those past the item's length: nothing of theirs is stored.
//
// Numbers.  Sums are float32; P and dS are rounded to bf16 once each, as operands beside bf16 q, k and dout (with 64 rows or keys
// or fewer that side's free half of S takes what that leaves as a second operand: dk and dv of few rows 2.4e-3 -> 1.7e-3 from 64 bits;
// as a branch in the one kernel it cost 25 % of every size).  delta is sum_e dout out as well,
// but out is rounded to bf16, and what that leaves is the same for all keys of a row: it does not average out (dq and dk were 3.3e-3 of
// their norm from 64 bits, 2.4e-3 without it).  With d' that delta, b = sum_k P (dP - d') is what it lacks, since sum_k P = 1: the dq
// kernel hands delta = d' + b to the dkv kernel, and subtracts b' M from dq, M = sum_k P k and b' the sum of dS as it was rounded: what
// rounding leaves then adds up along k - M alone, which is small where a row's weight lies on one key (dq of sharp rows 2.6e-3 -> 2.1e-3).
// Rows of one key have P = 1 whatever q and k are: their dq and that key's dk are 0, not what rounding leaves.
// Rows past their item's lengths may hold anything: a step's are cleared in shared memory before its products, an item's own reach only
// results that are not stored.
#pragma once
#include "cross_attention.cuh"

namespace wb {

constexpr int CRB_M = 128, CRB_STEP = 128;     // own rows of an item, rows of the other side a step
constexpr int CRB_STAGES = 4;
constexpr int CRB_GROUP_WARPS = 8, CRB_WARPS = 2 * CRB_GROUP_WARPS, CRB_THREADS = 64 + 32 * CRB_WARPS;
// TMEM: S of even and odd steps (over each half of it that half's P and dS, 32 columns each), dP, the two accumulators
constexpr uint32_t CRB_TM_S = 128, CRB_TM_D = 256, CRB_TM_ACC = 384, CRB_TM_COLS = 512;

struct CrossBwdSmem {
  static constexpr int TILE = CRB_M * 128;                  // 128 rows of 64 elements
  static constexpr int STATS_BYTES = 2 * CRB_STEP * 4;      // dkv: -lse / scale, then -delta, of the step's rows
  static constexpr int OFF_STEP = 4 * TILE;                 // the own tiles have two slots
  static constexpr int OFF_STATS = OFF_STEP + CRB_STAGES * 2 * TILE;
  static constexpr int OFF_B = OFF_STATS + CRB_STAGES * STATS_BYTES;    // dq: b and b' by [item parity][column half][row]
  static constexpr int OFF_BAR = OFF_B + 2 * 2 * CRB_M * 8;
  static constexpr int TOTAL = 1024 + OFF_BAR + 512;
  // dq: a split's share, over the rings when they are done: rows of 64 floats of M, 64 of dQ, b and b'
  static constexpr int SHARE_LD = 2 * CRA_HD + 4;
};
static_assert(CrossBwdSmem::TOTAL <= 227 * 1024, "one CTA an SM");
static_assert(CRB_M * CrossBwdSmem::SHARE_LD * 4 <= CrossBwdSmem::OFF_STATS - CrossBwdSmem::OFF_STEP, "a share fits the ring");

struct CrossBwdParams {
  CrossParams x;             // lse, out: the forward pass's
  const __nv_bfloat16* dout;
  long long do_batch, do_row;
  int do_items;              // as q_items, for dout
  float* stats;              // [batch][H][2][stats_ld]: -lse / scale, -delta, from the dq kernel to the dkv kernel
  int stats_ld;              // Tq rounded up to 128
  int want_dq;               // cross_bwd_kernel<false,.>: 0: delta alone
  __nv_bfloat16* dq;         // [batch][Tq][H 64]
  __nv_bfloat16* dk;         // [batch][Tk][Hk 64]
  __nv_bfloat16* dv;
};

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// -lse / scale and -sum_e dout out of a row of q, by the four threads of a quad; -infinity and 0 for one that takes no part.
__device__ __forceinline__ float2 cross_row_stats(const CrossBwdParams& p, int b, int h, int row, bool there, int t) {
  const CrossParams& x = p.x;
  float d = 0.0f, l = INFINITY;
  if (there) {
    const long long oi = (static_cast<long long>(b) * x.Tq + row) * x.H * CRA_HD + h * CRA_HD + 16 * t;
    const long long di = static_cast<long long>(b) * p.do_batch + static_cast<long long>(row) * p.do_row + h * CRA_HD + 16 * t;
    if (in_bounds(x.err, oi, 16, static_cast<long long>(x.batch) * x.Tq * x.H * CRA_HD, SITE_CROSS_OUT) &&
        in_bounds(x.err, di, 16, (x.batch - 1) * p.do_batch + (x.Tq - 1) * p.do_row + x.H * CRA_HD, SITE_CROSS_Q)) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 a = *reinterpret_cast<const uint4*>(x.out + oi + 8 * k), c = *reinterpret_cast<const uint4*>(p.dout + di + 8 * k);
        const uint32_t au[4] = {a.x, a.y, a.z, a.w}, cu[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d = fmaf(__uint_as_float(au[i] << 16), __uint_as_float(cu[i] << 16), d);
          d = fmaf(__uint_as_float(au[i] & 0xffff0000u), __uint_as_float(cu[i] & 0xffff0000u), d);
        }
      }
    }
    const long long li = (static_cast<long long>(b) * x.H + h) * x.Tq + row;
    if (in_bounds(x.err, li, 1, static_cast<long long>(x.batch) * x.H * x.Tq, SITE_CROSS_LSE)) l = x.lse[li] / x.scale;
  }
  d += __shfl_xor_sync(0xffffffffu, d, 1);
  d += __shfl_xor_sync(0xffffffffu, d, 2);
  return make_float2(-l, -d);
}

// own0, own1: K and V (DKV) or Q and dO; step0, step1: Q and dO (DKV) or K and V.  Boxes of 64 x 128 rows.
// TWICE: the step side has 64 rows or fewer in all.
template <bool DKV, bool TWICE>
__global__ void __launch_bounds__(CRB_THREADS, 1)
    cross_bwd_kernel(const __grid_constant__ CUtensorMap own0, const __grid_constant__ CUtensorMap own1,
                     const __grid_constant__ CUtensorMap step0, const __grid_constant__ CUtensorMap step1,
                     const __grid_constant__ CrossBwdParams p) {
  using S = CrossBwdSmem;
  const CrossParams& x = p.x;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base_u32 - smem_u32(smem_raw));
  uint64_t* m_full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);   // [2] an item's own tiles
  uint64_t* m_empty = m_full + 2;                                      // [2]
  uint64_t* full = m_empty + 2;                                        // [CRB_STAGES] a step's tiles
  uint64_t* empty = full + CRB_STAGES;                                 // [CRB_STAGES]
  uint64_t* s_full = empty + CRB_STAGES;                               // S and dP of a step
  uint64_t* d_free = s_full + 1;                                       // dP is in registers
  uint64_t* p_full = d_free + 1;                                       // [2] P and dS written, by parity of the step
  uint64_t* fixed = p_full + 2;                                        // a ragged step's tiles are cleared
  uint64_t* acc_full = fixed + 1;                                      // an item's sums
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* b_full = acc_empty + 1;                                    // every warp's share of b is written
  uint64_t* mma_done = b_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = warp_id();
  const int lane = lane_id();

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m_full[i], 1);
      mbar_init(&m_empty[i], 1);
      mbar_init(&p_full[i], CRB_WARPS);
    }
    for (int s = 0; s < CRB_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(d_free, CRB_WARPS);
    mbar_init(fixed, CRB_WARPS);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, CRB_WARPS);
    mbar_init(b_full, CRB_WARPS);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, CRB_TM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();

  const int own_T = DKV ? x.Tk : x.Tq, step_T = DKV ? x.Tq : x.Tk, heads = DKV ? x.Hk : x.H;
  const int n_tiles = (own_T + CRB_M - 1) / CRB_M;
  const int n_items = x.batch * heads * n_tiles;
  // CTAs of a cluster share an item's steps; such a grid has one item a cluster
  const int splits = DKV ? 1 : x.splits, rank = blockIdx.x % splits;
  const int it_first = blockIdx.x / splits, it_step = gridDim.x / splits;
  // every role walks the same items and steps
  struct Item {
    int b, h, r0;              // h: head of the own rows; r0: the first of them
    int own_len, step_len, per_head, steps;
    int t_first;               // first row of this CTA's steps
  };
  auto item_at = [&](int it) -> Item {
    Item r;
    const int bh = it / n_tiles;
    r.r0 = it % n_tiles * CRB_M;
    r.b = bh / heads;
    r.h = bh % heads;
    const int q_len = cross_len(x.q_lens, r.b, x.batch, x.Tq, x.err), kv_len = cross_len(x.kv_lens, r.b, x.batch, x.Tk, x.err);
    r.own_len = DKV ? kv_len : q_len;
    r.step_len = DKV ? q_len : kv_len;
    r.per_head = (r.step_len + CRB_STEP - 1) / CRB_STEP;
    r.steps = r.r0 < r.own_len ? r.per_head * (DKV ? x.group : 1) : 0;     // DKV: the group's heads one after another
    r.t_first = 0;
    if (!DKV && splits > 1) {
      const int j0 = r.steps * rank / splits;
      r.t_first = j0 * CRB_STEP;
      r.steps = r.steps * (rank + 1) / splits - j0;
    }
    return r;
  };
  // rows of a step that starts at t0, and whether its tail holds rows that take no part (behind the last row TMA fills in zeros)
  auto next_t0 = [](const Item& i, int t0) { return t0 + CRB_STEP >= i.step_len ? 0 : t0 + CRB_STEP; };
  auto ragged = [&](const Item& i, int t0) { return t0 + CRB_STEP > i.step_len && i.step_len < step_T; };

  if (warp == 0) {
    if (elect_one()) {
      uint32_t n = 0;                        // steps so far; may pass 32 bits, where its low ones go on as they should
      int c = 0;                             // items with steps so far
      bool ok = true;
      for (int it = it_first; it < n_items && ok; it += it_step) {
        const Item i = item_at(it);
        if (i.steps == 0) continue;
        const int slot = c & 1;
        const int q_at = i.b * x.q_items, do_at = i.b * p.do_items, kv_at = i.b * x.kv_items;
        if (!mbar_wait(&m_empty[slot], ((c >> 1) & 1) ^ 1u, x.err, abort_flag, 43)) { ok = false; break; }
        mbar_arrive_expect_tx(&m_full[slot], 2 * S::TILE);
        tma_load_3d(smem + 2 * slot * S::TILE, &own0, &m_full[slot], i.h * CRA_HD, i.r0, DKV ? kv_at : q_at);
        tma_load_3d(smem + (2 * slot + 1) * S::TILE, &own1, &m_full[slot], i.h * CRA_HD, i.r0, DKV ? kv_at : do_at);
        ++c;
        int h = DKV ? i.h * x.group : i.h / x.group, t0 = i.t_first;
        for (int j = 0; j < i.steps; ++j, ++n) {
          const int st = n % CRB_STAGES;
          if (!mbar_wait(&empty[st], ((n / CRB_STAGES) & 1) ^ 1u, x.err, abort_flag, 44)) { ok = false; break; }
          mbar_arrive_expect_tx(&full[st], 2 * S::TILE + (DKV ? S::STATS_BYTES : 0));
          uint8_t* dst = smem + S::OFF_STEP + st * 2 * S::TILE;
          tma_load_3d(dst, &step0, &full[st], h * CRA_HD, t0, DKV ? q_at : kv_at);
          tma_load_3d(dst + S::TILE, &step1, &full[st], h * CRA_HD, t0, DKV ? do_at : kv_at);
          if (DKV) {
            const float* src = p.stats + (static_cast<long long>(i.b) * x.H + h) * 2 * p.stats_ld + t0;
            uint8_t* sd = smem + S::OFF_STATS + st * S::STATS_BYTES;
            bulk_load(sd, src, CRB_STEP * 4, &full[st]);
            bulk_load(sd + CRB_STEP * 4, src + p.stats_ld, CRB_STEP * 4, &full[st]);
          }
          t0 = next_t0(i, t0);
          if (DKV && t0 == 0) ++h;
        }
      }
      if (!ok) {   // copies already in flight land long before this (their barriers may never be counted out)
        const uint64_t w0 = globaltimer();
        while (globaltimer() - w0 < 10000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t step_at = smem_u32(smem + S::OFF_STEP), own_at = smem_u32(smem);
      constexpr uint32_t IDESC_ACC = make_idesc(128, CRA_HD, 1u) | IDESC_B_MN;
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) { return mbar_wait(bar, parity, x.err, abort_flag, site); };
      bool ok = true;
      uint32_t n = 0;
      int c = 0, fixes = 0;
      // the step before, whose sums are issued behind the scores of this one
      uint32_t pn = 0;
      int pc = 0, p_halves = 0;
      bool p_any = false, p_first = false, p_last = false;
      auto sums = [&]() -> bool {
        if (!p_any) return true;
        const int st = pn % CRB_STAGES;
        if (!wait(&p_full[pn & 1], (pn >> 1) & 1, 45)) return false;
        if (p_first && !wait(acc_empty, (pc & 1) ^ 1u, 46)) return false;
        tc_fence_after();
        const uint32_t n0 = sw128_mn_desc_lo(step_at + st * 2 * S::TILE, S::TILE), n1 = DKV ? n0 + (S::TILE >> 4) : n0;
        const uint32_t src = tmem + (pn & 1) * CRB_TM_S, acc = tmem + CRB_TM_ACC;
        if (DKV || p.want_dq) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (!TWICE && k >= 4 && p_halves < 2) break;
            const uint32_t a = src + k / 4 * 64 + k % 4 * 8, b = (TWICE ? k % 4 : k) * (2048 >> 4);
            mma_f16_tmem_a_lo<IDESC_ACC>(acc, a, n1 + b, !p_first || k != 0);
            mma_f16_tmem_a_lo<IDESC_ACC>(acc + CRA_HD, a + 32, n0 + b, !p_first || k != 0);
          }
        }
        mma_commit(&empty[st]);
        if (p_last) mma_commit(acc_full);
        p_any = false;
        return true;
      };
      for (int it = it_first; it < n_items && ok; it += it_step) {
        const Item i = item_at(it);
        if (i.steps == 0) continue;
        const int slot = c & 1;
        const uint32_t a0 = sw128_desc_lo(own_at + 2 * slot * S::TILE), a1 = a0 + (S::TILE >> 4);
        ok = wait(&m_full[slot], (c >> 1) & 1, 47);
        int t0 = i.t_first;
        for (int j = 0; j < i.steps && ok; ++j, ++n) {
          const int st = n % CRB_STAGES;
          const int halves = i.step_len - t0 > 64 ? 2 : 1;
          ok = wait(&full[st], (n / CRB_STAGES) & 1, 48);
          // the sums before a ragged step go first: its tiles are cleared when the softmax comes to it
          if (ok && ragged(i, t0)) ok = sums() && wait(fixed, fixes++ & 1, 49);
          if (!ok) break;
          tc_fence_after();
          const uint32_t b0 = sw128_desc_lo(step_at + st * 2 * S::TILE), b1 = b0 + (S::TILE >> 4);
          auto scores = [&](uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (halves == 2) mma_bf16_lo<make_idesc(128, 128, 1u)>(d, a + 2 * k, b + 2 * k, k != 0);
              else mma_bf16_lo<make_idesc(128, 64, 1u)>(d, a + 2 * k, b + 2 * k, k != 0);
          };
          // the sums that read this S buffer were issued before, and run before
          scores(tmem + (n & 1) * CRB_TM_S, a0, b0);
          if (n > 0) ok = wait(d_free, (n - 1) & 1, 50);
          if (!ok) break;
          tc_fence_after();
          scores(tmem + CRB_TM_D, a1, b1);
          mma_commit(s_full);
          if (j + 1 == i.steps) mma_commit(&m_empty[slot]);
          ok = sums();
          p_any = true;
          pn = n;
          pc = c;
          p_halves = halves;
          p_first = j == 0;
          p_last = j + 1 == i.steps;
          t0 = next_t0(i, t0);
        }
        ++c;
      }
      if (ok) sums();
      mma_commit(mma_done);
      mbar_drain(mma_done, 0);
    }
  } else {
    const int half = (warp - 2) >> 3;                // this warp's 64 columns of a step
    const int quarter = warp & 3;
    const int sub = ((warp - 2) >> 2) & 1;
    const int lane_base = quarter * 32 + sub * 16;
    const uint32_t lane_off = static_cast<uint32_t>(lane_base) << 16;
    const int t = lane & 3, cq = 2 * t;
    const int ra = lane_base + (lane >> 2);          // this thread's own rows: ra and ra + 8
    float2* const b_part = reinterpret_cast<float2*>(smem + S::OFF_B);
    const uint64_t c2 = f32x2_pack(x.c, x.c);
    auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, x.err, abort_flag, site));
    };
    bool ok = true;
    uint32_t n = 0;
    int c = 0;

    // results of an item: DKV: the first half's warps store dv, the second's dk; else 32 columns of dq - b' M each
    auto finish = [&](const Item& i, int ci, float za, float zb) -> bool {
      const bool any = i.steps > 0;
      uint32_t v[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) v[k] = 0;
      float2 ba = {}, bb = {};
      // a split's 32 columns of M and dQ, for the join behind the roles
      auto share = [&](const uint32_t (&m)[16], const uint32_t (&d)[16]) {
        float* at = reinterpret_cast<float*>(smem + S::OFF_STEP) + ra * S::SHARE_LD + half * 32 + cq;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float* w = at + (k & 1) * 8 * S::SHARE_LD + k / 2 * 8;
          *reinterpret_cast<float2*>(w) = make_float2(__uint_as_float(m[2 * k]), __uint_as_float(m[2 * k + 1]));
          *reinterpret_cast<float2*>(w + CRA_HD) = make_float2(__uint_as_float(d[2 * k]), __uint_as_float(d[2 * k + 1]));
        }
      };
      if (any) {
        if (!DKV) {
          if (!wait(b_full, ci & 1, 51)) return false;
          const float2* b_of = b_part + (ci & 1) * 2 * CRB_M + ra;
          ba = make_float2(b_of[0].x + b_of[CRB_M].x, b_of[0].y + b_of[CRB_M].y);
          bb = make_float2(b_of[8].x + b_of[CRB_M + 8].x, b_of[8].y + b_of[CRB_M + 8].y);
        }
        if (!DKV && splits == 1) {
          const long long si = (static_cast<long long>(i.b) * x.H + i.h) * 2 * p.stats_ld + p.stats_ld + i.r0 + ra;
          if (half == 0 && t < 2 &&
              in_bounds(x.err, si, 9, static_cast<long long>(x.batch) * x.H * 2 * p.stats_ld, SITE_CROSS_STATS))
            p.stats[si + 8 * t] = i.r0 + ra + 8 * t >= i.own_len ? 0.0f : t ? zb - bb.x : za - ba.x;         // -delta
        }
        if (!wait(acc_full, ci & 1, 52)) return false;
        tc_fence_after();
        const uint32_t acc = tmem + lane_off + CRB_TM_ACC;
        if (DKV) {
          tmem_ld_16x256b_x8(acc + half * CRA_HD, v);
        } else if (p.want_dq) {
          uint32_t m[16], d[16];
          tmem_ld_16x256b_x4(acc + half * 32, m);
          tmem_ld_16x256b_x4(acc + CRA_HD + half * 32, d);
          tmem_ld_wait();
          if (splits > 1) share(m, d);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            v[k] = __float_as_uint(fmaf(-(k & 2 ? bb.y : ba.y), __uint_as_float(m[k]), __uint_as_float(d[k])));
        }
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty);
      }
      if (!DKV && splits > 1) {
        if (!any) {
          const uint32_t zeros[16] = {};
          share(zeros, zeros);
        }
        if (half == 0 && t == 0) {
          float* b_at = reinterpret_cast<float*>(smem + S::OFF_STEP) + ra * S::SHARE_LD + 2 * CRA_HD;
          *reinterpret_cast<float2*>(b_at) = ba;
          *reinterpret_cast<float2*>(b_at + 8 * S::SHARE_LD) = bb;
        }
        return true;
      }
      if (!DKV && !p.want_dq) return true;
      __nv_bfloat16* const dst = !DKV ? p.dq : half ? p.dk : p.dv;
      const float k = DKV && half == 0 ? 1.0f : (DKV ? i.own_len : i.step_len) == 1 ? 0.0f : x.scale;
      const long long ld = static_cast<long long>(heads) * CRA_HD;
      const long long extent = static_cast<long long>(x.batch) * own_T * ld;
#pragma unroll
      for (int e8 = 0; e8 < 2; ++e8) {
        const int r = i.r0 + ra + 8 * e8;
        const bool there = any && r < i.own_len;
#pragma unroll
        for (int q = 0; q < (DKV ? 2 : 1); ++q) {
          uint32_t w[4];
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const int e = 16 * q + 4 * kk + 2 * e8;
            w[kk] = there ? pack_bf16(k * __uint_as_float(v[e]), k * __uint_as_float(v[e + 1])) : 0u;
          }
          const uint4 u = quad_transpose(w[0], w[1], w[2], w[3], t);
          const long long o = (static_cast<long long>(i.b) * own_T + r) * ld + i.h * CRA_HD + 32 * (DKV ? q : half) + 8 * t;
          if (r < own_T && in_bounds(x.err, o, 8, extent, SITE_CROSS_OUT)) *reinterpret_cast<uint4*>(dst + o) = u;
        }
      }
      return true;
    };

    Item last;                                       // the item whose results are still to be stored
    int last_c = -1;
    float last_za = 0.0f, last_zb = 0.0f;
    for (int it = it_first; it < n_items && ok; it += it_step) {
      const Item i = item_at(it);
      float la = 0.0f, lb = 0.0f, za = 0.0f, zb = 0.0f;      // rows' -lse / scale and -delta
      if (!DKV && i.r0 < i.own_len && i.step_len > 0) {
        const float2 sa = cross_row_stats(p, i.b, i.h, i.r0 + ra, i.r0 + ra < i.own_len, t);
        const float2 sb = cross_row_stats(p, i.b, i.h, i.r0 + ra + 8, i.r0 + ra + 8 < i.own_len, t);
        la = sa.x;
        lb = sb.x;
        za = sa.y;
        zb = sb.y;
        // every row of a tile has an entry; -delta of one is written when b is known (split: corrected then)
        const long long si = (static_cast<long long>(i.b) * x.H + i.h) * 2 * p.stats_ld + i.r0 + ra;
        if (half == 0 && t < 2 && rank == 0 &&
            in_bounds(x.err, si, p.stats_ld + 9, static_cast<long long>(x.batch) * x.H * 2 * p.stats_ld, SITE_CROSS_STATS)) {
          p.stats[si + 8 * t] = t ? lb : la;
          if (splits > 1) p.stats[si + p.stats_ld + 8 * t] = t ? zb : za;
        }
      }
      if (!DKV && half == 0 && it + it_step < n_items) {     // the next item's rows of out, for its statistics
        const Item next = item_at(it + it_step);
        const int row = next.r0 + lane_base + lane;
        if (lane < 16 && row < next.own_len)
          prefetch_l2(x.out + (static_cast<long long>(next.b) * x.Tq + row) * x.H * CRA_HD + next.h * CRA_HD);
      }
      if (i.steps == 0) {
        ok = finish(i, 0, 0.0f, 0.0f);
        continue;
      }
      uint64_t ba2 = 0, bb2 = 0;                     // this thread's share of b of the two rows
      float bra = 0.0f, brb = 0.0f;                  // this thread's share of b'
      int t0 = i.t_first;
      for (int j = 0; j < i.steps; ++j, ++n) {
        const int st = n % CRB_STAGES;
        const int rows = i.step_len - t0;            // that take part, in this step
        if (DKV || ragged(i, t0)) {                  // the statistics come with the step's tiles
          if (!wait(&full[st], (n / CRB_STAGES) & 1, 53)) { ok = false; break; }
        }
        if (ragged(i, t0)) {
          uint4* tile = reinterpret_cast<uint4*>(smem + S::OFF_STEP + st * 2 * S::TILE);
          for (int k = rows * 8 + static_cast<int>(threadIdx.x) - 64; k < CRB_STEP * 8; k += 32 * CRB_WARPS)
            tile[k] = tile[k + S::TILE / 16] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(fixed);
        }
        if (!wait(s_full, n & 1, 54)) { ok = false; break; }
        tc_fence_after();
        // TWICE: the second half's warps form the same P and dS, and store what rounding them left
        const int cols = TWICE ? 0 : 64 * half;      // this warp's first column
        if (rows > cols) {
          // s[4k], s[4k+1]: own row ra, columns 8k + cq, + 1; s[4k+2], s[4k+3]: row ra + 8
          const uint32_t s_tm = tmem + lane_off + (n & 1) * CRB_TM_S;
          uint32_t s[32], d[32];
          tmem_ld_16x256b_x8(s_tm + cols, s);
          tmem_ld_16x256b_x8(tmem + lane_off + CRB_TM_D + cols, d);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(d_free);
          if (!DKV && rows < cols + 64) {
            // keys that take no part: P = 0 from a score of -infinity, and dS = 0
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (cols + 8 * kk + cq + (e & 1) >= rows) s[4 * kk + e] = 0xff800000u;
          }
          const float2* stats = reinterpret_cast<const float2*>(smem + S::OFF_STATS + st * S::STATS_BYTES) + cols / 2 + t;
          const bool rest = TWICE && half;
          uint32_t pw[16], dw[16];
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            uint64_t nl = 0, nd = 0;
            if (DKV) {                               // of the step's rows 8k + cq and + 1
              nl = *reinterpret_cast<const uint64_t*>(stats + 4 * kk);
              nd = *reinterpret_cast<const uint64_t*>(stats + CRB_STEP / 2 + 4 * kk);
            }
#pragma unroll
            for (int e8 = 0; e8 < 2; ++e8) {
              if (!DKV) {
                nl = e8 ? f32x2_pack(lb, lb) : f32x2_pack(la, la);
                nd = e8 ? f32x2_pack(zb, zb) : f32x2_pack(za, za);
              }
              const uint64_t sv = f32x2_pack(__uint_as_float(s[4 * kk + 2 * e8]), __uint_as_float(s[4 * kk + 2 * e8 + 1]));
              const uint64_t dv = f32x2_pack(__uint_as_float(d[4 * kk + 2 * e8]), __uint_as_float(d[4 * kk + 2 * e8 + 1]));
              float a, e;
              f32x2_unpack(f32x2_mul(f32x2_add(sv, nl), c2), a, e);
              a = ex2_approx(a);
              e = ex2_approx(e);
              uint32_t w = pack_bf16(a, e);
              pw[2 * kk + e8] = rest ? pack_bf16_rest(a, e, w) : w;
              const uint64_t ds = f32x2_mul(f32x2_add(dv, nd), f32x2_pack(a, e));
              if (!DKV && !rest) {
                if (e8) bb2 = f32x2_add(bb2, ds);
                else ba2 = f32x2_add(ba2, ds);
              }
              f32x2_unpack(ds, a, e);
              w = pack_bf16(a, e);
              dw[2 * kk + e8] = rest ? pack_bf16_rest(a, e, w) : w;
            }
          }
          // over the 64 columns of S that this warp has read (or that are free); shared columns once all warps have read them
          if (TWICE && !half) {
            if (!wait(d_free, n & 1, 55)) { ok = false; break; }
            tc_fence_after();
          }
          tmem_st_16x128b_x8(s_tm + 64 * half, pw);
          tmem_st_16x128b_x8(s_tm + 64 * half + 32, dw);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[n & 1]);
          if (!DKV) {                                // b', while the products run: 3 % of the backward pass; with mma.sync and ones 11 %
            uint64_t u0 = 0, u1 = 0;
#pragma unroll
            for (int m = 0; m < 16; m += 2) {
              u0 = f32x2_add(u0, f32x2_pack(__uint_as_float(dw[m] << 16), __uint_as_float(dw[m] & 0xffff0000u)));
              u1 = f32x2_add(u1, f32x2_pack(__uint_as_float(dw[m + 1] << 16), __uint_as_float(dw[m + 1] & 0xffff0000u)));
            }
            float y0, y1, y2, y3;
            f32x2_unpack(u0, y0, y1);
            f32x2_unpack(u1, y2, y3);
            bra += y0 + y1;
            brb += y2 + y3;
          }
        } else {
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(d_free);
            mbar_arrive(&p_full[n & 1]);
          }
        }
        if (last_c >= 0) {
          if (!finish(last, last_c, last_za, last_zb)) { ok = false; break; }
          last_c = -1;
        }
        t0 = next_t0(i, t0);
      }
      if (!ok) break;
      if (!DKV) {
        // b of a row: four threads of this warp and four of the other half's
        float ba, bb, y;
        f32x2_unpack(ba2, ba, y);
        ba += y;
        f32x2_unpack(bb2, bb, y);
        bb += y;
        ba += __shfl_xor_sync(0xffffffffu, ba, 1);
        bb += __shfl_xor_sync(0xffffffffu, bb, 1);
        ba += __shfl_xor_sync(0xffffffffu, ba, 2);
        bb += __shfl_xor_sync(0xffffffffu, bb, 2);
        bra += __shfl_xor_sync(0xffffffffu, bra, 1);
        brb += __shfl_xor_sync(0xffffffffu, brb, 1);
        bra += __shfl_xor_sync(0xffffffffu, bra, 2);
        brb += __shfl_xor_sync(0xffffffffu, brb, 2);
        float2* b_of = b_part + (c & 1) * 2 * CRB_M + half * CRB_M + ra;
        if (t == 0) {
          b_of[0] = make_float2(ba, bra);
          b_of[8] = make_float2(bb, brb);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b_full);
      }
      last = i;
      last_c = c++;
      last_za = za;
      last_zb = zb;
    }
    if (ok && last_c >= 0) finish(last, last_c, last_za, last_zb);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, CRB_TM_COLS);
  if (DKV || splits == 1) return;
  // the shares of an item's splits, a part of the rows each: dq = scale (sum dQ - (sum b') (sum M)), -delta less b
  cluster_sync();
  const Item i = item_at(it_first);
  const int r0 = CRB_M * rank / splits, r1 = CRB_M * (rank + 1) / splits;
  const long long ld = static_cast<long long>(heads) * CRA_HD;
  for (int k = threadIdx.x; k < (r1 - r0) * (CRA_HD / 4); k += CRB_THREADS) {
    const int r = r0 + k / (CRA_HD / 4), e = k % (CRA_HD / 4) * 4, row = i.r0 + r;
    if (row >= own_T) break;
    const uint32_t at = smem_u32(smem + S::OFF_STEP) + r * S::SHARE_LD * 4;
    float4 m[CRA_MAX_SPLITS], d[CRA_MAX_SPLITS], b[CRA_MAX_SPLITS];
#pragma unroll
    for (int q = 0; q < CRA_MAX_SPLITS; ++q) {
      if (q >= splits) continue;
      const uint32_t from = cluster_map(at, q);
      m[q] = ld_cluster_f32x4(from + e * 4);
      d[q] = ld_cluster_f32x4(from + (CRA_HD + e) * 4);
      b[q] = ld_cluster_f32x4(from + 2 * CRA_HD * 4);
    }
#pragma unroll
    for (int q = 1; q < CRA_MAX_SPLITS; ++q) {
      if (q >= splits) continue;
      m[0] = make_float4(m[0].x + m[q].x, m[0].y + m[q].y, m[0].z + m[q].z, m[0].w + m[q].w);
      d[0] = make_float4(d[0].x + d[q].x, d[0].y + d[q].y, d[0].z + d[q].z, d[0].w + d[q].w);
      b[0].x += b[q].x;
      b[0].y += b[q].y;
    }
    const bool there = row < i.own_len;
    const long long si = (static_cast<long long>(i.b) * x.H + i.h) * 2 * p.stats_ld + p.stats_ld + row;
    if (e == 0 && there && in_bounds(x.err, si, 1, static_cast<long long>(x.batch) * x.H * 2 * p.stats_ld, SITE_CROSS_STATS))
      p.stats[si] -= b[0].x;
    if (!p.want_dq) continue;
    const float f = -b[0].y, c = i.step_len == 1 ? 0.0f : x.scale;
    const uint32_t w0 = pack_bf16(c * fmaf(f, m[0].x, d[0].x), c * fmaf(f, m[0].y, d[0].y));
    const uint32_t w1 = pack_bf16(c * fmaf(f, m[0].z, d[0].z), c * fmaf(f, m[0].w, d[0].w));
    const long long o = (static_cast<long long>(i.b) * own_T + row) * ld + i.h * CRA_HD + e;
    if (in_bounds(x.err, o, 4, static_cast<long long>(x.batch) * own_T * ld, SITE_CROSS_OUT))
      *reinterpret_cast<uint2*>(p.dq + o) = there ? make_uint2(w0, w1) : make_uint2(0u, 0u);
  }
  cluster_sync();                                  // the others have read this CTA's share
}

}  // namespace wb
