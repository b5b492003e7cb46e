// The four contractions of a vocabulary head's loss and its gradient, on tcgen05 (sm_103a).
//
// n rows of hidden states x (bf16 [n, d], compacted: rows that take no part are gone), a projection
// matrix w (bf16 [V, d]), logits s = x w^T that are never stored:
//   HEAD_LSE      s tile by tile -> per row and tile (max, sum 2^((s - max) c)) and the targets' logits
//   HEAD_DLOGITS  s again for a piece of the vocabulary -> D = softmax - target, bf16 [n, piece]
//   HEAD_GRADS    for the piece, in one launch: D w, added to float32 slabs of dx, and D^T x', the
//                 piece's rows of dw
// D stays a piece (the workspace bounds it), so memory does not grow with n V; recomputing s costs one
// of the four products.  All operands are read where they lie: w and x' as MN-major B tiles, D as an
// MN-major A tile for dw, so nothing is transposed in memory.
//
// Two forms.  PAIR: two CTAs (a cluster, one SM each) make one tile of 256 rows x up to 256 columns: each
// loads 128 rows of A and half of B's columns: 32 KB per 64 of k, which an SM's 64 bytes a clock from L2
// bring in the 512 clocks of its MMAs.  Single: one CTA, 128 rows: 48 KB for the same MMAs.  The tensor pipe
// was active for 75 to 78 % (pair) and 73 % (single) of the SMs' time in HEAD_DLOGITS, 81 % and 72 to 79 % in
// the gradient products (3000 x 1280 against 20000).  The single form has the finer rows, starts sooner and wins
// where a product is short.
// Per CTA, as in the other GEMMs of this library: warp 0 lane 0 loads a ring of stages with TMA; warp 1
// lane 0 (of the pair's first CTA) issues the MMAs into one of two 256-column TMEM accumulators; warps 2-17
// run the epilogue of the tile before on their CTA's 128 rows: warp w has TMEM lane quarter w % 4 and a
// quarter of the columns.  Every wait is bounded.  The rows that take part are only known on the device
// (*n_rows); all roles read them and walk the same tiles.
#pragma once
#include "gemm.cuh"

namespace wb {

enum HeadKind : int { HEAD_LSE, HEAD_DLOGITS, HEAD_GRADS };

constexpr int HEAD_BN = 256, HEAD_BK = 64;   // widest tile, elements of k per stage
constexpr int head_bm(bool pair) { return pair ? 256 : 128; }

// HEAD_LSE stores no tile, only partials: its staging area is the exchange of those, and a stage more fits.
template <int KIND, bool PAIR>
struct HeadSmem {
  static constexpr int A_BYTES = 128 * HEAD_BK * 2;
  static constexpr int B_BYTES = (PAIR ? HEAD_BN / 2 : HEAD_BN) * HEAD_BK * 2;
  static constexpr int MN_BLOCK = 64 * HEAD_BK * 2;      // 64 M / N elements x 64 k of an MN-major tile
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = (PAIR ? 5 : 3) + (KIND == HEAD_LSE);
  // 32 rows x 128 bytes per epilogue warp (128-byte swizzle); with rows of 64 bytes and a stage more the
  // backward pass of 10752 x 1280 took 2.80 ms against 2.71
  static constexpr int BOX_BYTES = 32 * 128;
  static constexpr int OFF_EPI = STAGES * STAGE_BYTES;
  static constexpr int OFF_BAR = OFF_EPI + (KIND == HEAD_LSE ? 2 * 4 * 3 * 128 * 4 : GEMM_EPI_WARPS * BOX_BYTES);
  static constexpr int TOTAL = 1024 + OFF_BAR + 512;
};
// Byte offset of 16-byte chunk j of row r in such a box.
__device__ __forceinline__ uint32_t box128_off(int r, int j) { return static_cast<uint32_t>(r * 128 + ((j ^ (r & 7)) << 4)); }
static_assert(HeadSmem<HEAD_GRADS, true>::TOTAL <= 227 * 1024 && HeadSmem<HEAD_LSE, false>::TOTAL <= 227 * 1024 &&
                  HeadSmem<HEAD_GRADS, false>::TOTAL <= 227 * 1024,
              "one CTA per SM");

struct HeadMaps {
  CUtensorMap a0, a1;        // x (LSE, DLOGITS); D for dx (K-major), D for dw (MN-major)
  CUtensorMap b0, b1;        // w (K-major); w for dx (MN-major), x' for dw (MN-major)
  CUtensorMap o0, o1;        // D; slabs of dx, dw
};

struct HeadParams {
  const int* n_rows;         // device: rows that take part, at most m_cap; null: all of them
  int m_cap;                 // rows of the call
  int V, d;
  int v0, vc;                // this piece of the vocabulary (LSE: all of it)
  int bn;                    // columns of a tile, a multiple of 32
  int a_rows;                // rows of a load of x or D: 128, or fewer where the call has fewer (what lies in the
                             // rest of the tile's rows reaches only rows that are not there)
  int panel;                 // column tiles walked together (LSE, DLOGITS)
  int dx_splits;             // GRADS: slabs, 0 without dx
  int want_dw;
  int first_piece;           // dx: store instead of add
  float scale_log2;          // log2(e) / temperature
  // by row of x: its label (cross entropy), or its source row and the number of its sorted entries
  const int64_t* labels;     // LSE without compaction: the labels themselves
  const int* row_tgt;        // null without compaction: the row itself
  const int* row_cnt;        // null: cross entropy
  const int* tgt_idx;        // distillation: [source row][k], sorted
  const float* tgt_p;
  int k;
  float label_p;             // cross entropy: weight of the label
  float smooth;              // what every column's target has on top (label smoothing / V)
  // LSE out
  float2* part;              // [column tile][part_ld]: (max logit, sum of 2^((logit - max) scale_log2))
  float* part_sum;           // [column tile][part_ld]: plain sum of logits, null without smoothing
  long long part_ld;
  float* tgt_s;              // [row][k]: logits at the targets
  int dl_cols;               // columns of D's buffer
  // DLOGITS in
  const float* row_lse;      // by compact row
  float inv_t;
  // dw
  const float* g_scale;      // device scalar that x' was divided by
  float out_scale;
  uint32_t* err;
};

template <int KIND, bool PAIR>
__global__ void __launch_bounds__(GEMM_THREADS, 1)
    head_gemm_kernel(const __grid_constant__ HeadMaps maps, const __grid_constant__ HeadParams p) {
  using S = HeadSmem<KIND, PAIR>;
  constexpr int BM = head_bm(PAIR);
  constexpr int STAGES = S::STAGES;
  constexpr bool LOGITS = KIND != HEAD_GRADS;
  constexpr uint32_t TMEM_COLS = 2 * HEAD_BN;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base_u32 - smem_u32(smem_raw));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);   // [STAGES], the first CTA's count both
  uint64_t* empty = full + STAGES;                                   // [STAGES]
  uint64_t* tfull = empty + STAGES;                                  // [2]
  uint64_t* tempty = tfull + 2;                                      // [2], the first CTA's count both
  uint64_t* red_full = tempty + 2;                                   // [2][4]: LSE partials of a quarter
  uint64_t* mma_done = red_full + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = warp_id();
  const int lane = lane_id();
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], (PAIR ? 2 : 1) * GEMM_EPI_WARPS);
      for (int q = 0; q < 4; ++q) mbar_init(&red_full[4 * a + q], 3);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (PAIR) tmem_alloc_pair(tmem_slot, TMEM_COLS);
    else tmem_alloc(tmem_slot, TMEM_COLS);
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();      // the peer's barriers are set up too
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();

  // ---- tiles: the same walk in every role of both CTAs ----
  int n = p.n_rows ? *p.n_rows : p.m_cap;
  n = n < 0 ? 0 : n > p.m_cap ? p.m_cap : n;
  const int bn = p.bn;
  const int row_tiles = n > 0 ? (n + BM - 1) / BM : 1;     // with no rows: one tile of zeros
  const int n_tiles = ((LOGITS ? p.vc : p.d) + bn - 1) / bn;
  const int kb_d = (p.d + HEAD_BK - 1) / HEAD_BK, kb_v = (p.vc + HEAD_BK - 1) / HEAD_BK,
            kb_n = ((n > 0 ? n : 1) + HEAD_BK - 1) / HEAD_BK;
  const long long dw_tiles = LOGITS || !p.want_dw ? 0 : static_cast<long long>((p.vc + BM - 1) / BM) * n_tiles;
  const long long dx_tiles = static_cast<long long>(row_tiles) * n_tiles;
  const long long total = LOGITS ? dx_tiles : dw_tiles + dx_tiles * p.dx_splits;
  struct Tile {
    int mt, nt, split, kb0, kb1;
    bool dw;
  };
  auto tile_at = [&](long long t) -> Tile {
    Tile r;
    r.split = 0;
    r.kb0 = 0;
    r.dw = false;
    if (LOGITS) {
      // panels of column tiles, all rows through each: a panel of w is read once from memory and the
      // rows again from L2 (they are the smaller side)
      const long long per_panel = static_cast<long long>(row_tiles) * p.panel;
      const int pn = static_cast<int>(t / per_panel);
      const long long q = t - pn * per_panel;
      const int left = n_tiles - pn * p.panel;
      const int w = left < p.panel ? left : p.panel;
      r.mt = static_cast<int>(q / w);
      r.nt = pn * p.panel + static_cast<int>(q % w);
      r.kb1 = kb_d;
    } else if (t < dw_tiles) {
      r.dw = true;
      r.mt = static_cast<int>(t / n_tiles);
      r.nt = static_cast<int>(t % n_tiles);
      r.kb1 = kb_n;
    } else {
      const long long u = t - dw_tiles;
      r.split = static_cast<int>(u / dx_tiles);
      const long long q = u - r.split * dx_tiles;
      r.mt = static_cast<int>(q / n_tiles);
      r.nt = static_cast<int>(q % n_tiles);
      r.kb0 = static_cast<int>(static_cast<long long>(kb_v) * r.split / p.dx_splits);
      r.kb1 = static_cast<int>(static_cast<long long>(kb_v) * (r.split + 1) / p.dx_splits);
    }
    return r;
  };
  const long long t_first = PAIR ? blockIdx.x >> 1 : blockIdx.x, t_step = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (warp == 0) {
    // ------------------------------ TMA producer ---------------------------
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const int half = PAIR ? bn / 2 : bn;         // this CTA's columns of B
      const int mn_loads = (half + 63) / 64;
      const uint32_t b_bytes = LOGITS ? half * 128 : mn_loads * S::MN_BLOCK;
      auto load = [&](uint8_t* dst, const CUtensorMap* m, int stg, int c0, int c1) {
        if (PAIR) tma_load_2d_pair(dst, m, cluster_addr(&full[stg], 0), c0, c1);
        else tma_load_2d(dst, m, &full[stg], c0, c1);
      };
      for (long long t = t_first; t < total && ok; t += t_step) {
        const Tile tl = tile_at(t);
        const int row0 = tl.mt * BM + static_cast<int>(rank) * 128;
        const int col0 = tl.nt * bn + static_cast<int>(rank) * half;
        for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, p.err, abort_flag, 24)) { ok = false; break; }
          if (rank == 0)
            mbar_arrive_expect_tx(&full[stage], (PAIR ? 2 : 1) * ((tl.dw ? S::A_BYTES : p.a_rows * 128) + b_bytes));
          uint8_t* sa = smem + stage * S::STAGE_BYTES;
          uint8_t* sb = sa + S::A_BYTES;
          if (LOGITS) {
            load(sa, &maps.a0, stage, kb * HEAD_BK, row0);
            load(sb, &maps.b0, stage, kb * HEAD_BK, p.v0 + col0);
          } else if (tl.dw) {
            for (int j = 0; j < 2; ++j)
              load(sa + j * S::MN_BLOCK, &maps.a1, stage, row0 + 64 * j, kb * HEAD_BK);
            for (int j = 0; j < mn_loads; ++j)
              load(sb + j * S::MN_BLOCK, &maps.b1, stage, col0 + 64 * j, kb * HEAD_BK);
          } else {
            load(sa, &maps.a0, stage, kb * HEAD_BK, row0);
            for (int j = 0; j < mn_loads; ++j)
              load(sb + j * S::MN_BLOCK, &maps.b0, stage, col0 + 64 * j, p.v0 + kb * HEAD_BK);
          }
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {  // copies already in flight land long before this (their barrier may never be counted out)
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 10000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer -----------------------------
    if (lane == 0 && rank == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int local = 0;
      auto commit = [&](uint64_t* bar) {
        if (PAIR) mma_commit_pair(bar);
        else mma_commit(bar);
      };
      const uint32_t idesc0 = make_idesc(BM, bn, 1u) | (LOGITS ? 0u : IDESC_B_MN);
      for (long long t = t_first; t < total && ok; t += t_step, ++local) {
        const Tile tl = tile_at(t);
        const int acc = local & 1;
        if (!mbar_wait(&tempty[acc], ((local >> 1) & 1) ^ 1u, p.err, abort_flag, 25)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * HEAD_BN;
        const uint32_t idesc = idesc0 | (tl.dw ? IDESC_A_MN : 0u);
        for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, p.err, abort_flag, 26)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * S::STAGE_BYTES);
          const uint32_t sb = sa + S::A_BYTES;
          // a descriptor advances by the byte offset / 16 (addresses stay below 256 KB): K-major 32 bytes a
          // K16 step, MN-major 2048
          const uint64_t ad = tl.dw ? sw128_mn_desc(sa, S::MN_BLOCK) : sw128_desc(sa);
          const uint64_t bd = LOGITS ? sw128_desc(sb) : sw128_mn_desc(sb, S::MN_BLOCK);
          const uint64_t a_step = tl.dw ? 128 : 2;
          constexpr uint64_t b_step = LOGITS ? 2 : 128;
#pragma unroll
          for (int k = 0; k < HEAD_BK / 16; ++k)
            if (PAIR) mma_bf16_pair(d_tmem, ad + k * a_step, bd + k * b_step, idesc, kb != tl.kb0 || k != 0);
            else mma_bf16(d_tmem, ad + k * a_step, bd + k * b_step, idesc, kb != tl.kb0 || k != 0);
          commit(&empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (ok) commit(&tfull[acc]);
      }
      commit(mma_done);
    }
  } else {
    // ------------------------------- epilogue ------------------------------
    const int ew = warp - 2;
    const int quarter = warp & 3;                // TMEM lane quarter this warp may access
    const int cg = ew >> 2;                      // column group
    // its chunks of 32 columns, 0 to 2: LSE an even share, the others 64 columns or none
    const int ch0 = KIND == HEAD_LSE ? bn / 32 * cg / 4 : min(2 * cg, bn / 32);
    const int ch1 = KIND == HEAD_LSE ? bn / 32 * (cg + 1) / 4 : min(2 * cg + 2, bn / 32);
    uint8_t* const box = smem + S::OFF_EPI + ew * S::BOX_BYTES;
    auto box_free = [&]() {                      // its last store has read it
      if (lane == 0) bulk_wait_read0();
      __syncwarp();
    };
    // LSE: (max, sum, plain sum) of a warp's columns for the quarter's first warp, two tiles deep
    float* red = reinterpret_cast<float*>(smem + S::OFF_EPI);        // [2][4 quarters][3][4 groups][32]
    auto release = [&](int a) {                  // one lane a warp: this warp has read accumulator a
      if (PAIR) mbar_arrive_cluster(cluster_addr(&tempty[a], 0));
      else mbar_arrive(&tempty[a]);
    };
    const float c = p.scale_log2;
    const float g_out = KIND == HEAD_GRADS && p.want_dw ? *p.g_scale * p.out_scale : 1.0f;
    bool ok = true;
    int local = 0;
    for (long long t = t_first; t < total && ok; t += t_step, ++local) {
      const Tile tl = tile_at(t);
      const int acc = local & 1;
      const uint32_t acc_phase = (local >> 1) & 1;
      const int m0 = tl.mt * BM + static_cast<int>(rank) * 128 + quarter * 32;   // first row of this warp
      const int m = m0 + lane;
      const bool row_ok = m < n;
      const int ncol0 = tl.nt * bn + ch0 * 32;         // first column inside the piece / the width
      // the row's next target at or after this warp's first column, found while the MMAs run
      const int lo = p.v0 + ncol0;
      int pos = 0, cnt = 0, next = 0x7fffffff;
      long long tb = 0;
      float lse = 0.0f, smooth = 0.0f;
      if (LOGITS && row_ok && in_bounds(p.err, m, 1, p.m_cap, SITE_HEAD_ROWS)) {
        if (KIND == HEAD_DLOGITS) {
          lse = p.row_lse[m];
          smooth = p.smooth;
        }
        const long long tl64 = p.labels ? p.labels[m] : p.row_tgt ? p.row_tgt[m] : m;
        const int tgt = tl64 < 0 || tl64 > 0x7ffffffe ? -1 : static_cast<int>(tl64);
        if (!p.row_cnt) {
          if (tgt >= lo && tgt < p.V) next = tgt;
        } else if (in_bounds(p.err, tgt, 1, p.m_cap, SITE_HEAD_ROWS)) {
          tb = static_cast<long long>(tgt) * p.k;
          cnt = max(p.row_cnt[m], 0);
          int hi = cnt;
          while (pos < hi) {
            const int mid = (pos + hi) >> 1;
            if (p.tgt_idx[tb + mid] < lo) pos = mid + 1;
            else hi = mid;
          }
          if (pos < cnt) next = p.tgt_idx[tb + pos];
        }
      }
      // the same answer in all lanes: the loads from TMEM are a whole warp's
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], acc_phase, p.err, abort_flag, 27))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * HEAD_BN;

      if constexpr (KIND == HEAD_LSE) {
        float mx = -INFINITY, l = 0.0f, sum = 0.0f;
        for (int ch = ch0; ch < ch1; ++ch) {
          const int n0 = tl.nt * bn + ch * 32;
          if (n0 >= p.vc) break;
          float v[32];
          tmem_ld32(t_row + ch * 32, v);
          tmem_ld_wait();
          // targets in these 32 columns are rare: one column at a time, read again for all lanes
          while (true) {
            const unsigned pend = __ballot_sync(0xffffffffu, next < n0 + 32);
            if (!pend) break;
            const int col = __shfl_sync(0xffffffffu, next, __ffs(pend) - 1) - n0;
            const float s = tmem_ld1(t_row + ch * 32 + col);
            tmem_ld_wait();
            if (next - n0 == col) {
              const long long ti = static_cast<long long>(m) * p.k + pos;
              if (in_bounds(p.err, ti, 1, static_cast<long long>(p.m_cap) * p.k, SITE_HEAD_TARGET)) p.tgt_s[ti] = s;
              ++pos;
              next = pos < cnt ? p.tgt_idx[tb + pos] : 0x7fffffff;
            }
          }
          if (n0 + 32 > p.vc) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (n0 + i >= p.vc) v[i] = -INFINITY;
          }
          if (p.part_sum) {
#pragma unroll
            for (int i = 0; i < 32; ++i) sum += n0 + i < p.vc ? v[i] : 0.0f;
          }
          float x0 = fmaxf(v[0], v[1]), x1 = fmaxf(v[2], v[3]);
#pragma unroll
          for (int i = 4; i < 32; i += 4) {
            x0 = fmax3(x0, v[i], v[i + 1]);
            x1 = fmax3(x1, v[i + 2], v[i + 3]);
          }
          const float mn = fmaxf(mx, fmaxf(x0, x1));
          const float mo = mn == -INFINITY ? 0.0f : mn;     // columns that are all -inf add nothing
          // the difference first, then the scale: it is never positive.  (In one operation, v c - round(max c), what the
          // rounding leaves of large logits is an exponent: 32 entries at -1e30 made a sum of infinity.)
          float s0 = 0.0f, s1 = 0.0f;
          const uint64_t c2 = f32x2_pack(c, c), n2 = f32x2_pack(-mo, -mo);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float a, b;
            f32x2_unpack(f32x2_mul(f32x2_add(f32x2_pack(v[i], v[i + 1]), n2), c2), a, b);
            s0 += ex2_approx(a);
            s1 += ex2_approx(b);
          }
          l = l * ex2_approx((mx - mo) * c) + (s0 + s1);
          mx = mn;
        }
        float* r3 = red + ((acc * 4 + quarter) * 3) * 128;    // [3][4][32]
        if (cg != 0) {
          tc_fence_before();
          r3[cg * 32 + lane] = mx;
          r3[128 + cg * 32 + lane] = l;
          r3[256 + cg * 32 + lane] = sum;
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&red_full[4 * acc + quarter]);
            release(acc);
          }
        } else {
          if (!__all_sync(0xffffffffu, mbar_wait(&red_full[4 * acc + quarter], acc_phase, p.err, abort_flag, 28))) {
            ok = false;
            break;
          }
          float mm = mx;
#pragma unroll
          for (int q = 1; q < 4; ++q) mm = fmaxf(mm, r3[q * 32 + lane]);
          const float mo = mm == -INFINITY ? 0.0f : mm;
          l *= ex2_approx((mx - mo) * c);
#pragma unroll
          for (int q = 1; q < 4; ++q) {
            l += r3[128 + q * 32 + lane] * ex2_approx((r3[q * 32 + lane] - mo) * c);
            sum += r3[256 + q * 32 + lane];
          }
          // the accumulator goes back only now: the tile after next then finds the exchange area read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) release(acc);
          const long long pi = static_cast<long long>(tl.nt) * p.part_ld + m;
          if (row_ok && in_bounds(p.err, pi, 1, static_cast<long long>(n_tiles) * p.part_ld, SITE_HEAD_PART)) {
            p.part[pi] = make_float2(mm, l);
            if (p.part_sum) p.part_sum[pi] = sum;
          }
        }
      } else {
        for (int ch = ch0; ch < ch1; ++ch) {
          const int n0 = tl.nt * bn + ch * 32;
          float v[32];
          tmem_ld32(t_row + ch * 32, v);
          tmem_ld_wait();
          if (ch == ch1 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) release(acc);
          }
          if (KIND == HEAD_GRADS && !tl.dw) {
            if (n0 >= p.d || m0 >= p.m_cap) continue;
            if (tl.kb0 == tl.kb1) {          // a short last piece can leave a split without any k
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0.0f;
            }
            box_free();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(box + box128_off(lane, j)) =
                  make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (p.first_piece) tma_store_3d(&maps.o0, box, n0, m0, tl.split);
              else tma_reduce_add_3d(&maps.o0, box, n0, m0, tl.split);
              bulk_commit();
            }
            continue;
          }
          if constexpr (KIND == HEAD_DLOGITS) {
            // s / T is rounded before the difference: it is then never above the lse that the forward pass rounded from the
            // same sums (as a packed pair the product was measured to be fused with the difference, hence single ones);
            // and no softmax is above 1, however far rounding puts a large logit (a NaN stays).  Against one fused step:
            // 77 x 384 both ways 61.5 us / 61.1, 14336 x 1280 the same within the noise
            constexpr float LOG2E = 1.4426950408889634f;
            const uint64_t l2 = f32x2_pack(-lse, -lse), e2 = f32x2_pack(LOG2E, LOG2E);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float a, b;
              f32x2_unpack(f32x2_mul(f32x2_add(f32x2_pack(__fmul_rn(v[i], p.inv_t), __fmul_rn(v[i + 1], p.inv_t)), l2), e2), a, b);
              v[i] = ex2_approx(min_nan(a, 0.0f)) - smooth;
              v[i + 1] = ex2_approx(min_nan(b, 0.0f)) - smooth;
            }
            const int end = p.v0 + n0 + 32;
            while (__any_sync(0xffffffffu, next < end)) {
              if (next < end) {
                const int col = next - (end - 32);
                const float pt = p.tgt_p ? p.tgt_p[tb + pos] : p.label_p;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (i == col) v[i] -= pt;
                ++pos;
                next = pos < cnt ? p.tgt_idx[tb + pos] : 0x7fffffff;
              }
            }
            // rows and columns outside are zeros: they are factors of the products that follow
            if (!row_ok || end > p.V) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!row_ok || p.v0 + n0 + i >= p.V) v[i] = 0.0f;
            }
            if (m0 >= kb_n * HEAD_BK) continue;     // past the rows that dw's sum runs over
          } else {                                        // dw
            if (p.v0 + m0 >= p.V) continue;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= g_out;
          }
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
          // two chunks fill the box; the store clips what lies past the width
          if (ch == ch0) box_free();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(box + box128_off(lane, 4 * (ch - ch0) + j)) =
                make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
          if (ch + 1 < ch1) continue;
          fence_proxy_async_smem();
          __syncwarp();
          const int b0 = tl.nt * bn + ch0 * 32;
          if (lane == 0 && b0 < (KIND == HEAD_DLOGITS ? p.dl_cols : p.d)) {
            if (KIND == HEAD_DLOGITS) tma_store_2d(&maps.o0, box, b0, m0);
            else tma_store_2d(&maps.o1, box, b0, p.v0 + m0);
            bulk_commit();
          }
        }
        if (ch0 == ch1) {                         // a narrow tile: no column for this warp
          __syncwarp();
          if (lane == 0) release(acc);
        }
      }
    }
    if (lane == 0) bulk_wait0();   // stores complete before the CTA (and its smem) goes away
  }

  tc_fence_before();
  __syncthreads();
  // every MMA is done and has signalled this CTA's barriers (they signal in order); then the peer's
  // arrivals here are over too
  if (threadIdx.x == 32) mbar_drain(mma_done, 0);
  __syncthreads();
  if (PAIR) cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    if (PAIR) tmem_dealloc_pair(tmem_base, TMEM_COLS);
    else tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

}  // namespace wb
