// The four contractions of a vocabulary head's loss and its gradient, on tcgen05 (sm_103a).
//
// n rows of hidden states x (bf16 [n, d], compacted: rows that take no part are gone), a projection
// matrix w (bf16 [V, d]), logits s = x w^T that are never stored:
//   HEAD_LSE      s tile by tile -> per row and tile (max, sum 2^(s c - max)) and the targets' logits
//   HEAD_DLOGITS  s again for a piece of the vocabulary -> D = softmax - target, bf16 [n, piece]
//   HEAD_DX       D w      for the piece, added to float32 slabs
//   HEAD_DW       D^T x'   for the piece's rows of dw
// D stays a piece (the workspace bounds it), so memory does not grow with n V; recomputing s costs one
// of the four products.  All three operands are read where they lie: w and x' as MN-major B tiles,
// D as an MN-major A tile for dw, so nothing is transposed in memory.
//
// Roles as in the other GEMMs of this library: warp 0 lane 0 loads a ring of 4 stages with TMA
// (128 x 64 of A, 64 x 256 of B), warp 1 lane 0 issues the MMAs into one of two 256-column TMEM
// accumulators, warps 2-17 run the epilogue of the tile before: warp w has TMEM lane quarter w % 4 and
// 64 of the 256 columns.  Every wait is bounded.  The rows that take part are only known on the
// device (*n_rows); all roles read them and walk the same tiles.
#pragma once
#include "gemm.cuh"

namespace wb {

enum HeadKind : int { HEAD_LSE, HEAD_DLOGITS, HEAD_DX, HEAD_DW };

constexpr int HEAD_BM = 128, HEAD_BN = 256, HEAD_BK = 64;

struct HeadSmem {
  static constexpr int A_BYTES = HEAD_BM * HEAD_BK * 2;
  static constexpr int B_BYTES = HEAD_BN * HEAD_BK * 2;
  static constexpr int MN_BLOCK = 64 * HEAD_BK * 2;      // 64 M / N elements x 64 k of an MN-major tile
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = 4;
  static constexpr int BOX_BYTES = 32 * 64;              // 32 rows x 64 bytes per epilogue warp (64-byte swizzle)
  static constexpr int OFF_EPI = STAGES * STAGE_BYTES;
  static constexpr int OFF_BAR = OFF_EPI + GEMM_EPI_WARPS * BOX_BYTES;
  static constexpr int TOTAL = 1024 + OFF_BAR + 512;
};
static_assert(HeadSmem::TOTAL <= 227 * 1024, "one CTA per SM");

struct HeadParams {
  const int* n_rows;         // device: rows that take part, at most m_cap
  int m_cap;                 // rows of the call
  int V, d;
  int v0, vc;                // this piece of the vocabulary (LSE: all of it)
  int panel;                 // column tiles walked together (LSE, DLOGITS)
  int k_splits;              // DX: slabs
  int first_piece;           // DX: store instead of add
  float scale_log2;          // log2(e) / temperature
  // targets of compact row i: entries [src(i) * k, + cnt(src(i))) sorted by index, src = row_src
  const int* row_src;
  const int* tgt_idx;
  const float* tgt_p;        // null: every entry weighs label_p
  const int* tgt_cnt;        // null: k entries
  int k;
  float label_p;
  float smooth;              // what every column's target has on top (label smoothing / V)
  // LSE out
  float2* part;              // [column tile][part_ld]: (max, sum) in log2 units
  float* part_sum;           // [column tile][part_ld]: plain sum of logits, null without smoothing
  long long part_ld;
  float* tgt_s;              // [row][k]: logits at the targets
  // DLOGITS in
  const float* lse;          // by source row, natural units
  // DW
  const float* g_scale;      // device scalar that x' was divided by
  float out_scale;
  uint32_t* err;
};

template <int KIND>
__global__ void __launch_bounds__(GEMM_THREADS, 1)
    head_gemm_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                     const __grid_constant__ CUtensorMap omap, const __grid_constant__ HeadParams p) {
  using S = HeadSmem;
  constexpr int STAGES = S::STAGES;
  constexpr bool A_MN = KIND == HEAD_DW, B_MN = KIND == HEAD_DX || KIND == HEAD_DW;
  constexpr uint32_t IDESC =
      make_idesc(HEAD_BM, HEAD_BN, 1u) | (A_MN ? IDESC_A_MN : 0u) | (B_MN ? IDESC_B_MN : 0u);
  constexpr uint32_t TMEM_COLS = 2 * HEAD_BN;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base_u32 - smem_u32(smem_raw));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);   // [STAGES]
  uint64_t* empty = full + STAGES;                                   // [STAGES]
  uint64_t* tfull = empty + STAGES;                                  // [2]
  uint64_t* tempty = tfull + 2;                                      // [2]
  uint64_t* red_full = tempty + 2;                                   // [2][4]: LSE partials of a quarter
  uint64_t* mma_done = red_full + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = warp_id();
  const int lane = lane_id();
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], GEMM_EPI_WARPS);
      for (int q = 0; q < 4; ++q) mbar_init(&red_full[4 * a + q], 3);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();

  // ---- tiles: the same walk in every role ----
  int n = *p.n_rows;
  n = n < 0 ? 0 : n > p.m_cap ? p.m_cap : n;
  const int row_tiles = n > 0 ? (n + HEAD_BM - 1) / HEAD_BM : 1;     // with no rows: one tile of zeros
  const int v_tiles_m = (p.vc + HEAD_BM - 1) / HEAD_BM;
  const int m_tiles = KIND == HEAD_DW ? v_tiles_m : row_tiles;
  const int n_tiles = KIND == HEAD_LSE || KIND == HEAD_DLOGITS ? (p.vc + HEAD_BN - 1) / HEAD_BN
                                                               : (p.d + HEAD_BN - 1) / HEAD_BN;
  const int kb_all = KIND == HEAD_DX ? (p.vc + HEAD_BK - 1) / HEAD_BK
                     : KIND == HEAD_DW ? ((n > 0 ? n : 1) + HEAD_BK - 1) / HEAD_BK
                                       : (p.d + HEAD_BK - 1) / HEAD_BK;
  const int splits = KIND == HEAD_DX ? p.k_splits : 1;
  const long long per_split = static_cast<long long>(m_tiles) * n_tiles;
  const long long total = per_split * splits;
  struct Tile {
    int mt, nt, split, kb0, kb1;
  };
  auto tile_at = [&](long long t) -> Tile {
    Tile r;
    if (KIND == HEAD_LSE || KIND == HEAD_DLOGITS) {
      // panels of column tiles, all rows through each: a panel of w is read once from memory and the
      // rows again from L2 (they are the smaller side)
      const long long per_panel = static_cast<long long>(m_tiles) * p.panel;
      const int pn = static_cast<int>(t / per_panel);
      const long long q = t - pn * per_panel;
      const int left = n_tiles - pn * p.panel;
      const int w = left < p.panel ? left : p.panel;
      r.mt = static_cast<int>(q / w);
      r.nt = pn * p.panel + static_cast<int>(q % w);
      r.split = 0;
    } else {
      r.split = static_cast<int>(t / per_split);
      const long long q = t - r.split * per_split;
      r.mt = static_cast<int>(q / n_tiles);
      r.nt = static_cast<int>(q % n_tiles);
    }
    r.kb0 = static_cast<int>(static_cast<long long>(kb_all) * r.split / splits);
    r.kb1 = static_cast<int>(static_cast<long long>(kb_all) * (r.split + 1) / splits);
    return r;
  };

  if (warp == 0) {
    // ------------------------------ TMA producer ---------------------------
    if (lane == 0) {
      tma_prefetch_desc(&amap);
      tma_prefetch_desc(&bmap);
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, last_parity = 0;
      bool ok = true;
      for (long long t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const Tile tl = tile_at(t);
        for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, p.err, abort_flag, 24)) { ok = false; break; }
          mbar_arrive_expect_tx(&full[stage], S::STAGE_BYTES);
          uint8_t* sa = smem + stage * S::STAGE_BYTES;
          uint8_t* sb = sa + S::A_BYTES;
          if constexpr (A_MN) {
            for (int j = 0; j < HEAD_BM / 64; ++j)
              tma_load_2d(sa + j * S::MN_BLOCK, &amap, &full[stage], tl.mt * HEAD_BM + 64 * j, kb * HEAD_BK);
          } else {
            tma_load_2d(sa, &amap, &full[stage], kb * HEAD_BK, tl.mt * HEAD_BM);
          }
          if constexpr (B_MN) {
            const int k_row = kb * HEAD_BK + (KIND == HEAD_DX ? p.v0 : 0);
            for (int j = 0; j < HEAD_BN / 64; ++j)
              tma_load_2d(sb + j * S::MN_BLOCK, &bmap, &full[stage], tl.nt * HEAD_BN + 64 * j, k_row);
          } else {
            tma_load_2d(sb, &bmap, &full[stage], kb * HEAD_BK, p.v0 + tl.nt * HEAD_BN);
          }
          issued_mask |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {  // let every copy already in flight land before the CTA exits
        for (int s = 0; s < STAGES; ++s)
          if (issued_mask & (1u << s)) mbar_drain(&full[s], (last_parity >> s) & 1u);
      }
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer -----------------------------
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int local = 0;
      for (long long t = blockIdx.x; t < total && ok; t += gridDim.x, ++local) {
        const Tile tl = tile_at(t);
        const int acc = local & 1;
        if (!mbar_wait(&tempty[acc], ((local >> 1) & 1) ^ 1u, p.err, abort_flag, 25)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * HEAD_BN;
        for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, p.err, abort_flag, 26)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * S::STAGE_BYTES);
          const uint32_t sb = sa + S::A_BYTES;
#pragma unroll
          for (int k = 0; k < HEAD_BK / 16; ++k) {
            const uint64_t ad = A_MN ? sw128_mn_desc(sa + k * 2048, S::MN_BLOCK) : sw128_desc(sa + k * 32);
            const uint64_t bd = B_MN ? sw128_mn_desc(sb + k * 2048, S::MN_BLOCK) : sw128_desc(sb + k * 32);
            mma_bf16(d_tmem, ad, bd, IDESC, kb != tl.kb0 || k != 0);
          }
          mma_commit(&empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (ok) mma_commit(&tfull[acc]);
      }
      mma_commit(mma_done);     // no MMA reads smem or writes TMEM any more when the CTA leaves
      mbar_drain(mma_done, 0);
    }
  } else {
    // ------------------------------- epilogue ------------------------------
    constexpr int COLS = HEAD_BN / 4;
    const int ew = warp - 2;
    const int quarter = warp & 3;                // TMEM lane quarter this warp may access
    const int cg = ew >> 2;                      // column group
    uint8_t* box = smem + S::OFF_EPI + ew * S::BOX_BYTES;
    // LSE: (max, sum, plain sum) of this warp's 64 columns for the quarter's first warp, two tiles deep
    float* red = reinterpret_cast<float*>(smem + S::OFF_EPI);        // [2][4 quarters][3][4 groups][32]
    const float c = p.scale_log2;
    const float g_out = KIND == HEAD_DW ? *p.g_scale * p.out_scale : 1.0f;
    bool ok = true;
    int local = 0;
    for (long long t = blockIdx.x; t < total && ok; t += gridDim.x, ++local) {
      const Tile tl = tile_at(t);
      const int acc = local & 1;
      const uint32_t acc_phase = (local >> 1) & 1;
      const int m0 = tl.mt * HEAD_BM + quarter * 32;   // first row of this warp's slab
      const int m = m0 + lane;
      const bool row_ok = m < n;
      const int ncol0 = tl.nt * HEAD_BN + cg * COLS;   // first column inside the piece / the width
      // the row's next target at or after this warp's first column, found while the MMAs run
      const int lo = p.v0 + ncol0;
      int pos = 0, cnt = 0, next = 0x7fffffff, src = 0;
      long long tb = 0;
      float lse2 = 0.0f, smooth = 0.0f;
      if ((KIND == HEAD_LSE || KIND == HEAD_DLOGITS) && row_ok &&
          in_bounds(p.err, m, 1, p.m_cap, SITE_HEAD_ROWS)) {
        src = p.row_src[m];
        if (in_bounds(p.err, src, 1, p.m_cap, SITE_HEAD_ROWS)) {
          tb = static_cast<long long>(src) * p.k;
          cnt = p.tgt_cnt ? p.tgt_cnt[src] : p.k;
          int hi = cnt;
          while (pos < hi) {
            const int mid = (pos + hi) >> 1;
            if (p.tgt_idx[tb + mid] < lo) pos = mid + 1;
            else hi = mid;
          }
          if (pos < cnt) next = p.tgt_idx[tb + pos];
          if (KIND == HEAD_DLOGITS) {
            lse2 = p.lse[src] * 1.4426950408889634f;
            smooth = p.smooth;
          }
        }
      }
      if (!mbar_wait(&tfull[acc], acc_phase, p.err, abort_flag, 27)) { ok = false; break; }
      tc_fence_after();
      const uint32_t t_cols = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * HEAD_BN + cg * COLS;

      if constexpr (KIND == HEAD_LSE) {
        float mx = -INFINITY, l = 0.0f, sum = 0.0f;
#pragma unroll
        for (int ch = 0; ch < COLS / 32; ++ch) {
          const int n0 = ncol0 + ch * 32;
          if (n0 >= p.vc) continue;
          float v[32];
          tmem_ld32(t_cols + ch * 32, v);
          tmem_ld_wait();
          // targets in these 32 columns are rare: one column at a time, read again for all lanes
          const int end = lo + (ch + 1) * 32;
          while (true) {
            const unsigned pend = __ballot_sync(0xffffffffu, next < end);
            if (!pend) break;
            const int col = __shfl_sync(0xffffffffu, next, __ffs(pend) - 1) - lo;
            const float s = tmem_ld1(t_cols + col);
            tmem_ld_wait();
            if (next - lo == col) {
              if (in_bounds(p.err, static_cast<long long>(m) * p.k + pos, 1, static_cast<long long>(p.m_cap) * p.k,
                            SITE_HEAD_TARGET))
                p.tgt_s[static_cast<long long>(m) * p.k + pos] = s;
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
          const float mn = fmaxf(mx, fmaxf(x0, x1) * c);
          const float mo = mn == -INFINITY ? 0.0f : mn;     // columns that are all -inf add nothing
          float s0 = 0.0f, s1 = 0.0f;
          const uint64_t c2 = f32x2_pack(c, c), n2 = f32x2_pack(-mo, -mo);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float a, b;
            fma_f32x2(a, b, v[i], v[i + 1], c2, n2);
            s0 += ex2_approx(a);
            s1 += ex2_approx(b);
          }
          l = l * ex2_approx(mx - mo) + (s0 + s1);
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
            mbar_arrive(&tempty[acc]);
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
          l *= ex2_approx(mx - mo);
#pragma unroll
          for (int q = 1; q < 4; ++q) {
            l += r3[128 + q * 32 + lane] * ex2_approx(r3[q * 32 + lane] - mo);
            sum += r3[256 + q * 32 + lane];
          }
          // the accumulator goes back only now: the tile after next then finds the exchange area read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
          const long long pi = static_cast<long long>(tl.nt) * p.part_ld + m;
          if (row_ok && in_bounds(p.err, pi, 1, static_cast<long long>(n_tiles) * p.part_ld, SITE_HEAD_PART)) {
            p.part[pi] = make_float2(mm, l);
            if (p.part_sum) p.part_sum[pi] = sum;
          }
        }
      } else {
#pragma unroll
        for (int ch = 0; ch < COLS / 32; ++ch) {
          const int n0 = ncol0 + ch * 32;
          float v[32];
          tmem_ld32(t_cols + ch * 32, v);
          tmem_ld_wait();
          if (ch == COLS / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[acc]);
          }
          if constexpr (KIND == HEAD_DX) {
            if (n0 >= p.d || m0 >= p.m_cap) continue;
            if (tl.kb0 == tl.kb1) {          // a short last piece can leave a split without any k
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0.0f;
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {               // two boxes of 16 float columns
              if (n0 + 16 * hf >= p.d) continue;
              if (lane == 0) bulk_wait_read0();
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4*>(box + box_off(lane, j)) =
                    make_float4(v[16 * hf + 4 * j], v[16 * hf + 4 * j + 1], v[16 * hf + 4 * j + 2], v[16 * hf + 4 * j + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                if (p.first_piece) tma_store_3d(&omap, box, n0 + 16 * hf, m0, tl.split);
                else tma_reduce_add_3d(&omap, box, n0 + 16 * hf, m0, tl.split);
                bulk_commit();
              }
            }
          } else {
            if constexpr (KIND == HEAD_DLOGITS) {
              const uint64_t c2 = f32x2_pack(c, c), l2 = f32x2_pack(-lse2, -lse2);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                float a, b;
                fma_f32x2(a, b, v[i], v[i + 1], c2, l2);
                v[i] = ex2_approx(a) - smooth;
                v[i + 1] = ex2_approx(b) - smooth;
              }
              const int end = lo + (ch + 1) * 32;
              while (__any_sync(0xffffffffu, next < end)) {
                if (next < end) {
                  const int col = next - lo - ch * 32;
                  const float pt = p.tgt_p ? p.tgt_p[tb + pos] : p.label_p;
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (i == col) v[i] -= pt;
                  ++pos;
                  next = pos < cnt ? p.tgt_idx[tb + pos] : 0x7fffffff;
                }
              }
              // rows and columns outside are zeros: they are factors of the products that follow
              if (!row_ok || p.v0 + n0 + 32 > p.V) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!row_ok || p.v0 + n0 + i >= p.V) v[i] = 0.0f;
              }
              if (m0 >= p.m_cap) continue;
            } else {                                        // HEAD_DW
              if (n0 >= p.d || p.v0 + m0 >= p.V) continue;
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] *= g_out;
            }
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            if (lane == 0) bulk_wait_read0();       // the previous store has read the staging box
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(box + box_off(lane, j)) =
                  make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&omap, box, n0, (KIND == HEAD_DW ? p.v0 : 0) + m0);
              bulk_commit();
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait0();   // stores complete before the CTA (and its smem) goes away
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, TMEM_COLS);
}

}  // namespace wb
