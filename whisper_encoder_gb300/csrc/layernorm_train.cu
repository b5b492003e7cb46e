// LayerNorm for training: the forward pass that keeps its row statistics, and the backward pass with
// the reduction of the weight's and the bias's gradient.  Any width up to 10240, bf16 / f16 / f32.
//
//   t = round(x + r), mu = mean(t), rs = 1 / sqrt(mean((t - mu)^2) + eps), y = (t - mu) rs g + b
//   h = (t - mu) rs, u = g dy:
//   dx = rs (u - mean(u) - h mean(u h)) (+ dt),  dg = sum_rows dy h,  db = sum_rows dy
//
// Both passes are bound by memory: each element is read once and written once.  Statistics, row sums and
// the sums over rows are fp32, and the row statistics take their two passes over registers.
// Forward: a team of 1, 2, 4 or 8 warps (by the width) holds a row, at most 40 elements a lane; teams of
// one warp need no barrier.  Backward: see there.
#include <cstring>
#include <mutex>
#include <type_traits>

#include "../../include/wb.h"
#include "internal.h"
#include "ptx.cuh"

namespace wb {
namespace {

constexpr int LNT_MAX_D = 10240;
// Grid cap: well above what is resident, so that the SMs take rows as they get through them (152 * 8: 82 us, this 78).
constexpr int LNT_FWD_BLOCKS = 152 * 32;
constexpr int COL_SLICES = 32;            // column-sum kernel: slices of the partial rows per block

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

// VEC elements of T.  Where rows start on 16 bytes they are one load, of 16 bytes or (forward, 16-bit types) 8; in the
// ragged backward pass a pair whose second element lies 32 W columns on.
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

// ------------------------------ forward ------------------------------
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

// Pair i of a loaded vector as two floats, and back: 16-bit pairs as whole words (the forward pass of 48000 x 1280
// bf16 with a residual took 86 us converting element by element, 78 so).
template <typename T, typename Raw>
__device__ __forceinline__ uint64_t pair_of(const Raw& r, int i) {
  if constexpr (sizeof(T) == 4) {
    return f32x2_pack(r.e[2 * i], r.e[2 * i + 1]);
  } else {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      uint32_t w;
      memcpy(&w, r.e + 2 * i, 4);
      return f32x2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
      __half2 w;
      memcpy(&w, r.e + 2 * i, 4);
      const float2 f = __half22float2(w);
      return f32x2_pack(f.x, f.y);
    }
  }
}
template <typename T, typename Raw>
__device__ __forceinline__ void set_pair(Raw& r, int i, uint64_t v) {
  float lo, hi;
  f32x2_unpack(v, lo, hi);
  if constexpr (sizeof(T) == 4) {
    r.e[2 * i] = lo;
    r.e[2 * i + 1] = hi;
  } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const __nv_bfloat162 w = __floats2bfloat162_rn(lo, hi);
    memcpy(r.e + 2 * i, &w, 4);
  } else {
    const __half2 w = __floats2half2_rn(lo, hi);
    memcpy(r.e + 2 * i, &w, 4);
  }
}

constexpr int lnt_warps(int W) { return W < 4 ? 4 : W; }   // warps per block: one to four teams

// Rows are read into registers, all loads of a row before its first sum; columns past the row count as zeros, so that
// the sums have no branches (3000 x 10240 f32 88 us with them, 78 without).
// 48000 x 1280 bf16 with a residual: 78 us, 6.3 TB/s, 24000 x 1280 f32 76.  Rings of shared memory in front of the same
// arithmetic take 85 to 89 (16 warps an SM, one or two rows at a time).
template <typename T, int VEC, int NV, int W>
__global__ void __launch_bounds__(lnt_warps(W) * 32)
    ln_train_fwd_kernel(const T* __restrict__ x, const T* __restrict__ res, const float* __restrict__ g,
                        const float* __restrict__ bta, int rows, int d, float eps, T* __restrict__ y,
                        T* __restrict__ total, float2* __restrict__ stats, uint32_t* err) {
  constexpr int TEAMS = lnt_warps(W) / W, NP = VEC / 2;
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
      u[i] = Raw{};
      if (col < d && in_bounds(err, base + col, VEC, n_el, SITE_LNT_X)) {
        u[i] = *reinterpret_cast<const Raw*>(x + base + col);
        if (res) r[i] = *reinterpret_cast<const Raw*>(res + base + col);
      }
    }
    uint64_t v[NV * NP], acc[2] = {0, 0};                  // two chains of adds
    float lo, hi;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = ((i * W + wt) * 32 + lane) * VEC;
      if (col < d && res) {
        // the sum is rounded to the tensor's type first: what is normalised is what is stored
#pragma unroll
        for (int j = 0; j < NP; ++j) set_pair<T>(u[i], j, f32x2_add(pair_of<T>(u[i], j), pair_of<T>(r[i], j)));
        if (in_bounds(err, base + col, VEC, n_el, SITE_LNT_TOTAL))
          *reinterpret_cast<Raw*>(total + base + col) = u[i];
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        v[i * NP + j] = pair_of<T>(u[i], j);
        acc[j & 1] = f32x2_add(acc[j & 1], v[i * NP + j]);
      }
    }
    f32x2_unpack(f32x2_add(acc[0], acc[1]), lo, hi);
    const float mean = team_sum<W>(lo + hi, 0.0f, red[team], team, wt, lane, 0).x * inv_d;
    acc[0] = acc[1] = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float nm = ((i * W + wt) * 32 + lane) * VEC < d ? -mean : 0.0f;      // past the row: stays 0
      const uint64_t nm2 = f32x2_pack(nm, nm);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        v[i * NP + j] = f32x2_add(v[i * NP + j], nm2);
        acc[j & 1] = f32x2_fma(v[i * NP + j], v[i * NP + j], acc[j & 1]);
      }
    }
    f32x2_unpack(f32x2_add(acc[0], acc[1]), lo, hi);
    const float rstd = rsqrtf(team_sum<W>(lo + hi, 0.0f, red[team], team, wt, lane, 1).x * inv_d + eps);
    const uint64_t rs2 = f32x2_pack(rstd, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = ((i * W + wt) * 32 + lane) * VEC;
      if (col >= d || !in_bounds(err, base + col, VEC, n_el, SITE_LNT_Y)) continue;
      float gg[VEC], bb[VEC];
      load_params<VEC>(g + col, gg);
      load_params<VEC>(bta + col, bb);
      Raw o;
#pragma unroll
      for (int j = 0; j < NP; ++j)
        set_pair<T>(o, j, f32x2_fma(f32x2_mul(v[i * NP + j], rs2), f32x2_pack(gg[2 * j], gg[2 * j + 1]),
                                    f32x2_pack(bb[2 * j], bb[2 * j + 1])));
      *reinterpret_cast<Raw*>(y + base + col) = o;
    }
    if (wt == 0 && lane == 0 && in_bounds(err, row, 1, rows, SITE_LNT_STATS)) stats[row] = make_float2(mean, rstd);
  }
}

// ------------------------------ backward ------------------------------
// Teams as in the forward pass.  Each lane keeps its columns of dg and db in registers over all the rows of
// its team; a block adds its teams in order and leaves one partial row, and a second kernel adds those in
// block order: no atomics, the same result every time.  A team's rows come through its own ring of shared
// memory, filled by one lane with bulk copies, and are read from there twice (for the row's sums, then for
// dx), so that neither the rows in flight nor the row at hand cost registers.  The arithmetic is on packed
// pairs.  g lies in shared memory too: read from global memory twice a row, 32 bytes apart from lane to lane, it took
// more of the L1 than the rows themselves (98 us against 86 at 48000 x 1280 bf16 with dt, 6000 x 10240 128 against 86).
// Measured there: 82 us (6.0 TB/s); rows held in registers and read directly 274 us (216 registers, 8 warps an SM);
// four resident blocks a SM instead of one write more partial rows.
// Rows that do not start on 16 bytes (ragged) come through the same rings, copied with the elements that share their
// first and last 16 bytes, and are read element by element, lanes side by side: 10000 x 5123 bf16 with dt 182 us,
// 40000 x 387 45, 4097 x 1283 f32 27 (a block a row, read directly into registers: 1195, 165 and 27).
constexpr int LNT_WARPS = 32;    // per block of the ragged forward kernel, at most
constexpr int LNT_STAGES = 4;    // rows in flight per team, at most

// Sums of (a, b) over the block; `slot` as in team_sum.
__device__ __forceinline__ float2 block_sum(float a, float b, float2 (*red)[LNT_WARPS], int slot) {
  const int W = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if ((threadIdx.x & 31) == 0) red[slot][threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  a = b = 0.0f;
  for (int i = 0; i < W; ++i) {
    a += red[slot][i].x;
    b += red[slot][i].y;
  }
  return make_float2(a, b);
}

// Elements a lane: fifths of 40 for rows of one warp (short rows keep few registers), 40 for the rest.
constexpr int lane_elems(int d) { return d > 1280 ? 40 : (d + 255) / 256 * 8; }
// Warps of a block, one block an SM.  Rows of many elements a lane take few warps, whose registers hold more loads
// at once and whose rings then have two rows each; short rows take many, as their chains of sums are long for their
// bytes.  bf16 with dt, 8 / 12 / 16 warps: 48000 x 1280 82 / 86 / 86 us, 24000 x 2560 82 / 85 / 88, 60000 x 768
// 65 / 65 / 68, 80000 x 640 80 / 71 / 70, 100000 x 512 79 / 70 / 69, 100000 x 256 61 / 49 / 45; with 6 and 4 warps
// 48000 x 1280 takes 86 and 102.  f32: 24000 x 1280 82 / 85 / -, 50000 x 384 55 / 54 / -; four warps a row, 6000 x
// 5120: 89 / 85 / -.  Ragged rows are bound by the reads of single elements and want the warps: 40000 x 1283 bf16
// 191 / 156 / 138, 40000 x 901 101 / 86 / 80, 40000 x 1283 f32 174 / 135 / -.
constexpr int lnb_warps(int W, int es, int elems, bool ragged) {
  return W == 8 || (!ragged && W < 4 && elems >= 32) ? 8 : es == 2 && W < 4 && (ragged || elems <= 16) ? 16 : 12;
}
constexpr int LNB_RING = 224 * 1024;   // bytes of g and the rings of a block
// Bytes of a row in a ring: a ragged row does not start on 16 bytes and is copied with what lies around it.
__host__ __device__ constexpr int lnb_slot(int d, int es, bool ragged) {
  return ragged ? (d * es + 14 + 15) / 16 * 16 : d * es;
}

// Partial rows part[block] = [dg (d) | db (d)]; null where the caller wants dx alone.
template <typename T, int VEC, int NV, int W>
__global__ void __launch_bounds__(lnb_warps(W, sizeof(T), NV * VEC, VEC * sizeof(T) < 16) * 32, 1)
    ln_train_bwd_kernel(const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ g,
                        const float2* __restrict__ stats, const T* __restrict__ dt, int rows, int d,
                        T* __restrict__ dx, float* __restrict__ part, int stages, uint32_t* err) {
  constexpr int TEAMS = lnb_warps(W, sizeof(T), NV * VEC, VEC * sizeof(T) < 16) / W, NP = VEC / 2;    // pairs a vector
  constexpr bool RAGGED = VEC * sizeof(T) < 16;
  static_assert(!RAGGED || VEC == 2, "a pair of elements 32 W columns apart");
  static_assert((TEAMS * 3 * static_cast<int>(sizeof(T)) + 4) * (W * 32 * NV * VEC) + TEAMS * 3 * 32 <= LNB_RING,
                "g and a row of each team");
  using Raw = typename Pack<T, VEC>::Raw;
  extern __shared__ __align__(16) uint8_t ring[];     // g, [teams][stages][x, dy, dt][row]; at the end [teams][2 d]
  __shared__ uint64_t full[TEAMS][LNT_STAGES];
  __shared__ int abort_flag;
  __shared__ float2 red[TEAMS][2][W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / W, wt = warp % W;
  const float inv_d = 1.0f / static_cast<float>(d);
  const long long n_el = static_cast<long long>(rows) * d;
  const uint32_t bytes = lnb_slot(d, sizeof(T), RAGGED);
  const uint32_t stage_bytes = bytes * (dt ? 3 : 2);
  // g, by (vector, quarter of a vector, lane): neighbouring lanes read neighbouring 16 bytes (ragged: by column)
  float4* gs = reinterpret_cast<float4*>(ring);
  float* gs1 = reinterpret_cast<float*>(ring);
  constexpr int G4 = VEC / 4;
  uint8_t* mine = ring + W * NV * 32 * VEC * sizeof(float) + static_cast<size_t>(team) * stages * stage_bytes;
  if (threadIdx.x == 0) {
    for (int t = 0; t < TEAMS; ++t)
      for (int i = 0; i < LNT_STAGES; ++i) mbar_init(&full[t][i], 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  grid_dependency_wait();
  if (RAGGED) {
    for (int c = threadIdx.x; c < d; c += TEAMS * W * 32) gs1[c] = __ldg(g + c);
  } else if (team == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = ((i * W + wt) * 32 + lane) * VEC;
#pragma unroll
      for (int q = 0; q < G4; ++q)
        gs[((i * W + wt) * G4 + q) * 32 + lane] =
            col < d ? __ldg(reinterpret_cast<const float4*>(g + col) + q) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
  }
  __syncthreads();
  uint64_t ag[NV * NP], ab[NV * NP];         // this lane's columns of dg and db, in pairs
#pragma unroll
  for (int i = 0; i < NV * NP; ++i) ag[i] = ab[i] = 0;
  grid_dependents_launch();
  const bool feeder = wt == 0 && lane == 0;
  auto issue = [&](long long row, int stage) {
    uint8_t* to = mine + static_cast<size_t>(stage) * stage_bytes;
    if constexpr (!RAGGED) {
      mbar_arrive_expect_tx(&full[team][stage], stage_bytes);
      bulk_load(to, x + row * d, bytes, &full[team][stage]);
      bulk_load(to + bytes, dy + row * d, bytes, &full[team][stage]);
      if (dt) bulk_load(to + 2 * bytes, dt + row * d, bytes, &full[team][stage]);
    } else {
      // the whole 16 bytes that the row lies in, as far as the tensor has them; what is left of the last row by hand.
      // (dx over an input: the neighbours' elements in them may be old or new, and are not looked at.)
      constexpr int PER = 16 / sizeof(T);
      const long long lo = row * d / PER * PER, end = (row + 1) * d, whole = n_el / PER * PER;
      const long long hi = (end + PER - 1) / PER * PER;
      const uint32_t n = static_cast<uint32_t>((hi <= n_el ? hi : whole) - lo) * sizeof(T);
      if (hi > n_el) {
        for (long long e = whole; e < n_el; ++e) {
          reinterpret_cast<T*>(to)[e - lo] = x[e];
          reinterpret_cast<T*>(to + bytes)[e - lo] = dy[e];
          if (dt) reinterpret_cast<T*>(to + 2 * bytes)[e - lo] = dt[e];
        }
      }
      mbar_arrive_expect_tx(&full[team][stage], n * (dt ? 3 : 2));
      if (n) {
        bulk_load(to, x + lo, n, &full[team][stage]);
        bulk_load(to + bytes, dy + lo, n, &full[team][stage]);
        if (dt) bulk_load(to + 2 * bytes, dt + lo, n, &full[team][stage]);
      }
    }
  };
  const long long first = blockIdx.x + static_cast<long long>(gridDim.x) * team;     // few rows: one a block
  const long long step = static_cast<long long>(gridDim.x) * TEAMS;
  if (feeder)
    for (int s = 0; s < stages && first + s * step < rows; ++s) issue(first + s * step, s);
  auto stats_of = [&](long long row) {
    return row < rows && in_bounds(err, row, 1, rows, SITE_LNT_STATS) ? __ldg(stats + row) : make_float2(0.0f, 0.0f);
  };
  // column of a vector's first element, and of its second where rows are ragged
  auto col_of = [&](int i) { return RAGGED ? (2 * i * W + wt) * 32 + lane : ((i * W + wt) * 32 + lane) * VEC; };
  constexpr int NEXT = W * 32;
  auto load_gs = [&](int i, float (&o)[VEC]) {
    if constexpr (RAGGED) {
      const int c = col_of(i);
      o[0] = gs1[c];
      o[1] = c + NEXT < d ? gs1[c + NEXT] : 0.0f;
    } else {
#pragma unroll
      for (int q = 0; q < G4; ++q) {
        const float4 f = gs[((i * W + wt) * G4 + q) * 32 + lane];
        o[4 * q] = f.x; o[4 * q + 1] = f.y; o[4 * q + 2] = f.z; o[4 * q + 3] = f.w;
      }
    }
  };
  auto load_row = [&](const uint8_t* from, int col) -> Raw {
    if constexpr (RAGGED) {
      Raw r = {};
      r.e[0] = reinterpret_cast<const T*>(from)[col];
      if (col + NEXT < d) r.e[1] = reinterpret_cast<const T*>(from)[col + NEXT];
      return r;
    } else {
      return *reinterpret_cast<const Raw*>(from + col * sizeof(T));
    }
  };
  float2 ahead = stats_of(first);            // statistics of the next row, loaded a row early
  int stage = 0, slot = 0;
  uint32_t parity = 0;
  for (long long row = first; row < rows; row += step, slot ^= 1) {
    const long long base = row * d;
    const float2 st = ahead;
    ahead = stats_of(row + step);
    const uint64_t nm2 = f32x2_pack(-st.x, -st.x), rs2 = f32x2_pack(st.y, st.y);
    const uint8_t* at = mine + static_cast<size_t>(stage) * stage_bytes;
    if (RAGGED) at += base * sizeof(T) % 16;
    // a wait that runs out marks the error word and goes on: every thread keeps to the same barriers
    mbar_wait(&full[team][stage], parity, err, &abort_flag, 31);
    uint64_t c1p = 0, c2p = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = col_of(i);
      if (col >= d) continue;
      const Raw xv = load_row(at, col);
      const Raw yv = load_row(at + bytes, col);
      float gg[VEC];
      load_gs(i, gg);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int e = i * NP + j;
        const uint64_t y2 = pair_of<T>(yv, j);
        const uint64_t h2 = f32x2_mul(f32x2_add(pair_of<T>(xv, j), nm2), rs2);
        const uint64_t u2 = f32x2_mul(f32x2_pack(gg[2 * j], gg[2 * j + 1]), y2);
        ag[e] = f32x2_fma(y2, h2, ag[e]);
        ab[e] = f32x2_add(ab[e], y2);
        c1p = f32x2_add(c1p, u2);
        c2p = f32x2_fma(u2, h2, c2p);
      }
    }
    float lo, hi, c1, c2;
    f32x2_unpack(c1p, lo, hi);
    c1 = lo + hi;
    f32x2_unpack(c2p, lo, hi);
    c2 = lo + hi;
    const float2 c = team_sum<W>(c1, c2, red[team], team, wt, lane, slot);
    c1 = -c.x * inv_d;
    c2 = -c.y * inv_d;
    const uint64_t c12 = f32x2_pack(c1, c1), c22 = f32x2_pack(c2, c2);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = col_of(i);
      if (col >= d || !in_bounds(err, base + col, RAGGED ? 1 : VEC, n_el, SITE_LNT_Y)) continue;
      const Raw xv = load_row(at, col);
      const Raw yv = load_row(at + bytes, col);
      float gg[VEC];
      load_gs(i, gg);
      Raw tv, o;
      if (dt) tv = load_row(at + 2 * bytes, col);
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const uint64_t h2 = f32x2_mul(f32x2_add(pair_of<T>(xv, j), nm2), rs2);
        const uint64_t u2 = f32x2_fma(f32x2_pack(gg[2 * j], gg[2 * j + 1]), pair_of<T>(yv, j), c12);
        const uint64_t in = f32x2_fma(h2, c22, u2);
        set_pair<T>(o, j, dt ? f32x2_fma(in, rs2, pair_of<T>(tv, j)) : f32x2_mul(in, rs2));
      }
      if constexpr (RAGGED) {
        dx[base + col] = o.e[0];
        if (col + NEXT < d) dx[base + col + NEXT] = o.e[1];
      } else {
        *reinterpret_cast<Raw*>(dx + base + col) = o;
      }
    }
    // the team has read the stage for the second time: its next row may come
    if (W == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(W * 32) : "memory");
    if (feeder && row + stages * step < rows) issue(row + stages * step, stage);
    if (++stage == stages) { stage = 0; parity ^= 1u; }
  }
  if (!part) return;
  float* dst = part + static_cast<long long>(blockIdx.x) * 2 * d;
  const long long part_el = static_cast<long long>(gridDim.x) * 2 * d;
  uint64_t* acc = reinterpret_cast<uint64_t*>(ring);       // every copy has been waited for
  if (TEAMS > 1) __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = col_of(i);
    if (col >= d) continue;
    if constexpr (RAGGED) {
      float* to = reinterpret_cast<float*>(ring) + static_cast<size_t>(team) * 2 * d + col;
      float lo, hi;
      f32x2_unpack(ag[i], lo, hi);
      to[0] = lo;
      if (col + NEXT < d) to[NEXT] = hi;
      f32x2_unpack(ab[i], lo, hi);
      to[d] = lo;
      if (col + NEXT < d) to[d + NEXT] = hi;
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j) {                       // VEC divides d: pairs start on 8 bytes in both halves
        acc[(team * 2 * d + col) / 2 + j] = ag[i * NP + j];
        acc[(team * 2 * d + d + col) / 2 + j] = ab[i * NP + j];
      }
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += TEAMS * W * 32) {  // pairs of the 2 d sums, teams in order
    uint64_t sum = acc[c];
#pragma unroll
    for (int t = 1; t < TEAMS; ++t) sum = f32x2_add(sum, acc[t * d + c]);
    if (in_bounds(err, (dst - part) + 2 * c, 2, part_el, SITE_LNT_PART)) reinterpret_cast<uint64_t*>(dst)[c] = sum;
  }
}

// The forward pass of ragged rows: a block of up to 8 warps a row, single elements, read directly (4097 x 1283 f32
// 18 us, 40000 x 1283 bf16 with a residual 143; the team kernel above with single elements 29 and 809).  Wide rows
// take more warps rather than more loads a lane (with a residual, 11 loads against 20 or 40 in 8 warps: 10000 x 2561
// bf16 88 / 125 us, 10000 x 5123 188 / 467; 5000 x 10239 f16 10 loads in 32 warps 208, 40 in 8 331): 11 loads while 10
// warps hold a row, 10 loads while 16 do, 11 loads again while 16 do, then 10 in up to 32.  11 / 10 loads, bf16
// without a residual: 14692 x 3403 128 / 135, 14200 x 3521 150 / 132, 9998 x 5001 140 / 119, 9759 x 5123 138 / 187; with
// one 169 / 170, 195 / 169, 182 / 153, 179 / 231; f32 without one, half the rows: 66 / 75, 81 / 72, 75 / 66, 74 / 106.
template <typename T, int NV, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS > 16 ? 1 : WARPS > 8 ? 2 : NV <= 6 ? 6 : 3)
    ln_train_fwd_any_kernel(const T* __restrict__ x, const T* __restrict__ res, const float* __restrict__ g,
                            const float* __restrict__ bta, int rows, int d, float eps, T* __restrict__ y,
                            T* __restrict__ total, float2* __restrict__ stats, uint32_t* err) {
  __shared__ float2 red[2][LNT_WARPS];
  const int nt = blockDim.x, tid = threadIdx.x;
  const float inv_d = 1.0f / static_cast<float>(d);
  const long long n_el = static_cast<long long>(rows) * d;
  grid_dependency_wait();
  grid_dependents_launch();
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const long long base = row * d;
    T u[NV], r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = i * nt + tid;
      u[i] = r[i] = from_f32<T>(0.0f);
      if (col < d && in_bounds(err, base + col, 1, n_el, SITE_LNT_X)) {
        u[i] = x[base + col];
        if (res) r[i] = res[base + col];
      }
    }
    float v[NV], sm = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = i * nt + tid;
      if (res) {
        u[i] = from_f32<T>(to_f32<T>(u[i]) + to_f32<T>(r[i]));
        if (col < d && in_bounds(err, base + col, 1, n_el, SITE_LNT_TOTAL)) total[base + col] = u[i];
      }
      v[i] = to_f32<T>(u[i]);
      sm += v[i];
    }
    const float mean = block_sum(sm, 0.0f, red, 0).x * inv_d;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) q += i * nt + tid < d ? (v[i] - mean) * (v[i] - mean) : 0.0f;
    const float rstd = rsqrtf(block_sum(q, 0.0f, red, 1).x * inv_d + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = i * nt + tid;
      if (col < d && in_bounds(err, base + col, 1, n_el, SITE_LNT_Y))
        y[base + col] = from_f32<T>(fmaf((v[i] - mean) * rstd, __ldg(g + col), __ldg(bta + col)));
    }
    if (tid == 0 && in_bounds(err, row, 1, rows, SITE_LNT_STATS)) stats[row] = make_float2(mean, rstd);
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
#pragma unroll 8
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
int fwd_blocks(int rows, int d) {
  const int t = teams_per_block(d);
  const long long b = (static_cast<long long>(rows) + t - 1) / t;
  return static_cast<int>(b < LNT_FWD_BLOCKS ? b : LNT_FWD_BLOCKS);
}

int bwd_blocks(int rows) { return rows < 152 ? rows : 152; }   // a partial row each

// How rows are spread, by width, type and (backward) the tensors that a row is read from.
struct Spread {
  bool vec;      // rows start on 16 bytes
  int warps;     // per row
  int stages;    // backward: rows in flight per team, what the shared memory holds
  int blocks;    // backward: one an SM, at most one a row
  int any_nv;    // ragged forward pass: loads a lane, see there
  int any_warps;
};

Spread spread(int rows, int d, int dtype, int tensors) {
  const int es = dtype == WB_F32 ? 4 : 2;
  Spread s = {};
  s.vec = d % (16 / es) == 0;
  s.warps = team_warps(d);
  const int teams = lnb_warps(s.warps, es, lane_elems(d), !s.vec) / s.warps;
  const int fit = (LNB_RING - s.warps * 1280 * 4) / (teams * lnb_slot(d, es, !s.vec) * tensors);
  s.stages = fit < LNT_STAGES ? fit : LNT_STAGES;
  s.blocks = bwd_blocks(rows);
  const int need = (d + 32 * 8 - 1) / (32 * 8);
  s.any_nv = need <= 2 ? need : need <= 4 ? 4 : need <= 6 ? 6 : need <= 10 ? 10
             : d <= 11 * 32 * 10 || (d > 10 * 32 * 16 && d <= 11 * 32 * 16) ? 11 : 10;
  s.any_warps = (d + 32 * s.any_nv - 1) / (32 * s.any_nv);
  return s;
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

std::mutex g_lnt_mu;

// Raises a kernel's limit of dynamic shared memory once per device, so that launches stay legal inside a
// graph capture.
template <typename K>
cudaError_t ring_attr(K kern, uint64_t* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev > 63) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_lnt_mu);
  if (*done & (1ull << dev)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LNB_RING);
  if (e == cudaSuccess) *done |= 1ull << dev;
  return e;
}

template <typename T, int VEC, int NV, int W>
cudaError_t go(const BwdArgs<T>& a, const Spread& sp, cudaStream_t s) {
  static uint64_t done = 0;
  const cudaError_t e = ring_attr(ln_train_bwd_kernel<T, VEC, NV, W>, &done);
  if (e != cudaSuccess) return e;
  constexpr int WARPS = lnb_warps(W, sizeof(T), NV * VEC, VEC * sizeof(T) < 16);
  constexpr size_t TEAMS = WARPS / W;
  size_t smem = W * NV * 32 * VEC * sizeof(float) +
                TEAMS * sp.stages * (a.dt ? 3 : 2) * lnb_slot(a.d, sizeof(T), VEC * sizeof(T) < 16);
  const size_t sums = TEAMS * 2 * a.d * sizeof(float);
  if (smem < sums) smem = sums;
  return launch_pdl(ln_train_bwd_kernel<T, VEC, NV, W>, dim3(sp.blocks), dim3(WARPS * 32), smem, s, a.dy, a.x, a.g,
                    a.stats, a.dt, a.rows, a.d, a.dx, a.part, sp.stages, a.err);
}
template <typename T, int VEC>
cudaError_t bwd_by_width(const BwdArgs<T>& a, const Spread& sp, cudaStream_t s) {
  constexpr int FULL = 40 / VEC;                           // lane_elems(d) of them
  if (sp.warps == 2) return go<T, VEC, FULL, 2>(a, sp, s);
  if (sp.warps == 4) return go<T, VEC, FULL, 4>(a, sp, s);
  if (sp.warps == 8) return go<T, VEC, FULL, 8>(a, sp, s);
  if (a.d <= 256) return go<T, VEC, FULL / 5, 1>(a, sp, s);
  if (a.d <= 512) return go<T, VEC, 2 * FULL / 5, 1>(a, sp, s);
  if (a.d <= 768) return go<T, VEC, 3 * FULL / 5, 1>(a, sp, s);
  if (a.d <= 1024) return go<T, VEC, 4 * FULL / 5, 1>(a, sp, s);
  return go<T, VEC, FULL, 1>(a, sp, s);
}

template <typename T, int VEC, int NV, int W>
cudaError_t go(const FwdArgs<T>& a, cudaStream_t s) {
  return launch_pdl(ln_train_fwd_kernel<T, VEC, NV, W>, dim3(fwd_blocks(a.rows, a.d)), dim3(lnt_warps(W) * 32), 0, s,
                    a.x, a.res, a.g, a.b, a.rows, a.d, a.eps, a.y, a.total, a.stats, a.err);
}
template <typename T, int NV, int WARPS = 8>
cudaError_t go_any(const FwdArgs<T>& a, const Spread& sp, cudaStream_t s) {
  return launch_pdl(ln_train_fwd_any_kernel<T, NV, WARPS>, dim3(a.rows < LNT_FWD_BLOCKS ? a.rows : LNT_FWD_BLOCKS),
                    dim3(32 * sp.any_warps), 0, s, a.x, a.res, a.g, a.b, a.rows, a.d, a.eps, a.y, a.total, a.stats,
                    a.err);
}
template <typename T>
cudaError_t any_by_width(const FwdArgs<T>& a, const Spread& sp, cudaStream_t s) {
  switch (sp.any_nv) {
    case 1: return go_any<T, 1>(a, sp, s);
    case 2: return go_any<T, 2>(a, sp, s);
    case 4: return go_any<T, 4>(a, sp, s);
    case 6: return go_any<T, 6>(a, sp, s);
    case 11: return go_any<T, 11, 16>(a, sp, s);
    default: return sp.any_warps <= 8 ? go_any<T, 10>(a, sp, s) : go_any<T, 10, 32>(a, sp, s);
  }
}

// Vectors of 8 bytes for 16-bit rows: g and b then are 16 neighbouring bytes a lane.  Against 16 bytes: 48000 x 1280
// bf16 without a residual 52 / 57 us, with one 77.5 / 77.9, 6000 x 10240 83 / 89; rows of two or four warps gain
// nothing (24000 x 2560 80 / 80) or lose (3001 x 5120 27.5 / 26.1), and take 16 bytes.
template <typename T>
cudaError_t fwd_by_width(const FwdArgs<T>& a, const Spread& sp, cudaStream_t s) {
  constexpr int WIDE = 16 / sizeof(T), VEC = 4, FULL = 40 / VEC;
  if (!sp.vec) return any_by_width(a, sp, s);
  if (sp.warps == 2) return go<T, WIDE, 40 / WIDE, 2>(a, s);
  if (sp.warps == 4) return go<T, WIDE, 40 / WIDE, 4>(a, s);
  if (sp.warps == 8) return go<T, VEC, FULL, 8>(a, s);
  if (a.d <= 256) return go<T, VEC, FULL / 5, 1>(a, s);
  if (a.d <= 512) return go<T, VEC, 2 * FULL / 5, 1>(a, s);
  if (a.d <= 768) return go<T, VEC, 3 * FULL / 5, 1>(a, s);
  if (a.d <= 1024) return go<T, VEC, 4 * FULL / 5, 1>(a, s);
  return go<T, VEC, FULL, 1>(a, s);
}

bool type_ok(int dtype) { return dtype == WB_BF16 || dtype == WB_F16 || dtype == WB_F32; }

template <typename T>
cudaError_t fwd_t(const void* x, const void* res, const float* g, const float* b, int rows, int d, float eps, void* y,
                  void* total, float* stats, const Spread& sp, uint32_t* err, cudaStream_t s) {
  const FwdArgs<T> a{static_cast<const T*>(x), static_cast<const T*>(res), g, b, rows, d, eps, static_cast<T*>(y),
                     static_cast<T*>(total), reinterpret_cast<float2*>(stats), err};
  return fwd_by_width<T>(a, sp, s);
}
template <typename T>
cudaError_t bwd_t(const void* dy, const void* x, const float* g, const float* stats, const void* dt, int rows, int d,
                  void* dx, float* part, const Spread& sp, uint32_t* err, cudaStream_t s) {
  const BwdArgs<T> a{static_cast<const T*>(dy), static_cast<const T*>(x), g, reinterpret_cast<const float2*>(stats),
                     static_cast<const T*>(dt), rows, d, static_cast<T*>(dx), part, err};
  return sp.vec ? bwd_by_width<T, 16 / sizeof(T)>(a, sp, s) : bwd_by_width<T, 2>(a, sp, s);
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
      !aligned8(stats))
    return WB_EINVAL;
  if (residual ? !aligned16(residual) || !total || !aligned16(total) : total != nullptr) return WB_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t* err = tc_err_ptr();
  if (!err) return WB_ECUDA;
  const Spread sp = spread(rows, d, dtype, 1);
  Prof pr(PC_TRAIN_LN, s);
  if (dtype == WB_BF16) WB_CUDA(fwd_t<__nv_bfloat16>(x, residual, g, b, rows, d, eps, y, total, stats, sp, err, s));
  else if (dtype == WB_F16) WB_CUDA(fwd_t<__half>(x, residual, g, b, rows, d, eps, y, total, stats, sp, err, s));
  else WB_CUDA(fwd_t<float>(x, residual, g, b, rows, d, eps, y, total, stats, sp, err, s));
  return WB_OK;
}

size_t wb_layernorm_backward_workspace_bytes(int rows, int d, int dtype) {
  if (rows < 1 || d < 1 || d > LNT_MAX_D || !type_ok(dtype)) return 0;
  return static_cast<size_t>(bwd_blocks(rows)) * 2 * d * sizeof(float);
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
  if (!dy || !x || !g || !stats || !dx || !aligned16(dy) || !aligned16(x) || !aligned16(g) || !aligned8(stats) ||
      !aligned16(dx) || (dtotal && !aligned16(dtotal)))
    return WB_EINVAL;
  if (dg && (!workspace || !aligned16(workspace) ||
             workspace_bytes < wb_layernorm_backward_workspace_bytes(rows, d, dtype)))
    return WB_EWORKSPACE;
  uint32_t* err = tc_err_ptr();
  if (!err) return WB_ECUDA;
  float* part = dg ? static_cast<float*>(workspace) : nullptr;
  const Spread sp = spread(rows, d, dtype, dtotal ? 3 : 2);
  Prof pr(PC_TRAIN_LN, s, dg ? 2 : 1);
  if (dtype == WB_BF16) WB_CUDA(bwd_t<__nv_bfloat16>(dy, x, g, stats, dtotal, rows, d, dx, part, sp, err, s));
  else if (dtype == WB_F16) WB_CUDA(bwd_t<__half>(dy, x, g, stats, dtotal, rows, d, dx, part, sp, err, s));
  else WB_CUDA(bwd_t<float>(dy, x, g, stats, dtotal, rows, d, dx, part, sp, err, s));
  if (dg)
    WB_CUDA(launch_pdl(ln_train_colsum_kernel, dim3((2 * d + 31) / 32), dim3(32 * COL_SLICES), 0, s,
                       static_cast<const float*>(part), sp.blocks, d, dg, db, err));
  return WB_OK;
}

}  // extern "C"
