// Clipped policy loss on per-token log-probabilities, with a KL term against a reference, and its gradient.
//
// With nll = -log p of a sampled token (what the vocabulary losses give as a row's loss), d = old_nll - nll
// and x = nll - ref_nll, a token of a sequence with advantage A has
//   l = -min(e^d A, clip(e^d, 1 - lo, 1 + hi) A) + beta (e^x - x - 1),
//   dl/dnll = (clipped ? 0 : e^d A) + beta (e^x - 1),
// and the loss is sum w l with w = 1 / N over the N tokens that take part, or 1 / (B n_b): the mean over the B
// sequences that have tokens of the means over their n_b tokens.
//
// Bound by memory (16 bytes a token forward, 20 backward, 4 more with a reference), below a million tokens by the launches.
// Forward: a team of 1 to 8 warps of a block takes a sequence; a block leaves one partial row, and a second kernel joins those
// in order, in every one of its blocks, and turns counts into weights.  Up to 128 sequences of 512 tokens are one block's, in
// one launch: 8 x 77 tokens take 5.5 us against 8.2 with two.  Towards that limit the one block is the slower form: 16 x 448 tokens take it
// 5.2 us, 64 x 448 10.2 and 128 x 512 18.0, where two launches take 6.5 for 129 x 512 (all among other calls; 8 x 77 so 3.5).
// No atomics: the same call gives the same bits.
// 16001 x 448 tokens: forward 28 us, of which the join takes 4 (the sums 5 TB/s), backward 22 (6.5 TB/s).  Four tokens side by side a load
// where they lie on 16 bytes: one at a time it took 30 and 25, half of the issue slots on addresses.  6 blocks an SM with half the loads
// each: 26, but 1024 x 448 tokens 8.6 for 8.3; prefetching a warp's next sequence into L2: 28.
//
// Numbers.  Whether a token is clipped is decided on d against log1p(hi) and log1p(-lo), both as unevaluated sums of
// two float32 (the rounding of a difference is exact in float32): one rounding near the border would turn a
// whole gradient on or off.  e^x - x - 1 is x^2 / 2 for small x: below 1/2 its series, above it the
// difference of expm1, which loses two bits at most.  An advantage of zero gives zero, whatever e^d is.  A lane adds up to 32 of a
// sequence's tokens in one float32, the rest of its share (sequences of more than 8192 tokens) as pairs.
#include <cmath>
#include <type_traits>

#include "../../include/wb.h"
#include "internal.h"
#include "ptx.cuh"

namespace wb {
namespace {

constexpr int POL_THREADS = 256, POL_WARPS = POL_THREADS / 32;
constexpr int POL_MAX_BLOCKS = 608;       // 4 on each SM
constexpr int POL_TILE = 4;               // tokens of a thread and step, backward
constexpr int POL_SUM_TILE = 8;           // forward: its loads in flight
constexpr int POL_FLUSH = 4;              // forward: steps of them that a lane adds in one float32
constexpr int POL_LANE_TOKENS = POL_FLUSH * POL_SUM_TILE;
constexpr int POL_SMALL_S = 128, POL_SMALL_T = 512, POL_SMALL_THREADS = 1024;

struct PolicyArgs {
  const float* nll;
  const float* old_nll;
  const float* ref_nll;      // or null
  const float* adv;
  const int64_t* labels;
  long long S, T;
  int adv_tok;               // one for each token, else one for each sequence
  float hi0, hi1, lo0, lo1;  // log1p(hi), log1p(-lo): value and what its rounding left
  float hold_hi, hold_lo;    // 1 + hi, 1 - lo
  float beta;
  int per_sequence;
  uint32_t* err;
};

struct Token {
  float loss, kl, grad;
  bool clipped;
};

// x^2/2 + x^3/6 + ... for |x| < 1/2: the first term left out, x^10 / 10! relative to x^2 / 2, is below 2^-28.
__device__ __forceinline__ float exp_minus_x_minus_1(float x, float em1) {
  float p = fmaf(x, 1.0f / 9.0f, 1.0f);
  p = fmaf(x * (1.0f / 8.0f), p, 1.0f);
  p = fmaf(x * (1.0f / 7.0f), p, 1.0f);
  p = fmaf(x * (1.0f / 6.0f), p, 1.0f);
  p = fmaf(x * (1.0f / 5.0f), p, 1.0f);
  p = fmaf(x * (1.0f / 4.0f), p, 1.0f);
  p = fmaf(x * (1.0f / 3.0f), p, 1.0f);
  return fabsf(x) < 0.5f ? 0.5f * x * x * p : em1 - x;
}

// What the sign of an advantage decides, once a sequence where it is the sequence's: clipped is sign d above border.
struct Side {
  float adv, sign, b0, b1;   // border: value and what its rounding left
  float held;                // a clipped token's loss
};
__device__ __forceinline__ Side policy_side(const PolicyArgs& a, float adv) {
  const bool up = adv > 0.0f;
  return Side{adv, up ? 1.0f : adv < 0.0f ? -1.0f : 0.0f, up ? a.hi0 : -a.lo0, up ? a.hi1 : -a.lo1, -(up ? a.hold_hi : a.hold_lo) * adv};
}

template <bool REF>
__device__ __forceinline__ Token policy_token(const PolicyArgs& a, const Side& k, float nll, float old_nll, float ref) {
  Token t;
  const float d = old_nll - nll, ds = d * k.sign;
  const float bb = d - old_nll;
  const float e = (old_nll - (d - bb)) - (nll + bb);       // d + e is the difference itself
  t.clipped = (ds > k.b0) | ((ds == k.b0) & (e * k.sign > k.b1));
  const float ra = k.adv == 0.0f ? 0.0f : expf(d) * k.adv;
  t.loss = t.clipped ? k.held : -ra;
  t.grad = t.clipped ? 0.0f : ra;
  t.kl = 0.0f;
  if (REF) {
    const float x = nll - ref;
    const float em1 = expm1f(x);
    t.kl = exp_minus_x_minus_1(x, em1);
    if (a.beta != 0.0f) {                                // a weight of zero leaves a KL of infinity out
      t.loss = fmaf(a.beta, t.kl, t.loss);
      t.grad = fmaf(a.beta, em1, t.grad);
    }
  }
  return t;
}

// Tokens at..at + 3 * step, as many as `there` says; VEC: side by side, on 16 bytes.  A label counts by its sign, which is in its upper word.
template <bool REF, bool VEC, bool TOK>
__device__ __forceinline__ void load4(const PolicyArgs& a, long long at, int step, const bool (&there)[4], int (&lab)[4], float (&nll)[4],
                                      float (&old)[4], float (&ref)[4], float (&adv)[4]) {
  const int* hi = reinterpret_cast<const int*>(a.labels) + 1;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lab[i] = -1;
      nll[i] = old[i] = ref[i] = 0.0f;
      if (TOK) adv[i] = 0.0f;
    }
    if (!there[0] || !in_bounds(a.err, at, 4, a.S * a.T, SITE_POLICY_IN)) return;
    const int4 l0 = *reinterpret_cast<const int4*>(a.labels + at), l1 = *reinterpret_cast<const int4*>(a.labels + at + 2);
    const float4 n = *reinterpret_cast<const float4*>(a.nll + at), o = *reinterpret_cast<const float4*>(a.old_nll + at);
    lab[0] = l0.y; lab[1] = l0.w; lab[2] = l1.y; lab[3] = l1.w;
    nll[0] = n.x; nll[1] = n.y; nll[2] = n.z; nll[3] = n.w;
    old[0] = o.x; old[1] = o.y; old[2] = o.z; old[3] = o.w;
    if (REF) {
      const float4 r = *reinterpret_cast<const float4*>(a.ref_nll + at);
      ref[0] = r.x; ref[1] = r.y; ref[2] = r.z; ref[3] = r.w;
    }
    if (TOK) {
      const float4 v = *reinterpret_cast<const float4*>(a.adv + at);
      adv[0] = v.x; adv[1] = v.y; adv[2] = v.z; adv[3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long t = at + static_cast<long long>(i) * step;
      lab[i] = -1;
      nll[i] = old[i] = ref[i] = 0.0f;
      if (TOK) adv[i] = 0.0f;
      if (!there[i] || !in_bounds(a.err, t, 1, a.S * a.T, SITE_POLICY_IN)) continue;
      lab[i] = hi[2 * t];
      nll[i] = a.nll[t];
      old[i] = a.old_nll[t];
      if (REF) ref[i] = a.ref_nll[t];
      if (TOK) adv[i] = a.adv[t];
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A running sum and what its roundings left.  Units for float64 are so few (16 cycles a warp's addition) that a sequence's nine
// operations in one lane were half of the forward pass over 16001 sequences, and the join of 608 rows a microsecond.
struct Sum2 {
  float s, c;
  __device__ __forceinline__ void add(float v) {
    const float t = s + v, b = t - s;
    c += (s - (t - b)) + (v - b);
    s = t;
  }
  __device__ __forceinline__ void add(const Sum2& v) {
    add(v.s);
    c += v.c;
  }
  // (what an infinite sum's roundings left is no number)
  __device__ __forceinline__ float value32() const { return isfinite(s) ? s + c : s; }
  __device__ __forceinline__ double value() const { return isfinite(s) ? static_cast<double>(s) + static_cast<double>(c) : static_cast<double>(s); }
};

// Sums of loss, KL and clipped tokens over sequences (each divided by its sequence's tokens where sequences count the same), tokens,
// and sequences with tokens.
struct PolicyPart {
  Sum2 loss, kl, clipped;
  long long tokens, seqs;
};

struct SeqSum {
  float loss, kl;
  int clipped, count;
};

// This warp's share of a sequence, in every lane: warp `part` of W.  No branches among the tokens of a step: they overlap.
// LONG: a lane has more than POL_FLUSH steps (in every call the pairs took 2 to 5 % with a reference: 16001 x 448 tokens 40.3 us for 39.5).
template <bool REF, bool VEC, bool TOK, bool LONG>
__device__ __forceinline__ SeqSum policy_sequence(const PolicyArgs& a, long long s, int part, int W) {
  SeqSum r = {0.0f, 0.0f, 0, 0};
  const long long base = s * a.T;
  const Side side_s = policy_side(a, !TOK && in_bounds(a.err, s, 1, a.S, SITE_POLICY_IN) ? a.adv[s] : 0.0f);
  constexpr int GROUPS = POL_SUM_TILE / 4;
  const int T = static_cast<int>(a.T), first = (part * 32 + static_cast<int>(lane_id())) * (VEC ? 4 : 1);
  const int step = VEC ? 1 : W * 32, group = W * 32 * 4;                        // between a lane's tokens, and its groups of four
  // what a lane of a long sequence has added so far: of 4096 equal losses in one float32 the roundings were 2^-15 of the sum, of 65536
  // 2^-11
  Sum2 loss = {0.0f, 0.0f}, kl = {0.0f, 0.0f};
  int steps = 0;
  for (int t0 = first; t0 < T; t0 += GROUPS * group) {
    if (LONG && steps++ == POL_FLUSH) {
      loss.add(r.loss);
      if (REF) kl.add(r.kl);
      r.loss = r.kl = 0.0f;
      steps = 1;
    }
    int lab[GROUPS][4];
    float nll[GROUPS][4], old[GROUPS][4], ref[GROUPS][4], adv[GROUPS][4];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      bool there[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) there[i] = g * group + i * step < T - t0;
      load4<REF, VEC, TOK>(a, base + t0 + g * group, step, there, lab[g], nll[g], old[g], ref[g], adv[g]);
    }
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool on = lab[g][i] >= 0;
        const Token k = policy_token<REF>(a, TOK ? policy_side(a, adv[g][i]) : side_s, nll[g][i], old[g][i], ref[g][i]);
        r.loss += on ? k.loss : 0.0f;
        if (REF) r.kl += on ? k.kl : 0.0f;
        r.clipped += on & k.clipped;
        r.count += on;
      }
    }
  }
  if (LONG) {
    loss.add(r.loss);
    r.loss = loss.value32();
    if (REF) {
      kl.add(r.kl);
      r.kl = kl.value32();
    }
  }
  r.loss = warp_sum(r.loss);
  if (REF) r.kl = warp_sum(r.kl);
  r.clipped = __reduce_add_sync(0xffffffffu, r.clipped);
  r.count = __reduce_add_sync(0xffffffffu, r.count);
  return r;
}

__device__ __forceinline__ void policy_add(PolicyPart& sum, const SeqSum& r, int per_sequence) {
  if (r.count == 0) return;
  const float n = static_cast<float>(r.count);
  sum.loss.add(per_sequence ? r.loss / n : r.loss);
  sum.kl.add(per_sequence ? r.kl / n : r.kl);
  sum.clipped.add(per_sequence ? static_cast<float>(r.clipped) / n : static_cast<float>(r.clipped));
  sum.tokens += r.count;
  sum.seqs += 1;
}
__device__ __forceinline__ void policy_join(PolicyPart& sum, const PolicyPart& p) {
  sum.loss.add(p.loss);
  sum.kl.add(p.kl);
  sum.clipped.add(p.clipped);
  sum.tokens += p.tokens;
  sum.seqs += p.seqs;
}
__device__ __forceinline__ Sum2 shfl_xor(const Sum2& v, int o) {
  return Sum2{__shfl_xor_sync(0xffffffffu, v.s, o), __shfl_xor_sync(0xffffffffu, v.c, o)};
}
// The 32 lanes' rows, in every lane.
__device__ __forceinline__ PolicyPart policy_warp_join(PolicyPart p) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const PolicyPart q = {shfl_xor(p.loss, o), shfl_xor(p.kl, o), shfl_xor(p.clipped, o), __shfl_xor_sync(0xffffffffu, p.tokens, o),
                          __shfl_xor_sync(0xffffffffu, p.seqs, o)};
    policy_join(p, q);
  }
  return p;
}
__device__ __forceinline__ float policy_weight(int count, int per_sequence, double f) {
  return count == 0 ? 0.0f : static_cast<float>(per_sequence ? f / count : f);
}

// W warps a sequence.
template <bool REF, bool VEC, bool TOK, bool LONG>
__global__ void __launch_bounds__(POL_THREADS, 4) policy_sum_kernel(const __grid_constant__ PolicyArgs a, int W, int* counts,
                                                                 PolicyPart* part, int parts) {
  __shared__ SeqSum red[POL_WARPS];
  __shared__ PolicyPart join[POL_WARPS];
  const int teams = POL_WARPS / W;
  const int lane = lane_id(), warp = warp_id(), team = warp / W, in_team = warp % W;
  grid_dependency_wait();
  grid_dependents_launch();
  PolicyPart sum = {};
  // all teams of a block make the same number of rounds: there are barriers inside
  for (long long s0 = static_cast<long long>(blockIdx.x) * teams; s0 < a.S; s0 += static_cast<long long>(gridDim.x) * teams) {
    const long long s = s0 + team;
    SeqSum r = {0.0f, 0.0f, 0, 0};
    if (s < a.S) r = policy_sequence<REF, VEC, TOK, LONG>(a, s, in_team, W);
    if (W > 1) {
      if (lane == 0) red[warp] = r;
      __syncthreads();
      r = red[team * W];
      for (int i = 1; i < W; ++i) {
        r.loss += red[team * W + i].loss;
        r.kl += red[team * W + i].kl;
        r.clipped += red[team * W + i].clipped;
        r.count += red[team * W + i].count;
      }
      __syncthreads();
    }
    if (in_team == 0 && lane == 0 && s < a.S) {
      if (in_bounds(a.err, s, 1, a.S, SITE_POLICY_OUT)) counts[s] = r.count;
      policy_add(sum, r, a.per_sequence);
    }
  }
  if (in_team == 0 && lane == 0) join[team] = sum;
  __syncthreads();
  if (threadIdx.x == 0 && in_bounds(a.err, blockIdx.x, 1, parts, SITE_POLICY_OUT)) {
    PolicyPart all = join[0];
    for (int i = 1; i < teams; ++i) policy_join(all, join[i]);
    part[blockIdx.x] = all;
  }
}

// All of it in one block: a warp takes every 32nd sequence.
template <bool REF, bool TOK>
__global__ void __launch_bounds__(POL_SMALL_THREADS) policy_small_kernel(const __grid_constant__ PolicyArgs a, float* stats,
                                                                         float* weight) {
  constexpr int WARPS = POL_SMALL_THREADS / 32;
  __shared__ PolicyPart join[WARPS];
  __shared__ int counts[POL_SMALL_S];
  __shared__ double factor;
  const int lane = lane_id(), warp = warp_id();
  grid_dependency_wait();
  grid_dependents_launch();
  PolicyPart sum = {};
  for (int s = warp; s < a.S; s += WARPS) {
    static_assert(POL_SMALL_T <= 32 * POL_LANE_TOKENS, "not LONG");
    const SeqSum r = policy_sequence<REF, false, TOK, false>(a, s, 0, 1);
    if (lane == 0) {
      counts[s] = r.count;
      policy_add(sum, r, a.per_sequence);
    }
  }
  if (lane == 0) join[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    static_assert(WARPS == 32, "a row for each lane");
    const PolicyPart all = policy_warp_join(join[lane]);
    const long long n = a.per_sequence ? all.seqs : all.tokens;
    const double f = n > 0 ? 1.0 / static_cast<double>(n) : 0.0;
    if (lane == 0) {
      factor = f;
      stats[0] = static_cast<float>(all.loss.value() * f);
      stats[1] = static_cast<float>(all.kl.value() * f);
      stats[2] = static_cast<float>(all.clipped.value() * f);
    }
  }
  __syncthreads();
  const int s = threadIdx.x;
  if (s < a.S && in_bounds(a.err, s, 1, a.S, SITE_POLICY_OUT)) weight[s] = policy_weight(counts[s], a.per_sequence, factor);
}

// stats = (loss, mean KL, share of clipped tokens); weight of each sequence's tokens.  The weights need the counts alone: only the first
// block adds the sums.
__global__ void __launch_bounds__(POL_THREADS) policy_join_kernel(const PolicyPart* part, int parts, const int* counts, long long S,
                                                                  int per_sequence, float* stats, float* weight, uint32_t* err) {
  __shared__ PolicyPart join[POL_WARPS];
  grid_dependency_wait();
  grid_dependents_launch();
  PolicyPart sum = {};
  constexpr int LOADS = (POL_MAX_BLOCKS + POL_THREADS - 1) / POL_THREADS;
  PolicyPart p[LOADS];
#pragma unroll
  for (int k = 0; k < LOADS; ++k) {
    const int i = threadIdx.x + k * POL_THREADS;
    p[k] = {};
    if (i < parts) p[k] = part[i];
  }
#pragma unroll
  for (int k = 0; k < LOADS; ++k) {
    if (blockIdx.x == 0) {
      policy_join(sum, p[k]);
    } else {
      sum.tokens += p[k].tokens;
      sum.seqs += p[k].seqs;
    }
  }
  if (blockIdx.x == 0) {
    sum = policy_warp_join(sum);
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum.tokens += __shfl_xor_sync(0xffffffffu, sum.tokens, o);
      sum.seqs += __shfl_xor_sync(0xffffffffu, sum.seqs, o);
    }
  }
  if (lane_id() == 0) join[warp_id()] = sum;
  __syncthreads();
  long long n = 0;
#pragma unroll
  for (int i = 0; i < POL_WARPS; ++i) n += per_sequence ? join[i].seqs : join[i].tokens;
  const double f = n > 0 ? 1.0 / static_cast<double>(n) : 0.0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    sum = join[0];
    for (int i = 1; i < POL_WARPS; ++i) policy_join(sum, join[i]);
    stats[0] = static_cast<float>(sum.loss.value() * f);
    stats[1] = static_cast<float>(sum.kl.value() * f);
    stats[2] = static_cast<float>(sum.clipped.value() * f);
  }
  const long long s = static_cast<long long>(blockIdx.x) * POL_THREADS + threadIdx.x;
  if (s < S && in_bounds(err, s, 1, S, SITE_POLICY_OUT)) {
    weight[s] = policy_weight(counts[s], per_sequence, f);
  }
}

// Quotients by T of indexes below 2^31 (Granlund and Montgomery's division by an invariant: shift = ceil(log2 T),
// mul = floor(2^(31 + shift) / T) + 1).
struct Divide {
  uint32_t mul;
  int shift;                 // 0: T = 1
};
__host__ __device__ inline uint32_t quotient(const Divide& d, uint32_t n) {
  return d.shift ? static_cast<uint32_t>((static_cast<uint64_t>(n) * d.mul >> 32) >> (d.shift - 1)) : n;
}

template <bool REF, bool VEC, bool TOK>
__global__ void __launch_bounds__(POL_THREADS) policy_grad_kernel(const __grid_constant__ PolicyArgs a, const Divide by_T, const float* dloss,
                                                                  const float* weight, float* dnll) {
  grid_dependency_wait();
  grid_dependents_launch();
  const long long n_el = a.S * a.T;
  const float dl = *dloss;
  const long long span = static_cast<long long>(POL_THREADS) * POL_TILE;
  constexpr int STEP = VEC ? 1 : POL_THREADS;
  // 64-bit division only where 31 bits do not hold the index
  auto sequence = [&](long long t) -> long long { return n_el <= 0x7fffffff ? quotient(by_T, static_cast<uint32_t>(t)) : t / a.T; };
  for (long long i0 = blockIdx.x * span + threadIdx.x * (VEC ? POL_TILE : 1); i0 < n_el; i0 += gridDim.x * span) {
    static_assert(POL_TILE == 4, "load4");
    int lab[4];
    float nll[4], old[4], ref[4], adv[4], w[4], grad[4];
    bool there[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) there[i] = i0 + i * STEP < n_el;
    load4<REF, VEC, TOK>(a, i0, STEP, there, lab, nll, old, ref, adv);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long t = i0 + i * STEP;
      if (VEC && i > 0) {                                // T is a multiple of 4: one sequence's
        w[i] = w[0];
        if (!TOK) adv[i] = adv[0];
        continue;
      }
      w[i] = 0.0f;
      if (!TOK) adv[i] = 0.0f;
      if (!there[i] || !in_bounds(a.err, t, 1, n_el, SITE_POLICY_IN)) continue;
      const long long s = sequence(t);
      if (!TOK) adv[i] = a.adv[s];
      w[i] = weight[s];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      grad[i] = lab[i] < 0 ? 0.0f : policy_token<REF>(a, policy_side(a, adv[i]), nll[i], old[i], ref[i]).grad * (w[i] * dl);
    if constexpr (VEC) {
      if (in_bounds(a.err, i0, 4, n_el, SITE_POLICY_OUT)) *reinterpret_cast<float4*>(dnll + i0) = make_float4(grad[0], grad[1], grad[2], grad[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (there[i] && in_bounds(a.err, i0 + i * STEP, 1, n_el, SITE_POLICY_OUT)) dnll[i0 + i * STEP] = grad[i];
    }
  }
}

int policy_blocks(long long units) {
  return static_cast<int>(units < 1 ? 1 : units < POL_MAX_BLOCKS ? units : POL_MAX_BLOCKS);
}

// Warps a sequence: as many as leave each lane at most 16 tokens, up to a whole block.  More of them for few sequences make more partial rows:
// 1024 x 448 tokens forward 11.9 us with one warp, 13.2 with four.
int policy_warps(long long T) {
  int w = 1;
  while (w < POL_WARPS && T > 512LL * w) w *= 2;
  return w;
}

bool aligned_to(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Arguments that both directions share.
wb_status policy_args(PolicyArgs& a, const float* nll, const float* old_nll, const float* ref_nll, const float* advantage,
                      int advantage_per_token, const int64_t* labels, int64_t S, int64_t T, double clip_low, double clip_high,
                      float kl_weight, bool& empty) {
  if (S < 0 || T < 0 || S > (1LL << 31) || T > (1LL << 30) || (T > 0 && S > (1LL << 40) / T)) return WB_EINVAL;
  if (!(clip_low >= 0.0 && clip_low <= 1.0) || !(clip_high >= 0.0 && clip_high <= 1e30)) return WB_EINVAL;
  if (!std::isfinite(kl_weight) || (kl_weight != 0.0f && !ref_nll && S > 0 && T > 0)) return WB_EINVAL;
  empty = S == 0 || T == 0;
  if (empty) return WB_OK;
  if (!nll || !old_nll || !advantage || !labels || !aligned_to(nll, 4) || !aligned_to(old_nll, 4) || !aligned_to(ref_nll, 4) ||
      !aligned_to(advantage, 4) || !aligned_to(labels, 8))
    return WB_EINVAL;
  const double hi = std::log1p(clip_high), lo = std::log1p(-clip_low);
  a.nll = nll;
  a.old_nll = old_nll;
  a.ref_nll = ref_nll;
  a.adv = advantage;
  a.labels = labels;
  a.S = S;
  a.T = T;
  a.adv_tok = advantage_per_token ? 1 : 0;
  a.hi0 = static_cast<float>(hi);
  a.hi1 = static_cast<float>(hi - a.hi0);
  a.lo0 = static_cast<float>(lo);
  a.lo1 = std::isfinite(lo) ? static_cast<float>(lo - a.lo0) : 0.0f;
  a.hold_hi = static_cast<float>(1.0 + clip_high);
  a.hold_lo = static_cast<float>(1.0 - clip_low);
  a.beta = kl_weight;
  a.per_sequence = 0;
  a.err = nullptr;
  return WB_OK;
}

// Four tokens side by side are of one sequence and lie on 16 bytes.
bool policy_vec(const PolicyArgs& a) {
  return a.T % 4 == 0 && aligned16(a.nll) && aligned16(a.old_nll) && aligned16(a.ref_nll) && aligned16(a.labels) &&
         (!a.adv_tok || aligned16(a.adv));
}

// f(with a reference, vec, an advantage for each token), as types.
template <typename F>
cudaError_t choose(const PolicyArgs& a, bool vec, F f) {
  const std::true_type yes;
  const std::false_type no;
  auto tok = [&](auto r, auto v) { return a.adv_tok ? f(r, v, yes) : f(r, v, no); };
  if (a.ref_nll) return vec ? tok(yes, yes) : tok(yes, no);
  return vec ? tok(no, yes) : tok(no, no);
}

bool policy_small(int64_t S, int64_t T) { return S <= POL_SMALL_S && T <= POL_SMALL_T; }

struct PolicyWs {
  size_t part, counts, total;
};
PolicyWs policy_ws(int64_t S) {
  Carver c;
  PolicyWs w;
  w.part = c.take(sizeof(PolicyPart) * POL_MAX_BLOCKS);
  w.counts = c.take(sizeof(int) * static_cast<size_t>(S));
  w.total = c.off;
  return w;
}

}  // namespace
}  // namespace wb

using namespace wb;

extern "C" {

size_t wb_policy_loss_workspace_bytes(int64_t S, int64_t T) {
  if (S < 1 || T < 1 || S > (1LL << 31) || T > (1LL << 30) || S > (1LL << 40) / T) return 0;
  return policy_small(S, T) ? 0 : policy_ws(S).total;
}

wb_status wb_policy_loss(const float* nll, const float* old_nll, const float* ref_nll, const float* advantage,
                         int advantage_per_token, const int64_t* labels, int64_t S, int64_t T, double clip_low,
                         double clip_high, float kl_weight, int per_sequence, float* stats, float* weight, void* workspace,
                         size_t workspace_bytes, void* stream) {
  PolicyArgs a;
  bool empty = false;
  const wb_status st = policy_args(a, nll, old_nll, ref_nll, advantage, advantage_per_token, labels, S, T, clip_low, clip_high,
                                   kl_weight, empty);
  if (st != WB_OK) return st;
  if (!stats || !aligned_to(stats, 4) || (S > 0 && (!weight || !aligned_to(weight, 4)))) return WB_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (empty) {
    WB_CUDA(cudaMemsetAsync(stats, 0, 3 * sizeof(float), s));
    if (S > 0) WB_CUDA(cudaMemsetAsync(weight, 0, sizeof(float) * static_cast<size_t>(S), s));
    return WB_OK;
  }
  const bool small = policy_small(S, T);
  if (!small && (!workspace || !aligned16(workspace) || workspace_bytes < policy_ws(S).total)) return WB_EWORKSPACE;
  a.per_sequence = per_sequence != 0;
  a.err = tc_err_ptr();
  if (!a.err) return WB_ECUDA;
  if (small) {
    Prof pr(PC_POLICY, s);
    WB_CUDA(choose(a, false, [&](auto ref, auto, auto tok) {
      return launch_pdl(policy_small_kernel<decltype(ref)::value, decltype(tok)::value>, dim3(1), dim3(POL_SMALL_THREADS), 0, s, a, stats, weight);
    }));
    return WB_OK;
  }
  const PolicyWs w = policy_ws(S);
  auto* part = reinterpret_cast<PolicyPart*>(static_cast<char*>(workspace) + w.part);
  int* counts = reinterpret_cast<int*>(static_cast<char*>(workspace) + w.counts);
  const int warps = policy_warps(T);
  const int teams = POL_WARPS / warps;
  const int blocks = policy_blocks((S + teams - 1) / teams);
  Prof pr(PC_POLICY, s, 2);
  const bool is_long = T > 32LL * warps * POL_LANE_TOKENS;
  WB_CUDA(choose(a, policy_vec(a), [&](auto ref, auto vec, auto tok) {
    constexpr bool R = decltype(ref)::value, V = decltype(vec)::value, K = decltype(tok)::value;
    return launch_pdl(is_long ? policy_sum_kernel<R, V, K, true> : policy_sum_kernel<R, V, K, false>, dim3(blocks), dim3(POL_THREADS), 0, s, a, warps,
                      counts, part, blocks);
  }));
  WB_CUDA(launch_pdl(policy_join_kernel, dim3(static_cast<unsigned>((S + POL_THREADS - 1) / POL_THREADS)), dim3(POL_THREADS), 0, s,
                     static_cast<const PolicyPart*>(part), blocks, static_cast<const int*>(counts), static_cast<long long>(S),
                     a.per_sequence, stats, weight, a.err));
  return WB_OK;
}

wb_status wb_policy_loss_backward(const float* dloss, const float* nll, const float* old_nll, const float* ref_nll,
                                  const float* advantage, int advantage_per_token, const int64_t* labels, const float* weight,
                                  int64_t S, int64_t T, double clip_low, double clip_high, float kl_weight, float* dnll,
                                  void* stream) {
  PolicyArgs a;
  bool empty = false;
  const wb_status st = policy_args(a, nll, old_nll, ref_nll, advantage, advantage_per_token, labels, S, T, clip_low, clip_high,
                                   kl_weight, empty);
  if (st != WB_OK) return st;
  if (empty) return WB_OK;
  if (!dloss || !weight || !dnll || !aligned_to(dloss, 4) || !aligned_to(weight, 4) || !aligned_to(dnll, 4)) return WB_EINVAL;
  a.err = tc_err_ptr();
  if (!a.err) return WB_ECUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Prof pr(PC_POLICY, s);
  const long long span = static_cast<long long>(POL_THREADS) * POL_TILE;
  const long long units = (a.S * a.T + span - 1) / span;
  const int blocks = static_cast<int>(units < 8LL * POL_MAX_BLOCKS ? units : 8LL * POL_MAX_BLOCKS);
  Divide by_T{0, 0};
  while ((1LL << by_T.shift) < T) ++by_T.shift;
  by_T.mul = by_T.shift ? static_cast<uint32_t>((1ull << (31 + by_T.shift)) / static_cast<uint64_t>(T) + 1) : 0;
  WB_CUDA(choose(a, policy_vec(a) && aligned16(dnll), [&](auto ref, auto vec, auto tok) {
    return launch_pdl(policy_grad_kernel<decltype(ref)::value, decltype(vec)::value, decltype(tok)::value>, dim3(blocks), dim3(POL_THREADS), 0, s, a,
                      by_T, dloss, weight, dnll);
  }));
  return WB_OK;
}

}  // extern "C"
