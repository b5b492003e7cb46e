// The global norm of many gradients and clipping by it: norm = sqrt(sum over all tensors of g^2), and
// out_i = g_i * min(1, max_norm / norm), in place or into tensors of the same type or float32.
//
// Bound by memory: every gradient is read for the norm and, where it has to be scaled, once more for that.
// Both passes cut the tensors into chunks of 32 KB (gradients' bytes) that a grid of resident blocks
// takes in turn; the table of tensors travels as a kernel argument (up to 32 KB), so that nothing is
// uploaded and a call can be captured.  The second pass walks the chunks from the end: what the first
// pass read last is still in L2.
// 79 M bf16 elements: norm alone 27 us, in place 74, into tensors of the same type 77, into float32 106.  Beside memory there is
// float64: every thread joins the partial sums and takes the root and the quotient.  Its pipe is busy for 12 % of the scaling pass and
// 20 % of the norm's over 64 M elements (9 and 5 us), and a small call pays the same before its first store: 3.6 M float32 in 20
// tensors take 18 us for a floor of 4.
//
// Numbers.  A thread adds the squares of at most 128 elements in 32 bits (four or eight chains), the rest of the sum is in
// 64 bits and in a fixed order: the same call gives the same bits.  Squares of elements above 2^63 are
// infinite in 32 bits, and of elements below 2^-63 they lose digits or vanish: a thread whose sum is infinite or below 2^-90 although an
// element is not zero reads its elements again, scaled by 2^-100 or 2^100, so that the norm is right over
// the whole range of the types.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <type_traits>

#include "../../include/wb.h"
#include "internal.h"
#include "ptx.cuh"

namespace wb {
namespace {

constexpr int CLIP_THREADS = 256;
constexpr int CLIP_LOADS = 8;                                    // of 16 bytes a thread and chunk
constexpr int CLIP_CHUNK_BYTES = CLIP_THREADS * CLIP_LOADS * 16;
constexpr int CLIP_BLOCKS_PER_SM = 4;
constexpr int CLIP_MAX_BLOCKS = 1024;                            // of a launch: partial sums it leaves
// Entries of a launch's table.  Two sizes: arguments are copied with the launch.
constexpr int CLIP_TABLE = 960, CLIP_TABLE_SMALL = 96;

struct ClipEntry {
  const void* g;
  void* out;
  long long n;
  uint32_t chunk0;       // the entry's first chunk
  uint16_t head;         // elements before g's first 16-byte boundary (all of them taken with the first chunk)
  uint8_t type, out_type;
};
template <int N>
struct ClipTable {
  int n;                 // entries
  uint32_t chunks;       // of all of them
  uint32_t* err;
  ClipEntry e[N];
};
static_assert(sizeof(ClipTable<CLIP_TABLE>) + 64 <= 32764, "kernel arguments");

struct ClipScale {
  const double* part;
  int parts;
  float max_norm;
  float* norm;           // written by the first block, null in all but the first launch
};

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

template <typename T>
constexpr int clip_vec() { return 16 / static_cast<int>(sizeof(T)); }
template <typename T>
constexpr int clip_elems() { return CLIP_CHUNK_BYTES / static_cast<int>(sizeof(T)); }

// 16 bytes of T as floats
__device__ __forceinline__ void widen(const uint4& w, float (&v)[4], float) {
  v[0] = __uint_as_float(w.x);
  v[1] = __uint_as_float(w.y);
  v[2] = __uint_as_float(w.z);
  v[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void widen(const uint4& w, float (&v)[8], __nv_bfloat16) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const uint4& w, float (&v)[8], __half) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Range of the entry's elements that chunk c of it covers: [lo, hi), of which [lo, a) come before the first
// 16-byte boundary.
struct ClipSpan {
  long long lo, a, hi;
};
template <typename T>
__device__ __forceinline__ ClipSpan clip_span(const ClipEntry& e, uint32_t c) {
  ClipSpan s;
  s.a = e.head + static_cast<long long>(c) * clip_elems<T>();
  s.lo = c == 0 ? 0 : s.a;
  s.hi = min(e.n, s.a + clip_elems<T>());
  s.a = min(s.a, s.hi);
  return s;
}

// The elements of a span that thread t has, one by one: the same ones as the vector path's.
template <typename T, typename F>
__device__ __forceinline__ void clip_each(const ClipSpan& s, F f) {
  constexpr int V = clip_vec<T>();
  const int t = threadIdx.x;
  if (s.lo + t < s.a) f(s.lo + t);
  for (long long i = s.a + t * V; i < s.hi; i += CLIP_THREADS * V)
    for (long long j = i; j < min(i + V, s.hi); ++j) f(j);
}

template <typename T>
__device__ __forceinline__ double clip_sum_squares(const ClipEntry& e, uint32_t c, uint32_t* err) {
  constexpr int V = clip_vec<T>();
  const T* g = static_cast<const T*>(e.g);
  const ClipSpan s = clip_span<T>(e, c);
  const int t = threadIdx.x;
  float acc[V];
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  auto one = [&](long long i) {
    if (!in_bounds(err, i, 1, e.n, SITE_CLIP_IN)) return;
    const float x = to_f32(g[i]);
    bits |= __float_as_uint(x) & 0x7fffffffu;
    acc[0] = fmaf(x, x, acc[0]);
  };
  if (s.lo + t < s.a) one(s.lo + t);
  if (s.hi - s.a == clip_elems<T>()) {
    uint4 w[CLIP_LOADS];
    const uint4* p = reinterpret_cast<const uint4*>(g + s.a) + t;
    if (in_bounds(err, s.a, clip_elems<T>(), e.n, SITE_CLIP_IN)) {
#pragma unroll
      for (int k = 0; k < CLIP_LOADS; ++k) w[k] = p[k * CLIP_THREADS];
    }
#pragma unroll
    for (int k = 0; k < CLIP_LOADS; ++k) {
      float v[V];
      widen(w[k], v, T());
      bits |= (w[k].x | w[k].y | w[k].z | w[k].w) & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(v[i], v[i], acc[i]);
    }
  } else {
    for (long long i = s.a + t * V; i < s.hi; i += CLIP_THREADS * V) {
      if (i + V <= s.hi) {
        if (!in_bounds(err, i, V, e.n, SITE_CLIP_IN)) continue;
        const uint4 w = *reinterpret_cast<const uint4*>(g + i);
        float v[V];
        widen(w, v, T());
        bits |= (w.x | w.y | w.z | w.w) & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu);
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(v[j], v[j], acc[j]);
      } else {
        for (long long j = i; j < s.hi; ++j) one(j);
      }
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) sum += acc[i];
  if (sum >= 0x1p-90f && sum <= 0x1.fffffep127f) return static_cast<double>(sum);
  if (bits == 0) return 0.0;
  // outside of what squares in 32 bits can hold (or not finite at all): the same elements, scaled
  const bool large = !(sum < 0x1p-90f);
  const float k = large ? 0x1p-100f : 0x1p100f;
  float r = 0.0f;
  clip_each<T>(s, [&](long long i) {
    if (!in_bounds(err, i, 1, e.n, SITE_CLIP_IN)) return;
    const float x = to_f32(g[i]) * k;
    r = fmaf(x, x, r);
  });
  return static_cast<double>(r) * (large ? 0x1p200 : 0x1p-200);
}

// Sum over the block in a fixed order; every thread gets it.
__device__ __forceinline__ double clip_block_sum(double v) {
  __shared__ double red[CLIP_THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane_id() == 0) red[warp_id()] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < CLIP_THREADS / 32; ++i) v += red[i];
  return v;
}

// The entry of chunk c: the last one that starts at or before it (entries without elements have no chunk).
template <int N>
__device__ __forceinline__ int clip_find(const ClipTable<N>& t, uint32_t c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].chunk0 <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int N>
__global__ void __launch_bounds__(CLIP_THREADS, CLIP_BLOCKS_PER_SM)
    clip_norm_kernel(const __grid_constant__ ClipTable<N> t, double* part, int parts) {
  grid_dependency_wait();
  grid_dependents_launch();
  double sum = 0.0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const ClipEntry& e = t.e[clip_find(t, c)];
    const uint32_t k = c - e.chunk0;
    if (e.type == WB_BF16) sum += clip_sum_squares<__nv_bfloat16>(e, k, t.err);
    else if (e.type == WB_F16) sum += clip_sum_squares<__half>(e, k, t.err);
    else sum += clip_sum_squares<float>(e, k, t.err);
  }
  sum = clip_block_sum(sum);
  if (threadIdx.x == 0 && in_bounds(t.err, blockIdx.x, 1, parts, SITE_CLIP_PART)) part[blockIdx.x] = sum;
}

// N elements of T, one load, as floats; and back
template <int N, typename T>
__device__ __forceinline__ void load_wide(const T* g, float (&v)[N]) {
  if constexpr (sizeof(T) * N == 16) {
    widen(*reinterpret_cast<const uint4*>(g), v, T());
  } else {
    static_assert(sizeof(T) == 2 && N == 4, "8 bytes");
    const uint2 w = *reinterpret_cast<const uint2*>(g);
    float u[8];
    widen(make_uint4(w.x, w.y, 0, 0), u, T());
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = u[i];
  }
}
__device__ __forceinline__ void narrow(const float (&v)[4], float s, float* out) {
  *reinterpret_cast<float4*>(out) = make_float4(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
}
__device__ __forceinline__ void narrow(const float (&v)[8], float s, __nv_bfloat16* out) {
  *reinterpret_cast<uint4*>(out) = make_uint4(pack_bf16(v[0] * s, v[1] * s), pack_bf16(v[2] * s, v[3] * s),
                                              pack_bf16(v[4] * s, v[5] * s), pack_bf16(v[6] * s, v[7] * s));
}
__device__ __forceinline__ void narrow(const float (&v)[8], float s, __half* out) {
  *reinterpret_cast<uint4*>(out) = make_uint4(pack_f16(v[0] * s, v[1] * s), pack_f16(v[2] * s, v[3] * s),
                                              pack_f16(v[4] * s, v[5] * s), pack_f16(v[6] * s, v[7] * s));
}

// Vectors are 16 bytes of the output: float32 from 16 bits by 8-byte loads, so that a warp's stores are whole lines (with 16-byte
// loads each store left every second 16 bytes to the next one: 79 M elements 130 us for the whole call, now 108).
template <typename T, typename O>
__device__ __forceinline__ void clip_scale(const ClipEntry& e, uint32_t c, float k, uint32_t* err) {
  constexpr int V = 16 / static_cast<int>(sizeof(O)), BATCH = CLIP_LOADS;
  constexpr int ROUNDS = clip_elems<T>() / (V * CLIP_THREADS * BATCH);
  const T* g = static_cast<const T*>(e.g);
  O* out = static_cast<O*>(e.out);
  const ClipSpan s = clip_span<T>(e, c);
  const int t = threadIdx.x;
  // a factor of 1 copies: products would change a NaN's bits
  const bool copy = std::is_same<T, O>::value && k == 1.0f;
  auto one = [&](long long i) {
    if (!in_bounds(err, i, 1, e.n, SITE_CLIP_OUT)) return;
    if (copy) reinterpret_cast<T*>(out)[i] = g[i];
    else out[i] = from_f32<O>(to_f32(g[i]) * k);
  };
  // two tensors whose 16-byte boundaries lie at different elements go one element at a time
  if (reinterpret_cast<uintptr_t>(out + e.head) & 15u) {
    for (long long i = s.lo + t; i < s.hi; i += CLIP_THREADS) one(i);
    return;
  }
  if (s.lo + t < s.a) one(s.lo + t);
  // one load in flight a thread, as g and out may be the same memory to the compiler: 79 M bf16 87 us, 77 scaled
  if (copy) {
    constexpr int W = clip_vec<T>();
    for (long long i = s.a + t * W; i < s.hi; i += CLIP_THREADS * W) {
      if (i + W <= s.hi) {
        if (in_bounds(err, i, W, e.n, SITE_CLIP_OUT)) *reinterpret_cast<uint4*>(out + i) = *reinterpret_cast<const uint4*>(g + i);
      } else {
        for (long long j = i; j < s.hi; ++j) one(j);
      }
    }
    return;
  }
  if (s.hi - s.a == clip_elems<T>()) {
    if (!in_bounds(err, s.a, clip_elems<T>(), e.n, SITE_CLIP_OUT)) return;
#pragma unroll 1
    for (int r = 0; r < ROUNDS; ++r) {
      const long long at = s.a + (static_cast<long long>(r) * BATCH * CLIP_THREADS + t) * V;
      float v[BATCH][V];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) load_wide<V>(g + at + i * CLIP_THREADS * V, v[i]);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) narrow(v[i], k, out + at + i * CLIP_THREADS * V);
    }
    return;
  }
  for (long long i = s.a + t * V; i < s.hi; i += CLIP_THREADS * V) {
    if (i + V <= s.hi) {
      if (!in_bounds(err, i, V, e.n, SITE_CLIP_OUT)) continue;
      float v[V];
      load_wide<V>(g + i, v);
      narrow(v, k, out + i);
    } else {
      for (long long j = i; j < s.hi; ++j) one(j);
    }
  }
}

// The norm from the partial sums (every block, in the same order) and the factor: below 1 only where a finite
// norm is above max_norm.
__device__ __forceinline__ float clip_factor(const ClipScale& s, uint32_t* err, double& norm) {
  double v = 0.0;
  for (int i = threadIdx.x; i < s.parts; i += CLIP_THREADS)
    if (in_bounds(err, i, 1, s.parts, SITE_CLIP_PART)) v += s.part[i];
  norm = sqrt(clip_block_sum(v));
  const float n32 = static_cast<float>(norm);
  if (s.norm && blockIdx.x == 0 && threadIdx.x == 0) *s.norm = n32;
  return norm > s.max_norm && isfinite(n32) ? static_cast<float>(s.max_norm / norm) : 1.0f;
}

// A factor below float32's normal range, in float64: gradients of 2^119 clipped to 2^-27 are ordinary numbers, although the factor would be
// 0 in float32, or keep few of its digits.
template <typename T, typename O>
__device__ __forceinline__ void clip_scale_tiny(const ClipEntry& e, uint32_t c, double f, uint32_t* err) {
  const T* g = static_cast<const T*>(e.g);
  O* out = static_cast<O*>(e.out);
  const ClipSpan s = clip_span<T>(e, c);
  for (long long i = s.lo + threadIdx.x; i < s.hi; i += CLIP_THREADS)
    if (in_bounds(err, i, 1, e.n, SITE_CLIP_OUT)) out[i] = from_f32<O>(static_cast<float>(static_cast<double>(to_f32(g[i])) * f));
}
template <int N>
__device__ __forceinline__ void clip_scale_tiny(const ClipTable<N>& t, double f) {
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const ClipEntry& e = t.e[clip_find(t, c)];
    const uint32_t j = c - e.chunk0;
    const bool wide = e.out_type == WB_F32;
    if (e.type == WB_F32) clip_scale_tiny<float, float>(e, j, f, t.err);
    else if (e.type == WB_F16) wide ? clip_scale_tiny<__half, float>(e, j, f, t.err) : clip_scale_tiny<__half, __half>(e, j, f, t.err);
    else if (wide) clip_scale_tiny<__nv_bfloat16, float>(e, j, f, t.err);
    else clip_scale_tiny<__nv_bfloat16, __nv_bfloat16>(e, j, f, t.err);
  }
}

template <int N>
__global__ void __launch_bounds__(CLIP_THREADS, CLIP_BLOCKS_PER_SM)
    clip_scale_kernel(const __grid_constant__ ClipTable<N> t, const ClipScale s) {
  grid_dependency_wait();
  grid_dependents_launch();
  double norm;
  const float k = clip_factor(s, t.err, norm);
  if (k < 0x1p-126f && s.max_norm > 0.0f) {
    clip_scale_tiny(t, s.max_norm / norm);
    return;
  }
  for (uint32_t i = blockIdx.x; i < t.chunks; i += gridDim.x) {
    const uint32_t c = t.chunks - 1 - i;
    const ClipEntry& e = t.e[clip_find(t, c)];
    if (k == 1.0f && e.out == e.g) continue;       // nothing to do in place
    const uint32_t j = c - e.chunk0;
    if (e.type == WB_BF16) {
      if (e.out_type == WB_BF16) clip_scale<__nv_bfloat16, __nv_bfloat16>(e, j, k, t.err);
      else clip_scale<__nv_bfloat16, float>(e, j, k, t.err);
    } else if (e.type == WB_F16) {
      if (e.out_type == WB_F16) clip_scale<__half, __half>(e, j, k, t.err);
      else clip_scale<__half, float>(e, j, k, t.err);
    } else {
      clip_scale<float, float>(e, j, k, t.err);
    }
  }
}

__global__ void __launch_bounds__(CLIP_THREADS) clip_finish_kernel(const ClipScale s, uint32_t* err) {
  grid_dependency_wait();
  grid_dependents_launch();
  double norm;
  clip_factor(s, err, norm);
}

int elem_bytes(int type) { return type == WB_F32 ? 4 : 2; }

// Elements of a chunk, and before the first 16-byte boundary.
long long chunk_elems(int type) { return CLIP_CHUNK_BYTES / elem_bytes(type); }
long long head_elems(const void* p, long long n, int type) {
  const long long h = static_cast<long long>((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / elem_bytes(type);
  return h < n ? h : n;
}

struct ClipCall {
  const void* const* grads;
  void* const* outs;
  const int64_t* numel;
  const int32_t* types;
  const int32_t* out_types;
  int n;
};

template <int N>
void fill(ClipTable<N>& t, const ClipCall& a, int first, int last, uint32_t* err) {
  t.n = last - first;
  t.err = err;
  uint32_t c = 0;
  for (int i = first; i < last; ++i) {
    ClipEntry& e = t.e[i - first];
    e.g = a.grads[i];
    e.out = a.outs ? a.outs[i] : nullptr;
    e.n = a.numel[i];
    e.type = static_cast<uint8_t>(a.types[i]);
    e.out_type = static_cast<uint8_t>(a.outs ? a.out_types[i] : a.types[i]);
    e.chunk0 = c;
    const long long head = head_elems(e.g, e.n, e.type);
    e.head = static_cast<uint16_t>(head);
    const long long body = e.n - head, per = chunk_elems(e.type);
    if (e.n > 0) c += static_cast<uint32_t>(body > 0 ? (body + per - 1) / per : 1);
  }
  t.chunks = c;
}

int clip_grid(uint32_t chunks) {
  const int most = std::min(CLIP_MAX_BLOCKS, sm_count() * CLIP_BLOCKS_PER_SM);
  return static_cast<int>(std::min<uint32_t>(chunks > 0 ? chunks : 1, static_cast<uint32_t>(most)));
}

template <int N>
cudaError_t clip_launches(const ClipCall& a, float max_norm, float* norm, double* part, uint32_t* err, cudaStream_t s) {
  ClipTable<N> t;
  int parts = 0;
  for (int first = 0; first < a.n; first += N) {
    fill(t, a, first, std::min(a.n, first + N), err);
    const int grid = clip_grid(t.chunks);
    const cudaError_t e = launch_pdl(clip_norm_kernel<N>, dim3(grid), dim3(CLIP_THREADS), 0, s, t, part + parts, grid);
    if (e != cudaSuccess) return e;
    parts += grid;
  }
  ClipScale sc{part, parts, max_norm, norm};
  if (!a.outs) return launch_pdl(clip_finish_kernel, dim3(1), dim3(CLIP_THREADS), 0, s, sc, err);
  // the last tensors first: they were read last
  for (int first = (a.n - 1) / N * N; first >= 0; first -= N) {
    if (a.n > N) fill(t, a, first, std::min(a.n, first + N), err);
    const cudaError_t e = launch_pdl(clip_scale_kernel<N>, dim3(clip_grid(t.chunks)), dim3(CLIP_THREADS), 0, s, t, sc);
    if (e != cudaSuccess) return e;
    sc.norm = nullptr;
  }
  return cudaSuccess;
}

// Tables, and so launches of a pass, that n tensors take.
int clip_tables(int n) { return n <= CLIP_TABLE_SMALL ? 1 : (n + CLIP_TABLE - 1) / CLIP_TABLE; }

struct Extent {
  uintptr_t lo, hi;
};

bool type_ok(int t) { return t == WB_BF16 || t == WB_F16 || t == WB_F32; }

}  // namespace
}  // namespace wb

using namespace wb;

extern "C" {

size_t wb_clip_grad_norm_workspace_bytes(int n_tensors) {
  if (n_tensors < 1 || n_tensors > WB_CLIP_MAX_TENSORS) return 0;
  return static_cast<size_t>(clip_tables(n_tensors)) * CLIP_MAX_BLOCKS * sizeof(double);
}

wb_status wb_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* numel, const int32_t* dtypes,
                            const int32_t* out_dtypes, int n_tensors, float max_norm, float* norm, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (n_tensors < 0 || n_tensors > WB_CLIP_MAX_TENSORS || !norm || (reinterpret_cast<uintptr_t>(norm) & 3u)) return WB_EINVAL;
  if (outs && !(max_norm >= 0.0f)) return WB_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n_tensors == 0) {
    WB_CUDA(cudaMemsetAsync(norm, 0, sizeof(float), s));
    return WB_OK;
  }
  if (!grads || !numel || !dtypes || (outs && !out_dtypes)) return WB_EINVAL;
  for (int i = 0; i < n_tensors; ++i) {
    if (!type_ok(dtypes[i])) return WB_EUNSUPPORTED;
    if (outs && out_dtypes[i] != dtypes[i] && out_dtypes[i] != WB_F32) return WB_EUNSUPPORTED;
    if (numel[i] < 0 || numel[i] > (1LL << 40)) return WB_EINVAL;
    if (numel[i] == 0) continue;
    if (!grads[i] || reinterpret_cast<uintptr_t>(grads[i]) % elem_bytes(dtypes[i])) return WB_EINVAL;
    if (outs && (!outs[i] || reinterpret_cast<uintptr_t>(outs[i]) % elem_bytes(out_dtypes[i]))) return WB_EINVAL;
    if (outs && outs[i] == grads[i] && out_dtypes[i] != dtypes[i]) return WB_EINVAL;
  }
  if (outs) {
    // what is written overlaps nothing but, exactly, its own gradient
    Extent* x = new (std::nothrow) Extent[2 * static_cast<size_t>(n_tensors)];
    if (!x) return WB_EINVAL;
    int m = 0;
    for (int i = 0; i < n_tensors; ++i) {
      if (numel[i] == 0) continue;
      const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]), o = reinterpret_cast<uintptr_t>(outs[i]);
      x[m++] = Extent{g, g + static_cast<uintptr_t>(numel[i]) * elem_bytes(dtypes[i])};
      if (o != g) x[m++] = Extent{o, o + static_cast<uintptr_t>(numel[i]) * elem_bytes(out_dtypes[i])};
    }
    std::sort(x, x + m, [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
    bool apart = true;
    for (int i = 1; i < m; ++i) apart = apart && x[i - 1].hi <= x[i].lo;
    delete[] x;
    if (!apart) return WB_EINVAL;
  }
  if (!workspace || !aligned16(workspace) || workspace_bytes < wb_clip_grad_norm_workspace_bytes(n_tensors))
    return WB_EWORKSPACE;
  uint32_t* err = tc_err_ptr();
  if (!err) return WB_ECUDA;
  const ClipCall a{grads, outs, numel, dtypes, out_dtypes, n_tensors};
  double* part = static_cast<double*>(workspace);
  Prof pr(PC_CLIP, s, clip_tables(n_tensors) + (outs ? clip_tables(n_tensors) : 1));
  if (n_tensors <= CLIP_TABLE_SMALL) WB_CUDA(clip_launches<CLIP_TABLE_SMALL>(a, max_norm, norm, part, err, s));
  else WB_CUDA(clip_launches<CLIP_TABLE>(a, max_norm, norm, part, err, s));
  return WB_OK;
}

}  // extern "C"
