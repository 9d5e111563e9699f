// clip.cuh -- global gradient norm over many tensors, and clipping.
//
// norm = sqrt(sum over all tensors of sum g^2), coef = min(1, max_norm /
// (norm + 1e-6)), out = coef * g: the clip of the training step (optim.cuh)
// for gradients that do not lie in one flat buffer.
//
// Two launches whatever the number of tensors (up to CLIP_MAX_TENSORS a
// launch): the tensors' addresses and sizes travel in the kernel parameters,
// so nothing is copied to the device and a captured call replays as it is.
// Every tensor is cut into pieces of CLIP_PIECE bytes; block b takes the
// pieces b, b + grid, ...  The first kernel adds the squares in fp64 (a square
// of any fp32 value is a normal fp64 number, so nothing overflows or vanishes;
// the fp64 pipes keep pace with HBM) and leaves one partial per block; the
// second has every block add the partials in the same order, so that no third
// launch and no counter is needed, and then scales.  No atomics: the result
// depends on the sizes alone.  Memory bounds both: the gradients are read twice
// (the second pass walks backwards, so that it finds what L2 still holds) and
// written once; the second read and the write are skipped when the clip is off
// or changes nothing in place.  B200, 114 M fp32 elements in 49 tensors to other
// memory: 227 us (1.37 GB, 6.0 TB/s).
#pragma once
#include "common.cuh"

// blocks of a launch at most, and partials it leaves: 8 for each of 148 SMs, where 6 (sums,
// 38 registers) and 3 (scaling, 79) are resident at a time; the others follow behind them
constexpr int CLIP_BLOCKS = 1184;
constexpr int CLIP_THREADS = 256;
constexpr int CLIP_PIECE = 32768;        // bytes: eight 16-byte loads a thread, all in flight
constexpr int CLIP_MAX_TENSORS = 1024;   // a launch (28 KB of kernel parameters)
constexpr int CLIP_FEW_TENSORS = 128;    // the small table of the common case

template <int CAP> struct ClipTable {
  const void* g[CAP];
  void* out[CAP];
  unsigned long long size_bf16[CAP];  // elements * 2 + (1 if bf16)
  int piece0[CAP + 1];                // first piece of each tensor; [n] = all pieces
  int n;
};

// Tensor that piece c belongs to (piece0 ascends; empty tensors have no piece).
template <int CAP>
__device__ __forceinline__ int clip_find(const ClipTable<CAP>& t, int c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.piece0[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double sq_f64(float x) { const double d = x; return d * d; }

template <typename T>
__device__ __forceinline__ double clip_piece_sumsq(const T* __restrict__ g, long long n) {
  constexpr int E = 16 / sizeof(T), U = CLIP_PIECE / 16 / CLIP_THREADS;
  double s0 = 0.0, s1 = 0.0;
  if ((reinterpret_cast<uintptr_t>(g) & 15) == 0) {
    const long long nv = n / E;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = (long long)u * CLIP_THREADS + threadIdx.x;
      v[u] = i < nv ? __ldcg(reinterpret_cast<const uint4*>(g) + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const T* e = reinterpret_cast<const T*>(&v[u]);
#pragma unroll
      for (int k = 0; k < E; k += 2) { s0 += sq_f64(to_f(e[k])); s1 += sq_f64(to_f(e[k + 1])); }
    }
    const long long r = nv * E + threadIdx.x;
    if (r < n) s0 += sq_f64(to_f(g[r]));
  } else {
    for (long long i = threadIdx.x; i < n; i += CLIP_THREADS) s0 += sq_f64(to_f(g[i]));
  }
  return s0 + s1;
}

template <int CAP>
__global__ void __launch_bounds__(CLIP_THREADS) clip_sumsq_kernel(const __grid_constant__ ClipTable<CAP> t,
                                                                  double* __restrict__ part) {
  pdl_wait();
  __shared__ double sh[32];
  double s = 0.0;
  for (int c = blockIdx.x; c < t.piece0[t.n]; c += gridDim.x) {
    const int k = clip_find(t, c);
    const long long n = (long long)(t.size_bf16[k] >> 1);
    const bool lp = t.size_bf16[k] & 1;
    const long long per = lp ? CLIP_PIECE / 2 : CLIP_PIECE / 4, e0 = (long long)(c - t.piece0[k]) * per;
    const long long m = n - e0 < per ? n - e0 : per;
    s += lp ? clip_piece_sumsq(static_cast<const bf16*>(t.g[k]) + e0, m)
            : clip_piece_sumsq(static_cast<const float*>(t.g[k]) + e0, m);
  }
  s = warp_sum_d(s);
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  if (lane == 0) sh[wid] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double r = 0.0;
    for (int w = 0; w < CLIP_THREADS / 32; ++w) r += sh[w];
    part[blockIdx.x] = r;
  }
}

// out may be g itself: every element is read and written by the same thread.
template <typename T>
__device__ __forceinline__ void clip_piece_scale(const T* g, T* out, long long n, float coef) {
  constexpr int E = 16 / sizeof(T), U = CLIP_PIECE / 16 / CLIP_THREADS;
  if (((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
    const long long nv = n / E;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = (long long)u * CLIP_THREADS + threadIdx.x;
      if (i < nv) v[u] = __ldcg(reinterpret_cast<const uint4*>(g) + i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = (long long)u * CLIP_THREADS + threadIdx.x;
      if (i >= nv) continue;
      T* e = reinterpret_cast<T*>(&v[u]);
#pragma unroll
      for (int k = 0; k < E; ++k) e[k] = from_f<T>(to_f(e[k]) * coef);
      __stcs(reinterpret_cast<uint4*>(out) + i, v[u]);
    }
    const long long r = nv * E + threadIdx.x;
    if (r < n) out[r] = from_f<T>(to_f(g[r]) * coef);
  } else {
    for (long long i = threadIdx.x; i < n; i += CLIP_THREADS) out[i] = from_f<T>(to_f(g[i]) * coef);
  }
}

// parts: partials of all sum launches of the call.  max_norm = 0: norm only.
template <int CAP>
__global__ void __launch_bounds__(CLIP_THREADS) clip_scale_kernel(const __grid_constant__ ClipTable<CAP> t,
                                                                  const double* __restrict__ part, int parts,
                                                                  float max_norm, int in_place,
                                                                  float* __restrict__ norm_out, unsigned* err) {
  pdl_wait();
  __shared__ double sh[32];
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += CLIP_THREADS) s += part[i];
  s = warp_sum_d(s);
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  if (lane == 0) sh[wid] = s;
  __syncthreads();
  double total = 0.0;
  for (int w = 0; w < CLIP_THREADS / 32; ++w) total += sh[w];
  const double norm = sqrt(total);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (norm_out) *norm_out = (float)norm;
    if (!isfinite(norm)) set_error(err, GPT_EBIT_NONFINITE);
  }
  if (max_norm <= 0.f && in_place) return;
  // a norm that is not finite leaves the gradients as they are
  const float coef = max_norm > 0.f && isfinite(norm) ? (float)fmin(1.0, (double)max_norm / (norm + 1e-6)) : 1.f;
  if (coef == 1.f && in_place) return;
  for (int c = t.piece0[t.n] - 1 - (int)blockIdx.x; c >= 0; c -= (int)gridDim.x) {
    const int k = clip_find(t, c);
    const long long n = (long long)(t.size_bf16[k] >> 1);
    const bool lp = t.size_bf16[k] & 1;
    const long long per = lp ? CLIP_PIECE / 2 : CLIP_PIECE / 4, e0 = (long long)(c - t.piece0[k]) * per;
    const long long m = n - e0 < per ? n - e0 : per;
    if (lp) clip_piece_scale(static_cast<const bf16*>(t.g[k]) + e0, static_cast<bf16*>(t.out[k]) + e0, m, coef);
    else clip_piece_scale(static_cast<const float*>(t.g[k]) + e0, static_cast<float*>(t.out[k]) + e0, m, coef);
  }
}
