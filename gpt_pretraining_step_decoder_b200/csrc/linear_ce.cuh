// linear_ce.cuh -- softmax cross entropy of z = softcap(x W^T) over a large
// vocabulary without keeping the logits, and its gradient.
//
//   lse_i = log sum_v exp(z_iv),   loss_i = lse_i - z_i,target   (0 if ignored)
//   dz_iv = (exp(z_iv - lse_i) - [v = target_i]) g_i (1 - (z_iv / cap)^2)
//   dx = dz W,   dW = dz^T x
//
// bf16: the forward pass is one tensor-core GEMM whose epilogue reduces every
// 128-column half tile of a row to (max, sum of exp) in registers, so nothing
// of size N x V is ever written; ce_combine_kernel joins a row's pairs.  The
// backward pass walks the vocabulary in pieces: the logits of a piece once more,
// turned into dz (bf16) in that GEMM's epilogue, then the two gradient products
// on it; dx is summed over the pieces in fp32.  Three products of 2 N V d
// operations bound it.  fp32: the same pieces through plain FFMA products, with
// fp32 logits of one piece at a time in the workspace.
#pragma once
#include "common.cuh"

// (m, s) + (m2, s2) of sums s e^m; an empty part has m = -inf, s = 0
__device__ __forceinline__ void lse_join(float& m, float& s, float m2, float s2) {
  const float mx = fmaxf(m, m2);
  if (mx == -INFINITY) { s += s2; return; }  // both empty (a NaN sum stays)
  s = s * __expf(m - mx) + s2 * __expf(m2 - mx);
  m = mx;
}

// Loss of one row; counts it if its target is one.  Targets below -1 or past
// the vocabulary raise the input error and are ignored.
__device__ __forceinline__ float ce_row_loss(float lse, float zt, int y, int V, int& valid, unsigned* err) {
  valid = y >= 0 && y < V;
  if (y < -1 || y >= V) set_error(err, GPT_EBIT_INPUT);
  return valid ? lse - zt : 0.f;
}

// Block of 32 rows x 32 groups of half tiles; stats [n_tiles, N], so that a
// warp reads 32 neighbouring rows.  Leaves each row's lse and loss, and the
// block's loss sum (fp64) and count for ce_mean_kernel.
__global__ void __launch_bounds__(1024) ce_combine_kernel(const float2* __restrict__ stats, int n_tiles, int N, int V,
                                                          const int32_t* __restrict__ targets,
                                                          const float* __restrict__ ztgt, float* __restrict__ lse_out,
                                                          float* __restrict__ tok_loss, double2* __restrict__ part,
                                                          unsigned* err) {
  pdl_wait();
  __shared__ float2 sh[32][33];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + lane;
  float m = -INFINITY, s = 0.f;
  if (row < N) {
    constexpr int U = 4;  // pairs in flight per thread
    for (int j = grp; j < n_tiles; j += 32 * U) {
      float2 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = j + 32 * u < n_tiles ? stats[(long long)(j + 32 * u) * N + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int u = 0; u < U; ++u) lse_join(m, s, v[u].x, v[u].y);
    }
  }
  sh[grp][lane] = make_float2(m, s);
  __syncthreads();
  if (grp == 0) {
    for (int g = 1; g < 32; ++g) lse_join(m, s, sh[g][lane].x, sh[g][lane].y);
    double l = 0.0;
    int valid = 0;
    if (row < N) {
      const float lse = m + logf(s);
      const int y = targets[row];
      const float t = ce_row_loss(lse, y >= 0 && y < V ? ztgt[row] : 0.f, y, V, valid, err);
      if (lse_out) lse_out[row] = lse;
      if (tok_loss) tok_loss[row] = t;
      l = t;
    }
    l = warp_sum_d(l);
    const int c = __reduce_add_sync(0xffffffffu, valid);
    if (lane == 0) part[blockIdx.x] = make_double2(l, (double)c);
  }
}

// mean of the valid rows' losses, the blocks' sums added in a fixed order
__global__ void __launch_bounds__(1024) ce_mean_kernel(const double2* __restrict__ part, int parts,
                                                       float* __restrict__ loss, unsigned* err) {
  pdl_wait();
  __shared__ double sh[2][32];
  double l = 0.0, c = 0.0;
  for (int i = threadIdx.x; i < parts; i += blockDim.x) { const double2 p = part[i]; l += p.x; c += p.y; }
  l = warp_sum_d(l);
  c = warp_sum_d(c);
  if ((threadIdx.x & 31) == 0) { sh[0][threadIdx.x >> 5] = l; sh[1][threadIdx.x >> 5] = c; }
  __syncthreads();
  if (threadIdx.x == 0) {
    l = c = 0.0;
    for (int w = 0; w < 32; ++w) { l += sh[0][w]; c += sh[1][w]; }
    const float r = c > 0.0 ? (float)(l / c) : 0.f;
    if (!isfinite(r)) set_error(err, GPT_EBIT_NONFINITE);
    if (loss) *loss = r;
  }
}

// Gradient scale of every row: dtok[i], or dloss / count (dloss null: 1), 0 for
// ignored rows.  Every block counts the targets itself (they are few and in
// L2), so one launch does.
__global__ void __launch_bounds__(1024) ce_row_scale_kernel(const int32_t* __restrict__ targets, int N, int V,
                                                            const float* __restrict__ dloss,
                                                            const float* __restrict__ dtok, float* __restrict__ g,
                                                            unsigned* err) {
  pdl_wait();
  __shared__ int sh[32];
  float base = 0.f;
  if (!dtok) {
    int c = 0;
    for (int i = threadIdx.x; i < N; i += blockDim.x) { const int y = targets[i]; c += y >= 0 && y < V; }
    c = __reduce_add_sync(0xffffffffu, c);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = c;
    __syncthreads();
    c = __reduce_add_sync(0xffffffffu, sh[threadIdx.x & 31]);
    base = c > 0 ? (dloss ? *dloss : 1.f) / (float)c : 0.f;
  }
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < N; i += gridDim.x * blockDim.x) {
    const int y = targets[i];
    if (y < -1 || y >= V) set_error(err, GPT_EBIT_INPUT);
    g[i] = y >= 0 && y < V ? (dtok ? dtok[i] : base) : 0.f;
  }
}

// ---------------------------------------------------------------- fp32 pieces
// One block per row of a piece of fp32 logits z [N, width] (columns col0 ...):
// joins the piece's max and sum of exp to the row's, picks the target's logit.
// first: the row's pair starts here.
__global__ void __launch_bounds__(256) ce_piece_stats_kernel(const float* __restrict__ z, int width, int col0, int first,
                                                             float softcap, const int32_t* __restrict__ targets, int N,
                                                             float2* __restrict__ stats, float* __restrict__ ztgt) {
  pdl_wait();
  __shared__ float sh[32];
  const long long row = blockIdx.x;
  const float* r = z + row * width;
  auto cap = [&](float v) { return softcap > 0.f ? softcap * tanhf(v / softcap) : v; };
  float mx = -INFINITY;
  for (int i = threadIdx.x; i < width; i += blockDim.x) mx = fmaxf(mx, cap(r[i]));
  mx = block_max(mx, sh);
  const float ref = mx == -INFINITY ? 0.f : mx;
  float s = 0.f;
  for (int i = threadIdx.x; i < width; i += blockDim.x) s += expf(cap(r[i]) - ref);
  s = block_sum(s, sh);
  if (threadIdx.x == 0) {
    float m = mx;
    if (!first) {
      const float2 o = stats[row];
      const float t = fmaxf(m, o.x);
      if (t == -INFINITY) { s += o.y; }
      else { s = s * expf(m - t) + o.y * expf(o.x - t); m = t; }
    }
    stats[row] = make_float2(m, s);
    const int y = targets[row] - col0;
    if (targets[row] >= 0 && y >= 0 && y < width) ztgt[row] = cap(r[y]);
  }
}

// z -> dz in place
__global__ void __launch_bounds__(256) ce_piece_grad_kernel(float* __restrict__ z, int width, int col0, float softcap,
                                                            const int32_t* __restrict__ targets,
                                                            const float* __restrict__ lse,
                                                            const float* __restrict__ row_scale) {
  pdl_wait();
  const long long row = blockIdx.x;
  float* r = z + row * width;
  const float l = lse[row], g = row_scale[row];
  const int y = targets[row] - col0;
  for (int i = threadIdx.x; i < width; i += blockDim.x) {
    float v = r[i], slope = 1.f;
    if (softcap > 0.f) { const float t = tanhf(v / softcap); v = softcap * t; slope = 1.f - t * t; }
    r[i] = g != 0.f ? (expf(v - l) - (i == y ? 1.f : 0.f)) * slope * g : 0.f;
  }
}

// fp32 sum over the pieces -> dx (row pitch ld elements)
__global__ void __launch_bounds__(256) ce_dx_kernel(const float* __restrict__ acc, int N, int d, bf16* __restrict__ dx,
                                                    long long ld) {
  pdl_wait();
  const int c4 = d / 4;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < (long long)N * c4;
       i += (long long)gridDim.x * blockDim.x) {
    float v[4];
    load4(acc + i * 4, v);
    store4(dx + (i / c4) * ld + (i % c4) * 4, v);
  }
}
