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
// on it; dx is summed over the pieces in fp32.  dz is rounded to bf16 without the
// mean's factor dloss / count, which the products apply in fp32: where few rows have a target in
// common, dz = -(1 - p) with p near 0 is then exact instead of off by the same
// half step in every row.  Three products of 2 N V d
// operations bound it.  B200, in a stream of calls: 32768 x 50304 x 768 forward
// 1868 us (1355 TFLOP/s), 16384 x 65536 x 2048 backward with soft-cap 10.7 ms (1233
// TFLOP/s, under the power cap; 9.2 ms in a short run), 33 x 50304 x 768 forward 23.6 us
// (17.6 of them the one read of W, 4.4 TB/s).  fp32: the same pieces through plain FFMA products, with
// fp32 logits of one piece at a time in the workspace.
#pragma once
#include "gemm_tc.cuh"

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

// Block of 32 rows x G groups of pairs (a warp per group); stats [n_pairs, N],
// so that a warp reads 32 neighbouring rows; G neighbouring lanes then join the
// groups of one row.  Leaves each row's lse and loss and the block's loss sum
// (fp64) and count; the block that finishes last (`counter`, zeroed by the kernel
// before) adds those in block order and writes the mean.  G = 32 for few rows
// (latency: all pairs in flight at once), 8 for many (more blocks per SM hide
// it: 32768 rows of 100 pairs took 41 us with G = 32).
template <int G>
__global__ void __launch_bounds__(32 * G) ce_combine_kernel(const float2* __restrict__ stats, int n_tiles, int N, int V,
                                                            const int32_t* __restrict__ targets,
                                                            const float* __restrict__ ztgt, float* __restrict__ lse_out,
                                                            float* __restrict__ tok_loss, double2* __restrict__ part,
                                                            unsigned* __restrict__ counter, float* __restrict__ loss,
                                                            unsigned* err) {
  pdl_wait();
  __shared__ float2 sh[G][33];
  __shared__ double sums[2][32];
  __shared__ int last;
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int r = blockIdx.x * 32 + lane;
  const int br = threadIdx.x / G, row = blockIdx.x * 32 + br, g = threadIdx.x % G;  // the row that is joined below
  int y = -1;
  float zt = 0.f;
  if (g == 0 && row < N) {
    y = targets[row];
    zt = ztgt[row];  // written only where the target is one
  }
  float m = -INFINITY, s = 0.f;
  if (r < N) {
    constexpr int U = 16;  // pairs in flight per thread, joined at once
    for (int j = grp; j < n_tiles; j += G * U) {
      float2 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = j + G * u < n_tiles ? __ldcg(stats + (long long)(j + G * u) * N + r) : make_float2(-INFINITY, 0.f);
      float mx = m;
#pragma unroll
      for (int u = 0; u < U; ++u) mx = fmaxf(mx, v[u].x);
      const float ref = mx == -INFINITY ? 0.f : mx;  // nothing but empty parts: their sums are 0 (or NaN, which stays)
      s *= __expf(m - ref);
#pragma unroll
      for (int u = 0; u < U; ++u) s += v[u].y * __expf(v[u].x - ref);
      m = mx;
    }
  }
  sh[grp][lane] = make_float2(m, s);
  __syncthreads();
  m = sh[g][br].x;
  s = sh[g][br].y;
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1)
    lse_join(m, s, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o));
  if (g == 0) {
    int valid = 0;
    float t = 0.f;
    if (row < N) {
      const float lse = m + logf(s);
      t = ce_row_loss(lse, zt, y, V, valid, err);
      if (lse_out) lse_out[row] = lse;
      if (tok_loss) tok_loss[row] = t;
    }
    sums[0][br] = t;
    sums[1][br] = valid;
  }
  __syncthreads();
  if (grp == 0) {
    const double l = warp_sum_d(sums[0][lane]), c = warp_sum_d(sums[1][lane]);
    if (lane == 0) {
      part[blockIdx.x] = make_double2(l, c);
      __threadfence();
      last = atomicAdd(counter, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double l = 0.0, c = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += blockDim.x) {
    const double2 p = __ldcg(part + i);
    l += p.x;
    c += p.y;
  }
  l = warp_sum_d(l);
  c = warp_sum_d(c);
  if (lane == 0) { sums[0][grp] = l; sums[1][grp] = c; }
  __syncthreads();
  if (threadIdx.x == 0) {
    l = c = 0.0;
    for (int w = 0; w < G; ++w) { l += sums[0][w]; c += sums[1][w]; }
    const float mean = c > 0.0 ? (float)(l / c) : 0.f;
    if (!isfinite(mean)) set_error(err, GPT_EBIT_NONFINITE);
    if (loss) *loss = mean;
  }
}

// fp32: gradient scale of a row: dtok[i], or base = dloss / count (dloss null: 1),
// 0 for ignored rows.  With few rows every block counts the targets itself (they are
// in L2), so that no launch has to come first; for more ce_base_kernel counts them once.
struct CeRowScale {
  const int32_t* targets;
  const float* dloss;
  const float* dtok;
  int N, V;
  unsigned* err;
};
__device__ __forceinline__ float ce_scale_base(const CeRowScale& a) {
  if (a.dtok) return 0.f;
  __shared__ int sh[32];
  int c = __reduce_add_sync(0xffffffffu, count_targets(a.targets, a.N, a.V, threadIdx.x, blockDim.x));
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = c;
  __syncthreads();
  c = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) c += sh[w];
  return c > 0 ? (a.dloss ? *a.dloss : 1.f) / (float)c : 0.f;
}
__device__ __forceinline__ float ce_row_scale(const CeRowScale& a, float base, int i) {
  const int y = a.targets[i];
  if (y < -1 || y >= a.V) set_error(a.err, GPT_EBIT_INPUT);
  return y >= 0 && y < a.V ? (a.dtok ? a.dtok[i] : base) : 0.f;
}
// base alone, for more rows than the first product counts on the side
__global__ void __launch_bounds__(1024) ce_base_kernel(const CeRowScale a, float* __restrict__ base) {
  pdl_wait();
  const float b = ce_scale_base(a);
  if (threadIdx.x == 0) *base = b;
}

// ---------------------------------------------------------------- fp32 pieces
// One block per row of a piece of fp32 logits z [N, width] (columns col0 ...):
// joins the piece's max and sum of exp to the row's, picks the target's logit.
// first: the row's pair starts here.
__global__ void __launch_bounds__(256) ce_piece_stats_kernel(const float* __restrict__ z, int width, int col0, int first,
                                                             float softcap, const int32_t* __restrict__ targets, int N,
                                                             float2* __restrict__ stats, float* __restrict__ ztgt,
                                                             unsigned* __restrict__ counter) {
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0u;
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

// fp32 products of the pieces (FFMA): C[m, n] = sum_k A[m, k] B[n, k].  32 x 32
// tiles, so that the small decoders' products still make enough blocks; the 8
// warps of a block take every eighth chunk of 16 k's each, through shared memory
// of their own (no block barrier in the loop, the next chunk's loads in flight
// meanwhile), 4 x 8 results per thread in packed pairs, and the partial tiles are
// added in warp order.  Fewer tiles than SMs and a long K: K is also shared out
// over blocks, whose tiles the last one to finish adds in share order.  A chunk
// lies as [k][row ^ 8 (k / 4)], so that neither the writes of an operand that is
// contiguous along k nor the reads conflict.  A small call is latency (256 x 512 x 128,
// both launches: 12.2 us), a large one the shared-memory reads of 4 x 8 results (4096
// x 8192 x 1024: 6.3 ms, 33 TFLOP/s; 64 x 64 tiles with a chunk staged once for four
// warps 5.7, but a third slower at 400 x 3000 x 200).
struct CeProduct {
  const float* A; long long lda; int a_kmajor;
  const float* B; long long ldb; int b_kmajor;
  float* C; long long ldc;
  int M, N, K, beta, tiles;  // tiles = number of 32 x 32 tiles; 0: no product
  int splits;                // shares of K
  float* part;               // splits > 1: [tiles * splits][32 x 32]
  unsigned* counter;         // splits > 1: finished shares per tile, zero at the start
};
// gradient epilogue (dz instead of z); lse null: none
struct CeGrad {
  const float* lse;
  CeRowScale scale;
  const float* base;  // counted before (null: by every block)
  int col0;
  float softcap;
  unsigned* zero;  // CEP_TILES counters to zero for the next launch (null: none)
};
constexpr int CEP_KC = 16, CEP_WARPS = 8;
constexpr int CEP_TILES = 296;  // two blocks per SM: about as many as a split product makes
constexpr int CEP_SLOTS = 2 * CEP_TILES;  // partial tiles

// One lane's part of a 32 x 16 chunk (zeros beyond the operand): four times four
// neighbours along the contiguous dimension.
__device__ __forceinline__ void ce_load_chunk(float (&v)[4][4], const float* __restrict__ p, long long ld, int kmajor,
                                              bool vec, int r0, int rows, int k0, int k1) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + (kmajor ? (lane >> 2) + 8 * i : (lane & 7) * 4), k = k0 + (kmajor ? (lane & 3) * 4 : (lane >> 3) + 4 * i);
    const float* q = kmajor ? p + r * ld + k : p + k * ld + r;
    if (vec && (kmajor ? r < rows && k + 4 <= k1 : k < k1 && r + 4 <= rows)) {
      load4(q, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = (kmajor ? r < rows && k + j < k1 : k < k1 && r + j < rows) ? q[j] : 0.f;
    }
  }
}
__device__ __forceinline__ void ce_store_chunk(float (*s)[32], const float (&v)[4][4], int kmajor) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kmajor) {
      const int kq = lane & 3, r = ((lane >> 2) + 8 * i) ^ (8 * kq);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[4 * kq + j][r] = v[i][j];
    } else {
      store4(&s[(lane >> 3) + 4 * i][((lane & 7) * 4) ^ (8 * i)], v[i]);
    }
  }
}

// one or two products in one launch (dx and dW of a piece)
__global__ void __launch_bounds__(CEP_WARPS * 32, 2) ce_product_kernel(const CeProduct p0, const CeProduct p1,
                                                                       const CeGrad gr) {
  pdl_wait();
  // per warp: its chunks of A and B; then its partial tile
  __shared__ __align__(16) float sh[CEP_WARPS][2][CEP_KC][32];
  __shared__ int last;
  const int blocks0 = p0.tiles * p0.splits;
  const bool second = (int)blockIdx.x >= blocks0;
  const CeProduct& p = second ? p1 : p0;
  const int item = blockIdx.x - (second ? blocks0 : 0), tile = item / p.splits, nt = (p.N + 31) >> 5;
  const int m0 = tile / nt * 32, n0 = tile % nt * 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tm = (lane >> 2) * 4, tn = (lane & 3) * 8;  // this thread's 4 x 8 results
  float (*as)[32] = sh[warp][0];
  float (*bs)[32] = sh[warp][1];
  constexpr int STEP = CEP_WARPS * CEP_KC;
  const int share = ((p.K + p.splits * CEP_KC - 1) / (p.splits * CEP_KC)) * CEP_KC;
  const int kb = item % p.splits * share, k1 = min(p.K, kb + share);
  const bool veca = ((p.lda & 3) | (reinterpret_cast<uintptr_t>(p.A) & 15)) == 0;
  const bool vecb = ((p.ldb & 3) | (reinterpret_cast<uintptr_t>(p.B) & 15)) == 0;
  float acc[4][8] = {};
  float va[4][4], vb[4][4];
  int k0 = kb + warp * CEP_KC;
  const bool grad = gr.lse != nullptr && !second;
  if (k0 < k1) {
    ce_load_chunk(va, p.A, p.lda, p.a_kmajor, veca, m0, p.M, k0, k1);
    ce_load_chunk(vb, p.B, p.ldb, p.b_kmajor, vecb, n0, p.N, k0, k1);
  }
  if (gr.zero && blockIdx.x == 0)
    for (int i = threadIdx.x; i < CEP_TILES; i += CEP_WARPS * 32) gr.zero[i] = 0u;
  // while the first chunk is on its way
  const float base = !grad ? 0.f : gr.base ? *gr.base : ce_scale_base(gr.scale);
  for (; k0 < k1; k0 += STEP) {
    __syncwarp();
    ce_store_chunk(as, va, p.a_kmajor);
    ce_store_chunk(bs, vb, p.b_kmajor);
    __syncwarp();
    if (k0 + STEP < k1) {
      ce_load_chunk(va, p.A, p.lda, p.a_kmajor, veca, m0, p.M, k0 + STEP, k1);
      ce_load_chunk(vb, p.B, p.ldb, p.b_kmajor, vecb, n0, p.N, k0 + STEP, k1);
    }
#pragma unroll 4
    for (int k = 0; k < CEP_KC; ++k) {
      const int x = (k >> 2) * 8;
      float a[4], b[8];
      load4(&as[k][tm ^ x], a);
      load4(&bs[k][tn ^ x], *reinterpret_cast<float(*)[4]>(&b[0]));
      load4(&bs[k][(tn + 4) ^ x], *reinterpret_cast<float(*)[4]>(&b[4]));
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          tc::fma2v(acc[i][j], acc[i][j + 1], b[j], b[j + 1], a[i], acc[i][j], acc[i][j + 1]);
    }
  }
  __syncwarp();
  float* mine = &sh[warp][0][0][0] + tm * 32 + tn;  // partial tile [32][32]
#pragma unroll
  for (int i = 0; i < 4; ++i) { store4(mine + i * 32, &acc[i][0]); store4(mine + i * 32 + 4, &acc[i][4]); }
  __syncthreads();
  // four results per thread: row threadIdx / 8, four columns
  const int m = m0 + (threadIdx.x >> 3), nc = (threadIdx.x & 7) * 4;
  float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < CEP_WARPS; ++w) {
    float v[4];
    load4(&sh[w][0][0][0] + threadIdx.x * 4, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] += v[j];
  }
  if (p.splits > 1) {
    float4* part = reinterpret_cast<float4*>(p.part) + (long long)tile * p.splits * 256 + threadIdx.x;
    part[item % p.splits * 256] = make_float4(r[0], r[1], r[2], r[3]);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(p.counter + tile, 1u) == (unsigned)p.splits - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    r[0] = r[1] = r[2] = r[3] = 0.f;
    for (int s = 0; s < p.splits; ++s) {
      const float4 v = __ldcg(part + s * 256);
      r[0] += v.x; r[1] += v.y; r[2] += v.z; r[3] += v.w;
    }
  }
  if (m >= p.M) return;
  const float l = grad ? gr.lse[m] : 0.f, g = grad ? ce_row_scale(gr.scale, base, m) : 0.f;
  const int y = grad ? gr.scale.targets[m] - gr.col0 : -1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = n0 + nc + j;
    if (n >= p.N) continue;
    float v = r[j];
    if (grad) {  // (exp(z - lse) - [target]) * slope * scale; a row without a gradient stays out
      float slope = 1.f;
      if (gr.softcap > 0.f) { const float t = tanhf(v / gr.softcap); v = gr.softcap * t; slope = 1.f - t * t; }
      v = g != 0.f ? (expf(v - l) - (n == y ? 1.f : 0.f)) * slope * g : 0.f;
    }
    float* c = p.C + m * p.ldc + n;
    *c = (p.beta ? *c : 0.f) + v;
  }
}

// fp32 sum over the pieces, times *base (null: 1) -> dx (row pitch ld elements)
__global__ void __launch_bounds__(256) ce_dx_kernel(const float* __restrict__ acc, int N, int d,
                                                    const float* __restrict__ base, bf16* __restrict__ dx, long long ld) {
  pdl_wait();
  const float b = base ? *base : 1.f;
  const int c4 = d / 4;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < (long long)N * c4;
       i += (long long)gridDim.x * blockDim.x) {
    float v[4];
    load4(acc + i * 4, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] *= b;
    store4(dx + (i / c4) * ld + (i % c4) * 4, v);
  }
}
