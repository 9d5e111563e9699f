// fp8_block.cuh -- e4m3 quantization with one power-of-two scale for each
// group of 128 elements, of a matrix and of its transpose in one pass.
//
// scale = the least 2^e with amax <= 448 * 2^e over the group (1 x 128 of a
// row, or a 128 x 128 block), code = e4m3(x / scale) to nearest even.  With a
// power of two the division is exact, so a code depends on x and e alone, and
// the scale is one exponent byte (e + 127), the form in which the tensor cores
// take scales (tcgen05.mma block_scale), so the product needs no pass over its
// accumulators for them.
//
// Scale storage, "atoms" of 512 bytes for 128 rows x 4 groups (512 elements of
// K): scale of row r, group b at ((b / 4) * ceil(rows / 128) + r / 128) * 512
// + 16 (r % 32) + 4 (r % 128 / 32) + b % 4.  That is the order in which
// tcgen05.cp spreads an atom over tensor memory: lane r % 32, column
// r % 128 / 32, byte b % 4.
//
// Persistent blocks of 512 threads take a 128 x 128 tile at a time; each thread
// holds 4 rows x 8 columns of it in registers, from which both orientations are
// coded: x is read once.  A tile arrives by TMA (zeros beyond the matrix) while
// the one before it is coded; rows that are not 16-byte aligned take plain loads.
// The transposed codes pass through shared memory (4-byte slots, XORed so that
// neither the column-wise writes nor the row-wise reads conflict).  Memory bounds
// it: 2 or 4 bytes read and 1 or 2 written per element.  B200, both orientations:
// 32768 x 768 bf16 in row groups 20.9 us (101 MB, 4.8 TB/s; a 50 MB copy_ takes
// 20.4), 8192 x 2048 fp32 in blocks 19.4 us (101 MB, 5.2 TB/s).  256 threads of 8 x 8
// elements, tiles by plain loads: 41.8 and 27.9.
#pragma once
#include <cuda_fp8.h>
#include "gemm_tc.cuh"

// exponent byte of a group from the bits of its largest magnitude: 448 = 1.75 *
// 2^8, so amax = m 2^k needs 2^(k-8), one more where m > 1.75 (the carry).  0
// gives a scale of one, an infinity or a NaN the NaN scale 255.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits == 0u) return 127u;
  if (amax_bits >= 0x7f800000u) return 255u;
  const int e = (int)((amax_bits + 0x1fffffu) >> 23) - 8;
  return e < 0 ? 0u : (uint32_t)e;
}
// 1 / scale as fp32 (exact); the NaN scale gives NaN, hence NaN codes
__device__ __forceinline__ float scale_inv(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__host__ __device__ __forceinline__ long long scale_offset(long long r, long long b, long long row_atoms) {
  return ((b >> 2) * row_atoms + (r >> 7)) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (b & 3);
}

struct QuantArgs {
  long long rows, cols, ldx;
  uint8_t* q; long long ldq; uint8_t* sc;     // codes and scales of x; q null: not written
  uint8_t* qt; long long ldqt; uint8_t* sct;  // those of its transpose; qt null: not written
  int square;
  int tiles;
  unsigned* err;
};

// |a|, |b| joined to m; a NaN stays
__device__ __forceinline__ float absmax3(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  load4(p, *reinterpret_cast<float(*)[4]>(&v[0]));
  load4(p + 4, *reinterpret_cast<float(*)[4]>(&v[4]));
}
__device__ __forceinline__ void load8(const bf16* p, float (&v)[8]) {
  const uint4 t = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}

// (y0, y1) = (x0, x1) * (c0, c1), one instruction
__device__ __forceinline__ void mul2(float& y0, float& y1, float x0, float x1, float c0, float c1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(y0), "=f"(y1)
      : "f"(x0), "f"(x1), "f"(c0), "f"(c1));
}

constexpr int QUANT_THREADS = 512;

struct QuantShared {
  float colmax[16][128];    // per warp
  float rowmax[128];
  float colinv[128], rowinv[128];
  uint32_t tr[128 * 32];    // transposed codes: [column][4-row slot]
  uint64_t full;            // the tile in flight has landed
  int abort;
};

// FULL: no bounds to check; TMA: x's tile lies in `buf`, and `next` starts the
// copy of the tile after it once every thread has read its part.
template <bool FULL, bool TMA, typename T, typename Next>
__device__ __forceinline__ void quantize_tile(const T* __restrict__ x, const QuantArgs& a, long long rb, int cb,
                                              int cblocks, QuantShared& sh, const T* buf, Next next) {
  const long long row0 = rb * 128, col0 = (long long)cb * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int slot = warp * 2 + half, r0 = slot * 4;  // this thread's 4 rows and 8 columns of the tile
  const int c0 = l * 8;

  float v[4][8];
  if (TMA) {
#pragma unroll
    for (int i = 0; i < 4; ++i) load8(buf + (r0 + i) * 128 + c0, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const long long r = row0 + r0 + i, c = col0 + c0 + j;
        v[i][j] = r < a.rows && c < a.cols ? to_f(x[r * a.ldx + c]) : 0.f;
      }
  }
  // largest magnitudes (an infinity comes out on top, a NaN as NaN)
  float rmax[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    rmax[i] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) rmax[i] = absmax3(rmax[i], v[i][j], v[i][j + 1]);
  }
  {
    // over the 16 lanes of a row, the lanes sharing out the 4 rows: lane l ends
    // with row 2 (l / 8) + l / 4 % 2
    const float x0 = max_nan(l & 8 ? rmax[2] : rmax[0], __shfl_xor_sync(0xffffffffu, l & 8 ? rmax[0] : rmax[2], 8));
    const float x1 = max_nan(l & 8 ? rmax[3] : rmax[1], __shfl_xor_sync(0xffffffffu, l & 8 ? rmax[1] : rmax[3], 8));
    float m = max_nan(l & 4 ? x1 : x0, __shfl_xor_sync(0xffffffffu, l & 4 ? x0 : x1, 4));
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if ((l & 3) == 0) sh.rowmax[r0 + (l >> 3) * 2 + ((l >> 2) & 1)] = m;
  }
  if (!a.square && a.qt) {
    float cm[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cm[j] = absmax3(absmax3(0.f, v[0][j], v[1][j]), v[2][j], v[3][j]);
    // the two halves of the warp (other rows, same columns) share out the columns
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = max_nan(half ? cm[4 + j] : cm[j], __shfl_xor_sync(0xffffffffu, half ? cm[j] : cm[4 + j], 16));
    store4(&sh.colmax[warp][c0 + 4 * half], o);
  }
  __syncthreads();
  next();
  // a thread per row and per column: scale byte, its place, its inverse
  const int t = threadIdx.x & 127, which = threadIdx.x >> 7;
  if (which < 2) {
    float m;
    if (a.square) {
      // magnitudes order like their bit patterns, NaN above all
      m = max_nan(max_nan(sh.rowmax[lane], sh.rowmax[lane + 32]), max_nan(sh.rowmax[lane + 64], sh.rowmax[lane + 96]));
      m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    } else if (which == 0) {
      m = sh.rowmax[t];
    } else {
      m = 0.f;
      if (a.qt) {
#pragma unroll
        for (int w = 0; w < 16; ++w) m = max_nan(m, sh.colmax[w][t]);
      }
    }
    const uint32_t sb = scale_byte(__float_as_uint(m));
    (which == 0 ? sh.rowinv : sh.colinv)[t] = scale_inv(sb);
    // row r of x is row r of q, group cb; column c is row c of qt, group rb
    uint8_t* s = which == 0 ? a.sc : a.sct;
    if (which == 0 ? a.q != nullptr : a.qt != nullptr) {
      const long long r = (which == 0 ? row0 : col0) + t, rows = which == 0 ? a.rows : a.cols;
      const long long grp = which == 0 ? cb : rb, groups = which == 0 ? cblocks : (a.rows + 127) >> 7;
      s += scale_offset(r, grp, (rows + 127) >> 7);
      *s = r < rows ? (uint8_t)sb : 127;
      if (grp == groups - 1)  // the groups that fill the last atom
        for (int k = 1; k <= (int)((4 - (groups & 3)) & 3); ++k) s[k] = 127;
    }
  }
  __syncthreads();
  if (a.q) {
    float inv[4];
    load4(&sh.rowinv[r0], inv);
    uint8_t* d = a.q + (row0 + r0) * a.ldq + col0 + c0;
#pragma unroll
    for (int i = 0; i < 4; ++i, d += a.ldq) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; j += 2) mul2(y[j], y[j + 1], v[i][j], v[i][j + 1], inv[i], inv[i]);
      uint2 o;
      o.x = e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16);
      o.y = e4m3x2(y[4], y[5]) | (e4m3x2(y[6], y[7]) << 16);
      if (!FULL && row0 + r0 + i >= a.rows) continue;
      if (FULL || col0 + c0 + 8 <= a.cols) {
        *reinterpret_cast<uint2*>(d) = o;
      } else {
        for (int j = 0; j < 8; ++j)
          if (col0 + c0 + j < a.cols) d[j] = (uint8_t)((j < 4 ? o.x : o.y) >> (8 * (j & 3)));
      }
    }
  }
  if (a.qt) {
    float inv[8];
    load4(&sh.colinv[c0], *reinterpret_cast<float(*)[4]>(&inv[0]));
    load4(&sh.colinv[c0 + 4], *reinterpret_cast<float(*)[4]>(&inv[4]));
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 2) mul2(v[i][j], v[i][j + 1], v[i][j], v[i][j + 1], inv[j], inv[j + 1]);
    uint32_t* trow = sh.tr + c0 * 32 + (slot ^ (2 * l));
#pragma unroll
    for (int j = 0; j < 8; ++j) trow[j * 32] = e4m3x2(v[0][j], v[1][j]) | (e4m3x2(v[2][j], v[3][j]) << 16);
    __syncthreads();
    uint8_t* d = a.qt + (col0 + slot) * a.ldqt + row0 + l * 8;
#pragma unroll
    for (int k = 0; k < 4; ++k, d += 32 * a.ldqt) {
      const int c = k * 32 + slot;
      const uint2 o = *reinterpret_cast<const uint2*>(&sh.tr[c * 32 + ((2 * l) ^ (2 * (c >> 3)))]);
      if (!FULL && col0 + c >= a.cols) continue;
      const long long r = row0 + l * 8;
      if (FULL || r + 8 <= a.rows) {
        *reinterpret_cast<uint2*>(d) = o;
      } else {
        for (int j = 0; j < 8; ++j)
          if (r + j < a.rows) d[j] = (uint8_t)((j < 4 ? o.x : o.y) >> (8 * (j & 3)));
      }
    }
  }
}

constexpr int QUANT_BLOCKS = 2;  // resident per SM
// x's tile, then QuantShared
template <typename T> constexpr int quant_smem() { return 128 * 128 * (int)sizeof(T) + (int)sizeof(QuantShared); }

template <typename T, bool TMA>
__global__ void __launch_bounds__(QUANT_THREADS, QUANT_BLOCKS)
    fp8_block_quantize_kernel(const __grid_constant__ CUtensorMap map, const T* __restrict__ x, const QuantArgs a) {
  pdl_wait();
  extern __shared__ __align__(128) uint8_t quant_smem_raw[];
  T* buf = reinterpret_cast<T*>(quant_smem_raw);
  QuantShared& sh = *reinterpret_cast<QuantShared*>(quant_smem_raw + 128 * 128 * sizeof(T));
  const int cblocks = (int)((a.cols + 127) >> 7);
  auto fetch = [&](int tile) {
    if (!TMA || threadIdx.x != 0 || tile >= a.tiles) return;
    tc::mbar_expect_tx(&sh.full, 128 * 128 * sizeof(T));
    tc::tma_load_2d(buf, &map, &sh.full, tile % cblocks * 128, tile / cblocks * 128);
  };
  if (TMA) {
    if (threadIdx.x == 0) {
      tc::mbar_init(&sh.full, 1);
      sh.abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
  }
  fetch(blockIdx.x);
  uint32_t phase = 0;
  for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const long long rb = tile / cblocks;
    const int cb = tile % cblocks;
    auto next = [&] { fetch(tile + (int)gridDim.x); };
    // a copy that never lands: reported, the codes are void, later waits return at once
    if (TMA) tc::mbar_wait(&sh.full, phase, &sh.abort, a.err);
    phase ^= 1;
    if (rb * 128 + 128 <= a.rows && (long long)cb * 128 + 128 <= a.cols)
      quantize_tile<true, TMA>(x, a, rb, cb, cblocks, sh, buf, next);
    else
      quantize_tile<false, TMA>(x, a, rb, cb, cblocks, sh, buf, next);
    __syncthreads();  // the shared tables are free for the next tile
  }
}
