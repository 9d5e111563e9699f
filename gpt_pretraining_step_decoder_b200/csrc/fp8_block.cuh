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
// One block per 128 x 128 tile, 256 threads; each thread holds 8 rows x 8
// columns of it in registers, from which both orientations are coded: x is read
// once.  The transposed codes pass through shared memory (8-byte slots, XORed
// so that neither the column-wise writes nor the row-wise reads conflict).
// Memory bounds it: 2 or 4 bytes read and 1 or 2 written per element.
#pragma once
#include <cuda_fp8.h>
#include "common.cuh"

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
  int square, vec;                            // vec: 16-byte loads are aligned
};

template <typename T>
__global__ void __launch_bounds__(256) fp8_block_quantize_kernel(const T* __restrict__ x, const QuantArgs a) {
  pdl_wait();
  __shared__ uint32_t colmax[8][128];
  __shared__ uint32_t blockmax[8];
  __shared__ __align__(16) uint2 tr[128 * 16];  // transposed codes: [column][8-row slot]
  const int cblocks = (int)((a.cols + 127) >> 7);
  const long long rb = blockIdx.x / cblocks;
  const int cb = (int)(blockIdx.x % cblocks);
  const long long row0 = rb * 128, col0 = (long long)cb * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  const int r0 = warp * 16 + half * 8;  // this thread's 8 rows and 8 columns of the tile
  const int c0 = l * 8;
  const bool full = row0 + 128 <= a.rows && col0 + 128 <= a.cols && a.vec;

  float v[8][8];
  if (full) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const T* p = x + (row0 + r0 + i) * a.ldx + col0 + c0;
      load4(p, *reinterpret_cast<float(*)[4]>(&v[i][0]));
      load4(p + 4, *reinterpret_cast<float(*)[4]>(&v[i][4]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const long long r = row0 + r0 + i, c = col0 + c0 + j;
        v[i][j] = r < a.rows && c < a.cols ? to_f(x[r * a.ldx + c]) : 0.f;
      }
  }
  // largest magnitudes, as bit patterns (they order like the values; infinities
  // and NaN come out on top)
  uint32_t rmax[8], cmax[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { rmax[i] = 0u; cmax[i] = 0u; }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = __float_as_uint(v[i][j]) & 0x7fffffffu;
      rmax[i] = max(rmax[i], b);
      cmax[j] = max(cmax[j], b);
    }
  if (a.square) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, rmax[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) blockmax[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, blockmax[w]);
#pragma unroll
    for (int i = 0; i < 8; ++i) { rmax[i] = m; cmax[i] = m; }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) rmax[i] = max(rmax[i], __shfl_xor_sync(0xffffffffu, rmax[i], o));
    if (a.qt) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t m = max(cmax[j], __shfl_xor_sync(0xffffffffu, cmax[j], 16));
        if (half == 0) colmax[warp][c0 + j] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0u;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max(m, colmax[w][c0 + j]);
        cmax[j] = m;
      }
    }
  }
  if (a.q) {
    const long long row_atoms = (a.rows + 127) >> 7;
    const int last = cb == cblocks - 1 ? (4 - (cblocks & 3)) & 3 : 0;  // groups that fill the last atom
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long long r = row0 + r0 + i;
      const uint32_t sb = scale_byte(rmax[i]);
      if (l == 0) {
        uint8_t* s = a.sc + scale_offset(r, cb, row_atoms);
        *s = r < a.rows ? (uint8_t)sb : 127;
        for (int k = 1; k <= last; ++k) s[k] = 127;
      }
      const float inv = scale_inv(sb);
      uint2 o;
      o.x = e4m3x2(v[i][0] * inv, v[i][1] * inv) | (e4m3x2(v[i][2] * inv, v[i][3] * inv) << 16);
      o.y = e4m3x2(v[i][4] * inv, v[i][5] * inv) | (e4m3x2(v[i][6] * inv, v[i][7] * inv) << 16);
      if (r >= a.rows) continue;
      uint8_t* d = a.q + r * a.ldq + col0 + c0;
      if (col0 + c0 + 8 <= a.cols) {
        *reinterpret_cast<uint2*>(d) = o;
      } else {
        for (int j = 0; j < 8; ++j)
          if (col0 + c0 + j < a.cols) d[j] = (uint8_t)((j < 4 ? o.x : o.y) >> (8 * (j & 3)));
      }
    }
  }
  if (a.qt) {
    const long long col_atoms = (a.cols + 127) >> 7, rblocks = (a.rows + 127) >> 7;
    const int last = rb == rblocks - 1 ? (int)((4 - (rblocks & 3)) & 3) : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t sb = scale_byte(cmax[j]);
      const long long c = col0 + c0 + j;
      if (warp == 0 && half == 0) {
        uint8_t* s = a.sct + scale_offset(c, rb, col_atoms);
        *s = c < a.cols ? (uint8_t)sb : 127;
        for (int k = 1; k <= last; ++k) s[k] = 127;
      }
      const float inv = scale_inv(sb);
      uint2 o;
      o.x = e4m3x2(v[0][j] * inv, v[1][j] * inv) | (e4m3x2(v[2][j] * inv, v[3][j] * inv) << 16);
      o.y = e4m3x2(v[4][j] * inv, v[5][j] * inv) | (e4m3x2(v[6][j] * inv, v[7][j] * inv) << 16);
      tr[(c0 + j) * 16 + ((r0 >> 3) ^ l)] = o;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = k * 16 + (threadIdx.x >> 4), slot = threadIdx.x & 15;
      const uint2 o = tr[c * 16 + (slot ^ (c >> 3))];
      if (col0 + c >= a.cols) continue;
      const long long r = row0 + slot * 8;
      uint8_t* d = a.qt + (col0 + c) * a.ldqt + r;
      if (r + 8 <= a.rows) {
        *reinterpret_cast<uint2*>(d) = o;
      } else {
        for (int j = 0; j < 8; ++j)
          if (r + j < a.rows) d[j] = (uint8_t)((j < 4 ? o.x : o.y) >> (8 * (j & 3)));
      }
    }
  }
}
