// quant_f8.cuh -- 8-bit floating point (E4M3) operands with a scale per block
// of 128, as the FP8 products read them.
//
// Activations [R, K]: one scale per row and 128 features, the least power of
// two s with amax <= 448 s (s = 1 for a block of zeros, at least 2^-126).
// Dividing by a power of two is exact, so the only rounding is that of x / s
// to E4M3 (nearest even), and codes do not depend on how the quotient is
// computed.  A value that is not finite becomes the NaN code and does not
// count in amax.  Weights [n, rows, cols]: the same rule over 128 x 128 blocks.
//
// Bound by memory: 2 or 4 bytes read and 1 written per value (16384 x 2688 bf16 in
// 21.5 us, 6.2 TB/s; 16384 x 1856 float32 in 23.6 us, 6.5 TB/s).  Eight lanes
// hold a block (16 values each), so its maximum is three shuffles away and each
// lane stores 16 bytes; blocks of all rows are numbered through, which keeps
// every lane busy at any K.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace nh {
namespace f8 {

constexpr int BLK = 128;

// exponent of the block's scale from the bits of its largest magnitude (finite):
// 448 = 1.75 * 2^8
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
  if (amax_bits == 0) return 0;
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -126);
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
constexpr uint32_t INF_BITS = 0x7f800000u;

// Two values times a power of two as a pair of codes (low byte first).  Scaled
// finite values never pass 448, so only Inf and NaN give the NaN code.
// (The conversion saturates: an Inf has to be made a NaN first.)
__device__ __forceinline__ uint32_t encode2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// v times a power of two; Inf becomes NaN (Inf * 0)
__device__ __forceinline__ float scaled(float v, float inv) { return fmaf(v, inv, v * 0.0f); }

// relu(v) that keeps a NaN, and its square
__device__ __forceinline__ float relu_nan(float v) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float relu2_nan(float v) {
  const float r = relu_nan(v);
  return r * r;
}

// 16 values of a row as they lie in global memory
struct Bf16x16 {
  uint32_t w[8];
};
struct F32x16 {
  float v[16];
};
__device__ __forceinline__ void load16(const __nv_bfloat16* p, bool in, Bf16x16& r) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 u = in ? q[h] : make_uint4(0, 0, 0, 0);
    r.w[4 * h] = u.x;
    r.w[4 * h + 1] = u.y;
    r.w[4 * h + 2] = u.z;
    r.w[4 * h + 3] = u.w;
  }
}
__device__ __forceinline__ void load16(const float* p, bool in, F32x16& r) {
  const float4* q = reinterpret_cast<const float4*>(p);
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const float4 f = in ? q[h] : make_float4(0.f, 0.f, 0.f, 0.f);
    r.v[4 * h] = f.x;
    r.v[4 * h + 1] = f.y;
    r.v[4 * h + 2] = f.z;
    r.v[4 * h + 3] = f.w;
  }
}
__device__ __forceinline__ float value(const Bf16x16& r, int i) {
  return __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
}
__device__ __forceinline__ float value(const F32x16& r, int i) { return r.v[i]; }
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> { using type = Bf16x16; };
template <> struct Raw<float> { using type = F32x16; };

// Bits of the largest magnitude of 16 values, as integers (two bf16 at a time);
// Inf and NaN come out on top, and only where there are any they are left out one
// by one.
__device__ __forceinline__ uint32_t amax_any(const Bf16x16& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, r.w[i] & 0x7fff7fffu);
  return max(m & 0xffff0000u, m << 16);
}
__device__ __forceinline__ uint32_t amax_any(const F32x16& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; i += 2) m = __vimax3_u32(m, mag_bits(r.v[i]), mag_bits(r.v[i + 1]));
  return m;
}
template <typename R>
__device__ __forceinline__ uint32_t amax16(const R& r) {
  uint32_t m = amax_any(r);
  if (m >= INF_BITS) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t b = mag_bits(value(r, i));
      m = max(m, b < INF_BITS ? b : 0u);
    }
  }
  return m;
}

template <typename R>
__device__ __forceinline__ uint4 encode16(const R& r, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = scaled(value(r, 4 * i + j), inv);
    w[i] = encode2(s[0], s[1]) | (encode2(s[2], s[3]) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows of activations.  inv_row == null: codes [R, K], scales [R, KB].  With
// inv_row [R, k]: each row is stored to its k permuted rows instead (ids < 0:
// no row), so the routed experts read their tokens in expert order.
//
// Here and in the kernels that read what this one writes, nothing that a launch
// before may have written goes through the read-only path (__ldg, or const with
// __restrict__): that path wants memory which nobody writes while the grid lives, and a
// grid may become resident while the one before it still runs.
template <typename Tin>
__global__ void __launch_bounds__(256) quantize_rows(const Tin* x, uint32_t units, int K, int KB,
                                                     uint8_t* codes, float* scales,
                                                     const int32_t* inv_row, int k) {
  pdl_wait();
  pdl_trigger();
  const int sub = threadIdx.x & 7;
  const uint32_t u = blockIdx.x * (blockDim.x >> 3) + (threadIdx.x >> 3);
  const unsigned group = 0xffu << (threadIdx.x & 24);
  if (u < units) {
    const uint32_t row = u / (uint32_t)KB, b = u - row * (uint32_t)KB;
    const int col = (int)b * BLK + sub * 16;
    typename Raw<Tin>::type v;
    load16(x + (size_t)row * K + col, col < K, v);
    uint32_t m = amax16(v);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(group, m, o));
    const int e = scale_exp(m);
    const uint4 q = encode16(v, pow2(-e));
    if (inv_row == nullptr) {
      if (col < K) *reinterpret_cast<uint4*>(codes + (size_t)row * K + col) = q;
      if (sub == 0) scales[u] = pow2(e);
    } else {
      for (int j0 = 0; j0 < k; j0 += 8) {
        int to[8];           // asked for together, ahead of the stores
#pragma unroll
        for (int j = 0; j < 8; ++j) to[j] = j0 + j < k ? inv_row[(size_t)row * k + j0 + j] : -1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (to[j] < 0) continue;
          if (col < K) *reinterpret_cast<uint4*>(codes + (size_t)to[j] * K + col) = q;
          if (sub == 0) scales[(size_t)to[j] * KB + b] = pow2(e);
        }
      }
    }
  }
}

// One 128 x 128 block of a weight per CTA: thread = half a row (64 values).
template <typename Tin>
__global__ void __launch_bounds__(256) quantize_blocks(const Tin* w, int rows, int cols, int RB,
                                                       int CB, uint8_t* codes, float* scales) {
  __shared__ uint32_t part[8];
  pdl_wait();
  pdl_trigger();
  const int64_t blk = blockIdx.x;
  const int64_t mat = blk / ((int64_t)RB * CB);
  const int in = (int)(blk - mat * RB * CB);
  const int r = (in / CB) * BLK + (threadIdx.x >> 1);
  const int c0 = (in % CB) * BLK + (threadIdx.x & 1) * 64;
  const size_t at = ((size_t)mat * rows + r) * cols;
  typename Raw<Tin>::type v[4];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    load16(w + at + c0 + 16 * i, r < rows && c0 + 16 * i < cols, v[i]);
    m = max(m, amax16(v[i]));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, part[i]);
  const int e = scale_exp(m);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r < rows && c0 + 16 * i < cols)
      *reinterpret_cast<uint4*>(codes + at + c0 + 16 * i) = encode16(v[i], pow2(-e));
  if (threadIdx.x == 0) scales[blk] = pow2(e);
}

// y_acc[t] += sum over j of w_j rows[inv_row[t, j]], in slot order: the down projection
// leaves a token's k rows apart and they meet here, so a result does not depend on
// the order in which tiles end.  Adding tiles to y_acc as they end does, and saves a
// launch and the rows' way to memory and back: 128 experts of 2688 x 1856, 6 taken, in
// a graph with this kernel and without: 8 tokens 75 and 72 us, 301 tokens 241 and 235,
// 16384 tokens 1.95 and 1.79 ms.  One add to an element of y_acc, atomic, since the
// shared expert may add to it at the same time.  `parts` blocks share a token, a thread
// holds four features; rows of eight slots are asked for at once.
__global__ void __launch_bounds__(256) combine_rows(const float* rows, const int32_t* inv_row,
                                                    const float* perm_w, int parts, int k,
                                                    int quads, float* y_acc) {
  const int t = blockIdx.x / parts;
  const int q = (blockIdx.x - t * parts) * blockDim.x + threadIdx.x;
  int row[8];
  float w[8];
  auto slots = [&](int j0) {       // rows and weights of slots j0 ..; no row: id out of range
#pragma unroll
    for (int j = 0; j < 8; ++j) row[j] = j0 + j < k ? inv_row[(size_t)t * k + j0 + j] : -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = row[j] >= 0 ? perm_w[row[j]] : 0.f;
  };
  // The permute was complete before the down projection, the launch before, began: the
  // first slots are asked for ahead of the wait for its rows.
  slots(0);
  pdl_wait();
  pdl_trigger();
  if (q >= quads) return;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j0 = 0; j0 < k; j0 += 8) {
    if (j0) slots(j0);
    float4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = row[j] >= 0
                 ? __ldcs(reinterpret_cast<const float4*>(rows) + (size_t)row[j] * quads + q)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum.x = fmaf(w[j], v[j].x, sum.x);
      sum.y = fmaf(w[j], v[j].y, sum.y);
      sum.z = fmaf(w[j], v[j].z, sum.z);
      sum.w = fmaf(w[j], v[j].w, sum.w);
    }
  }
  red_add_f32x4(y_acc + ((size_t)t * quads + q) * 4, sum.x, sum.y, sum.z, sum.w);
}

}  // namespace f8
}  // namespace nh
