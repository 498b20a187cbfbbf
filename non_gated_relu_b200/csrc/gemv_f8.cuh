// gemv_f8.cuh -- block-scaled FP8 product of at most 32 dense rows: the decode
// form of the FP8 shared expert and linear layer.
//
//   out[r, n] = epi( sum_b sx[r, b] sw[n / 128, b] (xq[r] . wq[n] over block b) )
//
// Bound by the weights' bytes.  A CTA takes 16 weight rows over the whole K and its 8 warps take K blocks of 128 in turn, so the bytes
// of a task are all asked for at once: lane (g, q) loads 16 bytes of rows g and
// g + 8 at 16 q of each half block, straight into the fragments of
// mma.sync m16n8k32 (E4M3, float32 accumulate).  The order of features inside
// an MMA is free as long as both operands agree, so word i of a lane's 16
// bytes is k-slot i for weights and activations alike.  Each block's product
// starts from zero and enters the running sum times its two scales; the warps'
// sums are added in warp order, so a result does not depend on scheduling.
//
// Up to 8 rows the activations come unquantized: the four lanes that hold a
// token's block of 128 find its maximum with two shuffles and encode their words
// in registers, every CTA for itself, instead of a launch before this one.  3712 x
// 2688, 1 row: a call from the host takes 10 us in one launch and 15 in two; in a
// CUDA graph it is 5.1 against 4.0, because the second launch can ask for its
// weights ahead (asking for the values ahead, fewer blocks in flight and CTAs of
// four warps were all slower).
#pragma once

#include "gemm_tc.cuh"
#include "quant_f8.cuh"

namespace nh {
namespace f8v {

constexpr int WARPS = 8;
constexpr int MT = 16;      // weight rows of a task

enum Out : int {
  OUT_BF16 = 0,       // out bf16 [rows, N] = acc
  OUT_F32 = 1,        // out f32 [rows, N] = acc
  OUT_RELU2_F32 = 2,  // out f32 [rows, N] = relu(acc)^2   (quantized by the next kernel)
  OUT_ADD_F32 = 3,    // out f32 [rows, N] += acc, atomic adds
};

struct Args {
  const void* x;           // codes, or values, [rows, K]
  const float* xs;         // scales of codes [rows, KB]
  const uint8_t* w;        // codes [N, K]
  const float* ws;         // scales [ceil(N / 128), KB]
  int rows;                // at most NT
  int N, K, KB;
  int out_kind;
  void* out;               // [rows, N]
  int early_w;             // weights were complete before the previous launch in
                           // the stream began its work
};

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// One lane's 16 values at p, or zeros, as codes of a block whose other values lie
// in the lanes next to it; `e` is the exponent of the block's scale.
template <typename Tx>
__device__ __forceinline__ void quantize_block(const Tx* p, bool in0, bool in1, uint4& q0, uint4& q1,
                                               int& e) {
  typename f8::Raw<Tx>::type v0, v1;
  f8::load16(p, in0, v0);
  f8::load16(p + 64, in1, v1);
  uint32_t m = max(f8::amax16(v0), f8::amax16(v1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  e = f8::scale_exp(m);
  q0 = f8::encode16(v0, f8::pow2(-e));
  q1 = f8::encode16(v1, f8::pow2(-e));
}

// NT: rows, padded (8, 16, 32); U: K blocks of a warp in flight; Tx: uint8_t for
// codes, else the type of the values (NT = 8)
template <int NT, int U, typename Tx>
__global__ void __launch_bounds__(WARPS * 32, 2) f8_gemv(const Args a) {
  constexpr int NB = NT / 8;
  constexpr bool RAW = sizeof(Tx) > 1;
  static_assert(!RAW || NT == 8, "values are quantized for one tile of 8 tokens");
  __shared__ float red[WARPS][MT][NT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;
  const int n0 = blockIdx.x * MT;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  bool waited = false;
  auto wait_previous = [&]() {
    pdl_wait();
    pdl_trigger();
    waited = true;
  };
  if (!a.early_w) wait_previous();
  const uint8_t* w0 = a.w + ((size_t)n0 + gq) * a.K;
  const uint8_t* w1 = w0 + (size_t)8 * a.K;
  const float* ws = a.ws + (size_t)(n0 / 128) * a.KB;

  float acc[NB][4];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

  // x rows of this lane's fragment columns (token gq of each n-tile) and of its
  // accumulator columns (tokens 2 tq, 2 tq + 1); rows past the last repeat it and
  // are not stored
  const Tx* xp[NB];
  const float* sp[NB][2];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    xp[j] = static_cast<const Tx*>(a.x) + (size_t)min(8 * j + gq, a.rows - 1) * a.K;
    sp[j][0] = a.xs + (size_t)min(8 * j + 2 * tq, a.rows - 1) * a.KB;
    sp[j][1] = a.xs + (size_t)min(8 * j + 2 * tq + 1, a.rows - 1) * a.KB;
  }

  for (int b0 = warp; b0 < a.KB; b0 += WARPS * U) {
    uint4 wv[U][4];
    float sw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + u * WARPS;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int off = b * 128 + h * 64 + tq * 16;
        const bool in = b < a.KB && off < a.K;
        wv[u][2 * h] = in ? load_stream(w0 + off) : zero;
        wv[u][2 * h + 1] = in ? load_stream(w1 + off) : zero;
      }
      sw[u] = b < a.KB ? ws[b] : 0.f;
    }
    if (!waited) wait_previous();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + u * WARPS;
      if (b >= a.KB) break;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (8 * j >= a.rows) break;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const int off = b * 128 + tq * 16;
        uint4 xv[2];
        float s0, s1;
        if constexpr (RAW) {
          int e;
          quantize_block(xp[j] + off, off < a.K, off + 64 < a.K, xv[0], xv[1], e);
          s0 = f8::pow2(__shfl_sync(0xffffffffu, e, 8 * tq)) * sw[u];
          s1 = f8::pow2(__shfl_sync(0xffffffffu, e, 8 * tq + 4)) * sw[u];
        } else {
          xv[0] = off < a.K ? *reinterpret_cast<const uint4*>(xp[j] + off) : zero;
          xv[1] = off + 64 < a.K ? *reinterpret_cast<const uint4*>(xp[j] + off + 64) : zero;
          s0 = sp[j][0][b] * sw[u];
          s1 = sp[j][1][b] * sw[u];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 p = wv[u][2 * h], q = wv[u][2 * h + 1];
          mma_e4m3(d, p.x, q.x, p.y, q.y, xv[h].x, xv[h].y);
          mma_e4m3(d, p.z, q.z, p.w, q.w, xv[h].z, xv[h].w);
        }
        acc[j][0] = fmaf(s0, d[0], acc[j][0]);
        acc[j][1] = fmaf(s1, d[1], acc[j][1]);
        acc[j][2] = fmaf(s0, d[2], acc[j][2]);
        acc[j][3] = fmaf(s1, d[3], acc[j][3]);
      }
    }
  }
  if (!waited) wait_previous();   // a warp without a K block
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    red[warp][gq][8 * j + 2 * tq] = acc[j][0];
    red[warp][gq][8 * j + 2 * tq + 1] = acc[j][1];
    red[warp][gq + 8][8 * j + 2 * tq] = acc[j][2];
    red[warp][gq + 8][8 * j + 2 * tq + 1] = acc[j][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < MT * NT; i += WARPS * 32) {
    const int f = i % MT, c = i / MT;
    if (c >= a.rows) break;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v += red[w][f][c];
    const size_t at = (size_t)c * a.N + n0 + f;
    switch (a.out_kind) {
      case OUT_BF16: static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v); break;
      case OUT_F32: static_cast<float*>(a.out)[at] = v; break;
      case OUT_RELU2_F32: static_cast<float*>(a.out)[at] = f8::relu2_nan(v); break;
      default: red_add_f32(static_cast<float*>(a.out) + at, v);
    }
  }
}

}  // namespace f8v
}  // namespace nh
