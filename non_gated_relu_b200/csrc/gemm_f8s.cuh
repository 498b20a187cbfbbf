// gemm_f8s.cuh -- block-scaled FP8 product with the weights on the MMA M side:
// the routed experts' form for batches that leave an expert few rows, and the
// dense form of as many rows as give each SM one tile of 64.
//
//   acc[n, r] = sum_b sw[n / 128, b] sx[r, b] (wq[n] . xq[r] over K block b of 128)
//
// Up to about a hundred rows an expert, the experts' weights are all that
// matters: each is read once from memory and meets few rows.  A tile is 128
// weight rows (one scale block) against NT rows of the entry, so a K block
// stages 16 KB of weights and NT / 8 KB of activations, its MMAs (M = 128, N =
// NT, four of K = 32 from zero) take a fraction of the time the weights take to
// arrive, and the rate is that of memory as long as enough bytes are under way:
// two CTAs per SM, each with about 100 KB of stages (one CTA of 192 KB, as 128
// rows a tile would need, drew 3.7 TB/s where two draw 6).  Measured, one launch at
// a time under the profiler, 6 of 128 experts of 2688 x 1856 taken: 301 tokens (all
// hit): 106 and 107 us for the two projections, 6.0 TB/s; 8 tokens: 35 and 35.  As in
// the pair kernel each K block is its own accumulator, four in turn, drained
// into registers times its scales by eight warps (warp w: weight rows of quarter
// w mod 4, half of the columns); the weight scale is one number per block and the
// row scales are held by the lanes, one column each, and pass through shared
// memory.
//
// A launch that follows this call's own quantization starts on its first stages'
// weights before it waits for it (they were there before), which covers launch
// and tail.
//
// The end of a tile: a warp stores 32 neighbouring features of a row per
// instruction; relu^2 needs the maximum over the tile's 128 features, which lie
// in four warps: they exchange column maxima and then codes through shared
// memory, in two bounded barrier waits, and store whole 128-byte rows.
//
// Roles (320 threads): warp 0 producer, warp 1 tensor memory owner and MMA
// issuer, warps 2..9 drain.  All waits are bounded.
#pragma once

#include "gemm_f8.cuh"

namespace nh {
namespace f8s {

constexpr int BK = 128, UMMA_K = 32, M = 128;
constexpr int DRAINS = 8;
constexpr int THREADS = 64 + 32 * DRAINS;
constexpr int NBUF = 4;            // accumulators

enum Out : int {
  OUT_RELU2_F8 = 0,  // out E4M3 [rows, N] of relu(acc)^2, scales [rows, ceil(N / 128)]
  OUT_BF16 = 1,      // out bf16 [rows, N] = acc
  OUT_F32 = 2,       // out f32 [rows, N] = acc
  OUT_ADD_F32 = 3,   // out f32 [rows, N] += acc, atomic adds (one to an element)
};

struct Args {
  const float* xs;         // [rows, KB]
  const float* ws;         // [E, ceil(N / 128), KB]
  const int4* tiles;       // (expert, first row, rows <= NT, -) or null: dense rows
  const int32_t* num_tiles;
  int dense_rows;
  int N, K, KB;
  void* out;
  float* out_scales;       // OUT_RELU2_F8
  int* status;
  uint64_t timeout_ns;
  int early_w;             // weights and tile table were complete before the
                           // previous launch in the stream began its work
};

template <int NT, int STAGES, int CTAS>
struct Shape {
  static constexpr int W_BYTES = M * BK;
  static constexpr int X_BYTES = NT * BK;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int TMEM_COLS = NBUF * NT;
  static constexpr int NBAR = 2 * STAGES + 2 * NBUF + 1 + 4;
  static constexpr int CODES = NT * 144;              // [NT][128] codes, rows 144 bytes apart
  static constexpr int SMEM = STAGES * STAGE_BYTES + 1024 + CODES + 8 * NT * 4 + NBAR * 8 + 16;
  static_assert(SMEM * CTAS <= 227 * 1024, "shared memory of an SM");
  static_assert(TMEM_COLS * CTAS <= 512 && TMEM_COLS >= 32, "tensor memory");
  static_assert(STAGE_BYTES % 1024 == 0, "stage alignment");
};

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// NC accumulator columns of this thread's weight row
template <int NC>
__device__ __forceinline__ void load_columns(uint32_t taddr, uint32_t (&v)[NC]) {
  if constexpr (NC % 32 == 0) {
#pragma unroll
    for (int c = 0; c < NC; c += 32) f8g::tmem_ld32(taddr + c, v + c);
  } else {
#pragma unroll
    for (int c = 0; c < NC; c += 8) tmem_ld8(taddr + c, v + c);
  }
}

template <int NT>
__device__ __forceinline__ int4 entry(const Args& g, int m) {
  if (g.tiles) return g.tiles[m];
  return make_int4(0, m * NT, min(NT, g.dense_rows - m * NT), 0);
}

template <int NT, int STAGES, int CTAS, int OUT>
__global__ void __launch_bounds__(THREADS, CTAS)
    f8_swap_gemm(const __grid_constant__ CUtensorMap map_x,
                 const __grid_constant__ CUtensorMap map_w, const Args g) {
  using S = Shape<NT, STAGES, CTAS>;
  constexpr int NC = NT / 2;                  // columns of a drain warp
  constexpr int CL = (NC + 31) / 32;          // columns whose scales a lane holds
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  uint8_t* const codes = base_ptr + STAGES * S::STAGE_BYTES;                  // [NT][144]
  uint32_t* const amax = reinterpret_cast<uint32_t*>(codes + S::CODES);       // [4][NT]
  float* const col_scales = reinterpret_cast<float*>(amax + 4 * NT);          // [DRAINS][NC]
  const uint32_t bar0 = base + STAGES * S::STAGE_BYTES + S::CODES + 8 * NT * 4;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + NBUF + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 2 * NBUF);
  // per column half: maxima written, codes written
  auto half_bar = [&](int h, int w) { return bar0 + 8u * (2 * STAGES + 2 * NBUF + 1 + 2 * h + w); };
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(codes + S::CODES + 8 * NT * 4 + S::NBAR * 8);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < NBUF; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), DRAINS);
    }
    mbar_init(drain_bar, 1);
    for (int i = 0; i < 4; ++i) mbar_init(half_bar(0, 0) + 8u * i, DRAINS / 2);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_w);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), S::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // the producer of an early launch waits after its first weights
  const bool early = g.early_w != 0;
  if (!early || warp != 0) pdl_wait();
  pdl_trigger();
  const WaitCtl wc{abort_flag, g.status, g.timeout_ns};

  const int n_blocks = (g.N + M - 1) / M;
  const int num_m = g.tiles ? *g.num_tiles : (g.dense_rows + NT - 1) / NT;
  const int step_m = gridDim.x / n_blocks, step_nb = gridDim.x - step_m * n_blocks;
  f8g::TileWalk t{(int)blockIdx.x / n_blocks, (int)blockIdx.x % n_blocks};
  const int nk = g.KB;

  if (warp == 0) {
    // ---------------- producer ----------------
    int stage = 0;
    uint32_t phase = 0;
    long issued = 0;
    bool ok = true;
    if (early) {
      // weights of the first stages, then the wait, then their activations
      f8g::TileWalk e = t;
      int kb = 0, ahead = 0;
      for (; ahead < STAGES && e.m < num_m; ++ahead) {
        if (f8g::elect_one()) {
          mbar_arrive_expect_tx(full_bar(ahead), S::STAGE_BYTES);
          tma_load_3d(base + ahead * S::STAGE_BYTES, &map_w, full_bar(ahead), kb * BK, e.nb * M,
                      entry<NT>(g, e.m).x);
        }
        if (++kb == nk) {
          kb = 0;
          e.next(n_blocks, step_m, step_nb);
        }
      }
      pdl_wait();
      e = t;
      kb = 0;
      for (int s = 0; s < ahead; ++s) {
        if (f8g::elect_one())
          tma_load_2d(base + s * S::STAGE_BYTES + S::W_BYTES, &map_x, full_bar(s), kb * BK,
                      entry<NT>(g, e.m).y);
        if (++kb == nk) {
          kb = 0;
          e.next(n_blocks, step_m, step_nb);
        }
      }
      issued = ahead;
    }
    long skip = issued;        // stages of the loop below that are under way already
    for (; ok && t.m < num_m; t.next(n_blocks, step_m, step_nb)) {
      const int4 ent = entry<NT>(g, t.m);
      for (int kb = 0; kb < nk; ++kb) {
        if (skip > 0) {
          --skip;
        } else {
          ok = __all_sync(0xffffffffu, mbar_wait_spin(empty_bar(stage), phase ^ 1u, wc, SITE_TC_PRODUCER));
          if (!ok) break;
          if (f8g::elect_one()) {
            const uint32_t sw = base + stage * S::STAGE_BYTES;
            mbar_arrive_expect_tx(full_bar(stage), S::STAGE_BYTES);
            tma_load_3d(sw, &map_w, full_bar(stage), kb * BK, t.nb * M, ent.x);
            tma_load_2d(sw + S::W_BYTES, &map_x, full_bar(stage), kb * BK, ent.y);
          }
          ++issued;
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      const long first = issued > STAGES ? issued - STAGES : 0;
      for (long i = first; i < issued; ++i)
        tc::mbar_drain(full_bar((int)(i % STAGES)), (uint32_t)((i / STAGES) & 1), g.timeout_ns,
                       g.status);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    int stage = 0;
    uint32_t phase = 0, use = 0;
    bool ok = true, any = false;
    const uint64_t sdesc0 = make_sdesc_sw128(base);
    const uint32_t idesc = f8g::make_idesc_e4m3(M, NT);
    for (; ok && t.m < num_m; t.next(n_blocks, step_m, step_nb)) {
      for (int kb = 0; kb < nk; ++kb, ++use) {
        const uint32_t a = use % NBUF;
        ok = __all_sync(0xffffffffu,
                        mbar_wait_spin(full_bar(stage), phase, wc, SITE_TC_MMA) &&
                            mbar_wait_spin(tempty_bar(a), ((use / NBUF) & 1u) ^ 1u, wc, SITE_TC_MMA));
        if (!ok) break;
        tc_fence_after();
        const uint64_t dw = sdesc0 + (uint64_t)(stage * (S::STAGE_BYTES >> 4));
        const uint64_t dx = dw + (S::W_BYTES >> 4);
        if (f8g::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < BK / UMMA_K; ++kk)
            umma_f8(tmem_base + a * NT, dw + kk * (UMMA_K >> 4), dx + kk * (UMMA_K >> 4), idesc,
                    kk != 0);
          umma_commit(tfull_bar(a));
          umma_commit(empty_bar(stage));
        }
        any = true;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && any && f8g::elect_one()) {
      umma_commit(drain_bar);
      tc::mbar_drain(drain_bar, 0, g.timeout_ns, g.status);
    }
  } else {
    // ---------------- drain: 32 weight rows x NC columns per warp ----------------
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tq = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * NC);
    float* const scales = col_scales + (warp - 2) * NC;
    uint32_t use = 0, tiles_done = 0;
    bool ok = true;
    for (; ok && t.m < num_m; t.next(n_blocks, step_m, step_nb)) {
      const int4 ent = entry<NT>(g, t.m);
      const float* ws = g.ws + ((size_t)ent.x * n_blocks + t.nb) * nk;
      const float* xs[CL];
      float sx[CL], sw = *ws;
#pragma unroll
      for (int i = 0; i < CL; ++i) {
        // columns past the entry repeat its last row and are not stored
        const int c = half * NC + min(lane + 32 * i, NC - 1);
        xs[i] = g.xs + (size_t)(ent.y + min(c, ent.z - 1)) * nk;
        sx[i] = *xs[i];
      }
      float acc[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[c] = 0.f;
      for (int kb = 0; kb < nk; ++kb, ++use) {
        const uint32_t a = use % NBUF;
        // the columns' scales, read back four to a load (one shuffle a column takes
        // an SM's shuffle unit longer than the weights of 64 columns need to arrive)
        __syncwarp();
#pragma unroll
        for (int i = 0; i < CL; ++i)
          if (lane + 32 * i < NC) scales[lane + 32 * i] = sx[i] * sw;
        __syncwarp();
        if (kb + 1 < nk) {
          sw = ws[kb + 1];
#pragma unroll
          for (int i = 0; i < CL; ++i) sx[i] = xs[i][kb + 1];
        }
        ok = __all_sync(0xffffffffu, mbar_wait_spin(tfull_bar(a), (use / NBUF) & 1u, wc, SITE_TC_EPILOGUE));
        if (!ok) break;
        tc_fence_after();
        uint32_t v[NC];
        load_columns<NC>(tq + a * NT, v);
        f8g::tmem_wait();
        f8g::pin(v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) f8g::arrive_relaxed(tempty_bar(a));
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const float4 s = *reinterpret_cast<const float4*>(scales + c);
          acc[c] = fmaf(s.x, __uint_as_float(v[c]), acc[c]);
          acc[c + 1] = fmaf(s.y, __uint_as_float(v[c + 1]), acc[c + 1]);
          acc[c + 2] = fmaf(s.z, __uint_as_float(v[c + 2]), acc[c + 2]);
          acc[c + 3] = fmaf(s.w, __uint_as_float(v[c + 3]), acc[c + 3]);
        }
      }
      if (!ok) break;
      const int cols = min(NC, ent.z - half * NC);         // <= 0: none in this half
      const int f = t.nb * M + quarter * 32 + lane;        // this lane's feature
      if constexpr (OUT != OUT_RELU2_F8) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (c < cols && f < g.N) {
            const size_t at = (size_t)(ent.y + half * NC + c) * g.N + f;
            if constexpr (OUT == OUT_BF16)
              static_cast<__nv_bfloat16*>(g.out)[at] = __float2bfloat16_rn(acc[c]);
            else if constexpr (OUT == OUT_F32)
              static_cast<float*>(g.out)[at] = acc[c];
            else
              red_add_f32(static_cast<float*>(g.out) + at, acc[c]);
          }
      } else {
        uint32_t top[CL];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          acc[c] = f8::relu2_nan(acc[c]);
          const uint32_t b = f8::mag_bits(acc[c]);
          const uint32_t m = __reduce_max_sync(0xffffffffu, b < f8::INF_BITS && f < g.N ? b : 0u);
          if (lane == (c & 31)) top[c / 32] = m;
        }
#pragma unroll
        for (int i = 0; i < CL; ++i)
          if (lane + 32 * i < NC) amax[quarter * NT + half * NC + lane + 32 * i] = top[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(half_bar(half, 0));
        ok = __all_sync(0xffffffffu, mbar_wait(half_bar(half, 0), tiles_done & 1u, wc, SITE_TC_EPILOGUE));
        if (!ok) break;
        int ex[CL];
#pragma unroll
        for (int i = 0; i < CL; ++i) {
          const int c = half * NC + min(lane + 32 * i, NC - 1);
          ex[i] = f8::scale_exp(max(max(amax[c], amax[NT + c]), max(amax[2 * NT + c], amax[3 * NT + c])));
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float v = f8::scaled(acc[c], f8::pow2(-__shfl_sync(0xffffffffu, ex[c / 32], c & 31)));
          codes[(half * NC + c) * 144 + quarter * 32 + lane] = (uint8_t)f8::encode2(v, v);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(half_bar(half, 1));
        ok = __all_sync(0xffffffffu, mbar_wait(half_bar(half, 1), tiles_done & 1u, wc, SITE_TC_EPILOGUE));
        if (!ok) break;
        ++tiles_done;
        // rows of this half, four to an instruction, every fourth such to this warp
        const int word = lane & 7, n = min(M, g.N - t.nb * M);
        for (int c0 = 4 * quarter; c0 < cols; c0 += 16) {
          const int c = c0 + (lane >> 3);
          if (c < cols && 16 * word < n)
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g.out) +
                                      (size_t)(ent.y + half * NC + c) * g.N + t.nb * M + 16 * word) =
                *reinterpret_cast<const uint4*>(codes + (half * NC + c) * 144 + 16 * word);
        }
        if (quarter == 0) {
#pragma unroll
          for (int i = 0; i < CL; ++i) {
            const int c = lane + 32 * i;
            if (c < cols)
              g.out_scales[(size_t)(ent.y + half * NC + c) * n_blocks + t.nb] = f8::pow2(ex[i]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, S::TMEM_COLS);
  }
}

}  // namespace f8s
}  // namespace nh
