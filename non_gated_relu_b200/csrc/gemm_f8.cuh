// gemm_f8.cuh -- block-scaled FP8 product on CTA pairs (tcgen05 cta_group::2,
// kind::f8f6f4): the prefill form of the FP8 experts, shared expert and linear
// layer.
//
//   acc[r, n] = sum_b sx[r, b] sw[n / 128, b] (xq[r] . wq[n] over K block b of 128)
//
// The two scales change with every K block, so the product of a block cannot
// stay in the tensor-memory accumulator: each block is one accumulator (four
// MMAs of K = 32 starting from zero), two accumulators take turns, and drain
// warps read one into registers and add it up times its scales, while the tensor
// cores fill the other.  A tile is 256 rows x 256 features for a pair of CTAs
// (each stages 128 rows of both operands).  Per K block of a tile the MMAs take
// 512 cycles and the multiply-adds 256 of each SM's float32 units; what sets the
// rate is how long an accumulator is away from the tensor cores: a drain warp
// takes its 128 columns in four loads, each in flight while the one before is
// added, and hands the accumulator back before it adds the last.  They wait without
// the sleep hint (a K block of a lone pair 461 -> 449 ns).  Measured: a K
// block every 700 to 850 cycles and 2000 to 3500 for the end of a tile.  One launch at
// a time, under the profiler: 16384 x 3712 x 2688 in 160 us (2.0 PFLOP/s), the experts'
// two products of 16384 tokens (128 experts of 2688 x 1856, 6 taken) in 652 and 722.
// Calls one after the other run at the power limit: the linear call takes 207 us, 22 of
// them the quantization, the experts' 1.95 ms.
// A thread owns one row and 128 features, which makes the
// scale one number per thread and block, and leaves the maximum of a (row, 128
// features) block of the output inside one thread, where the next projection's
// quantization needs it.
//
// Roles (384 threads): warp 0 TMA producer (both CTAs); warp 1 tensor memory
// owner and, in the leader, MMA issuer; warps 4..11 drain (warp w: row quarter
// w mod 4, feature half (w - 4) / 4).  The first four warps hand registers to
// the other eight, whose sums would spill in an even split.  Producer and
// issuer run their loops as whole warps and elect a lane for the instruction
// itself: descriptors and addresses then stay in uniform registers (one lane in
// a branch of its own needed 700 cycles to issue a K block, this way it takes 140).  Tiles are dealt
// out in turn (tile i to pair i mod pairs): they all take the same time.  Both
// CTAs' copies complete on the leader's stage barrier, MMA completion is
// committed to both CTAs, the peer's drains arrive on the leader's barriers.
// Every wait is bounded, as in the bf16 kernels.
#pragma once

#include "gemm_tc.cuh"
#include "quant_f8.cuh"

namespace nh {
namespace f8g {

constexpr int BK = 128;        // K of a stage: one block of scales, one 128-byte row
constexpr int UMMA_K = 32;
constexpr int MP = 256, NT = 256, HALF = 128;
constexpr int STAGES = 6;
constexpr int EPI_WARPS = 8;
constexpr int COLS = 128;      // features of a drain warp's rows: one scale block
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr int REGS_ROLES = 48, REGS_DRAIN = 224;   // per thread, after the split
constexpr int REGS_NEEDED = 128 * REGS_ROLES + 32 * EPI_WARPS * REGS_DRAIN;
constexpr int OP_BYTES = HALF * BK;
constexpr int STAGE_BYTES = 2 * OP_BYTES;
constexpr int TMEM_COLS = 2 * NT;
constexpr int NBAR = 2 * STAGES + 3;
constexpr int STORE_BYTES = EPI_WARPS * 32 * 128;  // 128 bytes of each drained row
constexpr int SMEM = STAGES * STAGE_BYTES + 1024 + STORE_BYTES + NBAR * 8 + 16;
static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");

enum Out : int {
  OUT_BF16 = 0,        // out bf16 [rows, N] = acc
  OUT_F32 = 1,         // out f32 [rows, N] = acc
  OUT_RELU2_F8 = 2,    // out E4M3 [rows, N] of relu(acc)^2, scales [rows, ceil(N / 128)]
  OUT_ADD_F32 = 3,     // out f32 [rows, N] += acc, atomic adds (one to an element)
};

struct Args {
  const float* xs;         // [rows, KB]
  const float* ws;         // [E, ceil(N / 128), KB]
  const int4* tiles;       // (expert, first row, rows <= 256, -) or null: dense rows
  const int32_t* num_tiles;
  int dense_rows;
  int N, K, KB;
  void* out;
  float* out_scales;       // OUT_RELU2_F8
  int64_t ldo;
  int* status;
  uint64_t timeout_ns;
};

// D (+)= A B^T over both CTAs' shared memory, E4M3 in, f32 accumulate, M = 256
__device__ __forceinline__ void umma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D f32, A and B E4M3 (format 0), both K-major
__device__ __forceinline__ uint32_t make_idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 32 accumulator columns of this thread's row; the values are there after
// tmem_wait and pin.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      :
        "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// pin: volatile statements keep their order, so what uses the pinned registers
// cannot move ahead of the wait before it.
__device__ __forceinline__ void tmem_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Arrive on a barrier (a shared::cluster address) without releasing memory: what
// it hands over is tensor memory that has been read (tcgen05.wait::ld and
// tcgen05.fence order that), no memory contents.  A releasing arrive waits for
// the lane's global loads in flight, 200 to 300 cycles for every accumulator.
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Arrive once on the barrier at the same place in both CTAs when all prior pair
// MMAs of this thread complete.
__device__ __forceinline__ void umma_commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// acc += s v for 32 columns
__device__ __forceinline__ void add_scaled(float* acc, const uint32_t (&v)[32], float s) {
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] = fmaf(s, __uint_as_float(v[i]), acc[i]);
}

// A pair's tiles, `pairs` apart: (tile entry m, feature block nb)
struct TileWalk {
  int m, nb;
  __device__ __forceinline__ void next(int n_blocks, int step_m, int step_nb) {
    m += step_m;
    nb += step_nb;
    if (nb >= n_blocks) {
      nb -= n_blocks;
      ++m;
    }
  }
};

__device__ __forceinline__ int4 entry(const Args& g, int m) {
  if (g.tiles) return g.tiles[m];
  return make_int4(0, m * MP, min(MP, g.dense_rows - m * MP), 0);
}

// MMA N of a tile with n_eff features left: whole multiples of 32 (weight rows
// past N arrive as zeros and their columns are not stored)
__device__ __forceinline__ int mma_n(int n_eff) { return (n_eff + 31) & ~31; }

// relu of a row's first n features in place (n a multiple of 16), and the bits of
// the largest finite square.  Squaring keeps the order of what is not negative, so
// the maximum is taken before it, as an integer, where Inf and NaN come out on top:
// only then the squares are looked at one by one.
__device__ __forceinline__ uint32_t relu_amax(int n, float (&acc)[COLS]) {
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < COLS; c += 16) {
    if (c >= n) break;
#pragma unroll
    for (int i = c; i < c + 16; i += 2) {
      acc[i] = f8::relu_nan(acc[i]);
      acc[i + 1] = f8::relu_nan(acc[i + 1]);
      m = __vimax3_u32(m, f8::mag_bits(acc[i]), f8::mag_bits(acc[i + 1]));
    }
  }
  const float top = __uint_as_float(m);
  const uint32_t sq = f8::mag_bits(top * top);
  if (m < f8::INF_BITS && sq < f8::INF_BITS) return sq;
  m = 0;
#pragma unroll
  for (int i = 0; i < COLS; ++i) {
    const uint32_t b = f8::mag_bits(acc[i] * acc[i]);
    if (i < n && b < f8::INF_BITS) m = max(m, b);
  }
  return m;
}

// The end of a tile: a warp's 32 rows x 128 features, a lane's row in acc.  A
// store of 16 bytes by every lane to its own row touches 32 lines (a tile's
// stores took 5000 to 9000 cycles that way, its K loop 15000), so the rows cross
// shared memory 128 bytes at a time and leave four to an instruction: 16-byte
// word j of row r waits in slot j ^ (r mod 8).  row0: first row; rows: how many
// exist; n: features that exist (a multiple of 16).
template <int OUT>
__device__ __forceinline__ void finish_rows(const Args& g, int row0, int rows, int f0, int n,
                                            float (&acc)[COLS], uint4* stage, int lane) {
  constexpr bool F32 = OUT == OUT_F32 || OUT == OUT_ADD_F32;
  constexpr int PER = F32 ? 4 : (OUT == OUT_BF16 ? 8 : 16);   // features of a 16-byte word
  constexpr int PASSES = COLS / (8 * PER);
  const int mine = row0 + min(lane, rows - 1);
  float w = 1.f;          // OUT_RELU2_F8: one over the row's scale
  if constexpr (OUT == OUT_RELU2_F8) {
    const int e = f8::scale_exp(relu_amax(n, acc));
    w = f8::pow2(-e);
    if (lane < rows)
      g.out_scales[(size_t)mine * ((g.N + 127) / 128) + f0 / 128] = f8::pow2(e);
  }
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = (p * 8 + j) * PER;
      uint4 word;
      if constexpr (F32) {
        word = make_uint4(__float_as_uint(acc[c]), __float_as_uint(acc[c + 1]),
                          __float_as_uint(acc[c + 2]), __float_as_uint(acc[c + 3]));
      } else if constexpr (OUT == OUT_BF16) {
        word = make_uint4(pack_bf16x2(acc[c], acc[c + 1]), pack_bf16x2(acc[c + 2], acc[c + 3]),
                          pack_bf16x2(acc[c + 4], acc[c + 5]), pack_bf16x2(acc[c + 6], acc[c + 7]));
      } else {
        f8::F32x16 sq;
#pragma unroll
        for (int i = 0; i < 16; ++i) sq.v[i] = acc[c + i] * acc[c + i];
        word = f8::encode16(sq, w);
      }
      stage[lane * 8 + (j ^ (lane & 7))] = word;
    }
    __syncwarp();
    const int j = lane & 7, c = (p * 8 + j) * PER;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      const uint4 word = stage[r * 8 + (j ^ (r & 7))];
      const int64_t row = row0 + r;
      if (r < rows && c < n) {
        const size_t at = (size_t)row * g.ldo + f0 + c;
        if constexpr (OUT == OUT_ADD_F32)
          red_add_f32x4(static_cast<float*>(g.out) + at, __uint_as_float(word.x),
                        __uint_as_float(word.y), __uint_as_float(word.z), __uint_as_float(word.w));
        else if constexpr (OUT == OUT_F32)
          *reinterpret_cast<uint4*>(static_cast<float*>(g.out) + at) = word;
        else if constexpr (OUT == OUT_BF16)
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(g.out) + at) = word;
        else
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g.out) + at) = word;
      }
    }
  }
}

template <int OUT>
__global__ void __launch_bounds__(THREADS, 1)
    f8_pair_gemm(const __grid_constant__ CUtensorMap map_x,
                 const __grid_constant__ CUtensorMap map_w, const Args g) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const uint32_t bar0 = base + STAGES * STAGE_BYTES + STORE_BYTES;
  uint4* const stores = reinterpret_cast<uint4*>(base_ptr + STAGES * STAGE_BYTES);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  // a stage's MMAs are done: the producer may refill it, and the accumulator
  // that they wrote may be drained
  auto done_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * STAGES + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 2);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + STAGES * STAGE_BYTES + STORE_BYTES + NBAR * 8);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(done_bar(s), 1);
    }
    for (uint32_t a = 0; a < 2; ++a) mbar_init(tempty_bar(a), 2 * EPI_WARPS);   // both CTAs' drains
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_w);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // the peer's barriers are initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const WaitCtl wc{abort_flag, g.status, g.timeout_ns};

  const int num_m = g.tiles ? *g.num_tiles : (g.dense_rows + MP - 1) / MP;
  const int n_blocks = (g.N + NT - 1) / NT;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int step_m = pairs / n_blocks, step_nb = pairs - step_m * n_blocks;
  TileWalk t{pair / n_blocks, pair % n_blocks};
  const int nk = g.KB;

  // the split draws on what the block was launched with: the host checks that
  // the kernel's registers cover REGS_NEEDED before any launch
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_ROLES));
    if (warp == 0) {
      // ---------------- producer ----------------
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      bool ok = true;
      const uint32_t full0 = map_to_rank(full_bar(0), 0);   // the leader's stage barriers
      for (; ok && t.m < num_m; t.next(n_blocks, step_m, step_nb)) {
        const int nb = t.nb;
        const int4 ent = entry(g, t.m);
        const int x_row = ent.y + (int)rank * HALF;
        const int w_row = nb * NT + (int)rank * (mma_n(min(NT, g.N - nb * NT)) / 2);
        for (int kb = 0; kb < nk; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait_spin(done_bar(stage), phase ^ 1u, wc,
                                                      SITE_TC_PRODUCER));
          if (!ok) break;
          const uint32_t sx = base + stage * STAGE_BYTES, sw = sx + OP_BYTES;
          const uint32_t fb = full0 + 8u * stage;
          if (elect_one()) {
            if (leader) mbar_arrive_expect_tx(full_bar(stage), 2u * STAGE_BYTES);
            tma_load_2d_pair(sx, &map_x, fb, kb * BK, x_row);
            tma_load_3d_pair(sw, &map_w, fb, kb * BK, w_row, ent.x);
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader && lane == 0) {
        // the leader's stage barriers count both CTAs' copies: wait for those in flight
        const long first = issued > STAGES ? issued - STAGES : 0;
        for (long i = first; i < issued; ++i)
          tc::mbar_drain(full_bar((int)(i % STAGES)), (uint32_t)((i / STAGES) & 1), g.timeout_ns,
                         g.status);
      }
    } else if (warp == 1 && leader) {
      // ---------------- MMA issuer ----------------
      int stage = 0;
      uint32_t phase = 0, use = 0;
      bool ok = true, any = false;
      const uint64_t sdesc0 = make_sdesc_sw128(base);
      for (; ok && t.m < num_m; t.next(n_blocks, step_m, step_nb)) {
        const int nb = t.nb;
        const uint32_t idesc = make_idesc_e4m3(MP, mma_n(min(NT, g.N - nb * NT)));
        for (int kb = 0; kb < nk; ++kb, ++use) {
          const uint32_t acc = use & 1u;
          ok = __all_sync(0xffffffffu,
                          mbar_wait_spin(full_bar(stage), phase, wc, SITE_TC_MMA) &&
                              mbar_wait_spin(tempty_bar(acc), ((use >> 1) & 1u) ^ 1u, wc, SITE_TC_MMA));
          if (!ok) break;
          tc_fence_after();
          // start addresses count 16-byte units in the descriptor's low bits
          const uint64_t dx = sdesc0 + (uint64_t)(stage * (STAGE_BYTES >> 4));
          const uint64_t dw = dx + (OP_BYTES >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BK / UMMA_K; ++kk)
              umma_f8_pair(tmem_base + acc * NT, dx + kk * (UMMA_K >> 4), dw + kk * (UMMA_K >> 4),
                           idesc, kk != 0);
            umma_commit_both(done_bar(stage));
          }
          any = true;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // the lane that issued them commits and waits for the MMAs in flight
      if (!ok && any && elect_one()) {
        umma_commit_pair(drain_bar);
        tc::mbar_drain(drain_bar, 0, g.timeout_ns, g.status);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_DRAIN));
    // ---------------- drain: 32 rows x 128 features per warp ----------------
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tq = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * COLS);
    const uint32_t tempty0 = map_to_rank(tempty_bar(0), 0);   // the leader's
    const int first = (int)rank * HALF + quarter * 32;        // the warp's rows in a tile
    uint32_t use = 0, phase = 0;
    int stage = 0;
    bool ok = true;
    for (; ok && t.m < num_m; t.next(n_blocks, step_m, step_nb)) {
      const int4 ent = entry(g, t.m);
      const int f0 = t.nb * NT + half * COLS;
      const int n = min(COLS, g.N - f0);           // <= 0: no features in this half
      const float* xs = g.xs + (size_t)(ent.y + min(first + lane, ent.z - 1)) * nk;
      const float* ws = g.ws + ((size_t)ent.x * ((g.N + 127) / 128) + (n > 0 ? f0 / 128 : 0)) * nk;
      float sx = *xs, sw = *ws;
      float acc[COLS];
#pragma unroll
      for (int i = 0; i < COLS; ++i) acc[i] = 0.f;
      for (int kb = 0; kb < nk; ++kb, ++use) {
        const uint32_t a = use & 1u, from = tq + a * NT;
        // the warp leaves together, also where a wait runs out for some lanes
        ok = __all_sync(0xffffffffu, mbar_wait_spin(done_bar(stage), phase, wc, SITE_TC_EPILOGUE));
        if (!ok) break;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        tc_fence_after();
        // four loads of 32 columns, each in flight while the one before is added;
        // the accumulator goes back before the last is added
        uint32_t v0[32], v1[32];
        if (n > 0) tmem_ld32(from, v0);
        const float s = sx * sw;
        if (kb + 1 < nk) {
          sx = xs[kb + 1];
          sw = ws[kb + 1];
        }
        if (n > 0) {
          tmem_wait();
          pin(v0);
          tmem_ld32(from + 32, v1);
          add_scaled(acc, v0, s);
          tmem_wait();
          pin(v1);
          tmem_ld32(from + 64, v0);
          add_scaled(acc + 32, v1, s);
          tmem_wait();
          pin(v0);
          tmem_ld32(from + 96, v1);
          add_scaled(acc + 64, v0, s);
          tmem_wait();
          pin(v1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_relaxed(tempty0 + 8u * a);
        if (n > 0) add_scaled(acc + 96, v1, s);
      }
      if (ok && n > 0 && first < ent.z)
        finish_rows<OUT>(g, ent.y + first, min(32, ent.z - first), f0, n, acc,
                         stores + (warp - 4) * 256, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // no CTA leaves while its peer may still touch its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

}  // namespace f8g
}  // namespace nh
