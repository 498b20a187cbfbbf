// gate.cuh -- the router's choice from its logits, and its gradient.
//
// Per token, with l the logits as the router reads them (NaN counts as -inf,
// an expert that cannot be taken; +inf as the largest float32):
//   s = sigmoid(l)  or  softmax(l) over the E experts
//   c = s + bias (bias selects only, it never enters a weight); -inf where l = -inf
//   group value = its largest c, or the sum of its two largest (a missing second
//   counts 0); the topk_group best groups stay; the k best experts of those,
//   (c desc, id asc); groups tie to the lower group
//   w_j = alpha s_j / sum of the chosen s   (norm)   or   alpha s_j
//
// The choice is that of exact scores.  Without a bias and without a sum over
// two experts the logits order the experts as their scores do, so the float32
// logits are compared themselves.  Otherwise c is computed in float32 first;
// a token in which two neighbours that the choice or its order depends on are
// closer than the float32 error of c (and are not the same logit and bias), or a
// kept and a dropped group closer than theirs, is chosen again from scores in 64
// bits, by the same warp.
//
// Weights are computed from the chosen logits alone where norm is set, scaled
// by the largest of them (softmax) or by min(0, largest) (sigmoid), so that
// experts whose scores all underflow still share the token as they should.
//
// One warp per token; lane i holds experts [i PER, (i + 1) PER) in registers,
// so the lowest lane that holds a maximum holds the lowest id.  A pick is one
// integer max over the warp (redux) on order-preserving keys.  Bound by
// instruction issue (about 1200 a token with groups, bias and 256 experts, the
// compare and integer pipe first): 16384 tokens, 256 experts, sigmoid, bias, 4 of 8
// groups by their two best: 26 to 31 us a call (bf16 logits without a bias, whose
// exact ties at the k-th place go to 64 bits: 34); the gradient 9.4 us, where its
// bytes would take 2.8.
#pragma once

#include "common.cuh"

namespace nh {
namespace gate {

constexpr int WARPS = 8;
constexpr unsigned FULL = 0xffffffffu;

struct Args {
  const void* logits;     // [T, E] (float or bf16)
  const float* bias;      // [E] or null
  int32_t* idx;           // [T, k] out (forward), in (backward)
  float* w;               // [T, k] out (forward)
  const float* dw;        // [T, k] in (backward)
  void* dlogits;          // [T, E] out (backward), the logits' type
  int64_t T;
  int E, G, tg, k;
  int softmax, norm, top2;
  float alpha;
};

__device__ __forceinline__ float clean(float l) {
  // fmaxf drops a NaN; -0 becomes +0: they tie
  return fminf(fmaxf(l, -INFINITY), 3.402823466e38f) + 0.0f;
}

// order-preserving key of a float that is not NaN; 0 is below every key
__device__ __forceinline__ uint32_t key_of(float v) {
  const int u = __float_as_int(v);
  return (uint32_t)u ^ ((uint32_t)(u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
  return of_key(__reduce_max_sync(FULL, key_of(v)));
}

// Row values [lane PER, lane PER + PER), cleaned; -inf past E.  16-byte loads
// where rows and lanes start on them.
template <int PER>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float (&l)[PER]) {
  const int e0 = lane * PER;
  if (PER >= 4 && (E % 4) == 0) {
#pragma unroll
    for (int i = 0; i + 3 < PER; i += 4) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e0 + i < E) v = *reinterpret_cast<const float4*>(row + e0 + i);
      l[i] = clean(v.x);
      l[i + 1] = clean(v.y);
      l[i + 2] = clean(v.z);
      l[i + 3] = clean(v.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = e0 + i < E ? clean(row[e0 + i]) : -INFINITY;
  }
}

template <int PER>
__device__ __forceinline__ void load_row(const __nv_bfloat16* row, int E, int lane,
                                         float (&l)[PER]) {
  const int e0 = lane * PER;
  if (PER >= 4 && (E % 4) == 0) {
#pragma unroll
    for (int i = 0; i + 3 < PER; i += 4) {
      uint2 u = make_uint2(0xff80ff80u, 0xff80ff80u);   // -inf
      if (e0 + i < E) u = *reinterpret_cast<const uint2*>(row + e0 + i);
      l[i] = clean(__uint_as_float(u.x << 16));
      l[i + 1] = clean(__uint_as_float(u.x & 0xffff0000u));
      l[i + 2] = clean(__uint_as_float(u.y << 16));
      l[i + 3] = clean(__uint_as_float(u.y & 0xffff0000u));
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      l[i] = e0 + i < E ? clean(__bfloat162float(row[e0 + i])) : -INFINITY;
  }
}

template <int PER>
__device__ __forceinline__ void store_row(float* row, int E, int lane, const float (&v)[PER]) {
  const int e0 = lane * PER;
  if (PER >= 4 && (E % 4) == 0) {
#pragma unroll
    for (int i = 0; i + 3 < PER; i += 4)
      if (e0 + i < E)
        *reinterpret_cast<float4*>(row + e0 + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i < E) row[e0 + i] = v[i];
  }
}

template <int PER>
__device__ __forceinline__ void store_row(__nv_bfloat16* row, int E, int lane,
                                          const float (&v)[PER]) {
  const int e0 = lane * PER;
  if (PER >= 4 && (E % 4) == 0) {
#pragma unroll
    for (int i = 0; i + 3 < PER; i += 4)
      if (e0 + i < E)
        *reinterpret_cast<uint2*>(row + e0 + i) =
            make_uint2(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i < E) row[e0 + i] = __float2bfloat16_rn(v[i]);
  }
}

template <int PER>
__device__ __forceinline__ uint32_t max_key(const uint32_t (&key)[PER]) {
  uint32_t m = key[0];
#pragma unroll
  for (int i = 1; i < PER; i += 2)
    m = i + 1 < PER ? __vimax3_u32(m, key[i], key[i + 1]) : max(m, key[i]);
  return m;
}

// sigmoid without overflow or cancellation at either end
__device__ __forceinline__ float sigmoid(float l) {
  const float e = expf(-fabsf(l));
  return (l < 0.f ? e : 1.f) / (1.f + e);
}

// This lane's part of the chosen experts' summed score: lanes j < k hold their
// chosen logit l (-inf: cannot be taken, part 0), the others -inf.
__device__ __forceinline__ float share(float l, bool softmax) {
  float top = warp_max(l);
  if (top == -INFINITY) top = 0.f;
  float u;
  if (softmax) {
    u = expf(l - top);
  } else if (top > -80.f) {
    u = sigmoid(l);
  } else {   // all underflow, or nearly: e^-top sigmoid(l), where sigmoid(l) = e^l
    u = expf(l - top);
  }
  const float z = warp_sum(u);
  return z > 0.f ? u / z : 0.f;
}

// value of a pair (largest, second largest) as a group value
template <typename V>
__device__ __forceinline__ V group_value(V v1, V v2, bool top2) {
  return top2 && v2 != -INFINITY ? v1 + v2 : v1;
}

template <typename V>
__device__ __forceinline__ void top2_add(V v, V& v1, V& v2) {
  if (v > v1) {
    v2 = v1;
    v1 = v;
  } else if (v > v2) {
    v2 = v;
  }
}

// How far the exact value of a group may lie from its float32 value gs: tol_s for the
// scores, and half a unit in the last place of either c and of their sum, 2^-23 (|v1| +
// |v2|) together.  The sum of two of opposite sign is small where its error is not, so
// each group brings its own error, and a kept group is certain only if it stays above
// every dropped one.  2^-22 covers the rounding of gs +- e, too.  A group without a
// usable expert is exactly -inf; one past float32's range is never certain.
struct Reach {
  float lo, hi;
  __device__ __forceinline__ Reach(float gs, float v1, float v2, bool top2, float tol_s) {
    const float size = fabsf(v1) + (top2 && v2 != -INFINITY ? fabsf(v2) : 0.f);
    const float e = tol_s + 0x1p-22f * size;
    lo = gs - e;
    hi = gs + e;
    if (v1 == -INFINITY) {
      lo = INFINITY;
      hi = -INFINITY;
    } else if (!(size < INFINITY)) {
      lo = -INFINITY;
      hi = INFINITY;
    }
  }
};
// Is the lowest end of the kept groups (lo) not above the highest of the dropped (hi)?
__device__ __forceinline__ bool overlap(float kept_lo, float dropped_hi) {
  return !(-warp_max(-kept_lo) > warp_max(dropped_hi));
}

// Groups by value from shared memory, any group size: lane q reduces groups q
// and q + 32, starting at its own place in the group so that the lanes' reads
// spread over the banks.  Returns the kept groups as a mask; `close` (float)
// is set where a kept and a dropped group are within their errors (Reach).
template <typename V>
__device__ __forceinline__ uint64_t keep_groups(const V* c, int G, int g, int tg, bool top2,
                                                int lane, float tol_s, bool* close) {
  V gs[2], v1s[2], v2s[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int q = lane + 32 * r;
    V v1 = -INFINITY, v2 = -INFINITY;
    if (q < G)
      for (int i = 0, p = q % g; i < g; ++i) {
        top2_add(c[q * g + p], v1, v2);
        if (++p == g) p = 0;
      }
    gs[r] = group_value(v1, v2, top2);
    v1s[r] = v1;
    v2s[r] = v2;
  }
  int rank[2] = {0, 0};
  for (int q = 0; q < G; ++q) {
    const V o = __shfl_sync(FULL, q < 32 ? gs[0] : gs[1], q & 31);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int me = lane + 32 * r;
      rank[r] += (o > gs[r] || (o == gs[r] && q < me)) ? 1 : 0;
    }
  }
  uint64_t keep = 0;
#pragma unroll
  for (int r = 0; r < 2; ++r)
    keep |= (uint64_t)__ballot_sync(FULL, lane + 32 * r < G && rank[r] < tg) << (32 * r);
  if (close) {
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (lane + 32 * r >= G) continue;
      const Reach at((float)gs[r], (float)v1s[r], (float)v2s[r], top2, tol_s);
      if (rank[r] < tg)
        lo = fminf(lo, at.lo);
      else
        hi = fmaxf(hi, at.hi);
    }
    *close = overlap(lo, hi);
  }
  return keep;
}

// The choice from 64-bit scores (rare): writes pick j to lane j's `e`.
template <int PER, typename Tin>
__device__ __noinline__ int choose_f64(const Tin* row, const Args& a, double* c, int lane) {
  const int E = a.E, g = E / a.G, e0 = lane * PER;
  float l[PER];
  load_row<PER>(row, E, lane, l);
  double s[PER];
  if (a.softmax) {
    float mine = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) mine = fmaxf(mine, l[i]);
    float top = warp_max(mine);
    if (top == -INFINITY) top = 0.f;
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      s[i] = exp((double)l[i] - (double)top);
      z += s[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(FULL, z, o);
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = z > 0.0 ? s[i] / z : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
  }
  uint32_t live = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i;
    if (e < E) {
      s[i] = l[i] == -INFINITY ? -INFINITY : s[i] + (a.bias ? (double)a.bias[e] : 0.0);
      c[e] = s[i];
      live |= 1u << i;
    }
  }
  __syncwarp();
  if (a.tg < a.G) {
    const uint64_t keep = keep_groups<double>(c, a.G, g, a.tg, a.top2, lane, 0.f, nullptr);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i < E && !((keep >> ((e0 + i) / g)) & 1ull)) live &= ~(1u << i);
  }
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    double bv = 0.0;
    int be = -1;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (((live >> i) & 1u) && (be < 0 || s[i] > bv)) {
        bv = s[i];
        be = e0 + i;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(FULL, bv, o);
      const int oe = __shfl_xor_sync(FULL, be, o);
      if (oe >= 0 && (be < 0 || ov > bv || (ov == bv && oe < be))) {
        bv = ov;
        be = oe;
      }
    }
    const int i = be - e0;
    if (i >= 0 && i < PER) live &= ~(1u << i);
    if (lane == j) mine = be;
  }
  return mine;
}

// The keys that reach `floor_key`, with their experts, into cand (32 of them at
// most); returns how many there are.
template <int PER>
__device__ __forceinline__ int gather(const uint32_t (&key)[PER], uint32_t floor_key, int e0,
                                      int lane, uint2* cand) {
  int found = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const unsigned who = __ballot_sync(FULL, key[i] >= floor_key);
    if (key[i] >= floor_key) {
      const int at = found + __popc(who & ((1u << lane) - 1u));
      if (at < 32) cand[at] = make_uint2(key[i], (uint32_t)(e0 + i));
    }
    found += __popc(who);
  }
  return found;
}

// A few candidates in the order of their 64-bit scores, one to a lane: pick j to
// lane j.  A tenth of the time of choose_f64, whose lanes score all their experts
// one after the other.
template <int PER, typename Tin>
__device__ __noinline__ int order_f64(const Tin* row, const Args& a, const uint2* cand, int n,
                                      int lane) {
  double top = 0.0, z = 1.0;
  if (a.softmax) {
    float l[PER];
    load_row<PER>(row, a.E, lane, l);
    float mine = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) mine = fmaxf(mine, l[i]);
    const float t = warp_max(mine);
    top = t == -INFINITY ? 0.0 : (double)t;
    z = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) z += exp((double)l[i] - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(FULL, z, o);
  }
  int e = 0x7fffffff;
  double c = -INFINITY;
  if (lane < n) {
    e = (int)cand[lane].y;
    const double l = (double)clean(to_f32(row[e]));
    if (l != -INFINITY) {
      c = a.softmax ? exp(l - top) / z : 1.0 / (1.0 + exp(-l));
      if (a.bias) c += (double)a.bias[e];
    }
  }
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const double o = __shfl_sync(FULL, c, j);
    const int oe = __shfl_sync(FULL, e, j);
    rank += (o > c || (o == c && oe < e)) ? 1 : 0;
  }
  int mine = 0;
  for (int j = 0; j < n; ++j) {
    const int r = __shfl_sync(FULL, rank, j), oe = __shfl_sync(FULL, e, j);
    if (r == lane) mine = oe;
  }
  return mine;
}

template <int PER, typename Tin>
__global__ void __launch_bounds__(WARPS * 32, PER <= 8 ? 5 : 3) gate_forward(const Args a) {
  extern __shared__ double smem[];   // [WARPS][E]
  __shared__ uint2 cand[WARPS][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x * (int64_t)WARPS + warp;
  if (t >= a.T) return;
  const int E = a.E, g = E / a.G, k = a.k, e0 = lane * PER;
  const Tin* row = static_cast<const Tin*>(a.logits) + t * E;
  float l[PER];
  load_row<PER>(row, E, lane, l);

  const bool grouped = a.tg < a.G;
  const bool by_score = a.bias != nullptr || (grouped && a.top2);
  float top = 0.f, z = 1.f;      // of the softmax over all experts
  if (a.softmax && (by_score || !a.norm)) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = fmaxf(m, l[i]);
    top = warp_max(m);
    if (top == -INFINITY) top = 0.f;
    float p = 0.f;
    if (a.norm) {
#pragma unroll
      for (int i = 0; i < PER; ++i) p += __expf(l[i] - top);
    } else {   // z is part of the weights too
#pragma unroll
      for (int i = 0; i < PER; ++i) p += expf(l[i] - top);
    }
    z = warp_sum(p);
    if (z == 0.f) z = 1.f;
  }
  float c[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) c[i] = l[i];
  if (by_score) {
    // Scores that only choose: the approximate exponential and divide, 2 + 1.2
    // |x| and 2 units in the last place (their documented bounds), a third of the
    // instructions.
    if (a.softmax) {
      const float iz = 1.f / z;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (l[i] != -INFINITY) c[i] = __expf(l[i] - top) * iz;
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (l[i] != -INFINITY) c[i] = __fdividef(1.f, 1.f + __expf(-fmaxf(l[i], -80.f)));
    }
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (l[i] != -INFINITY) c[i] += a.bias[e0 + i];   // past E, too, l is -inf
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] += 0.0f;
  }
  // Twice the error of a score, in u = 2^-24.  sigmoid, e = exp(-l): s (1 - s) <=
  // 1/4 of e's 4 + 2.4 |l| (s (1 - s) |l| <= 0.23: under 1.6 together), the add 1,
  // the divide 4: under 7.  softmax, of a value <= 1 / z: e^-d (4 + 2.4 d) <= 4,
  // the rounding of l - top under 1, z's terms under 12 (512 of them at the d that
  // counts most) and its PER + 5 adds, two roundings: under PER + 24.  The add of
  // the bias is counted at the comparison.
  const float tol_s = a.softmax ? (PER + 14) * 0x1p-22f / z : 0x1p-20f;
  bool again = false;

  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = e0 + i < E ? key_of(c[i]) : 0u;
  if (grouped) {
    const int width = g / PER;
    bool close = false;
    if (g % PER == 0 && (width & (width - 1)) == 0) {
      // a group is `width` whole lanes: its two largest by a butterfly
      float v1 = -INFINITY, v2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < PER; ++i) top2_add(c[i], v1, v2);
      for (int o = 1; o < width; o <<= 1) {
        const float o1 = __shfl_xor_sync(FULL, v1, o), o2 = __shfl_xor_sync(FULL, v2, o);
        v2 = fmaxf(fminf(v1, o1), fmaxf(v2, o2));
        v1 = fmaxf(v1, o1);
      }
      const float gs = group_value(v1, v2, a.top2);
      const int me = lane / width;
      int rank = 0;
      for (int q = 0; q < a.G; ++q) {
        const float o = __shfl_sync(FULL, gs, q * width);
        rank += (o > gs || (o == gs && q < me)) ? 1 : 0;
      }
      if (by_score) {
        const Reach at(gs, v1, v2, a.top2, tol_s);
        close = overlap(me < a.G && rank < a.tg ? at.lo : INFINITY,
                        me < a.G && rank >= a.tg ? at.hi : -INFINITY);
      }
      if (rank >= a.tg) {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = 0u;
      }
    } else {
      float* cs = reinterpret_cast<float*>(smem + (size_t)warp * E);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e0 + i < E) cs[e0 + i] = c[i];
      __syncwarp();
      const uint64_t keep =
          keep_groups<float>(cs, a.G, g, a.tg, a.top2, lane, tol_s, by_score ? &close : nullptr);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e0 + i < E && !((keep >> ((e0 + i) / g)) & 1ull)) key[i] = 0u;
    }
    again = close;
  }

  // the k best, lane j the j-th; with scores one more, whose distance counts
  int my_e = 0;
  uint32_t my_key = 0u, next_key = 0u;
  const int rounds = by_score ? k + 1 : k;
  uint32_t best = max_key<PER>(key);
  // Every one of the `rounds` best is at least the rounds-th largest of the lanes'
  // best keys.  The few keys that are (11 of 256 at 9 rounds) go to shared memory,
  // one to a lane, and each counts those before it: 150 instructions where one
  // maximum after the other takes 50 a round.
  uint32_t floor_key = 0u, left = best;
  for (int j = 0; j < rounds; ++j) {     // lanes with equal keys fall together: a lower floor
    floor_key = __reduce_max_sync(FULL, left);
    if (left == floor_key) left = 0u;
  }
  floor_key = max(floor_key, 1u);
  const int found = gather<PER>(key, floor_key, e0, lane, cand[warp]);
  const bool ranked = found <= 32 && rounds <= 32;
  if (ranked) {
    __syncwarp();
    const uint2 me = lane < found ? cand[warp][lane] : make_uint2(0u, 0u);
    int rank = 0;
    for (int j = 0; j < found; ++j) {
      const uint2 o = cand[warp][j];
      rank += (o.x > me.x || (o.x == me.x && o.y < me.y)) ? 1 : 0;
    }
    __syncwarp();
    if (lane < found && rank < rounds) cand[warp][rank] = me;
    __syncwarp();
    if (lane < min(found, rounds)) {
      my_key = cand[warp][lane].x;
      my_e = (int)cand[warp][lane].y;
    }
  } else {
    // many equal keys, few lanes with many kept experts, or k = 32
    for (int j = 0; j < rounds; ++j) {
      const uint32_t m = __reduce_max_sync(FULL, best);
      const int src = __ffs(__ballot_sync(FULL, best == m)) - 1;
      int e = 0;
      if (lane == src) {
        // the first of this lane's keys that is the maximum goes out of the race
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (key[i] == m) {
            key[i] = 0u;
            e = e0 + i;
            break;
          }
        best = max_key<PER>(key);
      }
      e = __shfl_sync(FULL, e, src);
      if (lane == j) {
        my_e = e;
        my_key = m;
      }
      if (j == 32) next_key = m;   // the runner-up at k = 32, which no lane holds
    }
  }
  const auto logit_of = [&](int e) { return clean(to_f32(row[e])); };
  if (by_score) {
    // neighbours closer than the error of their scores, and not equal inputs
    const float mine = of_key(my_key);
    const float l_me = lane <= k ? logit_of(my_e) : 0.f;
    const float b_me = lane <= k && a.bias ? a.bias[my_e] : 0.f;
    uint32_t after = __shfl_down_sync(FULL, my_key, 1);
    const float l_after = __shfl_down_sync(FULL, l_me, 1);
    const float b_after = __shfl_down_sync(FULL, b_me, 1);
    // equal inputs tie exactly and stay in id order; at the end of the k best
    // they do not count as such, since what comes after the runner-up is not seen
    const bool same = lane < k - 1 && l_me == l_after && b_me == b_after;
    if (lane == 31) after = next_key;
    const bool near = lane < k && after != 0u && !same && mine != -INFINITY &&
                      mine - of_key(after) <= tol_s + 0x1p-22f * fabsf(mine);
    const bool unsure = __any_sync(FULL, near);
    if (again || (unsure && !ranked)) {
      my_e = choose_f64<PER>(row, a, smem + (size_t)warp * E, lane);
    } else if (unsure) {
      // the groups are certain: whatever may be among the k best is within the
      // errors of the k-th
      const float last = of_key(__shfl_sync(FULL, my_key, k - 1));
      const float floor_c = last - (tol_s + 0x1p-22f * fabsf(last));
      __syncwarp();
      const int some = gather<PER>(key, max(key_of(floor_c), 1u), e0, lane, cand[warp]);
      __syncwarp();
      my_e = some >= k && some <= 32 ? order_f64<PER>(row, a, cand[warp], some, lane)
                                     : choose_f64<PER>(row, a, smem + (size_t)warp * E, lane);
    }
  }
  const float lj = lane < k ? logit_of(my_e) : -INFINITY;
  float wj;
  if (a.norm)
    wj = share(lj, a.softmax != 0);
  else
    wj = a.softmax ? expf(lj - top) / z : sigmoid(lj);
  if (lane < k) {
    a.idx[t * k + lane] = my_e;
    a.w[t * k + lane] = a.alpha * wj;
  }
}

// d logits from d weights.  With p_j the shares of the chosen experts, s the scores,
// and for raw softmax r the summed score of the experts not chosen:
//   norm, softmax   dl_j = alpha p_j sum_i p_i (dw_j - dw_i)
//   norm, sigmoid   the same times (1 - s_j)
//   raw,  sigmoid   dl_j = alpha dw_j s_j (1 - s_j)
//   raw,  softmax   dl_j = alpha s_j (r dw_j + sum_i s_i (dw_j - dw_i)), j chosen
//                   dl_n = -alpha s_n sum_i s_i dw_i, the others
// (from dw = alpha d(s_j / sum s): d log p_j = d log s_j - sum p d log s).  The sums
// over differences are dw_j - sum p dw and dw_j - sum s dw without their cancellation:
// where one expert has nearly all of the weight, those lose every digit of its
// gradient.  An expert named twice gets both parts, in slot order (with raw softmax its
// dw are summed first); an id outside [0, E) takes no part.  One write of each row, and
// its read only for raw softmax.
template <int PER, typename Tin>
__global__ void __launch_bounds__(WARPS * 32) gate_backward(const Args a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x * (int64_t)WARPS + warp;
  if (t >= a.T) return;
  const int E = a.E, k = a.k, e0 = lane * PER;
  const Tin* row = static_cast<const Tin*>(a.logits) + t * E;
  int e = -1;
  float dw = 0.f, lj = -INFINITY;
  if (lane < k) {
    e = a.idx[t * k + lane];
    if (e >= 0 && e < E) {
      dw = a.dw[t * k + lane];
      lj = clean(to_f32(row[e]));
    } else {
      e = -1;
    }
  }
  float out[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) out[i] = 0.f;
  float d;
  if (a.norm) {
    const float p = share(lj, a.softmax != 0);
    float sum = 0.f;
    for (int j = 0; j < k; ++j)
      sum = fmaf(__shfl_sync(FULL, p, j), dw - __shfl_sync(FULL, dw, j), sum);
    d = a.alpha * p * sum;
    if (!a.softmax) d *= sigmoid(-lj);
  } else if (!a.softmax) {
    d = a.alpha * dw * sigmoid(lj) * sigmoid(-lj);
  } else {
    float l[PER];
    load_row<PER>(row, E, lane, l);
    float m = l[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) m = fmaxf(m, l[i]);
    float top = warp_max(m);
    if (top == -INFINITY) top = 0.f;
    // slots of the same expert are one, the first of them
    uint32_t chosen = 0;
    float w = 0.f;
    bool first = e >= 0;
    for (int j = 0; j < k; ++j) {
      const int ej = __shfl_sync(FULL, e, j);
      const float dwj = __shfl_sync(FULL, dw, j);
      if (ej == e) {
        w += dwj;
        first = first && j >= lane;
      }
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (e0 + i == ej) chosen |= 1u << i;
    }
    float p = 0.f, others = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      out[i] = expf(l[i] - top);
      p += out[i];
      if (!((chosen >> i) & 1u)) others += out[i];
    }
    float z = warp_sum(p);
    if (z == 0.f) z = 1.f;
    const float r = warp_sum(others) / z;
    const float s = first ? expf(lj - top) / z : 0.f;
    float sum = r * w, all = 0.f;
    for (int j = 0; j < k; ++j) {
      const float sj = __shfl_sync(FULL, s, j), wj = __shfl_sync(FULL, w, j);
      sum = fmaf(sj, w - wj, sum);
      all = fmaf(sj, wj, all);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      out[i] = (chosen >> i) & 1u ? 0.f : -a.alpha * (out[i] / z) * all;
    d = a.alpha * s * sum;
  }
  for (int j = 0; j < k; ++j) {
    const int ej = __shfl_sync(FULL, e, j);
    const float dj = __shfl_sync(FULL, d, j);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e0 + i == ej) out[i] += dj;
  }
  store_row<PER>(static_cast<Tin*>(a.dlogits) + t * E, E, lane, out);
}

}  // namespace gate
}  // namespace nh
