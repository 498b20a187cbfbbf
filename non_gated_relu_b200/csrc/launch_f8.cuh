// launch_f8.cuh -- host side of the FP8 operators: tensor maps, kernel choice
// and launches.  Part of nh_moe.cu (inside namespace nh).

// uint8 [rows, row_bytes], box 128 bytes x box_rows, 128-byte swizzle
static nh_status map_u8_2d(CUtensorMap* m, const void* base, int64_t row_bytes, int64_t rows,
                           int box_rows) {
  auto fn = encode_fn();
  if (!fn) return fail(NH_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[2] = {(cuuint64_t)row_bytes, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  cuuint32_t box[2] = {(cuuint32_t)f8g::BK, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
                  es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(NH_ERR_CUDA, "cuTensorMapEncodeTiled (u8 2d) failed: %d", (int)r);
  return NH_OK;
}

static nh_status check_f8(const nh_fp8_weight* w, const char* name) {
  if (!w) return fail(NH_ERR_INVALID_ARG, "%s is NULL", name);
  NH_TRY(check_ptr(w->codes, name));
  return check_ptr(w->scales, name);
}

// One product: out = outkind(x W[e]^T) over tile entries or dense rows.
enum F8Out { F8_BF16, F8_F32, F8_RELU2, F8_ADD };
struct F8Call {
  const uint8_t* x;          // codes [x_rows, K]
  const float* xs;
  int64_t x_rows;
  const nh_fp8_weight* w;    // [n_exp, N, K]
  int n_exp;
  int64_t rows;              // output rows
  int N, K;
  const int4* tiles;
  const int32_t* num_tiles;
  int max_tiles;
  int tile_rows;             // of tile entries: below 256 with the weights on the M side
  F8Out out_kind;
  void* out;                 // F8_RELU2: codes, or float32 from the GEMV
  float* out_scales;         // F8_RELU2: their scales (not the GEMV)
  int* status;
  bool early_w;
};

// x: null for the call's codes, else values of x_type (at most F8_RAW_ROWS rows)
static nh_status launch_f8_gemv(const F8Call& c, cudaStream_t st, const void* x = nullptr,
                                bool x_bf16 = false) {
  f8v::Args a{};
  a.x = x ? x : c.x;
  a.xs = c.xs;
  a.w = c.w->codes;
  a.ws = c.w->scales;
  a.rows = (int)c.rows;
  a.N = c.N;
  a.K = c.K;
  a.KB = (int)f8_blocks(c.K);
  switch (c.out_kind) {
    case F8_BF16: a.out_kind = f8v::OUT_BF16; break;
    case F8_F32: a.out_kind = f8v::OUT_F32; break;
    case F8_RELU2: a.out_kind = f8v::OUT_RELU2_F32; break;
    default: a.out_kind = f8v::OUT_ADD_F32;
  }
  a.out = c.out;
  a.early_w = c.early_w ? 1 : 0;
  const dim3 g((unsigned)(c.N / f8v::MT)), b(f8v::WARPS * 32);
  if (x && x_bf16) return launch_k("f8_gemv", f8v::f8_gemv<8, 3, __nv_bfloat16>, g, b, 0, st, a);
  if (x) return launch_k("f8_gemv", f8v::f8_gemv<8, 3, float>, g, b, 0, st, a);
  if (c.rows <= 16) return launch_k("f8_gemv", f8v::f8_gemv<16, 2, uint8_t>, g, b, 0, st, a);
  return launch_k("f8_gemv", f8v::f8_gemv<32, 2, uint8_t>, g, b, 0, st, a);
}

// products with weights on the MMA M side
template <int NT, int STAGES, int CTAS>
static nh_status launch_f8_swap_as(const F8Call& c, int dev, cudaStream_t st) {
  using S = f8s::Shape<NT, STAGES, CTAS>;
  CUtensorMap mx, mw;
  NH_TRY(map_u8_2d(&mx, c.x, c.K, c.x_rows, NT));
  NH_TRY(map_u8_3d(&mw, c.w->codes, c.K, c.N, c.n_exp, f8s::BK, true));
  f8s::Args a{};
  a.xs = c.xs;
  a.ws = c.w->scales;
  a.tiles = c.tiles;
  a.num_tiles = c.num_tiles;
  a.dense_rows = (int)c.rows;
  a.N = c.N;
  a.K = c.K;
  a.KB = (int)f8_blocks(c.K);
  a.out = c.out;
  a.out_scales = c.out_scales;
  a.status = c.status;
  a.timeout_ns = timeout_ns();
  a.early_w = c.early_w ? 1 : 0;
  // an entry holds at least one row
  const int64_t m = c.tiles ? std::min<int64_t>(c.max_tiles, c.rows) : (c.rows + NT - 1) / NT;
  const int64_t tiles = m * ((c.N + f8s::M - 1) / f8s::M);
  const dim3 grid((unsigned)std::min<int64_t>(tiles, (int64_t)g_sm_count[dev] * CTAS));
  if (c.out_kind == F8_RELU2)
    return launch_k("f8_swap_gemm", f8s::f8_swap_gemm<NT, STAGES, CTAS, f8s::OUT_RELU2_F8>, grid,
                    dim3(f8s::THREADS), S::SMEM, st, mx, mw, a);
  if (c.out_kind == F8_F32)
    return launch_k("f8_swap_gemm", f8s::f8_swap_gemm<NT, STAGES, CTAS, f8s::OUT_F32>, grid,
                    dim3(f8s::THREADS), S::SMEM, st, mx, mw, a);
  if constexpr (NT == F8_DENSE_NT) {
    if (c.out_kind == F8_BF16)
      return launch_k("f8_swap_gemm", f8s::f8_swap_gemm<NT, STAGES, CTAS, f8s::OUT_BF16>, grid,
                      dim3(f8s::THREADS), S::SMEM, st, mx, mw, a);
    return launch_k("f8_swap_gemm", f8s::f8_swap_gemm<NT, STAGES, CTAS, f8s::OUT_ADD_F32>, grid,
                    dim3(f8s::THREADS), S::SMEM, st, mx, mw, a);
  }
  return fail(NH_ERR_UNSUPPORTED, "internal: dense rows take tiles of %d", F8_DENSE_NT);
}

static nh_status launch_f8_swap(const F8Call& c, int dev, cudaStream_t st) {
  switch (c.tile_rows) {
    case 16: return launch_f8_swap_as<16, 5, 2>(c, dev, st);
    case 32: return launch_f8_swap_as<32, 5, 2>(c, dev, st);
    default: return launch_f8_swap_as<64, 4, 2>(c, dev, st);
  }
}

template <int OUT>
static nh_status launch_f8_pair_as(const F8Call& c, const f8g::Args& a, int64_t tiles, int dev,
                                   cudaStream_t st) {
  CUtensorMap mx, mw;
  NH_TRY(map_u8_2d(&mx, c.x, c.K, c.x_rows, f8g::HALF));
  NH_TRY(map_u8_3d(&mw, c.w->codes, c.K, c.N, c.n_exp, f8g::BK, true));
  const int64_t pairs = std::min<int64_t>(tiles, g_f8_clusters[dev]);
  if (pairs <= 0) return NH_OK;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
  lc.blockDim = dim3(f8g::THREADS, 1, 1);
  lc.dynamicSmemBytes = f8g::SMEM;
  lc.stream = st;
  cudaLaunchAttribute at[3];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  at[2].id = cudaLaunchAttributePriority;
  at[2].val.priority = stream_priority(st);
  lc.attrs = at;
  lc.numAttrs = 3;
  NH_CUDA(cudaLaunchKernelEx(&lc, f8g::f8_pair_gemm<OUT>, mx, mw, a));
  return launch_check("f8_pair_gemm");
}

static nh_status launch_f8_pair(const F8Call& c, int dev, cudaStream_t st) {
  f8g::Args a{};
  a.xs = c.xs;
  a.ws = c.w->scales;
  a.tiles = c.tiles;
  a.num_tiles = c.num_tiles;
  a.dense_rows = (int)c.rows;
  a.N = c.N;
  a.K = c.K;
  a.KB = (int)f8_blocks(c.K);
  a.out = c.out;
  a.out_scales = c.out_scales;
  a.ldo = c.N;
  a.status = c.status;
  a.timeout_ns = timeout_ns();
  const int64_t m = c.tiles ? c.max_tiles : (c.rows + f8g::MP - 1) / f8g::MP;
  const int64_t tiles = m * ((c.N + f8g::NT - 1) / f8g::NT);
  switch (c.out_kind) {
    case F8_BF16: return launch_f8_pair_as<f8g::OUT_BF16>(c, a, tiles, dev, st);
    case F8_F32: return launch_f8_pair_as<f8g::OUT_F32>(c, a, tiles, dev, st);
    case F8_RELU2: return launch_f8_pair_as<f8g::OUT_RELU2_F8>(c, a, tiles, dev, st);
    default: return launch_f8_pair_as<f8g::OUT_ADD_F32>(c, a, tiles, dev, st);
  }
}

static bool f8_gemv_rows(const F8Call& c) { return !c.tiles && c.rows <= F8_GEMV_ROWS; }

static nh_status run_f8(const F8Call& c, int dev, cudaStream_t st) {
  if (c.rows == 0) return NH_OK;
  if (c.tiles && c.tile_rows < f8g::MP) return launch_f8_swap(c, dev, st);
  if (f8_gemv_rows(c)) return launch_f8_gemv(c, st);
  // Few rows: tiles of 128 features x 64 rows while each SM gets one at most, where
  // 256 x 256 tiles leave most SMs without.  Measured in a graph with the
  // quantization, these against those: N 3712, K 2688: 11.5 and 14.4 us for 64 rows,
  // 12.8 and 15.3 for 320 (145 tiles), and 16.6 against 16.1 for 448 (203); N 512, K
  // 4096, 100 rows: 16.4 and 18.9.
  const int64_t small = (c.rows + F8_DENSE_NT - 1) / F8_DENSE_NT * ((c.N + f8s::M - 1) / f8s::M);
  if (!c.tiles && small <= g_sm_count[dev]) return launch_f8_swap_as<F8_DENSE_NT, 4, 2>(c, dev, st);
  return launch_f8_pair(c, dev, st);
}

// Quantize R rows of C values; with inv_row each to its k permuted rows.
template <typename Tin>
static nh_status launch_quantize(const Tin* x, int64_t R, int C, uint8_t* codes, float* scales,
                                 const int32_t* inv_row, int k, cudaStream_t st) {
  const int64_t kb = f8_blocks(C), units = R * kb;
  if (units == 0) return NH_OK;
  if (units > 0x7fffffff) return fail(NH_ERR_UNSUPPORTED, "quantization of %lld blocks", (long long)units);
  return launch_k("quantize_rows", f8::quantize_rows<Tin>, dim3((unsigned)((units + 31) / 32)),
                  dim3(256), 0, st, x, (uint32_t)units, C, (int)kb, codes, scales, inv_row, k);
}

// Dense rows that a kernel left in float32 behind their quantized form
// (f8_hidden_bytes): where the GEMV writes its squared relu, or codes directly
struct F8Hidden {
  uint8_t* codes;
  float* scales;
  float* f32;
};
static F8Hidden f8_hidden(void* base, int64_t R, int64_t C) {
  char* b = static_cast<char*>(base);
  return {reinterpret_cast<uint8_t*>(b), reinterpret_cast<float*>(b + f8_scales_at(R, C)),
          reinterpret_cast<float*>(b + f8_rows_bytes(R, C))};
}

// Rows of the down projection, weighted and summed per token, into y_acc.
static nh_status launch_combine(const float* rows, const int32_t* inv_row, const float* perm_w,
                                int64_t T, int k, int H, float* y_acc, cudaStream_t st) {
  const int quads = H / 4;                        // H is a multiple of 64
  const int parts = (quads + 255) / 256;          // blocks of a token
  const int threads = ((quads + parts - 1) / parts + 31) / 32 * 32;
  if (T > 0x7fffffff / parts)
    return fail(NH_ERR_UNSUPPORTED, "combine of %lld tokens", (long long)T);
  return launch_k("combine_rows", f8::combine_rows, dim3((unsigned)(T * parts)), dim3(threads), 0, st,
                  rows, inv_row, perm_w, parts, k, quads, y_acc);
}

// A dense product of unquantized rows: in one launch up to F8_RAW_ROWS of them,
// else quantized to xq, xs first.  early_raw: the previous launch in the stream
// belongs to the same call.
static nh_status run_f8_dense(F8Call c, const void* x, bool bf16, uint8_t* xq, float* xs,
                              bool early_raw, int dev, cudaStream_t st) {
  if (c.rows <= F8_RAW_ROWS) {
    c.early_w = early_raw;
    return launch_f8_gemv(c, st, x, bf16);
  }
  if (bf16)
    NH_TRY(launch_quantize(static_cast<const __nv_bfloat16*>(x), c.rows, c.K, xq, xs, nullptr, 0, st));
  else
    NH_TRY(launch_quantize(static_cast<const float*>(x), c.rows, c.K, xq, xs, nullptr, 0, st));
  c.x = xq;
  c.xs = xs;
  c.x_rows = c.rows;
  c.early_w = true;
  return run_f8(c, dev, st);
}
