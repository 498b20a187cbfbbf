// api_f8.cuh -- C ABI of the FP8 operators.  Part of nh_moe.cu (inside extern "C").

static nh_status check_f8_dims(int64_t rows, int64_t cols, const char* what) {
  if (rows < 0 || cols < 1) return fail(NH_ERR_INVALID_ARG, "%s: sizes must be positive", what);
  if (cols % 16) return fail(NH_ERR_UNSUPPORTED, "%s: needs a multiple of 16 features", what);
  if (rows >= (int64_t(1) << 31) - 4096 || cols >= int64_t(1) << 30)
    return fail(NH_ERR_UNSUPPORTED, "%s: too large", what);
  return NH_OK;
}

nh_status nh_fp8_quantize(int64_t T, int64_t K, const void* x, int32_t dtype, uint8_t* codes,
                          float* scales, void* stream) {
  NH_TRY(check_f8_dims(T, K, "nh_fp8_quantize"));
  if (dtype != NH_F32 && dtype != NH_BF16) return fail(NH_ERR_INVALID_ARG, "unknown dtype");
  if (T == 0) return NH_OK;
  NH_TRY(check_ptr(x, "x"));
  NH_TRY(check_ptr(codes, "codes"));
  NH_TRY(check_ptr(scales, "scales"));
  int dev;
  NH_TRY(device_setup(&dev));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == NH_BF16)
    return launch_quantize(static_cast<const __nv_bfloat16*>(x), T, (int)K, codes, scales, nullptr, 0,
                           st);
  return launch_quantize(static_cast<const float*>(x), T, (int)K, codes, scales, nullptr, 0, st);
}

nh_status nh_fp8_quantize_weight(int64_t n_mat, int64_t rows, int64_t cols, const void* w,
                                 int32_t dtype, uint8_t* codes, float* scales, void* stream) {
  NH_TRY(check_f8_dims(rows, cols, "nh_fp8_quantize_weight"));
  if (n_mat < 0) return fail(NH_ERR_INVALID_ARG, "n_mat must be >= 0");
  if (dtype != NH_F32 && dtype != NH_BF16) return fail(NH_ERR_INVALID_ARG, "unknown dtype");
  const int64_t rb = f8_blocks(rows), cb = f8_blocks(cols);
  if (n_mat == 0 || rows == 0) return NH_OK;
  if (rb * cb > 0x7fffffff / n_mat)
    return fail(NH_ERR_UNSUPPORTED, "nh_fp8_quantize_weight: too many blocks");
  NH_TRY(check_ptr(w, "w"));
  NH_TRY(check_ptr(codes, "codes"));
  NH_TRY(check_ptr(scales, "scales"));
  int dev;
  NH_TRY(device_setup(&dev));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)(n_mat * rb * cb));
  if (dtype == NH_BF16)
    return launch_k("quantize_blocks", f8::quantize_blocks<__nv_bfloat16>, grid, dim3(256), 0, st,
                    static_cast<const __nv_bfloat16*>(w), (int)rows, (int)cols, (int)rb, (int)cb,
                    codes, scales);
  return launch_k("quantize_blocks", f8::quantize_blocks<float>, grid, dim3(256), 0, st,
                  static_cast<const float*>(w), (int)rows, (int)cols, (int)rb, (int)cb, codes, scales);
}

nh_status nh_fp8_linear_workspace_size(int64_t T, int64_t N, int64_t K, size_t* bytes) {
  if (!bytes) return fail(NH_ERR_INVALID_ARG, "bytes is NULL");
  NH_TRY(check_f8_dims(T, K, "nh_fp8_linear"));
  NH_TRY(check_f8_dims(0, N, "nh_fp8_linear"));
  *bytes = ALIGN + f8_rows_bytes(T, K);
  return NH_OK;
}

nh_status nh_fp8_linear(int64_t T, int64_t N, int64_t K, const void* x, int32_t x_dtype,
                        const nh_fp8_weight* w, void* y, int32_t y_dtype, void* ws, size_t ws_bytes,
                        void* stream) {
  size_t need;
  NH_TRY(nh_fp8_linear_workspace_size(T, N, K, &need));
  if ((x_dtype != NH_F32 && x_dtype != NH_BF16) || (y_dtype != NH_F32 && y_dtype != NH_BF16))
    return fail(NH_ERR_INVALID_ARG, "unknown dtype");
  NH_TRY(check_ptr(ws, "ws"));
  if (reinterpret_cast<uintptr_t>(ws) % ALIGN)
    return fail(NH_ERR_INVALID_ARG, "ws must be %zu-byte aligned", ALIGN);
  if (ws_bytes < need)
    return fail(NH_ERR_INVALID_ARG, "ws holds %zu bytes, %zu needed", ws_bytes, need);
  if (T == 0) return NH_OK;
  NH_TRY(check_ptr(x, "x"));
  NH_TRY(check_f8(w, "w"));
  NH_TRY(check_ptr(y, "y"));
  int dev;
  NH_TRY(f8_device_setup(&dev));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* xq = at<uint8_t>(ws, ALIGN);
  float* xs = at<float>(ws, ALIGN + f8_scales_at(T, K));
  F8Call c{};
  c.w = w;
  c.n_exp = 1;
  c.rows = T;
  c.N = (int)N;
  c.K = (int)K;
  c.out_kind = y_dtype == NH_BF16 ? F8_BF16 : F8_F32;
  c.out = y;
  c.status = static_cast<int*>(ws);
  return run_f8_dense(c, x, x_dtype == NH_BF16, xq, xs, false, dev, st);
}

// The two projections of the routed experts on the workspace.  `follows`: the
// previous launch in the stream belongs to the same call.
static nh_status f8_experts_up(const Plan& p, int64_t T, const void* x, const nh_fp8_weight* w,
                               void* ws, int dev, cudaStream_t st) {
  const nh_moe_ws_layout& L = p.lay;
  uint8_t* xq = at<uint8_t>(ws, L.x_perm);
  float* xs = at<float>(ws, L.x_perm + f8_scales_at(p.rows, p.H));
  NH_TRY(launch_quantize(static_cast<const __nv_bfloat16*>(x), T, p.H, xq, xs,
                         at<int32_t>(ws, L.inv_row), p.k, st));
  F8Call c{};
  c.x = xq;
  c.xs = xs;
  c.x_rows = p.rows;
  c.w = w;
  c.n_exp = p.E;
  c.rows = p.rows;
  c.N = p.I;
  c.K = p.H;
  c.tiles = at<int4>(ws, L.tiles);
  c.num_tiles = at<int32_t>(ws, L.num_tiles);
  c.max_tiles = L.max_tiles;
  c.tile_rows = L.tile_rows;
  c.status = at<int>(ws, L.status);
  c.early_w = true;   // the launch before is this call's quantization
  const F8Hidden h = f8_hidden(at<void>(ws, L.h), p.rows, p.I);
  c.out_kind = F8_RELU2;
  c.out = h.codes;
  c.out_scales = h.scales;
  return run_f8(c, dev, st);
}

static nh_status f8_experts_down(const Plan& p, int64_t T, const nh_fp8_weight* w, void* ws,
                                 float* y_acc, bool follows, int dev, cudaStream_t st) {
  const nh_moe_ws_layout& L = p.lay;
  const F8Hidden h = f8_hidden(at<void>(ws, L.h), p.rows, p.I);
  F8Call c{};
  c.x = h.codes;
  c.xs = h.scales;
  c.x_rows = p.rows;
  c.w = w;
  c.n_exp = p.E;
  c.rows = p.rows;
  c.N = p.H;
  c.K = p.I;
  c.tiles = at<int4>(ws, L.tiles);
  c.num_tiles = at<int32_t>(ws, L.num_tiles);
  c.max_tiles = L.max_tiles;
  c.tile_rows = L.tile_rows;
  float* rows = at<float>(ws, f8_down_rows_at(p));
  c.out_kind = F8_F32;
  c.out = rows;
  c.status = at<int>(ws, L.status);
  c.early_w = follows;
  NH_TRY(run_f8(c, dev, st));
  return launch_combine(rows, at<int32_t>(ws, L.inv_row), at<float>(ws, L.perm_w), T, p.k, p.H,
                        y_acc, st);
}

static nh_status f8_experts(const nh_moe_config* cfg, int64_t T, const void* x,
                            const nh_fp8_weight* w_up, const nh_fp8_weight* w_down, void* ws,
                            size_t ws_bytes, float* y_acc, void* stream, bool up, bool down) {
  NH_TRY(no_latent(cfg, "routed experts"));
  Plan p;
  NH_TRY(make_plan(cfg, T, &p));
  if (cfg->weight_format != NH_WEIGHTS_FP8)
    return fail(NH_ERR_INVALID_ARG, "config has no FP8 weights (weight_format)");
  NH_TRY(check_ws(p, ws, ws_bytes));
  if (up) NH_TRY(check_f8(w_up, "w_up"));
  if (down) NH_TRY(check_f8(w_down, "w_down"));
  if (T == 0) return NH_OK;
  if (up) NH_TRY(check_ptr(x, "x"));
  if (down) NH_TRY(check_ptr(y_acc, "y_acc"));
  int dev;
  NH_TRY(f8_device_setup(&dev));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (up) NH_TRY(f8_experts_up(p, T, x, w_up, ws, dev, st));
  if (down) NH_TRY(f8_experts_down(p, T, w_down, ws, y_acc, up, dev, st));
  return NH_OK;
}

nh_status nh_moe_experts_up_fp8(const nh_moe_config* cfg, int64_t T, const void* x,
                                const nh_fp8_weight* w_up, void* ws, size_t ws_bytes,
                                void* stream) {
  return f8_experts(cfg, T, x, w_up, nullptr, ws, ws_bytes, nullptr, stream, true, false);
}

nh_status nh_moe_experts_down_fp8(const nh_moe_config* cfg, int64_t T, const nh_fp8_weight* w_down,
                                  void* ws, size_t ws_bytes, float* y_acc, void* stream) {
  return f8_experts(cfg, T, nullptr, nullptr, w_down, ws, ws_bytes, y_acc, stream, false, true);
}

nh_status nh_moe_forward_fp8(const nh_moe_config* cfg, int64_t T, const void* x,
                             const nh_fp8_weight* w_up, const nh_fp8_weight* w_down, void* ws,
                             size_t ws_bytes, float* y_acc, void* stream) {
  return f8_experts(cfg, T, x, w_up, w_down, ws, ws_bytes, y_acc, stream, true, true);
}

static nh_status f8_shared(const nh_moe_config* cfg, int64_t T, const void* x,
                           const nh_fp8_weight* w_su, const nh_fp8_weight* w_sd, float* y_acc,
                           void* ws, size_t ws_bytes, void* stream, bool store) {
  size_t need;
  NH_TRY(nh_moe_shared_workspace_size(cfg, T, &need));
  if (cfg->weight_format != NH_WEIGHTS_FP8)
    return fail(NH_ERR_INVALID_ARG, "config has no FP8 weights (weight_format)");
  Plan p;
  NH_TRY(make_plan(cfg, T, &p));
  NH_TRY(check_ptr(ws, "ws_shared"));
  if (reinterpret_cast<uintptr_t>(ws) % ALIGN)
    return fail(NH_ERR_INVALID_ARG, "ws_shared must be %zu-byte aligned", ALIGN);
  if (ws_bytes < need)
    return fail(NH_ERR_INVALID_ARG, "ws_shared holds %zu bytes, %zu needed", ws_bytes, need);
  NH_TRY(check_f8(w_su, "w_shared_up"));
  NH_TRY(check_f8(w_sd, "w_shared_down"));
  if (T == 0) return NH_OK;
  NH_TRY(check_ptr(x, "x"));
  NH_TRY(check_ptr(y_acc, "y_acc"));
  int dev;
  NH_TRY(f8_device_setup(&dev));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* status = static_cast<int*>(ws);
  NH_CUDA(cudaMemsetAsync(status, 0, STATUS_BYTES, st));
  uint8_t* xq = at<uint8_t>(ws, ALIGN);
  float* xs = at<float>(ws, ALIGN + f8_scales_at(T, p.H));
  const F8Hidden h = f8_hidden(at<void>(ws, ALIGN + f8_rows_bytes(T, p.H)), T, p.S);
  F8Call up{};
  up.w = w_su;
  up.n_exp = 1;
  up.rows = T;
  up.N = p.S;
  up.K = p.H;
  up.status = status;
  // the GEMV leaves relu^2 in float32, to be quantized by what follows; the tiles'
  // ends quantize it themselves
  const bool gemv = f8_gemv_rows(up);
  up.out_kind = F8_RELU2;
  up.out = gemv ? static_cast<void*>(h.f32) : h.codes;
  up.out_scales = h.scales;
  NH_TRY(run_f8_dense(up, x, true, xq, xs, false, dev, st));
  F8Call down = up;
  down.w = w_sd;
  down.N = p.H;
  down.K = p.S;
  down.out_kind = store ? F8_F32 : F8_ADD;
  down.out = y_acc;
  if (gemv) return run_f8_dense(down, h.f32, false, h.codes, h.scales, true, dev, st);
  down.x = h.codes;
  down.xs = h.scales;
  down.x_rows = T;
  down.early_w = true;   // the launch before is this call's up projection
  return run_f8(down, dev, st);
}

nh_status nh_moe_shared_fp8(const nh_moe_config* cfg, int64_t T, const void* x,
                            const nh_fp8_weight* w_shared_up, const nh_fp8_weight* w_shared_down,
                            float* y_acc, void* ws_shared, size_t ws_shared_bytes, void* stream) {
  return f8_shared(cfg, T, x, w_shared_up, w_shared_down, y_acc, ws_shared, ws_shared_bytes, stream,
                   false);
}

nh_status nh_moe_shared_store_fp8(const nh_moe_config* cfg, int64_t T, const void* x,
                                  const nh_fp8_weight* w_shared_up,
                                  const nh_fp8_weight* w_shared_down, float* y_acc, void* ws_shared,
                                  size_t ws_shared_bytes, void* stream) {
  return f8_shared(cfg, T, x, w_shared_up, w_shared_down, y_acc, ws_shared, ws_shared_bytes, stream,
                   true);
}
