// api_gate.cuh -- C ABI of the gate.  Part of nh_moe.cu (inside extern "C").

nh_status nh_moe_gate(const nh_moe_gate_config* cfg, int64_t T, const void* logits,
                      const float* bias, int32_t* topk_idx, float* topk_w, void* stream) {
  NH_TRY(check_gate(cfg, T));
  if (T == 0) return NH_OK;
  NH_TRY(check_ptr(logits, "logits"));
  NH_TRY(check_ptr(topk_idx, "topk_idx"));
  NH_TRY(check_ptr(topk_w, "topk_w"));
  if (bias) NH_TRY(check_ptr(bias, "e_score_correction_bias"));
  int dev;
  NH_TRY(device_setup(&dev));
  gate::Args a = gate_args(cfg, T);
  a.logits = logits;
  a.bias = bias;
  a.idx = topk_idx;
  a.w = topk_w;
  return launch_gate(a, cfg->dtype == NH_BF16, false, static_cast<cudaStream_t>(stream));
}

nh_status nh_moe_gate_backward(const nh_moe_gate_config* cfg, int64_t T, const void* logits,
                               const int32_t* topk_idx, const float* d_topk_w, void* d_logits,
                               void* stream) {
  NH_TRY(check_gate(cfg, T));
  if (T == 0) return NH_OK;
  NH_TRY(check_ptr(logits, "logits"));
  NH_TRY(check_ptr(topk_idx, "topk_idx"));
  NH_TRY(check_ptr(d_topk_w, "d_topk_w"));
  NH_TRY(check_ptr(d_logits, "d_logits"));
  int dev;
  NH_TRY(device_setup(&dev));
  gate::Args a = gate_args(cfg, T);
  a.logits = logits;
  a.idx = const_cast<int32_t*>(topk_idx);
  a.dw = d_topk_w;
  a.dlogits = d_logits;
  return launch_gate(a, cfg->dtype == NH_BF16, true, static_cast<cudaStream_t>(stream));
}

nh_status nh_moe_route_scored(const nh_moe_config* cfg, int32_t score_func, int64_t T,
                              const void* x, const float* w_router, const float* bias,
                              int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes,
                              void* stream) {
  Plan p;
  NH_TRY(make_plan(cfg, T, &p));
  const nh_moe_gate_config gc = {p.E, p.G, p.tg, p.k, cfg->norm_topk_prob,
                                 cfg->routed_scaling_factor, score_func, cfg->group_score, NH_F32};
  NH_TRY(check_gate(&gc, T));
  NH_TRY(check_ptr(ws, "ws"));
  if (reinterpret_cast<uintptr_t>(ws) % ALIGN)
    return fail(NH_ERR_INVALID_ARG, "ws must be %zu-byte aligned", ALIGN);
  if (ws_bytes < p.lay.counts)
    return fail(NH_ERR_INVALID_ARG, "ws holds %zu bytes, %zu needed for routing", ws_bytes,
                p.lay.counts);
  if (T == 0) return NH_OK;
  NH_TRY(check_ptr(x, "x"));
  NH_TRY(check_ptr(w_router, "w_router"));
  NH_TRY(check_ptr(topk_idx, "topk_idx"));
  NH_TRY(check_ptr(topk_w, "topk_w"));
  if (bias) NH_TRY(check_ptr(bias, "e_score_correction_bias"));
  int dev;
  NH_TRY(device_setup(&dev));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  NH_CUDA(cudaMemsetAsync(at<int>(ws, p.lay.status), 0, STATUS_BYTES, st));
  float* logits = at<float>(ws, p.lay.logits);
  if (T > 32)
    NH_TRY(route_logits(p, T, x, w_router, ws, dev, st));
  else if (p.bf16)
    NH_TRY((launch_k("router_logits_small", router_logits_small<__nv_bfloat16>, dim3(p.E), dim3(256),
                     0, st, static_cast<const __nv_bfloat16*>(x), w_router, logits, (int)T, p.E,
                     p.H)));
  else
    NH_TRY((launch_k("router_logits_small", router_logits_small<float>, dim3(p.E), dim3(256), 0, st,
                     static_cast<const float*>(x), w_router, logits, (int)T, p.E, p.H)));
  gate::Args a = gate_args(&gc, T);
  a.logits = logits;
  a.bias = bias;
  a.idx = topk_idx;
  a.w = topk_w;
  return launch_gate(a, false, false, st);
}
