// launch_gate.cuh -- host side of the gate: checks and kernel choice.  Part of
// nh_moe.cu (inside namespace nh).

static nh_status check_gate(const nh_moe_gate_config* c, int64_t T) {
  if (!c) return fail(NH_ERR_INVALID_ARG, "gate config is NULL");
  if (c->n_routed_experts < 1) return fail(NH_ERR_INVALID_ARG, "n_routed_experts must be >= 1");
  if (c->n_group < 1 || c->n_routed_experts % c->n_group != 0)
    return fail(NH_ERR_INVALID_ARG, "n_routed_experts (%d) must be a multiple of n_group (%d)",
                c->n_routed_experts, c->n_group);
  if (c->topk_group < 1 || c->topk_group > c->n_group)
    return fail(NH_ERR_INVALID_ARG, "topk_group must be in [1, n_group]");
  const int g = c->n_routed_experts / c->n_group;
  if (c->num_experts_per_tok < 1 || (int64_t)c->num_experts_per_tok > (int64_t)c->topk_group * g)
    return fail(NH_ERR_INVALID_ARG, "num_experts_per_tok must be in [1, topk_group * E / n_group]");
  if (c->norm_topk_prob != 0 && c->norm_topk_prob != 1)
    return fail(NH_ERR_INVALID_ARG, "norm_topk_prob must be 0 or 1");
  if (!std::isfinite(c->routed_scaling_factor))
    return fail(NH_ERR_INVALID_ARG, "routed_scaling_factor must be finite");
  if (c->score_func != NH_SCORE_SIGMOID && c->score_func != NH_SCORE_SOFTMAX)
    return fail(NH_ERR_INVALID_ARG, "unknown score_func");
  if (c->group_score != NH_GROUP_SCORE_MAX && c->group_score != NH_GROUP_SCORE_TOP2)
    return fail(NH_ERR_INVALID_ARG, "unknown group_score");
  if (c->group_score == NH_GROUP_SCORE_TOP2 && g < 2)
    return fail(NH_ERR_INVALID_ARG, "the top-2 group score needs >= 2 experts per group");
  if (c->dtype != NH_F32 && c->dtype != NH_BF16) return fail(NH_ERR_INVALID_ARG, "unknown dtype");
  if (T < 0) return fail(NH_ERR_INVALID_ARG, "T must be >= 0");
  if (c->n_routed_experts > MAX_E) return fail(NH_ERR_UNSUPPORTED, "n_routed_experts > %d", MAX_E);
  if (c->n_group > MAX_G) return fail(NH_ERR_UNSUPPORTED, "n_group > %d", MAX_G);
  if (c->num_experts_per_tok > MAX_K)
    return fail(NH_ERR_UNSUPPORTED, "num_experts_per_tok > %d", MAX_K);
  if (T >= int64_t(1) << 31) return fail(NH_ERR_UNSUPPORTED, "T must be < 2^31");
  return NH_OK;
}

static gate::Args gate_args(const nh_moe_gate_config* c, int64_t T) {
  gate::Args a{};
  a.T = T;
  a.E = c->n_routed_experts;
  a.G = c->n_group;
  a.tg = c->topk_group;
  a.k = c->num_experts_per_tok;
  a.softmax = c->score_func == NH_SCORE_SOFTMAX;
  a.norm = c->norm_topk_prob;
  a.top2 = c->group_score == NH_GROUP_SCORE_TOP2;
  a.alpha = c->routed_scaling_factor;
  return a;
}

template <int PER>
static nh_status launch_gate_per(const gate::Args& a, bool bf16, bool backward, cudaStream_t st) {
  const dim3 grid((unsigned)((a.T + gate::WARPS - 1) / gate::WARPS)), block(gate::WARPS * 32);
  if (backward)
    return bf16 ? launch_k("gate_backward", gate::gate_backward<PER, __nv_bfloat16>, grid, block, 0, st, a)
                : launch_k("gate_backward", gate::gate_backward<PER, float>, grid, block, 0, st, a);
  const size_t smem = (size_t)gate::WARPS * a.E * sizeof(double);
  return bf16 ? launch_k("gate_forward", gate::gate_forward<PER, __nv_bfloat16>, grid, block, smem, st, a)
              : launch_k("gate_forward", gate::gate_forward<PER, float>, grid, block, smem, st, a);
}

// experts per lane: the least power of two that holds a row in one warp
static nh_status launch_gate(const gate::Args& a, bool bf16, bool backward, cudaStream_t st) {
  if (a.E <= 32) return launch_gate_per<1>(a, bf16, backward, st);
  if (a.E <= 64) return launch_gate_per<2>(a, bf16, backward, st);
  if (a.E <= 128) return launch_gate_per<4>(a, bf16, backward, st);
  if (a.E <= 256) return launch_gate_per<8>(a, bf16, backward, st);
  return launch_gate_per<16>(a, bf16, backward, st);
}
