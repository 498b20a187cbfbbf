"""Refusals of the gate and FP8 entry points, on the host: nothing is enqueued when an
argument check fails, so these need no GPU."""
import ctypes

import pytest

import non_gated_relu_b200 as nh
import synth

P = ctypes.c_void_p
OK = P(256)


def gate_cfg(**kw):
    base = dict(n_routed_experts=16, num_experts_per_tok=4, n_group=4, topk_group=2)
    base.update(kw)
    return nh.gate_config(**base)


@pytest.mark.parametrize("kw", [
    dict(n_routed_experts=0), dict(n_group=3), dict(n_group=0), dict(topk_group=0),
    dict(topk_group=5), dict(num_experts_per_tok=0), dict(num_experts_per_tok=9),
    dict(routed_scaling_factor=float("nan")), dict(routed_scaling_factor=float("inf")),
    dict(n_group=16, topk_group=4, group_score="top2")])
def test_gate_refuses_bad_configs(kw):
    lib, c = nh.load(), gate_cfg(**kw)
    for rc in (lib.nh_moe_gate(ctypes.byref(c), 4, OK, None, OK, OK, None),
               lib.nh_moe_gate_backward(ctypes.byref(c), 4, OK, OK, OK, OK, None)):
        assert rc == nh.NH_ERR_INVALID_ARG, kw


@pytest.mark.parametrize("field,value", [("score_func", 2), ("group_score", 5), ("dtype", 7),
                                         ("norm_topk_prob", 2)])
def test_gate_refuses_unknown_enums(field, value):
    lib, c = nh.load(), gate_cfg()
    setattr(c, field, value)
    assert lib.nh_moe_gate(ctypes.byref(c), 4, OK, None, OK, OK, None) == nh.NH_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(n_routed_experts=520, n_group=4),
                                dict(n_routed_experts=256, n_group=128, topk_group=128),
                                dict(n_routed_experts=64, n_group=1, topk_group=1,
                                     num_experts_per_tok=33)])
def test_gate_sizes_the_kernels_do_not_take(kw):
    lib, c = nh.load(), gate_cfg(**kw)
    assert lib.nh_moe_gate(ctypes.byref(c), 4, OK, None, OK, OK, None) == nh.NH_ERR_UNSUPPORTED


def test_gate_pointers_and_token_counts():
    lib, c = nh.load(), gate_cfg()
    ref = ctypes.byref(c)
    for args, word in (((None, None, OK, OK), b"logits"), ((OK, None, None, OK), b"topk_idx"),
                       ((OK, None, OK, None), b"topk_w"), ((OK, P(8), OK, OK), b"bias"),
                       ((P(264), None, OK, OK), b"aligned")):
        assert lib.nh_moe_gate(ref, 4, *args, None) == nh.NH_ERR_INVALID_ARG
        assert word in lib.nh_last_error()
    for args, word in (((None, OK, OK, OK), b"logits"), ((OK, None, OK, OK), b"topk_idx"),
                       ((OK, OK, None, OK), b"d_topk_w"), ((OK, OK, OK, None), b"d_logits")):
        assert lib.nh_moe_gate_backward(ref, 4, *args, None) == nh.NH_ERR_INVALID_ARG
        assert word in lib.nh_last_error()
    assert lib.nh_moe_gate(ref, -1, OK, None, OK, OK, None) == nh.NH_ERR_INVALID_ARG
    assert lib.nh_moe_gate(ref, 1 << 31, OK, None, OK, OK, None) == nh.NH_ERR_UNSUPPORTED
    assert lib.nh_moe_gate(None, 4, OK, None, OK, OK, None) == nh.NH_ERR_INVALID_ARG
    # no tokens: nothing to do, no pointers needed
    assert lib.nh_moe_gate(ref, 0, None, None, None, None, None) == nh.NH_OK
    assert lib.nh_moe_gate_backward(ref, 0, None, None, None, None, None) == nh.NH_OK


def test_gate_config_names():
    c = nh.gate_config(8, 2, scoring_func="softmax", group_score="top2", dtype="bf16")
    assert (c.score_func, c.group_score, c.dtype) == (nh.NH_SCORE_SOFTMAX, 1, nh.NH_BF16)
    for kw in (dict(scoring_func="relu"), dict(group_score="min"), dict(dtype="f16")):
        with pytest.raises(ValueError):
            nh.gate_config(8, 2, **kw)


def test_route_scored_checks():
    lib = nh.load()
    cfg = synth.CONFIGS["decode_bf16_t8"]
    c = nh.config_from(cfg)
    need = nh.workspace_layout(cfg, 8).counts
    ref = ctypes.byref(c)
    call = lib.nh_moe_route_scored
    assert call(ref, 2, 8, OK, OK, None, OK, OK, OK, need, None) == nh.NH_ERR_INVALID_ARG
    assert b"score_func" in lib.nh_last_error()
    assert call(ref, 1, 8, OK, OK, None, OK, OK, None, need, None) == nh.NH_ERR_INVALID_ARG
    assert call(ref, 1, 8, OK, OK, None, OK, OK, OK, need - 1, None) == nh.NH_ERR_INVALID_ARG
    assert b"needed" in lib.nh_last_error()
    assert call(ref, 1, 8, OK, OK, None, OK, OK, P(272), need, None) == nh.NH_ERR_INVALID_ARG
    assert call(ref, 1, 8, OK, None, None, OK, OK, OK, need, None) == nh.NH_ERR_INVALID_ARG
    assert call(ref, 1, 0, None, None, None, None, None, OK, need, None) == nh.NH_OK


def test_quantize_checks():
    lib = nh.load()
    q = lib.nh_fp8_quantize
    assert q(4, 24, OK, nh.NH_F32, OK, OK, None) == nh.NH_ERR_UNSUPPORTED      # 24 % 16
    assert q(4, 0, OK, nh.NH_F32, OK, OK, None) == nh.NH_ERR_INVALID_ARG
    assert q(-1, 32, OK, nh.NH_F32, OK, OK, None) == nh.NH_ERR_INVALID_ARG
    assert q(4, 32, OK, 9, OK, OK, None) == nh.NH_ERR_INVALID_ARG
    for args in ((None, OK, OK), (OK, None, OK), (OK, OK, None), (P(8), OK, OK)):
        assert q(4, 32, args[0], nh.NH_F32, args[1], args[2], None) == nh.NH_ERR_INVALID_ARG
    assert q(1 << 31, 32, OK, nh.NH_F32, OK, OK, None) == nh.NH_ERR_UNSUPPORTED
    assert q(0, 32, None, nh.NH_F32, None, None, None) == nh.NH_OK
    w = lib.nh_fp8_quantize_weight
    assert w(1, 8, 24, OK, nh.NH_F32, OK, OK, None) == nh.NH_ERR_UNSUPPORTED
    assert w(-1, 8, 32, OK, nh.NH_F32, OK, OK, None) == nh.NH_ERR_INVALID_ARG
    assert w(1, 8, 32, None, nh.NH_F32, OK, OK, None) == nh.NH_ERR_INVALID_ARG
    assert w(1 << 30, 1 << 20, 1 << 20, OK, nh.NH_F32, OK, OK, None) == nh.NH_ERR_UNSUPPORTED
    assert w(0, 8, 32, None, nh.NH_F32, None, None, None) == nh.NH_OK


def test_linear_checks():
    lib = nh.load()
    w = nh.Fp8Weight(256, 256)
    wr = ctypes.byref(w)
    need = nh.fp8_linear_workspace_size(4, 32, 48)
    assert need >= 256 + 4 * 48 + 4 * 4

    def call(T=4, N=32, K=48, x=OK, xd=nh.NH_BF16, w=wr, y=OK, yd=nh.NH_BF16, ws=OK, n=need):
        return lib.nh_fp8_linear(T, N, K, x, xd, w, y, yd, ws, n, None)

    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(ws=None), dict(n=need - 1),
               dict(xd=5), dict(yd=5), dict(T=-1), dict(ws=P(272)), dict(x=P(258)),
               dict(w=ctypes.byref(nh.Fp8Weight(0, 256))),
               dict(w=ctypes.byref(nh.Fp8Weight(256, 260)))):
        assert call(**kw) == nh.NH_ERR_INVALID_ARG, kw
    assert call(N=24) == nh.NH_ERR_UNSUPPORTED
    assert call(K=40) == nh.NH_ERR_UNSUPPORTED
    assert call(T=0, x=None, w=None, y=None) == nh.NH_OK
    with pytest.raises(nh.NHMoEError):
        nh.fp8_linear_workspace_size(4, 32, 40)


def test_fp8_weight_format_and_its_entry_points():
    lib = nh.load()
    base = synth.CONFIGS["decode_bf16_t8"]
    cfg = base.replace(weight_format="fp8")
    nh.validate(cfg)
    with pytest.raises(nh.NHMoEError) as e:
        nh.validate(cfg.replace(dtype="f32"))
    assert e.value.status == nh.NH_ERR_INVALID_ARG
    c, bf = nh.config_from(cfg), nh.config_from(base)
    q4 = nh.config_from(base.replace(weight_format="nvfp4"))
    w = nh.Fp8Weight(256, 256)
    wr = ctypes.byref(w)
    need, sneed = nh.workspace_size(cfg, 8), nh.shared_workspace_size(cfg, 8)
    ref = ctypes.byref(c)
    # FP8 configs are refused by the other formats' calls, and theirs by these
    for rc in (lib.nh_moe_forward(ref, 8, OK, OK, OK, OK, need, OK, None),
               lib.nh_moe_experts_up(ref, 8, OK, OK, OK, need, None),
               lib.nh_moe_experts_down(ref, 8, OK, OK, need, OK, None),
               lib.nh_moe_shared(ref, 8, OK, OK, OK, OK, OK, sneed, None),
               lib.nh_moe_shared_store(ref, 8, OK, OK, OK, OK, OK, sneed, None)):
        assert rc == nh.NH_ERR_INVALID_ARG and b"FP8" in lib.nh_last_error()
    n4 = nh.NvFp4Weight(256, 256, 256)
    rc = lib.nh_moe_forward_nvfp4(ref, 8, OK, ctypes.byref(n4), ctypes.byref(n4), OK, need, OK, None)
    assert rc == nh.NH_ERR_INVALID_ARG and b"FP8" in lib.nh_last_error()
    rc = lib.nh_moe_shared_nvfp4(ref, 8, OK, ctypes.byref(n4), ctypes.byref(n4), OK, OK, sneed, None)
    assert rc == nh.NH_ERR_INVALID_ARG
    for other in (bf, q4):
        r = ctypes.byref(other)
        big = 1 << 40
        for rc in (lib.nh_moe_forward_fp8(r, 8, OK, wr, wr, OK, big, OK, None),
                   lib.nh_moe_experts_up_fp8(r, 8, OK, wr, OK, big, None),
                   lib.nh_moe_experts_down_fp8(r, 8, wr, OK, big, OK, None),
                   lib.nh_moe_shared_fp8(r, 8, OK, wr, wr, OK, OK, big, None),
                   lib.nh_moe_shared_store_fp8(r, 8, OK, wr, wr, OK, OK, big, None)):
            assert rc == nh.NH_ERR_INVALID_ARG and b"no FP8" in lib.nh_last_error()
    # pointers and workspaces
    bad = ctypes.byref(nh.Fp8Weight(256, 0))
    for rc in (lib.nh_moe_forward_fp8(ref, 8, OK, wr, wr, OK, need - 1, OK, None),
               lib.nh_moe_forward_fp8(ref, 8, None, wr, wr, OK, need, OK, None),
               lib.nh_moe_forward_fp8(ref, 8, OK, None, wr, OK, need, OK, None),
               lib.nh_moe_forward_fp8(ref, 8, OK, wr, bad, OK, need, OK, None),
               lib.nh_moe_forward_fp8(ref, 8, OK, wr, wr, OK, need, None, None),
               lib.nh_moe_forward_fp8(ref, 8, OK, wr, wr, P(272), need, OK, None),
               lib.nh_moe_forward_fp8(ref, -1, OK, wr, wr, OK, need, OK, None),
               lib.nh_moe_shared_fp8(ref, 8, OK, wr, wr, OK, OK, sneed - 1, None),
               lib.nh_moe_shared_fp8(ref, 8, OK, wr, wr, None, OK, sneed, None),
               lib.nh_moe_shared_fp8(ref, 8, OK, wr, wr, OK, P(272), sneed, None)):
        assert rc == nh.NH_ERR_INVALID_ARG
    lat = nh.config_from(cfg.replace(latent_size=1024))
    rc = lib.nh_moe_forward_fp8(ctypes.byref(lat), 8, OK, wr, wr, OK, need, OK, None)
    assert rc == nh.NH_ERR_INVALID_ARG and b"latent_size" in lib.nh_last_error()


@pytest.mark.parametrize("T", [0, 1, 8, 9, 32, 33, 300, 5000])
def test_fp8_workspace_holds_codes_and_scales(T):
    cfg = synth.CONFIGS["decode_bf16_t8"].replace(weight_format="fp8")
    L = nh.workspace_layout(cfg, T)
    rows = T * cfg.k
    assert L.x_direct == 0 and L.swap_ab == int(L.tile_rows < 256)
    assert L.tile_rows in (16, 32, 64, 256)
    assert L.max_tiles >= -(-rows // L.tile_rows) + min(rows, cfg.E - 1)
    assert L.h - L.x_perm >= rows * (cfg.H + 4 * -(-cfg.H // 128))
    assert L.ready - L.h >= rows * (cfg.I + 4 * -(-cfg.I // 128))
    assert L.total_bytes == nh.workspace_size(cfg, T)


@pytest.mark.parametrize("n,world", [(1856, 2), (1856, 3), (3712, 4), (192, 2), (128, 1)])
def test_fp8_shards_are_whole_scale_blocks(n, world):
    from non_gated_relu_b200 import tp
    cuts = [tp.shard_range_fp8(n, world, r) for r in range(world)]
    assert cuts[0][0] == 0 and cuts[-1][1] == n
    assert all(a[1] == b[0] for a, b in zip(cuts, cuts[1:]))
    assert all(s % 128 == 0 and e > s and (e - s) % 64 == 0 for s, e in cuts)
    with pytest.raises(ValueError):
        tp.shard_range_fp8(n, -(-n // 128) + 1, 0)
    with pytest.raises(ValueError):
        tp.shard_range_fp8(n, world, world)


def test_fp8_shards_hold_the_weights_values():
    torch = pytest.importorskip("torch")
    import fp8_util as ref
    from non_gated_relu_b200 import tp
    gen = torch.Generator().manual_seed(0)
    cfg = synth.CONFIGS["decode_bf16_t8"].replace(
        weight_format="fp8", hidden_size=256, n_routed_experts=8, n_group=1, topk_group=1,
        moe_intermediate_size=320, moe_shared_expert_intermediate_size=448)
    q = {"up": ref.make_weight(gen, 8, 320, 256), "down": ref.make_weight(gen, 8, 256, 320),
         "shared_up": ref.make_weight(gen, 1, 448, 256), "shared_down": ref.make_weight(gen, 1, 256, 448)}
    for world in (1, 2, 3):
        parts = {k: [] for k in q}
        for r in range(world):
            c = tp.shard_config(cfg, world, r)
            sh = tp.shard_fp8(cfg, world, r, q)
            assert sh["up"][0].shape == (8, c.moe_intermediate_size, 256)
            assert sh["shared_down"][0].shape[2] == c.moe_shared_expert_intermediate_size
            for k in q:
                parts[k].append(ref.weight_values(*sh[k]))
        for k in q:
            got = torch.cat(parts[k], dim=2 if k.endswith("down") else 1)
            assert torch.equal(got, ref.weight_values(*q[k]))


def test_python_argument_checks():
    torch = pytest.importorskip("torch")
    c = nh.gate_config(16, 4)
    f = torch.zeros((2, 16))
    i, w = torch.zeros((2, 4), dtype=torch.int32), torch.zeros((2, 4))
    with pytest.raises(TypeError):
        nh.gate(c, f.half(), None, i, w)
    with pytest.raises(TypeError):
        nh.gate(c, f, None, i.long(), w)
    with pytest.raises(ValueError):
        nh.gate(c, f[:, :8], None, i, w)
    with pytest.raises(ValueError):
        nh.gate(c, torch.zeros((16, 2)).t(), None, i, w)       # not contiguous
    with pytest.raises(ValueError):
        nh.gate(c, f, torch.zeros(15), i, w)
    with pytest.raises(ValueError):
        nh.fp8_weight(torch.zeros((8, 16), dtype=torch.uint8), torch.zeros((1, 1)))
    with pytest.raises(TypeError):
        nh.fp8_quantize(torch.zeros((2, 16), dtype=torch.float64), None, None)
    if not torch.cuda.is_available():
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            nh.gate(c, f, None, i, w)                          # host tensors


def test_weights_of_another_device_are_refused(monkeypatch):
    pytest.importorskip("torch")
    w = nh.Fp8Weight(256, 256)
    w.shape, w.device = (1, 64, 128), 1
    monkeypatch.setattr(nh._types(), "current_device", lambda: 1)
    nh._fp8("w", w, (1, 64, 128))
    monkeypatch.setattr(nh._types(), "current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1"):
        nh._fp8("w", w, (1, 64, 128))


def test_unknown_weight_formats_are_refused():
    base = synth.CONFIGS["tiny_f32_t64"].replace(dtype="bf16", hidden_size=64)
    for fmt in ("FP8", "fp8_e4m3", "bf16", 3):
        with pytest.raises(ValueError, match="weight_format"):
            nh.config_from(base.replace(weight_format=fmt))
    for fmt, value in (("native", 0), ("nvfp4", 1), ("fp8", 2), (2, 2), (None, 0)):
        assert nh.config_from(base.replace(weight_format=fmt)).weight_format == value


def test_sigmoid_routers_refuse_other_scores():
    """The routers whose scores are sigmoids do not answer a config that asks for others."""
    torch = pytest.importorskip("torch")
    cfg = synth.CONFIGS["tiny_f32_t64"].replace(T=2, scoring_func="softmax")
    x = torch.zeros((2, cfg.hidden_size))
    for call in (lambda c: nh.route(c, x, x, None, x, x, x),
                 lambda c: nh.route_permute(c, x, x, None, x, x, x),
                 lambda c: nh.route_noalloc(c, x, x, None, x, x)):
        with pytest.raises(ValueError, match="route_scored"):
            call(cfg)
        with pytest.raises(ValueError, match="scoring_func"):
            call(cfg.replace(scoring_func="sqrtsoftplus"))
