"""FP8 (E4M3, a scale per block of 128): quantization, the linear product, the experts and
the block, against 64-bit references (fp8_util).

Tolerance of a product, derived: a product of two codes has 8 significant bits and is
exact; a block's 128 are summed by the tensor cores in at least 24 bits, 128 steps of
2^-23 of their magnitudes at most; the two scales' product and its multiply-add are 2
roundings; the blocks' and the warps' sums KB + 8 more: with S = sum |x| |w| of the
dequantized values,  |error| <= S (128 2^-23 + (KB + 10) 2^-24)."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import non_gated_relu_b200 as nh  # noqa: E402
import fp8_util as ref  # noqa: E402
import synth  # noqa: E402

DEV = "cuda"
B16, F32 = torch.bfloat16, torch.float32


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def gamma(K):
    return 128 * 2.0 ** -23 + (-(-K // 128) + 10) * 2.0 ** -24


# -- quantization -----------------------------------------------------------------------
def quantized(x):
    T, K = x.shape
    codes = torch.full((T + 1, K), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((T + 1, -(-K // 128)), -3.0, device=DEV)
    nh.fp8_quantize(x, codes[:T], scales[:T])
    torch.cuda.synchronize()
    assert (codes[T] == 0x55).all() and (scales[T] == -3).all(), "wrote past the last row"
    return codes[:T], scales[:T]


def same(a, b):
    return torch.equal(a.nan_to_num(nan=9e9), b.nan_to_num(nan=9e9))


@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("T,K", [(1, 16), (1, 128), (3, 144), (5, 112), (33, 1856), (257, 2688),
                                 (2000, 64)])
def test_quantize(T, K, dtype):
    gen = generator(T + K)
    # magnitudes over many binades, so that scales and subnormal codes vary
    x = torch.randn((T, K), generator=gen, device=DEV) * torch.exp2(
        torch.randint(-20, 20, (T, 1), generator=gen, device=DEV).float())
    x = (x * torch.exp2(torch.randint(-12, 1, (T, K), generator=gen, device=DEV).float())).to(dtype)
    codes, scales = quantized(x)
    q, s = ref.quantize_rows(x)
    assert torch.equal(scales.double(), s)
    assert torch.equal(ref.decode(codes), q)


@pytest.mark.parametrize("dtype", [B16, F32])
def test_quantize_borders(dtype):
    x = torch.zeros((12, 256), device=DEV)
    step = 1 + 2.0 ** (-7 if dtype == B16 else -23)
    x[0, 0] = 448.0                     # fits a scale of 1 exactly
    x[1, 0] = 448.0 * step              # just does not
    x[2, 127], x[2, 128] = 448.0 * 2 ** 10, -448.0 * 2.0 ** -10
    x[3, :17] = torch.arange(17, device=DEV) + 0.5      # ties between codes go to the even one
    x[3, 17:40] = 2.0 ** -9 * (torch.arange(23, device=DEV) / 4)
    x[3, 100] = 400.0
    x[4, 5] = torch.finfo(dtype).max
    x[5, 5] = torch.finfo(dtype).tiny
    x[6, 5], x[6, 6] = math.inf, 3.0    # not finite: NaN codes, the others by their own maximum
    x[7, 5], x[7, 200] = math.nan, -math.inf
    x[8] = math.nan
    x[9] = -0.0
    x[10, :128] = 1.0
    x[11, 3] = torch.finfo(dtype).tiny / 4              # subnormal
    x = x.to(dtype)
    codes, scales = quantized(x)
    q, s = ref.quantize_rows(x)
    assert torch.equal(scales.double(), s)
    assert same(ref.decode(codes), q)
    assert scales[0, 0] == 1 and scales[1, 0] == 2 and scales[9, 0] == 1
    assert scales[5, 0] == 2.0 ** -126 and scales[8, 0] == 1


def test_quantize_past_32_bits():
    K, T = 2688, (1 << 32) // 2688 + 40         # rows whose offset passes 2^32 elements
    x = torch.empty((T, K), dtype=B16, device=DEV)
    x.view(-1)[: 1 << 20].fill_(1.0)
    tail = torch.randn((32, K), generator=generator(1), device=DEV).to(B16)
    x[-32:] = tail
    codes = torch.empty((T, K), dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty((T, K // 128), device=DEV)
    nh.fp8_quantize(x, codes, scales)
    q, s = ref.quantize_rows(tail)
    assert torch.equal(scales[-32:].double(), s)
    assert torch.equal(ref.decode(codes[-32:]), q)
    assert (scales[:300] == 2.0 ** -8).all() and (codes[:300].float() == 256).all()


@pytest.mark.parametrize("dtype", [B16, F32])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 16), (2, 128, 128), (3, 200, 144), (1, 1856, 2688),
                                         (5, 129, 272)])
def test_quantize_weight(n, rows, cols, dtype):
    gen = generator(rows)
    w = (torch.randn((n, rows, cols), generator=gen, device=DEV) * 0.02).to(dtype)
    w[0, 0, 0] = 7.0
    codes, scales = nh.fp8_quantize_weight(w)
    q, s = ref.quantize_weight(w)
    assert torch.equal(scales.double(), s)
    assert torch.equal(ref.decode(codes), q)


# -- linear ---------------------------------------------------------------------------------
def linear(x, w, N, out=B16, ws=None):
    T, K = x.shape
    if ws is None:
        ws = torch.zeros(nh.fp8_linear_workspace_size(T, N, K), dtype=torch.uint8, device=DEV)
    y = torch.full((T + 1, N), -77.0, dtype=out, device=DEV)
    nh.fp8_linear(x, w, y[:T], ws)
    assert nh.check_device(ws) == 0
    assert (y[T] == -77).all(), "wrote past the last row"
    return y[:T]


def check_product(y, xv, wv, K):
    want = xv @ wv.t()
    tol = (xv.abs() @ wv.abs().t()) * gamma(K) + want.abs() * ref.EPS[y.dtype]
    err = (y.double() - want).abs()
    assert (err <= tol).all(), (float((err / tol.clamp(min=1e-300)).max()))
    return float((err.norm() / want.norm()).item())


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 64, 128, 129, 256, 257, 600])
@pytest.mark.parametrize("N,K", [(16, 16), (64, 128), (272, 144), (1856, 2688), (2688, 1856),
                                 (400, 1136)])
def test_linear(T, N, K):
    gen = generator(T * 31 + N)
    codes, scales = ref.make_weight(gen, 1, N, K)
    w = nh.fp8_weight(codes, scales)
    wv = ref.weight_values(codes[0], scales[0])
    x = torch.randn((T, K), generator=gen, device=DEV)
    check_product(linear(x.to(B16), w, N), ref.rows_values(x.to(B16)), wv, K)
    rel = check_product(linear(x, w, N, F32), ref.rows_values(x), wv, K)
    assert rel <= 2e-5


@pytest.mark.parametrize("T,N,K", [(9537, 16, 16), (9601, 64, 128), (3300, 272, 144),
                                   (2400, 400, 1136), (700, 1856, 144), (449, 3712, 2688),
                                   (320, 3712, 2688), (640, 1856, 2688), (321, 3712, 2688)])
def test_linear_many_rows(T, N, K):
    """On both sides of one tile of 128 features x 64 rows for each SM, where the form
    changes; last tiles of 1 to 63 rows and of 16 features."""
    gen = generator(T * 31 + N)
    codes, scales = ref.make_weight(gen, 1, N, K)
    w = nh.fp8_weight(codes, scales)
    wv = ref.weight_values(codes[0], scales[0])
    x = torch.randn((T, K), generator=gen, device=DEV)
    check_product(linear(x.to(B16), w, N), ref.rows_values(x.to(B16)), wv, K)
    assert check_product(linear(x, w, N, F32), ref.rows_values(x), wv, K) <= 2e-5


def test_linear_many_tiles():
    """More tiles than CTA pairs, a last tile of 32 features, and rows of every size."""
    gen = generator(4)
    T, N, K = 4999, 1824, 528
    codes, scales = ref.make_weight(gen, 1, N, K)
    x = (torch.randn((T, K), generator=gen, device=DEV) *
         torch.exp2(torch.randint(-30, 30, (T, 1), generator=gen, device=DEV).float()))
    check_product(linear(x, nh.fp8_weight(codes, scales), N, F32), ref.rows_values(x),
                  ref.weight_values(codes[0], scales[0]), K)


def test_linear_past_32_bits():
    """y passes 2^31 elements and 2^32 bytes."""
    gen = generator(6)
    T, N, K = 600_001, 4096, 64
    codes, scales = ref.make_weight(gen, 1, N, K)
    x = torch.randn((T, K), generator=gen, device=DEV).to(B16)
    y = linear(x, nh.fp8_weight(codes, scales), N)
    wv = ref.weight_values(codes[0], scales[0])
    for part in (slice(0, 300), slice(T - 300, T), slice(T // 2, T // 2 + 100)):
        check_product(y[part], ref.rows_values(x[part]), wv, K)


@pytest.mark.parametrize("T", [0])
def test_no_tokens(T):
    gen = generator(1)
    codes, scales = ref.make_weight(gen, 1, 64, 128)
    x = torch.empty((0, 128), dtype=B16, device=DEV)
    ws = torch.zeros(nh.fp8_linear_workspace_size(0, 64, 128), dtype=torch.uint8, device=DEV)
    nh.fp8_linear(x, nh.fp8_weight(codes, scales), torch.empty((0, 64), dtype=B16, device=DEV), ws)
    nh.fp8_quantize(x, torch.empty((0, 128), dtype=torch.uint8, device=DEV),
                    torch.empty((0, 1), device=DEV))
    cfg = config(0)
    c = nh.config_from(cfg)
    up, down = experts_case(cfg, gen)
    ws = torch.zeros(nh.workspace_size(c, 0), dtype=torch.uint8, device=DEV)
    x = torch.empty((0, cfg.H), dtype=B16, device=DEV)
    y = torch.empty((0, cfg.H), device=DEV)
    idx = torch.empty((0, cfg.k), dtype=torch.int32, device=DEV)
    nh.permute(c, x, idx, torch.empty((0, cfg.k), device=DEV), ws)
    nh.forward_fp8(c, x, nh.fp8_weight(*up), nh.fp8_weight(*down), ws, y)
    assert nh.check_device(ws) == 0


def test_tensors_off_the_device_are_refused():
    codes, scales = ref.make_weight(generator(1), 1, 64, 128)
    w = nh.fp8_weight(codes, scales)
    x, y = torch.zeros((4, 128), dtype=B16, device=DEV), torch.zeros((4, 64), dtype=B16, device=DEV)
    n = nh.fp8_linear_workspace_size(4, 64, 128)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    for args in ((x.cpu(), w, y, ws), (x, w, y.cpu(), ws), (x, w, y, ws.cpu())):
        with pytest.raises(ValueError):
            nh.fp8_linear(*args)
    with pytest.raises(ValueError):
        nh.fp8_linear(x, nh.fp8_weight(*ref.make_weight(generator(1), 1, 64, 256)), y, ws)
    with pytest.raises(ValueError):
        nh.fp8_linear(x.t().contiguous().t(), w, y, ws)         # strided
    with pytest.raises(ValueError):
        nh.fp8_weight(codes.cpu(), scales)
    with pytest.raises(nh.NHMoEError):
        nh.fp8_linear(x, w, y, ws[: n - 256])
    with pytest.raises(nh.NHMoEError):
        nh.fp8_linear(torch.zeros(4 * 128 + 4, dtype=B16, device=DEV)[4:].view(4, 128), w, y, ws)


def test_linear_non_finite_rows_stay_in_their_rows():
    gen = generator(9)
    for T in (5, 40, 300):
        N, K = 272, 400
        codes, scales = ref.make_weight(gen, 1, N, K)
        w = nh.fp8_weight(codes, scales)
        x = torch.randn((T, K), generator=gen, device=DEV)
        clean = linear(x, w, N, F32)
        x[1, 7], x[T - 1, 399] = math.nan, math.inf
        y = linear(x, w, N, F32)
        keep = torch.ones(T, dtype=torch.bool, device=DEV)
        keep[[1, T - 1]] = False
        assert y[~keep].isnan().all() and torch.equal(y[keep], clean[keep])
        # a NaN code in a weight row: its feature alone
        c2 = codes.clone()
        c2.view(torch.uint8)[0, 17, 399] = 0x7F
        x[1, 7], x[T - 1, 399] = 0.0, 0.0
        y = linear(x, nh.fp8_weight(c2, scales), N, F32)
        assert y[:, 17].isnan().all() and torch.isfinite(y[:, [16, 18]]).all()


def test_linear_is_the_same_every_time():
    gen = generator(12)
    for T in (8, 700):
        codes, scales = ref.make_weight(gen, 1, 1856, 2688)
        w = nh.fp8_weight(codes, scales)
        x = torch.randn((T, 2688), generator=gen, device=DEV).to(B16)
        first = linear(x, w, 1856, F32)
        for _ in range(5):
            assert torch.equal(first, linear(x, w, 1856, F32))
        # a row's result does not depend on the rows around it
        if T > 64:
            assert torch.equal(first[:300], linear(x[:300].contiguous(), w, 1856, F32))


def test_linear_right_after_the_weights_are_made():
    """The weights come from the launch before: no load of them may run ahead of it."""
    gen = generator(13)
    N, K = 3712, 2688
    ws = torch.zeros(nh.fp8_linear_workspace_size(300, N, K), dtype=torch.uint8, device=DEV)
    codes = torch.zeros((1, N, K), dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.zeros((1, 29, 21), device=DEV)
    w = nh.fp8_weight(codes, scales)
    for T in (1, 8, 300):
        x = torch.randn((T, K), generator=gen, device=DEV).to(B16)
        y = torch.empty((T, N), dtype=B16, device=DEV)
        for rep in range(8):
            full = torch.randn((1, N, K), generator=gen, device=DEV) * 2.0 ** rep
            torch.cuda.synchronize()
            nh.fp8_quantize_weight(full, codes, scales)
            nh.fp8_linear(x, w, y, ws)
            check_product(y, ref.rows_values(x), ref.weight_values(codes[0], scales[0]), K)


def test_linear_streams_and_graphs():
    gen = generator(14)
    N, K = 1856, 2688
    codes, scales = ref.make_weight(gen, 1, N, K)
    w = nh.fp8_weight(codes, scales)
    for T in (8, 300):
        x = torch.randn((T, K), generator=gen, device=DEV).to(B16)
        want = linear(x, w, N)
        n = nh.fp8_linear_workspace_size(T, N, K)
        # two streams at once, each with its own workspace
        wss = [torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
        ys = [torch.empty((T, N), dtype=B16, device=DEV) for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(6):
            for st, y, ws in zip(streams, ys, wss):
                nh.fp8_linear(x, w, y, ws, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for y in ys)
        # two graphs that share a workspace, replayed in turn
        graphs = []
        for y in ys:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                nh.fp8_linear(x, w, y, wss[0])
            graphs.append(g)
        x2 = x.flip(0).contiguous()
        x.copy_(x2)
        for y in ys:
            y.zero_()
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want.flip(0)) for y in ys)
        assert nh.check_device(wss[0]) == 0


# -- experts -----------------------------------------------------------------------------
def config(T=8, **kw):
    base = dict(T=T, hidden_size=256, n_routed_experts=16, n_group=4, topk_group=2,
                num_experts_per_tok=4, moe_intermediate_size=192,
                moe_shared_expert_intermediate_size=320, weight_format="fp8", w_std=0.05,
                wr_std=0.05)
    base.update(kw)
    return synth.MoEConfig("fp8", **base)


def experts_case(cfg, gen):
    up = ref.make_weight(gen, cfg.E, cfg.I, cfg.H)
    down = ref.make_weight(gen, cfg.E, cfg.H, cfg.I)
    return up, down


def run_experts(cfg, x, idx, w, up, down, split=False):
    """(y_acc float32, dequantized hidden rows, hidden scales, perm_token, offsets)"""
    T, c = x.shape[0], nh.config_from(cfg)
    ws = torch.zeros(nh.workspace_size(c, T), dtype=torch.uint8, device=DEV)
    y = torch.zeros((T + 1, cfg.H), device=DEV)
    fu, fd = nh.fp8_weight(*up), nh.fp8_weight(*down)
    nh.permute(c, x, idx, w, ws)
    if split:
        nh.experts_up_fp8(c, x, fu, ws)
        nh.experts_down_fp8(c, T, fd, ws, y[:T])
    else:
        nh.forward_fp8(c, x, fu, fd, ws, y[:T])
    assert nh.check_device(ws) == 0
    assert (y[T] == 0).all()
    L, rows, kb = nh.workspace_layout(c, T), T * cfg.k, -(-cfg.I // 128)
    codes = ws[L.h:L.h + rows * cfg.I].view(rows, cfg.I)
    at = L.h + -(-rows * cfg.I // 256) * 256
    scales = ws[at:at + 4 * rows * kb].view(F32).view(rows, kb)
    token = ws[L.perm_token:L.perm_token + 4 * rows].view(torch.int32).long()
    offs = ws[L.offsets:L.offsets + 4 * (cfg.E + 1)].view(torch.int32).tolist()
    return y[:T], codes, scales, token, offs


def check_experts(cfg, x, idx, w, up, down, split=False):
    """The hidden rows are a correct quantization of values within the product's
    tolerance of the exact ones, and y is their product, weighted and summed."""
    y, codes, scales, token, offs = run_experts(cfg, x, idx, w, up, down, split)
    xv = ref.rows_values(x)
    y64 = torch.zeros((x.shape[0], cfg.H), dtype=torch.float64, device=DEV)
    tol64 = torch.zeros_like(y64)
    for e in range(cfg.E):
        r = slice(offs[e], offs[e + 1])
        t = token[r]
        if t.numel() == 0:
            continue
        uv, dv = ref.weight_values(up[0][e], up[1][e]), ref.weight_values(down[0][e], down[1][e])
        pre = xv[t] @ uv.t()
        err = (xv[t].abs() @ uv.abs().t()) * gamma(cfg.H)
        lo, hi = torch.relu(pre - err) ** 2, torch.relu(pre + err) ** 2
        lo, hi = lo * (1 - 2.0 ** -22), hi * (1 + 2.0 ** -22)     # the square's rounding
        pad = torch.nn.functional.pad
        kb = scales.shape[1]
        blk = lambda v: pad(v, (0, kb * 128 - cfg.I)).view(-1, kb, 128).amax(dim=2)  # noqa: E731
        s = scales[r].double()
        assert ((s >= ref.block_scale(blk(lo))) & (s <= ref.block_scale(blk(hi)))).all()
        sp = ref.spread(s, cfg.I)
        h = ref.decode(codes[r])
        # nearest_e4m3 is monotone: the code lies between those of the two ends
        assert (h >= ref.nearest_e4m3((lo / sp).clamp(max=448))).all()
        assert (h <= ref.nearest_e4m3((hi / sp).clamp(max=448))).all()
        h = h * sp
        wt = torch.zeros(t.numel(), 1, dtype=torch.float64, device=DEV)
        slot = (idx[t] == e)
        wt[:, 0] = (w[t].double() * slot).sum(dim=1)
        y64.index_add_(0, t, wt * (h @ dv.t()))
        # one rounding more for the weight, and k adds into y_acc
        tol64.index_add_(0, t, wt.abs() * (h @ dv.abs().t()) * (gamma(cfg.I) + (cfg.k + 2) * 2.0 ** -24))
    assert ((y.double() - y64).abs() <= tol64 + 1e-30).all()
    return y


def routing(T, E, k, gen, skew=0.0):
    score = torch.randn((T, E), generator=gen, device=DEV) + skew * torch.randn(
        E, generator=gen, device=DEV)
    idx = score.topk(k, dim=1).indices.int()
    w = torch.rand((T, k), generator=gen, device=DEV) + 0.1
    return idx, w


@pytest.mark.parametrize("T", [1, 2, 8, 9, 15, 16, 17, 32, 33, 65, 135, 200, 300, 515, 516, 1500])
@pytest.mark.parametrize("kw", [
    dict(), dict(hidden_size=64, moe_intermediate_size=64),
    dict(hidden_size=704, moe_intermediate_size=576, n_routed_experts=8, num_experts_per_tok=2),
    dict(hidden_size=2688, moe_intermediate_size=1856, n_routed_experts=4, n_group=1, topk_group=1,
         num_experts_per_tok=3)])
def test_experts(T, kw):
    gen = generator(T)
    cfg = config(T, **kw)
    up, down = experts_case(cfg, gen)
    idx, w = routing(T, cfg.E, cfg.k, gen, skew=1.0)
    x = torch.randn((T, cfg.H), generator=gen, device=DEV).to(B16)
    a = check_experts(cfg, x, idx, w, up, down)
    b = check_experts(cfg, x, idx, w, up, down, split=True)
    # the same up to the order of the float32 adds of a token's k rows
    assert ((a - b).abs() <= 2.0 ** -22 * cfg.k * (a.abs().amax() + b.abs())).all()


@pytest.mark.parametrize("T", [1, 8, 9, 32, 33, 64, 65, 300, 321, 1500])
@pytest.mark.parametrize("H,S", [(256, 320), (64, 64), (2688, 3712)])
def test_shared(T, H, S):
    """Each hidden value lies between the codes of its exact value's two ends, and y between
    the products of those ends, but for the rounding of S terms and the add."""
    gen = generator(T + S)
    cfg = config(T, hidden_size=H, moe_shared_expert_intermediate_size=S)
    c = nh.config_from(cfg)
    su, sd = ref.make_weight(gen, 1, S, H), ref.make_weight(gen, 1, H, S)
    x = torch.randn((T, H), generator=gen, device=DEV).to(B16)
    ws = torch.zeros(nh.shared_workspace_size(c, T), dtype=torch.uint8, device=DEV)
    y = torch.full((T + 1, H), float("nan"), device=DEV)
    nh.shared_store_fp8(c, x, nh.fp8_weight(*su), nh.fp8_weight(*sd), y[:T], ws)
    y0 = torch.randn((T + 1, H), generator=gen, device=DEV)
    y1 = y0.clone()
    nh.shared_fp8(c, x, nh.fp8_weight(*su), nh.fp8_weight(*sd), y1[:T], ws)
    assert nh.check_device(ws) == 0
    assert y[T].isnan().all() and torch.equal(y0[T], y1[T])
    uv, dv = ref.weight_values(su[0][0], su[1][0]), ref.weight_values(sd[0][0], sd[1][0])
    xv = ref.rows_values(x)
    pre, err = xv @ uv.t(), (xv.abs() @ uv.abs().t()) * gamma(H)
    ends = (torch.relu(pre - err) ** 2 * (1 - 2.0 ** -22), torch.relu(pre + err) ** 2 * (1 + 2.0 ** -22))
    kb = -(-S // 128)
    pad = torch.nn.functional.pad
    sp = [ref.spread(ref.block_scale(pad(v, (0, kb * 128 - S)).view(T, kb, 128).amax(dim=2)), S)
          for v in ends]
    code = lambda v, s: ref.nearest_e4m3((v / s).clamp(max=448)) * s  # noqa: E731
    lo = torch.minimum(code(ends[0], sp[0]), code(ends[0], sp[1]))
    hi = torch.maximum(code(ends[1], sp[0]), code(ends[1], sp[1]))
    pos, neg = dv.clamp(min=0).t(), dv.clamp(max=0).t()
    tol = (hi @ dv.abs().t()) * gamma(S) + 1e-30
    low, high = lo @ pos + hi @ neg - tol, hi @ pos + lo @ neg + tol
    assert ((y[:T] >= low) & (y[:T] <= high)).all()
    add = y0[:T].double()
    edge = 2.0 ** -24 * (add.abs() + torch.maximum(low.abs(), high.abs()))
    assert ((y1[:T] >= add + low - edge) & (y1[:T] <= add + high + edge)).all()


def test_experts_with_weights_past_32_bits():
    """The last expert's codes lie past 2^32 bytes."""
    cfg = config(5, hidden_size=4224, moe_intermediate_size=2048, n_routed_experts=512,
                 n_group=1, topk_group=1, num_experts_per_tok=2)
    gen = generator(31)

    def big(rows, cols):
        codes = torch.zeros((cfg.E, rows, cols), dtype=torch.uint8, device=DEV)
        scales = torch.ones((cfg.E, -(-rows // 128), -(-cols // 128)), device=DEV)
        for e in (0, 3, cfg.E - 1):
            c, s = ref.make_weight(gen, 1, rows, cols)
            codes[e], scales[e] = c[0].view(torch.uint8), s[0]
        return codes, scales

    up, down = big(cfg.I, cfg.H), big(cfg.H, cfg.I)
    for T in (5, 300):
        idx = torch.tensor([[cfg.E - 1, 3]], dtype=torch.int32, device=DEV).repeat(T, 1)
        idx[1:3, 1] = 0
        w = torch.rand((T, 2), generator=gen, device=DEV)
        x = torch.randn((T, cfg.H), generator=gen, device=DEV).to(B16)
        check_experts(cfg, x, idx, w, up, down)


@pytest.mark.parametrize("T", [5, 32, 40, 700])
def test_every_token_takes_the_same_experts(T):
    """Whole batches in two experts, none in the others; slots with weight 0."""
    gen = generator(T)
    cfg = config(T, num_experts_per_tok=2)
    up, down = experts_case(cfg, gen)
    idx = torch.tensor([[11, 2]], dtype=torch.int32, device=DEV).repeat(T, 1)
    w = torch.rand((T, 2), generator=gen, device=DEV)
    w[::3, 1] = 0.0
    x = torch.randn((T, cfg.H), generator=gen, device=DEV).to(B16)
    check_experts(cfg, x, idx, w, up, down)


@pytest.mark.parametrize("T", [4, 32, 90])
def test_an_expert_named_twice(T):
    gen = generator(T)
    cfg = config(T)
    up, down = experts_case(cfg, gen)
    idx = torch.randint(0, 3, (T, 4), generator=gen, device=DEV).int()
    w = torch.rand((T, 4), generator=gen, device=DEV)
    x = torch.randn((T, cfg.H), generator=gen, device=DEV).to(B16)
    y, *_ = run_experts(cfg, x, idx, w, up, down)
    # the same token by one slot with the summed weight
    uniq = torch.zeros((T, 3), device=DEV).scatter_add_(1, idx.long(), w)
    c3 = cfg.replace(num_experts_per_tok=3)
    i3 = torch.arange(3, dtype=torch.int32, device=DEV).repeat(T, 1)
    want, *_ = run_experts(c3, x, i3, uniq, up, down)
    # each slot's weighted row is rounded on its own: one rounding a slot and add
    assert ((y - want).abs() <= 2.0 ** -20 * (want.abs().amax() + want.abs())).all()


def test_ids_out_of_range_are_reported_and_dropped():
    gen = generator(3)
    for T in (6, 300):
        cfg = config(T)
        c = nh.config_from(cfg)
        up, down = experts_case(cfg, gen)
        idx, w = routing(T, cfg.E, cfg.k, gen)
        x = torch.randn((T, cfg.H), generator=gen, device=DEV).to(B16)
        bad = idx.clone()
        bad[1, 2], bad[T - 1, 0] = cfg.E, -1
        ws = torch.zeros(nh.workspace_size(c, T), dtype=torch.uint8, device=DEV)
        y = torch.zeros((T, cfg.H), device=DEV)
        fu, fd = nh.fp8_weight(*up), nh.fp8_weight(*down)
        nh.permute(c, x, bad, w, ws)
        nh.forward_fp8(c, x, fu, fd, ws, y)
        assert nh.check_device(ws) == nh.NH_ERR_DEVICE_CHECK
        w0 = w.clone()
        w0[1, 2], w0[T - 1, 0] = 0.0, 0.0
        want, *_ = run_experts(cfg, x, idx, w0, up, down)
        assert ((y - want).abs() <= 2.0 ** -20 * (want.abs().amax() + want.abs())).all()


def test_experts_repeat_and_graph():
    gen = generator(21)
    for T in (8, 400):
        cfg = config(T, n_routed_experts=32, n_group=4)
        c = nh.config_from(cfg)
        up, down = experts_case(cfg, gen)
        fu, fd = nh.fp8_weight(*up), nh.fp8_weight(*down)
        idx, w = routing(T, cfg.E, cfg.k, gen)
        x = torch.randn((T, cfg.H), generator=gen, device=DEV).to(B16)
        ws = torch.zeros(nh.workspace_size(c, T), dtype=torch.uint8, device=DEV)
        y_acc = torch.zeros((T, cfg.H), device=DEV)
        y = torch.empty((T, cfg.H), dtype=B16, device=DEV)

        def go():
            nh.zero_acc(c, T, y_acc)
            nh.permute(c, x, idx, w, ws)
            nh.forward_fp8(c, x, fu, fd, ws, y_acc)
            nh.finalize(c, T, y_acc, y)

        go()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go()
        x.copy_(x.flip(0))
        idx.copy_(idx.flip(0))
        w.copy_(w.flip(0))
        for _ in range(3):
            g.replay()
        assert nh.check_device(ws) == 0
        want = check_experts(cfg, x, idx, w, up, down)
        # float32 adds in another order, then one rounding each
        assert ((y.float() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-5 * want.abs().amax()).all()


def test_products_on_several_streams_at_once():
    """A small-batch and a large-batch experts call, a linear call and a GEMV side by
    side: kernels that share SMs and tensor memory, each with its own workspace."""
    gen = generator(41)
    small, large = config(8, hidden_size=704, moe_intermediate_size=576), config(6000, n_routed_experts=8)
    jobs = []
    for cfg in (small, large):
        c = nh.config_from(cfg)
        up, down = experts_case(cfg, gen)
        fu, fd = nh.fp8_weight(*up), nh.fp8_weight(*down)
        idx, w = routing(cfg.T, cfg.E, cfg.k, gen)
        x = torch.randn((cfg.T, cfg.H), generator=gen, device=DEV).to(B16)
        ws = torch.zeros(nh.workspace_size(c, cfg.T), dtype=torch.uint8, device=DEV)
        y = torch.zeros((cfg.T, cfg.H), device=DEV)

        def experts(stream=None, c=c, T=cfg.T, fu=fu, fd=fd, idx=idx, w=w, x=x, ws=ws, y=y):
            nh.zero_acc(c, T, y, stream=stream)
            nh.permute(c, x, idx, w, ws, stream=stream)
            nh.forward_fp8(c, x, fu, fd, ws, y, stream=stream)
        jobs.append((experts, y, ws, False))
    for T in (4, 900):
        wt = nh.fp8_weight(*ref.make_weight(gen, 1, 1856, 2688))
        x = torch.randn((T, 2688), generator=gen, device=DEV).to(B16)
        y = torch.zeros((T, 1856), dtype=B16, device=DEV)
        ws = torch.zeros(nh.fp8_linear_workspace_size(T, 1856, 2688), dtype=torch.uint8, device=DEV)
        jobs.append((lambda stream=None, x=x, wt=wt, y=y, ws=ws: nh.fp8_linear(x, wt, y, ws, stream=stream),
                     y, ws, True))
    want = []
    for job, y, _, _ in jobs:
        job()
        torch.cuda.synchronize()
        want.append(y.clone())
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(12):
        for (job, *_), st in zip(jobs, streams):
            job(st)
    torch.cuda.synchronize()
    for (_, y, ws, same_bits), ref_y in zip(jobs, want):
        assert nh.check_device(ws) == 0
        if same_bits:
            assert torch.equal(y, ref_y)
        else:      # up to the order of the float32 adds of a token's k rows
            assert ((y - ref_y).abs() <= 2.0 ** -20 * (ref_y.abs().amax() + ref_y.abs())).all()


# -- the block ---------------------------------------------------------------------------
def block_and_parts(cfg, seed=0, bias=False):
    gen = generator(seed)
    he, f8 = cfg.HE, {}
    f8["up"] = ref.make_weight(gen, cfg.E, cfg.I, he)
    f8["down"] = ref.make_weight(gen, cfg.E, he, cfg.I)
    if cfg.n_shared_experts:
        f8["shared_up"] = ref.make_weight(gen, 1, cfg.S, cfg.H)
        f8["shared_down"] = ref.make_weight(gen, 1, cfg.H, cfg.S)
    wr = torch.randn((cfg.E, cfg.H), generator=gen, device=DEV) * cfg.H ** -0.5
    b = torch.randn(cfg.E, generator=gen, device=DEV) * 0.05 if bias else None
    fc = [None, None]
    if cfg.latent_size:
        fc = [(torch.randn((cfg.latent_size, cfg.H), generator=gen, device=DEV) * cfg.H ** -0.5).to(B16),
              (torch.randn((cfg.H, cfg.latent_size), generator=gen, device=DEV) *
               cfg.latent_size ** -0.5).to(B16)]
    blk = nh.NemotronHMoE(cfg, wr, fp8=f8, bias=b, w_latent_fc1=fc[0], w_latent_fc2=fc[1])
    return blk, f8, wr, b, fc, gen


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [1, 8, 32, 33, 64, 300])
@pytest.mark.parametrize("latent", [0, 128])
def test_block(T, score, latent):
    """Routing by the block's own choice; the products' part of the error is far below what
    a hidden code on the other side of an edge adds, which is bounded in the mean: a share
    of 8 gamma of the codes moves by a step of at most 2^-3, so y's relative error stays
    under 2^-3 sqrt(8 gamma) = 0.2 %, beside bf16's 2^-8."""
    cfg = config(T, scoring_func=score, latent_size=latent)
    blk, f8, wr, b, fc, gen = block_and_parts(cfg, T, bias=True)
    x = torch.randn((T, cfg.H), generator=gen, device=DEV).to(B16)
    y = blk.forward(x)
    assert blk.check(T) == 0
    bufs = blk.buffers(T)
    idx, w = bufs.topk_idx.long(), bufs.topk_w
    logits = (x.double() @ wr.double().t())
    widx, ww = ref.gate(logits, b, cfg.n_group, cfg.topk_group, cfg.k, score == "softmax", True,
                        False, cfg.routed_scaling_factor)
    # float32 logits may choose otherwise only where two scores nearly tie
    sc = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    sc = sc + b.double()
    differ = (idx != widx).any(dim=1)
    assert ((sc.gather(1, idx) - sc.gather(1, widx)).abs()[differ] < 1e-5).all()
    agree = ~differ
    assert ((w.double() - ww).abs()[agree] <= 1e-4 * ww[agree]).all()
    if latent:
        x_lat = bufs.x_lat
        want = x.double() @ fc[0].double().t()
        assert ((x_lat.double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-4).all()
        routed = ref.experts(x_lat, idx, w, f8["up"], f8["down"])
        routed = bufs.y_lat.double() @ fc[1].double().t() if _near(bufs.y_lat, routed) else None
    else:
        routed = ref.experts(x, idx, w, f8["up"], f8["down"])
    h = torch.relu(ref.rows_values(x) @ ref.weight_values(f8["shared_up"][0][0], f8["shared_up"][1][0]).t()) ** 2
    shared = ref.rows_values(h) @ ref.weight_values(f8["shared_down"][0][0], f8["shared_down"][1][0]).t()
    assert _near(y, routed + shared)
    # host input through the captured graph
    yh = blk(x.cpu())
    assert _near(yh.cuda(), routed + shared)


def _near(y, want):
    rel = ((y.double() - want).norm() / want.norm()).item()
    assert rel <= 2.0 ** -8 + 0.002, rel
    return True


@pytest.mark.parametrize("T", [8, 40, 700])
@pytest.mark.parametrize("world", [2, 3])
def test_tensor_parallel_ranks_sum_to_the_block(T, world):
    """Rank by rank on one GPU: hidden codes are those of the whole block (the cuts lie on
    scale blocks), so the float32 partials add up to its accumulator but for the order of
    the sums: E k K blocks' roundings of the terms' magnitudes."""
    from non_gated_relu_b200 import tp
    cfg = config(T, moe_intermediate_size=448, moe_shared_expert_intermediate_size=576)
    blk, f8, wr, b, _, gen = block_and_parts(cfg, T, bias=True)
    x = torch.randn((T, cfg.H), generator=gen, device=DEV).to(B16)
    whole = blk.forward(x, partial=True).clone()
    parts = []
    for r in range(world):
        rank = tp.TPNemotronHMoE(cfg, wr, fp8=f8, bias=b, world=world, rank=r)
        parts.append(rank.partial(x).clone())
        assert rank.block.check(T) == 0
    total = sum(parts)
    size = sum(p.abs() for p in parts) + whole.abs().amax()
    assert ((total - whole).abs() <= 2.0 ** -18 * size).all()
    assert _near(rank.output(total), whole.double())


def test_block_needs_its_weights():
    cfg = config(8)
    blk, f8, wr, *_ = block_and_parts(cfg)
    with pytest.raises(ValueError):
        nh.NemotronHMoE(cfg, wr)
    with pytest.raises(ValueError):
        nh.NemotronHMoE(cfg, wr, fp8={"up": f8["up"], "down": f8["down"]})
    with pytest.raises(ValueError):
        nh.NemotronHMoE(cfg, wr, fp8={**f8, "down": f8["up"]})
    with pytest.raises(ValueError):
        nh.NemotronHMoE(cfg.replace(scoring_func="relu"), wr, fp8=f8)


def test_weights_quantized_here_serve_the_block():
    """bf16 weights through fp8_quantize_weight give a block near the bf16 one: codes are
    within 2^-4 of each weight and activation, and errors of K terms add as their root."""
    cfg = config(16)
    gen = generator(5)
    r = lambda *s: (torch.randn(s, generator=gen, device=DEV) * 0.05).to(B16)  # noqa: E731
    up, down, su, sd = r(cfg.E, cfg.I, cfg.H), r(cfg.E, cfg.H, cfg.I), r(cfg.S, cfg.H), r(cfg.H, cfg.S)
    wr = torch.randn((cfg.E, cfg.H), generator=gen, device=DEV) * 0.05
    a = nh.NemotronHMoE(cfg.replace(weight_format="native"), wr, up, down, su, sd)
    q = nh.fp8_quantize_weight
    b = nh.NemotronHMoE(cfg, wr, fp8={"up": q(up), "down": q(down), "shared_up": q(su[None]),
                                      "shared_down": q(sd[None])})
    x = torch.randn((16, cfg.H), generator=gen, device=DEV).to(B16)
    ya, yb = a.forward(x).double(), b.forward(x).double()
    # five roundings to E4M3 a path (x, W_up twice through the square, h, W_down), 2^-4 each
    assert ((ya - yb).norm() / ya.norm()).item() <= 5 * 2.0 ** -4


# -- repeated calls ----------------------------------------------------------------------
@pytest.mark.parametrize("T,kw", [
    (1, {}), (8, {}), (32, {}), (33, {}), (301, {}), (1500, {}),
    (4000, dict(n_routed_experts=8, n_group=1, topk_group=1, num_experts_per_tok=6)),
    (700, dict(n_routed_experts=64, n_group=1, topk_group=1, num_experts_per_tok=20))])
def test_experts_repeat_bit_for_bit(T, kw):
    """A token's k rows meet in the order of its slots, whatever order the tiles end in: the
    same bits from every call, also beside a call on another stream, and in a graph."""
    gen = generator(T + 7)
    cfg = config(T, **kw)
    c = nh.config_from(cfg)
    up, down = experts_case(cfg, gen)
    fu, fd = nh.fp8_weight(*up), nh.fp8_weight(*down)
    idx, w = routing(T, cfg.E, cfg.k, gen, skew=1.0)
    x = torch.randn((T, cfg.H), generator=gen, device=DEV).to(B16)
    sets = [(torch.zeros(nh.workspace_size(c, T), dtype=torch.uint8, device=DEV),
             torch.zeros((T, cfg.H), device=DEV)) for _ in range(2)]

    def go(ws, y, stream=None):
        nh.zero_acc(c, T, y, stream=stream)
        nh.permute(c, x, idx, w, ws, stream=stream)
        nh.forward_fp8(c, x, fu, fd, ws, y, stream=stream)

    go(*sets[0])
    want = sets[0][1].clone()
    assert want.abs().amax() > 0
    for _ in range(8):
        go(*sets[0])
        assert torch.equal(sets[0][1], want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(8):
        for (ws, y), st in zip(sets, streams):
            go(ws, y, st)
    torch.cuda.synchronize()
    for ws, y in sets:
        assert nh.check_device(ws) == 0 and torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(*sets[0])
    for _ in range(4):
        sets[0][1].fill_(3.0)
        g.replay()
        assert torch.equal(sets[0][1], want)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [8, 32, 40, 700])
def test_block_repeats_bit_for_bit(T, score):
    """Routed and shared expert add once each to an accumulator that starts at zero (or the
    routed one to the shared one's values): no order between them changes a bit."""
    cfg = config(T, scoring_func=score)
    blk, *_, gen = block_and_parts(cfg, T, bias=True)
    x = torch.randn((T, cfg.H), generator=gen, device=DEV).to(B16)
    want = blk.forward(x, partial=True).clone()
    for _ in range(10):
        assert torch.equal(blk.forward(x, partial=True), want)
    assert blk.check(T) == 0


def test_experts_add_to_what_is_there():
    gen = generator(77)
    for T in (3, 200, 1500):
        cfg = config(T)
        c = nh.config_from(cfg)
        up, down = experts_case(cfg, gen)
        idx, w = routing(T, cfg.E, cfg.k, gen)
        x = torch.randn((T, cfg.H), generator=gen, device=DEV).to(B16)
        alone, *_ = run_experts(cfg, x, idx, w, up, down)
        start = torch.randn((T, cfg.H), generator=gen, device=DEV)
        y, ws = start.clone(), torch.zeros(nh.workspace_size(c, T), dtype=torch.uint8, device=DEV)
        nh.permute(c, x, idx, w, ws)
        nh.forward_fp8(c, x, nh.fp8_weight(*up), nh.fp8_weight(*down), ws, y)
        assert torch.equal(y, start + alone)      # one float32 add


# -- launches that follow one another closely ----------------------------------------------
@pytest.mark.parametrize("T", [9, 16, 32, 33, 64, 700, 2000])
def test_linear_right_after_the_weights_are_made_any_kernel(T):
    """No weight or scale is read ahead of the kernel that makes it: the GEMV behind the
    quantization, small tiles and pairs."""
    gen = generator(T + 50)
    N, K = 512, 1024
    x = torch.randn((T, K), generator=gen, device=DEV).to(B16)
    sets = [torch.randn((1, N, K), generator=gen, device=DEV).to(B16) * 2.0 ** i for i in range(4)]
    codes = torch.empty((1, N, K), dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty((1, N // 128, K // 128), device=DEV)
    w = nh.fp8_weight(codes, scales)
    ws = torch.zeros(nh.fp8_linear_workspace_size(T, N, K), dtype=torch.uint8, device=DEV)
    want = []
    for v in sets:
        nh.fp8_quantize_weight(v, codes, scales)
        torch.cuda.synchronize()
        y = torch.empty((T, N), device=DEV)
        nh.fp8_linear(x, w, y, ws)
        torch.cuda.synchronize()
        want.append(y)
    got = [torch.empty((T, N), device=DEV) for _ in range(24)]
    for i, y in enumerate(got):
        nh.fp8_quantize_weight(sets[i % 4], codes, scales)
        nh.fp8_linear(x, w, y, ws)
    torch.cuda.synchronize()
    assert nh.check_device(ws) == 0
    assert all(torch.equal(y, want[i % 4]) for i, y in enumerate(got))


@pytest.mark.parametrize("T", [1, 8, 32, 33, 200, 1500])
@pytest.mark.parametrize("split", [False, True])
def test_experts_right_after_weights_and_routing_change(T, split):
    """Weights rewritten and the permute made anew directly before each call, on one
    workspace: neither the weights nor the tile table nor the scales of the call before
    are seen."""
    gen = generator(T + 60)
    cfg = config(T)
    c = nh.config_from(cfg)
    E, H, I = cfg.E, cfg.H, cfg.I
    r = lambda *s: torch.randn(s, generator=gen, device=DEV).to(B16)  # noqa: E731
    sets = []
    for i in range(3):
        idx, w = routing(T, E, cfg.k, gen, skew=2.0)
        sets.append((r(E, I, H) * 2.0 ** -i, r(E, H, I) * 2.0 ** i, r(T, H), idx, w))
    up = (torch.empty((E, I, H), dtype=torch.uint8, device=DEV),
          torch.empty((E, -(-I // 128), -(-H // 128)), device=DEV))
    down = (torch.empty((E, H, I), dtype=torch.uint8, device=DEV),
            torch.empty((E, -(-H // 128), -(-I // 128)), device=DEV))
    fu, fd = nh.fp8_weight(*up), nh.fp8_weight(*down)
    ws = torch.zeros(nh.workspace_size(c, T), dtype=torch.uint8, device=DEV)

    def go(s, y, apart):
        pause = torch.cuda.synchronize if apart else (lambda: None)
        uv, dv, x, idx, w = s
        nh.zero_acc(c, T, y)
        nh.permute(c, x, idx, w, ws)
        pause()
        if split:
            nh.fp8_quantize_weight(uv, *up)
            pause()
            nh.experts_up_fp8(c, x, fu, ws)
            pause()
            nh.fp8_quantize_weight(dv, *down)
            pause()
            nh.experts_down_fp8(c, T, fd, ws, y)
        else:
            nh.fp8_quantize_weight(uv, *up)
            nh.fp8_quantize_weight(dv, *down)
            pause()
            nh.forward_fp8(c, x, fu, fd, ws, y)
        pause()

    want = [torch.empty((T, H), device=DEV) for _ in sets]
    for s, y in zip(sets, want):
        go(s, y, True)
    got = [torch.empty((T, H), device=DEV) for _ in range(18)]
    for i, y in enumerate(got):
        go(sets[i % 3], y, False)
    torch.cuda.synchronize()
    assert nh.check_device(ws) == 0
    assert all(torch.equal(y, want[i % 3]) for i, y in enumerate(got))


@pytest.mark.parametrize("T", [1, 8, 9, 32, 33, 300])
def test_shared_right_after_the_weights_are_made(T):
    gen = generator(T + 70)
    cfg = config(T)
    c = nh.config_from(cfg)
    H, S = cfg.H, cfg.S
    r = lambda *s: torch.randn(s, generator=gen, device=DEV).to(B16)  # noqa: E731
    sets = [(r(1, S, H) * 2.0 ** -i, r(1, H, S) * 2.0 ** i, r(T, H)) for i in range(3)]
    su = (torch.empty((1, S, H), dtype=torch.uint8, device=DEV),
          torch.empty((1, -(-S // 128), -(-H // 128)), device=DEV))
    sd = (torch.empty((1, H, S), dtype=torch.uint8, device=DEV),
          torch.empty((1, -(-H // 128), -(-S // 128)), device=DEV))
    fu, fd = nh.fp8_weight(*su), nh.fp8_weight(*sd)
    ws = torch.zeros(nh.shared_workspace_size(c, T), dtype=torch.uint8, device=DEV)

    def go(s, y, apart):
        nh.fp8_quantize_weight(s[0], *su)
        nh.fp8_quantize_weight(s[1], *sd)
        if apart:
            torch.cuda.synchronize()
        nh.shared_store_fp8(c, s[2], fu, fd, y, ws)
        if apart:
            torch.cuda.synchronize()

    want = [torch.empty((T, H), device=DEV) for _ in sets]
    for s, y in zip(sets, want):
        go(s, y, True)
    got = [torch.empty((T, H), device=DEV) for _ in range(18)]
    for i, y in enumerate(got):
        go(sets[i % 3], y, False)
    torch.cuda.synchronize()
    assert nh.check_device(ws) == 0
    assert all(torch.equal(y, want[i % 3]) for i, y in enumerate(got))


@pytest.mark.parametrize("handle", [False, True])
def test_weights_allocated_for_another_stream(handle):
    """Codes and scales that the call allocates may lie where the current stream still works
    for a tensor that is gone: its last write must not reach them."""
    gen = generator(83)
    w = torch.randn((1, 2048, 4096), generator=gen, device=DEV)
    want = nh.fp8_quantize_weight(w)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    old = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device=DEV) for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)            # some 20 ms of the current stream
    for t in old:
        t.fill_(0x55)
    del t, old
    got = nh.fp8_quantize_weight(w, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def test_experts_with_rows_past_32_bits():
    """Codes, down-projection rows and their offsets past 2^32: a batch that repeats one of
    1000 tokens gives the small batch's result in every repetition, bit for bit (both run
    on tiles of the same height, and a row's sums do not depend on its place)."""
    P, R = 1000, 270
    cfg = config(P, hidden_size=1024, moe_intermediate_size=64, n_routed_experts=16, n_group=1,
                 topk_group=1, num_experts_per_tok=16)
    assert R * P * cfg.k * cfg.H > 2 ** 32
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("needs 60 GB")
    c, gen = nh.config_from(cfg), generator(91)
    assert nh.workspace_layout(c, P).tile_rows == nh.workspace_layout(c, P * R).tile_rows
    up, down = experts_case(cfg, gen)
    idx, w = routing(P, cfg.E, cfg.k, gen)
    x = torch.randn((P, cfg.H), generator=gen, device=DEV).to(B16)
    want, *_ = run_experts(cfg, x, idx, w, up, down)
    T = P * R
    ws = torch.zeros(nh.workspace_size(c, T), dtype=torch.uint8, device=DEV)
    y = torch.zeros((T, cfg.H), device=DEV)
    xs, idxs, wts = x.repeat(R, 1), idx.repeat(R, 1), w.repeat(R, 1)
    nh.permute(c, xs, idxs, wts, ws)
    nh.forward_fp8(c, xs, nh.fp8_weight(*up), nh.fp8_weight(*down), ws, y)
    assert nh.check_device(ws) == 0
    assert (y.view(R, P, cfg.H) == want).all()
