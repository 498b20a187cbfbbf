"""The gate (choice and weights from router logits) and its gradient against their
definitions in 64 bits (fp8_util.gate, autograd of fp8_util.gate_weights) and against
differences of the kernel's own weights.

Tolerances.  A share is expf(l_j - top) over a sum: the rounding of l_j - top moves it by
|l_j - top| 2^-24, expf by 2 ulp = 2^-22, the sum of up to 512 by (16 + 5) 2^-24 (16 per
lane, 5 shuffles), divides and the factor by 3 roundings: rel <= (|l_j - top| + 32) 2^-24;
doubled below.  Raw sigmoids are closer.  Weights under 2^-120 may be flushed."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import non_gated_relu_b200 as nh  # noqa: E402
import fp8_util as ref  # noqa: E402

DEV = "cuda"


def run(logits, bias, G, tg, k, softmax, norm, top2, alpha=2.5):
    T, E = logits.shape
    cfg = nh.gate_config(E, k, G, tg, norm, alpha, "softmax" if softmax else "sigmoid",
                         "top2" if top2 else "max",
                         "bf16" if logits.dtype == torch.bfloat16 else "f32")
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T + 1, k), -7.0, device=DEV)
    nh.gate(cfg, logits, bias, idx[:T], w[:T])
    torch.cuda.synchronize()
    assert (idx[T] == -7).all() and (w[T] == -7).all(), "wrote past the last token"
    return cfg, idx[:T].long(), w[:T]


def check_w(w, want, lsel):
    l = ref.clean(lsel)
    top = l.amax(dim=1, keepdim=True)
    far = torch.where(l == -math.inf, 0.0, (top - l).nan_to_num(0.0)).clamp(max=200.0)
    tol = want.abs() * (far + 32) * 2.0 ** -23 + 2.0 ** -118
    bad = (w.double() - want).abs() > tol
    assert not bad.any(), (w[bad][:4], want[bad][:4])


def check(logits, bias, G, tg, k, softmax, norm, top2):
    _, idx, w = run(logits, bias, G, tg, k, softmax, norm, top2)
    widx, ww = ref.gate(logits, bias, G, tg, k, softmax, norm, top2, 2.5)
    bad = (idx != widx).any(dim=1)
    assert not bad.any(), (int(bad.sum()), idx[bad][:2], widx[bad][:2])
    check_w(w, ww, logits.gather(1, idx))


# (E, G, tg, k): whole lanes per group, groups across lanes, one group, all groups kept,
# every candidate taken, the largest of each
SHAPES = [(1, 1, 1, 1), (5, 1, 1, 5), (16, 4, 1, 2), (24, 3, 2, 8), (64, 8, 3, 6), (100, 10, 4, 8),
          (128, 8, 1, 6), (128, 1, 1, 6), (160, 8, 3, 6), (256, 8, 4, 8), (256, 8, 8, 8),
          (257, 1, 1, 3), (320, 64, 7, 8), (384, 2, 1, 32), (512, 64, 64, 32), (512, 16, 5, 8),
          (64, 64, 6, 6), (40, 20, 9, 18)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_choice_and_weights(shape, softmax, bias):
    E, G, tg, k = shape
    gen = torch.Generator(device=DEV).manual_seed(E * 7 + G + 2 * softmax + bias)
    for T, dtype, norm, top2, std in ((67, torch.float32, True, True, 1.5),
                                      (9, torch.bfloat16, False, False, 3.0),
                                      (1, torch.float32, False, True, 0.3),
                                      (130, torch.bfloat16, True, True, 0.5)):
        if top2 and E // G < 2:
            top2 = False
        logits = (torch.randn((T, E), generator=gen, device=DEV) * std).to(dtype)
        b = torch.randn(E, generator=gen, device=DEV) * 0.1 if bias else None
        check(logits, b, G, tg, k, softmax, norm, top2)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("top2", [False, True])
def test_ties_go_to_the_lowest_id(softmax, top2):
    gen = torch.Generator(device=DEV).manual_seed(3)
    for E, G, tg, k in ((128, 8, 3, 6), (160, 8, 3, 6), (512, 16, 5, 32)):
        logits = torch.randint(-2, 3, (96, E), generator=gen, device=DEV).float()
        logits[0] = 0.0
        logits[1] = -0.0
        logits[2, ::2] = -0.0                              # +0 and -0 tie
        for b in (None, torch.zeros(E, device=DEV),
                  torch.randint(0, 2, (E,), generator=gen, device=DEV).float() / 4):
            check(logits, b, G, tg, k, softmax, True, top2)


@pytest.mark.parametrize("softmax", [False, True])
def test_neighbours_closer_than_float32_scores(softmax):
    """Logits one float32 step apart where the score is flat: their float32 scores
    agree, or come out in the other order, and the exact scores decide."""
    gen = torch.Generator(device=DEV).manual_seed(11)
    E, G, tg, k = 128, 8, 3, 6
    base = 6.0 + torch.randint(0, 3, (200, E), generator=gen, device=DEV).float() * 0.25
    step = torch.randint(-3, 4, (200, E), generator=gen, device=DEV).int()
    logits = (base.view(torch.int32) + step).view(torch.float32)
    gap = torch.rand(E, generator=gen, device=DEV) * 2.0 ** -22
    for b in (torch.zeros(E, device=DEV), gap):
        check(logits, b, G, tg, k, softmax, True, True)
        check(logits, b, 1, 1, k, softmax, True, False)
    check(logits, None, G, tg, k, softmax, False, True)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("top2", [False, True])
def test_biases_near_the_ends_of_float32(softmax, top2):
    """Group values that overflow float32 are told apart all the same; a bias of +inf (not
    of the documented values) still gives k different experts, those first."""
    gen = torch.Generator(device=DEV).manual_seed(8)
    inf, big = math.inf, 3.2e38
    for E, G, tg, k in ((64, 8, 3, 6), (100, 10, 4, 8), (128, 1, 1, 6)):
        x = torch.randn((50, E), generator=gen, device=DEV)
        x[:5, ::3] = -inf
        x[5, E // 2:] = -inf
        for _ in range(4):
            at = torch.randint(0, 5, (E,), generator=gen, device=DEV)
            step = 1 + torch.rand(E, generator=gen, device=DEV) * 2.0 ** -6
            b = torch.tensor([big, -big, 2.9e38, 0.0, 1.0], device=DEV)[at] * step
            check(x, b, G, tg, k, softmax, True, top2)
        b = torch.zeros(E, device=DEV)
        b[3:3 + k] = inf
        _, idx, w = run(x, b, 1, 1, k, softmax, True, False)
        free = x[:, 3:3 + k].isfinite().all(dim=1)
        assert (idx[free] == torch.arange(3, 3 + k, device=DEV)).all()
        assert all(r.unique().numel() == k for r in idx) and w.isfinite().all()


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_masked_and_non_finite_rows(softmax, bias, norm):
    E, G, tg, k = 32, 4, 2, 6
    gen = torch.Generator(device=DEV).manual_seed(5)
    inf, low = math.inf, torch.finfo(torch.float32).min
    x = torch.randn((14, E), generator=gen, device=DEV)
    x[0] = -inf                                  # nothing can be taken
    x[1] = math.nan
    x[2] = low                                   # a mask of the lowest value
    x[3, 5:] = -inf                              # fewer left than k
    x[4, 5:] = low
    x[5, ::2] = math.nan
    x[6, 3] = inf
    x[7, 3:6] = inf
    x[8] = inf
    x[9] = -200.0 - torch.arange(E, device=DEV)  # every score underflows
    x[10] = 200.0 + torch.arange(E, device=DEV)  # every sigmoid is 1 in float32
    x[11, 1:] = -inf
    x[12, 8:] = -inf                             # one expert left in some groups
    x[12, 9] = 0.5
    x[12, 17] = 0.25
    x[13] = -inf
    x[13, 31] = low
    b = torch.randn(E, generator=gen, device=DEV) * 0.1 if bias else None
    for top2 in (False, True):
        check(x, b, G, tg, k, softmax, norm, top2)
    xb = x.to(torch.bfloat16)
    check(xb, b, G, tg, k, softmax, norm, True)


def test_no_tokens():
    run(torch.empty((0, 16), device=DEV), None, 1, 1, 2, True, True, False)


def choose_exact(logits, bias, G, tg, k, softmax):
    """The choice by groups of two from scores in 64 bits, whole batches at once."""
    l = logits.double()
    c = (torch.softmax(l, 1) if softmax else torch.sigmoid(l)) + bias.double()
    T, E = c.shape
    value = c.view(T, G, E // G).topk(2, dim=2).values.sum(dim=2)
    order = value.sort(dim=1, descending=True, stable=True).indices[:, :tg]
    keep = torch.zeros((T, G), dtype=torch.bool, device=DEV).scatter_(1, order, True)
    c = c.masked_fill(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    return c.sort(dim=1, descending=True, stable=True).indices[:, :k]


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("size", [4.0, 16.0, 64.0, 1024.0, 2.0 ** 20])
@pytest.mark.parametrize("g", [2, 3])
def test_near_groups_with_biases_of_mixed_sign(softmax, size, g):
    """Two groups whose two best have biases of opposite sign: sums within 1e-5, each of two
    float32 values that were rounded at the size of their biases."""
    gen = torch.Generator(device=DEV).manual_seed(int(size) + g)
    T = 200000
    u = torch.rand((T, 3), generator=gen, device=DEV).double() * 0.4 + 0.3
    near = (torch.rand(T, generator=gen, device=DEV).double() - 0.5) * 2e-5
    u = torch.cat([u, (u[:, 0] + u[:, 1] - u[:, 2] + near)[:, None]], dim=1)
    ok = (u[:, 3] > 0.05) & (u[:, 3] < 0.95)
    l = (torch.log(u) if softmax else torch.logit(u))[ok].float()
    logits = torch.full((l.shape[0], 2 * g), -3.0, device=DEV)
    at = torch.tensor([0, 1, g, g + 1], device=DEV)
    logits[:, at] = l
    bias = torch.full((2 * g,), -4.0 * size - 8, device=DEV)
    bias[at] = torch.tensor([1.0, -1.0, 1.37, -1.37], device=DEV) * size
    _, idx, _ = run(logits, bias, 2, 1, 2, softmax, True, True)
    want = choose_exact(logits, bias, 2, 1, 2, softmax)
    bad = (idx != want).any(dim=1)
    assert not bad.any(), (int(bad.sum()), idx[bad][:3], want[bad][:3])


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E,G,tg", [(64, 8, 4), (64, 8, 1), (60, 10, 3), (128, 64, 9), (512, 64, 20),
                                    (256, 8, 4)])
def test_groups_with_errors_of_different_size(softmax, E, G, tg):
    """Biases of mixed sign, other sizes in each group: the group that float32 misjudges need
    not be the first one dropped."""
    gen = torch.Generator(device=DEV).manual_seed(E + G + tg)
    g, T = E // G, 60000
    logits = torch.randn((T, E), generator=gen, device=DEV)
    size = torch.exp2(torch.randint(0, 15, (G,), generator=gen, device=DEV).float())
    size *= 1 + torch.rand(G, generator=gen, device=DEV)
    bias = torch.full((G, g), -2.0 ** 17, device=DEV)
    bias[:, 0], bias[:, -1] = -size, size
    _, idx, _ = run(logits, bias.view(-1), G, tg, min(2 * tg, 32), softmax, True, True)
    want = choose_exact(logits, bias.view(-1), G, tg, min(2 * tg, 32), softmax)
    bad = (idx != want).any(dim=1)
    assert not bad.any(), (int(bad.sum()), idx[bad][:3], want[bad][:3])


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_group_sums_past_either_end_of_float32(sign):
    gen = torch.Generator(device=DEV).manual_seed(19)
    for E, G, tg in ((8, 4, 2), (12, 4, 1), (64, 32, 5)):
        x = torch.randn((40, E), generator=gen, device=DEV)
        x[:8, : E // G] = -math.inf
        for _ in range(3):
            b = sign * 2.5e38 * (1 + torch.rand(E, generator=gen, device=DEV) * 0.25)
            check(x, b, G, tg, 2, False, True, True)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("G,tg", [(1, 1), (4, 2)])
def test_an_infinite_bias_does_not_raise_a_masked_expert(softmax, G, tg):
    """-inf logits stay -inf whatever their bias (+inf is not of the documented values)."""
    gen = torch.Generator(device=DEV).manual_seed(23)
    E, k = 32, 4
    x = torch.randn((64, E), generator=gen, device=DEV)
    masked = torch.rand((64, E), generator=gen, device=DEV) < 0.3
    masked[:, ::8] = True
    x[masked] = -math.inf
    b = torch.zeros(E, device=DEV)
    b[::8], b[1::16] = math.inf, math.inf
    _, idx, w = run(x, b, G, tg, k, softmax, True, True)
    assert not masked.gather(1, idx).any() and (w > 0).all()


# -- gradient ---------------------------------------------------------------------------
def reference_gradient(logits, idx, dw, softmax, norm, alpha):
    l = ref.clean(logits).requires_grad_(True)
    w = alpha * ref.gate_weights(l, idx, softmax, norm)
    (w * dw.double()).sum().backward()
    return l.grad


def gradient_and_size(logits, idx, dw, softmax, norm, alpha):
    """Gradient in 64 bits by sums over differences, which cancel nowhere, and the size of
    its terms: (d, size, slack), [T, E] each.  With raw softmax the dw of an expert that is
    named m times are added first: m - 1 roundings of at most their magnitudes, which enter
    the differences as they are, however small those come out (slack)."""
    l, dw = ref.clean(logits), dw.double()
    T, E = l.shape
    k = idx.shape[1]
    p = ref.gate_weights(l, idx, softmax, norm)                    # [T, k]
    zero = torch.zeros_like(l)
    if norm or not softmax:
        if norm:
            diff = dw[:, :, None] - dw[:, None, :]
            parts = p[:, :, None] * p[:, None, :] * diff
            d, size = parts.sum(dim=2), parts.abs().sum(dim=2)
            if not softmax:
                d, size = (v * torch.sigmoid(-l.gather(1, idx)) for v in (d, size))
        else:
            d = p * torch.sigmoid(-l.gather(1, idx)) * dw
            size = d.abs()
        return alpha * zero.scatter_add(1, idx, d), alpha * zero.scatter_add(1, idx, size), zero
    s = torch.softmax(l, 1)
    w, w_size = zero.scatter_add(1, idx, dw), zero.scatter_add(1, idx, dw.abs())
    taken = torch.zeros_like(l, dtype=torch.bool).scatter_(1, idx, True)
    sc = torch.where(taken, s, 0.0)
    r = torch.where(taken, 0.0, s).sum(dim=1, keepdim=True)
    adds = (zero.scatter_add(1, idx, torch.ones_like(dw)) - 1).clamp(min=0)
    w_err = adds * 2.0 ** -24 * w_size
    d, size = torch.empty_like(l), torch.empty_like(l)
    for t in range(T):
        diff = w[t][:, None] - w[t][None, :]
        own = s[t] * (r[t] * w[t] + (sc[t][None, :] * diff).sum(dim=1))
        mag = s[t] * (r[t] * w_size[t] + (sc[t][None, :] * diff.abs()).sum(dim=1))
        rest = -s[t] * (sc[t] * w[t]).sum()
        d[t] = torch.where(taken[t], own, rest)
        size[t] = torch.where(taken[t], mag, s[t] * (sc[t] * w_size[t]).sum())
    slack = s * (w_err + (sc * w_err).sum(dim=1, keepdim=True))
    return alpha * d, alpha * size, alpha * slack


def check_gradient(logits, idx, dw, softmax, norm, alpha=2.5):
    """Each term is a product of two shares, of rel (far + 32) 2^-24 each with far the distance
    to the largest logit that enters them, a difference and up to 4 factors (a sigmoid of
    -l: 6 roundings), in a sum of k + 2; one rounding of the result.  Doubled."""
    T, E = logits.shape
    k = idx.shape[1]
    cfg = nh.gate_config(E, k, 1, 1, norm, alpha, "softmax" if softmax else "sigmoid", "max",
                         "bf16" if logits.dtype == torch.bfloat16 else "f32")
    out = torch.full((T + 1, E), 9.0, dtype=logits.dtype, device=DEV)
    nh.gate_backward(cfg, logits, idx.int(), dw, out[:T])
    assert (out[T] == 9).all()
    want, size, slack = gradient_and_size(logits, idx, dw, softmax, norm, alpha)
    l = ref.clean(logits)
    over = l if softmax and not norm else l.gather(1, idx)
    far = (over.amax(dim=1, keepdim=True) - over.amin(dim=1, keepdim=True)).clamp(max=104.0)
    tol = (size * (2 * (far + 32) + k + 16) * 2.0 ** -23 + 2 * slack +
           ref.EPS[logits.dtype] * want.abs() + 1e-37)
    bad = (out[:T].double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), out[:T][bad][:4], want[bad][:4], tol[bad][:4])
    return out[:T], want


@pytest.mark.parametrize("gap", [0.0, 4.0, 8.0, 12.0, 16.0, 30.0])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_where_one_expert_dominates(gap, softmax, norm, dtype):
    gen = torch.Generator(device=DEV).manual_seed(int(gap) + 31)
    for E, k in ((64, 6), (128, 1), (40, 8), (512, 32)):
        T = 24
        logits = torch.randn((T, E), generator=gen, device=DEV)
        if not softmax:
            logits -= 2.0             # sigmoid shares fall off as exp where logits are low
        best = torch.randint(0, E, (T, 1), generator=gen, device=DEV)
        logits = logits.scatter(1, best, logits.amax(dim=1, keepdim=True) + (0.0 if softmax else -gap))
        logits = (logits - gap).scatter(1, best, logits.gather(1, best)).to(dtype)
        idx = logits.float().topk(k, dim=1).indices
        dw = torch.randn((T, k), generator=gen, device=DEV)
        out, want = check_gradient(logits, idx, dw, softmax, norm)
        if norm and k == 1:
            assert (out == 0).all()
        # the same where the heavy expert was not chosen, and where one is named twice
        check_gradient(logits, idx.flip(1).roll(1, dims=0), dw, softmax, norm)
        if k > 1:
            twice = idx.clone()
            twice[:, 1] = twice[:, 0]
            check_gradient(logits, twice, dw, softmax, norm)
        # against autograd, where that keeps its digits
        if gap <= 8:
            g = reference_gradient(logits, idx, dw, softmax, norm, 2.5)
            assert ((g - want).abs() <= 1e-9 * want.abs().amax(dim=1, keepdim=True) + 1e-12).all()


@pytest.mark.parametrize("gap", [8.0, 16.0])
def test_gradient_rows_of_softmax_sum_to_zero(gap):
    """sum over experts of dl is 0 for a softmax: what the heavy expert gains the others lose."""
    gen = torch.Generator(device=DEV).manual_seed(41)
    T, E, k = 200, 64, 6
    logits = torch.randn((T, E), generator=gen, device=DEV)
    logits[:, 5] += gap + 4
    idx = logits.topk(k, dim=1).indices
    dw = torch.randn((T, k), generator=gen, device=DEV)
    for norm in (False, True):
        out, want = check_gradient(logits, idx, dw, True, norm)
        total = out.double().sum(dim=1).abs()
        assert (total <= 2.0 ** -14 * out.double().abs().amax(dim=1)).all()


@pytest.mark.parametrize("shape", [(1, 1), (5, 5), (16, 2), (33, 3), (100, 8), (128, 6), (250, 8),
                                   (256, 8), (512, 32)])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient(shape, softmax, norm, dtype):
    E, k = shape
    gen = torch.Generator(device=DEV).manual_seed(E + k)
    for T in (1, 67):
        logits = (torch.randn((T, E), generator=gen, device=DEV) * 2).to(dtype)
        cfg, idx, w = run(logits, None, 1, 1, k, softmax, norm, False)
        dw = torch.randn((T, k), generator=gen, device=DEV)
        out = torch.full((T + 1, E), 9.0, dtype=dtype, device=DEV)
        nh.gate_backward(cfg, logits, idx.int(), dw, out[:T])
        assert (out[T] == 9).all()
        want = reference_gradient(logits, idx, dw, softmax, norm, 2.5)
        # every term is a product of shares (rel (|l - top| + 32) 2^-24 each, twice), dw
        # and alpha; sums of up to 32 such terms: their magnitudes bound the error
        scale = 2.5 * dw.double().abs().sum(dim=1, keepdim=True)
        share = torch.softmax(logits.double(), 1) if softmax and not norm else torch.zeros_like(want)
        if norm or not softmax:
            share = share.scatter(1, idx, w.double() / 2.5)
        tol = share * scale * (20 + 64 + k) * 2.0 ** -23 + ref.EPS[dtype] * want.abs() + 1e-37
        bad = (out[:T].double() - want).abs() > tol
        assert not bad.any(), (out[:T][bad][:4], want[bad][:4])
        if norm or not softmax:
            rest = torch.ones((T, E), dtype=torch.bool, device=DEV).scatter(1, idx, False)
            assert (out[:T][rest] == 0).all()


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_gradient_against_differences(softmax, norm):
    """Central differences of the kernel's own weights.  h = 2^-6: the third derivative of
    a share is below 1, so h^2 / 6 alpha |dw| sum is the formula's part, and the float32
    weights' (32 + 8) 2^-24 each over 2 h the rounding's."""
    E, k, alpha, h = 24, 5, 2.5, 2.0 ** -6
    gen = torch.Generator(device=DEV).manual_seed(8)
    # well apart, so that a step of h changes no choice
    logits = torch.stack([torch.randperm(E, generator=gen, device=DEV).float() / 8 for _ in range(4)])
    cfg, idx, _ = run(logits, None, 1, 1, k, softmax, norm, False, alpha)
    dw = torch.randn((4, k), generator=gen, device=DEV)
    out = torch.empty_like(logits)
    nh.gate_backward(cfg, logits, idx.int(), dw, out)
    scale = alpha * dw.abs().double().sum(dim=1)
    tol = scale * (h * h / 6 + 2 * 40 * 2.0 ** -24 / (2 * h))
    for e in range(E):
        loss = []
        for d in (h, -h):
            p = logits.clone()
            p[:, e] += d
            _, i2, w2 = run(p, None, 1, 1, k, softmax, norm, False, alpha)
            assert torch.equal(i2, idx)
            loss.append((w2.double() * dw.double()).sum(dim=1))
        diff = (loss[0] - loss[1]) / (2 * h)
        assert ((diff - out[:, e].double()).abs() <= tol).all(), e


@pytest.mark.parametrize("softmax", [False, True])
def test_gradient_of_repeated_and_foreign_ids(softmax):
    E, k = 16, 4
    gen = torch.Generator(device=DEV).manual_seed(2)
    logits = torch.randn((3, E), generator=gen, device=DEV)
    dw = torch.randn((3, k), generator=gen, device=DEV)
    out = torch.empty_like(logits)
    for norm in (False, True):
        cfg = nh.gate_config(E, k, norm_topk_prob=norm, routed_scaling_factor=2.5,
                             scoring_func="softmax" if softmax else "sigmoid")
        idx = torch.tensor([[3, 3, 5, 3], [0, 15, 0, 1], [2, 2, 2, 2]], dtype=torch.int32, device=DEV)
        nh.gate_backward(cfg, logits, idx, dw, out)
        want = reference_gradient(logits, idx.long(), dw, softmax, norm, 2.5)
        tol = 2.5 * dw.double().abs().sum(dim=1, keepdim=True) * 100 * 2.0 ** -23
        assert ((out.double() - want).abs() <= tol).all()
        # ids outside [0, E) take no part: as if the slot were not there
        idx = torch.tensor([[3, -1, 5, 16], [7, 1 << 30, 2, 1], [-5, -1, -2, 99]],
                           dtype=torch.int32, device=DEV)
        nh.gate_backward(cfg, logits, idx, dw, out)
        for t, slots in ((0, [0, 2]), (1, [0, 2, 3])):
            want = reference_gradient(logits[t:t + 1], idx[t:t + 1, slots].long(), dw[t:t + 1, slots],
                                      softmax, norm, 2.5)
            assert ((out[t:t + 1].double() - want).abs() <= tol[t]).all()
        assert (out[2] == 0).all()


@pytest.mark.parametrize("softmax", [False, True])
def test_gradient_of_masked_rows_is_finite(softmax):
    E, k = 16, 4
    x = torch.zeros((4, E), device=DEV)
    x[0] = -math.inf
    x[1, 2:] = -math.inf
    x[2] = torch.finfo(torch.float32).min
    x[3] = -300.0
    dw = torch.ones((4, k), device=DEV)
    dw[:, 0] = 3.0
    for norm in (False, True):
        cfg, idx, _ = run(x, None, 1, 1, k, softmax, norm, False)
        out = torch.full_like(x, math.nan)
        nh.gate_backward(cfg, x, idx.int(), dw, out)
        assert torch.isfinite(out).all()
        assert (out[0] == 0).all() and (out[1, 2:] == 0).all()


# -- as they are used -----------------------------------------------------------------------
def test_streams_and_graph():
    gen = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn((300, 128), generator=gen, device=DEV)
    dw = torch.randn((300, 6), generator=gen, device=DEV)
    cfg = nh.gate_config(128, 6, 8, 2, scoring_func="softmax", group_score="top2")

    def go(idx, w, d, stream=None):
        nh.gate(cfg, x, None, idx, w, stream=stream)
        nh.gate_backward(cfg, x, idx, dw, d, stream=stream)

    def outs():
        return (torch.empty((300, 6), dtype=torch.int32, device=DEV), torch.empty((300, 6), device=DEV),
                torch.empty((300, 128), device=DEV))

    a, b, c = outs(), outs(), outs()
    go(*a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    go(*b, stream=s)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        go(*c)
    for o in c:
        o.zero_()
    x2 = x.clone()
    x.copy_(x2.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert torch.equal(c[0], a[0].flip(0)) and torch.equal(c[1], a[1].flip(0))
    x.copy_(x2)
    dw.copy_(dw.clone())
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, c))


@pytest.mark.parametrize("T", [1, 8, 32, 33, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_route_scored_is_the_gate_on_the_routers_logits(T, dtype):
    import numpy as np
    import synth
    cfg = synth.CONFIGS["tiny_f32_t64"].replace(T=T, dtype=dtype, n_routed_experts=32, topk_group=2)
    xn, wrn, _, _, _ = synth.make_router_and_x(cfg)
    x = torch.from_numpy(xn).cuda()
    x = x.view(torch.bfloat16) if dtype == "bf16" else x
    wr = torch.from_numpy(np.ascontiguousarray(wrn)).cuda()
    bias = torch.linspace(-0.1, 0.1, 32, device=DEV)
    ws = torch.zeros(nh.workspace_size(cfg, T), dtype=torch.uint8, device=DEV)
    lay = nh.workspace_layout(cfg, T)
    for score, b in (("softmax", None), ("softmax", bias), ("sigmoid", bias)):
        idx = torch.empty((T, 2), dtype=torch.int32, device=DEV)
        w = torch.empty((T, 2), device=DEV)
        nh.route_scored(cfg, score, x, wr, b, idx, w, ws)
        assert nh.check_device(ws) == 0
        logits = ws[lay.logits:lay.logits + 4 * T * 32].view(torch.float32).view(T, 32)
        want = x.double() @ wr.double().t()
        # products and sums in float32: K roundings of the terms' magnitudes
        tol = (x.double().abs() @ wr.double().abs().t()) * 256 * 2.0 ** -23
        assert ((logits.double() - want).abs() <= tol).all()
        widx, ww = ref.gate(logits, b, 4, 2, 2, score == "softmax", True, False, 2.5)
        assert torch.equal(idx.long(), widx)
        check_w(w, ww, logits.gather(1, widx))
    if dtype == "f32":
        i2, w2 = torch.empty_like(idx), torch.empty_like(w)
        nh.route(cfg, x, wr, bias, i2, w2, ws)
        assert torch.equal(idx, i2)
