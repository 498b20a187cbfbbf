"""What the expert-routing and 8-bit operators compute, in plain torch, and the calls a user makes of them.

Five operators that belong together in a mixture-of-experts block:

  gate           the router's choice from its logits [T, E]: sigmoid or softmax scores, an optional
                 balance bias that only selects, groups of experts, top-k, renormalised weights
  gate_backward  the gradient of the routing weights with respect to the logits
  quantize       activations [T, K] to E4M3 with one power-of-two scale per token and 128 features
  linear         y = x W^T with E4M3 operands and a scale per block of 128 (x quantized in the call)
  experts        the routed experts of a block with such weights: permute, up, relu^2, down, combine

``own`` selects the library's kernels; otherwise ``run`` computes the plain form.  Sizes are those of
this repository's workloads (hidden 2688, experts 1856 wide, shared expert 3712 wide, 128 experts of
which 6 are taken; the 256-expert, 4096-wide stress block) and odd ones between them.
"""
import math
import types

import numpy as np
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
F32_MAX = 3.4028234663852886e38


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def _gate(op, T, E, G, tg, k, score, bias, norm, top2, dtype, name=None):
    c = dict(op=op, T=T, E=E, G=G, tg=tg, k=k, score=score, bias=bias, norm=norm, top2=top2,
             dtype=dtype)
    return dict(c, name=name) if name else c


def _quant(T, K, dtype, name=None):
    c = dict(op="quantize", T=T, K=K, dtype=dtype)
    return dict(c, name=name) if name else c


def _linear(T, N, K, out, name=None):
    c = dict(op="linear", T=T, N=N, K=K, out=out)
    return dict(c, name=name) if name else c


def _experts(T, H, I, E, k, name=None):
    c = dict(op="experts", T=T, H=H, I=I, E=E, k=k)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of the 128-expert block: softmax scores, one group of eight
        _gate("gate", 8, 128, 8, 1, 6, "softmax", False, True, False, "f32", "gate_decode_t8"),
        # prefill of a 256-expert block: sigmoid scores, balance bias, 4 of 8 groups by their two best
        _gate("gate", 16384, 256, 8, 4, 8, "sigmoid", True, True, True, "f32",
              "gate_prefill_t16384"),
        # a ragged training batch, raw softmax weights (a dense gradient), bf16 logits
        _gate("gate_backward", 2047, 128, 1, 1, 6, "softmax", False, False, False, "bf16",
              "gate_backward_t2047"),
        # the gradient of the 256-expert prefill's routing
        _gate("gate_backward", 16384, 256, 8, 4, 8, "sigmoid", False, True, True, "f32",
              "gate_backward_t16384"),
        # activations of a ragged batch between the projections (float32, 14.5 blocks per token)
        _quant(333, 1856, "f32", "quantize_t333"),
        # activations of a whole prefill
        _quant(16384, 2688, "bf16", "quantize_t16384"),
        # the shared expert's up projection for a single token
        _linear(1, 3712, 2688, "bf16", "linear_t1"),
        # a ragged batch through the shared expert's down projection
        _linear(777, 2688, 3712, "bf16", "linear_t777"),
        # the shared expert's up projection over a whole prefill
        _linear(16384, 3712, 2688, "bf16", "linear_t16384"),
        # one decode step of the 128-expert block
        _experts(8, 2688, 1856, 128, 6, "experts_decode_t8"),
        # a ragged batch in flight: about 14 rows an expert
        _experts(301, 2688, 1856, 128, 6, "experts_t301"),
        # prefill of the 128-expert block
        _experts(16384, 2688, 1856, 128, 6, "experts_prefill_t16384"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate_backward", "quantize", "linear", "experts"])
    if op in ("gate", "gate_backward"):
        G = rng.choice([1, 1, 2, 4, 8, 8, 16])
        g = rng.randint(max(2, 8 // G), 256 // G)
        tg = rng.randint(1, G)
        k = rng.randint(1, min(8, tg * g))
        return _gate(op, _log_int(rng, 1, 16384), G * g, G, tg, k, rng.choice(["sigmoid", "softmax"]),
                     op == "gate" and rng.random() < 0.5, rng.random() < 0.7, rng.random() < 0.5,
                     rng.choice(["f32", "bf16"]))
    if op == "quantize":
        return _quant(_log_int(rng, 1, 16384), 16 * _log_int(rng, 4, 168), rng.choice(["bf16", "f32"]))
    if op == "linear":
        return _linear(_log_int(rng, 1, 16384), 16 * _log_int(rng, 8, 232), 16 * _log_int(rng, 8, 168),
                       "bf16")
    E = rng.choice([8, 16, 32, 64, 128])
    return _experts(_log_int(rng, 1, 8192), 64 * rng.randint(4, 42), 64 * rng.randint(4, 29), E,
                    rng.randint(1, 6))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _weight(gen, n, rows, cols, std):
    """Seeded normal weights [n, rows, cols] as E4M3 codes and float32 scales amax / 448 per 128 x 128
    block, as a checkpoint stores them."""
    rb, cb = -(-rows // BLOCK), -(-cols // BLOCK)
    codes = torch.empty((n, rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((n, rb, cb), dtype=torch.float32, device="cuda")
    pad = torch.zeros((rb * BLOCK, cb * BLOCK), device="cuda")
    for i in range(n):
        pad[:rows, :cols].normal_(0.0, std, generator=gen)
        blocks = pad.view(rb, BLOCK, cb, BLOCK)
        s = blocks.abs().amax(dim=(1, 3)) / E4M3_MAX
        scales[i] = s
        q = (blocks / s[:, None, :, None]).clamp_(-E4M3_MAX, E4M3_MAX).view(rb * BLOCK, cb * BLOCK)
        codes[i] = q[:rows, :cols].to(torch.float8_e4m3fn)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = types.SimpleNamespace(kept={}, **{k: v for k, v in case.items() if k != "name"})

    def normal(*shape, std=1.0):
        return torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen)

    if s.op in ("gate", "gate_backward"):
        s.logits = normal(s.T, s.E, std=1.5).to(_dtype(s.dtype))
        s.bias_v = normal(s.E, std=0.05) if s.bias else None
        s.alpha = 2.5
        if s.op == "gate_backward":
            # the forward's choice, which a training step keeps for its backward pass
            s.idx = _choose(s.logits, s)[0].to(torch.int32)
            s.dw = normal(s.T, s.k)
    elif s.op == "quantize":
        s.x = normal(s.T, s.K).to(_dtype(s.dtype))
    elif s.op == "linear":
        s.x = normal(s.T, s.K).to(torch.bfloat16)
        s.codes, s.scales = _weight(gen, 1, s.N, s.K, 0.02)
    else:
        s.x = normal(s.T, s.H).to(torch.bfloat16)
        s.up, s.up_scales = _weight(gen, s.E, s.I, s.H, 0.02)
        s.down, s.down_scales = _weight(gen, s.E, s.H, s.I, 0.02)
        # some experts are more popular than others
        want = normal(s.T, s.E) + normal(s.E, std=0.3)
        score, idx = torch.topk(want, s.k, dim=1)
        s.idx = idx.to(torch.int32)
        s.w = 2.5 * torch.softmax(score, dim=1)
        # the plain form's room per expert
        s.room = int(torch.zeros(s.E, dtype=torch.int64, device="cuda").index_add_(
            0, idx.flatten(), torch.ones(s.T * s.k, dtype=torch.int64, device="cuda")).max())
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _clean(logits, dtype):
    """Logits as the router reads them: NaN counts as -inf (an expert that cannot be taken), +inf as
    the largest float32."""
    l = logits.to(dtype)
    return torch.where(torch.isnan(l), -math.inf, l).clamp(max=F32_MAX)


def _scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
    z = e.sum(dim=1, keepdim=True)
    return e / torch.where(z == 0, 1.0, z)


def _choose(logits, s):
    """(idx [T, k], clean logits, scores) in 64 bits: neighbouring scores decide the choice."""
    l = _clean(logits, torch.float64)
    sc = _scores(l, s.score)
    T, E = l.shape
    bias = getattr(s, "bias_v", None)
    # without a bias or a sum over two experts the logits order the experts as the scores do
    if bias is None and (s.tg == s.G or not s.top2):
        c = l
    else:
        c = torch.where(l == -math.inf, -math.inf, sc + (0.0 if bias is None else bias.double()))
    order = torch.sort(c, dim=1, descending=True, stable=True).indices
    if s.tg < s.G:
        best = torch.sort(c.view(T, s.G, E // s.G), dim=2, descending=True).values
        gs = best[:, :, 0]
        if s.top2:
            gs = gs + torch.where(best[:, :, 1] == -math.inf, 0.0, best[:, :, 1])
        groups = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, : s.tg]
        keep = torch.zeros((T, s.G), dtype=torch.int8, device=l.device).scatter_(1, groups, 1)
        kept = keep.gather(1, order // (E // s.G))
        order = order.gather(1, torch.sort(kept, dim=1, descending=True, stable=True).indices)
    return order[:, : s.k], l, sc


def _shares(lsel, s):
    """What part of the selected experts' summed score each has; 0 where none can be taken."""
    top = lsel.amax(dim=1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    if s.score == "softmax":
        u = torch.exp(lsel - top)
    else:
        m = top.clamp(max=0.0)
        u = torch.where(lsel < 0, torch.exp(lsel - m) / (1.0 + torch.exp(lsel.clamp(max=0.0))),
                        1.0 / (1.0 + torch.exp(-lsel.clamp(min=0.0))))
    z = u.sum(dim=1, keepdim=True)
    return u / torch.where(z == 0, 1.0, z)


def _plain_gate(s):
    idx, l, sc = _choose(s.logits, s)
    w = _shares(l.gather(1, idx), s) if s.norm else sc.gather(1, idx)
    return {"idx": idx.to(torch.int32), "w": (s.alpha * w).float()}


def _plain_gate_backward(s):
    l = _clean(s.logits, torch.float32)
    idx = s.idx.long()
    lsel = l.gather(1, idx)
    gone = 1.0 / (1.0 + torch.exp(lsel))              # 1 - sigmoid
    if s.norm:
        p = _shares(lsel, s)
        d = s.alpha * p * (s.dw - (p * s.dw).sum(dim=1, keepdim=True))
        if s.score == "sigmoid":
            d = d * gone
        out = torch.zeros_like(l).scatter_add_(1, idx, d)
    else:
        sc = _scores(l, s.score)
        picked = sc.gather(1, idx) * s.dw
        if s.score == "sigmoid":
            out = torch.zeros_like(l).scatter_add_(1, idx, s.alpha * picked * gone)
        else:
            out = torch.zeros_like(l).scatter_add_(1, idx, s.alpha * picked)
            out = out - s.alpha * sc * picked.sum(dim=1, keepdim=True)
    return out.to(s.logits.dtype)


def _quantize(x):
    """[R, K] float32 -> (E4M3 codes [R, K], scales [R, ceil(K / 128)]), the scale the least power of
    two at which the block's largest magnitude fits 448 (1 for a block of zeros)."""
    R, K = x.shape
    kb = -(-K // BLOCK)
    pad = torch.zeros((R, kb * BLOCK), device=x.device)
    pad[:, :K] = x
    b = pad.view(R, kb, BLOCK)
    amax = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(dim=2)
    mant, ex = torch.frexp(amax)                       # amax = mant 2^ex, 448 = 0.875 * 2^9
    ex = (ex - torch.where(mant <= 0.875, 9, 8)).clamp(min=-126)
    scale = torch.where(amax == 0, 1.0, torch.ldexp(torch.ones_like(amax), ex))
    q = b / scale[:, :, None]
    q = torch.where(torch.isfinite(q), q, math.nan)
    return q.view(R, kb * BLOCK)[:, :K].to(torch.float8_e4m3fn), scale


def _spread(scale, cols):
    return scale.repeat_interleave(BLOCK, dim=-1)[..., :cols]


def _dequantized(x):
    q, scale = _quantize(x)
    return q.float() * _spread(scale, x.shape[1])


def _weight_f32(codes, scales):
    rows, cols = codes.shape[-2:]
    sc = scales.repeat_interleave(BLOCK, dim=-2)[..., :rows, :]
    return codes.float() * _spread(sc, cols)


def _plain_quantize(s):
    q, scale = _quantize(s.x.float())
    return {"codes": q, "scales": scale}


def _plain_linear(s):
    y = _dequantized(s.x.float()) @ _weight_f32(s.codes[0], s.scales[0]).t()
    return y.to(_dtype(s.out))


def _plain_experts(s):
    flat = s.idx.flatten().long()
    by = torch.sort(flat, stable=True).indices         # assignments by expert, in token order
    e = flat[by]
    counts = torch.zeros(s.E, dtype=torch.int64, device=flat.device).index_add_(0, flat, torch.ones_like(flat))
    at = torch.arange(flat.numel(), device=flat.device) - (torch.cumsum(counts, 0) - counts)[e]
    x = torch.zeros((s.E, s.room, s.H), device=flat.device)
    x[e, at] = _dequantized(s.x.float())[by // s.k]
    h = torch.relu(torch.bmm(x, _weight_f32(s.up, s.up_scales).transpose(1, 2))).square()
    h = _dequantized(h.view(s.E * s.room, s.I)).view(s.E, s.room, s.I)
    o = torch.bmm(h, _weight_f32(s.down, s.down_scales).transpose(1, 2))
    place = torch.empty_like(flat)
    place[by] = e * s.room + at
    rows = o.view(s.E * s.room, s.H)[place].view(s.T, s.k, s.H)
    return (rows * s.w[:, :, None]).sum(dim=1).to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------------------
def _own_gate_config(nh, s):
    c = s.kept.get("cfg")
    if c is None:
        c = s.kept["cfg"] = nh.gate_config(
            n_routed_experts=s.E, n_group=s.G, topk_group=s.tg, num_experts_per_tok=s.k,
            norm_topk_prob=s.norm, routed_scaling_factor=s.alpha, scoring_func=s.score,
            group_score="top2" if s.top2 else "max", dtype=s.dtype)
    return c


def _own_gate(nh, s):
    idx = torch.empty((s.T, s.k), dtype=torch.int32, device="cuda")
    w = torch.empty((s.T, s.k), dtype=torch.float32, device="cuda")
    nh.gate(_own_gate_config(nh, s), s.logits, s.bias_v, idx, w)
    return {"idx": idx, "w": w}


def _own_gate_backward(nh, s):
    out = torch.empty_like(s.logits)
    nh.gate_backward(_own_gate_config(nh, s), s.logits, s.idx, s.dw, out)
    return out


def _own_quantize(nh, s):
    codes = torch.empty((s.T, s.K), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((s.T, -(-s.K // BLOCK)), dtype=torch.float32, device="cuda")
    nh.fp8_quantize(s.x, codes, scales)
    return {"codes": codes, "scales": scales}


def _own_linear(nh, s):
    if "ws" not in s.kept:
        s.kept["ws"] = torch.zeros(nh.fp8_linear_workspace_size(s.T, s.N, s.K), dtype=torch.uint8,
                                   device="cuda")
        s.kept["w"] = nh.fp8_weight(s.codes, s.scales)
    y = torch.empty((s.T, s.N), dtype=_dtype(s.out), device="cuda")
    nh.fp8_linear(s.x, s.kept["w"], y, s.kept["ws"])
    return y


def _own_experts(nh, s):
    if "cfg" not in s.kept:
        c = nh.config_from(types.SimpleNamespace(
            hidden_size=s.H, n_routed_experts=s.E, n_group=1, topk_group=1, num_experts_per_tok=s.k,
            moe_intermediate_size=s.I, moe_shared_expert_intermediate_size=s.I, n_shared_experts=0,
            norm_topk_prob=True, routed_scaling_factor=2.5, dtype="bf16", weight_format="fp8"))
        s.kept.update(
            cfg=c, up=nh.fp8_weight(s.up, s.up_scales), down=nh.fp8_weight(s.down, s.down_scales),
            ws=torch.zeros(nh.workspace_size(c, s.T), dtype=torch.uint8, device="cuda"),
            y_acc=torch.empty((s.T, s.H), dtype=torch.float32, device="cuda"))
    c, ws, y_acc = s.kept["cfg"], s.kept["ws"], s.kept["y_acc"]
    y = torch.empty((s.T, s.H), dtype=torch.bfloat16, device="cuda")
    nh.zero_acc(c, s.T, y_acc)
    nh.permute(c, s.x, s.idx, s.w, ws)
    nh.forward_fp8(c, s.x, s.kept["up"], s.kept["down"], ws, y_acc)
    nh.finalize(c, s.T, y_acc, y)
    return y


_PLAIN = {"gate": _plain_gate, "gate_backward": _plain_gate_backward, "quantize": _plain_quantize,
          "linear": _plain_linear, "experts": _plain_experts}
_OWN = {"gate": _own_gate, "gate_backward": _own_gate_backward, "quantize": _own_quantize,
        "linear": _own_linear, "experts": _own_experts}


def run(state):
    if own:
        import non_gated_relu_b200 as nh
        return _OWN[state.op](nh, state)
    return _PLAIN[state.op](state)


# ---------------------------------------------------------------------------------------------
# the least that each must read, write and compute
# ---------------------------------------------------------------------------------------------
def work(case):
    c = types.SimpleNamespace(**case)
    if c.op in ("gate", "gate_backward"):
        size = 2 if c.dtype == "bf16" else 4
        if c.op == "gate":
            return {"bytes": c.T * (c.E * size + c.k * 8) + (4 * c.E if c.bias else 0),
                    "flops": 4 * c.T * c.E}
        # renormalised and sigmoid weights need the chosen logits alone; raw softmax weights need all
        read = c.E if (c.score == "softmax" and not c.norm) else c.k
        return {"bytes": c.T * (read * size + c.k * 8 + c.E * size), "flops": 4 * c.T * (read + c.k)}
    if c.op == "quantize":
        size = 2 if c.dtype == "bf16" else 4
        return {"bytes": c.T * (c.K * (size + 1) + 4 * -(-c.K // BLOCK)), "flops": 3 * c.T * c.K}
    if c.op == "linear":
        size = 2 if c.out == "bf16" else 4
        scales = 4 * -(-c.N // BLOCK) * -(-c.K // BLOCK)
        return {"bytes": c.T * c.K * 2 + c.N * c.K + scales + c.T * c.N * size,
                "flops": 2 * c.T * c.N * c.K}
    # weights of the experts that at least one token takes (even routing)
    hit = c.E * (1.0 - (1.0 - c.k / c.E) ** c.T)
    return {"bytes": hit * 2 * c.H * c.I * (1 + 4 / BLOCK ** 2) + c.T * (4 * c.H + 8 * c.k),
            "flops": 4 * c.T * c.k * c.H * c.I}


# ---------------------------------------------------------------------------------------------
# the same outputs from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------
def _e4m3_values():
    v = np.zeros(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        mag = math.nan if (e == 15 and m == 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[code] = -mag if code & 128 else mag
    return torch.from_numpy(v).cuda()


def _exact_weight(codes, scales):
    v = _e4m3_values()[codes.view(torch.uint8).long()]
    r = torch.arange(codes.shape[0], device="cuda") // BLOCK
    c = torch.arange(codes.shape[1], device="cuda") // BLOCK
    return v * scales.double()[r][:, c]


def _exact_quantized(x):
    """(codes' values, scales) of [R, K] float64: finite inputs only."""
    R, K = x.shape
    kb = -(-K // BLOCK)
    codes, scales = torch.empty_like(x), torch.empty((R, kb), dtype=torch.float64, device=x.device)
    for b in range(kb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        top = v.abs().max(dim=1).values
        e = torch.full_like(top, -126.0)
        # the least e with top <= 448 * 2^e
        near = torch.floor(torch.log2(top.clamp(min=1e-300) / E4M3_MAX)) - 1
        for step in (0, 1, 2):
            fits = top <= E4M3_MAX * torch.exp2(near + step)
            e = torch.where(fits & (e == -126.0), (near + step).clamp(min=-126.0), e)
        sc = torch.where(top == 0, 1.0, torch.exp2(e))
        q = v / sc[:, None]
        grid = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = torch.round(q / grid) * grid
        scales[:, b] = sc
    return codes, scales


def _exact_values(x):
    codes, scales = _exact_quantized(x)
    return codes * scales[:, torch.arange(x.shape[1], device=x.device) // BLOCK]


def _exact_gate(s):
    l = s.logits.double().cpu().numpy()
    T, E = l.shape
    if s.score == "sigmoid":
        logs = -np.logaddexp(0.0, -l)
    else:
        logs = l - np.logaddexp.reduce(l, axis=1, keepdims=True)
    by_score = s.bias_v is not None or (s.top2 and s.tg < s.G)
    c = np.exp(logs) + (0.0 if s.bias_v is None else s.bias_v.double().cpu().numpy()) if by_score else l
    open_ = np.ones((T, E), bool)
    if s.tg < s.G:
        part = np.sort(c.reshape(T, s.G, -1), axis=2)
        gs = part[:, :, -1] + (part[:, :, -2] if s.top2 else 0.0)
        place = np.argsort(np.argsort(-gs, axis=1, kind="stable"), axis=1, kind="stable")
        open_ = np.repeat(place < s.tg, E // s.G, axis=1)
    idx = np.argsort(np.where(open_, -c, np.inf), axis=1, kind="stable")[:, : s.k]
    g = np.take_along_axis(logs, idx, axis=1)
    w = np.exp(g - np.logaddexp.reduce(g, axis=1, keepdims=True)) if s.norm else np.exp(g)
    return {"idx": None, "w": s.alpha * w}


def _exact_gate_backward(s):
    """The Jacobian of each token's k weights applied to dw."""
    l, idx, dw = s.logits.double(), s.idx.long(), s.dw.double()
    T, E = l.shape
    if s.score == "sigmoid":
        sc = torch.sigmoid(l)
        slope = sc * (1 - sc)
    else:
        sc = torch.softmax(l, dim=1)
    sel = sc.gather(1, idx)
    if s.norm:
        z = sel.sum(dim=1, keepdim=True)
        ds = dw / z - (dw * sel).sum(dim=1, keepdim=True) / z ** 2
    else:
        ds = dw
    full = torch.zeros_like(l).scatter_add_(1, idx, s.alpha * ds)     # gradient of the scores
    if s.score == "sigmoid":
        return full * slope
    return sc * (full - (sc * full).sum(dim=1, keepdim=True))


def exact(case, seed):
    s = prepare(case, seed)
    if s.op == "gate":
        return _exact_gate(s)
    if s.op == "gate_backward":
        return _exact_gate_backward(s)
    if s.op == "quantize":
        codes, scales = _exact_quantized(s.x.double())
        return {"codes": codes, "scales": scales}
    if s.op == "linear":
        return _exact_values(s.x.double()) @ _exact_weight(s.codes[0], s.scales[0]).t()
    x = _exact_values(s.x.double())
    y = torch.zeros((s.T, s.H), dtype=torch.float64, device="cuda")
    for e in range(s.E):
        t, j = torch.nonzero(s.idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        h = torch.relu(x[t] @ _exact_weight(s.up[e], s.up_scales[e]).t()) ** 2
        o = _exact_values(h) @ _exact_weight(s.down[e], s.down_scales[e]).t()
        y[t] += s.w[t, j].double()[:, None] * o
    return y
