"""References of the FP8 and gate tests, in 64 bits and by other means than the
kernels': E4M3 by search in the table of its values, scales by search over powers of
two, products in float64, the choice of experts by sorting in float64."""
from __future__ import annotations

import math

import torch

BLOCK = 128
EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, "e4m3": 2.0 ** -4}   # half a step


def e4m3_table():
    """Value of every code (0x7F and 0xFF are NaN), float64."""
    vals = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        vals.append(math.nan if (code & 0x7F) == 0x7F else (-v if code & 0x80 else v))
    return torch.tensor(vals, dtype=torch.float64)


def decode(codes):
    return e4m3_table().to(codes.device)[codes.view(torch.uint8).long()]


def nearest_e4m3(v):
    """Nearest E4M3 value of |v| <= 448, ties to the even code; NaN and Inf to NaN."""
    pos = e4m3_table()[:0x7F].to(v.device)
    a = v.abs().nan_to_num(nan=0.0, posinf=0.0).contiguous()
    hi = torch.searchsorted(pos, a).clamp(1, 0x7E)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    code = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    out = torch.copysign(pos[code], v)
    return torch.where(torch.isfinite(v), out, math.nan)


def block_scale(amax):
    """The least power of two s >= 2^-126 with amax <= 448 s; 1 where amax = 0."""
    s = torch.ones_like(amax)
    for e in range(128, -127, -1):
        s = torch.where(amax <= 448.0 * 2.0 ** e, 2.0 ** e, s)
    return torch.where(amax == 0, 1.0, s)


def _blocks(n):
    return -(-n // BLOCK)


def spread(scales, cols, rows=None):
    s = scales.double()
    if rows is not None:
        s = s.repeat_interleave(BLOCK, dim=-2)[..., :rows, :]
    return s.repeat_interleave(BLOCK, dim=-1)[..., :cols]


def quantize_rows(x):
    """x [R, K] -> (values of the codes, scales), float64."""
    x = x.double()
    R, K = x.shape
    pad = torch.zeros((R, _blocks(K) * BLOCK), dtype=torch.float64, device=x.device)
    pad[:, :K] = x
    b = pad.view(R, -1, BLOCK)
    s = block_scale(torch.where(torch.isfinite(b), b.abs(), 0.0).amax(dim=2))
    return nearest_e4m3((b / s[:, :, None]).view(R, -1)[:, :K]), s


def quantize_weight(w):
    """w [n, rows, cols] -> (values of the codes, scales), float64."""
    w = w.double()
    n, r, c = w.shape
    pad = torch.zeros((n, _blocks(r) * BLOCK, _blocks(c) * BLOCK), dtype=torch.float64,
                      device=w.device)
    pad[:, :r, :c] = w
    b = pad.view(n, _blocks(r), BLOCK, _blocks(c), BLOCK)
    s = block_scale(torch.where(torch.isfinite(b), b.abs(), 0.0).amax(dim=(2, 4)))
    return nearest_e4m3((b / s[:, :, None, :, None]).view(pad.shape)[:, :r, :c]), s


def rows_values(x):
    q, s = quantize_rows(x)
    return q * spread(s, x.shape[1])


def weight_values(codes, scales):
    return decode(codes) * spread(scales, codes.shape[-1], codes.shape[-2])


def make_weight(gen, n, rows, cols, std=0.05):
    """Seeded FP8 weight with arbitrary float32 scales (not powers of two)."""
    dev = gen.device
    v = torch.randn((n, rows, cols), generator=gen, device=dev) * 64.0
    codes = v.clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = std / 64.0 * torch.rand((n, _blocks(rows), _blocks(cols)), generator=gen, device=dev).add_(0.5)
    return codes, scales


def experts(x, idx, w, up, down):
    """Routed experts in float64: x [T, H], idx / w [T, k], up / down (codes, scales).
    Returns (y [T, H], bound [T, H]): the bound is what the quantization of the hidden
    rows may add where a float32 sum falls on the other side of a rounding edge."""
    T, H = x.shape
    xv = rows_values(x)
    y = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    for e in range(up[0].shape[0]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        h = torch.relu(xv[t] @ weight_values(up[0][e], up[1][e]).t()) ** 2
        o = rows_values(h) @ weight_values(down[0][e], down[1][e]).t()
        y.index_add_(0, t, w[t, j].double()[:, None] * o)
    return y


def clean(logits):
    l = logits.double()
    return torch.where(torch.isnan(l), -math.inf, l).clamp(max=torch.finfo(torch.float32).max)


def gate(logits, bias, G, tg, k, softmax, norm, top2, alpha):
    """(idx [T, k], w [T, k] float64) of the gate's definition, by sorting."""
    l = clean(logits)
    T, E = l.shape
    if softmax:
        top = l.amax(dim=1, keepdim=True)
        u = torch.exp(l - torch.where(top == -math.inf, 0.0, top))
        z = u.sum(dim=1, keepdim=True)
        s = u / torch.where(z == 0, 1.0, z)
    else:
        s = torch.sigmoid(l)
    if bias is None and not (top2 and tg < G):
        c = l
    else:
        c = torch.where(l == -math.inf, -math.inf, s + (0.0 if bias is None else bias.double()))
    idx = torch.empty((T, k), dtype=torch.int64)
    c_host, g = c.cpu().tolist(), E // G
    for t in range(T):
        row = c_host[t]
        vals = []
        for q in range(G):
            best = sorted(row[q * g:(q + 1) * g], reverse=True)
            vals.append(best[0] + (best[1] if top2 and best[1] != -math.inf else 0.0))
        kept = sorted(range(G), key=lambda q: (-vals[q], q))[:tg]
        cand = [e for q in kept for e in range(q * g, (q + 1) * g)]
        idx[t] = torch.tensor(sorted(cand, key=lambda e: (-row[e], e))[:k])
    idx = idx.to(l.device)
    return idx, alpha * gate_weights(l, idx, softmax, norm)


def gate_weights(l, idx, softmax, norm):
    """Weights (alpha = 1) of the choice idx, float64, from log scores; l cleaned."""
    if softmax:
        # relative to the largest: the sum's logarithm is lost beside 1e38
        top = l.amax(dim=1, keepdim=True)
        rel = l - torch.where(top == -math.inf, 0.0, top)
        z = torch.exp(rel).sum(dim=1, keepdim=True)
        logs = rel - torch.where(z == 0, 0.0, torch.log(z))
    else:
        logs = torch.nn.functional.logsigmoid(l)
    if softmax and norm:
        logs = l
    sel = logs.gather(1, idx)
    if not norm:
        return torch.exp(sel)
    top = sel.amax(dim=1, keepdim=True)
    u = torch.exp(sel - torch.where(top == -math.inf, 0.0, top))
    z = u.sum(dim=1, keepdim=True)
    return u / torch.where(z == 0, 1.0, z)
