"""Float64 definitions of the layers beside the gated delta rule, for the tests.

Plain loops over sequences and tokens on the CPU, written from the formulas in
include/pace.h; nothing here uses the library.
"""
import math

import torch

U32 = 2.0 ** -24                 # half a step of float32, relative
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def norm_rope(x, norm, weight, eps, pos, inv_freq, adjacent, scale):
    """x [tokens, heads, d] -> float64."""
    x = x.double()
    if norm == "l2":
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps)
    elif norm == "rms":
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if weight is not None:
            x = x * weight.double()
    y = x.clone()
    if inv_freq is not None:
        half = inv_freq.numel()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
            w = pos.double() * inv_freq[i].double()
            cos, sin = torch.cos(w)[:, None], torch.sin(w)[:, None]
            y[..., a] = x[..., a] * cos - x[..., b] * sin
            y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y * scale


def linear(q, k, v, decay, state, lens, scale):
    """Token by token; rows behind a sequence's end are NaN in `out`."""
    t, b, h, dk = q.shape
    dv = v.shape[3]
    M = torch.zeros((b, h, dk, dv), dtype=torch.float64) if state is None else state.double().clone()
    out = torch.full((t, b, h, dv), math.nan, dtype=torch.float64)
    for i in range(b):
        n = t if lens is None else min(max(int(lens[i]), 0), t)
        for s in range(n):
            M[i] = M[i] * decay.double()[:, None, None] + k[s, i].double()[:, :, None] * v[s, i].double()[:, None, :]
            out[s, i] = scale * torch.matmul(q[s, i].double()[:, None, :], M[i])[:, 0]
    return out, M


def quantize(x):
    """(codes, scales) of the last axis in groups of 64, float64 from exact quotients."""
    x = x.double().unflatten(-1, (-1, 64))
    top = x.abs().amax(-1, keepdim=True)
    codes = torch.where(top > 0, torch.round(7 * x / torch.where(top > 0, top, 1.0)), 0.0)
    return codes.flatten(-2), (top / 7).squeeze(-1)


def values(x):
    codes, s = quantize(x)
    return (codes.unflatten(-1, (-1, 64)) * s.unsqueeze(-1)).flatten(-2)


def attention(q, k, v, seen, scale, window, sinks, lens, count):
    """q [T, B, Hq, d]; k, v float64 [B, n, Hk, d]; seen bool [B, n]: positions
    with a page.  Returns (out, mass, reach): the result, sum_j p_j |v_j| and
    the largest scale * sum |q k| of a row, which error bounds need.  Rows
    t >= count[b] are NaN."""
    t, b, hq, d = q.shape
    g = hq // k.shape[2]
    out = torch.full((t, b, hq, d), math.nan, dtype=torch.float64)
    mass, reach = torch.zeros_like(out), torch.zeros((t, b, hq, 1), dtype=torch.float64)
    for i in range(b):
        n = min(max(int(lens[i]), 0), k.shape[1])
        c = t if count is None else min(max(int(count[i]), 0), t)
        j = torch.arange(n)
        for s in range(c):
            p = n - c + s
            see = (j <= p) & seen[i, :n]
            if window:
                see = see & ((j > p - window) | (j < sinks))
            see = see.nonzero()[:, 0]
            for h in range(hq):
                if see.numel() == 0:
                    out[s, i, h] = 0
                    continue
                kk, vv, qq = k[i, see, h // g], v[i, see, h // g], q[s, i, h].double()
                w = torch.softmax(scale * (kk @ qq), 0)
                out[s, i, h] = w @ vv
                mass[s, i, h] = w @ vv.abs()
                reach[s, i, h] = abs(scale) * float((kk.abs() @ qq.abs()).max())
    return out, mass, reach
