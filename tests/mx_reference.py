"""The MXFP8 operators in 64 bits, from their definitions, with bounds on what
float32 sums and the roundings may change."""
import numpy as np
import torch

GROUP = 32
F64 = torch.float64
E4M3 = torch.tensor([(-1) ** (c >> 7) * ((c & 7) * 2.0 ** -9 if (c >> 3 & 15) == 0 else
                                         (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10)) if c & 127 != 127 else np.nan
                     for c in range(256)], dtype=F64)


def values(codes, scales):
    """What codes and scale bytes stand for."""
    v = E4M3.to(codes.device)[codes.long()]
    return v * torch.exp2(scales.to(F64) - 127).repeat_interleave(GROUP, -1)


def exponents(y):
    """E of each group of the last dimension (by comparison with every power)."""
    powers = 448 * torch.exp2(torch.arange(-100, 121, device=y.device, dtype=F64))
    amax = torch.where(torch.isfinite(y), y.abs(), 0.0).unflatten(-1, (-1, GROUP)).amax(-1)
    return torch.searchsorted(powers, amax.contiguous()) - 100


def nearest(x):
    """x rounded to the nearest e4m3 value, ties to the even one, saturating."""
    x = x.clamp(-512, 512)  # (all from 448 on saturate)
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -6))
    step = torch.exp2((e - 4).to(F64))
    return (torch.round(x / step) * step).clamp(-448, 448)


def rounded(y):
    """y through MXFP8."""
    p = torch.exp2(exponents(y).to(F64)).repeat_interleave(GROUP, -1)
    return nearest(y / p) * p


def bytes_of(y):
    """Codes and scale bytes of y."""
    e = exponents(y)
    v = nearest(y / torch.exp2(e.to(F64)).repeat_interleave(GROUP, -1))
    grid = E4M3[:127].to(y.device)
    codes = torch.searchsorted(grid, v.abs().contiguous())
    codes = torch.where(torch.isnan(v), 127, codes + 128 * torch.signbit(y))
    return codes.to(torch.uint8), (e + 127).to(torch.uint8)


def quantized_bound(y, off):
    """How far codes may be from y where y itself is off by `off`: half a step of
    e4m3 (2^-4 of a value, 2^-10 of the scale for the smallest), under a scale that
    may be the next larger one where the largest value is within `off` of its limit."""
    top = (y.abs() + off).unflatten(-1, (-1, GROUP)).amax(-1)
    p = torch.exp2(exponents(top.repeat_interleave(GROUP, -1)).to(F64)).repeat_interleave(GROUP, -1)
    return off + torch.maximum(2.0 ** -4 * (y.abs() + off), 2.0 ** -10 * p)


def quantize(x, apart=16):
    """MXFP8 of float64 values as the operators take it: scale rows a multiple of `apart` (4 or more) bytes apart."""
    codes, scales = bytes_of(x)
    rows, n = scales.shape
    held = torch.full((rows, -(-n // apart) * apart), 255, dtype=torch.uint8, device=x.device)  # (what is behind a row counts for nothing)
    held[:, :n] = scales
    return codes, held[:, :n]


def activation(kind, z):
    if kind == "relu":
        return torch.where(z < 0, 0.0, z)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return z * 0.5 * torch.erfc(-z * 0.5 ** 0.5)
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def product(x, w):
    """x w^T and how far a float32 sum of its exact products may be off: the tensor
    cores add 32 products at a time to the sum, each such addition off by 2^-23 of
    the magnitudes at most; up to 8 partial sums and a few further operations."""
    K = x.shape[-1]
    return x @ w.T, (x.abs() @ w.abs().T) * (K / 32 + 16) * 2.0 ** -23


def linear(x, w, bias, act, residual):
    """y and its bound before the last rounding."""
    z, off = product(x, w)
    if bias is not None:
        z = z + bias.to(F64)
        off = off + 2.0 ** -24 * z.abs()
    if act == "swiglu":
        gate, up = z.chunk(2, -1)
        og, ou = off.chunk(2, -1)
        g = gate * torch.sigmoid(gate)
        y = g * up
        # |silu'| <= 1.1; silu and the product within 2^-20 of their values
        off = 1.1 * og * (up.abs() + ou) + g.abs() * ou + 2.0 ** -20 * y.abs()
    else:
        y = activation(act, z)
        # slopes at most 1.13; erf, exp and quotients within 2^-20, relative to z (1 + erf cancels for negative z)
        off = 1.13 * off + (2.0 ** -20 * z.abs() if act != "none" and act != "relu" else 0.0)
    if residual is not None:
        y = y + residual.to(F64)
        off = off + 2.0 ** -24 * y.abs()
    return y, off


def moe(x, ids, weights, w13, w2, residual):
    """out and its bound (before the last rounding); w13 and w2 by expert."""
    T, K = x.shape
    out = torch.zeros((T, K), dtype=F64, device=x.device) if residual is None else residual.to(F64)
    off = torch.zeros_like(out)
    mass = torch.zeros_like(out)
    steps = 0
    for e in range(len(w13)):
        g = torch.where(ids == e, weights.to(F64), 0.0).sum(1)
        t = torch.where((ids == e).any(1))[0]
        if t.numel() == 0:
            continue
        F = w2[e].shape[1]
        y, o = linear(x[t], w13[e], None, "swiglu", None)
        y = y * g[t, None]
        o = o * g[t, None].abs() + 2.0 ** -22 * y.abs()
        h = rounded(y)
        # where y is that near to a border of the rounding or of the scale, the other side of it
        lo, hi = y - o, y + o
        top = torch.maximum(lo.abs(), hi.abs())
        p = [torch.exp2(exponents(v).to(F64)).repeat_interleave(GROUP, -1) for v in (y, (y.abs() - o).clamp(min=0), top)]
        other = [nearest(v / q) * q for v in (lo, hi) for q in p]
        jump = torch.stack([(v - h).abs() for v in other]).amax(0)
        out = out.index_add(0, t, h @ w2[e].T)
        off = off.index_add(0, t, jump @ w2[e].abs().T)
        mass = mass.index_add(0, t, h.abs() @ w2[e].abs().T)
        steps += F / 32 + 1
    return out, off + mass * (steps + 16) * 2.0 ** -23 + 2.0 ** -24 * out.abs()


def route(x, topk, scoring, bias, renormalize, scale, groups, topk_groups):
    """ids and weights of numpy float64 logits, one token at a time."""
    T, E = x.shape
    ids, weights = np.full((T, topk), -1), np.zeros((T, topk))
    for t in range(T):
        ok = x[t] > -np.inf
        if not ok.any():
            continue
        with np.errstate(over="ignore"):
            if scoring == "softmax":
                s = np.where(ok, np.exp(x[t] - x[t][ok].max()), 0.0)
                s = s / s.sum()
            else:
                s = 1 / (1 + np.exp(-x[t]))
        rank = x[t] if bias is None and groups == 1 else s + (0 if bias is None else bias)
        rank = np.where(ok, rank, -np.inf)
        if groups > 1:
            best = np.sort(rank.reshape(groups, -1), 1)[:, -2:].sum(1)
            kept = [g for g in np.argsort(-best, kind="stable")[:topk_groups] if best[g] > -np.inf]
            rank = np.where(np.isin(np.arange(E) // (E // groups), kept), rank, -np.inf)
        order = [e for e in np.argsort(-rank, kind="stable")[:topk] if rank[e] > -np.inf]
        w = s[order]
        if renormalize:
            w = w / w.sum()
        ids[t, :len(order)] = order
        weights[t, :len(order)] = w * scale
    return ids, weights
