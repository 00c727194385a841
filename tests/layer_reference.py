"""Plain 64-bit computations of the operators in ``layer_ops``, on the CPU."""
import math

import torch

E4M3_MAX, SCALE_FLOOR = 448.0, 2.0 ** -100
BF16, FP32, E4M3 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4   # half a step, relative to the value
E4M3_TINY = 2.0 ** -10                               # half of e4m3's smallest step


def add_norm(x, weight=None, residual=None, eps=1e-6, norm=True):
    """(h, y, scale) in 64 bits"""
    h = x.double() + (0 if residual is None else residual.double())
    y = h
    if norm:
        y = h / (h.square().mean(-1, keepdim=True) + eps).sqrt()
        if weight is not None:
            y = y * weight.double()
    amax = y.abs().amax(-1)
    scale = torch.where(torch.isfinite(y).all(-1), amax.clamp(min=SCALE_FLOOR) / E4M3_MAX, math.nan)
    return h, y, scale


def linear(x, weight, x_scale=None, weight_scale=None, bias=None, residual=None, activation=None):
    """(out, bound): the product in 64 bits, and what fp32 sums of its products may be off by.

    A product instruction adds 16 (bf16) or 32 (e4m3) products to the sum, which is cut to 24 bits; what it cuts of
    the products before they are added is bounded alike.  So every 16 of k cost at most two steps, 2^-22, of the sum
    of the absolute products; the epilogue's four roundings another 2^-22."""
    a, w = x.double(), weight.double()
    y, mag = a @ w.t(), a.abs() @ w.abs().t()
    if x_scale is not None:
        s = x_scale.double()[:, None] * weight_scale.double()
        y, mag = y * s, mag * s.abs()
    if bias is not None:
        y, mag = y + bias.double(), mag + bias.double().abs()
    err = mag * (x.shape[1] / 16 + 1) * 2.0 ** -22
    half = weight.shape[0] // 2
    sig = torch.sigmoid(y)
    # activations: their slopes are below 1.13; silu's exponential is off by 2^-18; gelu's erfc by 1.2e-7 < 2^-22, its
    # exponent -y^2 / 2 and what is added to it (below 2) by three roundings of their sum, the exponential of the exact
    # exponent's rounded multiple of log2 e by as much again, and four more roundings: all relative to the result
    if activation == "silu":
        y, err = y * sig, 1.13 * err + (y * sig).abs() * 2.0 ** -18
    elif activation == "gelu":
        g = y * 0.5 * torch.special.erfc(-y / math.sqrt(2))
        y, err = g, 1.13 * err + g.abs() * (2.0 ** -20 + (y.square() / 2 + 2) * 2.0 ** -21) + 2.0 ** -126
    elif activation == "silu_gated":
        g = (y * sig)[:, :half]
        e = 1.13 * err[:, :half] + g.abs() * 2.0 ** -18
        err = e * y[:, half:].abs() + (g.abs() + e) * err[:, half:]
        y = g * y[:, half:]
    if residual is not None:
        y = y + residual.double()
    return y, err + y.abs() * 2.0 ** -23


def logprobs(logits, tokens=None, num_top=0):
    """(logprobs, ranks, entropy, top_ids, top_logprobs, scale): scale is what errors are relative to"""
    x = logits.double().reshape(-1, logits.shape[-1])
    R, V = x.shape
    lp, ent, scale = (torch.zeros(R, dtype=torch.float64) for _ in range(3))
    ranks = torch.full((R,), -1, dtype=torch.int32)
    ids, top = torch.full((R, num_top), -1, dtype=torch.int32), torch.zeros(R, num_top, dtype=torch.float64)
    tok = None if tokens is None else tokens.reshape(-1).tolist()
    for r in range(R):
        if tok is not None and not 0 <= tok[r] < V:
            continue
        z = x[r]
        if torch.isnan(z).any() or z.max().abs() == math.inf:
            lp[r] = ent[r] = math.nan
            top[r] = math.nan
            continue
        lse = torch.logsumexp(z, 0)
        p = torch.exp(z - lse)
        ent[r] = torch.special.entr(p).sum()
        scale[r] = 2 + math.log(V) + (p * (z - z.max()).clamp(min=-1e4)).sum().abs()
        v, order = torch.sort(z, stable=True, descending=True)
        if tok is not None:
            lp[r] = z[tok[r]] - lse
            ranks[r] = (order == tok[r]).nonzero().item()
        n = min(num_top, V)
        ids[r, :n], top[r, :n] = order[:n].int(), v[:n] - lse
        top[r, n:] = -math.inf
    shape = logits.shape[:-1]
    out = [lp.view(shape), ranks.view(shape), ent.view(shape), ids.view(*shape, num_top), top.view(*shape, num_top)]
    if tok is None:
        out[0] = out[1] = None
    return (*out, scale.view(shape))
