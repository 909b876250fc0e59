"""Attention with changed scores in 64 bits, from the definition (include/fa.h): the tests'
oracle.  Works on torch float64 tensors, dense [B, H, N, d]."""
import math

import torch


def visible(B, N, causal, key_range):
    i = torch.arange(N)
    see = torch.ones(B, N, N, dtype=torch.bool)
    if causal:
        see &= i[None, :] <= i[:, None]
    if key_range is not None:
        r = key_range.long().clamp(0, N)
        see &= (i >= r[:, :, :1]) & (i < r[:, :, 1:])
    return see


def scores(q, k, causal, scale, softcap, slopes, key_range):
    """s [B, Hq, N, N] (-inf where hidden) and d s / d(scale q.k)."""
    B, Hq, N, _ = q.shape
    kk = k.repeat_interleave(Hq // k.shape[1], 1)
    x = scale * (q @ kk.mT)
    t = torch.tanh(x / softcap) if softcap else None
    s = softcap * t if softcap else x
    if slopes is not None:
        i = torch.arange(N, dtype=torch.float64)
        s = s - slopes.double().view(1, -1, 1, 1) * (i[:, None] - i[None, :]).abs()
    see = visible(B, N, causal, key_range)[:, None]
    return s.masked_fill(~see, -math.inf), (1 - t * t if softcap else torch.ones_like(s))


def softmax(s):
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[..., None])
    return torch.where(torch.isfinite(lse)[..., None], p, torch.zeros_like(p)), lse


def forward(q, k, v, causal=False, scale=1.0, softcap=0.0, slopes=None, key_range=None):
    """O, LSE and sum_j P_ij |v_jc| (for the error bound)."""
    s, _ = scores(q, k, causal, scale, softcap, slopes, key_range)
    p, lse = softmax(s)
    vv = v.repeat_interleave(q.shape[1] // k.shape[1], 1)
    return p @ vv, lse, p @ vv.abs()


def backward(q, k, v, o, lse, do, causal=False, scale=1.0, softcap=0.0, slopes=None, key_range=None):
    """dQ, dK, dV from given O and LSE, by the formulas of include/fa.h, and the same sums over
    absolute values (for the error bound)."""
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    s, fac = scores(q, k, causal, scale, softcap, slopes, key_range)
    live = torch.isfinite(lse)[..., None]
    p = torch.where(live, torch.exp(s - torch.where(live, lse[..., None], torch.zeros_like(s))), torch.zeros_like(s))
    kk, vv = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    delta = (do * o).sum(-1, keepdim=True)
    dp = do @ vv.mT
    ds = p * (dp - delta) * fac * scale
    mag = p * fac * scale * ((do.abs() @ vv.abs().mT) + (do * o).abs().sum(-1, keepdim=True))
    heads = lambda x: x.view(B, Hkv, g, N, d).sum(2)
    exact = (ds @ kk, heads(ds.mT @ q), heads(p.mT @ do))
    sums = (ds.abs() @ kk.abs(), heads(ds.abs().mT @ q.abs()), heads(p.mT @ do.abs()))
    more = (mag @ kk.abs(), heads(mag.mT @ q.abs()), torch.zeros_like(v))
    return exact, sums, more
