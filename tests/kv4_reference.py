"""The 4-bit cache format and attention over it, written out in 64 bits on the CPU from the
format's definition (include/fa.h): the tests' oracle."""
import numpy as np

GROUP, CLAMP = 32, 57344.0

_half = np.arange(65536, dtype=np.uint16).view(np.float16).astype(np.float64)
_TABLE = np.unique(_half[np.isfinite(_half)])            # every fp16 number, ascending


def quantise(x):
    """Codes (int) [..., G, 32] and s, m (float64 holding fp16 numbers) [..., G] of x [..., d]."""
    y = np.asarray(x, dtype=np.float64)
    y = y.reshape(*y.shape[:-1], -1, GROUP)
    bad = ~np.isfinite(y).all(-1)
    y = np.clip(np.where(bad[..., None], 0.0, y), -CLAMP, CLAMP)
    lo, hi = y.min(-1), y.max(-1)
    m = _TABLE[np.searchsorted(_TABLE, lo, side="right") - 1]
    steps = _TABLE[_TABLE >= 0]
    at = np.searchsorted(steps, (hi - m) / 15.0)
    s = np.full_like(m, np.inf)
    for k in (1, 0, -1):
        c = steps[np.clip(at + k, 0, len(steps) - 1)]
        s = np.where(m + 15.0 * c >= hi, np.minimum(s, c), s)
    n = np.zeros(y.shape, dtype=np.int64)
    for k in range(15):
        n += (y >= (m + (k + 0.5) * s)[..., None]).astype(np.int64)
    n = np.where((s == 0)[..., None] | bad[..., None], 0, n)
    return n, np.where(bad, 0.0, s), np.where(bad, np.nan, m)


def pack(n, s, m, is_k):
    """(codes uint8 [..., d/2], params fp16 [..., 2G]) in the cache's layout."""
    G = n.shape[-2]
    w = n.reshape(*n.shape[:-2], G, 4, 8)                 # group, word, channel
    if is_k:
        w = np.swapaxes(w, -3, -2)                        # word c of group i at place c G + i
    w = w.reshape(*w.shape[:-3], 4 * G, 4, 2)
    codes = (w[..., 0] | (w[..., 1] << 4)).astype(np.uint8)
    codes = codes.reshape(*codes.shape[:-2], -1)
    params = np.concatenate((s, m), -1) if is_k else np.stack((s, m), -1).reshape(*s.shape[:-1], -1)
    return codes, params.astype(np.float16)


def values(n, s, m):
    """What a token stands for, [..., d] in 64 bits."""
    y = m[..., None] + n * s[..., None]
    return y.reshape(*y.shape[:-2], -1)


def decode(q, k, v, lens, causal, scale, softcap=0.0, slopes=None):
    """O, LSE in 64 bits of rows q [B, Hq, Nq, d] over k, v [B, Hkv, Nk, d], and for the error
    bound: sum_j P_j |v_j| like O, and the largest scale sum_c |q_c k_c| of each row."""
    B, Hq, Nq, d = q.shape
    g = Hq // k.shape[1]
    o = np.zeros((B, Hq, Nq, d))
    av = np.zeros((B, Hq, Nq, d))
    lse = np.full((B, Hq, Nq), -np.inf)
    size = np.zeros((B, Hq, Nq))
    for b in range(B):
        n = k.shape[2] if lens is None else max(0, min(int(lens[b]), k.shape[2]))
        j = np.arange(n)
        for h in range(Hq):
            kk, vv = k[b, h // g, :n], v[b, h // g, :n]
            for t in range(Nq):
                pos = n - Nq + t
                s = scale * (kk @ q[b, h, t])
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - slopes[h] * np.abs(pos - j)
                if causal:
                    s = np.where(j <= pos, s, -np.inf)
                if n == 0 or not np.isfinite(s).any():
                    continue
                top = s.max()
                e = np.exp(s - top)
                lse[b, h, t] = top + np.log(e.sum())
                p = e / e.sum()
                o[b, h, t] = p @ vv
                av[b, h, t] = p @ np.abs(vv)
                size[b, h, t] = scale * (np.abs(kk) @ np.abs(q[b, h, t])).max()
    return o, lse, av, size
