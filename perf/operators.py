"""The cases on which the score-modified attention and the 4-bit key/value cache are measured.

Five kinds of case, one per direction or form of an operator:

* ``fwd``    - fa.fwd with a tanh cap on the scores, a bias that falls with the distance, and/or a
               key range per query row (documents, prefixes, padding);
* ``bwd``    - fa.bwd of the same, from Q, K, V, O, LSE and dO;
* ``decode`` - fa.decode with the same scores: a few new query rows over a bf16 cache;
* ``store``  - fa.kv4_write of new tokens into a 4-bit cache, and fa.kv4_read of them;
* ``kv4``    - fa.decode_kv4: a few new query rows over the 4-bit cache.

``run`` computes them from elementary torch operations, or, with ``own``, by the library's calls.
"""
import math

import torch

own = False

GROUP = 32          # channels that share a scale and a minimum in the 4-bit cache
CLAMP = 57344.0     # values are clamped to this before they are quantised


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one short sequence of a small model with capped scores: launch latency
        dict(name="fwd capped 200", kind="fwd", B=1, Hq=4, Hkv=2, N=200, d=64, causal=True, cap=20.0,
             alibi=False, mask="none"),
        # training or prefill of a grouped-query model with capped scores at 4k
        dict(name="fwd capped gqa 4k", kind="fwd", B=2, Hq=32, Hkv=8, N=4096, d=128, causal=True, cap=50.0,
             alibi=False, mask="none"),
        # 8k rows packed with nine documents and padding, distance bias
        dict(name="fwd documents 8k", kind="fwd", B=1, Hq=16, Hkv=16, N=8192, d=128, causal=True, cap=0.0,
             alibi=True, mask="docs"),
        # gradient of the capped scores at 4k
        dict(name="bwd capped 4k", kind="bwd", B=2, Hq=16, Hkv=16, N=4096, d=128, causal=True, cap=50.0,
             alibi=False, mask="none"),
        # gradient with visible prefixes and a distance bias, an odd length, three heads a group
        dict(name="bwd prefix 1000", kind="bwd", B=2, Hq=6, Hkv=2, N=1000, d=64, causal=False, cap=0.0,
             alibi=True, mask="prefix"),
        # gradient at the largest head dimension, capped, documents
        dict(name="bwd documents d256", kind="bwd", B=2, Hq=8, Hkv=4, N=2048, d=256, causal=True, cap=30.0,
             alibi=False, mask="docs"),
        # one new token over a short cache: launch latency
        dict(name="decode capped 333", kind="decode", B=2, Hq=8, Hkv=2, Nq=1, Nk=333, d=64, causal=False,
             cap=30.0, alibi=False),
        # one new token of four long conversations
        dict(name="decode capped 64k", kind="decode", B=4, Hq=32, Hkv=8, Nq=1, Nk=65536, d=128, causal=False,
             cap=50.0, alibi=False),
        # one new token of 64 conversations written to their caches
        dict(name="store one token", kind="store", B=64, Hkv=8, n=1, room=4096, d=128),
        # two prompts of an odd length written to their caches
        dict(name="store prompt", kind="store", B=2, Hkv=8, n=16001, room=16384, d=128),
        # one new token over a short 4-bit cache: launch latency
        dict(name="kv4 short", kind="kv4", B=1, Hq=8, Hkv=2, Nq=1, Nk=256, d=64, causal=False, cap=0.0,
             alibi=False),
        # one new token of four long conversations over 4-bit caches
        dict(name="kv4 64k", kind="kv4", B=4, Hq=32, Hkv=8, Nq=1, Nk=65536, d=128, causal=False, cap=0.0,
             alibi=False),
    ]


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["fwd", "bwd", "decode", "store", "kv4"])
    d = rng.choice([64, 128, 256])
    cap, alibi = rng.choice([(20.0, False), (50.0, False), (0.0, True), (30.0, True)])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 3, 4, 8])
    if kind in ("fwd", "bwd"):
        N = _between(rng, 1, 6000)
        most = 2 ** 28 if kind == "bwd" else 2 ** 29
        while Hkv * g * N * N > most // (d // 64):
            N = N * 2 // 3
        B = rng.randint(1, max(1, min(4, most // (d // 64) // (Hkv * g * N * N))))
        mask = rng.choice(["none", "docs", "prefix"])
        return dict(kind=kind, B=B, Hq=Hkv * g, Hkv=Hkv, N=N, d=d, causal=mask == "docs" or rng.random() < 0.5,
                    cap=cap, alibi=alibi, mask=mask)
    if kind == "store":
        room = _between(rng, 1, 1024) * 64
        B = _between(rng, 1, 64)
        while B * Hkv * room * d > 2 ** 26:
            room = max(64, room // 128 * 64)
            B = max(1, B // 2)
        return dict(kind=kind, B=B, Hkv=Hkv, n=rng.choice([1, _between(rng, 1, room)]), room=room, d=d)
    Nk = _between(rng, 1, 60000)
    B = _between(rng, 1, 32)
    while B * Hkv * Nk * d > 2 ** 27:
        Nk, B = max(1, Nk * 2 // 3), max(1, B // 2)
    return dict(kind=kind, B=B, Hq=Hkv * g, Hkv=Hkv, Nq=rng.choice([1, 1, 2, 5]), Nk=Nk, d=d,
                causal=rng.random() < 0.5, cap=cap, alibi=alibi)


# ----------------------------------------------------------------------------------------- inputs

def _doc_lengths(N):
    """Nine document lengths, the longest sixteen times the shortest, that leave N // 16 rows of padding."""
    total = N - N // 16
    w = [2.0 ** (i / 2.0) for i in range(9)]
    cuts = [0] + [int(round(total * sum(w[:i + 1]) / sum(w))) for i in range(9)]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _prefixes(B, N):
    return [(b + 1) * N // (B + 2) for b in range(B)]


def _key_range(case, gen):
    """int32 [B, N, 2]: the keys lo <= j < hi that each query row may see (None: all)."""
    B, N = case["B"], case["N"]
    if case["mask"] == "none":
        return None
    rng = torch.zeros(B, N, 2, dtype=torch.int32)
    order = torch.randperm(B, generator=gen).tolist()
    for b in range(B):
        if case["mask"] == "docs":
            lengths, at = _doc_lengths(N), 0
            for i in torch.randperm(len(lengths), generator=gen).tolist():
                rng[b, at:at + lengths[i], 0] = at
                rng[b, at:at + lengths[i], 1] = at + lengths[i]
                at += lengths[i]
        else:
            rng[b, :, 1] = torch.clamp(torch.arange(1, N + 1, dtype=torch.int32), min=_prefixes(B, N)[order[b]])
    return rng.cuda()


def _slopes(case):
    H = case["Hq"]
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda") \
        if case["alibi"] else None


def _lengths(case, gen):
    """int32 [B]: valid keys, the first batch entry's all, the others from a quarter of them up."""
    n = torch.randint(max(1, case["Nk"] // 4), case["Nk"] + 1, (case["B"],), generator=gen)
    n[0] = case["Nk"]
    return n.to(torch.int32).cuda()


def _keys(shape, gen):
    """Keys with a few channels four times as large as the others, as trained models have."""
    k = torch.randn(shape, generator=gen, device="cuda")
    k[..., ::16] *= 4.0
    return k.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    bf = lambda *s, f=1.0: (torch.randn(s, generator=gen, device="cuda") * f).to(torch.bfloat16)  # noqa: E731
    st = dict(case)
    d, B, Hkv = case["d"], case["B"], case["Hkv"]
    if case["kind"] in ("fwd", "bwd"):
        N = case["N"]
        st["q"], st["k"], st["v"] = bf(B, case["Hq"], N, d, f=2.0), bf(B, Hkv, N, d), bf(B, Hkv, N, d)
        st["range"], st["slopes"] = _key_range(case, host), _slopes(case)
        if case["kind"] == "bwd":
            st["do"] = bf(B, case["Hq"], N, d)
            st["o"], st["lse"] = _plain_fwd(st)
    elif case["kind"] == "store":
        st["k"], st["v"] = _keys((B, Hkv, case["n"], d), gen), bf(B, Hkv, case["n"], d)
        st["start"] = torch.randint(case["room"] - case["n"] + 1, (B,), generator=host).to(torch.int32).cuda()
        st["cache"] = _new_cache(B, Hkv, case["room"], d)
    else:
        Nk = case["Nk"]
        st["q"], st["slopes"] = bf(B, case["Hq"], case["Nq"], d), _slopes(case)
        k, v = _keys((B, Hkv, Nk, d), gen), bf(B, Hkv, Nk, d)
        st["lens"] = _lengths(case, host)
        if case["kind"] == "decode":
            st["k"], st["v"] = k, v
        else:
            st["cache"] = _new_cache(B, Hkv, -(-Nk // 64) * 64, d)
            _plain_write(st["cache"], k, v, torch.zeros(B, dtype=torch.int32, device="cuda"))
    return st


# -------------------------------------------------------------------- plain forms: scaled scores

def _plain_scores(s, cap, slopes, qpos, kpos, shape):
    """Capped scores and their bias: s [..., rows, keys] after the scale, heads flattened as `shape`."""
    t = torch.tanh(s / cap) if cap else None
    s = cap * t if cap else s
    if slopes is not None:
        far = (qpos[..., :, None] - kpos).abs().to(s.dtype)
        s = s - slopes.to(s.dtype).view(shape) * far
    return s, t


def _visible(st):
    """[B or 1, N, N] truth values: key j is visible to query i."""
    N = st["N"]
    j = torch.arange(N, device="cuda")
    see = torch.ones(1, N, N, dtype=torch.bool, device="cuda")
    if st["causal"]:
        see = see & (j[None, :] <= j[:, None])
    if st["range"] is not None:
        see = see & (j >= st["range"][:, :, 0, None]) & (j < st["range"][:, :, 1, None])
    return see


def _softmax_parts(s):
    """Weights e, their sum l and the logsumexp of the rows of s; a row of -inf alone gets e = 0, l = 1, LSE = -inf."""
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    l = e.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(m, -math.inf))
    return e, torch.where(l > 0, l, torch.ones_like(l)), lse.squeeze(-1)


def _grouped(st):
    """Scaled, capped and biased scores [B, Hkv, g, N, N] of a fwd or bwd case, hidden ones -inf, and the tanh."""
    B, Hq, Hkv, N, d = (st[n] for n in ("B", "Hq", "Hkv", "N", "d"))
    g = Hq // Hkv
    q = st["q"].float().view(B, Hkv, g, N, d)
    pos = torch.arange(N, device="cuda")
    s = torch.matmul(q, st["k"].float().unsqueeze(2).transpose(-1, -2)) * (1.0 / math.sqrt(d))
    s, t = _plain_scores(s, st["cap"], st["slopes"], pos, pos, (Hkv, g, 1, 1))
    return s.masked_fill_(~_visible(st)[:, None, None], -math.inf), t


def _plain_fwd(st):
    B, Hq, Hkv, N, d = (st[n] for n in ("B", "Hq", "Hkv", "N", "d"))
    e, l, lse = _softmax_parts(_grouped(st)[0])
    o = torch.matmul(e, st["v"].float().unsqueeze(2)) / l
    return o.view(B, Hq, N, d).to(torch.bfloat16), lse.reshape(B, Hq, N)


def _plain_bwd(st):
    B, Hq, Hkv, N, d = (st[n] for n in ("B", "Hq", "Hkv", "N", "d"))
    g, scale = Hq // Hkv, 1.0 / math.sqrt(d)
    s, t = _grouped(st)
    lse = st["lse"].view(B, Hkv, g, N, 1)
    p = torch.where(torch.isfinite(lse), torch.exp(s - lse), torch.zeros_like(s))
    del s
    do = st["do"].float().view(B, Hkv, g, N, d)
    delta = (do * st["o"].float().view(B, Hkv, g, N, d)).sum(-1, keepdim=True)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = p * (torch.matmul(do, st["v"].float().unsqueeze(2).transpose(-1, -2)) - delta)
    del p
    if t is not None:
        ds = ds * (1.0 - t * t)
    dq = torch.matmul(ds, st["k"].float().unsqueeze(2)) * scale
    dk = torch.matmul(ds.transpose(-1, -2), st["q"].float().view(B, Hkv, g, N, d)).sum(2) * scale
    return dq.view(B, Hq, N, d).to(torch.bfloat16), dk.to(torch.bfloat16), dv.to(torch.bfloat16)


def _plain_cached(st, k, v):
    """New rows q over the caches k, v (fp32 values) of which the first lens[b] keys count."""
    B, Hq, Hkv, Nq, d = (st[n] for n in ("B", "Hq", "Hkv", "Nq", "d"))
    g, Nk = Hq // Hkv, k.shape[2]
    s = torch.matmul(st["q"].float().view(B, Hkv, g * Nq, d), k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    s = s.view(B, Hkv, g, Nq, Nk)
    key = torch.arange(Nk, device="cuda")
    pos = st["lens"].long()[:, None] - Nq + torch.arange(Nq, device="cuda")      # of each new row
    s, _ = _plain_scores(s, st["cap"], st["slopes"], pos[:, None, None], key, (Hkv, g, 1, 1))
    last = pos if st["causal"] else (st["lens"].long()[:, None] - 1).expand(B, Nq)
    e, l, lse = _softmax_parts(s.masked_fill(key > last[:, None, None, :, None], -math.inf))
    o = torch.matmul(e.view(B, Hkv, g * Nq, Nk), v).view(B, Hkv, g, Nq, d) / l
    return o.reshape(B, Hq, Nq, d).to(torch.bfloat16), lse.reshape(B, Hq, Nq)


# -------------------------------------------------------------------- plain forms: the 4-bit cache
#
# Each token holds, for every 32 channels, fp16 numbers m (the largest one not above the group's
# least value) and s (the least one with m + 15 s not below its largest), and for each channel the
# code n in 0..15 whose m + n s is nearest to the value, the larger one of two.  Codes lie in 32-bit
# words of 8 channels, the first channel in the lowest bits; V's words in the channels' order, K's
# with word c of group i at place c * groups + i.

def _new_cache(B, Hkv, room, d):
    z = lambda n, t: torch.zeros(B, Hkv, room, n, dtype=t, device="cuda")  # noqa: E731
    return (z(d // 2, torch.uint8), z(2 * d // GROUP, torch.float16), z(d // 2, torch.uint8), z(2 * d // GROUP, torch.float16))


def _step16(h, up):
    """The neighbour of the fp16 numbers h above (up) or below."""
    bits = h.view(torch.int16).to(torch.int32) & 0xFFFF
    away = (bits < 0x8000) == up                                # from zero
    zero = (bits & 0x7FFF) == 0
    stepped = torch.where(zero, torch.full_like(bits, 1 if up else 0x8001), bits + torch.where(away, 1, -1))
    return ((stepped + 0x8000) % 0x10000 - 0x8000).to(torch.int16).view(torch.float16)


def _plain_quantise(x):
    """Codes (int32) [..., G, 32], s and m (fp16) [..., G] of x [..., d]."""
    x = x.double().clamp(-CLAMP, CLAMP).unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1), x.amax(-1)
    m = lo.half()
    m = torch.where(m.double() > lo, _step16(m, False), m)
    s = ((hi - m.double()) / 15.0).half()
    s = torch.where(m.double() + 15.0 * s.double() < hi, _step16(s, True), s)
    low = _step16(s, False)
    s = torch.where((s > 0) & (m.double() + 15.0 * low.double() >= hi), low, s)
    step = torch.where(s > 0, s.double(), torch.ones_like(hi))[..., None]
    n = torch.floor((x - m.double()[..., None]) / step + 0.5).clamp(0, 15)
    return torch.where(s[..., None] > 0, n, torch.zeros_like(n)).to(torch.int32), s, m


def _pack(n, interleave):
    """Codes [..., G, 32] to bytes [..., d / 2]."""
    w = n.unflatten(-1, (4, 4, 2))                                             # [..., G, word, byte, nibble]
    w = w[..., 0] | (w[..., 1] << 4)
    if interleave:
        w = w.transpose(-3, -2)
    return w.flatten(-3).to(torch.uint8)


def _unpack(c, interleave):
    G = c.shape[-1] // 16
    w = c.unflatten(-1, (4, G, 4) if interleave else (G, 4, 4))
    w = w.transpose(-3, -2) if interleave else w
    return torch.stack((w & 15, w >> 4), -1).flatten(-3)                       # [..., G, 32]


def _plain_write(cache, k, v, start):
    kc, kp, vc, vp = cache
    n, s, m = _plain_quantise(k)
    at = (start.long()[:, None] + torch.arange(k.shape[2], device="cuda"))[:, None, :, None].expand(-1, k.shape[1], -1, -1)
    put = lambda t, x: t.scatter_(2, at.expand(*at.shape[:3], t.shape[-1]), x)  # noqa: E731
    put(kc, _pack(n, True))
    put(kp, torch.cat((s, m), -1))
    n, s, m = _plain_quantise(v)
    put(vc, _pack(n, False))
    put(vp, torch.stack((s, m), -1).flatten(-2))


def _plain_values(cache):
    """The values (fp32) that a cache's tokens stand for."""
    kc, kp, vc, vp = cache
    ks, km = kp.float().unflatten(-1, (2, -1)).unbind(-2)
    vs, vm = vp.float().unflatten(-1, (-1, 2)).unbind(-1)
    k = _unpack(kc, True).float() * ks[..., None] + km[..., None]
    v = _unpack(vc, False).float() * vs[..., None] + vm[..., None]
    return k.flatten(-2), v.flatten(-2)


def _plain_read(cache, start, n):
    at = (start.long()[:, None] + torch.arange(n, device="cuda"))[:, None, :, None]
    part = tuple(torch.gather(t, 2, at.expand(-1, t.shape[1], -1, t.shape[3])) for t in cache)
    return tuple(x.to(torch.bfloat16) for x in _plain_values(part))


# -------------------------------------------------------------------------------------------- run

def _own_run(st):
    from exact_io_aware_83_b200 import fa
    kind = st["kind"]
    if kind == "store":
        cache = fa.KV4Cache(*st["cache"])
        fa.kv4_write(cache, st["k"], st["v"], start=st["start"])
        return fa.kv4_read(cache, st["n"], start=st["start"])
    extra = dict(causal=st["causal"], softcap=st["cap"], alibi_slopes=st["slopes"])
    if kind == "fwd":
        return fa.fwd(st["q"], st["k"], st["v"], key_range=st["range"], **extra)
    if kind == "bwd":
        return fa.bwd(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], key_range=st["range"], **extra)
    if kind == "decode":
        return fa.decode(st["q"], st["k"], st["v"], seqlens_k=st["lens"], **extra)
    return fa.decode_kv4(st["q"], fa.KV4Cache(*st["cache"]), seqlens_k=st["lens"], **extra)


def run(state):
    if own:
        return _own_run(state)
    kind = state["kind"]
    if kind == "fwd":
        return _plain_fwd(state)
    if kind == "bwd":
        return _plain_bwd(state)
    if kind == "store":
        _plain_write(state["cache"], state["k"], state["v"], state["start"])
        return _plain_read(state["cache"], state["start"], state["n"])
    if kind == "decode":
        return _plain_cached(state, state["k"].float(), state["v"].float())
    return _plain_cached(state, *_plain_values(state["cache"]))


# ------------------------------------------------------------------------------------------- work

def _pairs(case):
    """Visible (query, key) pairs of one batch's head, summed over the batch."""
    B, N = case["B"], case["N"]
    half = N * (N + 1) // 2
    if case["mask"] == "docs":
        return B * sum(n * (n + 1) // 2 if case["causal"] else n * n for n in _doc_lengths(N))
    if case["mask"] == "prefix" and not case["causal"]:
        return sum(half + p * (p - 1) // 2 for p in _prefixes(B, N))
    return B * (half if case["causal"] else N * N)


def work(case):
    d, B, Hkv = case["d"], case["B"], case["Hkv"]
    if case["kind"] == "store":
        values = 2 * B * Hkv * case["n"] * d
        held = values // 2 + values // GROUP * 4
        return {"bytes": 4 * values + 2 * held, "flops": 8 * values}
    Hq = case["Hq"]
    if case["kind"] in ("fwd", "bwd"):
        N, pairs = case["N"], _pairs(case) * Hq
        qo, kv, rows = 2 * B * Hq * N * d, 2 * B * Hkv * N * d, 4 * B * Hq * N
        ranges = 8 * B * N if case["mask"] != "none" else 0
        if case["kind"] == "fwd":
            return {"bytes": 2 * qo + 2 * kv + rows + ranges, "flops": 4 * d * pairs}
        return {"bytes": 4 * qo + 4 * kv + rows + ranges, "flops": 10 * d * pairs}
    # the first batch entry has all keys, the others five eighths of them on average
    keys = int(case["Nk"] * (1 + 0.625 * (B - 1))) * Hkv
    row = 4 * d if case["kind"] == "decode" else d + 8 * d // GROUP
    return {"bytes": keys * row + 4 * B * Hq * case["Nq"] * d + 4 * B * Hq * case["Nq"],
            "flops": 4 * d * keys * (Hq // Hkv) * case["Nq"]}


# ------------------------------------------------------------------------------------------ exact

def _exact_row_block(q, k, cap, slope, i, j, see):
    """Scores in 64 bits of rows q over keys k, after the scale; hidden pairs -inf. Also d(score)/d(raw)."""
    raw = (q @ k.mT) / math.sqrt(q.shape[-1])
    grad = torch.ones_like(raw)
    if cap:
        u = torch.exp(-2.0 * raw.abs() / cap)
        grad = 4.0 * u / (1.0 + u) ** 2                                  # 1 / cosh^2
        raw = cap * raw.sign() * (1.0 - u) / (1.0 + u)
    if slope is not None:
        raw = raw - slope * (i[:, None] - j[None, :]).abs().double()
    return torch.where(see, raw, torch.full_like(raw, -math.inf)), grad


def _exact_rows(s, v):
    """O and LSE in 64 bits of score rows over values v."""
    lse = torch.logsumexp(s, -1)
    p = torch.where(torch.isfinite(lse)[:, None], torch.exp(s - lse[:, None]), torch.zeros_like(s))
    return p @ v, lse, p


def _exact_see(st, b):
    N = st["N"]
    i = torch.arange(N, device="cuda")
    lo, hi = torch.zeros_like(i), torch.full_like(i, N)
    if st["range"] is not None:
        lo, hi = st["range"][b].long().unbind(-1)
    if st["causal"]:
        hi = torch.minimum(hi, i + 1)
    return i, (i[None, :] >= lo[:, None]) & (i[None, :] < hi[:, None])


def _exact_groups(x):
    """What each value of x [..., d] becomes when it is held in 4 bits, in 64 bits."""
    x = x.double().clamp(-CLAMP, CLAMP)
    y = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    halves = torch.arange(65536, dtype=torch.int32, device="cuda")
    halves = ((halves + 0x8000) % 0x10000 - 0x8000).to(torch.int16).view(torch.float16).double()
    table = halves[torch.isfinite(halves)].unique()                       # every fp16 number, ascending
    m = table[torch.searchsorted(table, y.amin(-1).contiguous(), right=True) - 1]
    near = torch.searchsorted(table, ((y.amax(-1) - m) / 15.0).contiguous())
    s = torch.full_like(m, math.inf)
    for k in (1, 0, -1):                                                  # the least one that reaches the top
        c = table[(near + k).clamp(0, table.numel() - 1)]
        s = torch.where((c >= 0) & (m + 15.0 * c >= y.amax(-1)), torch.minimum(s, c), s)
    out = torch.zeros_like(y)
    for k in range(15):
        out += (y >= (m + (k + 0.5) * s)[..., None]).double()
    return (m[..., None] + out * s[..., None]).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    kind, B, Hkv = case["kind"], case["B"], case["Hkv"]
    if kind == "store":
        return tuple(_exact_groups(st[n]) for n in ("k", "v"))
    g = case["Hq"] // Hkv
    slopes = st["slopes"].double() if st["slopes"] is not None else None
    at = lambda b, h: (b, h // g)  # noqa: E731
    heads = [(b, h) for b in range(B) for h in range(case["Hq"])]
    if kind in ("fwd", "bwd"):
        q, k, v = (st[n].double() for n in ("q", "k", "v"))
        o, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for b, h in heads:
            i, see = _exact_see(st, b)
            s, grad = _exact_row_block(q[b, h], k[at(b, h)], case["cap"], slopes[h] if slopes is not None else None, i, i, see)
            if kind == "fwd":
                o[b, h], lse[b, h], _ = _exact_rows(s, v[at(b, h)])
                continue
            do, l = st["do"][b, h].double(), st["lse"][b, h].double()
            p = torch.where(torch.isfinite(l)[:, None], torch.exp(s - l[:, None]), torch.zeros_like(s))
            dv[at(b, h)] += p.mT @ do
            ds = p * (do @ v[at(b, h)].mT - (do * st["o"][b, h].double()).sum(-1, keepdim=True)) * grad / math.sqrt(case["d"])
            dq[b, h] = ds @ k[at(b, h)]
            dk[at(b, h)] += ds.mT @ q[b, h]
        return (o, lse) if kind == "fwd" else (dq, dk, dv)
    Nq, Nk = case["Nq"], case["Nk"]
    if kind == "kv4":  # the cache is an input: the values that it stands for
        kc, kp, vc, vp = st["cache"]
        G = case["d"] // GROUP
        ch = torch.arange(case["d"], device="cuda")
        kbyte = 4 * ((ch % GROUP) // 8 * G + ch // GROUP) + ch % 8 // 2
        k = ((kc[..., kbyte].long() >> (4 * (ch % 2))) & 15).double() * kp[..., ch // GROUP].double() + kp[..., G + ch // GROUP].double()
        v = ((vc[..., ch // 2].long() >> (4 * (ch % 2))) & 15).double() * vp[..., ch // GROUP * 2].double() + vp[..., ch // GROUP * 2 + 1].double()
    else:
        k, v = st["k"], st["v"]
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["q"].shape[:3], dtype=torch.float64, device="cuda")
    for b, h in heads:
        n = int(st["lens"][b])
        i, j = torch.arange(n - Nq, n, device="cuda"), torch.arange(n, device="cuda")
        see = (j[None, :] <= i[:, None]) if case["causal"] else torch.ones(Nq, n, dtype=torch.bool, device="cuda")
        s, _ = _exact_row_block(st["q"][b, h].double(), k[at(b, h)][:n].double(), case["cap"],
                                slopes[h] if slopes is not None else None, i, j, see)
        o[b, h], lse[b, h], _ = _exact_rows(s, v[at(b, h)][:n].double())
    return o, lse
