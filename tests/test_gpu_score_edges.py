"""Attention with changed scores at the edges of its arguments, on the GPU against 64-bit
references: key ranges that lie far apart or at the ends of int32, caps from the smallest fp32
number to the largest.  Bounds as in test_gpu_score.py unless a test gives its own."""
import math

import numpy as np
import pytest
import torch

import kv4_reference
import score_reference as ref
from exact_io_aware_83_b200 import fa
from test_gpu_kv4 import _cache_of, _f64
from test_gpu_score import _decode_ref, _draw, _guarded, _slopes, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("near,far", [((0, 128), (384, 640)), ((0, 100), (512, 520)), ((130, 140), (900, 1000)),
                                      ((0, 1), (1023, 1024)), ((0, 128), (128, 1024))])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (2, 1)])
def test_neighbouring_tiles_that_see_far_apart_keys(d, near, far, Hq, Hkv):
    # with an odd group one CTA takes two 128-row tiles, here with key blocks between those of the
    # two that neither sees; the two tiles in either order, one of them empty, then ordinary rows
    N = 1024
    lo, hi = torch.zeros(2, N, dtype=torch.int64), torch.full((2, N), N, dtype=torch.int64)
    for b, pair in enumerate(((near, far), (far, near))):
        for t, (a, z) in enumerate(pair):
            lo[b, 128 * t:128 * t + 128], hi[b, 128 * t:128 * t + 128] = a, z
        lo[b, 256:384], hi[b, 256:384] = 0, 0
        lo[b, 384:512], hi[b, 384:512] = pair[0]
    r = torch.stack((lo, hi), -1).to(torch.int32)
    q, k, v, do = _draw(2, Hq, Hkv, N, d, seed=d + Hq + near[0] + far[0])
    check(q, k, v, do, key_range=r)
    check(q, k, v, do, key_range=r, softcap=20.0, slopes=_slopes(Hq))


# Caps far above the scores.  The score c tanh(x / c) is then nearly x, whatever c, so nothing in
# these bounds may grow with the cap: a score s is off by the tanh's 5.4e-7 |s| and eight
# fp32 roundings (of 1 / c, c log2(e) and the products: 2^-24 |s| each), below 2^-19.5 |s| in all,
# on top of the product's 2^-17 A (A_i = scale max_j sum_c |q_c k_c|, which also bounds |s|).

LARGE = 2.0 ** -17 + 2.0 ** -19.5


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,Nq,Nk,lens", [(8, 2, 1, 5000, [5000, 1234]), (12, 1, 5, 700, [700, 129]),
                                               (2, 2, 3, 400, [400, 2])])
@pytest.mark.parametrize("softcap", [1e4, 1e6, 1e9])
def test_decode_with_caps_above_every_score(d, Hq, Hkv, Nq, Nk, lens, softcap):
    g = torch.Generator().manual_seed(Hq * 100 + Nq + d)
    q = (torch.randn(2, Hq, Nq, d, generator=g) * 3).to(torch.bfloat16)
    k, v = (torch.randn(2, Hkv, Nk, d, generator=g).to(torch.bfloat16) for _ in range(2))
    scale = 1 / math.sqrt(d)
    o, lse = fa.decode(q.cuda(), k.cuda(), v.cuda(), seqlens_k=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                       causal=True, softcap=softcap)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    o_r, lse_r, av, size = _decode_ref(q, k, v, lens, True, scale, softcap, None)
    delta = LARGE * size
    o, lse = _f64(o), _f64(lse)
    live = np.isfinite(lse_r)
    assert np.array_equal(np.isneginf(lse), ~live) and (o[~live] == 0).all()
    off = np.abs(lse[live] - lse_r[live]) - (delta[live] + 2.0 ** -20 * (1 + np.abs(lse_r[live])))
    assert (off <= 0).all(), float(off.max())
    # Up to 16 rows a K/V head (8 at d = 256) P is the sum of two bf16 numbers, 2^-16 off, and an
    # accumulator takes at most 2 * 5000 / 64 = 157 products, each 2^-22 of what has been added up:
    # 2^-14 with the sum of P; with more rows P is rounded to bf16, in the product and in its sum.
    bits = -14 if Hq // Hkv * Nq <= (8 if d == 256 else 16) else -6.9
    tol = 2.0 ** -8 * np.abs(o_r) + (2.0 ** bits + 2 * delta[..., None]) * av + 2.0 ** -30
    assert (np.abs(o - o_r) <= tol).all(), float((np.abs(o - o_r) / tol).max())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,Nq", [(8, 2, 1), (12, 1, 5)])
@pytest.mark.parametrize("softcap", [1e4, 1e6, 1e9])
def test_decode_kv4_with_caps_above_every_score(d, Hq, Hkv, Nq, softcap):
    # bounds of test_gpu_kv4.py, with |s| <= A in the place of the cap
    n, lens, scale = 700, [700, 401], 1 / math.sqrt(d)
    g = torch.Generator().manual_seed(Hq + d)
    q = (torch.randn(2, Hq, Nq, d, generator=g) * 3).to(torch.bfloat16)
    k, v = (torch.randn(2, Hkv, n, d, generator=g).to(torch.bfloat16) for _ in range(2))
    o, lse = fa.decode_kv4(q.cuda(), _cache_of(k, v, 704), softcap=softcap, causal=True,
                           seqlens_k=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    pk, pv = kv4_reference.quantise(_f64(k)), kv4_reference.quantise(_f64(v))
    big = np.repeat(np.abs(pk[2]) + 15 * pk[1], 32, -1)
    v64 = kv4_reference.values(*pv)
    o_r, lse_r, av, _ = kv4_reference.decode(_f64(q), kv4_reference.values(*pk), v64, lens, True, scale, softcap)
    A = scale * np.einsum("bhtc,bhc->bht", np.abs(_f64(q)), np.repeat(big.max(2), Hq // Hkv, 1))
    delta = LARGE * A + 2.0 ** -20
    tol = (2.0 ** -8 * np.abs(o_r) + (2.0 ** -10 + 2 * delta[..., None] + 2.0 ** -18) * av
           + 2.0 ** -24 * np.abs(v64).max())
    assert (np.abs(_f64(lse) - lse_r) <= delta + 2.0 ** -20 * (1 + np.abs(lse_r))).all(), \
        float(np.abs(_f64(lse) - lse_r).max())
    assert (np.abs(_f64(o) - o_r) <= tol).all(), float((np.abs(_f64(o) - o_r) / tol).max())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("softcap", [64.0, 100.0, 1e5, 1e7])
@pytest.mark.parametrize("causal,slopes", [(False, False), (True, False), (True, True)])
def test_small_scores_beside_rows_beyond_the_cap(d, softcap, causal, slopes):
    # every other query is so large that all its scores are at the cap: the rows between them, which
    # share their warps, must not lose what lies below the cap's own resolution
    B, Hq, N, scale = 1, 2, 260, 1 / math.sqrt(d)
    q, k, v, do = _draw(B, Hq, 1, N, d, seed=d + int(math.log2(softcap)), q_std=2.0)
    q[:, :, 1::2] *= 2.0 ** 30
    sl = _slopes(Hq) if slopes else None
    kw = dict(causal=causal, softcap=softcap)
    gpu = dict(kw, alibi_slopes=None if sl is None else sl.cuda())
    qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
    o, lse = fa.fwd(qd, kd, vd, **gpu)
    dq, dk, dv = fa.bwd(qd, kd, vd, o, lse, dod, **gpu)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    args = dict(kw, scale=scale, slopes=sl, key_range=None)
    q64, k64, v64, do64 = (t.double() for t in (q, k, v, do))
    o_r, lse_r, av = ref.forward(q64, k64, v64, **args)
    even = slice(0, N, 2)
    A = scale * (q64.abs() @ k64.abs().mT).amax(-1) + (0.0 if sl is None else float(sl.max()) * N)
    delta = (LARGE * A)[:, :, even]
    o_, lse_ = o.double().cpu(), lse.double().cpu()
    off = (lse_ - lse_r).abs()[:, :, even] - (delta + 6.25e-6 + 2.0 ** -20 * (1 + lse_r.abs()[:, :, even]))
    assert bool((off <= 0).all()), float(off.max())
    tol = 2.0 ** -8 * o_r.abs() + 2.0 ** -30
    tol = tol[:, :, even] + (2.0 ** -7 + 2.0 ** -12 + 2 * delta[..., None]) * av[:, :, even]
    assert bool(((o_ - o_r).abs()[:, :, even] <= tol).all())
    exact, sums, more = ref.backward(q64, k64, v64, o_, lse_, do64, **args)
    e, s, m = (t[0][:, :, even] for t in (exact, sums, more))
    tol = 2.0 ** -8 * e.abs() + (2.0 ** -8 + 2.0 ** -12 + 2 * delta[..., None]) * s + 2.0 ** -18 * m + 2.0 ** -30
    assert bool(((dq.double().cpu()[:, :, even] - e).abs() <= tol).all())
    assert all(bool(torch.isfinite(t).all()) for t in (dk, dv))


@pytest.mark.parametrize("d,N", [(128, 4193), (64, 1500), (256, 1500)])
@pytest.mark.parametrize("slopes", [False, True])
def test_large_cap_in_long_rows(d, N, slopes):
    # key blocks whole and in parts, and sizes that a smaller cap with slopes gives 128-query steps
    q, k, v, do = _draw(1, 1, 1, N, d, seed=d + N, q_std=2.0)
    check(q, k, v, do, causal=True, softcap=1e5, slopes=_slopes(1) if slopes else None)


LOWEST, HIGHEST = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
def test_range_bounds_at_the_ends_of_int32(d, causal):
    # the bounds count as clamped to 0 .. N: rows that name no key by the lowest or the highest
    # int32, beside rows that see keys and so bring in blocks beyond the first
    N = 520
    kinds = torch.tensor([(0, LOWEST), (HIGHEST, HIGHEST), (LOWEST, LOWEST), (LOWEST, HIGHEST), (LOWEST, 3), (500, HIGHEST),
                          (HIGHEST, LOWEST), (0, 519), (130, LOWEST + 1), (HIGHEST - 1, 400)], dtype=torch.int64)
    i = torch.arange(2 * N).view(2, N)
    r = kinds[(i * 7 + i // 11) % len(kinds)].to(torch.int32)
    q, k, v, do = _draw(2, 3, 1, N, d, seed=d + 17)
    out = check(q, k, v, do, causal=causal, key_range=r)
    none = (r[..., 1] <= 0) | (r[..., 0] >= N) | (r[..., 1] <= r[..., 0])
    assert bool((out[0].cpu().transpose(1, 2)[none] == 0).all()) and bool((out[2].cpu().transpose(1, 2)[none] == 0).all())


def check_near_zero(q, k, v, do, causal, softcap):
    """check, and in the gradients' bounds what a small cap makes of a score's error: the factor
    1 - tanh^2(x / cap) is taken at an x that is off by up to delta = 2^-17 A, which for |x| near
    delta or below may be anything between its values at |x| - delta and |x| + delta."""
    o, lse = check(q, k, v, do, causal=causal, softcap=softcap, backward=False)
    dev = [t.cuda() for t in (q, k, v)]
    got = fa.bwd(*dev, o, lse, do.cuda(), causal=causal, softcap=softcap)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    B, Hq, N, d = q.shape
    g, scale = Hq // k.shape[1], 1 / math.sqrt(d)
    args = dict(causal=causal, scale=scale, softcap=softcap, slopes=None, key_range=None)
    q64, k64, v64, do64, o64, lse64 = (t.double().cpu() for t in (q, k, v, do, o, lse))
    exact, sums, more = ref.backward(q64, k64, v64, o64, lse64, do64, **args)
    kk, vv = k64.repeat_interleave(g, 1), v64.repeat_interleave(g, 1)
    x = scale * (q64 @ kk.mT).abs()
    delta = 2.0 ** -17 * scale * (q64.abs() @ kk.abs().mT).amax(-1, keepdim=True)
    fac = lambda y: 1 - torch.tanh(y / softcap) ** 2
    off = torch.maximum(fac((x - delta).clamp(min=0)) - fac(x), fac(x) - fac(x + delta))
    p = torch.exp(ref.scores(q64, k64, causal, scale, softcap, None, None)[0] - lse64[..., None])
    w = p * scale * off * ((do64 @ vv.mT).abs() + (do64 * o64).sum(-1, keepdim=True).abs())
    heads = lambda t: t.view(B, -1, g, N, d).sum(2)
    extra = (w @ kk.abs(), heads(w.mT @ q64.abs()), torch.zeros_like(v64))
    for name, a, e, s, m, t in zip(("dQ", "dK", "dV"), got, exact, sums, more, extra):
        a = a.double().cpu()
        tol = (2.0 ** -8 * e.abs() + (2.0 ** -8 + 2.0 ** -12 + 2 * float(delta.max())) * s + 2.0 ** -18 * m
               + 2.0 ** -30 + t)
        assert bool(torch.isfinite(a).all()), name
        assert bool(((a - e).abs() <= tol).all()), (name, float(((a - e).abs() / tol).max()))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("softcap", [1e-9, 1e-6, 1e6])
def test_rows_of_zero_scores(d, causal, softcap):
    # whole warps of zero queries: all their scores are 0 at any cap, also one whose folded
    # polynomial does not exist in fp32
    q, k, v, do = _draw(1, 2, 1, 300, d, seed=d, q_std=2.0)
    q[:, 0] = 0
    q[:, 1, 64:256] = 0
    check_near_zero(q, k, v, do, causal, softcap)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("softcap", [1e-45, 1e-42, 1e-37, 1e-25, 1e25, 1e37, 3.4e38])
def test_caps_at_the_ends_of_fp32(d, softcap):
    # scores all but equal, or all but uncapped; zero rows among them
    N = 300
    q, k, v, do = _draw(1, 2, 1, N, d, seed=d, q_std=2.0)
    q[:, 0, 3:7] = 0
    q[:, 1, 128:192] = 0
    check_near_zero(q, k, v, do, True, softcap)
    for Nq in (1, 10):
        lens, scale = [N], 1 / math.sqrt(d)
        rows = q[:, :, :Nq].contiguous()
        o_r, lse_r, av, size = _decode_ref(rows, k, v, lens, True, scale, softcap, None)
        o, lse = fa.decode(rows.cuda(), k.cuda(), v.cuda(), causal=True, softcap=softcap)
        tol = 2.0 ** -8 * np.abs(o_r) + (2.0 ** -6.9 + 2 * LARGE * size[..., None]) * av + 2.0 ** -30
        assert (np.abs(_f64(o) - o_r) <= tol).all()
        assert (np.abs(_f64(lse) - lse_r) <= LARGE * size + 2.0 ** -20 * (1 + np.abs(lse_r))).all()
        pk, pv = kv4_reference.quantise(_f64(k)), kv4_reference.quantise(_f64(v))
        k64, v64 = kv4_reference.values(*pk), kv4_reference.values(*pv)
        o_r, lse_r, av, _ = kv4_reference.decode(_f64(rows), k64, v64, lens, True, scale, softcap)
        big = np.repeat(np.abs(pk[2]) + 15 * pk[1], 32, -1)
        delta = LARGE * scale * np.einsum("bhtc,bhc->bht", np.abs(_f64(rows)), np.repeat(big.max(2), 2, 1)) + 2.0 ** -20
        o, lse = fa.decode_kv4(rows.cuda(), _cache_of(k, v, 320), softcap=softcap, causal=True,
                               seqlens_k=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        tol = (2.0 ** -8 * np.abs(o_r) + (2.0 ** -10 + 2 * delta[..., None] + 2.0 ** -18) * av
               + 2.0 ** -24 * np.abs(v64).max())
        assert (np.abs(_f64(o) - o_r) <= tol).all()
        assert (np.abs(_f64(lse) - lse_r) <= delta + 2.0 ** -20 * (1 + np.abs(lse_r))).all()
    assert fa.fa_device_status(None) == fa.FA_OK


def test_status_reports_one_error_of_each_kind():
    # a wait that ran out and a position outside a cache: both are reported, one per call
    cache = fa.kv4_alloc(1, 1, 64, 64)
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    outside = torch.full((1,), 64, dtype=torch.int32, device="cuda")
    assert fa.fa_device_status(None) == fa.FA_OK
    fa.kv4_write(cache, x, x, start=outside)
    assert fa.load().fa_watchdog_selftest(1000, None) == fa.FA_OK
    got = [fa.fa_device_status(None) for _ in range(3)]
    assert sorted(got) == [fa.FA_OK, fa.FA_ERR_DEVICE_TIMEOUT, fa.FA_ERR_SEQLENS] and got[2] == fa.FA_OK, got
    # two of the same kind are one error
    for _ in range(2):
        fa.kv4_write(cache, x, x, start=outside)
    assert fa.fa_device_status(None) == fa.FA_ERR_SEQLENS
    assert fa.fa_device_status(None) == fa.FA_OK


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("splits", [1, 2, 3, 60, 148, 1024])
def test_decode_of_long_caches_in_few_and_many_pieces(d, splits):
    # pieces of dozens of blocks, which refill every stage of the ring many times, and heads that
    # dozens of pieces share; keys and values behind the last one are NaN.  P keeps 16 bits here:
    # bounds of test_decode_with_caps_above_every_score, the distance off by 2^-22 of its largest.
    B, Hq, Hkv, Nq, Nk, lens, scale = 3, 6, 2, 2, 9000, [8999, 17, 4352], 1 / math.sqrt(d)
    g = torch.Generator().manual_seed(d + splits)
    q = (torch.randn(B, Hq, Nq, d, generator=g) * 3).to(torch.bfloat16)
    k, v = (torch.randn(B, Hkv, Nk, d, generator=g).to(torch.bfloat16) for _ in range(2))
    for b in range(B):
        k[b, :, lens[b]:], v[b, :, lens[b]:] = float("nan"), float("nan")
    slopes = torch.tensor([2.0 ** -(8 + h) for h in range(Hq)])
    o, lse = fa.decode(q.cuda(), k.cuda(), v.cuda(), seqlens_k=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                       causal=True, softcap=20.0, alibi_slopes=slopes.cuda(), num_splits=splits)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    o_r, lse_r, av, size = _decode_ref(q, k, v, lens, True, scale, 20.0, slopes)
    delta = LARGE * size + 2.0 ** -22 * float(slopes.max()) * Nk
    tol = 2.0 ** -8 * np.abs(o_r) + (2.0 ** -14 + 2 * delta[..., None]) * av + 2.0 ** -30
    if splits < 60:  # a warp's accumulator takes 2 * 9000 / 64 products: 2^-22 of the running sum each
        tol += 2.0 ** -14 * av
    assert (np.abs(_f64(o) - o_r) <= tol).all(), float((np.abs(_f64(o) - o_r) / tol).max())
    assert (np.abs(_f64(lse) - lse_r) <= delta + 2.0 ** -20 * (1 + np.abs(lse_r))).all()
