"""The 4-bit key/value cache on the GPU: what kv4_write stores and kv4_read gives back, bit for
bit, and decode_kv4 against attention in 64 bits over the values that the cache stands for.

Bounds of decode_kv4, with u = 2^-11 (fp16 rounding): the scores are fp32 sums of at most 64
terms a group over 8 groups, each off by at most 2^-23 of what has been added up, which the
codes' bias of up to 15 s + |m| enlarges: delta = 2^-17 A + 2^-20, A the row's largest
scale sum_c |q_c| (|m| + 15 s) (2^-20 for exp2, tanh and the distance in fp32, times the score's
size where a cap or a distance is in play: 2^-21 |s|).  Each P V term carries the fp16 rounding
of p and of v, and 2 delta from p and its sum:
    |O - ref| <= 2^-8 |ref| + (2 u + 2 delta + 2^-18) (sum_j P_j |v_j|) + 2^-24 max|v|
(the last term: fp16 underflow of probabilities below 2^-14 of the row's running maximum).
    |LSE - ref| <= delta + 2^-20 (1 + |ref|).
"""
import math

import numpy as np
import pytest
import torch

import kv4_reference as ref
from exact_io_aware_83_b200 import fa

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.double().cpu().numpy()


def _bf16(x):
    return torch.tensor(np.asarray(x), dtype=torch.float32).to(torch.bfloat16)


def _values(kind, shape, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape)
    if kind == "channels":
        x[..., ::16] *= 8.0
    elif kind == "constant":
        x[:] = x[..., :1]
    elif kind == "tiny":
        x *= 2.0 ** rng.integers(-40, -12, shape)
    elif kind == "huge":
        x *= 2.0 ** rng.integers(8, 40, shape)
    elif kind == "ties":                       # min 0, max 15 / 4: borders at odd eighths
        x = rng.integers(0, 31, shape) / 8.0
        x[..., ::32], x[..., 1::32] = 0.0, 3.75
    elif kind == "offset":                     # a spread of one bf16 step around a large value
        x = 1000.0 + 4.0 * rng.integers(0, 3, shape)
    elif kind == "mixed":                      # magnitudes far apart within a group
        x *= 10.0 ** rng.integers(-30, 4, shape).astype(float)
    return _bf16(x)


def _fresh(B, Hkv, cap, d, fill=0xA5):
    cache = fa.kv4_alloc(B, Hkv, cap, d)
    for t in cache:
        t.view(torch.uint8).fill_(fill)
    return cache


def _expected(x, is_k):
    return ref.pack(*ref.quantise(_f64(x)), is_k)


def _same_bits(a, b):
    a, b = a.view(np.uint16), b.view(np.uint16)
    nan = lambda t: (t & 0x7FFF) > 0x7C00
    return np.array_equal(np.where(nan(a), 0x7FFF, a), np.where(nan(b), 0x7FFF, b))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["normal", "channels", "constant", "tiny", "huge", "ties", "offset", "mixed"])
def test_write_bits_and_read_back(d, kind):
    B, Hkv, n, cap = 2, 3, 37, 128
    k, v = _values(kind, (B, Hkv, n, d), 11 + d), _values(kind, (B, Hkv, n, d), 12 + d)
    start = torch.tensor([5, 91], dtype=torch.int32)
    cache = _fresh(B, Hkv, cap, d)
    fa.kv4_write(cache, k.cuda(), v.cuda(), start=start.cuda())
    kr, vr = fa.kv4_read(cache, n, start=start.cuda())
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    for x, back, codes, params, is_k in ((k, kr, cache.k_codes, cache.k_params, True),
                                         (v, vr, cache.v_codes, cache.v_params, False)):
        n_, s, m = ref.quantise(_f64(x))
        want_c, want_p = ref.pack(n_, s, m, is_k)
        codes, params = codes.cpu().numpy(), params.cpu().numpy()
        held = np.zeros((B, cap), dtype=bool)
        for b in range(B):
            at = slice(int(start[b]), int(start[b]) + n)
            held[b, at] = True
            assert _same_bits(params[b, :, at].copy(), want_p[b]), (kind, is_k)
            assert np.array_equal(codes[b, :, at], want_c[b]), (kind, is_k)
        for b in range(B):  # nothing else of the cache changed
            assert (codes[b][:, ~held[b]] == 0xA5).all()
            assert (np.ascontiguousarray(params[b][:, ~held[b]]).view(np.uint8) == 0xA5).all()
        assert torch.equal(back.cpu(), torch.from_numpy(ref.values(n_, s, m)).to(torch.bfloat16))
        # the code is the nearest one: half a step (s / 2), but for clamped values
        y = np.clip(_f64(x), -ref.CLAMP, ref.CLAMP)
        half = np.repeat(s / 2, 32, -1)
        assert (np.abs(ref.values(n_, s, m) - y) <= half).all()


@pytest.mark.parametrize("d", [64, 256])
def test_groups_with_nan_or_infinity_read_back_as_nan(d):
    x = _values("normal", (1, 1, 3, d), 5)
    x[0, 0, 0, 3], x[0, 0, 1, 40], x[0, 0, 2, d - 1] = float("nan"), float("inf"), float("-inf")
    cache = _fresh(1, 1, 64, d)
    fa.kv4_write(cache, x.cuda(), x.cuda())
    k, v = (t.float().cpu() for t in fa.kv4_read(cache, 3))
    bad = torch.zeros(3, d, dtype=torch.bool)
    bad[0, :32], bad[1, 32:64], bad[2, d - 32:] = True, True, True
    for t in (k, v):
        assert torch.equal(torch.isnan(t[0, 0]), bad)


def test_counts_and_positions_outside_the_cache():
    B, Hkv, n, cap, d = 5, 2, 9, 64, 64
    k, v = _values("normal", (B, Hkv, n, d), 1), _values("normal", (B, Hkv, n, d), 2)
    start, counts = [0, 60, -3, 2 ** 31 - 1, 7], [4, 9, 9, 2, 0]
    cache = _fresh(B, Hkv, cap, d)
    to = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    fa.kv4_write(cache, k.cuda(), v.cuda(), start=to(start), counts=to(counts))
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_ERR_SEQLENS
    want = np.full((B, Hkv, cap, d // 2), 0xA5, dtype=np.uint8)
    codes = _expected(v, False)[0]
    for b in range(B):
        for i in range(counts[b]):
            if 0 <= start[b] + i < cap:
                want[b, :, start[b] + i] = codes[b, :, i]
    assert np.array_equal(cache.v_codes.cpu().numpy(), want)
    # reading outside leaves those rows alone
    out = [torch.full((B, Hkv, n, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.kv4_read(cache, n, start=to(start), k=out[0], v=out[1])
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_ERR_SEQLENS
    assert (out[0][1, :, 4:] == 7).all() and (out[0][2, :, :3] == 7).all() and (out[0][3] == 7).all()
    assert fa.fa_device_status(None) == fa.FA_OK


def _cache_of(k, v, cap):
    """A cache that holds k, v [B, Hkv, n, d] from position 0 on, and NaN or junk behind."""
    B, Hkv, n, d = k.shape
    cache = _fresh(B, Hkv, cap, d, fill=0xFF)   # fp16 0xFFFF is a NaN
    fa.kv4_write(cache, k.cuda(), v.cuda())
    return cache


def check(q, k, v, lens, cap, causal=False, softcap=0.0, slopes=None, num_splits=None, scale=None):
    B, Hq, Nq, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    cache = _cache_of(k, v, cap)
    to = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
    sl = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda")
    out = torch.full((B * Hq * Nq * d + 256,), 3.0, dtype=torch.bfloat16, device="cuda")
    ls = torch.full((B * Hq * Nq + 128,), 3.0, dtype=torch.float32, device="cuda")
    o, lse = out[128:-128].view(B, Hq, Nq, d), ls[64:-64].view(B, Hq, Nq)
    fa.decode_kv4(q.cuda(), cache, seqlens_k=to(lens), causal=causal, scale=scale, softcap=softcap,
                  alibi_slopes=sl, num_splits=num_splits, out=o, lse=lse)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    assert (out[:128] == 3).all() and (out[-128:] == 3).all() and (ls[:64] == 3).all() and (ls[-64:] == 3).all()
    pk, pv = ref.quantise(_f64(k)), ref.quantise(_f64(v))
    k64, v64 = ref.values(*pk), ref.values(*pv)
    big = np.repeat(np.abs(pk[2]) + 15 * pk[1], 32, -1)
    o_r, lse_r, av, _ = ref.decode(_f64(q), k64, v64, lens, causal, scale, softcap,
                                   None if slopes is None else sl.double().cpu().numpy())
    g = Hq // k.shape[1]
    A = scale * np.einsum("bhtc,bhc->bht", np.abs(_f64(q)), np.repeat(big.max(2), g, 1))
    far = cap * max(slopes) if slopes is not None else 0.0
    delta = 2.0 ** -17 * A + 2.0 ** -20 + 2.0 ** -21 * (softcap + far)
    vmax = np.abs(v64).max()
    tol = 2.0 ** -8 * np.abs(o_r) + (2.0 ** -10 + 2 * delta[..., None] + 2.0 ** -18) * av + 2.0 ** -24 * vmax
    o64, lse64 = _f64(o), _f64(lse)
    empty = np.isneginf(lse_r)
    assert np.array_equal(np.isneginf(lse64), empty)
    assert (o64[empty] == 0).all()
    assert np.isfinite(o64).all()
    assert (np.abs(o64 - o_r) <= tol).all(), float((np.abs(o64 - o_r) / np.maximum(tol, 1e-30)).max())
    with np.errstate(invalid="ignore"):
        off = np.where(empty, 0.0, np.abs(lse64 - lse_r) - (delta + 2.0 ** -20 * (1 + np.abs(lse_r))))
    assert (off <= 0).all(), float(off.max())
    return o, lse


def _draw(B, Hq, Hkv, Nq, n, d, seed, q_std=1.0):
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((B, Hkv, n, d))
    k[..., ::16] *= 4.0
    return (_bf16(q_std * rng.standard_normal((B, Hq, Nq, d))), _bf16(k),
            _bf16(rng.standard_normal((B, Hkv, n, d))))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,cap", [(1, 64), (31, 64), (64, 64), (257, 320), (1000, 1024)])
def test_lengths(d, n, cap):
    q, k, v = _draw(2, 4, 2, 1, n, d, seed=n + d)
    check(q, k, v, [n, max(0, n // 2)], cap)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,Nq", [(1, 1, 1), (8, 1, 1), (12, 4, 3), (9, 1, 1), (32, 2, 1), (16, 1, 8), (5, 5, 7)])
def test_rows_per_head(d, Hq, Hkv, Nq):
    q, k, v = _draw(2, Hq, Hkv, Nq, 300, d, seed=Hq * 100 + Hkv * 10 + Nq + d)
    check(q, k, v, [300, 77], 320, causal=True)


@pytest.mark.parametrize("lens", [[0, 0], [0, 5], [1, 2], [200, 3]])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_without_keys(lens, causal):
    q, k, v = _draw(2, 4, 2, 5, 200, 128, seed=sum(lens))
    check(q, k, v, lens, 256, causal=causal)


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 16, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_splits(splits, d):
    # more splits than pieces of 64 tokens leave some without keys
    q, k, v = _draw(1, 6, 2, 2, 1500, d, seed=splits + d)
    check(q, k, v, [1500], 1536, num_splits=splits, causal=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("softcap,alibi", [(5.0, False), (50.0, False), (0.0, True), (20.0, True)])
def test_capped_and_biased_scores(d, softcap, alibi):
    q, k, v = _draw(2, 8, 2, 3, 700, d, seed=d + int(softcap), q_std=3.0)
    slopes = [2.0 ** (-h - 1) for h in range(8)] if alibi else None
    check(q, k, v, [700, 401], 704, causal=True, softcap=softcap, slopes=slopes)


def test_large_scores_move_the_maximum():
    # scores of several hundred: nearly one key per row, the running maximum rises many times
    q, k, v = _draw(1, 8, 2, 2, 2000, 128, seed=3, q_std=20.0)
    k = (k.float() * torch.linspace(0.1, 3.0, 2000).view(1, 1, -1, 1)).to(torch.bfloat16)
    check(q, k, v, [2000], 2048)
    check(q, k, v, [2000], 2048, num_splits=1)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 60])
def test_query_magnitudes(size):
    # the query's power-of-two scaling: tiny and huge rows, rows of zeros among them
    q, k, v = _draw(1, 4, 1, 2, 130, 64, seed=9)
    q = (q.float() * size).to(torch.bfloat16)
    q[0, 1] = 0
    check(q, k, v, [130], 192, scale=0.125 / size)


def test_nan_reaches_the_rows_that_see_it():
    q, k, v = _draw(1, 2, 1, 2, 100, 64, seed=4)
    k[0, 0, 99, 5] = float("nan")
    cache = _cache_of(k, v, 128)
    o, lse = fa.decode_kv4(q.cuda(), cache, seqlens_k=torch.tensor([100], dtype=torch.int32, device="cuda"),
                           causal=True)
    assert torch.isfinite(o[:, :, 0]).all() and torch.isnan(o[:, :, 1]).all() and torch.isnan(lse[:, :, 1]).all()


def test_long_cache_offsets_past_32_bits():
    # 2 x 16 heads x 2^20 tokens x 256 channels: 4 GB of codes a tensor, so the last head's
    # tokens, which decide the result, lie past 2^32 bytes minus 128 MB
    B, Hkv, cap, d = 2, 16, 1 << 20, 256
    cache = fa.kv4_alloc(B, Hkv, cap, d)
    for t in cache:
        t.zero_()
    q, k, v = _draw(B, Hkv, Hkv, 1, 64, d, seed=8)
    start = torch.full((B,), cap - 64, dtype=torch.int32, device="cuda")
    fa.kv4_write(cache, k.cuda(), v.cuda(), start=start)
    kr, vr = fa.kv4_read(cache, 64, start=start)
    pk, pv = ref.quantise(_f64(k)), ref.quantise(_f64(v))
    assert torch.equal(kr.cpu(), torch.from_numpy(ref.values(*pk)).to(torch.bfloat16))
    o, lse = fa.decode_kv4(q.cuda(), cache)
    # the other cap - 64 keys are zero: score 0, value 0
    s = np.einsum("bhtc,bhjc->bhtj", _f64(q), ref.values(*pk)) / 16.0
    z = np.exp(s).sum(-1) + cap - 64
    want = np.einsum("bhtj,bhjc->bhtc", np.exp(s), ref.values(*pv)) / z[..., None]
    assert np.abs(_f64(lse) - np.log(z)).max() <= 1e-4
    av = np.einsum("bhtj,bhjc->bhtc", np.exp(s), np.abs(ref.values(*pv))) / z[..., None]
    assert (np.abs(_f64(o) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -8 * av + 2.0 ** -24).all()


def test_same_call_twice_and_on_another_stream_gives_the_same_bits():
    q, k, v = _draw(3, 8, 2, 1, 900, 128, seed=6)
    cache = _cache_of(k, v, 960)
    lens = torch.tensor([900, 13, 500], dtype=torch.int32, device="cuda")
    qd = q.cuda()
    first = fa.decode_kv4(qd, cache, seqlens_k=lens, softcap=30.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = fa.decode_kv4(qd, cache, seqlens_k=lens, softcap=30.0)
    side.synchronize()
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])


def test_decode_loop_captured_in_a_graph():
    # a serving step - write the new token, attend to the cache - captured once and replayed with
    # growing lengths held in device memory, against the same steps run one by one
    B, Hq, Hkv, d, cap, steps, n0 = 3, 8, 2, 128, 256, 5, [100, 63, 0]
    q, k, v = _draw(B, Hq, Hkv, 1, 120, d, seed=21)
    new = [_draw(B, Hq, Hkv, 1, 1, d, seed=30 + i) for i in range(steps)]

    def begin():
        cache = _fresh(B, Hkv, cap, d, fill=0xFF)
        counts = torch.tensor(n0, dtype=torch.int32, device="cuda")
        fa.kv4_write(cache, k.cuda(), v.cuda(), counts=counts)
        return cache, torch.tensor(n0, dtype=torch.int32, device="cuda")

    cache, pos = begin()
    want = []
    for qn, kn, vn in new:
        fa.kv4_write(cache, kn.cuda(), vn.cuda(), start=pos)
        pos = pos + 1
        want.append(fa.decode_kv4(qn.cuda(), cache, seqlens_k=pos, causal=True, softcap=20.0))
    torch.cuda.synchronize()

    cache, pos = begin()
    lens = pos + 1
    qs, ks, vs = (t.cuda() for t in new[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.kv4_write(cache, ks, vs, start=pos)
        o, lse = fa.decode_kv4(qs, cache, seqlens_k=lens, causal=True, softcap=20.0)
    for i, (qn, kn, vn) in enumerate(new):
        qs.copy_(qn)
        ks.copy_(kn)
        vs.copy_(vn)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]), i
        pos += 1
        lens += 1
    assert fa.fa_device_status(None) == fa.FA_OK
