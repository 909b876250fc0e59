"""Attention with changed scores (softcap, alibi_slopes, key_range) on the GPU: forward, backward
and decode against 64-bit references.

Bounds.  The scores are fp32 sums over d products; tcgen05 may truncate, so each of the d
additions is taken at 2^-23 of the running magnitude, bounded by A_i = scale max_j sum_c |q_c k_c|:
delta = 2^-23 * 64 * A (random-walk allowance: 64 of the at most 256 additions all one way)
+ 2^-20 |s| (tanh polynomial 3.1e-7, exp2 and bias arithmetic) with |s| <= S, the largest finite
|s| of the case.  P is rounded to bf16 (2^-8) for the product with V, the polynomial exp2 adds
7.5e-5, and O is normalised by the sum of the rounded probabilities to within the same 2^-8 of
what the largest one does not carry:
    |O - ref| <= 2^-8 |ref| + (2 * 2^-8 + 2^-12 + 2 delta) sum_j P |v_j| + 2^-30
    |LSE - ref| <= delta + 1e-4 / 16 + 2^-20 (1 + |ref|).
Gradients: P and dS are rounded to bf16 (2^-8 each, dS also carries P's delta and 2^-20 of the
unsubtracted dP and Delta), results to bf16:
    |dX - ref| <= 2^-8 |ref| + (2^-8 + 2^-12 + 2 delta) sum |dS| |x| + 2^-18 sum (|dP| + |Delta|) P |x| + 2^-30.
"""
import math

import numpy as np
import pytest
import torch

import score_reference as ref
from exact_io_aware_83_b200 import fa

pytestmark = pytest.mark.gpu


def _draw(B, Hq, Hkv, N, d, seed, q_std=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda h, f=1.0: (torch.randn(B, h, N, d, generator=g) * f).to(torch.bfloat16)
    return r(Hq, q_std), r(Hkv), r(Hkv), r(Hq)


def _slopes(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)])


def _guarded(shape, dtype):
    n = math.prod(shape)
    buf = torch.full((n + 256,), 3.0, dtype=dtype, device="cuda")
    return buf, buf[128:128 + n].view(shape)


def _intact(*bufs):
    return all(bool((b[:128] == 3).all()) and bool((b[-128:] == 3).all()) for b in bufs)


def _delta(q, k, scale, kw):
    g = q.shape[1] // k.shape[1]
    A = scale * (q.double().abs() @ k.double().abs().repeat_interleave(g, 1).mT).amax(-1)
    s, _ = ref.scores(q.double(), k.double(), kw["causal"], scale, kw["softcap"], kw["slopes"], kw["key_range"])
    S = float(s[torch.isfinite(s)].abs().max()) if bool(torch.isfinite(s).any()) else 0.0
    return 2.0 ** -17 * A + 2.0 ** -20 * S


def check(q, k, v, do, causal=False, scale=None, softcap=0.0, slopes=None, key_range=None, backward=True):
    B, Hq, N, d = q.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    kw = dict(causal=causal, softcap=softcap, slopes=slopes, key_range=key_range)
    gpu = dict(causal=causal, scale=scale, softcap=softcap,
               alibi_slopes=None if slopes is None else slopes.cuda(),
               key_range=None if key_range is None else key_range.cuda())
    ob, o = _guarded(q.shape, torch.bfloat16)
    lb, lse = _guarded(q.shape[:3], torch.float32)
    qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
    fa.fwd(qd, kd, vd, out=o, lse=lse, **gpu)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    assert _intact(ob, lb), "write outside O or LSE"
    q64, k64, v64, do64 = (t.double() for t in (q, k, v, do))
    o_r, lse_r, av = ref.forward(q64, k64, v64, scale=scale, **kw)
    delta = _delta(q, k, scale, kw)
    empty = torch.isneginf(lse_r)
    o_, lse_ = o.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isneginf(lse_), empty)
    assert bool((o_[empty] == 0).all()) and bool(torch.isfinite(o_).all())
    tol = 2.0 ** -8 * o_r.abs() + (2.0 ** -7 + 2.0 ** -12 + 2 * delta[..., None]) * av + 2.0 ** -30
    assert bool(((o_ - o_r).abs() <= tol).all()), float(((o_ - o_r).abs() / tol).max())
    lerr = torch.where(empty, 0.0, (lse_ - lse_r).abs() - (delta + 6.25e-6 + 2.0 ** -20 * (1 + lse_r.abs())))
    assert bool((lerr <= 0).all()), float(lerr.max())
    if not backward:
        return o, lse
    bufs, outs = zip(*(_guarded(t.shape, torch.bfloat16) for t in (q, k, v)))
    ws = torch.full((fa.fa_bwd_score_workspace_bytes(B, Hq, k.shape[1], N, d),), 0x7F, dtype=torch.uint8, device="cuda")
    fa.bwd(qd, kd, vd, o, lse, dod, workspace=ws, dq=outs[0], dk=outs[1], dv=outs[2], **gpu)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    assert _intact(*bufs), "write outside a gradient"
    exact, sums, more = ref.backward(q64, k64, v64, o_, lse_, do64, scale=scale, **kw)
    dmax = float(delta.max())
    for name, x, e, s, m in zip(("dQ", "dK", "dV"), outs, exact, sums, more):
        x = x.double().cpu()
        assert bool(torch.isfinite(x).all()), name
        tol = 2.0 ** -8 * e.abs() + (2.0 ** -8 + 2.0 ** -12 + 2 * dmax) * s + 2.0 ** -18 * m + 2.0 ** -30
        assert bool(((x - e).abs() <= tol).all()), (name, float(((x - e).abs() / tol).max()))
    return (o, lse) + outs


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 300])
@pytest.mark.parametrize("causal", [False, True])
def test_capped(d, N, causal):
    q, k, v, do = _draw(2, 2, 1, N, d, seed=N + d, q_std=2.0)
    check(q, k, v, do, causal=causal, softcap=20.0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("softcap,q_std", [(50.0, 1.0), (5.0, 4.0), (1.0, 8.0), (0.01, 1.0), (1e6, 1.0)])
def test_cap_sizes(d, softcap, q_std):
    # from caps that leave the scores alone to caps that all scores exceed, so that both forms of
    # the tanh and blocks that mix them are taken
    q, k, v, do = _draw(1, 3, 3, 260, d, seed=int(softcap * 100) + d, q_std=q_std)
    q[:, 0] = (q[:, 0].float() * 0.02).to(torch.bfloat16)
    check(q, k, v, do, causal=True, softcap=softcap)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_distance_bias(d, causal, softcap):
    q, k, v, do = _draw(1, 4, 2, 400, d, seed=d, q_std=2.0)
    check(q, k, v, do, causal=causal, softcap=softcap, slopes=_slopes(4))


def _doc_range(B, N, cuts):
    cu = torch.tensor([list(c) for c in cuts], dtype=torch.int32)
    return fa.document_ranges(cu, N)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
def test_documents_and_padding(d, causal):
    N = 517
    r = _doc_range(2, N, [(0, 3, 130, 131, 400, 500), (7, 256, 256, 384, 517, 517)])
    q, k, v, do = _draw(2, 4, 2, N, d, seed=d + 1)
    check(q, k, v, do, causal=causal, key_range=r, softcap=25.0, slopes=_slopes(4))
    check(q, k, v, do, causal=causal, key_range=r)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefixes(d):
    N = 390
    q, k, v, do = _draw(3, 2, 2, N, d, seed=d + 2)
    check(q, k, v, do, key_range=fa.prefix_ranges(torch.tensor([0, 200, 390]), N), slopes=_slopes(2))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [False, True])
def test_arbitrary_ranges(d, causal):
    # ranges that jump from row to row, with gaps between neighbours, bounds outside 0 .. N, and
    # rows, tiles and whole batch entries that see nothing
    B, N = 3, 700
    g = torch.Generator().manual_seed(d)
    lo = torch.randint(-50, N, (B, N), generator=g)
    hi = lo + torch.randint(-20, 260, (B, N), generator=g)
    lo[0, 128:256], hi[0, 128:256] = 5, 5
    lo[0, 256:384], hi[0, 256:384] = 600, 10 ** 9
    lo[1], hi[1] = N, 0
    lo[2, :300], hi[2, :300] = -(10 ** 9), 1
    r = torch.stack((lo, hi), -1).to(torch.int32)
    q, k, v, do = _draw(B, 3, 1, N, d, seed=d + 3)
    out = check(q, k, v, do, causal=causal, key_range=r, slopes=_slopes(3))
    assert bool((out[2][1] == 0).all()) and bool((out[3][1] == 0).all()) and bool((out[4][1] == 0).all())


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (6, 2), (5, 5), (7, 1), (16, 1)])
def test_head_groups(Hq, Hkv):
    N = 333
    q, k, v, do = _draw(2, Hq, Hkv, N, 64, seed=Hq * 10 + Hkv)
    r = _doc_range(2, N, [(0, 100, 333), (0, 333, 333)])
    check(q, k, v, do, causal=True, softcap=15.0, slopes=_slopes(Hq), key_range=r)


def test_unchanged_scores_agree_with_the_dense_call():
    # a range of everything and a cap beyond every score: the dense call's result to rounding,
    # and a window as ranges the windowed call's
    N, d = 640, 128
    q, k, v, do = (t.cuda() for t in _draw(1, 4, 2, N, d, seed=5))
    i = torch.arange(N, device="cuda")
    full = torch.stack((torch.zeros_like(i), torch.full_like(i, N)), -1).to(torch.int32)[None].contiguous()
    win = torch.stack((i - 100, i + 31), -1).to(torch.int32)[None].contiguous()
    for kw, other in ((dict(key_range=full, causal=True), dict(causal=True)),
                      (dict(softcap=1e9), dict()), (dict(key_range=win), dict(window=(100, 30)))):
        o1, l1 = fa.fwd(q, k, v, **kw)
        o2, l2 = fa.fwd(q, k, v, **other)
        assert (o1.float() - o2.float()).abs().max() <= 2.0 ** -8 * 4
        assert (l1 - l2).abs().max() <= 1e-5
        for a, b in zip(fa.bwd(q, k, v, o1, l1, do, **kw), fa.bwd(q, k, v, o1, l1, do, **other)):
            assert (a.float() - b.float()).norm() <= 2.0 ** -7 * b.float().norm()


def test_gradients_against_differences():
    # <O, dO> through the 64-bit forward moved by +-h along random directions, against the GPU's
    # gradients: h^2 terms and 64-bit rounding stay below 1e-6, the gradients carry bf16 rounding
    # (relative 2^-8 an element, averaged over 4000 elements a direction)
    N, d = 96, 64
    q, k, v, do = _draw(1, 2, 1, N, d, seed=77, q_std=2.0)
    r = _doc_range(1, N, [(0, 40, 90)])
    kw = dict(causal=False, softcap=6.0, slopes=_slopes(2), key_range=r)
    out = check(q, k, v, do, **kw)
    grads = [t.double().cpu() for t in out[2:]]
    g = torch.Generator().manual_seed(1)
    base = [t.double() for t in (q, k, v)]
    for n in range(3):
        u = torch.randn(base[n].shape, generator=g, dtype=torch.float64)
        f = []
        for h in (1e-4, -1e-4):
            x = list(base)
            x[n] = x[n] + h * u
            f.append(float((ref.forward(*x, scale=1 / 8, **kw)[0] * do.double()).sum()))
        num = (f[0] - f[1]) / 2e-4
        ana = float((grads[n] * u).sum())
        bound = 2.0 ** -7 * float((grads[n] * u).norm()) * 4 + 2.0 ** -7 * float(grads[n].norm())
        assert abs(num - ana) <= bound, (n, num, ana, bound)


def test_large_scores_and_late_rows():
    q, k, v, do = _draw(1, 2, 2, 640, 128, seed=78, q_std=6.0)
    check(q, k, v, do, causal=True, softcap=100.0, scale=0.35)
    check(q, k, v, do, scale=0.35, slopes=torch.tensor([0.0, 3.0]))


def test_long_row_against_a_slice():
    # 8192 rows of documents, 16 heads: one head against the reference, row block by row block
    B, H, N, d = 1, 16, 8192, 128
    q, k, v, do = _draw(B, H, H, N, d, seed=8)
    r = _doc_range(1, N, [(0, 100, 1000, 1001, 4096, 8000)])
    kw = dict(causal=True, softcap=50.0, alibi_slopes=_slopes(H).cuda(), key_range=r.cuda())
    qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
    o, lse = fa.fwd(qd, kd, vd, **kw)
    dq, dk, dv = fa.bwd(qd, kd, vd, o, lse, dod, **kw)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    assert bool((o[:, :, 8000:] == 0).all()) and bool((dq[:, :, 8000:] == 0).all()) and bool((dk[:, :, 8000:] == 0).all())
    h = 11
    sl = slice(1001, 4096)
    one = [t[:, h:h + 1, sl].contiguous() for t in (q, k, v, do)]
    n = 4096 - 1001
    q64, k64, v64, do64 = (t.double() for t in one)
    args = dict(causal=True, scale=1 / math.sqrt(d), softcap=50.0, slopes=_slopes(H)[h:h + 1], key_range=None)
    o_r, lse_r, av = ref.forward(q64, k64, v64, **args)
    got = o[:, h:h + 1, sl].double().cpu()
    assert bool(((got - o_r).abs() <= 2.0 ** -8 * o_r.abs() + 2.0 ** -6.9 * av + 2.0 ** -30).all())
    assert (lse[:, h:h + 1, sl].double().cpu() - lse_r).abs().max() <= 1e-4
    exact, sums, more = ref.backward(q64, k64, v64, got, lse[:, h:h + 1, sl].double().cpu(), do64, **args)
    for x, e, s, m in zip((dq, dk, dv), exact, sums, more):
        x = x[:, h:h + 1, sl].double().cpu()
        assert bool(((x - e).abs() <= 2.0 ** -8 * e.abs() + 2.0 ** -7.5 * s + 2.0 ** -18 * m + 2.0 ** -30).all())


@pytest.mark.parametrize("kw", [dict(causal=True, softcap=50.0), dict(causal=False, softcap=3.0),
                                dict(causal=True, alibi=True), dict(causal=True, softcap=8.0, alibi=True)])
def test_long_rows_without_ranges(kw):
    # from 4096 rows on, d = 128 without ranges takes 128-query steps; an odd length, grouped
    # heads, small and large |score| / cap: one head and one group against the reference
    N, d, scale = 4193, 128, 1 / math.sqrt(128)
    q, k, v, do = _draw(1, 3, 1, N, d, seed=41, q_std=2.0)
    slopes = _slopes(3) if kw.get("alibi") else None
    gpu = dict(causal=kw["causal"], softcap=kw.get("softcap", 0.0), alibi_slopes=None if slopes is None else slopes.cuda())
    qd, kd, vd, dod = (t.cuda() for t in (q, k, v, do))
    o, lse = fa.fwd(qd, kd, vd, **gpu)
    bufs, outs = zip(*(_guarded(t.shape, torch.bfloat16) for t in (q, k, v)))
    fa.bwd(qd, kd, vd, o, lse, dod, dq=outs[0], dk=outs[1], dv=outs[2], **gpu)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK and _intact(*bufs)
    args = dict(causal=kw["causal"], scale=scale, softcap=kw.get("softcap", 0.0), key_range=None)
    want = [torch.zeros(t.shape, dtype=torch.float64) for t in (q, k, v)]
    sums = [torch.zeros(t.shape, dtype=torch.float64) for t in (q, k, v)]
    more = [torch.zeros(t.shape, dtype=torch.float64) for t in (q, k, v)]
    for h in range(3):
        hs = slice(h, h + 1)
        one = [t.double() for t in (q[:, hs], k, v)]
        sl = None if slopes is None else slopes[hs]
        o_r, lse_r, av = ref.forward(*one, slopes=sl, **args)
        got, l = o[:, hs].double().cpu(), lse[:, hs].double().cpu()
        assert bool(((got - o_r).abs() <= 2.0 ** -8 * o_r.abs() + 2.0 ** -6.9 * av + 2.0 ** -30).all())
        assert (l - lse_r).abs().max() <= 1e-4
        for acc, part in zip((want, sums, more), ref.backward(*one, got, l, do[:, hs].double(), slopes=sl, **args)):
            acc[0][:, hs] = part[0]
            acc[1] += part[1]
            acc[2] += part[2]
    for x, e, s, m in zip(outs, want, sums, more):
        x = x.double().cpu()
        assert bool(((x - e).abs() <= 2.0 ** -8 * e.abs() + 2.0 ** -7.5 * s + 2.0 ** -18 * m + 2.0 ** -30).all())


def test_captured_training_step():
    # forward and backward captured together and replayed on new inputs, against eager calls
    B, Hq, Hkv, N, d = 1, 4, 2, 300, 128
    r = _doc_range(B, N, [(0, 120, 290)]).cuda()
    kw = dict(causal=True, softcap=20.0, alibi_slopes=_slopes(Hq).cuda(), key_range=r)
    one = [t.cuda() for t in _draw(B, Hq, Hkv, N, d, seed=1)]
    two = [t.cuda() for t in _draw(B, Hq, Hkv, N, d, seed=2)]
    want_o, want_l = fa.fwd(*two[:3], **kw)
    want = fa.bwd(*two[:3], want_o, want_l, two[3], **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.fwd(*one[:3], **kw)
        grads = fa.bwd(*one[:3], o, lse, one[3], **kw)
    for a, b in zip(one, two):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want_o) and torch.equal(lse, want_l)
    assert torch.equal(grads[1], want[1]) and torch.equal(grads[2], want[2])
    # dQ's fp32 additions land in no fixed order: 2^-24 a term, then one bf16 rounding
    assert (grads[0].float() - want[0].float()).abs().max() <= 2.0 ** -7 * want[0].float().abs().max()


# ---------------------------------------------------------------------------------------- decode

def _decode_ref(q, k, v, lens, causal, scale, softcap, slopes):
    import kv4_reference
    return kv4_reference.decode(q.double().numpy(), k.double().numpy(), v.double().numpy(), lens, causal, scale,
                                softcap, None if slopes is None else slopes.double().numpy())


def _mixed_ranges(B, N, seed):
    # rows of every kind: none, one key, a stretch, all keys
    g = torch.Generator().manual_seed(seed)
    lo = torch.randint(0, N, (B, N), generator=g)
    hi = lo + torch.randint(0, N, (B, N), generator=g)
    kind = torch.randint(0, 4, (B, N), generator=g)
    lo, hi = torch.where(kind == 3, 0, lo), torch.where(kind == 3, N, torch.where(kind == 2, lo + 1, hi))
    return torch.stack((lo, torch.where(kind == 0, lo, hi)), -1).to(torch.int32)


@pytest.mark.parametrize("B,Hq,Hkv,N,d", [(2, 40, 40, 257, 64), (2, 40, 40, 257, 128), (2, 20, 20, 257, 256),
                                          (49, 2, 1, 300, 64), (1, 6, 2, 1500, 128), (1, 8, 1, 1300, 64),
                                          (1, 3, 1, 1100, 256)])
@pytest.mark.parametrize("causal", [False, True])
def test_many_and_few_key_blocks(B, Hq, Hkv, N, d, causal):
    # 240 units: whole key blocks; 147, 24, 11, 18: key blocks in parts
    q, k, v, do = _draw(B, Hq, Hkv, N, d, seed=N + d + B)
    check(q, k, v, do, causal=causal, softcap=30.0, slopes=_slopes(Hq), key_range=_mixed_ranges(B, N, N + Hq))


def test_many_batch_entries():
    # more entries than a grid's second dimension holds, one row each, every third without its key
    B = 70000
    q, k, v, do = _draw(B, 1, 1, 1, 64, seed=8)
    r = torch.zeros(B, 1, 2, dtype=torch.int32)
    r[:, 0, 1] = (torch.arange(B) % 3 != 0).int()
    check(q, k, v, do, softcap=10.0, key_range=r)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("softcap,q_std", [(50.0, 1.0), (8.0, 2.0), (1.0, 4.0)])
def test_capped_ranges(d, softcap, q_std):
    # hidden keys and rows without keys in blocks of small, larger and saturated scores
    q, k, v, do = _draw(2, 4, 2, 600, d, seed=d + int(softcap), q_std=q_std)
    check(q, k, v, do, softcap=softcap, key_range=_mixed_ranges(2, 600, d))


@pytest.mark.parametrize("d", [64, 256])
def test_parts_add_up_in_order(d):
    # the same gradient of K and V every time; one key block with all the queries, the rest with few
    B, Hq, Hkv, N = 1, 8, 1, 1200
    q, k, v, do = (t.cuda() for t in _draw(B, Hq, Hkv, N, d, seed=5))
    i = torch.arange(N, dtype=torch.int32, device="cuda")
    rg = torch.stack((torch.zeros_like(i), torch.where(i < 1100, 100, N)), -1)[None].int().contiguous()
    kw = dict(key_range=rg, alibi_slopes=_slopes(Hq).cuda())
    o, lse = fa.fwd(q, k, v, **kw)
    first = fa.bwd(q, k, v, o, lse, do, **kw)
    for _ in range(3):
        again = fa.bwd(q, k, v, o, lse, do, **kw)
        assert torch.equal(again[1], first[1]) and torch.equal(again[2], first[2])
    check(*(t.cpu() for t in (q, k, v, do)), slopes=_slopes(Hq), key_range=rg.cpu())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,Nq,Nk,lens,splits", [
    (4, 2, 1, 333, [333, 100], None), (8, 1, 1, 1000, [1000, 1], 3), (6, 2, 5, 700, [3, 700], 2),
    (12, 1, 5, 300, [300, 129], 1), (2, 2, 1, 64, [0, 64], 1)])
@pytest.mark.parametrize("softcap,alibi", [(8.0, False), (0.0, True), (30.0, True)])
def test_decode(d, Hq, Hkv, Nq, Nk, lens, splits, softcap, alibi):
    if Hq // Hkv * Nq > (64 if d == 256 else 128):
        pytest.skip("beyond decode's row limit")
    g = torch.Generator().manual_seed(Hq * 100 + Nq + d)
    q = (torch.randn(2, Hq, Nq, d, generator=g) * 3).to(torch.bfloat16)
    k, v = (torch.randn(2, Hkv, Nk, d, generator=g).to(torch.bfloat16) for _ in range(2))
    slopes = _slopes(Hq) if alibi else None
    scale = 1 / math.sqrt(d)
    kd, vd = k.cuda(), v.cuda()
    for b in range(2):  # what lies behind the last key must not matter
        kd[b, :, lens[b]:] = float("nan")
        vd[b, :, lens[b]:] = float("nan")
    o, lse = fa.decode(q.cuda(), kd, vd, seqlens_k=torch.tensor(lens, dtype=torch.int32, device="cuda"), causal=True,
                       softcap=softcap, alibi_slopes=None if slopes is None else slopes.cuda(), num_splits=splits)
    torch.cuda.synchronize()
    assert fa.fa_device_status(None) == fa.FA_OK
    o_r, lse_r, av, size = _decode_ref(q, k, v, lens, True, scale, softcap, slopes)
    delta = 2.0 ** -17 * size + 2.0 ** -20 * (softcap + (max(lens) * float(slopes.max()) if alibi else 0.0) + 1)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(lse_r)
    assert np.array_equal(np.isneginf(lse), empty) and (o[empty] == 0).all() and np.isfinite(o).all()
    # P is rounded to bf16 and O normalised by the sum of the rounded values
    tol = 2.0 ** -8 * np.abs(o_r) + (2.0 ** -7 + 2.0 ** -12 + 2 * delta[..., None]) * av + 2.0 ** -30
    assert (np.abs(o - o_r) <= tol).all(), float((np.abs(o - o_r) / tol).max())
    with np.errstate(invalid="ignore"):
        off = np.where(empty, 0.0, np.abs(lse - lse_r) - (delta + 2.0 ** -20 * (1 + np.abs(lse_r))))
    assert (off <= 0).all(), float(off.max())


def test_capped_model_trained_then_served():
    # the operators as a user has them together: a prompt through fwd, its keys and values into
    # a bf16 and a 4-bit cache, then new tokens through decode and decode_kv4; the bf16 decode
    # must continue the forward's rows, the 4-bit one agree with decode over the values read back
    B, Hq, Hkv, N, n0, d = 2, 8, 2, 200, 180, 128
    q, k, v, _ = (t.cuda() for t in _draw(B, Hq, Hkv, N, d, seed=31, q_std=2.0))
    kw = dict(causal=True, softcap=20.0, alibi_slopes=_slopes(Hq).cuda())
    o, lse = fa.fwd(q, k, v, **kw)
    lens = torch.full((B,), N, dtype=torch.int32, device="cuda")
    last = q[:, :, n0:n0 + 12].contiguous()
    part = torch.full((B,), n0 + 12, dtype=torch.int32, device="cuda")
    o1, l1 = fa.decode(last, k, v, seqlens_k=part, **kw)
    assert (o1.float() - o[:, :, n0:n0 + 12].float()).abs().max() <= 2.0 ** -7 * 4
    assert (l1 - lse[:, :, n0:n0 + 12]).abs().max() <= 1e-4
    cache = fa.kv4_alloc(B, Hkv, 256, d)
    fa.kv4_write(cache, k[:, :, :n0].contiguous(), v[:, :, :n0].contiguous())
    fa.kv4_write(cache, k[:, :, n0:].contiguous(), v[:, :, n0:].contiguous(),
                 start=torch.full((B,), n0, dtype=torch.int32, device="cuda"))
    kr, vr = fa.kv4_read(cache, N)
    tail = q[:, :, N - 3:].contiguous()
    o2, l2 = fa.decode_kv4(tail, cache, seqlens_k=lens, **kw)
    o3, l3 = fa.decode(tail, kr, vr, seqlens_k=lens, **kw)
    # kv4_read rounds the values to bf16: 2^-8 of each key and value
    assert (l2 - l3).abs().max() <= 0.1 and (o2.float() - o3.float()).abs().max() <= 0.1
    assert fa.fa_device_status(None) == fa.FA_OK
