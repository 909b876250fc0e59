"""Host-only checks of attention with changed scores: refusals before anything is launched, the
workspace size, the range helpers, and the tests' own 64-bit reference against torch autograd."""
import math

import pytest
import torch

import score_reference as ref
from exact_io_aware_83_b200 import fa

FAKE = 0x10000  # never dereferenced


def _fwd(**kw):
    a = dict(q=FAKE, lse=FAKE, o=FAKE, slopes=None, rng=None, B=1, Hq=2, Hkv=1, N=16, d=128, causal=0, cap=0.0, scale=0.1)
    a.update(kw)
    return fa.load().fa_fwd_score(a["q"], FAKE, FAKE, a["o"], a["lse"], a["slopes"], a["rng"], a["B"], a["Hq"],
                                  a["Hkv"], a["N"], a["d"], a["causal"], a["cap"], a["scale"], None)


def _bwd(**kw):
    a = dict(q=FAKE, lse=FAKE, o=FAKE, ws=FAKE, wsb=1 << 40, slopes=None, rng=None, B=1, Hq=2, Hkv=1, N=16, d=128,
             causal=0, cap=0.0, scale=0.1)
    a.update(kw)
    return fa.load().fa_bwd_score(a["q"], FAKE, FAKE, a["o"], a["lse"], FAKE, FAKE, FAKE, FAKE, a["ws"], a["wsb"],
                                  a["slopes"], a["rng"], a["B"], a["Hq"], a["Hkv"], a["N"], a["d"], a["causal"],
                                  a["cap"], a["scale"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), fa.FA_ERR_INVALID_ARG), (dict(lse=None), fa.FA_ERR_INVALID_ARG),
    (dict(N=0), fa.FA_ERR_INVALID_ARG), (dict(causal=2), fa.FA_ERR_INVALID_ARG),
    (dict(scale=0.0), fa.FA_ERR_INVALID_ARG), (dict(cap=-1.0), fa.FA_ERR_INVALID_ARG),
    (dict(cap=float("nan")), fa.FA_ERR_INVALID_ARG), (dict(cap=float("inf")), fa.FA_ERR_INVALID_ARG),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED), (dict(Hq=3, Hkv=2), fa.FA_ERR_GQA),
    (dict(o=FAKE + 8), fa.FA_ERR_ALIGN), (dict(slopes=FAKE + 2), fa.FA_ERR_ALIGN),
    (dict(rng=FAKE + 4), fa.FA_ERR_ALIGN),
])
def test_argument_errors(kw, code):
    assert _fwd(**kw) == code
    assert _bwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ws=None), fa.FA_ERR_WORKSPACE), (dict(wsb=100), fa.FA_ERR_WORKSPACE),
    (dict(ws=FAKE + 8), fa.FA_ERR_ALIGN),
    (dict(d=256, N=1 << 20, Hq=1), fa.FA_ERR_UNSUPPORTED),
    (dict(d=128, N=1 << 24, Hq=1), fa.FA_ERR_UNSUPPORTED),
])
def test_backward_argument_errors(kw, code):
    assert _bwd(**kw) == code


@pytest.mark.parametrize("cap,slopes,code", [(-1.0, None, fa.FA_ERR_INVALID_ARG), (0.0, FAKE + 1, fa.FA_ERR_ALIGN)])
def test_decode_argument_errors(cap, slopes, code):
    assert fa.load().fa_decode_score(FAKE, FAKE, FAKE, FAKE, FAKE, None, slopes, None, 0, 1, 2, 1, 1, 64, 128, 0, 1,
                                     cap, 0.1, None) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="valid-argument path needs no GPU")
def test_valid_arguments_without_a_device_report_cuda_error():
    kw = dict(cap=30.0, slopes=FAKE + 4, rng=FAKE + 8, causal=1)
    assert _fwd(**kw) == fa.FA_ERR_CUDA and _bwd(**kw) == fa.FA_ERR_CUDA
    assert fa.load().fa_decode_score(FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, None, 0, 1, 2, 1, 1, 64, 128, 0, 1,
                                     5.0, 0.1, None) == fa.FA_ERR_CUDA


def test_workspace_size():
    pad = lambda x: (x + 255) // 256 * 256
    # spans; with less than 148 units part counts, items, and fp32 dK and dV of every part
    for B, Hq, Hkv, N, d, parts in ((1, 2, 1, 100, 64, 8), (3, 4, 1, 5000, 128, 4), (2, 8, 8, 4096, 256, 0),
                                    (1, 8, 4, 2048, 256, 4), (1, 4, 4, 4736, 128, 0), (1, 3, 3, 6272, 128, 4)):
        blocks = B * ((N + 127) // 128)
        plan = pad(4 * blocks) + pad(16 * parts * blocks) + parts * Hkv * 128 * blocks * d * 8 if parts else 0
        assert fa.fa_bwd_score_workspace_bytes(B, Hq, Hkv, N, d) == \
            fa.fa_bwd_workspace_bytes(B, Hq, Hkv, N, d) + pad(8 * blocks) + pad(plan)
    assert fa.fa_bwd_score_workspace_bytes(1, 4, 3, 100, 64) == 0


def test_binding_refuses_combinations_and_cpu_tensors():
    q = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16)
    for kw in (dict(window=(4, 0)), dict(dropout_p=0.1), dict(block_mask=q)):
        win = fa._window(False, kw.get("window"))
        with pytest.raises(ValueError):
            fa._score_alone(win, kw.get("dropout_p", 0.0), kw.get("block_mask"))
    with pytest.raises(ValueError):
        fa.fwd(q, q, q, softcap=5.0)
    with pytest.raises(ValueError):
        fa._slopes(torch.zeros(4), 4, q.device)
    with pytest.raises(ValueError):
        fa._key_range(torch.zeros(1, 8, 2, dtype=torch.int32), 1, 8, q.device)


def test_range_helpers():
    r = fa.document_ranges(torch.tensor([[0, 3, 5, 5], [1, 2, 4, 7]], dtype=torch.int32), 8)
    assert r.dtype == torch.int32 and r.shape == (2, 8, 2)
    assert r[0].tolist() == [[0, 3]] * 3 + [[3, 5]] * 2 + [[0, 0]] * 3
    assert r[1].tolist() == [[0, 0], [1, 2], [2, 4], [2, 4], [4, 7], [4, 7], [4, 7], [0, 0]]
    p = fa.prefix_ranges(torch.tensor([3, 0, 9]), 6)
    assert p[..., 0].eq(0).all() and p[..., 1].tolist() == [[3, 3, 3, 4, 5, 6], [1, 2, 3, 4, 5, 6], [6] * 6]


@pytest.mark.parametrize("softcap,alibi,docs,causal", [(3.0, False, False, True), (0.0, True, True, False),
                                                       (2.0, True, True, True)])
def test_reference_gradients_are_autograds(softcap, alibi, docs, causal):
    g = torch.Generator().manual_seed(3)
    B, Hq, Hkv, N, d = 2, 4, 2, 19, 8
    q, k, v, do = (torch.randn(B, h, N, d, generator=g, dtype=torch.float64) for h in (Hq, Hkv, Hkv, Hq))
    kw = dict(causal=causal, scale=1 / math.sqrt(d), softcap=softcap,
              slopes=torch.tensor([0.5, 0.25, 0.1, 0.0]) if alibi else None,
              key_range=fa.document_ranges(torch.tensor([[0, 7, 19], [0, 2, 15]]), N) if docs else None)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    s, _ = ref.scores(leaves[0], leaves[1], causal, kw["scale"], softcap, kw["slopes"], kw["key_range"])
    live = torch.isfinite(s).any(-1, keepdim=True)
    p = torch.softmax(torch.where(live, s, torch.zeros_like(s)), -1) * live
    o = p @ leaves[2].repeat_interleave(Hq // Hkv, 1)
    o.backward(do)
    o_r, lse, _ = ref.forward(q, k, v, **kw)
    assert (o_r - o).abs().max() < 1e-12
    exact, _, _ = ref.backward(q, k, v, o_r, lse, do, **kw)
    for a, b in zip(exact, leaves):
        assert (a - b.grad).abs().max() < 1e-11
