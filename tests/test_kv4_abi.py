"""Host-only checks of the 4-bit cache's entry points: refusals before anything is launched, the
split and workspace sizes, and the tests' own 64-bit reference of the format."""
import numpy as np
import pytest
import torch

import kv4_reference as ref
from exact_io_aware_83_b200 import fa

FAKE = 0x10000  # never dereferenced


def _copy(which, **kw):
    a = dict(k=FAKE, v=FAKE, kc=FAKE, kp=FAKE, vc=FAKE, vp=FAKE, start=None, counts=None, B=1, Hkv=2, n=3, cap=128,
             d=128)
    a.update(kw)
    lib = fa.load()
    if which == "write":
        return lib.fa_kv4_write(a["k"], a["v"], a["kc"], a["kp"], a["vc"], a["vp"], a["start"], a["counts"], a["B"],
                                a["Hkv"], a["n"], a["cap"], a["d"], None)
    return lib.fa_kv4_read(a["kc"], a["kp"], a["vc"], a["vp"], a["k"], a["v"], a["start"], a["B"], a["Hkv"], a["n"],
                           a["cap"], a["d"], None)


@pytest.mark.parametrize("which", ["write", "read"])
@pytest.mark.parametrize("kw,code", [
    (dict(k=None), fa.FA_ERR_INVALID_ARG), (dict(vp=None), fa.FA_ERR_INVALID_ARG),
    (dict(n=-1), fa.FA_ERR_INVALID_ARG), (dict(B=0), fa.FA_ERR_INVALID_ARG),
    (dict(cap=0), fa.FA_ERR_INVALID_ARG), (dict(cap=100), fa.FA_ERR_UNSUPPORTED),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED), (dict(n=129), fa.FA_ERR_UNSUPPORTED),
    (dict(B=1 << 12, Hkv=1 << 12, cap=128), fa.FA_ERR_UNSUPPORTED),
    (dict(kc=FAKE + 8), fa.FA_ERR_ALIGN), (dict(start=FAKE + 2), fa.FA_ERR_ALIGN),
])
def test_copy_argument_errors(which, kw, code):
    assert _copy(which, **kw) == code


def _decode(**kw):
    a = dict(q=FAKE, kc=FAKE, kp=FAKE, vc=FAKE, vp=FAKE, o=FAKE, lse=FAKE, lens=None, slopes=None, ws=FAKE,
             wsb=1 << 30, B=2, Hq=8, Hkv=2, Nq=1, cap=1024, d=128, causal=0, splits=3, softcap=0.0, scale=0.1)
    a.update(kw)
    return fa.load().fa_decode_kv4(a["q"], a["kc"], a["kp"], a["vc"], a["vp"], a["o"], a["lse"], a["lens"],
                                   a["slopes"], a["ws"], a["wsb"], a["B"], a["Hq"], a["Hkv"], a["Nq"], a["cap"],
                                   a["d"], a["causal"], a["splits"], a["softcap"], a["scale"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), fa.FA_ERR_INVALID_ARG), (dict(vc=None), fa.FA_ERR_INVALID_ARG),
    (dict(lse=None), fa.FA_ERR_INVALID_ARG), (dict(Nq=0), fa.FA_ERR_INVALID_ARG),
    (dict(causal=2), fa.FA_ERR_INVALID_ARG), (dict(splits=0), fa.FA_ERR_INVALID_ARG),
    (dict(splits=1025), fa.FA_ERR_INVALID_ARG), (dict(scale=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), fa.FA_ERR_INVALID_ARG), (dict(softcap=-1.0), fa.FA_ERR_INVALID_ARG),
    (dict(softcap=float("inf")), fa.FA_ERR_INVALID_ARG), (dict(softcap=float("nan")), fa.FA_ERR_INVALID_ARG),
    (dict(d=80), fa.FA_ERR_UNSUPPORTED), (dict(cap=1000), fa.FA_ERR_UNSUPPORTED),
    (dict(Hq=8, Hkv=3), fa.FA_ERR_GQA), (dict(Hq=129, Hkv=1), fa.FA_ERR_UNSUPPORTED),
    (dict(B=1 << 24, Hkv=2, Hq=2, cap=64), fa.FA_ERR_UNSUPPORTED),
    (dict(ws=None), fa.FA_ERR_WORKSPACE), (dict(wsb=100), fa.FA_ERR_WORKSPACE),
    (dict(o=FAKE + 8), fa.FA_ERR_ALIGN), (dict(ws=FAKE + 8), fa.FA_ERR_ALIGN),
    (dict(lens=FAKE + 1), fa.FA_ERR_ALIGN), (dict(slopes=FAKE + 2), fa.FA_ERR_ALIGN),
])
def test_decode_argument_errors(kw, code):
    assert _decode(**kw) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="valid-argument path needs no GPU")
def test_valid_arguments_without_a_device_report_cuda_error():
    assert _copy("write") == fa.FA_ERR_CUDA and _copy("read") == fa.FA_ERR_CUDA
    assert _decode() == fa.FA_ERR_CUDA
    assert _decode(splits=1, ws=None, wsb=0, softcap=30.0, slopes=FAKE + 4) == fa.FA_ERR_CUDA


def test_splits_and_workspace():
    pad = lambda x: (x + 255) // 256 * 256
    # two partial results a piece: O, m and l of a tile of 8 rows (16 where there are more, d < 256)
    assert fa.fa_decode_kv4_workspace_bytes(2, 8, 2, 2, 1024, 64, 1) == 0
    assert fa.fa_decode_kv4_workspace_bytes(2, 8, 2, 2, 1024, 64, 4) == pad(4 * 2 * 8 * 66 * 4)
    assert fa.fa_decode_kv4_workspace_bytes(2, 8, 2, 3, 1024, 64, 4) == pad(4 * 2 * 16 * 66 * 4)
    assert fa.fa_decode_kv4_workspace_bytes(2, 8, 2, 3, 1024, 256, 4) == pad(4 * 2 * 8 * 258 * 4)
    assert fa.fa_decode_kv4_workspace_bytes(2, 8, 3, 3, 1024, 64, 4) == 0
    for B, Hq, Hkv, Nq, cap, dd in ((1, 1, 1, 1, 64, 64), (64, 32, 8, 1, 65536, 128), (1, 8, 8, 4, 1 << 20, 256)):
        assert 1 <= fa.fa_decode_kv4_num_splits(B, Hq, Hkv, Nq, cap, dd) <= 1024
    assert fa.fa_decode_kv4_num_splits(1, 8, 8, 1, 100, 128) == 0


def test_binding_checks():
    c = fa.KV4Cache(*(torch.zeros(1, 1, 64, n, dtype=t) for n, t in
                      ((32, torch.uint8), (4, torch.float16), (32, torch.uint8), (4, torch.float16))))
    x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: fa.kv4_write(c, x, x), lambda: fa.kv4_read(c, 2), lambda: fa.decode_kv4(x, c)):
        with pytest.raises(ValueError):    # not on the GPU
            call()
    for kw in (dict(cap=100), dict(d=96), dict(B=0), dict(cap=0)):
        a = dict(B=1, Hkv=1, cap=64, d=64)
        a.update(kw)
        with pytest.raises(ValueError):
            fa.kv4_alloc(**a, device="cpu")
    assert [tuple(t.shape) for t in fa.kv4_alloc(2, 3, 128, 128, device="cpu")] == [
        (2, 3, 128, 64), (2, 3, 128, 8), (2, 3, 128, 64), (2, 3, 128, 8)]


def test_reference_quantiser():
    # closed forms: 0 .. 15 are their own codes; a constant group has s = 0; the tie goes up
    x = np.tile(np.arange(16.0), 2)
    n, s, m = ref.quantise(x)
    assert np.array_equal(n[0], np.tile(np.arange(16), 2)) and s[0] == 1.0 and m[0] == 0.0
    n, s, m = ref.quantise(np.full(32, -2.5))
    assert (n == 0).all() and s[0] == 0.0 and m[0] == -2.5
    y = np.tile(np.arange(16.0), 2)
    y[7] = 4.5
    assert ref.quantise(y)[0][0, 7] == 5
    # nearest: no value is further than half a step off, and the top is reached
    z = np.random.default_rng(0).standard_normal((50, 96)).astype(np.float32).astype(np.float64)
    n, s, m = ref.quantise(z)
    assert (np.abs(ref.values(n, s, m) - z) <= np.repeat(s, 32, -1) / 2).all()
    # the layouts: K's word of channels 32 i + 8 c lies at c G + i
    codes = np.zeros((1, 4, 32), dtype=int)
    codes[0, 2, 8:16] = np.arange(1, 9)              # group 2, c = 1: channels 72 .. 79
    zero = np.zeros((1, 4))
    k, _ = ref.pack(codes, zero, zero, True)
    v, _ = ref.pack(codes, zero, zero, False)
    word = np.array([0x21, 0x43, 0x65, 0x87], dtype=np.uint8)
    assert np.array_equal(k[0, 4 * (1 * 4 + 2):][:4], word) and k.astype(int).sum() == word.astype(int).sum()
    assert np.array_equal(v[0, 4 * 9:][:4], word)
