"""Attention with changed scores at the edges of its arguments, on the GPU against 64-bit
references: key ranges that lie far apart or at the ends of int32, caps from the smallest fp32
number to the largest.  Bounds as in test_gpu_score.py unless a test gives its own."""
import math

import pytest
import torch

from exact_io_aware_83_b200 import fa
from test_gpu_score import _draw, _slopes, check

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
