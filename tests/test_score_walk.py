"""The key blocks that a forward CTA walks for its two query tiles when key ranges decide what
each tile sees (tile_walk in fa_fwd.cuh, compiled for the host with nvcc), and a model of the
forward's K/V ring over such a walk.

The MMA role frees the ring slot of a K block when a tile multiplies it, so the walk may hold no
block that neither tile sees: the model shows that the ring stalls on a walk with such a gap,
and that it runs through on tile_walk's.
"""
import itertools
import pathlib
import shutil
import subprocess

import pytest

ROOT = pathlib.Path(__file__).resolve().parents[1]
HARNESS = r'''
#include <cstdio>
#include "fa_fwd.cuh"
int main() {
  int f0, n0, f1, n1;
  while (scanf("%d %d %d %d", &f0, &n0, &f1, &n1) == 4) {
    const fa::TileWalk w = fa::tile_walk(f0, n0, f1, n1);
    printf("%d %d", w.a[0], w.a[1]);
    for (int j = 0; j < w.count; ++j) printf(" %d", w.block(j));
    printf("\n");
  }
  return 0;
}
'''

SPANS = [(0, 0), (0, 1), (0, 4), (1, 1), (2, 3), (3, 1), (3, 2), (4, 9), (5, 1), (9, 2), (14, 1), (60, 3)]
CASES = list(itertools.product(SPANS, SPANS))


@pytest.fixture(scope="module")
def walks(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not pathlib.Path(nvcc).exists():
        pytest.skip("nvcc not available")
    d = tmp_path_factory.mktemp("tile_walk")
    src = d / "harness.cu"
    src.write_text(HARNESS)
    exe = d / "harness"
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-I", str(ROOT / "include"),
                    "-I", str(ROOT / "exact_io_aware_83_b200" / "csrc"), "-o", str(exe), str(src)],
                   check=True, capture_output=True)
    text = "\n".join(" ".join(map(str, t0 + t1)) for t0, t1 in CASES)
    out = subprocess.run([str(exe)], input=text, check=True, capture_output=True, text=True).stdout.splitlines()
    assert len(out) == len(CASES)
    return {c: (tuple(v[:2]), v[2:]) for c, v in zip(CASES, (list(map(int, line.split())) for line in out))}


def _runs_through(a, n, count, slots):
    """The forward's ring: K_j, V_j of the walk's blocks in order through `slots` slots, freed by
    the MMA role's steps.  False when the loader waits for a slot that is never freed."""
    freed = set()
    landed = lambda seq: all(s in freed for s in range(seq % slots, seq, slots))  # earlier users of the slot
    first = [a[t] if n[t] else 1 << 30 for t in (0, 1)]
    last = [a[t] + n[t] - 1 for t in (0, 1)]
    if count == 0:
        return True
    if not landed(0):
        return False
    freed.add(0)
    for j in range(count):
        if not landed(2 * j + 1):
            return False
        knext = False
        for t in (0, 1):
            if j + 1 < first[t] or j > last[t] or j >= last[t]:
                continue
            if not knext and not landed(2 * j + 2):
                return False
            knext = True
        freed.add(2 * j + 1)
        if knext:
            freed.add(2 * j + 2)
    return True


def test_walk_holds_each_tiles_blocks_and_no_others(walks):
    for (t0, t1), (a, blocks) in walks.items():
        assert blocks == sorted({f + i for f, n in (t0, t1) for i in range(n)}), (t0, t1)
        for t, (f, n) in enumerate((t0, t1)):
            assert blocks[a[t]:a[t] + n] == list(range(f, f + n)), (t0, t1, t)


@pytest.mark.parametrize("slots", [4, 6])  # d = 128 and d = 64
def test_ring_runs_through_on_every_walk(walks, slots):
    for (t0, t1), (a, blocks) in walks.items():
        assert _runs_through(a, (t0[1], t1[1]), len(blocks), slots), (t0, t1)


@pytest.mark.parametrize("slots,far", [(4, 3), (6, 4)])
def test_ring_stalls_on_a_walk_with_blocks_of_neither_tile(slots, far):
    # tile 0 sees block 0, tile 1 a block `far` on, and the walk takes what lies between too
    assert not _runs_through((0, far), (1, 2), far + 2, slots)
    assert _runs_through((0, 1), (1, 2), 3, slots)
