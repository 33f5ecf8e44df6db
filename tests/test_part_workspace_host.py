"""The gradients' workspace holds the parts of the tiles that have some, not whole rows
of tiles of the result; and where every part lies, by a model of how the pairs walk
the sums."""

import random

import pytest

from bitlinear_bl_forward_b200 import bl
from bitlinear_bl_forward_b200 import build as blbuild

PAIRS = 74   # CTA pairs that the sums are dealt out to
TILE = 256 * 256 * 4   # the largest tile in fp32


@pytest.fixture(scope="module")
def L():
    blbuild.build()
    return bl.lib()


SIZES = (1, 16, 33, 128, 257, 512, 1000, 1024, 1792, 2049, 4096, 6144, 8192, 16384, 32768)


@pytest.mark.parametrize("K", [64, 320, 2560, 8192, 28672, 65536])
def test_part_workspace_is_bounded(L, K):
    # dealt-out stages: at most two parts a pair, the last tiles' ends included.  (512 x
    # 28672 -> 8192 took 969 MB, 6144 x 65536 -> 8192 2.2 GB, for results of 29 and 805.)
    for M in SIZES:
        for N in (8, 64, 256, 1000, 2560, 6912, 8192, 28672):
            assert L.bl_backward_input_workspace_bytes(M, K, N) <= 2 * PAIRS * TILE
            for flags in (0, 1, 2, 3):
                assert L.bl_backward_weight_workspace_bytes(M, K, N, flags) <= 2 * PAIRS * TILE


def pieces(tiles, whole, nkv, per, nk):
    """(tile behind the whole ones, first stage, end, chunk) as a pair walks a chunk."""
    rest = (tiles - whole) * nkv
    for c in range((rest + per - 1) // per):
        u, end = c * per, min(rest, (c + 1) * per)
        while u < end:
            t = u // nkv
            c0 = u - t * nkv
            yield t, c0, min(nk, c0 + end - u), c
            u = min(end, (t + 1) * nkv)


def test_every_part_has_a_place_of_its_own():
    rng = random.Random(5)
    for i in range(400):
        tiles, nk = rng.randint(1, 120), rng.randint(4, 200)
        if i % 2:   # whole waves of whole tiles, the other tiles' stages dealt out
            whole = tiles // PAIRS * PAIRS
            if whole == tiles:
                continue
            nkv, per = nk, max(2, ((tiles - whole) * nk + PAIRS - 1) // PAIRS)
        else:       # every tile in the same number of parts
            whole, want = 0, rng.randint(2, max(2, nk // 2))
            per = (nk + want - 1) // want
            nkv = per * ((nk + per - 1) // per)
        over = int(nkv % per != 0)
        chunks = ((tiles - whole) * nkv + per - 1) // per
        places = chunks - 1 + over * (tiles - whole - 1) + 1
        seen, covered = {}, {t: [] for t in range(tiles - whole)}
        for t, c0, c1, c in pieces(tiles, whole, nkv, per, nk):
            place = c + over * t
            assert c0 < c1 and 0 <= place < places and place not in seen
            seen[place] = t
            covered[t].append((c0, c1, place))
        for t, got in covered.items():
            # the join's walk: parts in a row from the tile's first chunk, all of the sum
            first = t * nkv // per
            parts = ((t + 1) * nkv - 1) // per - first + 1
            assert [p for *_, p in got] == [first + over * t + j for j in range(parts)]
            assert got[0][0] == 0 and got[-1][1] == nk
            assert all(a[1] == b[0] for a, b in zip(got, got[1:]))
        if i % 2:
            assert places <= 2 * PAIRS
