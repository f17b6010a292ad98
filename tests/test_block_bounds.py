"""A CPU model of index arithmetic of the 4-bit weights' kernels (no kernel runs): the
narrow cells' grid against the work list's capacity and the weights' bytes, and the tiles
that quantisation writes."""
import os
import re

import pytest

from mixture_experts_routed_amd import abi

CSRC = os.path.join(os.path.dirname(abi.__file__), "csrc")
TILE = 1088
SHAPES = [(4, 8, 128, 2816, 704), (1, 1, 8, 64, 8), (3, 2, 5, 8, 64), (8, 1, 8, 128, 256),
          (61, 3, 16, 328, 200), (2, 2, 1024, 1000, 72), (16, 4, 32, 4096, 1032)]


def ceil(a, b):
    return -(-a // b)


def source(name):
    with open(os.path.join(CSRC, name)) as fh:
        return fh.read()


def geom(Kd, N, gateup):
    m = 1 if gateup else 2
    return ceil(N, 256 * m), ceil(Kd, 32), m


@pytest.mark.parametrize("T,K,E,d,f", SHAPES)
@pytest.mark.parametrize("gateup", [True, False])
def test_narrow_cells(T, K, E, d, f, gateup):
    """every workgroup finds an item inside the list, and its wavefronts' steps make up the
    slice's tiles, inside the expert's weights"""
    # the grid: the capacity times the slices, rounded up where no list is read
    assert "return z.max_items * ((N + slice - 1) / slice);" in source("ffn.hip")
    assert re.search(r"it = items\[lb / slices\];", source("ffn_mx4.hip"))
    rows = T * K + min(E, T * K) * 15
    items = rows // 64 + 1 + min(E, ceil(rows, 16))
    Kd, N = (d, f) if gateup else (f, d)
    slices = ceil(N, 64 if gateup else 128)
    blocks = items * slices
    assert {lb // slices for lb in range(blocks)} == set(range(items))
    gs, nst, m = geom(Kd, N, gateup)
    total = abi.moe_mx4_weight_bytes(E, d, f, abi.MOE_W_GATE_UP if gateup else abi.MOE_W_DOWN)
    assert total == E * gs * nst * 4 * m * TILE
    step = 4 * m * TILE
    per = ceil(nst, 4)
    for e in (0, E - 1):
        for sl in range(slices):
            g, w = sl >> 2, sl & 3
            seen = []
            for wave in range(4):
                s0 = wave * per
                n = max(0, min(per, nst - s0))
                start = (((e * gs + g) * nst + s0) * 4 + w) * m * TILE
                for stream in range(m):
                    length = n * step - (w * m + stream) * TILE if n else 0
                    first = start + stream * TILE
                    assert length >= 0
                    if n:
                        assert first + length <= total
                        # the last step's tile lies inside the range that loads are held to
                        assert (n - 1) * step + TILE <= length
                seen += range(s0, s0 + n)
            assert seen == list(range(nst))


@pytest.mark.parametrize("E,d,f", [s[2:] for s in SHAPES if s[2] < 100])
@pytest.mark.parametrize("gateup", [True, False])
def test_tiles_of_quantisation(E, d, f, gateup):
    """each tile of the packed weights is written by one wavefront, from the rows and
    columns that the layout gives it"""
    Kd, N = (d, f) if gateup else (f, d)
    gs, nst, m = geom(Kd, N, gateup)
    seen = {}
    for e in range(E):
        for x in range(gs * nst * m):
            for w in range(4):
                mm, u = (x & 1, x >> 1) if m == 2 else (0, x)
                slice_, step = divmod(u, nst)
                n0 = (slice_ * 4 + w) * 64 * m + 64 * mm
                tile = (e * gs * nst + u) * 4 * m + w * m + mm
                assert tile not in seen
                seen[tile] = (e, 32 * step, n0)
    assert sorted(seen) == list(range(E * gs * nst * 4 * m))
    for tile, at in seen.items():
        # expert, column group, K-step, slice, stream
        t, stream = divmod(tile, m)
        t, w = divmod(t, 4)
        t, s = divmod(t, nst)
        e, g = divmod(t, gs)
        assert at == (e, 32 * s, (4 * g + w) * 64 * m + 64 * stream)
