"""A CPU model of the dense product's operand staging (no kernel runs): which
bytes each thread's load reads, where they land in LDS, and which of them each
lane's matrix fragment is read back from -- for operands with the reduction
along the rows and down the columns, both element sizes and the tile heights.
Every load lies in its operand or past the descriptor's end (zeros), the LDS
image is a permutation, and every fragment element is the element it stands
for."""
import numpy as np
import pytest

STEP = 128  # bytes of k per step of a row operand


def seg_xor(k, es):
    return ((k & 3) | ((k >> 1) & 4)) if es == 2 else ((k >> 2) & 3)


def stage(col, es, rows, nth, have, ld, K, k0):
    """LDS chunk -> byte offset from the descriptor's base (or None: zeros), as
    Operand::init / issue compute it; ld in bytes"""
    epc, bk = 16 // es, STEP // es
    cpr = rows // epc if col else 8
    out = {}
    if col:
        nrow = min(bk, K - k0)
        limit = (nrow - 1) * ld + min(have, rows) * es if nrow > 0 else 0
    else:
        limit = (min(have, rows) - 1) * ld + (K - k0) * es if K > k0 else 0
    for q in range(rows * 8):
        r, c = q // cpr, q % cpr
        if col:
            seg = 2 if es == 2 else 4
            lc = ((c // seg) ^ seg_xor(r, es)) * seg + c % seg
            off = r * ld + lc * 16 if lc * epc < have else None
        else:
            lc = c ^ ((r >> 1) & 7)
            off = r * ld + lc * 16 if r < have and k0 + lc * epc < K else None
        if off is not None and off >= limit:
            off = None  # past the descriptor: zeros
        if off is not None:
            assert off + 16 <= limit, "a chunk straddles the descriptor's end"
        assert q not in out
        out[q] = off
    assert len(out) % nth == 0
    return out


def frag(col, es, rows, first, ks, lane):
    """LDS (chunk, element) of the fragment's elements, in order"""
    epc = 16 // es
    if not col:
        r, c = first + (lane & 15), 4 * ks + (lane >> 4)
        q = r * 8 + (c ^ ((r >> 1) & 7))
        return [(q, i) for i in range(epc)]
    got = []
    if es == 2:
        for i in range(2):
            for j in range(4):
                # the transposing load: element j of lane l is element (l & 3)... of the
                # lane group's row j, column l & 15
                src = (lane & ~15) | (4 * j + ((lane & 15) >> 2))
                k = 32 * ks + 8 * (src >> 4) + 4 * i + ((src >> 2) & 3)
                seg = (first >> 4) ^ seg_xor(k, es)
                at = k * rows + seg * 16 + (src & 3) * 4 + (lane & 3)
                got.append((at // 8, at % 8))
    else:
        for j in range(4):
            k = 16 * ks + 4 * (lane >> 4) + j
            at = k * rows + ((first >> 4) ^ seg_xor(k, es)) * 16 + (lane & 15)
            got.append((at // 4, at % 4))
    return got


@pytest.mark.parametrize("col", [False, True])
@pytest.mark.parametrize("es", [2, 4])
@pytest.mark.parametrize("rows,nth", [(128, 256), (256, 512)])
@pytest.mark.parametrize("have,K,k0", [(10 ** 6, 10 ** 6, 0), (24, 40, 0), (8, 200, 128),
                                       (10 ** 6, 64, 64), (17, 65, 0), (129, 65, 64), (9, 1, 0)])
def test_fragments_are_the_elements_they_stand_for(col, es, rows, nth, have, K, k0):
    epc, bk = 16 // es, STEP // es
    # the length along an operand's rows is a whole number of chunks (its padded copy's)
    if col:
        have = -(-have // epc) * epc
    else:
        K = -(-K // epc) * epc
    ld = (max(K, 512) if not col else max(min(have, 4096), 512)) * es
    lds = stage(col, es, rows, nth, have, ld, K, k0)
    for first in range(0, rows, 16):
        for ks in range(2):
            for lane in (0, 1, 5, 15, 16, 31, 38, 63):
                per = 8 if es == 2 else 4
                for i, (q, el) in enumerate(frag(col, es, rows, first, ks, lane)):
                    r = first + (lane & 15)                       # row or column of the tile
                    k = per * 4 * ks + per * (lane >> 4) + i      # k within the step
                    off = lds[q]
                    live = r < have and k0 + k < K
                    if not live:
                        # zeros, or (16-byte chunks are whole by construction) never stored
                        assert off is None or r >= have or k0 + k >= K
                        if r < have and k0 + k >= K:
                            assert off is None  # the reduction must see zeros
                        continue
                    want = k * ld + r * es if col else r * ld + k * es
                    assert off is not None and off + el * es == want, (first, ks, lane, i)
