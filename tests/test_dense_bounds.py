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


def seg_xor(k, es, rows):
    return (k >> 2) & 1 if es == 4 else k & 2 if rows == 64 else (k & 3) << 1


def stage(col, es, rows, nth, have, ld, K, k0):
    """LDS chunk -> byte offset from the descriptor's base (or None: zeros), as
    Operand::init / issue compute it; ld in bytes"""
    epc, bk = 16 // es, STEP // es
    cpr = rows // epc if col else STEP // 16
    out = {}
    if col:
        nrow = min(bk, K - k0)
        limit = (nrow - 1) * ld + min(have, rows) * es if nrow > 0 else 0
    else:
        limit = (min(have, rows) - 1) * ld + (K - k0) * es if K > k0 else 0
    for q in range(rows * STEP // 16):
        r, c = q // cpr, q % cpr
        if col:
            seg = 2 if es == 2 else 8
            lc = ((c // seg) ^ seg_xor(r, es, rows)) * seg + c % seg
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


def frag(col, es, rows, i, g, lane):
    """LDS (chunk, element) of the elements of fragment i (32 rows), k-group g, in order"""
    epc = 16 // es
    if not col:
        r, c = 32 * i + (lane & 31), 2 * g + (lane >> 5)
        q = r * 8 + (c ^ ((r >> 1) & 7))
        return [(q, e) for e in range(epc)]
    got = []
    if es == 2:
        for half in range(2):
            for j in range(4):
                # the transposing load gives lane l, element j: what lane 4 j + (l & 15) / 4
                # of its 16 lanes points at, element l & 3
                src = (lane & ~15) | (4 * j + ((lane & 15) >> 2))
                k = 8 * (src >> 5) + ((src >> 2) & 3)
                seg = (2 * i + ((src >> 4) & 1)) ^ seg_xor(k, es, rows)
                at = (k + 4 * half + 16 * g) * rows + seg * 16 + (src & 3) * 4 + (lane & 3)
                got.append((at // 8, at % 8))
    else:
        for j in range(4):
            k = 4 * (lane >> 5)
            at = (k + j + 8 * g) * rows + (i ^ seg_xor(k, es, rows)) * 32 + (lane & 31)
            got.append((at // 4, at % 4))
    return got


@pytest.mark.parametrize("col", [False, True])
@pytest.mark.parametrize("es", [2, 4])
@pytest.mark.parametrize("rows,nth", [(64, 256), (128, 256), (256, 256)])
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
    size = bk // 4  # values of k in a group
    for i in range(rows // 32):
        for g in range(4):
            for lane in (0, 1, 5, 15, 16, 31, 32, 38, 49, 63):
                per = 8 if es == 2 else 4
                for e, (q, el) in enumerate(frag(col, es, rows, i, g, lane)):
                    r = 32 * i + (lane & 31)              # row or column of the tile
                    k = size * g + per * (lane >> 5) + e  # k within the step
                    off = lds[q]
                    if r >= have or k0 + k >= K:
                        assert off is None                # the reduction must see zeros
                        continue
                    want = k * ld + r * es if col else r * ld + k * es
                    assert off is not None and off + el * es == want, (i, g, lane, e)


@pytest.mark.parametrize("es", [2, 4])
@pytest.mark.parametrize("col", [False, True])
@pytest.mark.parametrize("rows", [64, 128, 256])
def test_reads_spread_over_the_banks(col, es, rows):
    """the lanes that the LDS serves together touch 32-bit banks evenly: 8 lanes of
    16 bytes (rows), 32 lanes of 8 bytes (columns, 16-bit types), 64 lanes of 4
    bytes (fp32), each at most once a bank of 64"""
    for g in range(4):
        for i in range(rows // 32):
            if not col:
                groups = [[r * 128 + (((2 * g + (l >> 5)) ^ ((r >> 1) & 7)) * 16) + 4 * w
                           for l in range(8 * p, 8 * p + 8) for r in [32 * i + (l & 31)]
                           for w in range(4)] for p in range(8)]
            elif es == 2:
                groups = [[((8 * (l >> 5) + ((l >> 2) & 3) + 16 * g) * rows
                            + ((2 * i + ((l >> 4) & 1)) ^ seg_xor((l >> 2) & 3, 2, rows)) * 16) * 2
                           + (l & 3) * 8 + 4 * w
                           for l in range(32 * p, 32 * p + 32) for w in range(2)] for p in range(2)]
            else:
                groups = [[((4 * (l >> 5) + 8 * g) * rows
                            + (i ^ seg_xor(4 * (l >> 5), 4, rows)) * 32 + (l & 31)) * 4
                           for l in range(64)]]
            for at in groups:
                banks = [(b // 4) % 64 for b in at]
                assert len(set(banks)) == len(banks)


@pytest.mark.parametrize("es", [2, 4])
def test_column_sums_read_only_their_rows(es):
    """a thread of the column sums takes 8 columns of a row: in one piece where they are
    all there (16-bit rows end with a whole chunk of 8, fp32 rows with one of 4)"""
    epc = 16 // es
    for n in list(range(epc, 40, epc)) + [256 - epc, 256, 256 + epc, 264]:
        seen = set()
        for c in range(0, -(-n // 256) * 256, 8):
            if c >= n:
                continue
            whole = es == 2 or c + 8 <= n
            cols = [c + i for i in range(8) if whole or c + i < n]
            assert max(cols) < n
            seen.update(cols)
        assert seen == set(range(n))
