"""The index arithmetic that the 4-bit weights' kernels call (csrc/mx4_index.hpp), compiled
for the host: the tiles that quantisation writes, and the steps and bytes of each
wavefront of a narrow cell."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from mixture_experts_routed_amd import abi

CSRC = os.path.join(os.path.dirname(abi.__file__), "csrc")
TILE = 1088
SHAPES = [(8, 64, 8), (5, 8, 64), (3, 128, 256), (2, 328, 200), (2, 1000, 72), (1, 264, 520),
          (4, 40, 1032), (2, 2816, 704)]  # E, d, f
HOST = """
#include "mx4_index.hpp"
using namespace moe;
extern "C" void geometry(int Kd, int N, int gate, int E, int64_t *o)
{
    const Mx4Tiles z = mx4_tiles(Kd, N, gate);
    o[0] = z.gs, o[1] = z.nst, o[2] = z.nm, o[3] = mx4_blocks(z), o[4] = (int64_t)mx4_bytes(z, E);
}
extern "C" void place(int Kd, int N, int gate, unsigned x, unsigned expert, int w, int64_t *o)
{
    const Mx4Place p = mx4_place(mx4_tiles(Kd, N, gate), x, expert, w);
    o[0] = p.k0, o[1] = p.n0, o[2] = p.src, o[3] = p.dst;
}
extern "C" void quarter(int Kd, int N, int gate, int expert, int slice, int wave, int64_t *o)
{
    const Mx4Quarter q = mx4_quarter(mx4_tiles(Kd, N, gate), expert, slice, wave);
    o[0] = q.first, o[1] = q.count, o[2] = (int64_t)q.at, o[3] = q.bytes[0], o[4] = q.bytes[1];
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    at = tmp_path_factory.mktemp("mx4")
    (at / "host.cpp").write_text(HOST)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared", "-I", CSRC,
                    str(at / "host.cpp"), "-o", str(at / "host.so")], check=True)
    lib = ctypes.CDLL(str(at / "host.so"))

    def call(name, n, *args):
        out = (ctypes.c_int64 * n)()
        getattr(lib, name)(*args, out)
        return list(out)

    return call


def sizes(E, d, f, gate):
    return (d, f) if gate else (f, d)


def packed_bytes(E, d, f, gate):
    return abi.moe_mx4_weight_bytes(E, d, f, abi.MOE_W_GATE_UP if gate else abi.MOE_W_DOWN)


def test_the_kernels_call_it():
    for name, call in (("mx4.hip", r"\bmx4_place\(z, blockIdx\.x, blockIdx\.y,"),
                       ("mx4.hip", r"dim3\(mx4_blocks\(z\), E\)"),
                       ("mx4.hip", r"return mx4_bytes\("), ("ffn_mx4.hip", r"\bmx4_quarter\(")):
        with open(os.path.join(CSRC, name)) as fh:
            assert re.search(call, fh.read()), (name, call)


@pytest.mark.parametrize("gate", [1, 0])
@pytest.mark.parametrize("E,d,f", SHAPES)
def test_each_tile_is_written_once_from_its_rows_and_columns(host, E, d, f, gate):
    Kd, N = sizes(E, d, f, gate)
    gs, nst, m, blocks, nbytes = host("geometry", 5, Kd, N, gate, E)
    assert nbytes == packed_bytes(E, d, f, gate)
    # as the layout is documented: expert, column group, K-step, slice, stream
    want = {}
    for e in (0, E - 1):
        for g in range(-(-N // (256 * m))):
            for s in range(-(-Kd // 32)):
                for w in range(4):
                    for st in range(m):
                        t = (((e * gs + g) * nst + s) * 4 + w) * m + st
                        want[t] = [32 * s, (4 * g + w) * 64 * m + 64 * st, e * Kd * N]
    got = {}
    for e in {0, E - 1}:
        for x in range(blocks):
            for w in range(4):
                *at, tile = host("place", 4, Kd, N, gate, x, e, w)
                assert tile not in got
                got[tile] = at
    assert got == want
    assert max(got) * TILE + TILE == nbytes


@pytest.mark.parametrize("gate", [1, 0])
@pytest.mark.parametrize("E,d,f", SHAPES)
def test_a_narrow_cell_s_wavefronts_take_every_step_once(host, E, d, f, gate):
    Kd, N = sizes(E, d, f, gate)
    gs, nst, m, _, _ = host("geometry", 5, Kd, N, gate, E)
    total, step = packed_bytes(E, d, f, gate), 4 * m * TILE
    for e in (0, E - 1):
        for sl in range(-(-N // (64 * m))):
            seen = []
            for wave in range(4):
                first, count, at, *length = host("quarter", 5, Kd, N, gate, e, sl, wave)
                assert count >= 0 and (count > 0) == (length[0] > 0)
                if not count:
                    assert length == [0, 0]
                    continue
                seen += range(first, first + count)
                for stream in range(m):
                    n = length[stream] if not gate else length[0]
                    begin = at + stream * TILE
                    tile = (((e * gs + sl // 4) * nst + first) * 4 + sl % 4) * m + stream
                    assert begin == tile * TILE and begin + n <= total
                    # the last step's tile is inside the range, the next wavefront's is not
                    assert (count - 1) * step + TILE <= n <= count * step
                if gate:
                    assert length[0] == length[1]
            assert seen == list(range(nst))


def test_large_matrices_pass_32_bits(host):
    """a down matrix of 2^22 rows and 256 columns, 1,024 experts"""
    Kd, N, E = 1 << 22, 256, 1024
    gs, nst, m, blocks, nbytes = host("geometry", 5, Kd, N, 0, E)
    assert nbytes == E * nst * 4 * m * TILE
    *_, src, tile = host("place", 4, Kd, N, 0, blocks - 1, E - 1, 3)
    assert src == (E - 1) * Kd * N and (tile + 1) * TILE == nbytes
    first, count, at, b0, b1 = host("quarter", 5, Kd, N, 0, E - 1, 1, 3)
    assert first + count == nst and at + b0 <= nbytes
    assert np.iinfo(np.uint32).max > b0 == count * 4 * m * TILE - m * TILE
