// Where the 4-bit weights' kernels find their tiles: index arithmetic in plain constant
// expressions, which kernels, launchers and host programs call alike (no HIP in here).
// The layout: expert, column group (4 slices), K-step of 32 rows, slice, stream; a tile
// is 32 x 64 weights.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {

// bytes of the codes, and of codes and scales, of a tile
constexpr uint32_t kMx4Codes = 1024, kMx4Tile = 1088;

// An expert's matrix of Kd rows and N columns: column groups, K-steps, streams of a slice
// (gate and up matrices one of 64 columns, down matrices two).
struct Mx4Tiles {
    int Kd, N, gs, nst, nm;
};
constexpr Mx4Tiles mx4_tiles(int Kd, int N, bool gateup)
{
    const int nm = gateup ? 1 : 2;
    return Mx4Tiles{Kd, N, (N + 256 * nm - 1) / (256 * nm), (Kd + 31) / 32, nm};
}
// bytes of E experts' matrices
constexpr size_t mx4_bytes(const Mx4Tiles &z, int E)
{
    return (size_t)E * z.gs * z.nst * 4 * z.nm * kMx4Tile;
}
// workgroups an expert whose four wavefronts take one tile each
constexpr unsigned mx4_blocks(const Mx4Tiles &z) { return (unsigned)z.gs * z.nst * z.nm; }

// The tile of wavefront w of an expert's workgroup x: a workgroup has the four slices'
// tiles of one K-step, column group and stream.
struct Mx4Place {
    int k0, n0;   // the tile's first row and column
    int64_t src;  // the expert's first weight
    int64_t dst;  // the tile
};
constexpr Mx4Place mx4_place(const Mx4Tiles &z, unsigned x, unsigned expert, int w)
{
    const int m = z.nm == 2 ? x & 1 : 0;
    const unsigned u = z.nm == 2 ? x >> 1 : x;
    const unsigned group = u / (unsigned)z.nst, step = u - group * z.nst;
    return Mx4Place{(int)step * 32, ((int)group * 4 + w) * 64 * z.nm + 64 * m,
                    (int64_t)expert * z.Kd * z.N,
                    ((int64_t)expert * z.gs * z.nst + u) * (4 * z.nm) + w * z.nm + m};
}

// A quarter of a slice's K-steps, wavefront `wave`'s of a narrow cell: steps [first, first +
// count), the first one's tile as a byte offset, and from each stream's first tile on the
// bytes that loads may touch (0: no steps). Steps are 4 * nm tiles apart.
struct Mx4Quarter {
    int first, count;
    size_t at;
    uint32_t bytes[2];
};
constexpr Mx4Quarter mx4_quarter(const Mx4Tiles &z, int expert, int slice, int wave)
{
    const int per = (z.nst + 3) / 4, first = wave * per;
    const int left = z.nst - first, some = per < left ? per : left, count = some > 0 ? some : 0;
    const int g = slice >> 2, w = slice & 3;
    const uint32_t span = (uint32_t)count * (4 * (uint32_t)z.nm * kMx4Tile);
    return Mx4Quarter{first, count,
                      ((((size_t)expert * z.gs + g) * z.nst + first) * 4 + w) * z.nm * kMx4Tile,
                      {count > 0 ? span - (uint32_t)(w * z.nm) * kMx4Tile : 0u,
                       count > 0 ? span - (uint32_t)(w * z.nm + z.nm - 1) * kMx4Tile : 0u}};
}

}  // namespace moe
