// Expert weights in microscaled 4-bit floating point for gfx950: quantisation
// into the layout that the grouped FFN streams, and the way back.
//
// Format: blocks of 32 weights along the reduction (K) share a scale 2^e, stored
// as the byte e + 127; a weight is an e2m1 code (sign, 2 exponent bits, 1
// fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times it. With M the block's largest
// magnitude, e is the least with M <= 6 * 2^e, within [-110, 120] (-110 for M =
// 0): no value is clamped (but above 6 * 2^120), and quantising what a block of
// this format stands for gives the same values again. Codes are nearest, ties to
// the even code. A block with a value that is not finite gets the byte 255 and
// reads back as NaN.
//
// Layout: packed_geom in ffn_cells.hpp, tiles of 32 x 64 weights, [64 lanes][4 columns]
// [8 K-values] of 4 bits and then 64 scale bytes: what one wavefront of the grouped
// FFN multiplies in one step. A wavefront here makes one tile: lane (nq, kg) reads
// rows 8 kg .. + 7 of columns 4 nq .. + 3 (a row's 16 lanes cover 64 columns),
// which are the lane's own 32 codes, and the block's maximum is 8 rows in
// registers and two lane exchanges.
//
// Both ways are bound by HBM. Measured at 128 experts of 2816 x 704, bf16 (642 MB either
// way): quantising 117 us (5.5 TB/s), back 95.5 us (6.7 TB/s); a copy of 2 GiB moves 4.9
// TB/s. Weights are read and written past the caches (a line is used once, by one
// wavefront): quantising 145 -> 117 us, back 100 -> 95.5. The codes are not (they stay
// for whoever reads them next): quantising would gain 9 us, reading back lose 15.
#include "launch.hpp"
#include "mfma.hpp"

namespace moe {

namespace {

constexpr int kMinExp = -110, kMaxExp = 120;

// All of a tile's place is the same for a wavefront (mx4_index.hpp), so one scalar division
// finds it: with a running tile number, divided in 64 bits per lane, quantising took 178 us,
// not 162.
__device__ __forceinline__ Mx4Place place(const Mx4Tiles &z)
{
    return mx4_place(z, blockIdx.x, blockIdx.y,
                     __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
}

template <typename T>
__global__ __launch_bounds__(256) void k_mx4_quantize(const T *__restrict__ src, const Mx4Tiles z,
                                                      unsigned char *__restrict__ dst)
{
    const int lane = threadIdx.x & 63, nq = lane & 15, kg = lane >> 4;
    const Mx4Place at = place(z);
    const int n = at.n0 + 4 * nq, k = at.k0 + 8 * kg;
    // (N is a multiple of 8: a lane's 4 columns are all inside or all outside.) Rows and
    // columns past the matrix read its last row or first columns and count as 0, so that
    // all eight loads are in flight at once.
    typename Vec<T, 4>::type raw[8];
    const T *from = src + at.src + (n < z.N ? n : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        raw[i] = __builtin_nontemporal_load(reinterpret_cast<const typename Vec<T, 4>::type *>(
            from + (int64_t)min(k + i, z.Kd - 1) * z.N));
    float v[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[i][c] = k + i < z.Kd && n < z.N ? to_f32(raw[i][c]) : 0.f;
    uint32_t word[4], scales = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        int m = 0;  // magnitudes order as their bits, what is not finite last
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_int(v[i][c]) & 0x7fffffff);
        m = max(m, __shfl_xor(m, 16));
        m = max(m, __shfl_xor(m, 32));
        const bool odd = m >= 0x7f800000;
        const float M = __int_as_float(m);
        const int x = __builtin_amdgcn_frexp_expf(M);
        int ex = __builtin_amdgcn_frexp_mantf(M) <= 0.75f ? x - 3 : x - 2;
        ex = m == 0 || odd ? kMinExp : min(max(ex, kMinExp), kMaxExp);
        const float inv = pow2f(-ex);
        uint32_t o = 0;
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[0][c] * inv, v[1][c] * inv, 1.f, 0);
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[2][c] * inv, v[3][c] * inv, 1.f, 1);
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[4][c] * inv, v[5][c] * inv, 1.f, 2);
        o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[6][c] * inv, v[7][c] * inv, 1.f, 3);
        word[c] = o;
        scales |= (odd ? 255u : (uint32_t)(ex + 127)) << (8 * c);
    }
    unsigned char *tile = dst + at.dst * kMx4Tile;
    *reinterpret_cast<uint4 *>(tile + 16 * lane) =
        make_uint4(word[0], word[1], word[2], word[3]);
    if (kg == 0) *reinterpret_cast<uint32_t *>(tile + kMx4Codes + 4 * nq) = scales;
}

// codes 2 j and 2 j + 1 of a word times their scale
template <int J> __device__ __forceinline__ float2 decode2(uint32_t w, float scale)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, J);
    return make_float2(v[0], v[1]);
}

template <typename T>
__global__ __launch_bounds__(256) void k_mx4_dequantize(const unsigned char *__restrict__ src,
                                                        const Mx4Tiles z, T *__restrict__ dst)
{
    const int lane = threadIdx.x & 63, nq = lane & 15, kg = lane >> 4;
    const Mx4Place at = place(z);
    const int n = at.n0 + 4 * nq, k = at.k0 + 8 * kg;
    if (n >= z.N) return;
    const unsigned char *tile = src + at.dst * kMx4Tile;
    const uint4 q = *reinterpret_cast<const uint4 *>(tile + 16 * lane);
    const uint32_t scales = *reinterpret_cast<const uint32_t *>(tile + kMx4Codes + 4 * nq);
    const uint32_t word[4] = {q.x, q.y, q.z, q.w};
    float v[8][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float s = __uint_as_float(((scales >> (8 * c)) & 0xffu) << 23);
        const float2 a = decode2<0>(word[c], s), b = decode2<1>(word[c], s);
        const float2 g = decode2<2>(word[c], s), h = decode2<3>(word[c], s);
        const float col[8] = {a.x, a.y, b.x, b.y, g.x, g.y, h.x, h.y};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i][c] = col[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k + i < z.Kd)
            Vec<T, 4>::template store<true>(dst + at.src + ((int64_t)(k + i) * z.N + n), v[i]);
}

// (a matrix of at most 2^30 weights has fewer than 2^24 tiles)
dim3 mx4_grid(const Mx4Tiles &z, int E) { return dim3(mx4_blocks(z), E); }

}  // namespace

size_t mx4_weight_bytes(int E, int Kd, int N, bool gateup)
{
    return mx4_bytes(mx4_tiles(Kd, N, gateup), E);
}

hipError_t launch_mx4_quantize(int dtype, const void *src, int E, int Kd, int N, bool gateup,
                               void *dst, hipStream_t s)
{
    const Mx4Tiles z = mx4_tiles(Kd, N, gateup);
    unsigned char *o = static_cast<unsigned char *>(dst);
    if (dtype == 0)
        hipLaunchKernelGGL(k_mx4_quantize<float>, mx4_grid(z, E), dim3(256), 0, s,
                           static_cast<const float *>(src), z, o);
    else if (dtype == 1)
        hipLaunchKernelGGL(k_mx4_quantize<_Float16>, mx4_grid(z, E), dim3(256), 0, s,
                           static_cast<const _Float16 *>(src), z, o);
    else
        hipLaunchKernelGGL(k_mx4_quantize<__bf16>, mx4_grid(z, E), dim3(256), 0, s,
                           static_cast<const __bf16 *>(src), z, o);
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(int dtype, const void *src, int E, int Kd, int N, bool gateup,
                                 void *dst, hipStream_t s)
{
    const Mx4Tiles z = mx4_tiles(Kd, N, gateup);
    const unsigned char *i = static_cast<const unsigned char *>(src);
    if (dtype == 0)
        hipLaunchKernelGGL(k_mx4_dequantize<float>, mx4_grid(z, E), dim3(256), 0, s, i, z,
                           static_cast<float *>(dst));
    else if (dtype == 1)
        hipLaunchKernelGGL(k_mx4_dequantize<_Float16>, mx4_grid(z, E), dim3(256), 0, s, i, z,
                           static_cast<_Float16 *>(dst));
    else
        hipLaunchKernelGGL(k_mx4_dequantize<__bf16>, mx4_grid(z, E), dim3(256), 0, s, i, z,
                           static_cast<__bf16 *>(dst));
    return hipGetLastError();
}

}  // namespace moe
