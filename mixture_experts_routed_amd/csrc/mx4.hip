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
// Layout: packed_geom in ffn.hip, tiles of 32 x 64 weights, [64 lanes][4 columns]
// [8 K-values] of 4 bits and then 64 scale bytes: what one wavefront of the grouped
// FFN multiplies in one step. A wavefront here makes one tile: lane (nq, kg) reads
// rows 8 kg .. + 7 of columns 4 nq .. + 3 (a row's 16 lanes cover 64 columns),
// which are the lane's own 32 codes, and the block's maximum is 8 rows in
// registers and two lane exchanges. Bound by HBM.
#include "launch.hpp"
#include "mfma.hpp"

namespace moe {

namespace {

constexpr int kMinExp = -110, kMaxExp = 120;

struct Mx4Tiles {
    int Kd, N, gs, nst, nm;
    int64_t total;  // tiles of all experts
};

// the tile's expert, its first row and its first column
__device__ __forceinline__ void place(const Mx4Tiles &z, int64_t t, int64_t *e, int *k0, int *n0)
{
    const int m = (int)(t % z.nm);
    t /= z.nm;
    const int w = (int)(t & 3);
    t >>= 2;
    *k0 = (int)(t % z.nst) * 32;
    t /= z.nst;
    *n0 = ((int)(t % z.gs) * 4 + w) * 64 * z.nm + 64 * m;
    *e = t / z.gs;
}

template <typename T>
__global__ __launch_bounds__(256) void k_mx4_quantize(const T *__restrict__ src, const Mx4Tiles z,
                                                      unsigned char *__restrict__ dst)
{
    const int lane = threadIdx.x & 63, nq = lane & 15, kg = lane >> 4;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < z.total;
         t += (int64_t)gridDim.x * 4) {
        int64_t e;
        int k0, n0;
        place(z, t, &e, &k0, &n0);
        const int n = n0 + 4 * nq, k = k0 + 8 * kg;
        // (N is a multiple of 8: a lane's 4 columns are all inside or all outside)
        float v[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int c = 0; c < 4; ++c) v[i][c] = 0.f;
            if (k + i < z.Kd && n < z.N)
                Vec<T, 4>::load(src + ((e * z.Kd + k + i) * (int64_t)z.N + n), v[i]);
        }
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
        unsigned char *tile = dst + t * kMx4Tile;
        *reinterpret_cast<uint4 *>(tile + 16 * lane) =
            make_uint4(word[0], word[1], word[2], word[3]);
        if (kg == 0) *reinterpret_cast<uint32_t *>(tile + kMx4Codes + 4 * nq) = scales;
    }
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
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < z.total;
         t += (int64_t)gridDim.x * 4) {
        int64_t e;
        int k0, n0;
        place(z, t, &e, &k0, &n0);
        const int n = n0 + 4 * nq, k = k0 + 8 * kg;
        if (n >= z.N) continue;
        const unsigned char *tile = src + t * kMx4Tile;
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
                Vec<T, 4>::store(dst + ((e * z.Kd + k + i) * (int64_t)z.N + n), v[i]);
    }
}

Mx4Tiles mx4_tiles(int E, int Kd, int N, bool gateup)
{
    Mx4Tiles z;
    z.Kd = Kd;
    z.N = N;
    z.nm = gateup ? 1 : 2;
    z.gs = (N + 256 * z.nm - 1) / (256 * z.nm);
    z.nst = (Kd + 31) / 32;
    z.total = (int64_t)E * z.gs * z.nst * 4 * z.nm;
    return z;
}

dim3 mx4_grid(const Mx4Tiles &z)
{
    const int64_t want = (z.total + 3) / 4;
    return dim3((unsigned)(want < (1 << 18) ? want : 1 << 18));
}

}  // namespace

size_t mx4_weight_bytes(int E, int Kd, int N, bool gateup)
{
    return (size_t)mx4_tiles(E, Kd, N, gateup).total * kMx4Tile;
}

hipError_t launch_mx4_quantize(int dtype, const void *src, int E, int Kd, int N, bool gateup,
                               void *dst, hipStream_t s)
{
    const Mx4Tiles z = mx4_tiles(E, Kd, N, gateup);
    unsigned char *o = static_cast<unsigned char *>(dst);
    if (dtype == 0)
        hipLaunchKernelGGL(k_mx4_quantize<float>, mx4_grid(z), dim3(256), 0, s,
                           static_cast<const float *>(src), z, o);
    else if (dtype == 1)
        hipLaunchKernelGGL(k_mx4_quantize<_Float16>, mx4_grid(z), dim3(256), 0, s,
                           static_cast<const _Float16 *>(src), z, o);
    else
        hipLaunchKernelGGL(k_mx4_quantize<__bf16>, mx4_grid(z), dim3(256), 0, s,
                           static_cast<const __bf16 *>(src), z, o);
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(int dtype, const void *src, int E, int Kd, int N, bool gateup,
                                 void *dst, hipStream_t s)
{
    const Mx4Tiles z = mx4_tiles(E, Kd, N, gateup);
    const unsigned char *i = static_cast<const unsigned char *>(src);
    if (dtype == 0)
        hipLaunchKernelGGL(k_mx4_dequantize<float>, mx4_grid(z), dim3(256), 0, s, i, z,
                           static_cast<float *>(dst));
    else if (dtype == 1)
        hipLaunchKernelGGL(k_mx4_dequantize<_Float16>, mx4_grid(z), dim3(256), 0, s, i, z,
                           static_cast<_Float16 *>(dst));
    else
        hipLaunchKernelGGL(k_mx4_dequantize<__bf16>, mx4_grid(z), dim3(256), 0, s, i, z,
                           static_cast<__bf16 *>(dst));
    return hipGetLastError();
}

}  // namespace moe
