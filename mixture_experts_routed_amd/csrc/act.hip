// Activation of a dense FFN with its checkpoint in 8 bits, for gfx950:
//   forward   h = act(g) u            (u optional: h = act(g))
//             g and u kept as e4m3 codes with one power-of-two scale per 32
//             columns of a row
//   backward  from the codes and dh:  dg = dh u act'(g), du = dh act(g),
//             h = act(g) u again (the operand of the next product's dw)
// Scale: with M the block's largest finite magnitude, 2^e is the least power
// of two with M <= 448 * 2^e (448: the largest e4m3 value), e within [-110,
// 120]; the byte holds e + 127. Dividing by 2^e is exact, so a code is the
// value itself rounded once to 3 fraction bits (relative error at most 2^-4,
// below 2^(e-6) absolute 2^(e-10)), and any reader decodes code * 2^e exactly. A
// value that is not finite has the code 0x7f (NaN) and no part in M.
//
// One pass, bound by HBM: a thread takes 8 columns (16 bytes of the 16-bit
// types), the 4 threads of a block of 32 share its maximum by two lane moves.
// Measured: forward, gated, 32,768 x 2,048 of bf16 (541 MB) 97-100 us, 5.4-5.6
// TB/s; backward, 32,768 x 768 of fp16 with h (253 MB) 40-47 us, 5.4-6.3 TB/s. (A
// copy of 2 GiB reaches 4.9 TB/s.)
#include "launch.hpp"
#include "mfma.hpp"

namespace moe {

namespace {

constexpr int kBlockCols = 32;
constexpr int kMinExp = -110, kMaxExp = 120;

// v[0..n) of columns c.. of a row; absent columns are 0
template <typename T, bool VEC>
__device__ __forceinline__ void load_part(const T *p, int left, float (&v)[8])
{
    if (VEC) return load8<T>(p, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(p[i]) : 0.f;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_part(T *p, int left, const float (&v)[8])
{
    if (VEC) return store8<T>(p, v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = from_f32<T>(v[i]);
}

template <bool VEC>
__device__ __forceinline__ uint2 load_codes(const uint8_t *p, int left)
{
    if (VEC) return *reinterpret_cast<const uint2 *>(p);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t *p, int left, uint2 v)
{
    if (VEC) {
        *reinterpret_cast<uint2 *>(p) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = (uint8_t)((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
}

// the codes of a thread's 8 values and, in *scale, its block's scale byte; the
// 4 threads of a block call it together
__device__ __forceinline__ uint2 encode8(const float (&v)[8], int *scale)
{
    int m = 0;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int a = __float_as_int(v[i]) & 0x7fffffff;
        const bool fin = a < 0x7f800000;
        odd |= !fin;
        m = max(m, fin ? a : 0);  // magnitudes order as their bits
    }
    m = max(m, dpp_move<kQuadXor1>(m, 0));
    m = max(m, dpp_move<kQuadXor2>(m, 0));
    const float M = __int_as_float(m);
    const int k = __builtin_amdgcn_frexp_expf(M);
    int e = __builtin_amdgcn_frexp_mantf(M) <= 0.875f ? k - 9 : k - 8;
    e = m == 0 ? kMinExp : min(max(e, kMinExp), kMaxExp);
    *scale = e + 127;
    const float inv = pow2f(-e);
    int w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int r = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, 0, false);
        w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, r, true);
    }
    if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((__float_as_int(v[i]) & 0x7fffffff) >= 0x7f800000)
                w[i >> 2] = (w[i >> 2] & ~(0xff << (8 * (i & 3)))) | (0x7f << (8 * (i & 3)));
    }
    return make_uint2((uint32_t)w[0], (uint32_t)w[1]);
}

__device__ __forceinline__ void decode8(uint2 c, int scale, float (&v)[8])
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    // 2^(scale - 127). At the largest scale, 2^120, the code that magnitudes of 248 *
    // 2^120 and more are rounded to stands for 2^128, and an infinity there would
    // make silu, gelu and their slopes NaN (-inf * 0): one step of the unit less
    // makes it fp32's largest value, and every value of such a block at most 2^-24 of
    // itself smaller. (Clamping the values took 1.5 % longer, in every block.)
    const float unit = __int_as_float((scale << 23) - (scale >= kMaxExp + 127 ? 1 : 0));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int w = (int)(h ? c.y : c.x);
        const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
        const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
        v[4 * h] = a[0] * unit;
        v[4 * h + 1] = a[1] * unit;
        v[4 * h + 2] = b[0] * unit;
        v[4 * h + 3] = b[1] * unit;
    }
}

struct ActArg {
    const void *g, *u, *dh;
    void *h, *dg, *du;
    uint8_t *g8, *gs, *u8, *us;
    int64_t ldg, ldu, lddh, ldh, lddg, lddu;
    uint32_t threads;  // rows * per_row
    uint32_t per_row;  // threads of a row: 4 per block of 32 columns
    int f, act;
};

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_act_forward(const ActArg p)
{
    const uint32_t q = blockIdx.x * 256u + threadIdx.x;
    if (q >= p.threads) return;  // whole blocks of 4 threads
    const uint32_t row = q / p.per_row, at = q - row * p.per_row;
    const int c = (int)at * 8, left = p.f - c, nb = (int)(p.per_row / 4);
    const bool have = left > 0;
    const int64_t code = (int64_t)row * p.f + c, block = (int64_t)row * nb + (at >> 2);
    float g[8] = {}, u[8] = {}, h[8];
    if (have) load_part<T, VEC>(static_cast<const T *>(p.g) + row * p.ldg + c, left, g);
    if (p.u && have) load_part<T, VEC>(static_cast<const T *>(p.u) + row * p.ldu + c, left, u);
    if (p.g8) {
        int s;
        const uint2 w = encode8(g, &s);
        if (have) store_codes<VEC>(p.g8 + code, left, w);
        if ((at & 3) == 0) p.gs[block] = (uint8_t)s;
        if (p.u) {
            const uint2 x = encode8(u, &s);
            if (have) store_codes<VEC>(p.u8 + code, left, x);
            if ((at & 3) == 0) p.us[block] = (uint8_t)s;
        }
    }
    if (!have) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        h[i] = act_apply(g[i], p.act);
        if (p.u) h[i] *= u[i];
    }
    store_part<T, VEC>(static_cast<T *>(p.h) + row * p.ldh + c, left, h);
}

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_act_backward(const ActArg p)
{
    const uint32_t q = blockIdx.x * 256u + threadIdx.x;
    if (q >= p.threads) return;
    const uint32_t row = q / p.per_row, at = q - row * p.per_row;
    const int c = (int)at * 8, left = p.f - c, nb = (int)(p.per_row / 4);
    if (left <= 0) return;
    const int64_t code = (int64_t)row * p.f + c, block = (int64_t)row * nb + (at >> 2);
    float g[8], u[8], dh[8], dg[8], h[8];
    decode8(load_codes<VEC>(p.g8 + code, left), p.gs[block], g);
    if (p.u8) decode8(load_codes<VEC>(p.u8 + code, left), p.us[block], u);
    load_part<T, VEC>(static_cast<const T *>(p.dh) + row * p.lddh + c, left, dh);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a;
        const float slope = act_slope(g[i], p.act, a);
        dg[i] = (p.u8 ? dh[i] * u[i] : dh[i]) * slope;
        h[i] = p.u8 ? a * u[i] : a;
        dh[i] *= a;
    }
    store_part<T, VEC>(static_cast<T *>(p.dg) + row * p.lddg + c, left, dg);
    if (p.u8) store_part<T, VEC>(static_cast<T *>(p.du) + row * p.lddu + c, left, dh);
    if (p.h) store_part<T, VEC>(static_cast<T *>(p.h) + row * p.ldh + c, left, h);
}

// rows per launch: thread indices stay in 32 bits
template <typename F> hipError_t in_rows(int T, int f, ActArg p, F run)
{
    p.f = f;
    p.per_row = (uint32_t)((f + kBlockCols - 1) / kBlockCols * 4);
    const int64_t most = ((int64_t)1 << 31) / p.per_row;
    for (int64_t r = 0; r < T; r += most) {
        const int64_t rows = T - r < most ? T - r : most;
        p.threads = (uint32_t)(rows * p.per_row);
        const hipError_t rc = run(p, r, dim3((p.threads + 255) / 256));
        if (rc != hipSuccess) return rc;
    }
    return hipSuccess;
}

bool rows_take_8(const void *p, int64_t ld)
{
    return !p || (ld % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0);
}

template <typename P> P *shift(P *p, int64_t bytes)
{
    return p ? reinterpret_cast<P *>(const_cast<char *>(reinterpret_cast<const char *>(p)) + bytes)
             : nullptr;
}

template <typename T> hipError_t act_t(bool back, int T_, const ActArg &all, bool vec, hipStream_t s)
{
    return in_rows(T_, all.f, all, [&](ActArg p, int64_t r, dim3 grid) {
        const int64_t es = sizeof(T), nb = p.per_row / 4;
        p.g = shift((const char *)all.g, r * all.ldg * es);
        p.u = shift((const char *)all.u, r * all.ldu * es);
        p.dh = shift((const char *)all.dh, r * all.lddh * es);
        p.h = shift((char *)all.h, r * all.ldh * es);
        p.dg = shift((char *)all.dg, r * all.lddg * es);
        p.du = shift((char *)all.du, r * all.lddu * es);
        p.g8 = shift(all.g8, r * p.f);
        p.u8 = shift(all.u8, r * p.f);
        p.gs = shift(all.gs, r * nb);
        p.us = shift(all.us, r * nb);
        if (back) {
            if (vec)
                hipLaunchKernelGGL((k_act_backward<T, true>), grid, dim3(256), 0, s, p);
            else
                hipLaunchKernelGGL((k_act_backward<T, false>), grid, dim3(256), 0, s, p);
        } else {
            if (vec)
                hipLaunchKernelGGL((k_act_forward<T, true>), grid, dim3(256), 0, s, p);
            else
                hipLaunchKernelGGL((k_act_forward<T, false>), grid, dim3(256), 0, s, p);
        }
        return hipGetLastError();
    });
}

hipError_t launch_act(bool back, int dtype, int T, const ActArg &p, bool vec, hipStream_t s)
{
    return dtype == 0 ? act_t<float>(back, T, p, vec, s)
           : dtype == 1 ? act_t<_Float16>(back, T, p, vec, s) : act_t<__bf16>(back, T, p, vec, s);
}

}  // namespace

hipError_t launch_act_forward(const void *g, int64_t ldg, const void *u, int64_t ldu, int dtype,
                              int act, int T, int f, void *h, int64_t ldh, uint8_t *g8, uint8_t *gs,
                              uint8_t *u8, uint8_t *us, hipStream_t s)
{
    ActArg p{};
    p.g = g;
    p.ldg = ldg;
    p.u = u;
    p.ldu = ldu;
    p.h = h;
    p.ldh = ldh;
    p.g8 = g8;
    p.gs = gs;
    p.u8 = u8;
    p.us = us;
    p.f = f;
    p.act = act;
    const bool vec = f % 8 == 0 && rows_take_8(g, ldg) && rows_take_8(u, ldu) && rows_take_8(h, ldh);
    return launch_act(false, dtype, T, p, vec, s);
}

hipError_t launch_act_backward(const uint8_t *g8, const uint8_t *gs, const uint8_t *u8,
                               const uint8_t *us, const void *dh, int64_t lddh, int dtype, int act,
                               int T, int f, void *dg, int64_t lddg, void *du, int64_t lddu,
                               void *h, int64_t ldh, hipStream_t s)
{
    ActArg p{};
    p.g8 = const_cast<uint8_t *>(g8);
    p.gs = const_cast<uint8_t *>(gs);
    p.u8 = const_cast<uint8_t *>(u8);
    p.us = const_cast<uint8_t *>(us);
    p.dh = dh;
    p.lddh = lddh;
    p.dg = dg;
    p.lddg = lddg;
    p.du = du;
    p.lddu = lddu;
    p.h = h;
    p.ldh = ldh;
    p.f = f;
    p.act = act;
    const bool vec = f % 8 == 0 && rows_take_8(dh, lddh) && rows_take_8(dg, lddg) &&
                     rows_take_8(du, lddu) && rows_take_8(h, ldh);
    return launch_act(true, dtype, T, p, vec, s);
}

}  // namespace moe
