// Norms around a block for gfx950, with its gate, scale and residual:
//   n = y / rms(y) w_post,  z = r + alpha gate n,  h = z / rms(z) w_pre
// and their gradients (the formulas stand at k_norm_backward).
//
// Everything is read and written once, so these kernels are bound by HBM. Up to
// kMaxCols columns a row lies in registers, 8 columns a thread: a group of threads (a
// wavefront, or a workgroup just wide enough) takes row after row and keeps the weights
// of its columns; up to 4,096 columns it issues the next row's loads before it reduces
// this one. (Of the gradients' rows above 4,096 columns some lie in scratch: threads_of.)
// Row sums are lane moves and, between wavefronts, one LDS word each and one barrier.
// Rows whose length, strides or addresses are not whole 16-byte chunks are taken an
// element a load (V = 1), thread t the columns t, t + n, ..., so that a wavefront's loads
// lie together. The weights' gradients are summed per thread over the group's rows,
// written as one partial row per group, and added over the groups in order by a second
// launch: results do not depend on timing. Longer rows are read again for each pass, an
// element a load.
//
// Measured: 32,768 rows of 2,560, fp32 y and residual, fp16 h: 245 us (1.17 GB, 4.8 TB/s;
// read again for each pass 669); in bf16 148 us (4.5 TB/s), gradients 305 (3.3). Gradients
// of 8,192 rows of 4,096, bf16, a gate per element, 102 us (537 MB, 5.3 TB/s) and 6 for the
// second launch (read again for each pass, 2,115 in all). 4 rows of 2,816: 3.5 us. A copy of
// 2 GiB moves 4.9 TB/s. Off that path, forward and gradients: 8,192 rows of 4,091, fp32 116
// and 182 us (4.6 and 4.4 TB/s), bf16 115 and 491 (2.3 and 0.8: the same number of loads for
// half the bytes, and 2-byte stores); 4,000 of 8,192, fp32 102 and 242 (5.1 and 3.2), bf16 47
// and 89; 2,048 of 16,384, fp32 246 and 1,406 (2.2 and 0.6), bf16 393 and 2,123.
// Not taken: loads or stores past the caches (forward 5 to 7% slower), columns in two
// runs of 4 a thread (forward with fp32 rows 5% faster, gradients 10 to 38% slower).
#include "lanes.hpp"
#include "launch.hpp"
#include "mfma.hpp"

namespace moe {

namespace {

constexpr int kMaxCols = 8192;   // of a row in registers: 1024 threads of 8
constexpr int kWaveCols = 512;   // of a row that a wavefront takes
constexpr int kLongThreads = 256;
// rows are summed scaled by this when their squares overflow: any sum of squares fits
constexpr float kDown = 8.271806125530277e-25f;  // 2^-80

enum : int { kGateNone = 0, kGateToken, kGateChannel, kGateFull };

// ---- a thread's 8 columns of a row -------------------------------------------

template <typename X> struct Cols {
    typedef X type __attribute__((ext_vector_type(8)));
};

// columns (V = 8: 8 tid ..; V = 1: tid + nt i) of a row, 0 past d
template <int V, typename X>
__device__ __forceinline__ typename Cols<X>::type load_cols(const X *row, int tid, int nt, int d)
{
    typename Cols<X>::type v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = X(0);
    if constexpr (V == 8) {
        if (8 * tid < d) {
            if constexpr (sizeof(X) == 2) {
                v = *reinterpret_cast<const typename Cols<X>::type *>(row + 8 * tid);
            } else {
                const float4_t *q = reinterpret_cast<const float4_t *>(row + 8 * tid);
                const float4_t a = q[0], b = q[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = a[i];
                    v[4 + i] = b[i];
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (tid + nt * i < d) v[i] = row[tid + nt * i];
    }
    return v;
}

template <int V, typename X>
__device__ __forceinline__ void store_cols(X *row, int tid, int nt, int d, const float (&v)[8])
{
    if constexpr (V == 8) {
        if (8 * tid < d) store8<X>(row + 8 * tid, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (tid + nt * i < d) row[tid + nt * i] = from_f32<X>(v[i]);
    }
}

template <typename X>
__device__ __forceinline__ void widen(const typename Cols<X>::type &c, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(c[i]);
}

// ---- the threads that share a row ----------------------------------------------

// WAVE: a wavefront (4 rows a workgroup), else the workgroup. Sums come in the same
// order to every thread.
template <bool WAVE> struct Team {
    int tid, nt;
    int64_t first, stride;  // rows
    float *lds;             // [2][2][16]
    int slot = 0;

    __device__ __forceinline__ explicit Team(float *s) : lds(s)
    {
        tid = WAVE ? threadIdx.x & 63 : threadIdx.x;
        nt = WAVE ? 64 : blockDim.x;
        first = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
        stride = WAVE ? (int64_t)gridDim.x * 4 : gridDim.x;
    }
    __device__ __forceinline__ float sum(float v)
    {
        v = group_sum<64>(v);
        if constexpr (WAVE) return v;
        float *s = lds + 32 * slot;
        slot ^= 1;  // (whoever writes a slot again has passed the barrier behind its reads)
        const int lane = threadIdx.x & 15;
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        return group_sum<16>(lane < (int)(blockDim.x >> 6) ? s[lane] : 0.f);
    }
    __device__ __forceinline__ float2 sum2(float a, float b)
    {
        a = group_sum<64>(a);
        b = group_sum<64>(b);
        if constexpr (WAVE) return make_float2(a, b);
        float *s = lds + 32 * slot;
        slot ^= 1;
        const int lane = threadIdx.x & 15;
        if ((threadIdx.x & 63) == 0) {
            s[threadIdx.x >> 6] = a;
            s[16 + (threadIdx.x >> 6)] = b;
        }
        __syncthreads();
        const bool have = lane < (int)(blockDim.x >> 6);
        return make_float2(group_sum<16>(have ? s[lane] : 0.f),
                           group_sum<16>(have ? s[16 + lane] : 0.f));
    }
    // 1 / sqrt(mean of v^2 + eps) over the row's d columns
    __device__ __forceinline__ float inverse_rms(const float (&v)[8], int d, float eps)
    {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a += v[i] * v[i];
        a = sum(a);
        if (a < __builtin_inff()) return 1.f / sqrtf(a / (float)d + eps);
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a += (v[i] * kDown) * (v[i] * kDown);
        a = sum(a);
        return kDown / sqrtf(a / (float)d + eps * kDown * kDown);
    }
};

// Most threads of a workgroup. The larger ones (more than 512 threads, at most 128 registers
// each) hold one row at a time. The forward kernels fit (71 to 121 registers); the gradients'
// hold three column sums beside the row and spill, by the compiler's count: whole chunks in
// fp32 76 registers, with 16-bit weights and an fp32 residual 16 to 23, with a 16-bit one none;
// an element a load 62 to 102, in fp32 397.
constexpr int threads_of(bool wave, bool ahead) { return wave ? 256 : ahead ? 512 : 1024; }

template <typename T, typename Y, typename R, int V, bool WAVE, bool AHEAD>
__global__ __launch_bounds__(threads_of(WAVE, AHEAD)) void k_norm(const NormCall p)
{
    __shared__ float s[64];
    Team<WAVE> team(s);
    const int tid = team.tid, nt = team.nt, d = p.d;
    const T *gate = static_cast<const T *>(p.gate);
    struct In {
        typename Cols<R>::type r;
        typename Cols<Y>::type y;
        typename Cols<T>::type g;
        float token;
    };
    auto load = [&](In &in, int64_t t) {
        in.r = load_cols<V>(static_cast<const R *>(p.r) + t * p.ldr, tid, nt, d);
        if (p.y) in.y = load_cols<V>(static_cast<const Y *>(p.y) + t * p.ldy, tid, nt, d);
        if (p.gate_kind == kGateFull) in.g = load_cols<V>(gate + t * p.ldgate, tid, nt, d);
        in.token = p.gate_kind == kGateToken ? to_f32(gate[t]) : 1.f;
    };
    int64_t t = team.first;
    if (t >= p.T) return;  // (the whole group)
    In in, next;
    load(in, t);
    typename Cols<T>::type wpost{}, wpre{}, channel{};
    if (p.w_post) wpost = load_cols<V>(static_cast<const T *>(p.w_post), tid, nt, d);
    if (p.w_pre) wpre = load_cols<V>(static_cast<const T *>(p.w_pre), tid, nt, d);
    if (p.gate_kind == kGateChannel) channel = load_cols<V>(gate, tid, nt, d);
    for (;;) {
        const int64_t t1 = t + team.stride;
        if (AHEAD && t1 < p.T) load(next, t1);
        float z[8], iy = 0.f, iz = 0.f;
        widen<R>(in.r, z);
        if (p.y) {
            float n[8], g[8];
            widen<Y>(in.y, n);
            if (p.w_post) {
                iy = team.inverse_rms(n, d, p.eps);
                widen<T>(wpost, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) n[i] = n[i] * iy * g[i];
            }
            if (p.gate_kind >= kGateChannel) {
                widen<T>(p.gate_kind == kGateFull ? in.g : channel, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) n[i] *= g[i];
            }
            const float a = p.alpha * in.token;
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] += a * n[i];
        }
        if (p.w_pre) iz = team.inverse_rms(z, d, p.eps);
        if (p.z) store_cols<V>(static_cast<R *>(p.z) + t * p.ldz, tid, nt, d, z);
        if (p.h) {
            float w[8];
            widen<T>(wpre, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = z[i] * iz * w[i];
            store_cols<V>(static_cast<T *>(p.h) + t * p.ldh, tid, nt, d, w);
        }
        if (p.stats && tid == 0) {
            p.stats[2 * t] = iy;
            p.stats[2 * t + 1] = iz;
        }
        t = t1;
        if (t >= p.T) break;
        if (AHEAD)
            in = next;
        else
            load(in, t);
    }
}

// ---- gradients -------------------------------------------------------------------
// With zn = z iz, yn = y iy (iy, iz: the saved 1 / rms), means over a row's columns:
//   dr = dz + iz (g - zn mean(g zn)),          g = dh w_pre
//   q = alpha gate dr,  dgate = alpha dr n
//   dy = iy (q w_post - yn mean(q w_post yn))  (without w_post: q)
//   dw_pre = sum of dh zn,  dw_post = sum of q yn over the rows
// The second mean needs dr: two reductions a row. In terms of the normalised values
// nothing overflows that the result does not.

constexpr int kParts = 3;  // column sums: dw_pre, dw_post, the channel gate's gradient

// groups of threads that take rows, each with its partial row: what fills the GPU
int groups_for(int T, int d)
{
    const int most = d <= kWaveCols ? 1024 : d <= 4096 ? 512 : 256;
    return T < most ? T : most;
}

template <typename T, typename Y, typename R, int V, bool WAVE, bool AHEAD>
__global__ __launch_bounds__(threads_of(WAVE, AHEAD)) void k_norm_backward(
    const NormBackwardCall p, float *__restrict__ part)
{
    __shared__ float s[64];
    Team<WAVE> team(s);
    const int tid = team.tid, nt = team.nt, d = p.d;
    const T *gate = static_cast<const T *>(p.gate);
    struct In {
        typename Cols<R>::type dz, z;
        typename Cols<T>::type dh, g;
        typename Cols<Y>::type y;
        float token;
        float2 inv;
    };
    auto load = [&](In &in, int64_t t) {
        in.inv = make_float2(p.stats[2 * t], p.stats[2 * t + 1]);
        if (p.w_pre) {
            in.z = load_cols<V>(static_cast<const R *>(p.z) + t * p.ldz, tid, nt, d);
            in.dh = load_cols<V>(static_cast<const T *>(p.dh) + t * p.lddh, tid, nt, d);
        }
        if (p.dz) in.dz = load_cols<V>(static_cast<const R *>(p.dz) + t * p.lddz, tid, nt, d);
        if (p.y) in.y = load_cols<V>(static_cast<const Y *>(p.y) + t * p.ldy, tid, nt, d);
        if (p.gate_kind == kGateFull) in.g = load_cols<V>(gate + t * p.ldgate, tid, nt, d);
        in.token = p.gate_kind == kGateToken ? to_f32(gate[t]) : 1.f;
    };
    int64_t t = team.first;
    if (t >= p.T) return;  // (the whole group)
    In in, next;
    load(in, t);
    typename Cols<T>::type wpost{}, wpre{}, channel{};
    if (p.w_post) wpost = load_cols<V>(static_cast<const T *>(p.w_post), tid, nt, d);
    if (p.w_pre) wpre = load_cols<V>(static_cast<const T *>(p.w_pre), tid, nt, d);
    if (p.gate_kind == kGateChannel) channel = load_cols<V>(gate, tid, nt, d);
    const float mean = 1.f / (float)d;
    float apre[8] = {}, apost[8] = {}, agate[8] = {};
    for (;;) {
        const int64_t t1 = t + team.stride;
        if (AHEAD && t1 < p.T) load(next, t1);
        float dr[8] = {};
        if (p.dz) widen<R>(in.dz, dr);
        if (p.w_pre) {
            float zn[8], g[8], w[8], a = 0.f;
            widen<R>(in.z, zn);
            widen<T>(in.dh, g);
            widen<T>(wpre, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                zn[i] *= in.inv.y;
                apre[i] += g[i] * zn[i];
                g[i] *= w[i];
                a += g[i] * zn[i];
            }
            a = team.sum(a) * mean;
#pragma unroll
            for (int i = 0; i < 8; ++i) dr[i] += in.inv.y * (g[i] - zn[i] * a);
        }
        store_cols<V>(static_cast<R *>(p.dr) + t * p.lddr, tid, nt, d, dr);
        if (p.y) {
            float yn[8], w[8], g[8], n, b = 0.f, c = 0.f;
            widen<Y>(in.y, yn);
            widen<T>(p.gate_kind == kGateFull ? in.g : channel, g);
            const bool each = p.gate_kind >= kGateChannel;
            if (p.w_post) {
                widen<T>(wpost, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) yn[i] *= in.inv.x;
            }
            const float at = p.alpha * in.token;
            float dg[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n = p.w_post ? yn[i] * w[i] : yn[i];
                dg[i] = p.alpha * dr[i] * n;
                const float q = (each ? at * g[i] : at) * dr[i];
                if (p.w_post) {
                    apost[i] += q * yn[i];
                    dr[i] = q * w[i];
                    b += dr[i] * yn[i];
                } else {
                    dr[i] = q;
                }
                c += dg[i];
            }
            if (p.gate_kind == kGateChannel) {
#pragma unroll
                for (int i = 0; i < 8; ++i) agate[i] += dg[i];
            }
            if (p.gate_kind == kGateFull && p.dgate)
                store_cols<V>(static_cast<T *>(p.dgate) + t * p.lddgate, tid, nt, d, dg);
            if (p.w_post || p.gate_kind == kGateToken) {
                const float2 m = team.sum2(b, c);
                if (p.w_post) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) dr[i] = in.inv.x * (dr[i] - yn[i] * (m.x * mean));
                }
                if (p.gate_kind == kGateToken && p.dgate && tid == 0)
                    static_cast<T *>(p.dgate)[t] = from_f32<T>(m.y);
            }
            if (p.dy) store_cols<V>(static_cast<Y *>(p.dy) + t * p.lddy, tid, nt, d, dr);
        }
        t = t1;
        if (t >= p.T) break;
        if (AHEAD)
            in = next;
        else
            load(in, t);
    }
    float *mine = part + team.first * kParts * d;
    if (p.dw_pre) store_cols<V>(mine, tid, nt, d, apre);
    if (p.dw_post) store_cols<V>(mine + d, tid, nt, d, apost);
    if (p.gate_kind == kGateChannel && p.dgate) store_cols<V>(mine + 2 * d, tid, nt, d, agate);
}

// ---- rows longer than kMaxCols -----------------------------------------------------

template <typename T> __device__ __forceinline__ float get(const void *p, bool f32, int64_t i)
{
    return f32 ? static_cast<const float *>(p)[i] : to_f32(static_cast<const T *>(p)[i]);
}
template <typename T> __device__ __forceinline__ void put(void *p, bool f32, int64_t i, float v)
{
    if (f32)
        static_cast<float *>(p)[i] = v;
    else
        static_cast<T *>(p)[i] = from_f32<T>(v);
}
template <typename T>
__device__ __forceinline__ float gate_of(const void *gate, int kind, int64_t ld, int64_t t, int c)
{
    const T *g = static_cast<const T *>(gate);
    return kind == kGateNone ? 1.f
                             : to_f32(g[kind == kGateToken     ? t
                                        : kind == kGateChannel ? (int64_t)c
                                                               : t * ld + c]);
}

template <typename T> __global__ __launch_bounds__(kLongThreads) void k_norm_long(const NormCall p)
{
    __shared__ float s[64];
    Team<false> team(s);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        // 1 / rms of a row given by element
        auto inverse = [&](auto at) {
            float a = 0.f;
            for (int c = threadIdx.x; c < p.d; c += kLongThreads) a += at(c) * at(c);
            a = team.sum(a);
            if (a < __builtin_inff()) return 1.f / sqrtf(a / (float)p.d + p.eps);
            a = 0.f;
            for (int c = threadIdx.x; c < p.d; c += kLongThreads) {
                const float v = at(c) * kDown;
                a += v * v;
            }
            a = team.sum(a);
            return kDown / sqrtf(a / (float)p.d + p.eps * kDown * kDown);
        };
        auto y = [&](int c) { return get<T>(p.y, p.y32, t * p.ldy + c); };
        const float iy = p.w_post ? inverse(y) : 0.f;
        auto z = [&](int c) {
            const float r = get<T>(p.r, p.r32, t * p.ldr + c);
            if (!p.y) return r;
            float n = y(c);
            if (p.w_post) n = n * iy * to_f32(static_cast<const T *>(p.w_post)[c]);
            return r + p.alpha * gate_of<T>(p.gate, p.gate_kind, p.ldgate, t, c) * n;
        };
        const float iz = p.w_pre ? inverse(z) : 0.f;
        for (int c = threadIdx.x; c < p.d; c += kLongThreads) {
            const float v = z(c);
            if (p.z) put<T>(p.z, p.r32, t * p.ldz + c, v);
            if (p.h)
                static_cast<T *>(p.h)[t * p.ldh + c] =
                    from_f32<T>(v * iz * to_f32(static_cast<const T *>(p.w_pre)[c]));
        }
        if (p.stats && threadIdx.x == 0) {
            p.stats[2 * t] = iy;
            p.stats[2 * t + 1] = iz;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kLongThreads) void k_norm_backward_long(const NormBackwardCall p,
                                                                     float *part)
{
    __shared__ float s[64];
    Team<false> team(s);
    float *mine = part + (int64_t)blockIdx.x * kParts * p.d;
    // (thread tid owns the columns tid, tid + kLongThreads, ... of each part)
    for (int k = 0; k < kParts; ++k)
        for (int c = threadIdx.x; c < p.d; c += kLongThreads) mine[(int64_t)k * p.d + c] = 0.f;
    const T *wpre = static_cast<const T *>(p.w_pre), *wpost = static_cast<const T *>(p.w_post);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const float iy = p.stats[2 * t], iz = p.stats[2 * t + 1];
        auto zn = [&](int c) { return get<T>(p.z, p.r32, t * p.ldz + c) * iz; };
        auto dh = [&](int c) { return to_f32(static_cast<const T *>(p.dh)[t * p.lddh + c]); };
        float a = 0.f;
        if (p.w_pre) {
            for (int c = threadIdx.x; c < p.d; c += kLongThreads)
                a += dh(c) * to_f32(wpre[c]) * zn(c);
            a = team.sum(a) / (float)p.d;
        }
        auto dr = [&](int c) {
            float v = p.dz ? get<T>(p.dz, p.r32, t * p.lddz + c) : 0.f;
            if (p.w_pre) v += iz * (dh(c) * to_f32(wpre[c]) - zn(c) * a);
            return v;
        };
        auto yv = [&](int c) { return get<T>(p.y, p.y32, t * p.ldy + c); };
        auto q = [&](int c) {
            return p.alpha * gate_of<T>(p.gate, p.gate_kind, p.ldgate, t, c) * dr(c);
        };
        float2 m = make_float2(0.f, 0.f);
        if (p.y) {
            for (int c = threadIdx.x; c < p.d; c += kLongThreads) {
                const float yn = p.w_post ? yv(c) * iy : yv(c);
                const float w = p.w_post ? to_f32(wpost[c]) : 1.f;
                if (p.w_post) m.x += q(c) * w * yn;
                if (p.gate_kind == kGateToken) m.y += p.alpha * dr(c) * yn * w;
            }
            m = team.sum2(m.x, m.y);
            m.x /= (float)p.d;
        }
        // (dr may lie on dz: each element is read and written by its own thread, last here)
        for (int c = threadIdx.x; c < p.d; c += kLongThreads) {
            const float r = dr(c);
            if (p.w_pre) mine[c] += dh(c) * zn(c);
            if (p.y) {
                const float yn = p.w_post ? yv(c) * iy : yv(c);
                const float w = p.w_post ? to_f32(wpost[c]) : 1.f;
                const float qc = q(c);
                if (p.w_post) mine[p.d + c] += qc * yn;
                const float dg = p.alpha * r * yn * w;
                if (p.gate_kind == kGateChannel) mine[2 * (int64_t)p.d + c] += dg;
                if (p.gate_kind == kGateFull && p.dgate)
                    static_cast<T *>(p.dgate)[t * p.lddgate + c] = from_f32<T>(dg);
                if (p.dy)
                    put<T>(p.dy, p.y32, t * p.lddy + c,
                           p.w_post ? iy * (qc * w - yn * m.x) : qc);
            }
            put<T>(p.dr, p.r32, t * p.lddr + c, r);
        }
        if (p.gate_kind == kGateToken && p.dgate && threadIdx.x == 0)
            static_cast<T *>(p.dgate)[t] = from_f32<T>(m.y);
    }
}

// ---- the groups' partial rows, added in order ---------------------------------------
// a workgroup: 64 columns of one part, 16 threads a column, each a run of the rows
constexpr int kJoinCols = 64, kJoinRuns = 16;

template <typename T>
__global__ __launch_bounds__(kJoinCols *kJoinRuns) void k_norm_join(const NormBackwardCall p,
                                                                   const float *__restrict__ part,
                                                                   int groups)
{
    __shared__ float s[kJoinRuns][kJoinCols];
    void *out[kParts] = {p.dw_pre, p.dw_post, p.gate_kind == kGateChannel ? p.dgate : nullptr};
    void *o = blockIdx.y == 0 ? out[0] : blockIdx.y == 1 ? out[1] : out[2];
    if (!o) return;
    const int col = threadIdx.x & (kJoinCols - 1), run = threadIdx.x / kJoinCols;
    const int c = blockIdx.x * kJoinCols + col;
    const int per = (groups + kJoinRuns - 1) / kJoinRuns;
    float a = 0.f;
    if (c < p.d) {
        const float *q = part + blockIdx.y * (int64_t)p.d + c;
        const int g1 = min(groups, (run + 1) * per);
#pragma unroll 8
        for (int g = run * per; g < g1; ++g) a += q[(int64_t)g * kParts * p.d];
    }
    s[run][col] = a;
    __syncthreads();
    if (run == 0 && c < p.d) {
        a = 0.f;
#pragma unroll
        for (int q = 0; q < kJoinRuns; ++q) a += s[q][col];
        put<T>(o, p.grad32, c, a);
    }
}

// ---- launchers -----------------------------------------------------------------------

// whether rows at p with stride ld are whole 16-byte chunks of 8 elements
bool whole(const void *p, int64_t ld)
{
    return !p || (ld % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0);
}

// threads of a workgroup that hold d columns, 8 each
int block_for(int d) { return d <= kWaveCols ? 256 : (d + 511) / 512 * 64; }

// the types of y and of r (with z) next to the weights'
template <typename T, typename F> hipError_t with_types(bool y32, bool r32, F run)
{
    if constexpr (sizeof(T) == 4) {
        return run(0.f, 0.f);
    } else {
        if (y32) return r32 ? run(0.f, 0.f) : run(0.f, T(0));
        return r32 ? run(T(0), 0.f) : run(T(0), T(0));
    }
}

template <typename T, typename Y, typename R, int V>
hipError_t norm_rows(const NormCall &c, hipStream_t s)
{
    const int nt = block_for(c.d);
    if (c.d <= kWaveCols) {
        const int64_t want = ((int64_t)c.T + 3) / 4;
        hipLaunchKernelGGL((k_norm<T, Y, R, V, true, true>), dim3((unsigned)(want < 2048 ? want : 2048)),
                           dim3(nt), 0, s, c);
        return hipGetLastError();
    }
    // 2,048 threads a unit: about twice what runs at once, since the kernels have 71 to 138
    // registers a thread (3 to 6 wavefronts a SIMD, not 8); the others begin as those end
    const int most = 256 * (2048 / nt);
    const dim3 grid((unsigned)(c.T < most ? c.T : most));
    if (nt <= 512)
        hipLaunchKernelGGL((k_norm<T, Y, R, V, false, true>), grid, dim3(nt), 0, s, c);
    else
        hipLaunchKernelGGL((k_norm<T, Y, R, V, false, false>), grid, dim3(nt), 0, s, c);
    return hipGetLastError();
}

template <typename T> hipError_t norm_t(const NormCall &c, hipStream_t s)
{
    if (c.d > kMaxCols) {
        hipLaunchKernelGGL(k_norm_long<T>, dim3(c.T < 4096 ? c.T : 4096), dim3(kLongThreads), 0, s, c);
        return hipGetLastError();
    }
    const bool vec = c.d % 8 == 0 && whole(c.r, c.ldr) && whole(c.y, c.ldy) && whole(c.z, c.ldz) &&
                     whole(c.h, c.ldh) && (c.gate_kind != kGateFull || whole(c.gate, c.ldgate));
    return with_types<T>(c.y32, c.r32, [&](auto y, auto r) {
        typedef decltype(y) Y;
        typedef decltype(r) R;
        return vec ? norm_rows<T, Y, R, 8>(c, s) : norm_rows<T, Y, R, 1>(c, s);
    });
}

template <typename T, typename Y, typename R, int V>
void backward_rows(const NormBackwardCall &c, float *part, int groups, hipStream_t s)
{
    const int nt = block_for(c.d);
    if (c.d <= kWaveCols)
        hipLaunchKernelGGL((k_norm_backward<T, Y, R, V, true, true>), dim3((groups + 3) / 4),
                           dim3(nt), 0, s, c, part);
    else if (nt <= 512)
        hipLaunchKernelGGL((k_norm_backward<T, Y, R, V, false, true>), dim3(groups), dim3(nt), 0, s,
                           c, part);
    else
        hipLaunchKernelGGL((k_norm_backward<T, Y, R, V, false, false>), dim3(groups), dim3(nt), 0,
                           s, c, part);
}

template <typename T> hipError_t backward_t(const NormBackwardCall &c, float *part, hipStream_t s)
{
    const int groups = groups_for(c.T, c.d);
    if (c.d > kMaxCols) {
        hipLaunchKernelGGL(k_norm_backward_long<T>, dim3(groups), dim3(kLongThreads), 0, s, c, part);
    } else {
        const bool vec = c.d % 8 == 0 && whole(c.dz, c.lddz) && whole(c.dh, c.lddh) &&
                         whole(c.z, c.ldz) && whole(c.y, c.ldy) && whole(c.dr, c.lddr) &&
                         whole(c.dy, c.lddy) &&
                         (c.gate_kind != kGateFull ||
                          (whole(c.gate, c.ldgate) && whole(c.dgate, c.lddgate)));
        (void)with_types<T>(c.y32, c.r32, [&](auto y, auto r) {
            typedef decltype(y) Y;
            typedef decltype(r) R;
            if (vec)
                backward_rows<T, Y, R, 8>(c, part, groups, s);
            else
                backward_rows<T, Y, R, 1>(c, part, groups, s);
            return hipSuccess;
        });
    }
    if (c.dw_pre || c.dw_post || (c.gate_kind == kGateChannel && c.dgate))
        hipLaunchKernelGGL(k_norm_join<T>, dim3((c.d + kJoinCols - 1) / kJoinCols, kParts),
                           dim3(kJoinCols * kJoinRuns), 0, s, c, part, groups);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormCall &c, hipStream_t s)
{
    return c.dtype == 0   ? norm_t<float>(c, s)
           : c.dtype == 1 ? norm_t<_Float16>(c, s)
                          : norm_t<__bf16>(c, s);
}

size_t norm_backward_workspace(int T, int d)
{
    return (size_t)groups_for(T, d) * kParts * d * 4;
}

hipError_t launch_norm_backward(const NormBackwardCall &c, void *ws, hipStream_t s)
{
    float *part = static_cast<float *>(ws);
    return c.dtype == 0   ? backward_t<float>(c, part, s)
           : c.dtype == 1 ? backward_t<_Float16>(c, part, s)
                          : backward_t<__bf16>(c, part, s);
}

}  // namespace moe
