// Norms around a block for gfx950, with its gate, scale and residual:
//   n = y / rms(y) w_post,  z = r + alpha gate n,  h = z / rms(z) w_pre
// and their gradients. A workgroup takes a row at a time, a thread the columns
// tid, tid + 256, ...; the weights' gradients are summed per workgroup and column,
// then over the workgroups in order.
#include "launch.hpp"
#include "mfma.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;

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

// sum over the workgroup, in every thread
__device__ __forceinline__ float block_sum(float v, float *s)
{
#pragma unroll
    for (int h = 32; h > 0; h >>= 1) v += __shfl_xor(v, h);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    float a = 0.f;
#pragma unroll
    for (int q = 0; q < kThreads / 64; ++q) a += s[q];
    return a;
}

constexpr float kDown = 8.271806125530277e-25f;  // 2^-80: sums of any squares fit

template <typename T>
__device__ __forceinline__ float gate_of(const void *gate, int kind, int64_t ld, int64_t t, int c)
{
    return kind == 0 ? 1.f
                     : to_f32(static_cast<const T *>(gate)[kind == 1   ? t
                                                           : kind == 2 ? (int64_t)c
                                                                       : t * ld + c]);
}

template <typename T> __global__ __launch_bounds__(kThreads) void k_norm(const NormCall p)
{
    __shared__ float s[kThreads / 64];
    const float inf = __builtin_inff();
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        // 1 / rms of a row given by element
        auto inverse = [&](auto at) {
            float a = 0.f;
            for (int c = threadIdx.x; c < p.d; c += kThreads) a += at(c) * at(c);
            a = block_sum(a, s);
            if (a < inf) return 1.f / sqrtf(a / (float)p.d + p.eps);
            a = 0.f;
            for (int c = threadIdx.x; c < p.d; c += kThreads) {
                const float v = at(c) * kDown;
                a += v * v;
            }
            a = block_sum(a, s);
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
        for (int c = threadIdx.x; c < p.d; c += kThreads) {
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

constexpr int kParts = 3;  // column sums: dw_pre, dw_post, the channel gate's gradient
int blocks_for(int T) { return T < 256 ? T : 256; }

template <typename T>
__global__ __launch_bounds__(kThreads) void k_norm_backward(const NormBackwardCall p, float *part)
{
    __shared__ float s[kThreads / 64];
    float *mine = part + (int64_t)blockIdx.x * kParts * p.d;
    for (int c = threadIdx.x; c < kParts * p.d; c += kThreads) mine[c] = 0.f;
    __syncthreads();
    const T *wpre = static_cast<const T *>(p.w_pre), *wpost = static_cast<const T *>(p.w_post);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const float iy = p.stats[2 * t], iz = p.stats[2 * t + 1];
        auto zn = [&](int c) { return get<T>(p.z, p.r32, t * p.ldz + c) * iz; };
        auto dh = [&](int c) { return to_f32(static_cast<const T *>(p.dh)[t * p.lddh + c]); };
        float a = 0.f;
        if (p.w_pre) {
            for (int c = threadIdx.x; c < p.d; c += kThreads) a += dh(c) * to_f32(wpre[c]) * zn(c);
            a = block_sum(a, s) / (float)p.d;
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
        float b = 0.f, g = 0.f;
        if (p.y) {
            for (int c = threadIdx.x; c < p.d; c += kThreads) {
                const float yn = p.w_post ? yv(c) * iy : yv(c);
                const float w = p.w_post ? to_f32(wpost[c]) : 1.f;
                if (p.w_post) b += q(c) * w * yn;
                if (p.gate_kind == 1) g += p.alpha * dr(c) * yn * w;
            }
            b = block_sum(b, s) / (float)p.d;
            g = block_sum(g, s);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.d; c += kThreads) {
            const float r = dr(c);
            if (p.w_pre) mine[c] += dh(c) * zn(c);
            if (p.y) {
                const float yn = p.w_post ? yv(c) * iy : yv(c);
                const float w = p.w_post ? to_f32(wpost[c]) : 1.f;
                const float qc = q(c);
                if (p.w_post) mine[p.d + c] += qc * yn;
                const float dg = p.alpha * r * yn * w;
                if (p.gate_kind == 2) mine[2 * p.d + c] += dg;
                if (p.gate_kind == 3 && p.dgate)
                    static_cast<T *>(p.dgate)[t * p.lddgate + c] = from_f32<T>(dg);
                if (p.dy) put<T>(p.dy, p.y32, t * p.lddy + c, p.w_post ? iy * (qc * w - yn * b) : qc);
            }
            put<T>(p.dr, p.r32, t * p.lddr + c, r);
        }
        if (p.gate_kind == 1 && p.dgate && threadIdx.x == 0)
            static_cast<T *>(p.dgate)[t] = from_f32<T>(g);
        __syncthreads();
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_norm_join(const NormBackwardCall p, const float *part,
                                                        int blocks)
{
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= p.d) return;
    void *out[kParts] = {p.dw_pre, p.dw_post, p.gate_kind == 2 ? p.dgate : nullptr};
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
        if (!out[k]) continue;
        float a = 0.f;
        for (int b = 0; b < blocks; ++b) a += part[((int64_t)b * kParts + k) * p.d + c];
        put<T>(out[k], p.grad32, c, a);
    }
}

template <typename T> hipError_t backward_t(const NormBackwardCall &c, float *part, hipStream_t s)
{
    const int blocks = blocks_for(c.T);
    hipLaunchKernelGGL(k_norm_backward<T>, dim3(blocks), dim3(kThreads), 0, s, c, part);
    if (c.dw_pre || c.dw_post || (c.gate_kind == 2 && c.dgate))
        hipLaunchKernelGGL(k_norm_join<T>, dim3((c.d + kThreads - 1) / kThreads), dim3(kThreads), 0,
                           s, c, part, blocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormCall &c, hipStream_t s)
{
    const dim3 grid(c.T < 65536 ? c.T : 65536);
    if (c.dtype == 0)
        hipLaunchKernelGGL(k_norm<float>, grid, dim3(kThreads), 0, s, c);
    else if (c.dtype == 1)
        hipLaunchKernelGGL(k_norm<_Float16>, grid, dim3(kThreads), 0, s, c);
    else
        hipLaunchKernelGGL(k_norm<__bf16>, grid, dim3(kThreads), 0, s, c);
    return hipGetLastError();
}

size_t norm_backward_workspace(int T, int d) { return (size_t)blocks_for(T) * kParts * d * 4; }

hipError_t launch_norm_backward(const NormBackwardCall &c, void *ws, hipStream_t s)
{
    float *part = static_cast<float *>(ws);
    return c.dtype == 0   ? backward_t<float>(c, part, s)
           : c.dtype == 1 ? backward_t<_Float16>(c, part, s)
                          : backward_t<__bf16>(c, part, s);
}

}  // namespace moe
