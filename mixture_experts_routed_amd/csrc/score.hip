// Routing by scores for gfx950, and the gradient of the logits.
//   s_e = softmax or sigmoid of the logits,  c_e = s_e + bias_e
//   groups of E / G experts: worth = sum of the group_top largest c; `keep` stay
//   the K largest c of those, ties to the lower index; w = scale s (/ sum of s)
// One wavefront per token, lane l holding experts l, l + 64, ...
#include "launch.hpp"
#include "mfma.hpp"

namespace moe {

namespace {

constexpr int kWaves = 4;  // tokens of a workgroup

__device__ __forceinline__ double wave_sum_f64(double v)
{
#pragma unroll
    for (int h = 32; h > 0; h >>= 1) v += __shfl_xor(v, h);
    return v;
}
__device__ __forceinline__ float wave_max_f32(float v)
{
#pragma unroll
    for (int h = 32; h > 0; h >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, h));
    return v;
}
__device__ __forceinline__ float wave_sum_f32(float v)
{
#pragma unroll
    for (int h = 32; h > 0; h >>= 1) v += __shfl_xor(v, h);
    return v;
}

template <int NJ>
__global__ __launch_bounds__(kWaves * 64) void k_route_scored(const ScoreCall p)
{
    extern __shared__ double s_c[];  // [kWaves][E], with groups
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= p.T) return;
    const float *row = p.logits + t * p.E;
    const double inf = __builtin_inf();
    double s[NJ], c[NJ];
    float l[NJ], m = -__builtin_inff();
    uint32_t there = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = lane + kWave * j;
        l[j] = e < p.E ? row[e] : -__builtin_inff();
        if (l[j] > -__builtin_inff()) {  // not NaN
            there |= 1u << j;
            m = __builtin_fmaxf(m, l[j]);
        }
    }
    if (p.sigmoid) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[j] = (there >> j & 1) ? 1.0 / (1.0 + exp(-(double)l[j])) : 0.0;
    } else {
        m = wave_max_f32(m);
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            // (+inf logits share everything)
            s[j] = !(there >> j & 1) ? 0.0
                   : m == __builtin_inff() ? (l[j] == m ? 1.0 : 0.0) : exp((double)l[j] - (double)m);
            sum += s[j];
        }
        sum = wave_sum_f64(sum);
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[j] = sum > 0.0 ? s[j] / sum : 0.0;
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = lane + kWave * j;
        c[j] = s[j];
        if (p.bias && e < p.E) {
            const float b = p.bias[e];
            if (!(b > -__builtin_inff())) there &= ~(1u << j);
            c[j] += (double)b;
        }
    }
    if (p.groups > 1) {
        double *mine = s_c + (int64_t)wave * p.E;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = lane + kWave * j;
            if (e < p.E) mine[e] = (there >> j & 1) ? c[j] : -inf;
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int n = p.E / p.groups;
        double worth = -inf, next = -inf;
        if (lane < p.groups)
            for (int i = 0; i < n; ++i) {
                const double v = mine[lane * n + i];
                if (v > worth) {
                    next = worth;
                    worth = v;
                } else if (v > next) {
                    next = v;
                }
            }
        if (p.group_top > 1 && next > -inf) worth += next;
        int before = 0;
        for (int g = 0; g < p.groups; ++g) {
            const double o = __shfl(worth, g);
            before += o > worth || (o == worth && g < lane);
        }
        const uint64_t kept = __ballot(lane < p.groups && before < p.keep);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = lane + kWave * j;
            if (e < p.E && !(kept >> (e / n) & 1)) there &= ~(1u << j);
        }
    }
    double my_s = 0.0, total = 0.0;
    float my_l = 0.f, top_l = 0.f;
    int my_id = -1;
    if (!p.bias) {  // by the logits, of which the score is a rising function
#pragma unroll
        for (int j = 0; j < NJ; ++j) c[j] = (double)l[j];
    }
    for (int k = 0; k < p.K; ++k) {
        double best = -inf;
        int id = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if ((there >> j & 1) && (c[j] > best || id == 0x7fffffff)) {
                best = c[j];
                id = lane + kWave * j;
            }
#pragma unroll
        for (int h = 32; h > 0; h >>= 1) {
            const double ob = __shfl_xor(best, h);
            const int oi = __shfl_xor(id, h);
            if (ob > best || (ob == best && oi < id)) {
                best = ob;
                id = oi;
            }
        }
        if (id == 0x7fffffff) break;  // (the same in every lane)
        const int slot = id >> 6, owner = id & 63;
        double v = 0.0;
        float q = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (j == slot) {
                v = s[j];
                q = l[j];
            }
        v = __shfl(v, owner);
        q = __shfl(q, owner);
        if (lane == owner) there &= ~(1u << slot);
        if (lane == k) {
            my_id = id;
            my_s = v;
            my_l = q;
        }
        top_l = k == 0 ? q : __builtin_fmaxf(top_l, q);
    }
    if (p.renorm && my_id >= 0) {
        // a common factor for scores that are all too small to add up
        const double base = p.sigmoid ? (double)__builtin_fminf(top_l, 0.f) : (double)top_l;
        if (p.sigmoid)
            my_s = my_l >= 0.f ? my_s : exp((double)my_l - base) / (1.0 + exp((double)my_l));
        else
            my_s = top_l == __builtin_inff() ? (my_l == top_l ? 1.0 : 0.0)
                                             : exp((double)my_l - base);
    }
    total = p.renorm ? wave_sum_f64(my_id >= 0 ? my_s : 0.0) : 1.0;
    if (lane < p.K) {
        p.ids[t * p.K + lane] = my_id;
        p.w[t * p.K + lane] = my_id >= 0 ? (float)((double)p.scale * (my_s / total)) : 0.f;
    }
}

template <typename T, int NJ>
__global__ __launch_bounds__(kWaves * 64) void k_route_scored_backward(const ScoreBackwardCall p)
{
    extern __shared__ float s_row[];  // [kWaves][E]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
    if (t >= p.T) return;
    float *mine = s_row + (int64_t)wave * p.E;
    const float *row = p.logits + t * p.E;
    const float inf = __builtin_inff();
    for (int e = lane; e < p.E; e += 64) mine[e] = 0.f;
    const int id = lane < p.K ? p.ids[t * p.K + lane] : -1;
    bool ok = (unsigned)id < (unsigned)p.E;
    const float l = ok ? row[id] : -inf;
    ok = ok && l > -inf;
    const float u = ok ? p.scale * p.dw[t * p.K + lane] : 0.f;
    float g = 0.f, total = 0.f;
    // softmax over all experts
    float pr[NJ], m = -inf, sum = 0.f;
    const bool dense = !p.sigmoid && !p.renorm;
    if (dense) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = lane + kWave * j;
            pr[j] = e < p.E ? __builtin_fmaxf(row[e], -inf) : -inf;
            m = __builtin_fmaxf(m, pr[j]);
        }
        m = wave_max_f32(m);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            pr[j] = m == -inf ? 0.f : m == inf ? (pr[j] == inf ? 1.f : 0.f) : expf(pr[j] - m);
            sum += pr[j];
        }
        sum = wave_sum_f32(sum);
#pragma unroll
        for (int j = 0; j < NJ; ++j) pr[j] = sum > 0.f ? pr[j] / sum : 0.f;
    }
    if (p.renorm) {
        const float top = wave_max_f32(ok ? l : -inf);
        const float base = p.sigmoid ? __builtin_fminf(top, 0.f) : top;
        float s = 0.f;
        if (ok) {
            if (p.sigmoid)
                s = l >= 0.f ? 1.f / (1.f + expf(-l)) : expf(l - base) / (1.f + expf(l));
            else
                s = top == inf ? (l == inf ? 1.f : 0.f) : expf(l - base);
        }
        const float S = wave_sum_f32(s);
        s = S > 0.f ? s / S : 0.f;
        g = s * (u - wave_sum_f32(s * u));
        if (p.sigmoid && ok) g *= 1.f / (1.f + expf(l));
    } else if (p.sigmoid) {
        if (ok) g = u * (1.f / (1.f + expf(-l))) * (1.f / (1.f + expf(l)));
    } else {
        if (ok) g = u * (m == inf ? (l == inf ? 1.f : 0.f) : expf(l - m)) / sum;
        total = wave_sum_f32(g);
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (ok) atomicAdd(mine + id, g);  // (one instruction: lanes of one address in order)
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = lane + kWave * j;
        if (e >= p.E) continue;
        float v = mine[e];
        if (dense) v -= pr[j] * total;
        if (p.add) v += to_f32(static_cast<const T *>(p.add)[t * p.E + e]);
        static_cast<T *>(p.dlogits)[t * p.E + e] = from_f32<T>(v);
    }
}

template <typename T, int NJ> hipError_t backward_t(const ScoreBackwardCall &c, hipStream_t s)
{
    hipLaunchKernelGGL((k_route_scored_backward<T, NJ>), dim3((c.T + kWaves - 1) / kWaves),
                       dim3(kWaves * 64), kWaves * (size_t)c.E * 4, s, c);
    return hipGetLastError();
}
template <int NJ> hipError_t backward_any(const ScoreBackwardCall &c, hipStream_t s)
{
    return c.dtype == 0   ? backward_t<float, NJ>(c, s)
           : c.dtype == 1 ? backward_t<_Float16, NJ>(c, s)
                          : backward_t<__bf16, NJ>(c, s);
}

}  // namespace

hipError_t launch_route_scored(const ScoreCall &c, hipStream_t s)
{
    const dim3 grid((c.T + kWaves - 1) / kWaves), block(kWaves * 64);
    const size_t lds = c.groups > 1 ? kWaves * (size_t)c.E * 8 : 0;
    if (c.E <= 2 * kWave)
        hipLaunchKernelGGL(k_route_scored<2>, grid, block, lds, s, c);
    else if (c.E <= 4 * kWave)
        hipLaunchKernelGGL(k_route_scored<4>, grid, block, lds, s, c);
    else if (c.E <= 8 * kWave)
        hipLaunchKernelGGL(k_route_scored<8>, grid, block, lds, s, c);
    else
        hipLaunchKernelGGL(k_route_scored<16>, grid, block, lds, s, c);
    return hipGetLastError();
}

hipError_t launch_route_scored_backward(const ScoreBackwardCall &c, hipStream_t s)
{
    return c.E <= 2 * kWave   ? backward_any<2>(c, s)
           : c.E <= 4 * kWave ? backward_any<4>(c, s)
           : c.E <= 8 * kWave ? backward_any<8>(c, s)
                              : backward_any<16>(c, s);
}

}  // namespace moe
