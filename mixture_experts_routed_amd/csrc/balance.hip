// Router losses of gfx950 and the gradient of the router logits.
//
// With p_te the softmax of token t's logits, c_e the entries routed to expert
// e, n_t the tokens with at least one valid id and n_a = sum c_e:
//   balance = E sum_e (c_e / n_a) P_e,  P_e = (1 / n_t) sum_t p_te
//   z       = (1 / n_t) sum_t lse_t^2,  lse_t = log sum_e exp(logit_te)
// (sums over the n_t tokens). Their gradient and that of the renormalised
// top-k weights w_k = exp(l_k) / sum over the picks, for upstream gradients
// gb, gz and dw:
//   dl_te = p_te (gb E / n_t (f_e - sum_j f_j p_tj) + 2 gz / n_t lse_t)
//           + sum over the picks k of e: w_k (dw_k - sum_j w_j dw_j),  f = c / n_a
// c_e counts entries and has no gradient.
//
// A row of logits is read once: G lanes hold it in registers (lane s columns s
// + G j), so both kernels are bound by the traffic of the logits (and of the
// gradient). The forward keeps each lane's columns' sums of p over the rows
// its group takes, adds the groups of a workgroup in order through LDS, and
// writes one partial row per workgroup; a second launch adds those in order
// (counts are integers), so results do not depend on timing.
#include <type_traits>

#include "launch.hpp"
#include "mfma.hpp"

namespace moe {

namespace {

template <int G> __device__ __forceinline__ float group_sum(float v)
{
    v += __int_as_float(dpp_move<kQuadXor1>(__float_as_int(v), 0));
    v += __int_as_float(dpp_move<kQuadXor2>(__float_as_int(v), 0));
    v += __int_as_float(dpp_move<kRowHalfMirror>(__float_as_int(v), 0));
    if (G >= 16) v += __int_as_float(dpp_move<kRowMirror>(__float_as_int(v), 0));
    if (G >= 32) v += __shfl_xor(v, 16);
    if (G >= 64) v += __shfl_xor(v, 32);
    return v;
}

template <int G> __device__ __forceinline__ float group_max(float v)
{
    v = fmaxf(v, __int_as_float(dpp_move<kQuadXor1>(__float_as_int(v), 0)));
    v = fmaxf(v, __int_as_float(dpp_move<kQuadXor2>(__float_as_int(v), 0)));
    v = fmaxf(v, __int_as_float(dpp_move<kRowHalfMirror>(__float_as_int(v), 0)));
    if (G >= 16) v = fmaxf(v, __int_as_float(dpp_move<kRowMirror>(__float_as_int(v), 0)));
    if (G >= 32) v = fmaxf(v, __shfl_xor(v, 16));
    if (G >= 64) v = fmaxf(v, __shfl_xor(v, 32));
    return v;
}

// the lanes of this lane's group in a wavefront ballot
template <int G> __device__ __forceinline__ uint64_t group_bits(uint64_t b, int lane)
{
    return G == 64 ? b : (b >> (lane & ~(G - 1))) & ((1ull << (G & 63)) - 1);
}

// Softmax of one row: v[j] = logit of column sub + G j (NaN and -inf: absent,
// p = 0) becomes p; returns the log of the sum of exponentials, 0 for a row
// with no logit at all (its p are all 0).
template <int G, int NJ>
__device__ __forceinline__ float softmax_row(const float *__restrict__ row, int E, int sub,
                                             float (&v)[NJ])
{
    float m = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = sub + G * j;
        v[j] = e < E ? row[e] : -__builtin_inff();
        if (__builtin_isnan(v[j])) v[j] = -__builtin_inff();
        m = fmaxf(m, v[j]);
    }
    m = group_max<G>(m);
    const bool none = m == -__builtin_inff();
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        v[j] = none ? 0.f : expf(v[j] - m);
        s += v[j];
    }
    s = group_sum<G>(s);
    const float inv = none ? 0.f : 1.f / s;
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] *= inv;
    return none ? 0.f : m + logf(s);
}

// Scratch of the forward pass: per workgroup a row of probability sums, a row
// of counts, the sum of lse^2 and the valid tokens.
struct BalanceScratch {
    float *prob;    // [blocks][E]
    int *cnt;       // [blocks][E]
    float *z;       // [blocks]
    int *tokens;    // [blocks]
    float *term;    // [join workgroups]: sum of c_e * (sum of p_e)
    int *entries;   // [join workgroups]: sum of c_e
    int *arrived;   // join workgroups done; cleared by the first launch
};

constexpr int kJoinCols = 32;

template <int G, int NJ>
__global__ __launch_bounds__(256) void k_balance_rows(const float *__restrict__ logits,
                                                      const int32_t *__restrict__ ids, int T, int E,
                                                      int K, const BalanceScratch w)
{
    constexpr int GPB = 256 / G;
    __shared__ float s_p[256 * NJ];  // [GPB][G * NJ]
    __shared__ int s_c[kMaxExperts];
    __shared__ float s_z[GPB];
    __shared__ int s_t[GPB];
    const int tid = threadIdx.x, lane = tid & 63, sub = tid & (G - 1), grp = tid / G;
    if (blockIdx.x == 0 && tid == 0) *w.arrived = 0;
    for (int e = tid; e < E; e += 256) s_c[e] = 0;
    __syncthreads();
    float acc[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] = 0.f;
    float z = 0.f;
    int tokens = 0;
    const int stride = (int)gridDim.x * GPB;
    // every lane of a wavefront makes the same number of rounds (the group
    // reductions need all of them)
    for (int64_t t0 = (int64_t)blockIdx.x * GPB; t0 < T; t0 += stride) {
        const int64_t t = t0 + grp;
        const bool have = t < T;
        const int64_t row = have ? t : T - 1;
        bool live = false;
        for (int k = 0; k < K; k += G) {
            const int id = have && k + sub < K ? ids[row * K + k + sub] : -1;
            const bool ok = (unsigned)id < (unsigned)E;
            if (ok) atomicAdd(&s_c[id], 1);
            live |= group_bits<G>(__ballot(ok), lane) != 0;
        }
        float v[NJ];
        const float lse = softmax_row<G, NJ>(logits + row * E, E, sub, v);
        if (live) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[j] += v[j];
            z += lse * lse;
            ++tokens;
        }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) s_p[grp * (G * NJ) + sub + G * j] = acc[j];
    if (sub == 0) {
        s_z[grp] = z;
        s_t[grp] = tokens;
    }
    __syncthreads();
    for (int e = tid; e < E; e += 256) {
        float p = 0.f;
#pragma unroll
        for (int q = 0; q < GPB; ++q) p += s_p[q * (G * NJ) + e];
        w.prob[(int64_t)blockIdx.x * E + e] = p;
        w.cnt[(int64_t)blockIdx.x * E + e] = s_c[e];
    }
    if (tid == 0) {
        float a = 0.f;
        int n = 0;
        for (int q = 0; q < GPB; ++q) {
            a += s_z[q];
            n += s_t[q];
        }
        w.z[blockIdx.x] = a;
        w.tokens[blockIdx.x] = n;
    }
}

// Partial rows added in order: workgroup b takes columns 32 b .. 32 b + 31, 8
// threads each; the workgroup that arrives last adds the workgroups' terms, in
// order, into the losses.
__global__ __launch_bounds__(256) void k_balance_join(int blocks, int E, const BalanceScratch w,
                                                      int32_t *__restrict__ cnt,
                                                      float *__restrict__ prob,
                                                      float *__restrict__ loss)
{
    __shared__ float s_p[8][kJoinCols];
    __shared__ int s_c[8][kJoinCols];
    __shared__ double s_z[256];
    __shared__ int s_t[256];
    __shared__ int s_last;
    const int tid = threadIdx.x, col = tid & (kJoinCols - 1), part = tid / kJoinCols;
    const int e = blockIdx.x * kJoinCols + col;
    float p = 0.f;
    int c = 0;
    if (e < E)
        for (int b = part; b < blocks; b += 8) {
            p += w.prob[(int64_t)b * E + e];
            c += w.cnt[(int64_t)b * E + e];
        }
    s_p[part][col] = p;
    s_c[part][col] = c;
    double z = 0.;
    int nt = 0;
    for (int b = tid; b < blocks; b += 256) {
        z += w.z[b];
        nt += w.tokens[b];
    }
    s_z[tid] = z;
    s_t[tid] = nt;
    for (int h = 128; h > 0; h >>= 1) {
        __syncthreads();
        if (tid < h) {
            s_z[tid] += s_z[tid + h];
            s_t[tid] += s_t[tid + h];
        }
    }
    __syncthreads();
    nt = s_t[0];
    const float tokens = (float)max(nt, 1);
    if (part == 0) {
        p = 0.f;
        c = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            p += s_p[q][col];
            c += s_c[q][col];
        }
        if (e < E) {
            prob[e] = p / tokens;
            cnt[e] = c;
        }
        s_p[0][col] = (float)c * p;
        s_c[0][col] = c;
    }
    __syncthreads();
    if (tid == 0) {
        float term = 0.f;
        int entries = 0;
        for (int q = 0; q < kJoinCols; ++q) {
            term += s_p[0][q];
            entries += s_c[0][q];
        }
        w.term[blockIdx.x] = term;
        w.entries[blockIdx.x] = entries;
        __threadfence();
        s_last = atomicAdd(w.arrived, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last || tid) return;
    __threadfence();
    double term = 0.;
    int64_t entries = 0;
    for (unsigned b = 0; b < gridDim.x; ++b) {
        term += __hip_atomic_load(w.term + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        entries += __hip_atomic_load(w.entries + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    cnt[E] = nt;
    cnt[E + 1] = (int)entries;
    loss[0] = (float)(E * term / ((double)tokens * (double)(entries > 0 ? entries : 1)));
    loss[1] = (float)(s_z[0] / (double)tokens);
}

template <int G, int NJ, typename T>
__global__ __launch_bounds__(256) void k_route_backward(
    const float *__restrict__ logits, const int32_t *__restrict__ ids, const float *__restrict__ w,
    const float *__restrict__ dw, const int32_t *__restrict__ cnt, const float *__restrict__ dloss,
    int T_, int E, int K, T *__restrict__ out)
{
    constexpr int GPB = 256 / G, KS = (64 + G - 1) / G;  // picks per lane (K <= 64)
    const int tid = threadIdx.x, lane = tid & 63, sub = tid & (G - 1), grp = tid / G;
    const float nt = (float)max(cnt[E], 1), na = (float)max(cnt[E + 1], 1);
    const float gb = dloss ? dloss[0] * (float)E / nt : 0.f;
    const float gz = dloss ? dloss[1] * 2.f / nt : 0.f;
    float f[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) f[j] = sub + G * j < E ? (float)cnt[sub + G * j] / na : 0.f;
    const int stride = (int)gridDim.x * GPB;
    for (int64_t t0 = (int64_t)blockIdx.x * GPB; t0 < T_; t0 += stride) {
        const int64_t t = t0 + grp;
        const bool have = t < T_;
        const int64_t row = have ? t : T_ - 1;
        int id[KS];
        float wk[KS], pw[KS];
        bool live = false;
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < KS; ++q) {
            id[q] = -1;
            wk[q] = pw[q] = 0.f;
            if (q * G < K) {
                const int k = q * G + sub;
                if (k < K) id[q] = ids[row * K + k];
                const bool ok = (unsigned)id[q] < (unsigned)E;
                if (!ok) id[q] = -1;
                if (ok && dw) {
                    wk[q] = w[row * K + k];
                    pw[q] = wk[q] * dw[row * K + k];
                }
                live |= group_bits<G>(__ballot(ok), lane) != 0;
                s += pw[q];
            }
        }
        s = group_sum<G>(s);
        float v[NJ];
        const float lse = softmax_row<G, NJ>(logits + row * E, E, sub, v);
        float fp = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) fp += f[j] * v[j];
        fp = group_sum<G>(fp);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            v[j] = live && dloss ? v[j] * (gb * (f[j] - fp) + gz * lse) : 0.f;
        if (dw) {
#pragma unroll
            for (int q = 0; q < KS; ++q)
                if (q * G < K) {
                    const float pick = pw[q] - wk[q] * s;
                    for (int k = 0; k < min(G, K - q * G); ++k) {
                        const int e = __shfl(id[q], k, G);
                        const float add = __shfl(pick, k, G);
#pragma unroll
                        for (int j = 0; j < NJ; ++j)
                            if (e == sub + G * j) v[j] += add;
                    }
                }
        }
        if (have)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                if (sub + G * j < E) out[row * E + sub + G * j] = from_f32<T>(v[j]);
    }
}

// lanes per row and columns per lane for E columns
template <typename F> hipError_t by_width(int E, F run)
{
    if (E <= 8) return run(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
    if (E <= 16) return run(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
    if (E <= 32) return run(std::integral_constant<int, 16>(), std::integral_constant<int, 2>());
    if (E <= 64) return run(std::integral_constant<int, 16>(), std::integral_constant<int, 4>());
    if (E <= 128) return run(std::integral_constant<int, 32>(), std::integral_constant<int, 4>());
    if (E <= 256) return run(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
    if (E <= 512) return run(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
    return run(std::integral_constant<int, 64>(), std::integral_constant<int, 16>());
}

int group_of(int E)
{
    return E <= 8 ? 8 : E <= 64 ? 16 : E <= 128 ? 32 : 64;
}

constexpr int kBalanceBlocks = 512;

int balance_blocks(int T, int E)
{
    const int per = 256 / group_of(E);
    const int64_t b = ((int64_t)T + per - 1) / per;
    return (int)(b < kBalanceBlocks ? b : kBalanceBlocks);
}

size_t place_scratch(int T, int E, char *p, BalanceScratch *w)
{
    const size_t blocks = balance_blocks(T, E), join = (E + kJoinCols - 1) / kJoinCols;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *q = p + at;
        at += (bytes + 255) / 256 * 256;
        return q;
    };
    w->prob = reinterpret_cast<float *>(take(blocks * E * 4));
    w->cnt = reinterpret_cast<int *>(take(blocks * E * 4));
    w->z = reinterpret_cast<float *>(take(blocks * 4));
    w->tokens = reinterpret_cast<int *>(take(blocks * 4));
    w->term = reinterpret_cast<float *>(take(join * 4));
    w->entries = reinterpret_cast<int *>(take(join * 4));
    w->arrived = reinterpret_cast<int *>(take(4));
    return at;
}

}  // namespace

int64_t balance_workspace(int T, int E)
{
    BalanceScratch w;
    return (int64_t)place_scratch(T, E, nullptr, &w);
}

hipError_t launch_balance_loss(const float *logits, const int32_t *ids, int T, int E, int K,
                               int32_t *cnt, float *prob, float *loss, void *ws, hipStream_t s)
{
    BalanceScratch w;
    place_scratch(T, E, static_cast<char *>(ws), &w);
    const int blocks = balance_blocks(T, E);
    const hipError_t rc = by_width(E, [&](auto g, auto nj) {
        hipLaunchKernelGGL((k_balance_rows<decltype(g)::value, decltype(nj)::value>), dim3(blocks),
                           dim3(256), 0, s, logits, ids, T, E, K, w);
        return hipGetLastError();
    });
    if (rc != hipSuccess) return rc;
    hipLaunchKernelGGL(k_balance_join, dim3((E + kJoinCols - 1) / kJoinCols), dim3(256), 0, s,
                       blocks, E, w, cnt, prob, loss);
    return hipGetLastError();
}

hipError_t launch_route_backward(const float *logits, const int32_t *ids, const float *w,
                                 const float *dw, const int32_t *cnt, const float *dloss, int T,
                                 int E, int K, void *dlogits, int dtype, hipStream_t s)
{
    return by_width(E, [&](auto g, auto nj) {
        constexpr int G = decltype(g)::value, NJ = decltype(nj)::value;
        const int64_t b = ((int64_t)T + 256 / G - 1) / (256 / G);
        const dim3 grid((unsigned)(b < 4096 ? b : 4096)), block(256);
        if (dtype == 0)
            hipLaunchKernelGGL((k_route_backward<G, NJ, float>), grid, block, 0, s, logits, ids, w,
                               dw, cnt, dloss, T, E, K, static_cast<float *>(dlogits));
        else if (dtype == 1)
            hipLaunchKernelGGL((k_route_backward<G, NJ, _Float16>), grid, block, 0, s, logits, ids,
                               w, dw, cnt, dloss, T, E, K, static_cast<_Float16 *>(dlogits));
        else
            hipLaunchKernelGGL((k_route_backward<G, NJ, __bf16>), grid, block, 0, s, logits, ids, w,
                               dw, cnt, dloss, T, E, K, static_cast<__bf16 *>(dlogits));
        return hipGetLastError();
    });
}

}  // namespace moe
