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
// A row of logits is read once: G lanes hold it in registers, V consecutive
// columns at a time (V = 4 where rows are whole 16-byte chunks, else 1), so
// both kernels are bound by the traffic of the logits (and of the gradient).
// The forward keeps each lane's columns' sums of p over the rows its group
// takes, adds the groups of a workgroup in order through LDS, and writes one
// partial row per workgroup; a second launch adds those in order (counts are
// integers), so results do not depend on timing. The backward adds the picks'
// term through LDS: each group has a row there, the picks' lanes add to it (one
// instruction, in lane order), and every lane reads its columns back.
//
// Measured, 32,768 tokens, 512 experts, 10 picks: losses 13.7-14.8 us for the rows
// (68 MB, 4.6-5.0 TB/s) and 6.2-6.5 us for the join, which is the latency of a
// second launch, a round of loads and one counter; gradient in fp16 22.4 us (105
// MB, 4.7 TB/s). 64 tokens, 8 experts: 4.3 us, one launch. Rows of the next round
// loaded ahead of this one's arithmetic gained nothing: 16 wavefronts a CU
// already cover the latency.
#include "launch.hpp"
#include "mfma.hpp"

namespace moe {

namespace {

// v of lanes l and l ^ 16 (l ^ 32) in one order for both: the swap of row
// halves between two copies of v
template <int D> __device__ __forceinline__ float2 both_halves(float v)
{
    typedef unsigned u2 __attribute__((ext_vector_type(2)));
    const unsigned x = __float_as_uint(v);
    const u2 r = D == 16 ? __builtin_bit_cast(u2, __builtin_amdgcn_permlane16_swap(x, x, false, false))
                         : __builtin_bit_cast(u2, __builtin_amdgcn_permlane32_swap(x, x, false, false));
    return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// sum (maximum) over the G lanes of a group, in every lane of it, on register
// moves; every lane of the group must be active (groups may differ)
template <int G, typename F> __device__ __forceinline__ float group_reduce(float v, F op)
{
    v = op(v, __int_as_float(dpp_move<kQuadXor1>(__float_as_int(v), 0)));
    v = op(v, __int_as_float(dpp_move<kQuadXor2>(__float_as_int(v), 0)));
    v = op(v, __int_as_float(dpp_move<kRowHalfMirror>(__float_as_int(v), 0)));
    if constexpr (G >= 16) v = op(v, __int_as_float(dpp_move<kRowMirror>(__float_as_int(v), 0)));
    if constexpr (G >= 32) {
        const float2 h = both_halves<16>(v);
        v = op(h.x, h.y);
    }
    if constexpr (G >= 64) {
        const float2 h = both_halves<32>(v);
        v = op(h.x, h.y);
    }
    return v;
}
template <int G> __device__ __forceinline__ float group_sum(float v)
{
    return group_reduce<G>(v, [](float a, float b) { return a + b; });
}
template <int G> __device__ __forceinline__ float group_max(float v)
{
    return group_reduce<G>(v, [](float a, float b) { return fmaxf(a, b); });
}

// the lanes of this lane's group in a wavefront ballot
template <int G> __device__ __forceinline__ uint64_t group_bits(uint64_t b, int lane)
{
    return G == 64 ? b : (b >> (lane & ~(G - 1))) & ((1ull << (G & 63)) - 1);
}

// column of value j of lane `sub` of its group
template <int G, int V> __device__ __forceinline__ int column(int sub, int j)
{
    return (sub + G * (j / V)) * V + j % V;
}

// v[j] = logit of column(j), -inf past E
template <int G, int NJ, int V>
__device__ __forceinline__ void load_row(const float *__restrict__ row, int E, int sub,
                                         float (&v)[NJ])
{
#pragma unroll
    for (int j = 0; j < NJ; j += V) {
        const int e = column<G, V>(sub, j);
        if constexpr (V == 4) {
            const float4_t x = e < E ? *reinterpret_cast<const float4_t *>(row + e)
                                     : float4_t{-__builtin_inff(), -__builtin_inff(),
                                                -__builtin_inff(), -__builtin_inff()};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j + i] = x[i];
        } else {
            v[j] = e < E ? row[e] : -__builtin_inff();
        }
    }
}

// Softmax of a loaded row (NaN and -inf: absent, p = 0): v becomes p; returns the
// log of the sum of exponentials, 0 for a row with no logit at all (p = 0).
// e^x as 2^(x log2 e) in two instructions: the product's rounding is off by
// |x| 2^-24 relative to p, as the rounding of x = l - m itself already is
// (with expf these kernels were bound by arithmetic: its range reduction is
// most of what a row costs).
template <int G, int NJ> __device__ __forceinline__ float softmax_row(float (&v)[NJ])
{
    float m = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        v[j] = __builtin_fmaxf(v[j], -__builtin_inff());  // NaN becomes -inf
        m = __builtin_fmaxf(m, v[j]);
    }
    m = group_max<G>(m);
    const bool none = m == -__builtin_inff();
    const float m0 = none ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        v[j] = __builtin_amdgcn_exp2f((v[j] - m0) * 1.44269504088896341f);
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

// columns of a workgroup of the second launch; 512 experts (the only count compared): 8,
// 16, 32 and 64 columns 9.4, 6.2, 6.0 and 6.9 us (arrivals at one counter wait for one
// another), 32 by 512 threads 6.3
constexpr int kJoinCols = 16;
constexpr int kRowThreads = 1024;  // of a workgroup of the forward's first launch

// the losses from sum over e of c_e times the sum of p_e, entries, sum of lse^2, tokens
__device__ __forceinline__ void write_losses(int E, double term, int64_t entries, double z, int nt,
                                             int32_t *__restrict__ cnt, float *__restrict__ loss)
{
    const double tokens = (double)max(nt, 1);
    cnt[E] = nt;
    cnt[E + 1] = (int)entries;
    loss[0] = (float)(E * term / (tokens * (double)(entries > 0 ? entries : 1)));
    loss[1] = (float)(z / tokens);
}

// ONE: a single workgroup, which writes the results itself (cnt, prob, loss)
template <int G, int NJ, int V, bool ONE>
__global__ __launch_bounds__(kRowThreads) void k_balance_rows(const float *__restrict__ logits,
                                                              const int32_t *__restrict__ ids,
                                                              int T, int E, int K,
                                                              const BalanceScratch w,
                                                              int32_t *__restrict__ cnt,
                                                              float *__restrict__ prob,
                                                              float *__restrict__ loss)
{
    constexpr int GPB = kRowThreads / G;
    __shared__ float s_p[kRowThreads * NJ];  // [GPB][G * NJ]
    __shared__ int s_c[kMaxExperts];
    __shared__ float s_z[GPB];
    __shared__ int s_t[GPB];
    const int tid = threadIdx.x, lane = tid & 63, sub = tid & (G - 1), grp = tid / G;
    if (!ONE && blockIdx.x == 0 && tid == 0) *w.arrived = 0;
    for (int e = tid; e < E; e += kRowThreads) s_c[e] = 0;
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
        float v[NJ];
        load_row<G, NJ, V>(logits + (have ? t : T - 1) * E, E, sub, v);
        bool live = false;
        for (int k = 0; k < K; k += G) {
            const int id = have && k + sub < K ? ids[t * K + k + sub] : -1;
            const bool ok = (unsigned)id < (unsigned)E;
            if (ok) atomicAdd(&s_c[id], 1);
            live |= group_bits<G>(__ballot(ok), lane) != 0;
        }
        const float lse = softmax_row<G, NJ>(v);
        if (live) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[j] += v[j];
            z += lse * lse;
            ++tokens;
        }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) s_p[grp * (G * NJ) + column<G, V>(sub, j)] = acc[j];
    if (sub == 0) {
        s_z[grp] = z;
        s_t[grp] = tokens;
    }
    __syncthreads();
    float a = 0.f;
    int n = 0;
    if (ONE || tid == 0)  // (the same order in every thread)
        for (int q = 0; q < GPB; ++q) {
            a += s_z[q];
            n += s_t[q];
        }
    const float tokens_ = (float)max(n, 1);
    float term = 0.f;  // ONE: of this thread's column (E <= kRowThreads)
    for (int e = tid; e < E; e += kRowThreads) {
        float p = 0.f;
#pragma unroll 8
        for (int q = 0; q < GPB; ++q) p += s_p[q * (G * NJ) + e];
        if constexpr (ONE) {
            prob[e] = p / tokens_;
            cnt[e] = s_c[e];
            term = (float)s_c[e] * p;
        } else {
            w.prob[(int64_t)blockIdx.x * E + e] = p;
            w.cnt[(int64_t)blockIdx.x * E + e] = s_c[e];
        }
    }
    if constexpr (ONE) {
        __syncthreads();
        s_p[tid] = term;
        __syncthreads();
        if (tid < 64) {  // lane l adds the columns l, l + 64, ...
            float s = 0.f;
            int c = 0;
            for (int e = tid; e < E; e += 64) {
                s += s_p[e];
                c += s_c[e];
            }
            s = group_sum<64>(s);
            c = wave_sum(c);
            if (tid == 0) write_losses(E, s, c, a, n, cnt, loss);
        }
    } else if (tid == 0) {
        w.z[blockIdx.x] = a;
        w.tokens[blockIdx.x] = n;
    }
}

// Partial rows added in order: workgroup b takes columns 16 b .. 16 b + 15, 16
// threads each; the workgroup that arrives last adds the workgroups' terms, in
// order, into the losses.
__global__ __launch_bounds__(256) void k_balance_join(int blocks, int E, const BalanceScratch w,
                                                      int32_t *__restrict__ cnt,
                                                      float *__restrict__ prob,
                                                      float *__restrict__ loss)
{
    constexpr int PARTS = 256 / kJoinCols;
    __shared__ float s_p[PARTS][kJoinCols];
    __shared__ int s_c[PARTS][kJoinCols];
    __shared__ double s_z[4];
    __shared__ int s_t[4];
    __shared__ int s_last;
    const int tid = threadIdx.x, col = tid & (kJoinCols - 1), part = tid / kJoinCols;
    const int e = blockIdx.x * kJoinCols + col;
    float p = 0.f;
    int c = 0;
    // (at most 256 rows: 16 a thread, all in flight together; a thread without one reads
    // the last row and adds nothing)
    if (e < E) {
        float q[256 / PARTS];
        int n[256 / PARTS];
#pragma unroll
        for (int i = 0; i < 256 / PARTS; ++i) {
            const int64_t at = (int64_t)min(part + PARTS * i, blocks - 1) * E + e;
            q[i] = w.prob[at];
            n[i] = w.cnt[at];
        }
#pragma unroll
        for (int i = 0; i < 256 / PARTS; ++i)
            if (part + PARTS * i < blocks) {
                p += q[i];
                c += n[i];
            }
    }
    s_p[part][col] = p;
    s_c[part][col] = c;
    // (at most 256 workgroups in the first launch) 64 at a time, then in order
    {
        double z = tid < blocks ? (double)w.z[tid] : 0.;
        int n = tid < blocks ? w.tokens[tid] : 0;
#pragma unroll
        for (int h = 32; h > 0; h >>= 1) {
            z += __shfl_xor(z, h);
            n += __shfl_xor(n, h);
        }
        if ((tid & 63) == 0) {
            s_z[tid >> 6] = z;
            s_t[tid >> 6] = n;
        }
    }
    __syncthreads();
    const int nt = s_t[0] + s_t[1] + s_t[2] + s_t[3];
    const double zsum = s_z[0] + s_z[1] + s_z[2] + s_z[3];
    const float tokens = (float)max(nt, 1);
    if (part == 0) {
        p = 0.f;
        c = 0;
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
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
    if (!s_last) return;
    __threadfence();
    // (at most 64 workgroups here: E <= 1024)
    float *terms = &s_p[0][0];
    int *counts = &s_c[0][0];
    if (tid < (int)gridDim.x) {
        terms[tid] = __hip_atomic_load(w.term + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        counts[tid] = __hip_atomic_load(w.entries + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (tid) return;
    double term = 0.;
    int64_t entries = 0;
    for (unsigned b = 0; b < gridDim.x; ++b) {
        term += terms[b];
        entries += counts[b];
    }
    write_losses(E, term, entries, zsum, nt, cnt, loss);
}

// What a wavefront's lanes did in LDS before stands before what they do after, for
// the compiler too (the hardware keeps one wavefront's LDS operations in order; no
// instruction comes of it)
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int G, int NJ, int V, typename T>
__global__ __launch_bounds__(256) void k_route_backward(
    const float *__restrict__ logits, const int32_t *__restrict__ ids, const float *__restrict__ w,
    const float *__restrict__ dw, const int32_t *__restrict__ cnt, const float *__restrict__ dloss,
    int T_, int E, int K, T *__restrict__ out)
{
    constexpr int GPB = 256 / G, KS = (64 + G - 1) / G;  // picks per lane (K <= 64)
    __shared__ float s_pick[GPB][G * NJ];
    const int tid = threadIdx.x, lane = tid & 63, sub = tid & (G - 1), grp = tid / G;
    float *mine = s_pick[grp];
    const float nt = (float)max(cnt[E], 1), na = (float)max(cnt[E + 1], 1);
    const float gb = dloss ? dloss[0] * (float)E / nt : 0.f;
    const float gz = dloss ? dloss[1] * 2.f / nt : 0.f;
    float f[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = column<G, V>(sub, j);
        f[j] = e < E ? gb * ((float)cnt[e] / na) : 0.f;
    }
    const int stride = (int)gridDim.x * GPB;
    for (int64_t t0 = (int64_t)blockIdx.x * GPB; t0 < T_; t0 += stride) {
        const int64_t t = t0 + grp;
        const bool have = t < T_;
        const int64_t row = have ? t : T_ - 1;
        float v[NJ];
        load_row<G, NJ, V>(logits + row * E, E, sub, v);
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
                float d = 0.f;
                if (k < K) {
                    id[q] = ids[row * K + k];
                    if (dw) {
                        wk[q] = w[row * K + k];
                        d = dw[row * K + k];
                    }
                }
                const bool ok = (unsigned)id[q] < (unsigned)E;
                if (!ok) id[q] = -1;
                wk[q] = ok ? wk[q] : 0.f;
                pw[q] = ok ? wk[q] * d : 0.f;
                live |= group_bits<G>(__ballot(ok), lane) != 0;
                s += pw[q];
            }
        }
        if (dw) {
            s = group_sum<G>(s);
            wave_order();  // (the reads of the row before)
#pragma unroll
            for (int j = 0; j < NJ; ++j) mine[column<G, V>(sub, j)] = 0.f;
            wave_order();
#pragma unroll
            for (int q = 0; q < KS; ++q)
                if (q * G < K && id[q] >= 0) atomicAdd(mine + id[q], pw[q] - wk[q] * s);
        }
        if (dloss && live) {
            const float lse = softmax_row<G, NJ>(v);
            float fp = 0.f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) fp += f[j] * v[j];
            // f holds gb f_e: p (gb f_e + (gz lse - gb sum f p))
            const float c = gz * lse - group_sum<G>(fp);
#pragma unroll
            for (int j = 0; j < NJ; ++j) v[j] *= f[j] + c;
        } else {
#pragma unroll
            for (int j = 0; j < NJ; ++j) v[j] = 0.f;
        }
        if (dw) {
            wave_order();
#pragma unroll
            for (int j = 0; j < NJ; ++j) v[j] += mine[column<G, V>(sub, j)];
        }
        if (have)
#pragma unroll
            for (int j = 0; j < NJ; j += V) {
                const int e = column<G, V>(sub, j);
                if (e < E) {
                    if constexpr (V == 4) {
                        const float x[4] = {v[j], v[j + 1], v[j + 2], v[j + 3]};
                        Vec<T, 4>::store(out + row * E + e, x);
                    } else {
                        out[row * E + e] = from_f32<T>(v[j]);
                    }
                }
            }
    }
}

// Lanes per row G, values per lane NJ and columns together V for E columns.
// vec: rows are whole 16-byte chunks. (4 columns a lane also for the smallest
// E: a few idle lanes cost nothing there.)
template <int G, int NJ, int V> struct Width {
    static constexpr int g = G, nj = NJ, v = V;
};
template <typename F> hipError_t by_width(int E, bool vec, F run)
{
    if (vec) {
        if (E <= 32) return run(Width<8, 4, 4>());
        if (E <= 64) return run(Width<16, 4, 4>());
        if (E <= 128) return run(Width<32, 4, 4>());
        if (E <= 256) return run(Width<64, 4, 4>());
        if (E <= 512) return run(Width<64, 8, 4>());
        return run(Width<64, 16, 4>());
    }
    if (E <= 8) return run(Width<8, 1, 1>());
    if (E <= 16) return run(Width<16, 1, 1>());
    if (E <= 32) return run(Width<16, 2, 1>());
    if (E <= 64) return run(Width<16, 4, 1>());
    if (E <= 128) return run(Width<32, 4, 1>());
    if (E <= 256) return run(Width<64, 4, 1>());
    if (E <= 512) return run(Width<64, 8, 1>());
    return run(Width<64, 16, 1>());
}

bool whole_rows(const void *p, int E, int es)
{
    return E % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * es) == 0;
}

// rows of logits that a workgroup of the forward's first launch takes at a time, as
// by_width groups its lanes
int rows_at_once(int E, bool vec)
{
    const int lanes = E <= (vec ? 32 : 8) ? 8 : E <= 64 ? 16 : E <= 128 ? 32 : 64;
    return kRowThreads / lanes;
}

// Workgroups of the forward's first launch: at most 256 (one per CU), each with a
// row in its first round; one, and no second launch, for batches that one workgroup
// takes in 4 rounds (64 tokens, 8 experts: 4 us in one launch, 9 in two; 8 rounds of
// 9 to 32 experts whose rows are not whole 16-byte chunks).
int balance_blocks(int T, int E, bool vec)
{
    if (T <= 4 * rows_at_once(E, true)) return 1;
    const int rows = rows_at_once(E, vec);
    const int64_t b = ((int64_t)T + rows - 1) / rows;
    return (int)(b < 256 ? b : 256);
}

size_t place_scratch(int blocks, int E, char *p, BalanceScratch *w)
{
    const size_t join = (E + kJoinCols - 1) / kJoinCols;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char *q = p + at;
        at += (bytes + 255) / 256 * 256;
        return q;
    };
    w->prob = reinterpret_cast<float *>(take((size_t)blocks * E * 4));
    w->cnt = reinterpret_cast<int *>(take((size_t)blocks * E * 4));
    w->z = reinterpret_cast<float *>(take((size_t)blocks * 4));
    w->tokens = reinterpret_cast<int *>(take((size_t)blocks * 4));
    w->term = reinterpret_cast<float *>(take(join * 4));
    w->entries = reinterpret_cast<int *>(take(join * 4));
    w->arrived = reinterpret_cast<int *>(take(4));
    return at;
}

}  // namespace

int64_t balance_workspace(int T, int E)
{
    // (for any address of the logits: the form with the fewer rows at once)
    BalanceScratch w;
    return (int64_t)place_scratch(balance_blocks(T, E, false), E, nullptr, &w);
}

hipError_t launch_balance_loss(const float *logits, const int32_t *ids, int T, int E, int K,
                               int32_t *cnt, float *prob, float *loss, void *ws, hipStream_t s)
{
    const bool vec = whole_rows(logits, E, 4);
    const int blocks = balance_blocks(T, E, vec);
    BalanceScratch w;
    place_scratch(blocks, E, static_cast<char *>(ws), &w);
    const hipError_t rc = by_width(E, vec, [&](auto z) {
        typedef decltype(z) Z;
        auto rows = blocks == 1 ? k_balance_rows<Z::g, Z::nj, Z::v, true>
                                : k_balance_rows<Z::g, Z::nj, Z::v, false>;
        hipLaunchKernelGGL(rows, dim3(blocks), dim3(kRowThreads), 0, s, logits, ids, T, E, K, w,
                           cnt, prob, loss);
        return hipGetLastError();
    });
    if (rc != hipSuccess || blocks == 1) return rc;
    hipLaunchKernelGGL(k_balance_join, dim3((E + kJoinCols - 1) / kJoinCols), dim3(256), 0, s,
                       blocks, E, w, cnt, prob, loss);
    return hipGetLastError();
}

template <typename T>
static hipError_t route_backward_t(const float *logits, const int32_t *ids, const float *w,
                                   const float *dw, const int32_t *cnt, const float *dloss, int T_,
                                   int E, int K, T *out, hipStream_t s)
{
    const bool vec = whole_rows(logits, E, 4) && whole_rows(out, E, sizeof(T));
    return by_width(E, vec, [&](auto z) {
        typedef decltype(z) Z;
        const int64_t b = ((int64_t)T_ + 256 / Z::g - 1) / (256 / Z::g);
        hipLaunchKernelGGL((k_route_backward<Z::g, Z::nj, Z::v, T>),
                           dim3((unsigned)(b < 2048 ? b : 2048)), dim3(256), 0, s, logits, ids, w,
                           dw, cnt, dloss, T_, E, K, out);
        return hipGetLastError();
    });
}

hipError_t launch_route_backward(const float *logits, const int32_t *ids, const float *w,
                                 const float *dw, const int32_t *cnt, const float *dloss, int T,
                                 int E, int K, void *dlogits, int dtype, hipStream_t s)
{
    if (dtype == 0)
        return route_backward_t(logits, ids, w, dw, cnt, dloss, T, E, K,
                                static_cast<float *>(dlogits), s);
    if (dtype == 1)
        return route_backward_t(logits, ids, w, dw, cnt, dloss, T, E, K,
                                static_cast<_Float16 *>(dlogits), s);
    return route_backward_t(logits, ids, w, dw, cnt, dloss, T, E, K,
                            static_cast<__bf16 *>(dlogits), s);
}

}  // namespace moe
