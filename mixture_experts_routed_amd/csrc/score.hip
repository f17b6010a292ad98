// Routing by scores for gfx950, and the gradient of the logits.
//   s_e = softmax or sigmoid of the logits,  c_e = s_e + bias_e
//   groups of E / G experts: worth = sum of the group_top largest c; `keep` stay
//   the K largest c of those, ties to the lower index; w = scale s (/ sum of s)
//
// Choices are those of 64-bit arithmetic, made in 32 bits where those tell: L lanes hold a
// row of logits, each with 4 consecutive columns at a time where rows are whole 16-byte
// chunks.
//  * The K-th largest of the lanes' own maxima bounds the K-th largest c from below.
//    What reaches the bound, less what 32 bits may be off, are the candidates, one a lane,
//    through LDS.
//  * A candidate's place is the number of candidates before it, so ordering them takes
//    one compare each, not K rounds over the row.
//  * What lies within the errors of its 32-bit values is too near to call: groups are
//    chosen again from 64-bit scores, a sigmoid's candidates placed again by theirs,
//    one a lane (2 rows of 1,000 at 512 experts). Rows where a softmax's biased scores
//    lie so near, and those with more candidates than lanes, are taken again as a whole
//    in 64 bits, one row a wavefront, a round per pick (exact_row). Without a bias experts
//    are compared by their logits, which are exact.
//
// Candidates stay few while K is at most half of the lanes: 11.6 for 10 picks of 512 experts
// (32 lanes), 10.3 for 8 of 128 (16 lanes). As K nears the number of lanes with columns (32
// experts have 8), the least of their maxima count and the bound falls; where open columns
// lie in fewer than K lanes (one group of 32 columns: 8 lanes) there is none. Shares of rows
// of normal logits that exact_row takes (a model of the bound), and the time of 32,768 such
// rows without a bias: 128 experts, 8 picks 0.6%, 23 us; 10 picks 16%, 63 us; 12 picks 75%,
// 120 us; 256 experts, 10 picks 20%, 80 us; 16 picks all, 181 us; 512 experts, 32 picks all,
// 389 us; 1,024 experts, 64 picks all, 1,594 us. Equal logits in more columns than lanes
// do the same: 96 us for 128 experts, 8 picks, 165 for 512, 10 picks. moe_route_topk, K rounds
// a row whatever the logits, takes 34, 42, 49, 49, 75, 192, 564, 34 and 66 us there.
//
// Bound by vector arithmetic, and the gradient by HBM. Measured at 32,768 tokens, 512
// experts, 10 picks: sigmoid scores with a bias, 4 of 8 groups by their two best, 41 us a
// call in a row of calls (46 on another GPU; a kernel trace from an idle one has 44 at least,
// 45 on average; 1,155 vector instructions a wavefront of two rows are 30 us of it; the 70 MB
// would copy in 14); gradient of softmax scores, onto an fp16 output with another added, 28 us
// (137 MB, 4.9 TB/s). 4 tokens, 128 experts: 3.8 us.
// What the steps were worth: a round over the row a pick, 158 us; candidates by the bound,
// ordered by counting, 91; groups and sigmoids settled within the row's lanes, not the
// whole row again, 44; the gradient's rows in registers, 60 -> 28.
#include "lanes.hpp"
#include "launch.hpp"
#include "mfma.hpp"

#include <type_traits>

namespace moe {

namespace {

constexpr int kWaves = 4;  // wavefronts of a workgroup
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kUlp = 5.9604644775390625e-8f;  // 2^-24
__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// LDS written by lanes of this wavefront is read by others of it
__device__ __forceinline__ void wave_lds_order()
{
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ double wave_sum_f64(double v)
{
#pragma unroll
    for (int h = 32; h > 0; h >>= 1) v += __shfl_xor(v, h);
    return v;
}

// A score up to a factor that all of a row's picks share, for their ratios: softmax
// exp(l - top); sigmoid times exp(-min(top, 0)), so that scores too small for the type
// still add up. top: the largest of the picks' logits.
__device__ __forceinline__ float ratio_score(bool sigmoid, float l, float top)
{
    if (sigmoid)
        return l >= 0.f ? 1.f / (1.f + expf(-l))
                        : expf(l - __builtin_fminf(top, 0.f)) / (1.f + expf(l));
    // (+inf logits share everything)
    return top == __builtin_inff() ? (l == top ? 1.f : 0.f) : expf(l - top);
}

// Row t in 64 bits, by the whole wavefront: lane l holds experts l, l + 64, ...;
// lds: E doubles of this wavefront (with groups).
template <int NJ>
__device__ __noinline__ void exact_row(const ScoreCall &p, int64_t t, double *lds)
{
    const int lane = threadIdx.x & 63;
    const float *row = p.logits + t * p.E;
    const double inf = __builtin_inf();
    double s[NJ], c[NJ];
    float l[NJ], m = neg_inf();
    uint32_t there = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int e = lane + kWave * j;
        l[j] = e < p.E ? row[e] : neg_inf();
        if (l[j] > neg_inf()) {  // not NaN
            there |= 1u << j;
            m = __builtin_fmaxf(m, l[j]);
        }
    }
    if (p.sigmoid) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[j] = (there >> j & 1) ? 1.0 / (1.0 + exp(-(double)l[j])) : 0.0;
    } else {
        m = group_max<64>(m);
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
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
            if (!(b > neg_inf())) there &= ~(1u << j);
            c[j] += (double)b;
        }
    }
    if (p.groups > 1) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int e = lane + kWave * j;
            if (e < p.E) lds[e] = (there >> j & 1) ? c[j] : -inf;
        }
        wave_lds_order();
        const int n = p.E / p.groups;
        double worth = -inf, next = -inf;
        if (lane < p.groups)
            for (int i = 0; i < n; ++i) {
                const double v = lds[lane * n + i];
                if (v > worth) {
                    next = worth;
                    worth = v;
                } else if (v > next) {
                    next = v;
                }
            }
        wave_lds_order();
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
    if (!p.bias) {  // by the logits
#pragma unroll
        for (int j = 0; j < NJ; ++j) c[j] = (double)l[j];
    }
    double my_s = 0.0;
    float my_l = 0.f, top = 0.f;
    int my_id = -1;
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
        top = k == 0 ? q : __builtin_fmaxf(top, q);
    }
    double total = 1.0;
    if (p.renorm) {
        my_s = my_id >= 0 ? (double)ratio_score(p.sigmoid, my_l, top) : 0.0;
        total = wave_sum_f64(my_s);
    }
    if (lane < p.K) {
        p.ids[t * p.K + lane] = my_id;
        p.w[t * p.K + lane] = my_id >= 0 ? (float)((double)p.scale * (my_s / total)) : 0.f;
    }
}

struct Candidate {
    float key;
    int col;
};

// LDS of a wavefront: the scores of its rows (R rows of at most 16 L columns: 4 KB in
// 32 bits, 8 in 64), later its candidates (64) and their scores in 64 bits behind 4 KB
constexpr int kLdsBytes = 8192;

// an image of a float (not NaN) that orders as it does among whole numbers, and back
__device__ __forceinline__ int order_of(float v)
{
    const int b = __float_as_int(v);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int k)
{
    return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}
template <int L> __device__ __forceinline__ int lanes_max(int v)
{
    constexpr int lo = -2147483647 - 1;  // (the identity: moves fold into the maxima)
    v = max(v, dpp_move<kQuadXor1>(v, lo));
    v = max(v, dpp_move<kQuadXor2>(v, lo));
    v = max(v, dpp_move<kRowHalfMirror>(v, lo));
    v = max(v, dpp_move<kRowMirror>(v, lo));
    if constexpr (L >= 32) {
        const float2 h = both_halves<16>(__int_as_float(v));
        v = max(__float_as_int(h.x), __float_as_int(h.y));
    }
    if constexpr (L >= 64) {
        const float2 h = both_halves<32>(__int_as_float(v));
        v = max(__float_as_int(h.x), __float_as_int(h.y));
    }
    return v;
}

// The groups that stay, of the c in LDS (s: this row's E values; groups <= L, one
// wavefront's lanes): bit g P of the result for group g, with P lanes a group. near (in
// 32 bits): whether the least worth that stays and the best that does not are too near
// to call when each c is off by tol and a rounding of itself.
template <int L, typename F>
__device__ __forceinline__ uint64_t choose_groups(const ScoreCall &p, const F *s, int P, float tol,
                                                  bool *near)
{
    const int lane = threadIdx.x & 63, sub = lane & (L - 1);
    const int n = p.E / p.groups, g0 = sub / P;
    const F inf = (F)__builtin_inf();
    F worth = -inf, next = -inf;
    if (g0 < p.groups) {
        const F *q = s + g0 * n;
#pragma unroll 4
        for (int i = sub & (P - 1); i < n; i += P) {  // the two largest
            const F v = q[i];
            if constexpr (sizeof(F) == 4) {  // (the median of the three is the second largest)
                next = __builtin_amdgcn_fmed3f(worth, next, v);
            } else {
                const F less = v > worth ? worth : v;
                next = less > next ? less : next;
            }
            worth = v > worth ? v : worth;
        }
    }
    for (int h = 1; h < P; h <<= 1) {
        const F oa = __shfl_xor(worth, h), oc = __shfl_xor(next, h);
        const F less = oa > worth ? worth : oa;
        next = oc > next ? oc : next;
        next = less > next ? less : next;
        worth = oa > worth ? oa : worth;
    }
    const F size = worth > -inf ? __builtin_fabs(worth) + (next > -inf ? __builtin_fabs(next) : 0) : 0;
    if (p.group_top > 1 && next > -inf) worth += next;
    int before = 0;
    for (int g = 0; g < p.groups; ++g) {
        const F o = __shfl(worth, (lane & ~(L - 1)) + g * P);
        before += o > worth || (o == worth && g < g0);
    }
    const bool in = g0 < p.groups, stay = in && before < p.keep;
    if constexpr (sizeof(F) == 4) {
        const float low = -group_max<L>(stay ? -worth : -inf);
        const float high = group_max<L>(in && !stay ? worth : -inf);
        // (high -inf: no group is left out, or absent ones)
        *near = high > -inf && !(low - high > 4.f * tol + 4.f * kUlp * group_max<L>(size));
    }
    return group_bits<L>(__ballot(stay), lane);
}

// c of a row in 64 bits into s, by the row's L lanes
template <int L>
__device__ __forceinline__ void exact_scores(const ScoreCall &p, const float *row, float m,
                                             double *s)
{
    const int sub = threadIdx.x & (L - 1);
    double sum = 1.;
    auto softmax = [&](float l) {
        return !(l > neg_inf())         ? 0.
               : m == __builtin_inff() ? (l == m ? 1. : 0.)
                                       : exp((double)l - (double)m);
    };
    if (!p.sigmoid) {
        sum = 0.;
        for (int e = sub; e < p.E; e += L) sum += softmax(row[e]);
#pragma unroll
        for (int h = 1; h < L; h <<= 1) sum += __shfl_xor(sum, h);
    }
    for (int e = sub; e < p.E; e += L) {
        const float l = row[e], b = p.bias ? p.bias[e] : 0.f;
        const double c = p.sigmoid ? 1. / (1. + exp(-(double)l)) : softmax(l) / sum;
        s[e] = l > neg_inf() && b > neg_inf() ? c + (double)b : -__builtin_inf();
    }
}

template <int L, int NJ, int V>
__global__ __launch_bounds__(kWaves * 64) void k_route_scored(const ScoreCall p, uint32_t magic)
{
    constexpr int R = 64 / L;
    static_assert(R * L * NJ * 8 <= kLdsBytes && 4096 + 64 * (sizeof(Candidate) + 8) <= kLdsBytes,
                  "LDS");
    __shared__ double s_all[kWaves][kLdsBytes / 8];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane / L, sub = lane & (L - 1);
    double *lds = s_all[wave];
    float *s_c = reinterpret_cast<float *>(lds) + r * (L * NJ);
    Candidate *cand = reinterpret_cast<Candidate *>(lds + 512) + r * L;
    const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * R;
    if (t0 >= p.T) return;  // (the whole wavefront)
    const bool have = t0 + r < p.T;
    const int64_t t = have ? t0 + r : p.T - 1;
    const float inf = __builtin_inff();

    // Absent: -inf. A NaN logit becomes it here, before anything is compared (its image
    // among whole numbers would lie above every score's); a NaN bias fails b > -inf.
    float l[NJ], b[NJ], key[NJ];
    load_row<L, NJ, V>(p.logits + t * p.E, p.E, sub, l);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        l[j] = __builtin_fmaxf(l[j], -inf);
        b[j] = 0.f;
    }
    if (p.bias) load_row<L, NJ, V>(p.bias, p.E, sub, b);
    // largest logit, and the softmax's denominator where it counts
    float m = -inf, sum = 1.f, tol = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) m = __builtin_fmaxf(m, l[j]);
    m = group_max<L>(m);
    const bool scored = p.bias || p.groups > 1;  // every expert's score is needed
    if (!p.sigmoid && (scored || !p.renorm)) {
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float x = m == inf       ? (l[j] == inf ? 1.f : 0.f)
                            : l[j] > -inf ? __builtin_amdgcn_exp2f((l[j] - m) * kLog2e)
                                          : 0.f;
            key[j] = x;
            sum += x;
        }
        sum = group_sum<L>(sum);
    }
    if (scored) {
        // s in 32 bits. How far it may be off, with smax the row's largest score:
        // sigmoid, the argument's rounding and four of an ulp or less, relative
        // (1 - s) (1.5 |l| + 2) + 3 half-ulps, and s (1 - s) |l| <= 0.28 where l > -1.3;
        // softmax, arguments 2.5 |l - m| (with p |l - m| <= 0.37 pmax, and ln E on
        // average in the sum), 22 additions, and the rest below 6
        if (p.sigmoid) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                key[j] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-l[j] * kLog2e));
            const float smax = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-m * kLog2e));
            tol = kUlp * smax * (8.f + 1.5f * __builtin_fmaxf(0.f, -m)) + 0x1p-120f;
            tol = m > -inf ? tol : 0.f;  // (0 times inf: a row without experts)
        } else {
            const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) key[j] *= inv;
            tol = kUlp * inv * 48.f + 0x1p-120f;
        }
    }
    bool unsure = false;
    if (scored) {  // c of every expert; -inf: absent
#pragma unroll
        for (int j = 0; j < NJ; ++j) key[j] = l[j] > -inf && b[j] > -inf ? key[j] + b[j] : -inf;
    }
    if (p.groups > 1) {  // (at most L)
#pragma unroll
        for (int j = 0; j < NJ; j += V) {
            const int e = column<L, V>(sub, j);
#pragma unroll
            for (int i = 0; i < V; ++i) s_c[e + i] = key[j + i];
        }
        wave_lds_order();
        const int n = p.E / p.groups;
        int P = L;  // lanes of a group
        while (P * p.groups > L) P >>= 1;
        bool near = false;
        uint64_t kept = choose_groups<L>(p, s_c, P, tol, &near);
        if (__ballot(near)) {
            double *c = lds + r * (L * NJ);
            wave_lds_order();
            exact_scores<L>(p, p.logits + t * p.E, m, c);
            wave_lds_order();
            kept = choose_groups<L>(p, c, P, 0.f, &near);
            wave_lds_order();
        }
        if (!p.bias) {  // by the logits
#pragma unroll
            for (int j = 0; j < NJ; ++j) key[j] = l[j];
        }
        const bool quads = V == 4 && n % 4 == 0;  // 4 columns lie in one group
        bool open = false;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            if (j % V == 0 || !quads) {
                const int e = column<L, V>(sub, j);
                const int g = n == 1 ? e : (int)__umulhi((uint32_t)e, magic);
                open = L <= 32 ? (uint32_t)kept >> (g * P & 31) & 1 : kept >> (g * P & 63) & 1;
            }
            key[j] = open ? key[j] : -inf;  // (columns past E have -inf)
        }
    } else if (!p.bias) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) key[j] = l[j];
    }

    // a bound of the K-th largest key: the K-th largest of the lanes' maxima
    float best = key[0];
#pragma unroll
    for (int j = 1; j < NJ; ++j) best = __builtin_fmaxf(best, key[j]);
    const int none = order_of(-inf);
    int mine_best = order_of(best), bound_k = none;
    for (int k = 0; k < p.K; ++k) {
        bound_k = lanes_max<L>(mine_best);
        mine_best = mine_best == bound_k ? none : mine_best;
    }
    const float bound = value_of(bound_k);
    // two keys of biased scores are apart if they differ by more than this and kUlp
    // times 4 their size; the candidates reach so far below the bound
    const float far = 2.f * tol;
    const float from = p.bias ? bound - (far + 4.f * kUlp * __builtin_fabsf(bound)) : bound;
    const float least = __builtin_fmaxf(from, -__FLT_MAX__);  // (not -inf: absent)
    int count = 0;
#pragma unroll
    for (int j = 0; j < NJ; ++j) count += key[j] >= least;
    const int upto = wave_inclusive_scan(count, lane);
    const int prior = __shfl(upto, r == 0 ? 0 : r * L - 1);
    const int start = r == 0 ? 0 : prior;
    const int n = __shfl(upto, r * L + L - 1) - start;  // of this row
    unsure |= n > L || __builtin_isnan(from);
    wave_lds_order();
    if (n <= L) {
        Candidate *at = cand + (upto - count - start);
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (key[j] >= least) *at++ = Candidate{key[j], column<L, V>(sub, j)};
    }
    wave_lds_order();
    const bool mine_ok = n <= L && sub < n;
    Candidate me = {0.f, 0};
    if (mine_ok) me = cand[sub];
    const float *row = p.logits + t * p.E;
    const float my_l = mine_ok ? row[me.col] : -inf;
    const float apart = far + 4.f * kUlp * __builtin_fabsf(me.key);
    int place = 0, close = 0;  // (close counts the candidate itself)
    const int most = wave_max(n <= L ? n : 0);
    for (int i = 0; i < most; ++i) {
        const Candidate o = cand[i < L ? i : 0];
        const bool in = i < n;
        place += in && (o.key > me.key || (o.key == me.key && o.col < me.col));
        close += in && !(__builtin_fabsf(o.key - me.key) > apart);
    }
    bool pick = mine_ok && place < p.K;
    if (p.bias && __ballot(pick && close > 1)) {
        // too near to call in 32 bits
        if (p.sigmoid) {  // a candidate's c in 64 bits needs its logit and bias alone
            double *exact = lds + 512 + 64 + r * L;
            double c = 0.;
            if (mine_ok) {
                c = 1. / (1. + exp(-(double)my_l)) + (double)p.bias[me.col];
                exact[sub] = c;
            }
            wave_lds_order();
            place = 0;
            for (int i = 0; i < n && n <= L; ++i)
                place += exact[i] > c || (exact[i] == c && cand[i].col < me.col);
            pick = mine_ok && place < p.K;
        } else {  // the whole row, but for experts of the same logit and bias
            bool near = false;
            if (pick && close > 1) {
                const float my_b = p.bias[me.col];
                for (int i = 0; i < n; ++i) {
                    const Candidate o = cand[i];
                    if (i != sub && !(__builtin_fabsf(o.key - me.key) > apart))
                        near |= !(row[o.col] == my_l && p.bias[o.col] == my_b);
                }
            }
            unsure |= group_bits<L>(__ballot(near), lane) != 0;
        }
    }

    const float top = group_max<L>(pick ? my_l : -inf);
    float s = 0.f;
    if (pick) {
        if (p.renorm)
            s = ratio_score(p.sigmoid, my_l, top);
        else if (p.sigmoid)
            s = 1.f / (1.f + expf(-my_l));
        else
            s = ratio_score(false, my_l, m) / sum;
    }
    if (p.renorm) {
        const float total = group_sum<L>(s);
        s = pick ? s / total : 0.f;
    }
    if (have && !unsure) {
        if (pick) {
            p.ids[t * p.K + place] = me.col;
            p.w[t * p.K + place] = p.scale * s;
        } else if (sub >= n && sub < p.K) {  // (fewer experts than picks: n < K)
            p.ids[t * p.K + sub] = -1;
            p.w[t * p.K + sub] = 0.f;
        }
    }
    uint64_t again = __ballot(unsure && have && sub == 0);
    while (again) {
        const int first = __ffsll((unsigned long long)again) - 1;
        again &= again - 1;
        const ScoreCall cold = p;  // (by address: p itself stays in scalar registers)
        exact_row<L * NJ / 64>(cold, t0 + first / L, lds);
    }
}

// workgroups for rows of L lanes each
template <int L> unsigned row_blocks(int64_t rows)
{
    constexpr int per = kWaves * (64 / L);
    return (unsigned)((rows + per - 1) / per);
}

template <int L, int NJ> hipError_t scored_t(const ScoreCall &c, hipStream_t s)
{
    const int n = c.E / c.groups;
    const uint32_t magic = n > 1 ? (uint32_t)((((uint64_t)1 << 32) + n - 1) / n) : 0;
    const bool quads = c.E % 4 == 0 && reinterpret_cast<uintptr_t>(c.logits) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(c.bias) % 16 == 0;
    return in_parts(c.T, kMostThreads / L, [&](int64_t t, int64_t rows) {
        ScoreCall p = c;
        p.logits += t * c.E;
        p.ids += t * c.K;
        p.w += t * c.K;
        p.T = (int)rows;
        const dim3 grid(row_blocks<L>(rows)), block(kWaves * 64);
        if (quads)
            hipLaunchKernelGGL((k_route_scored<L, NJ, 4>), grid, block, 0, s, p, magic);
        else
            hipLaunchKernelGGL((k_route_scored<L, NJ, 1>), grid, block, 0, s, p, magic);
        return hipGetLastError();
    });
}

// ---- gradient ------------------------------------------------------------------
// L lanes hold a row of dlogits; the picks' terms are added through a row of LDS (one
// instruction a round of L picks, lanes of one address in order). Bound by the traffic
// of dlogits and `add`; the logits are read at the picks alone but for softmax weights
// that are not renormalised.

template <typename T, int L, int NJ, int V>
__global__ __launch_bounds__(kWaves * 64) void k_route_scored_backward(const ScoreBackwardCall p)
{
    constexpr int R = 64 / L;
    __shared__ float s_all[kWaves][R * L * NJ];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane / L, sub = lane & (L - 1);
    float *mine = s_all[wave] + r * (L * NJ);
    const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * R;
    if (t0 >= p.T) return;  // (the whole wavefront)
    const bool have = t0 + r < p.T;
    const int64_t t = have ? t0 + r : p.T - 1;
    const float *row = p.logits + t * p.E;
    const float inf = __builtin_inff();
    const int id = sub < p.K ? p.ids[t * p.K + sub] : -1;  // (K <= L)
    bool ok = (unsigned)id < (unsigned)p.E;
    const float l = ok ? row[id] : -inf;
    ok = ok && l > -inf;
    const float u = ok ? p.scale * p.dw[t * p.K + sub] : 0.f;
    float add[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) add[j] = 0.f;
    if (p.add) {
        const T *q = static_cast<const T *>(p.add) + t * p.E;
#pragma unroll
        for (int j = 0; j < NJ; j += V) {
            const int e = column<L, V>(sub, j);
            if (e >= p.E) continue;
            float x[V];
            Vec<T, V>::load(q + e, x);
#pragma unroll
            for (int i = 0; i < V; ++i) add[j + i] = x[i];
        }
    }
    float pr[NJ], m = -inf, sum = 0.f, g = 0.f, total = 0.f;
    const bool dense = !p.sigmoid && !p.renorm;
    if (dense) {
        load_row<L, NJ, V>(row, p.E, sub, pr);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            pr[j] = __builtin_fmaxf(pr[j], -inf);
            m = __builtin_fmaxf(m, pr[j]);
        }
        m = group_max<L>(m);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            pr[j] = m == inf    ? (pr[j] == inf ? 1.f : 0.f)
                    : m == -inf ? 0.f
                                : __builtin_amdgcn_exp2f((pr[j] - m) * kLog2e);
            sum += pr[j];
        }
        sum = group_sum<L>(sum);
        if (ok) g = u * ratio_score(false, l, m) / sum;
        total = group_sum<L>(g) / (sum > 0.f ? sum : 1.f);
    } else if (p.renorm) {
        const float top = group_max<L>(ok ? l : -inf);
        float s = ok ? ratio_score(p.sigmoid, l, top) : 0.f;
        const float S = group_sum<L>(s);
        s = S > 0.f ? s / S : 0.f;
        g = s * (u - group_sum<L>(s * u));
        if (p.sigmoid && ok) g *= 1.f / (1.f + expf(l));
    } else if (ok) {
        g = u * (1.f / (1.f + expf(-l))) * (1.f / (1.f + expf(l)));
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) mine[column<L, V>(sub, j)] = 0.f;
    wave_lds_order();
    if (ok) atomicAdd(mine + id, g);
    wave_lds_order();
    if (!have) return;
    T *out = static_cast<T *>(p.dlogits) + t * p.E;
#pragma unroll
    for (int j = 0; j < NJ; j += V) {
        const int e = column<L, V>(sub, j);
        if (e >= p.E) continue;
        float x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = mine[e + i] + add[j + i];
            if (dense) x[i] -= pr[j + i] * total;
        }
        Vec<T, V>::store(out + e, x);
    }
}

template <typename T, int L, int NJ> hipError_t backward_t(const ScoreBackwardCall &c, hipStream_t s)
{
    const bool quads = c.E % 4 == 0 && reinterpret_cast<uintptr_t>(c.logits) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(c.add) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(c.dlogits) % 16 == 0;
    return in_parts(c.T, kMostThreads / L, [&](int64_t t, int64_t rows) {
        ScoreBackwardCall p = c;
        p.logits += t * c.E;
        p.ids += t * c.K;
        p.dw += t * c.K;
        if (p.add) p.add = static_cast<const T *>(p.add) + t * c.E;
        p.dlogits = static_cast<T *>(p.dlogits) + t * c.E;
        p.T = (int)rows;
        const dim3 grid(row_blocks<L>(rows)), block(kWaves * 64);
        if (quads)
            hipLaunchKernelGGL((k_route_scored_backward<T, L, NJ, 4>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((k_route_scored_backward<T, L, NJ, 1>), grid, block, 0, s, p);
        return hipGetLastError();
    });
}

// lanes of a row and columns of a lane, for E experts: the fewest lanes that hold a row
// with 16 columns each, and one of K things each (picks, groups). (As many picks as that
// make most rows exact_row's: figures at the head.)
template <typename F> hipError_t with_lanes(int E, int K, F run)
{
    using std::integral_constant;
    if (K <= 16 && E <= 256)
        return E <= 64    ? run(integral_constant<int, 16>(), integral_constant<int, 4>())
               : E <= 128 ? run(integral_constant<int, 16>(), integral_constant<int, 8>())
                          : run(integral_constant<int, 16>(), integral_constant<int, 16>());
    if (K <= 32 && E <= 512)
        return E <= 256 ? run(integral_constant<int, 32>(), integral_constant<int, 8>())
                        : run(integral_constant<int, 32>(), integral_constant<int, 16>());
    return E <= 256 ? run(integral_constant<int, 64>(), integral_constant<int, 4>())
                    : run(integral_constant<int, 64>(), integral_constant<int, 16>());
}

}  // namespace

hipError_t launch_route_scored(const ScoreCall &c, hipStream_t s)
{
    return with_lanes(c.E, c.K > c.groups ? c.K : c.groups, [&](auto lanes, auto columns) {
        return scored_t<decltype(lanes)::value, decltype(columns)::value>(c, s);
    });
}

hipError_t launch_route_scored_backward(const ScoreBackwardCall &c, hipStream_t s)
{
    return with_lanes(c.E, c.K, [&](auto lanes, auto columns) {
        constexpr int L = decltype(lanes)::value, NJ = decltype(columns)::value;
        return c.dtype == 0   ? backward_t<float, L, NJ>(c, s)
               : c.dtype == 1 ? backward_t<_Float16, L, NJ>(c, s)
                              : backward_t<__bf16, L, NJ>(c, s);
    });
}

}  // namespace moe
