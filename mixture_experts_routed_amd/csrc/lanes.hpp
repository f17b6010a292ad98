// Rows of experts in groups of lanes of a wavefront: sums and maxima on register moves,
// and how a group holds a row.
#pragma once

#include "common.hpp"

namespace moe {

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

}  // namespace moe
