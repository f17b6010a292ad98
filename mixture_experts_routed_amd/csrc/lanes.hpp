// Sums and maxima over groups of lanes of a wavefront, on register moves.
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

}  // namespace moe
