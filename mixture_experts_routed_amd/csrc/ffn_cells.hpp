// Cells of the grouped expert FFN: what one workgroup of a projection computes, for
// each weight layout, and its kernel. The design stands at the head of ffn.hip, which
// launches the 16- and 32-bit layouts; ffn_mx4.hip has the 4-bit weights' kernels (a
// source of its own for the time that compiling takes).
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "plan_wave.hpp"

#include <type_traits>

namespace moe {

constexpr int kMT = kItemRows / 16;     // 16-row m-tiles per work item
constexpr int kWavesPerBlock = 4;
constexpr int kNpl = 4;                 // columns per lane and B stream
// Packed weight layout (kPacked, written once by k_pack): a matrix [E][Kd][N] becomes, per expert, column group g (4 slices
// of 64*m columns), K-step s, wave slice w and stream m (gate/up: m = 1 stream
// of 64 columns; down: m = 2 halves of 64 columns), a 4 KB tile of 4 x 64
// 16-byte words, word [c][lane] = what MFMA lane `lane` takes as its c-th B
// operand of the step: 16-bit types: the 8 K-values 32s + 8*(lane>>4) + i of
// column (4g+w)*64m + 64*stream + 4*(lane&15) + c; fp32: 4 columns
// (4g+w)*64m + 64*stream + 4*(lane&15) .. +3 of K-row 16s + 4*(lane>>4) + c.
// Outside [0,Kd) x [0,N) the words hold zeros. A workgroup's K range of one
// column group is then one contiguous run of 16 KB (x m) steps.
//
// Microscaled 4-bit weights (kMx4, written by mx4.hip) have the same order of
// tiles with 16-bit K-steps; a tile is 1024 bytes of codes and 64 of scales:
// word [lane] (16 bytes) holds the 4 columns' operands of that lane as above, 8
// codes of 4 bits each (K-value i in bits 4 i of dword c), and scale byte
// 4*(lane&15) + c the power of two 2^(byte - 127) of the 32 K-values of that
// column: a K-step is one block of the format.
struct PackedGeom {
    int gs, nst, m;       // column groups, K-steps, streams
    uint32_t tile_bytes;  // of one K-step of one slice's stream
    uint32_t step_bytes;  // bytes of one K-step of one column group
};

__host__ __device__ inline PackedGeom packed_geom(int Kd, int N, bool gateup, int es,
                                                  bool mx4 = false)
{
    PackedGeom z;
    z.m = gateup ? 1 : 2;
    const int kstep = es == 2 ? 32 : 16;
    z.gs = (N + 256 * z.m - 1) / (256 * z.m);
    z.nst = (Kd + kstep - 1) / kstep;
    z.tile_bytes = mx4 ? kMx4Tile : 4096u;
    z.step_bytes = 4 * z.tile_bytes * (uint32_t)z.m;
    return z;
}

// ---- raw buffer loads -----------------------------------------------------
// A buffer resource covering exactly one operand range: loads past its end
// return zeros without touching memory (range-checked by the hardware), which
// zero-fills the K tail of the weights, the rows past a work item's end and
// the steps past the end of a K split.
// Word 3 = 0x00020000: raw (untyped) buffer on gfx9-family GPUs.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                             0x00020000);
}

// Cache policy of a buffer load: 0 = default; kNT = non-temporal (the weights
// are read exactly once, so they should not displace the reused row tiles).
constexpr int kNT = 2;

// s_waitcnt vmcnt(n), expcnt and lgkmcnt left at their maximum (no wait)
constexpr int wait_vm(int n) { return 0x0F70 | n; }

template <int BYTES, int POLICY = 0> struct Ld;
template <int POLICY> struct Ld<8, POLICY> {
    typedef uint2 type;
    static __device__ __forceinline__ uint2 run(__amdgpu_buffer_rsrc_t r, uint32_t v, uint32_t s)
    {
        return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, v, s, POLICY));
    }
};
template <int POLICY> struct Ld<16, POLICY> {
    typedef uint4 type;
    static __device__ __forceinline__ uint4 run(__amdgpu_buffer_rsrc_t r, uint32_t v, uint32_t s)
    {
        return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, v, s, POLICY));
    }
};

// stores of outputs that this kernel does not read again: non-temporal
__device__ __forceinline__ void store_nt(float4 *p, float4 v)
{
    typedef float f4 __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(f4{v.x, v.y, v.z, v.w}, reinterpret_cast<f4 *>(p));
}
__device__ __forceinline__ void store_nt(uint2 *p, uint2 v)
{
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    __builtin_nontemporal_store(u2{v.x, v.y}, reinterpret_cast<u2 *>(p));
}
__device__ __forceinline__ void store_nt(uint4 *p, uint4 v)
{
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    __builtin_nontemporal_store(u4{v.x, v.y, v.z, v.w}, reinterpret_cast<u4 *>(p));
}

// Stores of the down projection's y, which the combine reads next: buffer
// stores with cache policy sc1 only. Measured on the prefill layer against
// non-temporal stores: the down projection ~15 us and the combine ~7 us faster
// (its y reads then hit the Infinity Cache). Default-policy stores were slower
// than both, and sc1 stores of the gate/up output h gained nothing.
constexpr int kSC1 = 16;
template <int POLICY = kSC1>
__device__ __forceinline__ void store_sc1(__amdgpu_buffer_rsrc_t r, uint32_t off, float4 v)
{
    typedef unsigned u4 __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), r, off, 0, POLICY);
}

// ---- per element type: MFMA and conversion -------------------------------
template <typename T> struct Elt;

template <> struct Elt<_Float16> {
    static constexpr int KR = 8;  // K-values per lane per MFMA
    static __device__ __forceinline__ float4_t mfma(uint4 a, uint4 b, float4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a),
                                                      __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
    }
    // 8 codes of 4 bits times their scale (exact within the type's range)
    static __device__ __forceinline__ uint4 mx4(uint32_t codes, float scale)
    {
        return make_uint4(
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 0)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 1)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 2)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, 3)));
    }
    static __device__ __forceinline__ uint32_t pack2(float lo, float hi)
    {
        const _Float16 l = (_Float16)lo, h = (_Float16)hi;
        return (uint32_t)__builtin_bit_cast(uint16_t, l) |
               ((uint32_t)__builtin_bit_cast(uint16_t, h) << 16);
    }
};

template <> struct Elt<__bf16> {
    static constexpr int KR = 8;
    static __device__ __forceinline__ float4_t mfma(uint4 a, uint4 b, float4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ uint4 mx4(uint32_t codes, float scale)
    {
        return make_uint4(
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2)),
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3)));
    }
    static __device__ __forceinline__ uint32_t pack2(float lo, float hi)
    {
        const __bf16 l = (__bf16)lo, h = (__bf16)hi;  // round to nearest even
        return (uint32_t)__builtin_bit_cast(uint16_t, l) |
               ((uint32_t)__builtin_bit_cast(uint16_t, h) << 16);
    }
};

template <> struct Elt<float> {
    static constexpr int KR = 4;
};

// silu(z) = z / (1 + e^-z), with the hardware reciprocal (about 1 ulp) in
// place of an IEEE division: an order of magnitude below the error of the
// fp16/bf16 SwiGLU output it feeds, and a fraction of the epilogue's time
__device__ __forceinline__ float silu(float z)
{
    return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// 16-bit B operand: RP consecutive K-rows of 4 columns each (row i = K-value
// i). Column c of them as RP/2 words of an MFMA operand (element i = K-row i).
template <int RP>
__device__ __forceinline__ void column_of_rows(const uint2 (&r)[RP], int c, uint32_t (&o)[RP / 2])
{
#pragma unroll
    for (int p = 0; p < RP / 2; ++p) {
        const uint32_t lo = (c < 2) ? r[2 * p].x : r[2 * p].y;
        const uint32_t hi = (c < 2) ? r[2 * p + 1].x : r[2 * p + 1].y;
        o[p] = (c & 1) ? ((lo >> 16) | (hi & 0xffff0000u)) : ((lo & 0xffffu) | (hi << 16));
    }
}

__device__ __forceinline__ uint4 column_of_rows(const uint2 (&r)[8], int c)
{
    uint32_t o[4];
    column_of_rows<8>(r, c, o);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int q)
{
    return q == 0 ? v.x : q == 1 ? v.y : q == 2 ? v.z : v.w;
}

__device__ __forceinline__ float lanef(const uint4 &v, int q)
{
    return __builtin_bit_cast(float, word(v, q));
}

__device__ __forceinline__ uint4 mask4(uint4 v, uint32_t m)
{
    return make_uint4(v.x & m, v.y & m, v.z & m, v.w & m);
}

// A lane's weights of one K-step and stream in 4 bits: the 4 columns' codes and
// scale bytes; column c as an MFMA operand
struct Mx4Word {
    uint4 codes;
    uint32_t scales;
};
__device__ __forceinline__ Mx4Word load_mx4(__amdgpu_buffer_rsrc_t r, uint32_t tile, int lane)
{
    Mx4Word w;
    w.codes = Ld<16>::run(r, tile + (uint32_t)lane * 16u, 0u);
    w.scales = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(
        r, tile + (uint32_t)(lane & 15) * 4u, kMx4Codes, 0);
    return w;
}
template <typename T> __device__ __forceinline__ uint4 mx4_operand(const Mx4Word &w, int c)
{
    return Elt<T>::mx4(word(w.codes, c), __uint_as_float(((w.scales >> (8 * c)) & 0xffu) << 23));
}

// Arguments of one grouped GEMM launch.
//   gate/up: A = xs [rows][d] (or x [a_rows][d] when GATHERED), B0 = W_gate,
//            B1 = W_up [E][d][f], out = h [rows][f] (type T).
//   down:    A = h [rows][f], B0 = W_down [E][f][d], out = y [rows][d] (fp32),
//            stok / sw for the epilogue.
// With nsplit > 1 the epilogue instead writes fp32 partial sums: split s at
// part + s * plane, row r at r * 2N (gate: columns [0, N), up: [N, 2N)) or at
// r * N (down, without the router weight).
// The item count and the work items are separate __restrict__ kernel
// arguments: provably read-only, they are fetched with scalar loads.
struct GemmArgs {
    const void *A;
    const void *B0;
    const void *B1;
    const int32_t *stok;
    const float *sw;
    void *out;
    float *part;
    int64_t plane;
    int a_rows;
    int Kd, N;
    int nsplit;       // K splits per (item, column group)
    int split_steps;  // K-steps per split
    int skip_quads;   // 1: the items in runs of 4 (the first ctl[1]) are left to k_big
    // down projection, compact outputs: out holds binary16 rows and yexp their
    // exponents, block-major: yexp[b * estride + row] for the kY16Block columns
    // of block b (estride = max_rows); nullptr: fp32 y
    int8_t *yexp;
    int64_t estride;
};

__device__ __forceinline__ void store_b64(__amdgpu_buffer_rsrc_t r, uint32_t off, uint2 v,
                                          int policy_sc1)
{
    typedef unsigned u2 __attribute__((ext_vector_type(2)));
    if (policy_sc1)
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, v), r, off, 0, kSC1);
    else
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, v), r, off, 0, kNT);
}

// One row of a down cell in the compact format. This lane holds the row's
// values v[m][c] at columns col + m * 64 + c; the 16 lanes of its DPP row hold
// the row's columns [col0, col0 + 128), one exponent block. Lanes whose
// columns lie past N contribute nothing and store nothing, but take part in
// the row maximum (every lane of the row must be active here). ry covers the
// item's rows of binary16 y; rl is the row within the item. Stores: sc1
// (policy_sc1) or non-temporal. Returns the row's exponent (the same in all
// 16 lanes); the caller stores the exponents (store_y16_exponents).
__device__ __forceinline__ int store_y16_row(const GemmArgs &p, __amdgpu_buffer_rsrc_t ry, int rl,
                                             int col, const float (&v)[2][4], int policy_sc1)
{
    constexpr int HALF = 16 * kNpl;
    const int N = p.N;
    float M = 0.0f;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            M = __builtin_fmaxf(M, col + m * HALF < N ? __builtin_fabsf(v[m][c]) : 0.0f);
    const int e = y16_exponent(row16_fmax(M));
    const float scale = pow2f(e);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        if (col + m * HALF >= N) continue;
        float q[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) q[c] = v[m][c] * scale;
        store_b64(ry, (uint32_t)((rl * N + col + m * HALF) * 2),
                  make_uint2(Elt<_Float16>::pack2(q[0], q[1]), Elt<_Float16>::pack2(q[2], q[3])),
                  policy_sc1);
    }
    return e;
}

// The exponents of a wavefront's 64 rows of one block, in one store: ev[mt][r]
// is the exponent of row 16 mt + 4 kg + r (kg = the lane's DPP row), so lane
// (kg, nq) already holds row 16 (nq >> 2) + 4 kg + (nq & 3) -- the 64 lanes
// hold the 64 rows once each -- and stores it if `real` (its row holds an
// entry). yexp_block = the block's exponents, row0 = the item's first row.
template <int NMT>
__device__ __forceinline__ void store_y16_exponents(int8_t *yexp_block, int64_t row0,
                                                    const int (&ev)[NMT][4], int rl, bool real)
{
    const int nq = threadIdx.x & 15;
    int e = 0;
#pragma unroll
    for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) e = (mt == (nq >> 2) && r == (nq & 3)) ? ev[mt][r] : e;
    if (real) yexp_block[row0 + rl] = (int8_t)e;
}

// Epilogue of one wavefront: acc[m][mt][c][r] is the output at row
// 16*mt + 4*kg + r of item `it` and column col + c (+ HALF for m = 1 of the
// down projection). rinfo[l] = (router weight, token) of the item's row l.
template <typename T, bool GATEUP, int NMT, bool MAY_SPLIT = true>
__device__ __forceinline__ void store_cells(const GemmArgs &p, const WorkItem &it, int col, int kg,
                                            const float4_t (&acc)[2][NMT][kNpl],
                                            const float2 *__restrict__ rinfo, int split)
{
    constexpr int ES = sizeof(T);
    constexpr int HALF = GATEUP ? 0 : 16 * kNpl;
    const int N = p.N;
    const bool partial = MAY_SPLIT && p.nsplit > 1;
    if constexpr (!GATEUP && ES == 2) {
        if (p.yexp && !partial) {
            // compact y: every lane stays for the row maxima (no early exit by column)
            const int col0 = col - kNpl * (threadIdx.x & 15);
            if (col0 >= N) return;  // the whole slice lies past N (wave-uniform)
            const __amdgpu_buffer_rsrc_t ry =
                make_rsrc(static_cast<uint16_t *>(p.out) + (int64_t)it.row0 * N,
                          (uint32_t)(it.nrows * N * 2));
            int ev[NMT][4];
#pragma unroll
            for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    ev[mt][r] = 0;
                    const int rl = 16 * mt + 4 * kg + r;
                    if (rl >= it.nrows) continue;  // uniform over the DPP row
                    const float2 ri = rinfo[rl];
                    if (__float_as_int(ri.y) < 0) continue;  // pad rows are never combined
                    float v[2][4];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int c = 0; c < 4; ++c) v[m][c] = ri.x * acc[m][mt][c][r];
                    ev[mt][r] = store_y16_row(p, ry, rl, col, v, 1);
                }
            const int nq = threadIdx.x & 15;
            const int rl = 16 * (nq >> 2) + 4 * kg + (nq & 3);
            const bool real = rl < it.nrows && __float_as_int(rinfo[rl].y) >= 0;
            store_y16_exponents<NMT>(p.yexp + (col0 / kY16Block) * p.estride, it.row0, ev, rl,
                                     real);
            return;
        }
    }
    if (col >= N) return;
#pragma unroll
    for (int mt = 0; mt < NMT; ++mt) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int rl = 16 * mt + 4 * kg + r;
            if (rl >= it.nrows) continue;
            const int64_t row = it.row0 + rl;
            if constexpr (GATEUP) {
                if (partial) {
                    // pad rows: the reduction writes their zero h without reading
                    if (__float_as_int(rinfo[rl].y) < 0) continue;
                    float *P = p.part + split * p.plane + row * 2 * N + col;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        *reinterpret_cast<float4 *>(P + m * N) =
                            make_float4(acc[m][mt][0][r], acc[m][mt][1][r], acc[m][mt][2][r],
                                        acc[m][mt][3][r]);
                    continue;
                }
                float hv[kNpl];
#pragma unroll
                for (int c = 0; c < kNpl; ++c) hv[c] = silu(acc[0][mt][c][r]) * acc[1][mt][c][r];
                T *H = static_cast<T *>(p.out) + row * N + col;
                if constexpr (ES == 2)
                    store_nt(reinterpret_cast<uint2 *>(H),
                             make_uint2(Elt<T>::pack2(hv[0], hv[1]), Elt<T>::pack2(hv[2], hv[3])));
                else
                    store_nt(reinterpret_cast<float4 *>(H), make_float4(hv[0], hv[1], hv[2], hv[3]));
            } else {
                const float2 ri = rinfo[rl];
                if (__float_as_int(ri.y) < 0) continue;  // pad rows are never combined
                const float g = partial ? 1.0f : ri.x;
                float *P = p.part + split * p.plane + row * N + col;
                // the item's rows of y, as one descriptor (range-checked stores)
                const __amdgpu_buffer_rsrc_t ry =
                    make_rsrc(static_cast<float *>(p.out) + (int64_t)it.row0 * N,
                              (uint32_t)(it.nrows * N * 4));
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    if (col + m * HALF >= N) continue;
                    const float4 v = make_float4(g * acc[m][mt][0][r], g * acc[m][mt][1][r],
                                                 g * acc[m][mt][2][r], g * acc[m][mt][3][r]);
                    if (partial)
                        *reinterpret_cast<float4 *>(P + m * HALF) = v;
                    else
                        store_sc1(ry, (uint32_t)((rl * N + col + m * HALF) * 4), v);
                }
            }
        }
    }
}

// (router weight, token) of the item's rows for the epilogue; the gate/up
// projection has no router weight (sw is not passed) and needs the tokens only
// (ltok != nullptr: the item's tokens from LDS, ltok[l] for its row l)
template <bool WITH_SW>
__device__ __forceinline__ void load_rinfo(const GemmArgs &p, const WorkItem &it, int l,
                                           float2 *__restrict__ rinfo, const int *ltok = nullptr)
{
    const bool ok = l < it.nrows;
    const int64_t r = it.row0 + (ok ? l : 0);
    const int t = ok ? (ltok ? ltok[l] : p.stok[r]) : -1;
    rinfo[l] = make_float2(WITH_SW && ok ? p.sw[r] : 0.f, __int_as_float(t));
}

// Launches with fewer cells than this (the GPU's workgroup slots: 2 per CU)
// stream their weights deep (see wide_cells)
constexpr int kDeepBelowCells = 512;

// Pipeline depth of the wide cells for NMT m-tiles: stage = 32 B-operand + 4
// A-operand VGPRs, accumulators = 32*NMT VGPRs; S stages + accumulators stay
// <= ~232.
constexpr int stages_for(int nmt) { return nmt >= 4 ? 2 : nmt == 3 ? 3 : nmt == 2 ? 4 : 5; }

// Shared A tile of one K-step: 64 rows x 32 K (16-bit) or 64 rows x 16 K
// (fp32), 64 bytes per row, double-buffered: 2 x 4 KB of LDS per workgroup.
constexpr int kATileU4 = kItemRows * 64 / 16;
// Shared B tile of the tall cells: per column slice 2 matrices x 64 lanes x
// 64 bytes (4 fragments of 16 bytes per lane), double-buffered.
constexpr int tall_buf_u4(int nslices) { return nslices * 2 * 64 * 4; }
constexpr int kLdsU4 = 2 * tall_buf_u4(2) > 2 * kATileU4 ? 2 * tall_buf_u4(2) : 2 * kATileU4;

// Wide cells: a workgroup of 4 wavefronts computes one work item (<= 64 rows)
// against 4 adjacent column slices of 16*kNpl columns, one per wavefront.
//  * A (the item's rows) is shared: per K-step each wavefront loads 16 rows x
//    64 bytes (one 16-byte load per lane) into registers, writes them to an LDS
//    slot, and after one barrier every wavefront reads its MFMA A-fragments
//    from LDS. One copy of A per workgroup instead of one per wavefront.
//  * B (the weights) is private to each wavefront: lane l supplies MFMA column
//    (l & 15) and K-group (l >> 4); it loads KR K-rows x kNpl columns of each
//    weight matrix per step (16 lanes cover one 16*kNpl-column row segment) and
//    transposes them in registers, so MFMA c produces the logical columns
//    kNpl*j + c, j = 0..15.
//  * S-stage register ring: the loads of step s+S-1 are issued before the
//    MFMAs of step s; the loop body is straight-line code, so they stay in
//    flight. The per-step barrier keeps the 4 wavefronts in step, so together
//    they read 4 adjacent row segments of every weight row.
//  * depth of the weight stream, one policy per launch (ctl[2]): when most
//    items are single (each streams its expert's weights from HBM once) the
//    launch runs shallow: the row operand's K-tail mask is applied as it is
//    loaded, so a wavefront waits for the step it has just issued (all but
//    its last few loads) before computing, about one step per wavefront in
//    flight. More only queues in the memory system: on a 2,048-token prefill
//    layer (512 experts, single items) masking at the use, with S-1 steps in
//    flight, was 4% slower. When most items are in runs (skewed routing; the
//    runs' tiles are re-read from L2) the mask moves to the use and the ring
//    keeps S-1 steps in flight: 7% faster on the down projection of a skewed
//    2,048-token chunk. Shallow single items beside deep runs in one launch
//    measured slower than either policy. A launch of fewer cells than the GPU
//    holds at once (kDeepBelowCells, two per CU) runs deep too: no other
//    workgroup shares a CU's memory pipe, so a workgroup's own bytes in flight
//    set its rate (decode's down projection, 186 cells: 30.3 -> 25.1 us).
// GATHERED (gate/up only): A is the token activation x [a_rows][Kd] and row r
// of the item reads x[stok[r]] -- the gather fused into the A-tile loads.
// The K range is [kb, ke) (a split of the reduction, or all of it).
template <typename T, bool GATEUP, bool GATHERED, int WF, bool DEEP, int NMT>
__device__ __forceinline__ void wide_cells(const GemmArgs &p, const WorkItem it, int slice,
                                           int kb, int ke, int split, uint4 *__restrict__ a_lds,
                                           float2 *__restrict__ rinfo, const int *ltok)
{
    constexpr int NPL = kNpl;
    constexpr int ES = sizeof(T);
    constexpr int KR = Elt<T>::KR;
    constexpr int KSTEP = 4 * KR;
    constexpr int NMAT = 2;       // two B streams (see below)
    constexpr int LB = NPL * ES;  // bytes per lane per row
    const T *A = static_cast<const T *>(p.A);
    const T *B0 = static_cast<const T *>(p.B0);
    const T *B1 = static_cast<const T *>(p.B1);
    const int Kd = p.Kd, N = p.N;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int nq = lane & 15, kg = lane >> 4;
    // GATEUP: slice = 16*NPL columns of both W_gate and W_up. Down: slice =
    // 2*16*NPL columns of W_down, as two halves 16*NPL columns apart, so that
    // each fp32 store instruction of the epilogue covers whole 64-byte runs.
    constexpr int SW = GATEUP ? 16 * NPL : 32 * NPL;  // columns per slice
    constexpr int HALF = GATEUP ? 0 : 16 * NPL;       // column offset of stream 1
    const int col = slice * SW + NPL * nq;
    const bool slice_ok = slice * SW < N;  // wave-uniform

    // operand ranges: this expert's weight rows [kb, ke) (empty for a surplus
    // slice: its loads return zeros without memory traffic), this item's rows
    __amdgpu_buffer_rsrc_t rb0, rb1;
    uint32_t vcol, rowb, bstep;  // lane offset, B row stride, B bytes per K-step
    if constexpr (WF == kPacked) {
        // this wavefront's tiles (g, s, w, m) for s in [s0, s1): 4 KB each,
        // one K-step apart (16 KB x streams)
        const int g = slice >> 2, w = slice & 3;
        const PackedGeom z = packed_geom(Kd, N, GATEUP, ES);
        const int s0 = kb / KSTEP, s1 = (ke + KSTEP - 1) / KSTEP;
        const size_t tb =
            ((((size_t)it.expert * z.gs + g) * z.nst + s0) * 4 + w) * z.m * z.tile_bytes;
        const uint32_t span = (uint32_t)(s1 - s0) * z.step_bytes;
        const uint32_t r0 = (uint32_t)__builtin_amdgcn_readfirstlane(
            (int)(slice_ok ? span - (uint32_t)(w * z.m) * z.tile_bytes : 0u));
        const uint32_t r1 = (uint32_t)__builtin_amdgcn_readfirstlane(
            (int)(slice_ok ? span - (uint32_t)(w * z.m + z.m - 1) * z.tile_bytes : 0u));
        const char *b0c = static_cast<const char *>(p.B0);
        rb0 = make_rsrc(b0c + tb, r0);
        rb1 = GATEUP ? make_rsrc(static_cast<const char *>(p.B1) + tb, r0)
                     : make_rsrc(b0c + tb + z.tile_bytes, r1);
        vcol = (uint32_t)lane * 16;
        rowb = 1024;  // between fragments c of one lane
        bstep = z.step_bytes;
    } else {
        const size_t wofs = (size_t)it.expert * Kd * N + (size_t)kb * N;
        const uint32_t kbytes = (uint32_t)((size_t)(ke - kb) * N * ES);
        const uint32_t wbytes = slice_ok ? kbytes : 0u;
        rb0 = make_rsrc(B0 + wofs, wbytes);
        // ((ke-kb)*N >= 8*8 >= HALF, so the second range never underflows;
        // readfirstlane keeps the wave-uniform value in an SGPR)
        const uint32_t wbytes1 = (uint32_t)__builtin_amdgcn_readfirstlane(
            (int)(slice_ok ? kbytes - (uint32_t)(HALF * ES) : 0u));
        rb1 = GATEUP ? make_rsrc(B1 + wofs, wbytes) : make_rsrc(B0 + wofs + HALF, wbytes1);
        rowb = (uint32_t)N * ES;  // bytes per weight row
        vcol = (uint32_t)col * ES;
        bstep = (uint32_t)KSTEP * rowb;
    }
    // this thread's share of the A tile: row tid/4, 16-byte chunk tid%4
    const int arow = tid >> 2, achunk = (tid & 3) * (16 / ES);
    __amdgpu_buffer_rsrc_t ra;
    uint32_t va0;
    if constexpr (GATHERED) {
        // all of x (< 2 GiB, checked by the host); a pad row (token -1) or a
        // row past the item starts at 2^31, outside the range: it reads zeros
        ra = make_rsrc(A, (uint32_t)((size_t)p.a_rows * Kd * ES));
        const int t = arow < it.nrows ? (ltok ? ltok[arow] : p.stok[it.row0 + arow]) : -1;
        va0 = (unsigned)t < (unsigned)p.a_rows ? (uint32_t)t * (uint32_t)Kd * ES : 0x80000000u;
    } else {
        ra = make_rsrc(A + (size_t)it.row0 * Kd, (uint32_t)((size_t)it.nrows * Kd * ES));
        va0 = (uint32_t)arow * (uint32_t)Kd * ES;
    }

    // made visible to all wavefronts by the barriers of the K loop (gate/up
    // needs the tokens only for its partial sums)
    if (!GATEUP || p.nsplit > 1)
        if (tid < kItemRows) load_rinfo<!GATEUP>(p, it, tid, rinfo, ltok);

    float4_t acc[NMAT][NMT][NPL];
#pragma unroll
    for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
            for (int c = 0; c < NPL; ++c) acc[m][mt][c] = float4_t{0.f, 0.f, 0.f, 0.f};

    // packed: 4 fragments (fp32: 4 rows) of 16 bytes per stream and step
    constexpr int NB = WF == kPacked ? 4 : KR;
    constexpr int LBB = WF == kPacked ? 16 : LB;
    typedef typename Ld<LBB>::type BT;
    struct Stage {
        BT b[NMAT][NB];
        uint4 a;
    };
    auto load = [&](Stage &st, int k0) {
        const uint32_t vb = WF == kPacked ? vcol + (uint32_t)((k0 - kb) / KSTEP) * bstep
                                          : vcol + (uint32_t)(k0 + KR * kg - kb) * rowb;
#pragma unroll
        for (int i = 0; i < NB; ++i) st.b[0][i] = Ld<LBB, kNT>::run(rb0, vb, (uint32_t)i * rowb);
#pragma unroll
        for (int i = 0; i < NB; ++i) st.b[1][i] = Ld<LBB, kNT>::run(rb1, vb, (uint32_t)i * rowb);
        // K past the range: the weights read as zero; zero A too so that no
        // non-finite value of a neighbouring row can leak in as 0 * inf.
        // Shallow: masked here, which makes the wavefront wait for the step's
        // loads right after issuing them; deep: masked at its use
        const int ka = k0 + achunk;
        st.a = Ld<16>::run(ra, va0 + (uint32_t)ka * ES, 0u);
        if constexpr (!DEEP) st.a = mask4(st.a, ka < ke ? 0xffffffffu : 0u);
    };
    auto compute = [&](const Stage &st, int step) {
        uint4 *slot = a_lds + (step & 1) * kATileU4;
        const int ka = kb + step * KSTEP + achunk;
        slot[tid] = DEEP ? mask4(st.a, ka < ke ? 0xffffffffu : 0u) : st.a;
        __syncthreads();
        uint4 af[NMT];
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt) af[mt] = slot[(16 * mt + nq) * 4 + kg];
        if constexpr (ES == 2) {
#pragma unroll
            for (int c = 0; c < NPL; ++c) {
#pragma unroll
                for (int m = 0; m < NMAT; ++m) {
                    uint4 fb;
                    if constexpr (WF == kPacked)
                        fb = st.b[m][c];
                    else
                        fb = column_of_rows(st.b[m], c);
#pragma unroll
                    for (int mt = 0; mt < NMT; ++mt)
                        acc[m][mt][c] = Elt<T>::mfma(af[mt], fb, acc[m][mt][c]);
                }
            }
        } else {
            // fp32: sub-step q uses K = k0 + 4*kg + q in both operands
#pragma unroll
            for (int q = 0; q < KR; ++q)
#pragma unroll
                for (int m = 0; m < NMAT; ++m)
#pragma unroll
                    for (int c = 0; c < NPL; ++c) {
                        const float b = lanef(st.b[m][q], c);
#pragma unroll
                        for (int mt = 0; mt < NMT; ++mt)
                            acc[m][mt][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                lanef(af[mt], q), b, acc[m][mt][c], 0, 0, 0);
                    }
        }
    };

    constexpr int S = stages_for(NMT);
    const int nsteps = (ke - kb + KSTEP - 1) / KSTEP;
    Stage st[S];
    // deep: the prologue's loads stay in step order (the load-count waits at
    // the loop head are taken over both entries into it)
#pragma unroll
    for (int j = 0; j < S - 1; ++j) {
        load(st[j], kb + j * KSTEP);
        if constexpr (DEEP) __builtin_amdgcn_sched_barrier(0);
    }
    for (int s = 0; s < nsteps; s += S) {
#pragma unroll
        for (int j = 0; j < S; ++j) {
            // steps past the range load zero weights (no memory traffic) and add 0
            load(st[(j + S - 1) % S], kb + (s + j + S - 1) * KSTEP);
            __builtin_amdgcn_sched_barrier(0);
            compute(st[j], s + j);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    store_cells<T, GATEUP, NMT>(p, it, col, kg, acc, rinfo, split);
}

// Wide cells over weights in 4 bits. Rows, columns and accumulators as above; what
// differs follows from a K-step's weights being 17/64 of the bytes:
//  * the matrix cores and the conversion of codes to operands (4 instructions of two
//    values each an operand, v_cvt_scalef32_pk_{f16,bf16}_fp4, which takes the block's
//    scale) now take as long as the stream, so nothing may wait: the operand of the
//    next column is made while this one's MFMAs run, the row operands of the next
//    step are read from LDS in the middle of this step, behind its one barrier, and
//    written there at its start;
//  * a wavefront keeps S - 1 steps (of 1 KB and 64 bytes a stream) in flight: two
//    registers' worth of loads an operand, in place of 16.
// Steps past the range load zeros (code 0, scale 2^-127), which add nothing.
// Measured, 2,048 tokens, 512 experts, top-10, 2,560 x 768, fp16: gate/up 256 us (1.07 GB
// of weights: 4.2 TB/s), down 159 us (0.53 GB, and 210 MB of fp32 written). In the form
// that 16-bit weights' cells have, with a conversion in front, 379 and 222. Stamps show
// what bounds them: routing is uneven (99 experts have more than 64 rows, and each of
// their items reads the weights again), and of a workgroup's 16 to 25 us the item, the
// row list and the first loads take 3, the last sums 1.4 (down: 5, its stores).
// Workgroups that take cell after cell (512, 1,024 or 1,536 of them) were slower.
constexpr int mx4_stages(int nmt) { return nmt >= 4 ? 4 : 6; }

template <typename T, bool GATEUP, bool GATHERED, int NMT>
__device__ __forceinline__ void wide_cells_mx4(const GemmArgs &p, const WorkItem it, int slice,
                                               int kb, int ke, int split,
                                               uint4 *__restrict__ a_lds,
                                               float2 *__restrict__ rinfo, const int *ltok)
{
    constexpr int SW = GATEUP ? 16 * kNpl : 32 * kNpl;  // columns per slice
    const int Kd = p.Kd, N = p.N;
    const int tid = threadIdx.x, lane = tid & 63;
    const int nq = lane & 15, kg = lane >> 4;
    const int col = slice * SW + kNpl * nq;

    // this wavefront's tiles (g, s, w, m) for s in [s0, s1), one K-step apart
    const PackedGeom z = packed_geom(Kd, N, GATEUP, 2, true);
    const int g = slice >> 2, w = slice & 3;
    const int s0 = kb / 32, nsteps = (ke - kb + 31) / 32;
    const size_t tb = ((((size_t)it.expert * z.gs + g) * z.nst + s0) * 4 + w) * z.m * kMx4Tile;
    const uint32_t span = (uint32_t)nsteps * z.step_bytes;
    const bool slice_ok = slice * SW < N;  // a surplus slice reads zeros, no memory
    const uint32_t r0 = (uint32_t)__builtin_amdgcn_readfirstlane(
        (int)(slice_ok ? span - (uint32_t)(w * z.m) * kMx4Tile : 0u));
    const uint32_t r1 = (uint32_t)__builtin_amdgcn_readfirstlane(
        (int)(slice_ok ? span - (uint32_t)(w * z.m + z.m - 1) * kMx4Tile : 0u));
    const char *b0c = static_cast<const char *>(p.B0);
    const __amdgpu_buffer_rsrc_t rb0 = make_rsrc(b0c + tb, r0);
    const __amdgpu_buffer_rsrc_t rb1 =
        GATEUP ? make_rsrc(static_cast<const char *>(p.B1) + tb, r0)
               : make_rsrc(b0c + tb + kMx4Tile, r1);
    // made visible to all wavefronts by the barriers of the K loop
    if (!GATEUP || p.nsplit > 1)
        if (tid < kItemRows) load_rinfo<!GATEUP>(p, it, tid, rinfo, ltok);

    float4_t acc[2][NMT][kNpl];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
            for (int c = 0; c < kNpl; ++c) acc[m][mt][c] = float4_t{0.f, 0.f, 0.f, 0.f};

    constexpr int S = mx4_stages(NMT);
    static_assert(S % 2 == 0, "the row operands alternate between two sets");
    struct Stage {
        Mx4Word b[2];
        uint4 a;
    };
    Stage st[S];
    uint4 af[2][NMT];
    auto load_b = [&](Stage &q, int step) {
        q.b[0] = load_mx4(rb0, (uint32_t)step * z.step_bytes, lane);
        q.b[1] = load_mx4(rb1, (uint32_t)step * z.step_bytes, lane);
    };
    // the first weights are asked for before the item's tokens are known
#pragma unroll
    for (int j = 0; j < S - 1; ++j) load_b(st[j], j);
    __builtin_amdgcn_sched_barrier(0);
    // this thread's share of the A tile: row tid/4, 16-byte chunk tid%4
    const int arow = tid >> 2, achunk = (tid & 3) * 8;
    __amdgpu_buffer_rsrc_t ra;
    uint32_t va;
    if constexpr (GATHERED) {
        ra = make_rsrc(p.A, (uint32_t)((size_t)p.a_rows * Kd * 2));
        const int t = arow < it.nrows ? (ltok ? ltok[arow] : p.stok[it.row0 + arow]) : -1;
        va = (unsigned)t < (unsigned)p.a_rows ? (uint32_t)t * (uint32_t)Kd * 2 : 0x80000000u;
    } else {
        ra = make_rsrc(static_cast<const T *>(p.A) + (size_t)it.row0 * Kd,
                       (uint32_t)((size_t)it.nrows * Kd * 2));
        va = (uint32_t)arow * (uint32_t)Kd * 2;
    }
    auto load_a = [&](Stage &q, int step) {
        q.a = Ld<16>::run(ra, va + (uint32_t)(kb + 32 * step + achunk) * 2, 0u);
    };
    // row operands of a step to its LDS slot; zeros past the K range, where the next
    // row's values (or the next split's) were loaded
    auto put = [&](const Stage &q, int step) {
        a_lds[(step & 1) * kATileU4 + tid] =
            mask4(q.a, kb + 32 * step + achunk < ke ? 0xffffffffu : 0u);
    };
    auto take = [&](uint4 (&a)[NMT], int step) {
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt)
            a[mt] = a_lds[(step & 1) * kATileU4 + (16 * mt + nq) * 4 + kg];
    };
    // step s: its operands in q and a; the loads of step s + S - 1 into qf
    auto step = [&](int s, const Stage &q, const Stage &qn, Stage &qf, const uint4 (&a)[NMT],
                    uint4 (&an)[NMT]) {
        load_b(qf, s + S - 1);
        load_a(qf, s + S - 1);
        __builtin_amdgcn_sched_barrier(0);
        uint4 fb[2];
        fb[0] = mx4_operand<T>(q.b[0], 0);
        put(qn, s + 1);
#pragma unroll
        for (int f = 0; f < 8; ++f) {
            const int m = f & 1, c = f >> 1;
            if (f + 1 < 8) fb[(f + 1) & 1] = mx4_operand<T>(q.b[(f + 1) & 1], (f + 1) >> 1);
#pragma unroll
            for (int mt = 0; mt < NMT; ++mt)
                acc[m][mt][c] = Elt<T>::mfma(a[mt], fb[f & 1], acc[m][mt][c]);
            if (f == 3) {
                __syncthreads();  // step s + 1's rows are in LDS
                take(an, s + 1);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int j = 0; j < S - 1; ++j) load_a(st[j], j);
    __builtin_amdgcn_sched_barrier(0);
    put(st[0], 0);
    __syncthreads();
    take(af[0], 0);
    int s = 0;
    for (; s + S <= nsteps; s += S) {
#pragma unroll
        for (int j = 0; j < S; ++j)
            step(s + j, st[j], st[(j + 1) % S], st[(j + S - 1) % S], af[j & 1], af[(j + 1) & 1]);
    }
#pragma unroll
    for (int j = 0; j < S - 1; ++j)
        if (s + j < nsteps)
            step(s + j, st[j], st[(j + 1) % S], st[(j + S - 1) % S], af[j & 1], af[(j + 1) & 1]);
    store_cells<T, GATEUP, NMT>(p, it, col, kg, acc, rinfo, split);
}

// Tall cells: a run of R consecutive items of one expert (R = 2 is dispatched;
// the R = 4 shape, one column slice over 256 rows, measured slower). The 4
// wavefronts take row block rb = wave % R (item i0 + rb, 64 rows) and column
// slice cs = wave / R of the C = 4/R slices of the workgroup, so the C
// slices' weight tile is loaded once per K-step and shared through LDS by R
// wavefronts each:
//  * producers: the 256 threads split the tile into units of (slice, matrix,
//    MFMA lane); a thread loads RP = KR*C/2 K-rows x 4 columns of its unit,
//    transposes them in registers (16-bit) and writes the MFMA B fragments of
//    that lane to LDS;
//  * consumers: every wavefront reads its slice's fragments from LDS and its
//    own rows' A fragments straight from memory (16-byte loads per lane).
// Every wavefront computes 4 m-tiles (a short last item computes zero rows).
// The weight loads keep the default cache policy here: the other runs of the
// same expert read the same tile, often while it is still in L2.
template <typename T, bool GATEUP, bool GATHERED, int WF, bool DEEP, int R>
__device__ __forceinline__ void tall_cells(const GemmArgs &p, const WorkItem *__restrict__ items,
                                           int i0, int nitems, int g, int j, int kb, int ke,
                                           int split, uint4 *__restrict__ lds,
                                           float2 *__restrict__ rinfo)
{
    constexpr int NPL = kNpl;
    constexpr int ES = sizeof(T);
    constexpr int KR = Elt<T>::KR;
    constexpr int KSTEP = 4 * KR;
    constexpr int NMAT = 2;
    constexpr int NMT = kMT;
    constexpr int C = 4 / R;    // column slices per workgroup
    constexpr int H = 2 / C;    // producer threads per (slice, matrix, lane) unit
    constexpr int RP = KR / H;  // weight rows per producer thread
    constexpr int SW = GATEUP ? 16 * NPL : 32 * NPL;
    constexpr int HALF = GATEUP ? 0 : 16 * NPL;
    constexpr int LB = NPL * ES;
    constexpr int BUF = tall_buf_u4(C);
    static_assert(H * C == 2 && RP * H == KR, "tall cell shape");
    const T *A = static_cast<const T *>(p.A);
    const T *B0 = static_cast<const T *>(p.B0);
    const T *B1 = static_cast<const T *>(p.B1);
    const int Kd = p.Kd, N = p.N;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nq = lane & 15, kg = lane >> 4;

    // consumer role: item i0 + rb of the run, column slice cs
    const int rb = wave % R, cs = wave / R;
    const WorkItem first = items[i0];
    const int expert = first.expert;
    WorkItem it = first;
    if (rb != 0) {
        if (i0 + rb < nitems) it = items[i0 + rb];
        if (i0 + rb >= nitems || it.expert != expert) it.nrows = 0;
    }
    const int col = (4 * g + C * j + cs) * SW + NPL * nq;

    // producer role: unit (slice pcs, matrix pm, lane plu), rows RP*hh.. of it
    const int pcs = C == 1 ? 0 : (wave >> 1);
    const int pm = C == 1 ? (wave >> 1) : (wave & 1);
    const int plu = C == 1 ? ((tid >> 1) & 63) : lane;
    const int hh = C == 1 ? (tid & 1) : 0;
    const int pslice = 4 * g + C * j + pcs;
    // packed: a producer thread copies 4/H whole fragments (fp32: rows) of its unit
    constexpr int PNB = WF == kPacked ? 4 / H : RP;
    __amdgpu_buffer_rsrc_t rbp;
    uint32_t rowb, vpb, bstep;
    if constexpr (WF == kPacked) {
        const PackedGeom z = packed_geom(Kd, N, GATEUP, ES);
        const int s0 = kb / KSTEP, s1 = (ke + KSTEP - 1) / KSTEP;
        const int wp = C * j + pcs, mm = GATEUP ? 0 : pm;  // tile slot in the group
        const size_t tb =
            (((((size_t)expert * z.gs + g) * z.nst + s0) * 4 + wp) * z.m + mm) * z.tile_bytes;
        const uint32_t span = (uint32_t)(s1 - s0) * z.step_bytes;
        const uint32_t pbytes = (uint32_t)__builtin_amdgcn_readfirstlane(
            (int)(pslice * SW >= N ? 0u : span - (uint32_t)(wp * z.m + mm) * z.tile_bytes));
        const char *bb = static_cast<const char *>(GATEUP && pm ? p.B1 : p.B0);
        rbp = make_rsrc(bb + tb, pbytes);
        rowb = 1024;
        vpb = (uint32_t)(hh * PNB) * 1024 + (uint32_t)plu * 16;
        bstep = z.step_bytes;
    } else {
        const size_t wofs = (size_t)expert * Kd * N + (size_t)kb * N;
        const uint32_t kbytes = (uint32_t)((size_t)(ke - kb) * N * ES);
        // pm and pslice are wave-uniform: keep the range and base in SGPRs
        const uint32_t pbytes = (uint32_t)__builtin_amdgcn_readfirstlane((int)(
            pslice * SW >= N ? 0u
                             : (GATEUP || pm == 0) ? kbytes : kbytes - (uint32_t)(HALF * ES)));
        const T *pbase = GATEUP ? (pm ? B1 + wofs : B0 + wofs) : B0 + wofs + pm * HALF;
        rbp = make_rsrc(pbase, pbytes);
        rowb = (uint32_t)N * ES;
        vpb = (uint32_t)(pslice * SW + NPL * (plu & 15)) * ES +
              (uint32_t)(KR * (plu >> 4) + RP * hh) * rowb;
        bstep = (uint32_t)KSTEP * rowb;
    }

    // A: 4 m-tiles of this wavefront's item; lane row 16*mt + nq, K chunk kg
    __amdgpu_buffer_rsrc_t ra;
    uint32_t va[NMT];
    if constexpr (GATHERED) {
        ra = make_rsrc(A, (uint32_t)((size_t)p.a_rows * Kd * ES));
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt) {
            const int rl = 16 * mt + nq;
            const int t = rl < it.nrows ? p.stok[it.row0 + rl] : -1;
            va[mt] = (unsigned)t < (unsigned)p.a_rows ? (uint32_t)t * (uint32_t)Kd * ES : 0x80000000u;
        }
    } else {
        ra = make_rsrc(A + (size_t)it.row0 * Kd, (uint32_t)((size_t)it.nrows * Kd * ES));
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt) va[mt] = (uint32_t)(16 * mt + nq) * (uint32_t)Kd * ES;
    }

    float2 *my_rinfo = rinfo + wave * kItemRows;
    if (!GATEUP || p.nsplit > 1) load_rinfo<!GATEUP>(p, it, lane, my_rinfo);

    float4_t acc[NMAT][NMT][NPL];
#pragma unroll
    for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
            for (int c = 0; c < NPL; ++c) acc[m][mt][c] = float4_t{0.f, 0.f, 0.f, 0.f};

    constexpr int LBB = WF == kPacked ? 16 : LB;
    typedef typename Ld<LBB>::type BT;
    struct Stage {
        BT b[PNB];
        uint4 a[NMT];
    };
    auto load = [&](Stage &st, int k0) {
        const uint32_t vb = vpb + (uint32_t)((k0 - kb) / KSTEP) * bstep;
#pragma unroll
        for (int i = 0; i < PNB; ++i) st.b[i] = Ld<LBB>::run(rbp, vb, (uint32_t)i * rowb);
        // A past the K range masked here (shallow) or at its use (deep), as in
        // the wide cells
        const int ka = k0 + KR * kg;
        const uint32_t am = ka < ke ? 0xffffffffu : 0u;
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt) {
            st.a[mt] = Ld<16>::run(ra, va[mt] + (uint32_t)ka * ES, 0u);
            if constexpr (!DEEP) st.a[mt] = mask4(st.a[mt], am);
        }
    };
    // fragment (or fp32 row) q of lane l of slice s, matrix m in a buffer
    auto frag = [&](int s, int m, int q, int l) { return ((s * NMAT + m) * 4 + q) * 64 + l; };
    auto compute = [&](const Stage &st, int step) {
        uint4 *buf = lds + (step & 1) * BUF;
        const uint32_t am = kb + step * KSTEP + KR * kg < ke ? 0xffffffffu : 0u;
        uint4 a[NMT];
#pragma unroll
        for (int mt = 0; mt < NMT; ++mt) a[mt] = DEEP ? mask4(st.a[mt], am) : st.a[mt];
        if constexpr (WF == kPacked) {
#pragma unroll
            for (int i = 0; i < PNB; ++i) buf[frag(pcs, pm, PNB * hh + i, plu)] = st.b[i];
        } else if constexpr (ES == 2) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t o[RP / 2];
                column_of_rows<RP>(st.b, c, o);
                if constexpr (RP == 8)
                    buf[frag(pcs, pm, c, plu)] = make_uint4(o[0], o[1], o[2], o[3]);
                else
                    reinterpret_cast<uint2 *>(buf)[2 * frag(pcs, pm, c, plu) + hh] =
                        make_uint2(o[0], o[1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < RP; ++i) buf[frag(pcs, pm, RP * hh + i, plu)] = st.b[i];
        }
        __syncthreads();
        if constexpr (ES == 2) {
#pragma unroll
            for (int c = 0; c < NPL; ++c)
#pragma unroll
                for (int m = 0; m < NMAT; ++m) {
                    const uint4 fb = buf[frag(cs, m, c, lane)];
#pragma unroll
                    for (int mt = 0; mt < NMT; ++mt)
                        acc[m][mt][c] = Elt<T>::mfma(a[mt], fb, acc[m][mt][c]);
                }
        } else {
#pragma unroll
            for (int q = 0; q < KR; ++q)
#pragma unroll
                for (int m = 0; m < NMAT; ++m) {
                    const uint4 bq = buf[frag(cs, m, q, lane)];
#pragma unroll
                    for (int c = 0; c < NPL; ++c)
#pragma unroll
                        for (int mt = 0; mt < NMT; ++mt)
                            acc[m][mt][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                lanef(a[mt], q), lanef(bq, c), acc[m][mt][c], 0, 0, 0);
                }
        }
    };

    // register ring depth: 16-bit 4 (one slice) or 3 (two slices) stages;
    // fp32 stages are larger, 2
    constexpr int S = ES == 2 ? (C == 1 ? 4 : 3) : 2;
    const int nsteps = (ke - kb + KSTEP - 1) / KSTEP;
    Stage st[S];
#pragma unroll
    for (int jj = 0; jj < S - 1; ++jj) {  // as in the wide cells
        load(st[jj], kb + jj * KSTEP);
        if constexpr (DEEP) __builtin_amdgcn_sched_barrier(0);
    }
    for (int s = 0; s < nsteps; s += S) {
#pragma unroll
        for (int jj = 0; jj < S; ++jj) {
            load(st[(jj + S - 1) % S], kb + (s + jj + S - 1) * KSTEP);
            __builtin_amdgcn_sched_barrier(0);
            compute(st[jj], s + jj);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    store_cells<T, GATEUP, NMT>(p, it, col, kg, acc, my_rinfo, split);
}

// A wide cell of the item's number of m-tiles. ltok: the item's token rows in LDS
// (ltok[r] for row r), or nullptr: from stok
template <typename T, bool GATEUP, bool GATHERED, int WF, bool DEEP>
__device__ __forceinline__ void single_cell(const GemmArgs &p, const WorkItem it, int g, int kb,
                                            int ke, int split, uint4 *__restrict__ lds,
                                            float2 *__restrict__ rinfo, const int *ltok)
{
    // wave-uniform by construction, so the buffer descriptors live in SGPRs
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slice = g * kWavesPerBlock + wave;
    auto cell = [&](auto nmt) {
        constexpr int NMT = decltype(nmt)::value;
        if constexpr (WF == kMx4)
            wide_cells_mx4<T, GATEUP, GATHERED, NMT>(p, it, slice, kb, ke, split, lds, rinfo, ltok);
        else
            wide_cells<T, GATEUP, GATHERED, WF, DEEP, NMT>(p, it, slice, kb, ke, split, lds, rinfo,
                                                           ltok);
    };
    switch ((it.nrows + 15) >> 4) {  // m-tiles of this item (uniform per workgroup)
    case 1: cell(std::integral_constant<int, 1>()); break;
    case 2: cell(std::integral_constant<int, 2>()); break;
    case 3: cell(std::integral_constant<int, 3>()); break;
    default: cell(std::integral_constant<int, kMT>()); break;
    }
}

// The cell of item i: a tall cell for an item in a run, else a wide cell.
template <typename T, bool GATEUP, bool GATHERED, int WF, bool DEEP>
__device__ __forceinline__ void gemm_cell(const GemmArgs &p, const WorkItem *__restrict__ items,
                                          const WorkItem it, int i, int nitems, int g, int kb,
                                          int ke, int split, uint4 *__restrict__ lds,
                                          float2 *__restrict__ rinfo)
{
    [[maybe_unused]] const int run = it.run & 0xff, j = (it.run >> 8) & 0xff;
    if constexpr (WF == kMx4) {
        // items in runs too: their weights come from L2 the second time, and a wide
        // cell takes less time than a tall one of the same work (down projection of
        // the prefill layer, 64 rows each: 25 against 30 us)
        single_cell<T, GATEUP, GATHERED, WF, DEEP>(p, it, g, kb, ke, split, lds, rinfo, nullptr);
    } else {
        // a run of 4 is taken as two runs of 2 (4-item cells, one column slice of
        // 256 rows each: the skewed long prompt's layer 0.8% slower)
        if (run == 4 && j < 4 && i >= j)
            tall_cells<T, GATEUP, GATHERED, WF, DEEP, 2>(p, items, i - (j & 1), nitems, g, j & 1,
                                                         kb, ke, split, lds, rinfo);
        else if (run == 2 && j < 2 && i >= j)
            tall_cells<T, GATEUP, GATHERED, WF, DEEP, 2>(p, items, i - j, nitems, g, j, kb, ke,
                                                         split, lds, rinfo);
        else
            single_cell<T, GATEUP, GATHERED, WF, DEEP>(p, it, g, kb, ke, split, lds, rinfo,
                                                       nullptr);
    }
}

// One workgroup per (work item, group of 4 column slices, K split).
// WP (gathered gate/up of a call planned here, WavePlan wp): workgroup 0
// writes the plan and the work list for the later kernels (plan_wave_body,
// one wavefront, LDS borrowed from the tiles), workgroups 1-7 have nothing
// to do, and workgroup 8 + b finds the item of its logical block b from the
// ids (wave_plan_item: every item is single, so there are no runs and no list
// to read) and keeps the item's tokens in LDS for its A-operand rows. A
// template instance of its own, so that the other launches' code is
// untouched.
template <typename T, bool GATEUP, bool GATHERED, int WF, bool WP = false>
__global__ __launch_bounds__(256, 2) void k_expert_gemm(const GemmArgs p,
                                                        const int32_t *__restrict__ ctl,
                                                        const WorkItem *__restrict__ items,
                                                        const WavePlan wp)
{
    __shared__ uint4 lds[kLdsU4];
    __shared__ float2 rinfo[kWavesPerBlock * kItemRows];
    constexpr int SW = GATEUP ? 16 * kNpl : 32 * kNpl;  // columns per slice
    constexpr int KSTEP = 4 * Elt<T>::KR;
    const int gs = (p.N + 4 * SW - 1) / (4 * SW);       // column groups per item
    const int per_item = gs * p.nsplit;
    if constexpr (WP) {
        static_assert(GATEUP && GATHERED, "planned here: the gathered gate/up launch only");
        static_assert(2 * kMaxExperts * 4 <= kLdsU4 * 16, "plan counters fit the tile LDS");
        __shared__ int s_tok[kItemRows];
        __shared__ WorkItem s_item;
        __shared__ int s_nb[2];
        if (blockIdx.x < 8) {
            if (blockIdx.x == 0 && threadIdx.x < kWave) {
                int *ls = reinterpret_cast<int *>(lds);
                plan_wave_body(wp.ids, wp.w, wp.nent, wp.E, wp.K, wp.tm, wp.nbits, wp.cnt,
                               wp.eoff, wp.boff, wp.tiles, wp.stok, wp.sw, wp.pos, wp.meta,
                               const_cast<int32_t *>(ctl), const_cast<WorkItem *>(items),
                               wp.max_items, wp.max_rows, 0, ls, ls + kMaxExperts);
            }
            return;  // (no barrier in these workgroups)
        }
        if (threadIdx.x < kWave) {
            int n, b;
            WorkItem w_it;
            wave_plan_item(wp.ids, wp.nent, wp.E, wp.K, wp.tm, wp.nbits, wp.max_rows, per_item,
                           blockIdx.x - 8, &n, &b, &w_it, s_tok);
            if (threadIdx.x == 0) {
                s_nb[0] = n;
                s_nb[1] = b;
                s_item = w_it;
            }
        }
        __syncthreads();
        const int nitems = s_nb[0], lb = s_nb[1];
        if (lb < 0) return;  // whole workgroup, after its only barrier outside the cell
        const WorkItem it = s_item;
        const int rem = lb - (lb / per_item) * per_item;
        const int g = rem / p.nsplit, split = rem - g * p.nsplit;
        const int kb = split * p.split_steps * KSTEP;
        const int ke = min(p.Kd, kb + p.split_steps * KSTEP);
        if (WF == kMx4 || nitems * per_item < kDeepBelowCells)  // (no runs)
            single_cell<T, true, true, WF, true>(p, it, g, kb, ke, split, lds, rinfo, s_tok);
        else
            single_cell<T, true, true, WF, false>(p, it, g, kb, ke, split, lds, rinfo, s_tok);
    } else {
        const int nitems = ctl[0];
        const int ifirst = p.skip_quads ? min(ctl[1], nitems) : 0;
        const int lb = xcd_logical_block((nitems - ifirst) * per_item);
        if (lb < 0) return;  // whole workgroup: no barrier reached
        const int il = lb / per_item;  // item ifirst + il
        const int i = ifirst + il;
        const int rem = lb - il * per_item;
        const int g = rem / p.nsplit, split = rem - g * p.nsplit;
        const int kb = split * p.split_steps * KSTEP;
        const int ke = min(p.Kd, kb + p.split_steps * KSTEP);
        const WorkItem it = items[i];
        // weight-stream depth of the launch: deep when at least half the items
        // are in runs or when the cells do not fill the GPU's workgroup slots,
        // else shallow (the same for every workgroup)
        if (WF == kMx4 || 2 * ctl[2] >= nitems ||
            (nitems - ifirst) * per_item < kDeepBelowCells)
            gemm_cell<T, GATEUP, GATHERED, WF, true>(p, items, it, i, nitems, g, kb, ke, split,
                                                         lds, rinfo);
        else
            gemm_cell<T, GATEUP, GATHERED, WF, false>(p, items, it, i, nitems, g, kb, ke,
                                                          split, lds, rinfo);
    }
}

// ---- launching ---------------------------------------------------------------

inline const int32_t *ctl_of(const void *scratch) { return static_cast<const int32_t *>(scratch); }
inline const WorkItem *items_of(const void *scratch)
{
    return reinterpret_cast<const WorkItem *>(static_cast<const char *>(scratch) + kCtlBytes);
}

inline GemmArgs gemm_args(const FfnShape &z, const void *scratch, bool gateup)
{
    GemmArgs p{};
    p.part = reinterpret_cast<float *>(static_cast<char *>(const_cast<void *>(scratch)) +
                                       z.part_offset);
    p.nsplit = gateup ? z.split_gu : z.split_dn;
    p.split_steps = gateup ? z.steps_gu : z.steps_dn;
    p.plane = gateup ? z.plane_gu : z.plane_dn;
    return p;
}

// the gate/up cells; gathered: rows from x through stok; wp with ids: planned here
template <typename T, int WF>
hipError_t gateup_cells(const GemmArgs &p, int64_t blocks, bool gathered, const void *scratch,
                        const WavePlan *wp, hipStream_t s)
{
    const dim3 grid((unsigned)blocks);
    const WavePlan none{};
    if (gathered && wp && wp->ids)  // planned here: 8 workgroups before the cells'
        hipLaunchKernelGGL((k_expert_gemm<T, true, true, WF, true>), dim3(grid.x + 8), dim3(256),
                           0, s, p, ctl_of(scratch), items_of(scratch), *wp);
    else if (gathered)
        hipLaunchKernelGGL((k_expert_gemm<T, true, true, WF>), grid, dim3(256), 0, s, p,
                           ctl_of(scratch), items_of(scratch), none);
    else
        hipLaunchKernelGGL((k_expert_gemm<T, true, false, WF>), grid, dim3(256), 0, s, p,
                           ctl_of(scratch), items_of(scratch), none);
    return hipGetLastError();
}

template <typename T, int WF>
hipError_t down_cells(const GemmArgs &p, int64_t blocks, const void *scratch, hipStream_t s)
{
    hipLaunchKernelGGL((k_expert_gemm<T, false, false, WF>), dim3((unsigned)blocks), dim3(256), 0,
                       s, p, ctl_of(scratch), items_of(scratch), WavePlan{});
    return hipGetLastError();
}

// the cells of 4-bit weights (ffn_mx4.hip; dtype: the C ABI's code, not fp32); narrow: one
// column slice a workgroup, unsplit
hipError_t gateup_cells_mx4(int dtype, const GemmArgs &p, int64_t blocks, bool narrow,
                            bool gathered, const void *scratch, const WavePlan *wp, hipStream_t s);
hipError_t down_cells_mx4(int dtype, const GemmArgs &p, int64_t blocks, bool narrow,
                          const void *scratch, hipStream_t s);

}  // namespace moe
