// The dense matrix product of gfx950 beside the routed layer, and its gradients:
//   out = act(x W + b) + r          x [T][d], W [d][n], out [T][n]
//   dx = dz W^T, dw = x^T dz, db = sum over the rows of dz
//
// All three products are one kernel, D[m][n] = sum_k A(m, k) B(k, n), whose
// operands lie in memory either with k contiguous ("rows": row i holds A(i, .))
// or with k as the row index ("columns": row k holds B(k, .)):
//   forward  A = x rows,     B = W columns
//   dx       A = dz rows,    B = W rows
//   dw       A = x columns,  B = dz columns
// A workgroup of 4 wavefronts computes a BM x BN tile in K-steps of 128 bytes
// of k (64 values of the 16-bit types, 32 of fp32), whole lines of a row
// operand. LDS holds three steps of A and two of B. A step is four k-groups;
// the fragments of a group are read into registers three groups before its
// matrix instructions, so a step's buffers are read out after its first group,
// and from then on the memory loads of B's step after next and of A's third
// step on go out into them (straight into LDS, no registers). They have until
// the end of the next step's (A: the one after it) first group, which is where
// the only barrier of a step stands. The loads are written in assembly so that
// the compiler does not count them: it would let every LDS read wait for all
// loads in flight. They have no register result; the kernel waits for them
// itself.
// In LDS the 16-byte chunks are permuted so that the reads of a wavefront
// spread over the banks:
//   rows:     chunk c of row r (8 chunks, 128 bytes) sits at c ^ ((r >> 1) & 7)
//   columns:  the columns that a lane group reads together (16 of the 16-bit
//             types, 32 of fp32) are a segment; segment s of row k sits at
//             s ^ 2 (k & 3) (fp32: s ^ ((k >> 2) & 1)), so that the rows that are
//             read together lie in different banks.
// Columns of the 16-bit types are read with the transposing LDS load (4 rows x
// 16 columns per 16 lanes), so no operand is rearranged in memory or registers.
// The matrix instruction is given B's fragment first: a lane then holds 4
// consecutive columns of one output row. The epilogue passes the accumulators
// through LDS, so that a lane finishes and stores 8 consecutive columns and a
// row is written in whole lines (and its code exists once, not per register).
//
// Operands whose rows are not whole 16-byte chunks (a stride or a contiguous
// length that is not a multiple of 8, fp32: 4) are first copied into rows
// padded with zeros in the workspace (k_pad_rows): one pass more over that
// operand, and one kernel for every size. Few tiles over a long reduction are
// cut along k (split); the partial sums, fp32 planes in the workspace, are
// added in split order by a second launch that applies the epilogue, so the
// result does not depend on timing.
//
// What bounds them, measured (times in a stream of calls, bf16 / fp16):
//   32,768 x 2,048 over 4,096     500 us, 1.10 PFLOP/s     power: the matrix cores are
//   8,192 x 4,096 over 2,048      118 us, 1.16 PFLOP/s     busy 59-72 % of the cycles at
//   4,096 x 2,048 over 8,192      114 + 17 us (2 ranges)   a clock that falls from 2.4 to
//                                 2 GHz under them; the same product of zeros takes 0.7
//                                 of the time
//   2,048 x 512 over 2,560        14.5 us, 370 TFLOP/s     operands into LDS: 168 MB for
//                                 256 tiles of 64 x 64, 14 TB/s
//   4 x 2,816 over 704            7.4 us                   one memory round trip after
//                                 another on 44 workgroups: first loads, 4 MB of w, the
//                                 store (an empty kernel of them: 1.4 us in such a trace)
#include "launch.hpp"
#include "mfma.hpp"

namespace moe {

namespace {

constexpr int kStepBytes = 128;  // bytes of k per K-step of a row operand
constexpr int kGroups = 4;       // k-groups of a step

typedef float float16_t __attribute__((ext_vector_type(16)));

// D[32][32] += A[32][16] B[16][32] (fp32: four of k = 2): lane l holds row
// (column) l & 31 of A (B) with k = 8 (l >> 5) .. + 7 (fp32: 4 (l >> 5) .. + 3,
// element j of both operands meeting in the j-th instruction), and of D column
// l & 31, rows 8 q + 4 (l >> 5) .. + 3 in registers 4 q .. 4 q + 3. A wavefront
// alone on its SIMD issues the 32x32 form at full rate, the 16x16 form at 0.6
// of it (2.4 against 1.4 PFLOP/s over the GPU).
// in_place is the same in assembly, with the accumulator in accumulation
// registers: a tile that takes all 256 of them leaves the compiler none to
// move them through, and it then copies accumulators around the instructions.
// Its operands come from LDS reads and its results are first read long after
// (the kernel waits there), so that no wait states are missing.
template <typename T> struct Mma;
template <> struct Mma<_Float16> {
    static __device__ __forceinline__ void run(uint4 a, uint4 b, float16_t &c)
    {
        c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a),
                                                   __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ void in_place(uint4 a, uint4 b, float16_t &c)
    {
#ifdef __HIP_DEVICE_COMPILE__
        asm("v_mfma_f32_32x32x16_f16 %0, %1, %2, %0"
            : "+a"(c)
            : "v"(__builtin_bit_cast(half8_t, a)), "v"(__builtin_bit_cast(half8_t, b)));
#endif
    }
};
template <> struct Mma<__bf16> {
    static __device__ __forceinline__ void run(uint4 a, uint4 b, float16_t &c)
    {
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                    __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ void in_place(uint4 a, uint4 b, float16_t &c)
    {
#ifdef __HIP_DEVICE_COMPILE__
        asm("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0"
            : "+a"(c)
            : "v"(__builtin_bit_cast(bf16x8_t, a)), "v"(__builtin_bit_cast(bf16x8_t, b)));
#endif
    }
};
template <> struct Mma<float> {
    static __device__ __forceinline__ void run(uint4 a, uint4 b, float16_t &c)
    {
        const float4_t x = __builtin_bit_cast(float4_t, a), y = __builtin_bit_cast(float4_t, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[j], y[j], c, 0, 0, 0);
    }
};

}  // namespace

// What the epilogue does with a tile; out_kind / res_kind: element type codes
// of the C ABI (0 fp32, else T).
struct Epilogue {
    const void *bias;      // [N] of T, or null
    const void *residual;  // [M][ldr], or null; may be out itself
    void *out;
    int64_t ldr, ldo;
    int res_f32, out_f32, act;
    int vec;               // rows of out and residual start at 16-byte boundaries
    int plain;             // vec, and no bias, activation or residual
};

struct GemmArg {
    const char *A, *B;
    int64_t lda, ldb;  // bytes per row
    int M, N, K;
    int a_cols, b_cols;  // length of an operand's rows as they lie (whole 16-byte chunks), elements
    int mt, nt;          // tiles
    int split, steps;    // K splits, K-steps per split
    float *part;         // split > 1: partial planes [split][M][pitch]
    int pitch;           // N rounded up to whole chunks of 8
    Epilogue e;
};

namespace {

template <int W> __device__ __forceinline__ void act_all(float (&v)[W], int act)
{
    switch (act) {
    case kActRelu:
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = act_apply(v[i], kActRelu);
        break;
    case kActSilu:
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = act_apply(v[i], kActSilu);
        break;
    case kActGelu:
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = act_apply(v[i], kActGelu);
        break;
    default: break;
    }
}

// columns c .. c + 7 of row r (those below N); c is a multiple of 8. NT: whole
// chunks are stored non-temporally (outputs that are larger than the caches)
template <typename T, bool NT = false>
__device__ __forceinline__ void finish8(const Epilogue &e, int64_t r, int c, int N, float (&v)[8])
{
    const int64_t ro = r * e.ldo + c, rr = r * e.ldr + c;
    const bool whole = e.vec && c + 8 <= N;
    if (e.bias) {
        const T *b = static_cast<const T *>(e.bias) + c;
        if (c + 8 <= N) {
            float q[8];
            load8<T>(b, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += q[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < N) v[i] += to_f32(b[i]);
        }
    }
    act_all<8>(v, e.act);
    if (e.residual) {
        if (whole) {
            float q[8];
            if (e.res_f32)
                load8<float>(static_cast<const float *>(e.residual) + rr, q);
            else
                load8<T>(static_cast<const T *>(e.residual) + rr, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += q[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < N)
                    v[i] += e.res_f32 ? static_cast<const float *>(e.residual)[rr + i]
                                      : to_f32(static_cast<const T *>(e.residual)[rr + i]);
        }
    }
    if (whole) {
        if (e.out_f32)
            store8<float, NT>(static_cast<float *>(e.out) + ro, v);
        else
            store8<T, NT>(static_cast<T *>(e.out) + ro, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < N) {
            if (e.out_f32)
                static_cast<float *>(e.out)[ro + i] = v[i];
            else
                static_cast<T *>(e.out)[ro + i] = from_f32<T>(v[i]);
        }
}

// the same for whole chunks without bias, activation and residual
template <typename T, bool NT>
__device__ __forceinline__ void store_plain(const Epilogue &e, int64_t r, int c, const float (&v)[8])
{
    if (e.out_f32)
        store8<float, NT>(static_cast<float *>(e.out) + r * e.ldo + c, v);
    else
        store8<T, NT>(static_cast<T *>(e.out) + r * e.ldo + c, v);
}

// LDS byte address of a shared object
__device__ __forceinline__ uint32_t lds_at(const void *p)
{
#ifdef __HIP_DEVICE_COMPILE__
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
#else
    (void)p;
    return 0;
#endif
}

// A buffer resource (word 3: raw buffer of the gfx9 family) in two halves: base
// address; range in bytes and that word. A load past the range returns zeros; a
// range of 0 bytes makes every load zeros.
struct Rsrc {
    uint64_t lo, hi;
};
__device__ __forceinline__ Rsrc rsrc_of(const char *base, uint32_t bytes)
{
    return Rsrc{reinterpret_cast<uint64_t>(base) & 0xffffffffffffull,
                (uint64_t)bytes | (0x00020000ull << 32)};
}

// 64 lanes x 16 bytes from the buffer at each lane's `off` to LDS at `to` + 16 lane;
// counted by vmcnt, which the compiler does not know of here. Sets m0, which
// nothing else in these kernels uses (a clobber of it cannot be declared). The
// compiler does not see a buffer load here and keeps no wait states before it:
// a resource word that a vector instruction has just written may be read by a
// scalar move, not by a buffer load, so it goes through s[96:99]; the moves are
// also the wait state that the load needs behind m0.
__device__ __forceinline__ void load_to_lds(uint32_t to, uint32_t off, const Rsrc &r)
{
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_mov_b32 m0, %0\n\ts_mov_b64 s[96:97], %2\n\ts_mov_b64 s[98:99], %3\n\t"
                 "buffer_load_dwordx4 %1, s[96:99], 0 offen lds"
                 :
                 : "s"(to), "v"(off), "s"(r.lo), "s"(r.hi)
                 : "memory", "s96", "s97", "s98", "s99");
#else
    (void)to, (void)off, (void)r;
#endif
}

// One operand's part of a workgroup's tile: ROWS output rows (or columns) of
// it, NTH threads; COL: the operand is in columns form; NF: 32-row fragments
// of a wavefront. Loads of every STRIDE-th K-step are issued in order: advance()
// makes the next one current.
template <typename T, bool COL, int ROWS, int NTH, int NF, int STRIDE = 1>
struct Operand {
    static constexpr int ES = sizeof(T), EPC = 16 / ES, BK = kStepBytes / ES;
    static constexpr int AHEAD = BK * STRIDE;           // values of k per advance()
    static constexpr int BYTES = ROWS * kStepBytes;     // of a step
    static constexpr int CHUNKS = BYTES / 16;
    static constexpr int LOADS = CHUNKS / NTH;          // per thread and step
    static constexpr int CPR = COL ? ROWS / EPC : kStepBytes / 16;  // chunks per LDS row
    static constexpr int SEG = ES == 2 ? 2 : 8;         // columns form: chunks per segment
    static_assert(CHUNKS % NTH == 0, "whole loads");
    static_assert(ROWS >= 64, "the permutation needs 4 (fp32: 2) segments");

    // the permutation of row k's segments (columns form); rows of 64 columns of
    // the 16-bit types are half the banks long: two rows already lie apart
    static __device__ __forceinline__ int seg_xor(int k)
    {
        return ES == 4 ? (k >> 2) & 1 : ROWS == 64 ? k & 2 : (k & 3) << 1;
    }

    const char *base;    // rows form: the tile's first row; columns: the current step's first row
    int64_t ld;
    uint32_t bytes;      // range of the current step's loads
    uint32_t full, tail; // columns form: bytes of a whole step; of a row's part of the tile
    int left;            // values of k from the current step on
    int kc;              // rows form: the k within a step of this thread's chunks
    uint32_t off[LOADS];
    uint32_t at[COL ? NF : kGroups];  // LDS byte of this lane's fragments in a buffer

    // K: values of k that the operand holds (rows form: a multiple of EPC); the
    // first step starts at k0
    __device__ __forceinline__ void init(const char *p, int64_t ld_, int first, int total, int K,
                                         int k0, int tid, int frag0)
    {
        ld = ld_;
        left = K - k0 + AHEAD;  // (advance() comes before the first step)
        const int have = min(ROWS, total - first);
        kc = 0;
        if (COL) {
            base = p + (int64_t)first * ES + ((int64_t)k0 - AHEAD) * ld;
            tail = (uint32_t)(have * ES);
            full = (uint32_t)((BK - 1) * ld) + tail;
        } else {
            base = p + (int64_t)first * ld;
            bytes = (uint32_t)((have - 1) * ld) + (uint32_t)(K * ES);
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int q = i * NTH + tid;
            const int r = q / CPR, c = q % CPR;
            if (COL) {
                const int lc = ((c / SEG) ^ seg_xor(r)) * SEG + c % SEG;
                off[i] = lc * EPC < have ? (uint32_t)r * (uint32_t)ld + (uint32_t)lc * 16u : kOutside;
            } else {
                const int lc = c ^ ((r >> 1) & 7);  // the same for every i
                kc = lc * EPC;
                off[i] = r < have ? (uint32_t)r * (uint32_t)ld + (uint32_t)lc * 16u +
                                        (uint32_t)((k0 - AHEAD) * ES)
                                  : kOutside;
            }
        }
        const int lane = tid & 63;
        if (!COL) {
            const int r = frag0 * 32 + (lane & 31);
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
                at[g] = (uint32_t)(r * kStepBytes + ((2 * g + (lane >> 5)) ^ ((r >> 1) & 7)) * 16);
        } else {
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                if (ES == 2) {
                    const int k = 8 * (lane >> 5) + ((lane >> 2) & 3);
                    const int seg = (2 * (frag0 + i) + ((lane >> 4) & 1)) ^ seg_xor(k);
                    at[i] = (uint32_t)((k * ROWS + seg * 16) * 2 + (lane & 3) * 8);
                } else {
                    const int k = 4 * (lane >> 5);
                    at[i] = (uint32_t)((k * ROWS + ((frag0 + i) ^ seg_xor(k)) * 32 + (lane & 31)) * 4);
                }
            }
        }
    }

    __device__ __forceinline__ void advance()
    {
        left -= AHEAD;
        if (COL) {
            base += (int64_t)AHEAD * ld;
            bytes = left >= BK ? full : left > 0 ? (uint32_t)((left - 1) * ld) + tail : 0u;
        } else {
            // (a row past the operand's end stays outside: the range ends below 2^31)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) off[i] += kStepBytes * STRIDE;
        }
    }

    // the i-th load of the current step into the buffer at `to`; k past the end reads zeros
    __device__ __forceinline__ void issue(uint32_t to, int i, int wave) const
    {
        const bool cut = !COL && kc >= left;
        load_to_lds(to + (uint32_t)(i * NTH + wave * 64) * 16u, cut ? kOutside : off[i],
                    rsrc_of(base, bytes));
    }

    // fragment i of this wavefront, k-group g, from the buffer at L (LDS byte)
    __device__ __forceinline__ uint4 frag(uint32_t L, int i, int g) const
    {
#ifdef __HIP_DEVICE_COMPILE__
        if constexpr (!COL) {
            typedef uint32_t u4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) const u4 *p;
            const u4 v = ((p)(uintptr_t)(L + at[g]))[i * 2 * kStepBytes];
            return make_uint4(v[0], v[1], v[2], v[3]);
        } else if constexpr (ES == 2) {
            typedef short s4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s4 *p;
            const p q = (p)(uintptr_t)(L + at[i]) + g * 4 * ROWS;  // 16 rows per group
            const s4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(q);
            const s4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16(q + ROWS);  // 4 rows on
            const uint2 a = __builtin_bit_cast(uint2, v), b = __builtin_bit_cast(uint2, w);
            return make_uint4(a.x, a.y, b.x, b.y);
        } else {
            typedef __attribute__((address_space(3))) const uint32_t *p;
            const p q = (p)(uintptr_t)(L + at[i]) + g * 8 * ROWS;
            return make_uint4(q[0], q[ROWS], q[2 * ROWS], q[3 * ROWS]);
        }
#else
        return make_uint4(0, 0, 0, 0);
#endif
    }
};

// WM x WN = 4 wavefronts, each (BM / WM) x (BN / WN) of the tile
template <typename T, bool AC, bool BC, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(256, (BM + BN > 256 ? 1 : 2)) void k_gemm(const GemmArg p)
{
    constexpr int NTH = WM * WN * 64, BK = kStepBytes / (int)sizeof(T);
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
    constexpr bool BIG = TM * TN == 16;  // accumulators take all accumulation registers
    typedef Operand<T, AC, BM, NTH, TM> OpA;
    typedef Operand<T, BC, BN, NTH, TN> OpB;
    constexpr uint32_t LDS_BYTES = 3 * OpA::BYTES + 2 * OpB::BYTES;
    __shared__ uint4 lds[LDS_BYTES / 16];
    static_assert(NTH == 256 && 3 * OpA::LOADS + 2 * OpB::LOADS < 64, "4 wavefronts; vmcnt has 6 bits");
    const int lb = xcd_logical_block(p.mt * p.nt * p.split);
    if (lb < 0) return;  // whole workgroup: no barrier reached
    const int tile = lb / p.split, split = lb - tile * p.split;
    // 8 rows of tiles at a time, so that the tiles that one XCD works on share
    // both operands
    const int band = tile / (8 * p.nt), in = tile - band * 8 * p.nt;
    const int bh = min(8, p.mt - band * 8);
    const int tn = in / bh, tm = band * 8 + in - tn * bh;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave - wm * WN;
    const int s0 = split * p.steps;
    const int s1 = min(s0 + p.steps, (p.K + BK - 1) / BK);

    OpA a;
    OpB b;
    // (the rows of a row operand hold k up to its padded length)
    a.init(p.A, p.lda, tm * BM, AC ? p.a_cols : p.M, AC ? p.K : p.a_cols, s0 * BK, tid, wm * TM);
    b.init(p.B, p.ldb, tn * BN, BC ? p.b_cols : p.N, BC ? p.K : p.b_cols, s0 * BK, tid, wn * TN);

    float16_t acc[TM][TN];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    };

    // LDS: three steps of A, then two of B
    const uint32_t base = lds_at(lds), base_b = base + 3 * OpA::BYTES;
    auto load_a = [&](uint32_t to, int i) {
        if (i == 0) a.advance();
        a.issue(to, i, wave);
    };
    auto load_b = [&](uint32_t to, int i) {
        if (i == 0) b.advance();
        b.issue(to, i, wave);
    };
    // fragments of the four k-groups, read in the order in which they are needed
    uint4 fa[kGroups][TM], fb[kGroups][TN];
    auto read = [&](uint32_t la, uint32_t lb_, int g, int q) {
        if (q == 0 || q > TN)
            fa[g][q == 0 ? 0 : q - TN] = a.frag(la, q == 0 ? 0 : q - TN, g);
        else
            fb[g][q - 1] = b.frag(lb_, q - 1, g);
    };
    // matrix instructions of k-group g; between them the fragments of the group
    // three further on, from la and lb_, and the memory loads: B's of the step
    // after next in group 1, A's of the third step on in groups 2 and 3
    constexpr int MMAS = TM * TN, GAP = MMAS / (TM + TN);
    static_assert(GAP * (TM + TN) == MMAS, "");
    auto group = [&](int g, uint32_t la, uint32_t lb_, uint32_t ta, uint32_t tb) {
#pragma unroll
        for (int q = 0; q < MMAS; ++q) {
            if (q % GAP == 0) read(la, lb_, (g + 3) % kGroups, q / GAP);
            if (g == 1)
#pragma unroll
                for (int i = q * OpB::LOADS / MMAS; i < (q + 1) * OpB::LOADS / MMAS; ++i)
                    load_b(tb, i);
            if (g >= 2) {
                const int at = (g - 2) * MMAS + q;
#pragma unroll
                for (int i = at * OpA::LOADS / (2 * MMAS); i < (at + 1) * OpA::LOADS / (2 * MMAS); ++i)
                    load_a(ta, i);
            }
            if constexpr (BIG)
                Mma<T>::in_place(fb[g][q % TN], fa[g][q / TN], acc[q / TN][q % TN]);
            else
                Mma<T>::run(fb[g][q % TN], fa[g][q / TN], acc[q / TN][q % TN]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    {  // (every range of k has a step)
        auto all_a = [&](uint32_t to) {
#pragma unroll
            for (int i = 0; i < OpA::LOADS; ++i) load_a(to, i);
        };
        auto all_b = [&](uint32_t to) {
#pragma unroll
            for (int i = 0; i < OpB::LOADS; ++i) load_b(to, i);
        };
        all_a(base);
        all_b(base_b);
        all_a(base + OpA::BYTES);
        all_b(base_b + OpB::BYTES);
        all_a(base + 2 * OpA::BYTES);
        clear();  // (while the loads are on their way)
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier"
                     :
                     : "n"(2 * OpA::LOADS + OpB::LOADS)
                     : "memory");
#pragma unroll
        for (int g = 0; g < 3; ++g)
#pragma unroll
            for (int q = 0; q < TM + TN; ++q) read(base, base_b, g, q);
        uint32_t a0 = base, a1 = base + OpA::BYTES, a2 = base + 2 * OpA::BYTES;
        uint32_t b0 = base_b, b1 = base_b + OpB::BYTES;
        // A step past the end of k reads zeros.
        for (int s = s0; s < s1; ++s) {
            group(0, a0, b0, 0, 0);
            // this step's buffers are read out by this wavefront, and all loads but
            // those of A two steps on have landed; with the barrier, by and for everyone
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(OpA::LOADS) : "memory");
            __builtin_amdgcn_sched_barrier(0);
            group(1, a1, b1, a0, b0);
            group(2, a1, b1, a0, b0);
            group(3, a1, b1, a0, b0);
            const uint32_t x = a0, y = b0;
            a0 = a1;
            a1 = a2;
            a2 = x;
            b0 = b1;
            b1 = y;
        }
        // nothing in flight into LDS, and every wavefront done with it; the last
        // matrix results readable
        asm volatile("s_nop 15\n\ts_nop 15\n\ts_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }

    const int row0 = tm * BM + wm * TM * 32, col0 = tn * BN + wn * TN * 32;
    if (p.split > 1) {
        float *plane = p.part + (int64_t)split * p.M * p.pitch;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int m = row0 + i * 32 + (lane & 31);
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = col0 + j * 32 + 8 * q + 4 * (lane >> 5);
                    const float16_t &c = acc[i][j];
                    if (m < p.M && n < p.pitch)
                        *reinterpret_cast<float4_t *>(plane + (int64_t)m * p.pitch + n) =
                            float4_t{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
                }
        }
        return;
    }
    // Each wavefront's own part of LDS holds 32 of its rows; rows are padded by
    // 4 floats, which spreads the rows of a store over the banks.
    constexpr int COLS = TN * 32, PITCH = COLS + 4, LPR = COLS / 8;
    static_assert(32 * PITCH * 4 * 4 <= (int)LDS_BYTES, "fits");
    float *mine = reinterpret_cast<float *>(lds) + wave * (32 * PITCH);
#pragma unroll
    for (int h = 0; h < TM; ++h) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float16_t &c = acc[h][j];
                *reinterpret_cast<float4_t *>(mine + (lane & 31) * PITCH + j * 32 + 8 * q +
                                              4 * (lane >> 5)) =
                    float4_t{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
            }
        // (LDS operations of one wavefront stay in order; the compiler keeps it)
        asm volatile("" ::: "memory");
        const int n = col0 + (lane % LPR) * 8;
        auto one = [&](int r, bool plain) __attribute__((always_inline)) {
            const int m = row0 + h * 32 + r;
            if (m >= p.M || n >= p.N) return;
            float v[8];
            load8<float>(mine + r * PITCH + (lane % LPR) * 8, v);
            if (plain)
                store_plain<T, BIG>(p.e, m, n, v);
            else
                finish8<T, BIG>(p.e, m, n, p.N, v);
        };
        if (p.e.plain && n + 8 <= p.N) {
#pragma unroll 4
            for (int r = lane / LPR; r < 32; r += 64 / LPR) one(r, true);
        } else {
#pragma unroll 2
            for (int r = lane / LPR; r < 32; r += 64 / LPR) one(r, false);
        }
        asm volatile("" ::: "memory");
    }
}

// 64 x 64 tiles for products that are too small to fill the GPU with larger
// ones: every wavefront computes the whole tile over one k-group of each step
// (wavefront w group w), and the partial tiles are added, in order, through LDS
// at the end. Four buffers hold four steps; the loads of step s + 3 go out when
// step s is read. Such a product waits for memory and for its barriers, not for
// the matrix cores: two of these workgroups run on a CU, or, where there is no
// more than one for every CU, one of TEAMS = 2 times 4 wavefronts, each with
// buffers of its own and every other step (2,048 x 512 outputs over 2,560
// values of k: 17 us with 256 workgroups of one team).
constexpr int kSmall = 64, kSmallBuffers = 4;
template <typename T, bool AC, bool BC, int TEAMS>
__global__ __launch_bounds__(256 * TEAMS, 2) void k_gemm_small(const GemmArg p)
{
    constexpr int NTH = 256, BK = kStepBytes / (int)sizeof(T), NB = kSmallBuffers;
    typedef Operand<T, AC, kSmall, NTH, 2, TEAMS> OpA;
    typedef Operand<T, BC, kSmall, NTH, 2, TEAMS> OpB;
    constexpr uint32_t BUF = OpA::BYTES + OpB::BYTES;
    constexpr int LOADS = OpA::LOADS + OpB::LOADS;
    __shared__ uint4 lds[TEAMS * NB * BUF / 16];
    const int lb = xcd_logical_block(p.mt * p.nt * p.split);
    if (lb < 0) return;  // whole workgroup: no barrier reached
    const int tile = lb / p.split, split = lb - tile * p.split;
    const int tm = tile / p.nt, tn = tile - tm * p.nt;
    const int lane = threadIdx.x & 63;
    const int team = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    const int tid = threadIdx.x & 255;  // in the team
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // (whole rounds of the teams: a step past the end of k reads zeros)
    const int s0 = split * p.steps;
    const int s1 = min(s0 + p.steps, (p.K + BK - 1) / BK);
    const int rounds = (s1 - s0 + TEAMS - 1) / TEAMS;
    const int k0 = (s0 + team) * BK;
    OpA a;
    OpB b;
    a.init(p.A, p.lda, tm * kSmall, AC ? p.a_cols : p.M, AC ? p.K : p.a_cols, k0, tid, 0);
    b.init(p.B, p.ldb, tn * kSmall, BC ? p.b_cols : p.N, BC ? p.K : p.b_cols, k0, tid, 0);
    float16_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    const uint32_t base = lds_at(lds) + (uint32_t)team * NB * BUF;
    auto next = [&](uint32_t q) { return q + BUF == base + NB * BUF ? base : q + BUF; };
    auto load = [&](uint32_t to) {
        a.advance();
        b.advance();
#pragma unroll
        for (int i = 0; i < OpA::LOADS; ++i) a.issue(to, i, wave);
#pragma unroll
        for (int i = 0; i < OpB::LOADS; ++i) b.issue(to + OpA::BYTES, i, wave);
    };
    {  // (every range of k has a step)
        uint32_t rd = base, wr = base;
#pragma unroll
        for (int q = 0; q < NB - 1; ++q) {
            load(wr);
            wr = next(wr);
        }
        for (int s = 0; s < rounds; ++s) {
            // this step has landed and the one before is read out; for everyone
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier"
                         :
                         : "n"((NB - 2) * LOADS)
                         : "memory");
            load(wr);
            wr = next(wr);
            uint4 fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // (the group is the wavefront's: uniform, so a scalar branch)
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
                    if (g == wave) {
                        fa[i] = a.frag(rd, i, g);
                        fb[i] = b.frag(rd + OpA::BYTES, i, g);
                    }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) Mma<T>::run(fb[j], fa[i], acc[i][j]);
            rd = next(rd);
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    // 32 rows at a time: the wavefronts' parts side by side, then one thread per
    // 8 columns of a row
    constexpr int PITCH = kSmall + 4, PART = 32 * PITCH, PARTS = 4 * TEAMS;
    static_assert(PARTS * PART * 4 <= (int)(TEAMS * NB * BUF), "fits");
    float *f = reinterpret_cast<float *>(lds);
    float *plane = p.part + (int64_t)split * p.M * p.pitch;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (i) __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float16_t &c = acc[i][j];
                *reinterpret_cast<float4_t *>(f + (team * 4 + wave) * PART + (lane & 31) * PITCH +
                                              j * 32 + 8 * q + 4 * (lane >> 5)) =
                    float4_t{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
            }
        __syncthreads();
        const int r = tid >> 3, m = tm * kSmall + i * 32 + r, n = tn * kSmall + (tid & 7) * 8;
        if (team == 0 && m < p.M && n < p.N) {
            float v[8] = {};
#pragma unroll
            for (int w = 0; w < PARTS; ++w) {
                float q[8];
                load8<float>(f + w * PART + r * PITCH + (tid & 7) * 8, q);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += q[k];
            }
            if (p.split > 1) {
                store8<float>(plane + (int64_t)m * p.pitch + n, v);
            } else {
                finish8<T>(p.e, m, n, p.N, v);
            }
        }
    }
}

// The split products' partial planes added in split order, then the epilogue:
// one thread per 8 columns of a row. Bound by reading the planes (9 of 2,560 x
// 504: 46 MB in 10 us, 4.6 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void k_gemm_reduce(const float *__restrict__ part, int M, int N,
                                                     int pitch, int split, const Epilogue e)
{
    const int per = pitch / 8;
    const int64_t total = (int64_t)M * per, plane = (int64_t)M * pitch;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < total;
         q += (int64_t)gridDim.x * 256) {
        const int64_t r = q / per;
        const int c = (int)(q - r * per) * 8;
        float v[8] = {};
        const float *s = part + r * pitch + c;
#pragma unroll 4
        for (int i = 0; i < split; ++i) {
            float z[8];
            load8<float>(s + i * plane, z);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += z[j];
        }
        finish8<T>(e, r, c, N, v);
    }
}

// dst [R][ldd] = src [R][C] (row stride lds), columns C .. ldd zero; in units of
// `unit` bytes: the element, or 2 or 4 of the 16-bit types (2 of fp32) together
// where a row is whole units and starts at one.
struct PadJob {
    const char *src;
    char *dst;
    int64_t lds, R;
    int C, ldd, unit;
    int blocks;  // workgroups of the launch that take it
};
// an operation's operands, in one launch
struct PadJobs {
    PadJob j[3];
    int n;
};

// one 16-byte chunk of dst per thread
template <typename U> __device__ __forceinline__ void pad_rows(const PadJob &p, int64_t first)
{
    constexpr int EPC = 16 / sizeof(U);
    const U *src = reinterpret_cast<const U *>(p.src);
    U *dst = reinterpret_cast<U *>(p.dst);
    const int per = p.ldd / EPC;
    for (int64_t q = first; q < p.R * per; q += (int64_t)p.blocks * 256) {
        const int64_t r = q / per;
        const int c = (int)(q - r * per) * EPC;
        typedef U vec __attribute__((ext_vector_type(EPC)));
        vec v;
#pragma unroll
        for (int i = 0; i < EPC; ++i) v[i] = c + i < p.C ? src[r * p.lds + c + i] : U(0);
        *reinterpret_cast<vec *>(dst + r * p.ldd + c) = v;
    }
}

// Bound by memory: 32,768 and 2,560 rows of 500 (71 MB in and out) 13.6 us, 5.2 TB/s
// (two launches: 18 us; 509 x 1,003 and 1,003 x 517 of fp32: 5.8 us, two launches 7.6).
__global__ __launch_bounds__(256) void k_pad_rows(const PadJobs all)
{
    int job = 0, block = blockIdx.x;
    while (job + 1 < all.n && block >= all.j[job].blocks) block -= all.j[job++].blocks;
    const PadJob &p = all.j[job];
    const int64_t first = (int64_t)block * 256 + threadIdx.x;
    if (p.unit == 8)
        pad_rows<uint64_t>(p, first);
    else if (p.unit == 4)
        pad_rows<uint32_t>(p, first);
    else
        pad_rows<uint16_t>(p, first);
}

// Column sums of dz [rows][n]: a workgroup adds `per` rows from blockIdx.y * per
// on, over 256 columns: 32 threads of 8 columns, 8 of every 8th row, joined in
// order through LDS. Its sums go to part [gridDim.y][n], or with one block of
// rows straight into db. VEC: rows are whole 16-byte chunks. Bound by memory, with
// a launch of its own: 8,192 x 2,048 of bf16 (34 MB) 7 us, 4.8 TB/s, and 4.5 us for the join.
constexpr int kSumCols = 256;
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void k_colsum(const T *__restrict__ dz, int64_t ld, int rows,
                                                int n, int per, float *__restrict__ part,
                                                void *__restrict__ db, int db_f32)
{
    __shared__ float s[8][kSumCols];
    const int cg = threadIdx.x & 31, rg = threadIdx.x >> 5;
    const int c = blockIdx.x * kSumCols + cg * 8;
    const int64_t r0 = (int64_t)blockIdx.y * per, r1 = r0 + per < rows ? r0 + per : rows;
    float v[8] = {};
    if (c < n)
#pragma unroll 4
        for (int64_t r = r0 + rg; r < r1; r += 8) {
            const T *p = dz + r * ld + c;
            float q[8];
            // (fp32 rows of whole chunks may end 4 columns into these 8)
            if (VEC && (sizeof(T) == 2 || c + 8 <= n)) {
                load8<T>(p, q);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] = c + i < n ? to_f32(p[i]) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += q[i];
        }
    store8<float>(&s[rg][cg * 8], v);
    __syncthreads();
    const int m = blockIdx.x * kSumCols + threadIdx.x;
    if (m >= n) return;
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) t += s[q][threadIdx.x];
    if (gridDim.y > 1)
        part[(int64_t)blockIdx.y * n + m] = t;
    else if (db_f32)
        static_cast<float *>(db)[m] = t;
    else
        static_cast<T *>(db)[m] = from_f32<T>(t);
}

// the blocks' sums added: 32 columns a workgroup, 8 threads each
template <typename T>
__global__ __launch_bounds__(256) void k_colsum_join(const float *__restrict__ part, int blocks,
                                                     int n, void *__restrict__ db, int db_f32)
{
    __shared__ float s[8][32];
    const int cg = threadIdx.x & 31, bg = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cg;
    float v = 0.f;
    if (c < n)
#pragma unroll 8
        for (int b = bg; b < blocks; b += 8) v += part[(int64_t)b * n + c];
    s[bg][cg] = v;
    __syncthreads();
    if (bg || c >= n) return;
    v = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) v += s[q][cg];
    if (db_f32)
        static_cast<float *>(db)[c] = v;
    else
        static_cast<T *>(db)[c] = from_f32<T>(v);
}

// ---- host side ---------------------------------------------------------------

int elem_size(int dtype) { return dtype == 0 ? 4 : 2; }
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Product {
    int64_t mt, nt;
    int tile;  // 64, 128 or 256 rows and columns
    int split, steps;
    int64_t part_bytes;
};

// Estimated microseconds of M x N outputs over `steps` K-steps in tiles of
// `tile`, cut into `split` along k. A workgroup alone on its CU takes c per
// step, two of them together c2 each; `fixed` is the launch with the first
// loads and the last stores. The constants are fits to measurements on the
// shapes named (tile 64 / 128 / 256, best split, 16-bit types):
//   4 x 2,816 over 704             6.5 /  7.8 / 12
//   64 x 512 over 2,560            9.7 / 10.5 / 16
//   1,024 x 1,024 over 1,024       8.6 / 11.7 / 27
//   2,048 x 512 over 2,560        14.9 / 18.5 / 28
//   512 x 2,048 over 4,096          26 /   22 / 32
//   2,048 x 2,048 over 2,048        38 /   26 / 42
//   2,560 x 512 over 32,768        159 /  112 / 95
//   32,768 x 2,048 over 4,096        - /  555 / 485
// and, in fp32 (bound by the matrix cores), 512 x 512 over 1,024: 14.8 / 21,
// 2,048 x 2,048 over 2,048: 164 / 134. The estimate names each row's fastest, but is
// off by up to a fifth for it, and twice by more than the choice turns on: 512 x
// 2,048 over 4,096 is estimated at 23.7 / 23.4 in tiles of 64 / 128, 2,560 x 512 over
// 32,768 at 105 / 104 in tiles of 128 / 256. Sizes near such a border may get the
// slower tile.
double product_us(int64_t M, int64_t N, int64_t steps, int dtype, int tile, int64_t split)
{
    const double wgs = (double)(div_up(M, tile) * div_up(N, tile) * split);
    const double n = (double)div_up(steps, split);
    const double full = wgs < 256 ? wgs / 256 : 1;  // share of the CUs (their power and L2)
    double t;
    if (tile == 256) {
        t = 5 + (double)div_up((int64_t)wgs, 256) * (4 + n * (0.9 + 0.8 * full * full));
    } else {
        const double c = dtype == 0 ? (tile == 64 ? 0.6 : 1.9)
                         : tile == 64 ? 0.2 + 0.1 * full : 0.42 + 0.12 * full;
        const double c2 = dtype == 0 ? 2 * c : tile == 64 ? 0.5 : 1.1;
        t = (tile == 64 ? 4.5 : 6) +
            (wgs <= 256 ? n * c : (double)div_up((int64_t)wgs, 512) * (1 + n * c2));
    }
    if (split > 1) t += 2 + (double)split * (double)M * (double)N * 8 / 5e6;
    return t;
}

Product product_of(int64_t M, int64_t N, int64_t K, int dtype)
{
    const int64_t steps = div_up(K, kStepBytes / elem_size(dtype));
    Product z{};
    double best = 0;
    for (int tile = 64; tile <= (dtype == 0 ? 128 : 256); tile *= 2) {
        const int64_t mt = div_up(M, tile), nt = div_up(N, tile);
        for (int64_t s = 1; s <= 16; ++s) {
            // splits of at least two steps, of a product that does not fill the GPU
            if (s > 1 && (2 * s > steps || mt * nt * s > (tile == 256 ? 256 : 512))) break;
            const double t = product_us(M, N, steps, dtype, tile, s);
            if (z.tile && t >= best) continue;
            best = t;
            z.mt = mt;
            z.nt = nt;
            z.tile = tile;
            z.split = (int)s;
        }
    }
    z.steps = (int)up(div_up(steps, z.split), 2);  // (whole rounds of two teams)
    z.split = (int)div_up(steps, z.steps);
    z.part_bytes = z.split > 1 ? up((int64_t)z.split * M * up(N, 8) * 4, 256) : 0;
    return z;
}

// a row-major [R][C] operand as the kernels read it: its padded copy's place
struct Padded {
    bool copy;
    int64_t cols, bytes;  // row length of the copy; its size
};

Padded padded(int64_t R, int64_t C, int64_t ld, int dtype)
{
    const int64_t epc = 16 / elem_size(dtype);
    Padded z;
    z.copy = C % epc || ld % epc;
    z.cols = up(C, epc);
    z.bytes = z.copy ? up(R * z.cols * elem_size(dtype), 256) : 0;
    return z;
}

struct Matrix {
    const char *p;
    int64_t ld;  // bytes
    int cols;
};

// the operand where it lies, or where its padded copy will be, which `jobs` then makes
Matrix place(const void *src, int64_t R, int64_t C, int64_t ld, int dtype, char *dst, PadJobs *jobs)
{
    const Padded z = padded(R, C, ld, dtype);
    const int es = elem_size(dtype);
    if (!z.copy) return Matrix{static_cast<const char *>(src), ld * es, (int)z.cols};
    PadJob &p = jobs->j[jobs->n++];
    p.unit = C * es % 8 == 0 && ld * es % 8 == 0 ? 8 : C * es % 4 == 0 && ld * es % 4 == 0 ? 4 : 2;
    const int64_t per = p.unit / es, blocks = div_up(R * (z.cols * es / 16), 256);
    p.src = static_cast<const char *>(src);
    p.dst = dst;
    p.lds = ld / per;
    p.R = R;
    p.C = (int)(C / per);
    p.ldd = (int)(z.cols / per);
    p.blocks = (int)(blocks < 8192 ? blocks : 8192);
    return Matrix{dst, z.cols * es, (int)z.cols};
}

hipError_t launch_pads(const PadJobs &jobs, hipStream_t s)
{
    if (!jobs.n) return hipSuccess;
    int blocks = 0;
    for (int i = 0; i < jobs.n; ++i) blocks += jobs.j[i].blocks;
    hipLaunchKernelGGL(k_pad_rows, dim3(blocks), dim3(256), 0, s, jobs);
    return hipGetLastError();
}

template <typename T, bool AC, bool BC>
hipError_t launch_product(const Matrix &A, const Matrix &B, int M, int N, int K, const Product &z,
                          float *part, const Epilogue &e, hipStream_t s)
{
    GemmArg g;
    g.A = A.p;
    g.B = B.p;
    g.lda = A.ld;
    g.ldb = B.ld;
    g.M = M;
    g.N = N;
    g.K = K;
    g.a_cols = A.cols;
    g.b_cols = B.cols;
    g.mt = (int)z.mt;
    g.nt = (int)z.nt;
    g.split = z.split;
    g.steps = z.steps;
    g.part = part;
    g.pitch = (int)up(N, 8);
    g.e = e;
    g.e.plain = e.vec && !e.bias && !e.residual && e.act == kActNone;
    const dim3 grid((unsigned)up(z.mt * z.nt * z.split, 8)), block(256);
    if (z.tile == kSmall) {
        if (z.mt * z.nt * z.split <= 256)
            hipLaunchKernelGGL((k_gemm_small<T, AC, BC, 2>), grid, dim3(512), 0, s, g);
        else
            hipLaunchKernelGGL((k_gemm_small<T, AC, BC, 1>), grid, block, 0, s, g);
    } else if constexpr (sizeof(T) == 2) {
        if (z.tile == 256)
            hipLaunchKernelGGL((k_gemm<T, AC, BC, 256, 256, 2, 2>), grid, block, 0, s, g);
        else
            hipLaunchKernelGGL((k_gemm<T, AC, BC, 128, 128, 2, 2>), grid, block, 0, s, g);
    } else {
        hipLaunchKernelGGL((k_gemm<T, AC, BC, 128, 128, 2, 2>), grid, block, 0, s, g);
    }
    if (z.split > 1) {
        const int64_t parts = (int64_t)M * (g.pitch / 8);
        const dim3 rgrid((unsigned)(parts / 256 + 1 < 8192 ? parts / 256 + 1 : 8192));
        hipLaunchKernelGGL(k_gemm_reduce<T>, rgrid, dim3(256), 0, s, part, M, N, g.pitch, z.split, e);
    }
    return hipGetLastError();
}

// rows that start at 16-byte boundaries (p itself is 16-byte aligned)
bool rows_aligned(const void *p, int64_t ld, int es) { return !p || ld * es % 16 == 0; }

template <typename T>
hipError_t linear_t(const LinearCall &c, char *ws, hipStream_t s)
{
    const LinearSpace z = linear_space(c.T, c.d, c.n, c.ldx, c.ldw, c.dtype);
    const int es = elem_size(c.dtype);
    PadJobs jobs{};
    const Matrix X = place(c.x, c.T, c.d, c.ldx, c.dtype, ws + z.x, &jobs);
    const Matrix W = place(c.w, c.d, c.n, c.ldw, c.dtype, ws + z.w, &jobs);
    const hipError_t rc = launch_pads(jobs, s);
    if (rc != hipSuccess) return rc;
    Epilogue e;
    e.bias = c.bias;
    e.residual = c.residual;
    e.out = c.out;
    e.ldr = c.ldr;
    e.ldo = c.ldo;
    e.res_f32 = c.res_dtype == 0;
    e.out_f32 = c.out_dtype == 0;
    e.act = c.act;
    e.vec = rows_aligned(c.out, c.ldo, e.out_f32 ? 4 : es) &&
            rows_aligned(c.residual, c.ldr, e.res_f32 ? 4 : es);
    return launch_product<T, false, true>(X, W, c.T, c.n, c.d,
                                          product_of(c.T, c.n, c.d, c.dtype),
                                          reinterpret_cast<float *>(ws + z.part), e, s);
}

template <typename T>
hipError_t linear_backward_t(const LinearBackwardCall &c, char *ws, hipStream_t s)
{
    const LinearBackwardSpace z = linear_backward_space(
        c.T, c.d, c.n, c.ldx, c.ldw, c.lddz, c.dtype, c.dx, c.dw, c.db);
    const int es = elem_size(c.dtype);
    Matrix X{}, W{}, D{};
    PadJobs jobs{};
    if (c.dx || c.dw) D = place(c.dz, c.T, c.n, c.lddz, c.dtype, ws + z.dz, &jobs);
    if (c.dx) W = place(c.w, c.d, c.n, c.ldw, c.dtype, ws + z.w, &jobs);
    if (c.dw) X = place(c.x, c.T, c.d, c.ldx, c.dtype, ws + z.x, &jobs);
    hipError_t rc = launch_pads(jobs, s);
    if (rc != hipSuccess) return rc;
    float *part = reinterpret_cast<float *>(ws + z.part);
    Epilogue e{};
    if (c.dx) {
        e.out = c.dx;
        e.ldo = c.lddx;
        e.out_f32 = es == 4;
        e.vec = rows_aligned(c.dx, c.lddx, es);
        rc = launch_product<T, false, false>(D, W, c.T, c.d, c.n,
                                             product_of(c.T, c.d, c.n, c.dtype), part, e, s);
        if (rc != hipSuccess) return rc;
    }
    if (c.dw) {
        e.out = c.dw;
        e.ldo = c.lddw;
        e.out_f32 = c.grad_dtype == 0;
        e.vec = rows_aligned(c.dw, c.lddw, e.out_f32 ? 4 : es);
        rc = launch_product<T, true, true>(X, D, c.d, c.n, c.T,
                                           product_of(c.d, c.n, c.T, c.dtype), part, e, s);
        if (rc != hipSuccess) return rc;
    }
    if (c.db) {
        const int blocks = z.db_blocks, per = (int)div_up(c.T, blocks);
        // (the padded copy, where there is one)
        const bool vec = D.p || !padded(c.T, c.n, c.lddz, c.dtype).copy;
        const T *dz = D.p ? reinterpret_cast<const T *>(D.p) : static_cast<const T *>(c.dz);
        const int64_t ld = D.p ? D.ld / es : c.lddz;
        const dim3 grid((c.n + kSumCols - 1) / kSumCols, blocks);
        auto sum = vec ? k_colsum<T, true> : k_colsum<T, false>;
        hipLaunchKernelGGL(sum, grid, dim3(256), 0, s, dz, ld, c.T, c.n, per, part, c.db, c.grad_dtype == 0 ? 1 : 0);
        if (blocks > 1)
            hipLaunchKernelGGL(k_colsum_join<T>, dim3((c.n + 31) / 32), dim3(256), 0, s, part,
                               blocks, c.n, c.db, c.grad_dtype == 0 ? 1 : 0);
    }
    return hipGetLastError();
}

}  // namespace

// (a launch's threads, at most 512 a workgroup, are counted in 32 bits)
bool linear_fits(int M, int N, int K, int dtype)
{
    const Product z = product_of(M, N, K, dtype);
    return z.mt * z.nt * z.split <= ((int64_t)1 << 23) - 8;
}

void linear_shape(int M, int N, int K, int dtype, int *tile, int *split)
{
    const Product z = product_of(M, N, K, dtype);
    *tile = z.tile;
    *split = z.split;
}

LinearSpace linear_space(int T, int d, int n, int64_t ldx, int64_t ldw, int dtype)
{
    LinearSpace z;
    z.x = 0;
    z.w = z.x + padded(T, d, ldx, dtype).bytes;
    z.part = z.w + padded(d, n, ldw, dtype).bytes;
    z.total = z.part + product_of(T, n, d, dtype).part_bytes;
    return z;
}

LinearBackwardSpace linear_backward_space(int T, int d, int n, int64_t ldx, int64_t ldw,
                                          int64_t lddz, int dtype, bool dx, bool dw, bool db)
{
    LinearBackwardSpace z;
    z.x = 0;
    z.w = z.x + (dw ? padded(T, d, ldx, dtype).bytes : 0);
    z.dz = z.w + (dx ? padded(d, n, ldw, dtype).bytes : 0);
    z.part = z.dz + (dx || dw ? padded(T, n, lddz, dtype).bytes : 0);
    int64_t most = 0;
    auto need = [&](int64_t b) { most = b > most ? b : most; };
    if (dx) need(product_of(T, d, n, dtype).part_bytes);
    if (dw) need(product_of(d, n, T, dtype).part_bytes);
    // the column sums: about 512 workgroups, of at least 64 rows
    const int64_t want = 512 / div_up(n, kSumCols), most_blocks = div_up(T, 64);
    z.db_blocks = (int)(want < 1 ? 1 : want < most_blocks ? want : most_blocks);
    if (db && z.db_blocks > 1) need(up((int64_t)z.db_blocks * n * 4, 256));
    z.total = z.part + most;
    return z;
}

hipError_t launch_linear(const LinearCall &c, void *ws, hipStream_t s)
{
    char *b = static_cast<char *>(ws);
    return c.dtype == 0 ? linear_t<float>(c, b, s)
           : c.dtype == 1 ? linear_t<_Float16>(c, b, s) : linear_t<__bf16>(c, b, s);
}

hipError_t launch_linear_backward(const LinearBackwardCall &c, void *ws, hipStream_t s)
{
    char *b = static_cast<char *>(ws);
    return c.dtype == 0 ? linear_backward_t<float>(c, b, s)
           : c.dtype == 1 ? linear_backward_t<_Float16>(c, b, s) : linear_backward_t<__bf16>(c, b, s);
}

}  // namespace moe
