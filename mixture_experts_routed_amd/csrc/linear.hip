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
// A workgroup computes a BM x BN tile in K-steps of 128 bytes of k (64 values
// of the 16-bit types, 32 of fp32). A step's operands go from memory straight
// into one of two LDS buffers (buffer loads with the LDS flag), one step ahead
// of the matrix instructions that read the other. In LDS the 16-byte chunks
// are permuted so that the reads of a wavefront meet every bank once:
//   rows:     chunk c of row r (8 chunks, 128 bytes) sits at c ^ ((r >> 1) & 7)
//   columns:  the 16 columns that one lane group reads (32 bytes of the 16-bit
//             types, 64 of fp32) are a segment; segment s of row k sits at
//             s ^ f(k), f taking 8 (4) values over the rows read together.
// Columns of the 16-bit types are read with the transposing LDS load (4 rows x
// 16 columns per 16 lanes), so no operand is rearranged in memory or registers.
// The matrix instruction is given B's fragment first: a lane then holds 4
// consecutive columns of one output row, which the epilogue stores together.
//
// Operands whose rows are not whole 16-byte chunks (a stride or a contiguous
// length that is not a multiple of 8, fp32: 4) are first copied into rows
// padded with zeros in the workspace (k_pad_rows): one pass more over that
// operand, and one kernel for every size. Few tiles over a long reduction are
// cut along k (split); the partial sums, fp32 planes in the workspace, are
// added in split order by a second launch that applies the epilogue, so the
// result does not depend on timing.
#include "launch.hpp"
#include "mfma.hpp"

namespace moe {

namespace {

constexpr int kStepBytes = 128;  // bytes of k per K-step of a row operand

template <typename T> struct Mma;
template <> struct Mma<_Float16> {
    static __device__ __forceinline__ float4_t run(uint4 a, uint4 b, float4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a),
                                                      __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
    }
};
template <> struct Mma<__bf16> {
    static __device__ __forceinline__ float4_t run(uint4 a, uint4 b, float4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    }
};
// fp32: lane group q of 16 lanes holds k = 4q .. 4q+3 of a 16-wide step; the
// instruction takes one k per group, so element j of both operands meets in
// the j-th of four
template <> struct Mma<float> {
    static __device__ __forceinline__ float4_t run(uint4 a, uint4 b, float4_t c)
    {
        const float4_t x = __builtin_bit_cast(float4_t, a), y = __builtin_bit_cast(float4_t, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[j], y[j], c, 0, 0, 0);
        return c;
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
    int vec;               // rows of out and residual take 4 columns at a time
};

struct GemmArg {
    const char *A, *B;
    int64_t lda, ldb;  // bytes per row
    int M, N, K;
    int a_cols, b_cols;  // length of an operand's rows as they lie (whole 16-byte chunks), elements
    int mt, nt;          // tiles
    int split, steps;    // K splits, K-steps per split
    float *part;         // split > 1: partial planes [split][M][N]
    Epilogue e;
};

namespace {

// 4 consecutive columns c..c+3 of row r (those below N)
template <typename T>
__device__ __forceinline__ void finish4(const Epilogue &e, int64_t r, int c, int N, float4_t z)
{
    float v[4] = {z[0], z[1], z[2], z[3]};
    if (e.vec && c + 4 <= N) {
        if (e.bias) {
            float b[4];
            Vec<T, 4>::load(static_cast<const T *>(e.bias) + c, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += b[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = act_apply(v[i], e.act);
        if (e.residual) {
            float q[4];
            if (e.res_f32)
                Vec<float, 4>::load(static_cast<const float *>(e.residual) + r * e.ldr + c, q);
            else
                Vec<T, 4>::load(static_cast<const T *>(e.residual) + r * e.ldr + c, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += q[i];
        }
        if (e.out_f32)
            Vec<float, 4>::store(static_cast<float *>(e.out) + r * e.ldo + c, v);
        else
            Vec<T, 4>::store(static_cast<T *>(e.out) + r * e.ldo + c, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (c + i >= N) break;
        float s = v[i];
        if (e.bias) s += to_f32(static_cast<const T *>(e.bias)[c + i]);
        s = act_apply(s, e.act);
        if (e.residual)
            s += e.res_f32 ? static_cast<const float *>(e.residual)[r * e.ldr + c + i]
                           : to_f32(static_cast<const T *>(e.residual)[r * e.ldr + c + i]);
        if (e.out_f32)
            static_cast<float *>(e.out)[r * e.ldo + c + i] = s;
        else
            static_cast<T *>(e.out)[r * e.ldo + c + i] = from_f32<T>(s);
    }
}

// One operand's part of a workgroup's tile: ROWS output rows (or columns) of
// it, NTH threads; COL: the operand is in columns form.
template <typename T, bool COL, int ROWS, int NTH>
struct Operand {
    static constexpr int ES = sizeof(T), EPC = 16 / ES, BK = kStepBytes / ES;
    static constexpr int CHUNKS = ROWS * 8;             // 16-byte chunks of a step
    static constexpr int LOADS = CHUNKS / NTH;          // per thread
    static constexpr int CPR = COL ? ROWS / EPC : 8;    // chunks per LDS row
    static_assert(CHUNKS % NTH == 0, "whole loads");

    // the permutation of row k's segments (columns form)
    static __device__ __forceinline__ int seg_xor(int k)
    {
        return ES == 2 ? ((k & 3) | ((k >> 1) & 4)) : ((k >> 2) & 3);
    }

    const char *base;   // first byte of the tile's rows (rows form: at k = 0)
    int64_t ld;
    int have;           // rows (columns) of the operand from the tile's first on
    int K;              // values of k that it holds (rows form: a multiple of EPC)
    uint32_t off[LOADS];
    int kc;             // rows form: the k within a step of this thread's chunks

    __device__ __forceinline__ void init(const char *p, int64_t ld_, int first, int total, int K_,
                                         int tid)
    {
        ld = ld_;
        K = K_;
        have = total - first;
        base = COL ? p + (int64_t)first * ES : p + (int64_t)first * ld;
        kc = 0;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int q = i * NTH + tid;
            const int r = q / CPR, c = q % CPR;
            if (COL) {
                constexpr int SEG = ES == 2 ? 2 : 4;  // chunks per segment
                const int lc = ((c / SEG) ^ seg_xor(r)) * SEG + c % SEG;
                off[i] = lc * EPC < have ? (uint32_t)r * (uint32_t)ld + (uint32_t)lc * 16u : kOutside;
            } else {
                const int lc = c ^ ((r >> 1) & 7);  // the same for every i
                kc = lc * EPC;
                off[i] = r < have ? (uint32_t)r * (uint32_t)ld + (uint32_t)lc * 16u : kOutside;
            }
        }
    }

    // the loads of the step that starts at k0 into the LDS buffer L; k past K gives zeros
    // (device pass only: with this body in a member function, the host pass of
    // the compiler leaves out the launch stubs of some of the kernel's instances)
    __device__ __forceinline__ void issue(uint4 *L, int k0, int wave) const
    {
#ifdef __HIP_DEVICE_COMPILE__
        __amdgpu_buffer_rsrc_t r;
        if (COL) {
            const int rows = min(BK, K - k0);
            const int64_t bytes = (int64_t)(rows - 1) * ld + (int64_t)min(have, ROWS) * ES;
            r = buffer_of(base + (int64_t)k0 * ld, rows > 0 ? (uint32_t)bytes : 0u);
        } else {
            const int64_t bytes = (int64_t)(min(have, ROWS) - 1) * ld + (int64_t)(K - k0) * ES;
            r = buffer_of(base + (int64_t)k0 * ES, K > k0 ? (uint32_t)bytes : 0u);
        }
        const bool cut = !COL && k0 + kc >= K;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(L + i * NTH + wave * 64), 16,
                                                     cut ? kOutside : off[i], 0, 0, 0);
#endif
    }

    // MFMA fragment of the 16 rows (columns) from `first` of the tile, k-group
    // ks of the step: 16-bit: lane l holds row first + (l & 15), k = 32 ks +
    // 8 (l >> 4) .. + 7; fp32: k = 16 ks + 4 (l >> 4) .. + 3
    static __device__ __forceinline__ uint4 frag(const uint4 *L, int first, int ks, int lane)
    {
        if (!COL) {
            const int r = first + (lane & 15), c = 4 * ks + (lane >> 4);
            return L[r * 8 + (c ^ ((r >> 1) & 7))];
        }
        if constexpr (ES == 2) {
            typedef short s4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s4 *p4;
            const uint16_t *h = reinterpret_cast<const uint16_t *>(L);
            s4 v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = 32 * ks + 8 * (lane >> 4) + 4 * i + ((lane >> 2) & 3);
                const int seg = (first >> 4) ^ seg_xor(k);
                v[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (p4)(const_cast<uint16_t *>(h) + k * ROWS + seg * 16 + (lane & 3) * 4));
            }
            const uint2 a = __builtin_bit_cast(uint2, v[0]), b = __builtin_bit_cast(uint2, v[1]);
            return make_uint4(a.x, a.y, b.x, b.y);
        } else {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(L);
            uint32_t v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = 16 * ks + 4 * (lane >> 4) + j;
                v[j] = w[k * ROWS + ((first >> 4) ^ seg_xor(k)) * 16 + (lane & 15)];
            }
            return make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
};

// WM x WN wavefronts, each (BM / WM) x (BN / WN) of the tile
template <typename T, bool AC, bool BC, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM *WN * 64) void k_gemm(const GemmArg p)
{
    constexpr int NTH = WM * WN * 64, BK = kStepBytes / (int)sizeof(T);
    constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
    constexpr int KS = 2;  // k-groups of a step
    __shared__ uint4 L0[(BM + BN) * 8], L1[(BM + BN) * 8];
    const int lb = xcd_logical_block(p.mt * p.nt * p.split);
    if (lb < 0) return;  // whole workgroup: no barrier reached
    const int tile = lb / p.split, split = lb - tile * p.split;
    const int tm = tile / p.nt, tn = tile - tm * p.nt;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave - wm * WN;

    Operand<T, AC, BM, NTH> a;
    Operand<T, BC, BN, NTH> b;
    // (the rows of a row operand hold k up to its padded length)
    a.init(p.A, p.lda, tm * BM, AC ? p.a_cols : p.M, AC ? p.K : p.a_cols, tid);
    b.init(p.B, p.ldb, tn * BN, BC ? p.b_cols : p.N, BC ? p.K : p.b_cols, tid);

    float4_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = float4_t{0.f, 0.f, 0.f, 0.f};

    const int s0 = split * p.steps;
    const int s1 = min(s0 + p.steps, (p.K + BK - 1) / BK);
    auto issue = [&](uint4 *L, int s) {
        a.issue(L, s * BK, wave);
        b.issue(L + BM * 8, s * BK, wave);
    };
    // this wavefront's loads landed and its LDS reads done; then all of them
    auto meet = [&]() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
    auto compute = [&](const uint4 *L) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint4 fa[TM], fb[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i)
                fa[i] = Operand<T, AC, BM, NTH>::frag(L, (wm * TM + i) * 16, ks, lane);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                fb[j] = Operand<T, BC, BN, NTH>::frag(L + BM * 8, (wn * TN + j) * 16, ks, lane);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = Mma<T>::run(fb[j], fa[i], acc[i][j]);
        }
    };
    if (s0 < s1) {
        issue(L0, s0);
        meet();
        for (int s = s0; s < s1; s += 2) {
            if (s + 1 < s1) issue(L1, s + 1);
            compute(L0);
            meet();
            if (s + 1 >= s1) break;
            if (s + 2 < s1) issue(L0, s + 2);
            compute(L1);
            meet();
        }
    }

#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = tm * BM + (wm * TM + i) * 16 + (lane & 15);
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int n = tn * BN + (wn * TN + j) * 16 + 4 * (lane >> 4);
            if (n >= p.N) continue;
            if (p.split > 1) {
                float *o = p.part + ((int64_t)split * p.M + m) * p.N + n;
                if (n + 4 <= p.N && (p.N & 3) == 0)
                    *reinterpret_cast<float4_t *>(o) = acc[i][j];
                else
                    for (int q = 0; q < 4 && n + q < p.N; ++q) o[q] = acc[i][j][q];
            } else {
                finish4<T>(p.e, m, n, p.N, acc[i][j]);
            }
        }
    }
}

// The split products' partial planes added in split order, then the epilogue:
// one thread per 4 columns of a row.
template <typename T>
__global__ __launch_bounds__(256) void k_gemm_reduce(const float *__restrict__ part, int M, int N,
                                                     int split, const Epilogue e)
{
    const int per = (N + 3) / 4;
    const int64_t total = (int64_t)M * per;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < total;
         q += (int64_t)gridDim.x * 256) {
        const int64_t r = q / per;
        const int c = (int)(q - r * per) * 4;
        float4_t z = {0.f, 0.f, 0.f, 0.f};
        const float *s = part + r * N + c;
        if ((N & 3) == 0) {
            for (int i = 0; i < split; ++i) {
                z += *reinterpret_cast<const float4_t *>(s);
                s += (int64_t)M * N;
            }
        } else {
            for (int i = 0; i < split; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + j < N) z[j] += s[j];
                s += (int64_t)M * N;
            }
        }
        finish4<T>(e, r, c, N, z);
    }
}

// dst [R][ldd] = src [R][C] (rows of lds elements), columns C .. ldd zero; U is
// the raw element, one 16-byte chunk of dst per thread
template <typename U>
__global__ __launch_bounds__(256) void k_pad_rows(const U *__restrict__ src, int64_t lds, int64_t R,
                                                  int C, U *__restrict__ dst, int ldd)
{
    constexpr int EPC = 16 / sizeof(U);
    const int per = ldd / EPC;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < R * per;
         q += (int64_t)gridDim.x * 256) {
        const int64_t r = q / per;
        const int c = (int)(q - r * per) * EPC;
        typedef U vec __attribute__((ext_vector_type(EPC)));
        vec v;
#pragma unroll
        for (int i = 0; i < EPC; ++i) v[i] = c + i < C ? src[r * lds + c + i] : U(0);
        *reinterpret_cast<vec *>(dst + r * ldd + c) = v;
    }
}

// Column sums of dz [T][n] over the rows [b * per, (b + 1) * per), b =
// blockIdx.y, into part [gridDim.y][n] (or, with one block of rows, straight
// into db). A workgroup covers 64 columns; its 4 wavefronts take every fourth
// row and are added in order through LDS.
template <typename T>
__global__ __launch_bounds__(256) void k_colsum(const T *__restrict__ dz, int64_t ld, int rows,
                                                int n, int per, float *__restrict__ part,
                                                void *__restrict__ db, int db_f32)
{
    __shared__ float s[4][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    const int r0 = blockIdx.y * per, r1 = min(rows, r0 + per);
    float v = 0.f;
    if (c < n)
        for (int r = r0 + w; r < r1; r += 4) v += to_f32(dz[(int64_t)r * ld + c]);
    s[w][lane] = v;
    __syncthreads();
    if (w || c >= n) return;
    v = ((s[0][lane] + s[1][lane]) + s[2][lane]) + s[3][lane];
    if (gridDim.y > 1)
        part[(int64_t)blockIdx.y * n + c] = v;
    else if (db_f32)
        static_cast<float *>(db)[c] = v;
    else
        static_cast<T *>(db)[c] = from_f32<T>(v);
}

template <typename T>
__global__ __launch_bounds__(256) void k_colsum_join(const float *__restrict__ part, int blocks,
                                                     int n, void *__restrict__ db, int db_f32)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= n) return;
    float v = 0.f;
    for (int b = 0; b < blocks; ++b) v += part[(int64_t)b * n + c];
    if (db_f32)
        static_cast<float *>(db)[c] = v;
    else
        static_cast<T *>(db)[c] = from_f32<T>(v);
}

// ---- host side ---------------------------------------------------------------

constexpr int kBM = 128, kBN = 128;
constexpr int kSlots = 512;       // workgroups of a 128 x 128 tile that the GPU holds at once
constexpr int kMinSplitSteps = 4;

int elem_size(int dtype) { return dtype == 0 ? 4 : 2; }
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Product {
    int64_t mt, nt;
    int split, steps;
    int64_t part_bytes;
};

Product product_of(int64_t M, int64_t N, int64_t K, int dtype)
{
    Product z;
    z.mt = div_up(M, kBM);
    z.nt = div_up(N, kBN);
    const int64_t steps = div_up(K, kStepBytes / elem_size(dtype));
    int64_t s = kSlots / (z.mt * z.nt);
    s = s < steps / kMinSplitSteps ? s : steps / kMinSplitSteps;
    s = s < 1 ? 1 : s;
    z.steps = (int)div_up(steps, s);
    z.split = (int)div_up(steps, z.steps);
    z.part_bytes = z.split > 1 ? up((int64_t)z.split * M * N * 4, 256) : 0;
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

hipError_t place(const void *src, int64_t R, int64_t C, int64_t ld, int dtype, const Padded &z,
                 char *dst, hipStream_t s, Matrix *m)
{
    const int es = elem_size(dtype);
    m->cols = (int)z.cols;
    if (!z.copy) {
        m->p = static_cast<const char *>(src);
        m->ld = ld * es;
        return hipSuccess;
    }
    m->p = dst;
    m->ld = z.cols * es;
    const int64_t chunks = R * (z.cols * es / 16);
    const dim3 grid((unsigned)(chunks / 256 + 1 < 4096 ? chunks / 256 + 1 : 4096)), block(256);
    if (es == 2)
        hipLaunchKernelGGL(k_pad_rows<uint16_t>, grid, block, 0, s,
                           static_cast<const uint16_t *>(src), ld, R, (int)C,
                           reinterpret_cast<uint16_t *>(dst), (int)z.cols);
    else
        hipLaunchKernelGGL(k_pad_rows<uint32_t>, grid, block, 0, s,
                           static_cast<const uint32_t *>(src), ld, R, (int)C,
                           reinterpret_cast<uint32_t *>(dst), (int)z.cols);
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
    g.e = e;
    const dim3 grid((unsigned)up(z.mt * z.nt * z.split, 8)), block(256);
    hipLaunchKernelGGL((k_gemm<T, AC, BC, kBM, kBN, 2, 2>), grid, block, 0, s, g);
    if (z.split > 1) {
        const int64_t quads = (int64_t)M * ((N + 3) / 4);
        const dim3 rgrid((unsigned)(quads / 256 + 1 < 8192 ? quads / 256 + 1 : 8192));
        hipLaunchKernelGGL(k_gemm_reduce<T>, rgrid, dim3(256), 0, s, part, M, N, z.split, e);
    }
    return hipGetLastError();
}

bool rows_take_4(const void *p, int64_t ld, int es)
{
    return !p || (ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * es) == 0);
}

template <typename T>
hipError_t linear_t(const LinearCall &c, char *ws, hipStream_t s)
{
    const LinearSpace z = linear_space(c.T, c.d, c.n, c.ldx, c.ldw, c.dtype);
    const int es = elem_size(c.dtype);
    Matrix X, W;
    hipError_t rc = place(c.x, c.T, c.d, c.ldx, c.dtype, padded(c.T, c.d, c.ldx, c.dtype),
                          ws + z.x, s, &X);
    if (rc != hipSuccess) return rc;
    rc = place(c.w, c.d, c.n, c.ldw, c.dtype, padded(c.d, c.n, c.ldw, c.dtype), ws + z.w, s, &W);
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
    e.vec = rows_take_4(c.out, c.ldo, e.out_f32 ? 4 : es) &&
            rows_take_4(c.residual, c.ldr, e.res_f32 ? 4 : es);
    return launch_product<T, false, true>(X, W, c.T, c.n, c.d,
                                          product_of(c.T, c.n, c.d, c.dtype),
                                          reinterpret_cast<float *>(ws + z.part), e, s);
}

template <typename T>
hipError_t linear_backward_t(const LinearBackwardCall &c, char *ws, hipStream_t s)
{
    const LinearBackwardSpace z = linear_backward_space(
        c.T, c.d, c.n, c.dx || c.dw ? c.ldx : c.d, c.ldw, c.lddz, c.dtype, c.dx, c.dw, c.db);
    const int es = elem_size(c.dtype);
    Matrix X{}, W{}, D{};
    hipError_t rc = hipSuccess;
    if (c.dx || c.dw)
        rc = place(c.dz, c.T, c.n, c.lddz, c.dtype, padded(c.T, c.n, c.lddz, c.dtype), ws + z.dz, s,
                   &D);
    if (rc == hipSuccess && c.dx)
        rc = place(c.w, c.d, c.n, c.ldw, c.dtype, padded(c.d, c.n, c.ldw, c.dtype), ws + z.w, s, &W);
    if (rc == hipSuccess && c.dw)
        rc = place(c.x, c.T, c.d, c.ldx, c.dtype, padded(c.T, c.d, c.ldx, c.dtype), ws + z.x, s, &X);
    if (rc != hipSuccess) return rc;
    float *part = reinterpret_cast<float *>(ws + z.part);
    Epilogue e{};
    if (c.dx) {
        e.out = c.dx;
        e.ldo = c.lddx;
        e.out_f32 = es == 4;
        e.vec = rows_take_4(c.dx, c.lddx, es);
        rc = launch_product<T, false, false>(D, W, c.T, c.d, c.n,
                                             product_of(c.T, c.d, c.n, c.dtype), part, e, s);
        if (rc != hipSuccess) return rc;
    }
    if (c.dw) {
        e.out = c.dw;
        e.ldo = c.lddw;
        e.out_f32 = c.grad_dtype == 0;
        e.vec = rows_take_4(c.dw, c.lddw, e.out_f32 ? 4 : es);
        rc = launch_product<T, true, true>(X, D, c.d, c.n, c.T,
                                           product_of(c.d, c.n, c.T, c.dtype), part, e, s);
        if (rc != hipSuccess) return rc;
    }
    if (c.db) {
        const int blocks = z.db_blocks, per = (int)div_up(c.T, blocks);
        hipLaunchKernelGGL(k_colsum<T>, dim3((c.n + 63) / 64, blocks), dim3(256), 0, s,
                           static_cast<const T *>(c.dz), c.lddz, c.T, c.n, per, part, c.db,
                           c.grad_dtype == 0 ? 1 : 0);
        if (blocks > 1)
            hipLaunchKernelGGL(k_colsum_join<T>, dim3((c.n + 255) / 256), dim3(256), 0, s, part,
                               blocks, c.n, c.db, c.grad_dtype == 0 ? 1 : 0);
    }
    return hipGetLastError();
}

}  // namespace

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
    // rows of dz per workgroup of the column sums: at least 64
    const int64_t want = 1024 / div_up(n, 64);
    const int64_t most_blocks = div_up(T, 64);
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
