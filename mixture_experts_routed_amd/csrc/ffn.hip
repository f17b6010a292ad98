// Grouped expert FFN for gfx950 on the expert-sorted rows of the routing plan:
//   gate/up:  H = D( silu(XS_e W_gate[e]) * (XS_e W_up[e]) )   (SwiGLU in the epilogue)
//   down:     Y = sw * (H_e W_down[e])                          (fp32, weight in the epilogue)
//
// Sources: "Batched resident MoE experts on Apple Silicon: a flat parallel
// expert pass", section 1 -- per (token, expert, weight) job: gate/up
// projection, gated activation, weighted down projection; "Round 4 Track C:
// Prefill MoE Plan ... & Epilogue / Gather Audit", section 1, finding 5 --
// the SwiGLU output is kept in half precision, and section 2 -- grouped
// GEMMs over tm-row tiles dominate the layer's time.
//
// Design (MI355X): at 512 experts x ~48 rows each, the weights (6 GB at the
// prefill shape) are streamed once and every weight element meets only a few
// dozen rows, so these GEMMs are bound by HBM, not by the matrix cores.
//  * Work list: each expert's rows cut into items of <= 64 rows. A workgroup
//    (4 wavefronts) covers 4 x 64 output rows-by-columns "cells" of one
//    expert; per item there are ceil(N / (4 slices)) workgroups, so the grid
//    is (items x column groups x K-splits) whatever the shape of the cells.
//  * Wide cells (an expert with a single item, the common case): the 4
//    wavefronts share the item's rows (A tile through LDS) and each streams its
//    own column slice of the weights straight into registers.
//  * Tall cells (runs of 2 items of one expert; a run of 4 is two runs of 2):
//    the wavefronts take different row blocks of the same column slices and
//    share the weight tile through LDS, so such an expert's weights are read
//    once per 128 rows instead of once per 64 rows.
//  * Split-K when the host-side bound on work items is too small to fill the
//    256 CUs (decode-sized batches): each split accumulates a K range into an
//    fp32 partial plane, and a reduce kernel adds the planes in split order
//    and applies the epilogue (SwiGLU, or the router weight).
//  * Matrix cores: v_mfma_f32_16x16x32_{f16,bf16} (v_mfma_f32_16x16x4_f32 for
//    fp32). The weights are row-major [K][N] (N contiguous) but an MFMA lane
//    needs 8 consecutive K of one column. Each lane loads 8 K-rows x 4
//    columns (8-byte loads; 16 lanes cover one 128-byte row segment) and
//    transposes the 8x4 block in registers into 4 B-fragments: fragment c
//    feeds MFMA c, whose 16 columns are the logical columns 4*j + c of the
//    slice. No repacking of the weights by the caller.
//  * Loads of K-step s+S-1 are issued before the MFMAs of step s.
//  * Packed weights (moe_pack_weights, once at load time): each wavefront's
//    K range of a column slice is one contiguous run of 4 KB tiles already in
//    MFMA lane order (16-byte loads, no transposes).
//  * Big cells (packed 16-bit weights, experts with hundreds of rows, as in a
//    long prompt planned as one call): runs of 4 items x 256 weight columns on
//    8 wavefronts, operands loaded straight into LDS (k_big, below), which
//    turns those experts from weight streaming into matrix-core work.
//  * Weights in microscaled 4 bits (moe_mx4_quantize): tiles in the packed
//    order, made into operands in registers. Every item is a wide cell, or in
//    small launches a set of narrow ones (ffn_mx4.hip).
// The cells are in ffn_cells.hpp.
#include "ffn_cells.hpp"

namespace moe {

// output columns per 8-wavefront big-cell workgroup: h columns (gate/up) or y
// columns (down)
constexpr int big_cols(bool gateup) { return gateup ? 128 : 256; }

int ffn_rows_per_item() { return kItemRows; }

size_t packed_weight_bytes(int E, int Kd, int N, bool gateup, int dtype)
{
    const PackedGeom z = packed_geom(Kd, N, gateup, dtype == 0 ? 4 : 2);
    return (size_t)E * z.gs * z.nst * z.step_bytes;
}

// One 16-byte word of the packed layout per thread (grid-stride); U is the
// raw element (uint16_t for f16/bf16, uint32_t for fp32): bits are copied.
template <typename U>
__global__ __launch_bounds__(256) void k_pack(const U *__restrict__ src, int Kd, int N, int gs,
                                              int nst, int nm, uint4 *__restrict__ dst,
                                              size_t total)
{
    for (size_t idx = (size_t)blockIdx.x * 256 + threadIdx.x; idx < total;
         idx += (size_t)gridDim.x * 256) {
        const int l = (int)(idx & 63), c = (int)((idx >> 6) & 3);
        size_t t = idx >> 8;
        const int m = (int)(t % nm);
        t /= nm;
        const int w = (int)(t & 3);
        t >>= 2;
        const int s = (int)(t % nst);
        t /= nst;
        const int g = (int)(t % gs);
        const size_t e = t / gs;
        const int n0 = (4 * g + w) * 64 * nm + 64 * m + 4 * (l & 15);
        auto val = [&](int k, int n) -> uint32_t {
            return (k < Kd && n < N) ? (uint32_t)src[(e * Kd + k) * (size_t)N + n] : 0u;
        };
        uint32_t o[4];
        if constexpr (sizeof(U) == 2) {
            const int n = n0 + c, k0 = 32 * s + 8 * (l >> 4);
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = val(k0 + 2 * q, n) | (val(k0 + 2 * q + 1, n) << 16);
        } else {
            const int k = 16 * s + 4 * (l >> 4) + c;
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = val(k, n0 + q);
        }
        dst[idx] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

hipError_t launch_pack(int dtype, const void *src, int E, int Kd, int N, bool gateup, void *dst,
                       hipStream_t s)
{
    const PackedGeom z = packed_geom(Kd, N, gateup, dtype == 0 ? 4 : 2);
    const size_t total = (size_t)E * z.gs * z.nst * z.step_bytes / 16;
    const size_t want = (total + 255) / 256;
    const unsigned blocks = (unsigned)(want < (1u << 18) ? want : (1u << 18));
    if (dtype == 0)
        hipLaunchKernelGGL(k_pack<uint32_t>, dim3(blocks), dim3(256), 0, s,
                           static_cast<const uint32_t *>(src), Kd, N, z.gs, z.nst, z.m,
                           static_cast<uint4 *>(dst), total);
    else
        hipLaunchKernelGGL(k_pack<uint16_t>, dim3(blocks), dim3(256), 0, s,
                           static_cast<const uint16_t *>(src), Kd, N, z.gs, z.nst, z.m,
                           static_cast<uint4 *>(dst), total);
    return hipGetLastError();
}

// Items are ceil(cnt_e / 64) per active expert, so their number is at most
// (active experts) + (entries beyond one per active expert) / 64; with rows
// padded to tm this is bounded from max_rows as below.
int64_t ffn_max_items(int E, int tm, int64_t max_rows)
{
    const int64_t per_tile = (max_rows + tm - 1) / tm;
    return max_rows / kItemRows + 1 + (E < per_tile ? E : per_tile);
}

// A run of 4 items spans more than 3 * 64 rows of one expert.
int64_t ffn_max_quads(int64_t max_rows) { return max_rows / (3 * kItemRows + 1); }

// ---- host-side shape of the two grouped GEMMs ------------------------------
namespace {

// columns of one workgroup's 4 slices: gate/up 4 x 64, down 4 x 128
int group_cols(bool gateup) { return kWavesPerBlock * (gateup ? 16 * kNpl : 32 * kNpl); }

// Split-K is used when the bound on (item, column group) cells is below
// kSplitBelowCells, three quarters of the 256 CUs: then each projection's
// reduction is cut into enough K ranges for about kTargetCells workgroups,
// two per CU. Above it, a split gains less than its reduction launch costs
// (decode, 2,816 x 704 bf16: the down projection's 246 cells unsplit took
// 29.7 us, split in two 27.1 us plus 4.6 us to reduce), while the gate/up
// projection's 123 cells, each streaming 2.9 MB, take 51 us split 5 ways
// (3: 54, 4: 52; 6 ways no longer fits one round of workgroups: 61).
constexpr int64_t kSplitBelowCells = 192;
constexpr int64_t kTargetCells = 512;
// The 8-wavefront kernel takes the runs of 4 items when the plan bound allows
// this many rows per expert on average.
constexpr int64_t kBigMinRowsPerExpert = 64;
constexpr int kMinStepsPerSplit = 8;
constexpr int kMaxSplit = 8;

void split_for(int64_t cells, int Kd, int kstep, int *nsplit, int *steps)
{
    const int nsteps = (Kd + kstep - 1) / kstep;
    int s = 1;
    if (cells < kSplitBelowCells) s = (int)((kTargetCells + cells - 1) / cells);
    s = s < kMaxSplit ? s : kMaxSplit;
    const int smax = nsteps / kMinStepsPerSplit > 1 ? nsteps / kMinStepsPerSplit : 1;
    s = s < smax ? s : smax;
    const int per = (nsteps + s - 1) / s;
    *steps = per;
    *nsplit = (nsteps + per - 1) / per;  // every split has >= 1 step
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

FfnShape ffn_shape(int E, int tm, int64_t max_rows, int d, int f, int dtype)
{
    FfnShape z;
    z.max_items = ffn_max_items(E, tm, max_rows);
    z.max_rows = max_rows;
    const int kstep = dtype == 0 ? 16 : 32;
    const int64_t gs_gu = (f + group_cols(true) - 1) / group_cols(true);
    const int64_t gs_dn = (d + group_cols(false) - 1) / group_cols(false);
    split_for(z.max_items * gs_gu, d, kstep, &z.split_gu, &z.steps_gu);
    split_for(z.max_items * gs_dn, f, kstep, &z.split_dn, &z.steps_dn);
    z.blocks_gu = (z.max_items * gs_gu * z.split_gu + 7) / 8 * 8;
    z.blocks_dn = (z.max_items * gs_dn * z.split_dn + 7) / 8 * 8;
    // big cells (packed 16-bit weights, experts with hundreds of rows)
    const bool big = dtype != 0 && max_rows >= kBigMinRowsPerExpert * (int64_t)E;
    z.big_gu = big && z.split_gu == 1;
    z.big_dn = big && z.split_dn == 1;
    z.blocks_big_gu = (ffn_max_quads(max_rows) * ((f + big_cols(true) - 1) / big_cols(true)) + 7) / 8 * 8;
    z.blocks_big_dn = (ffn_max_quads(max_rows) * ((d + big_cols(false) - 1) / big_cols(false)) + 7) / 8 * 8;
    z.plane_gu = max_rows * 2 * (int64_t)f;
    z.plane_dn = max_rows * (int64_t)d;
    const size_t pg = z.split_gu > 1 ? (size_t)z.split_gu * z.plane_gu * 4 : 0;
    const size_t pd = z.split_dn > 1 ? (size_t)z.split_dn * z.plane_dn * 4 : 0;
    z.part_offset = round256(kCtlBytes + (size_t)z.max_items * sizeof(WorkItem));
    z.scratch_bytes = z.part_offset + (pg > pd ? pg : pd);
    return z;
}

// Work list: each expert's row range [eoff[e], eoff[e+1]) cut into items of at
// most kItemRows rows; runs of 4 items first (item_slot). Ranges are clamped
// to [0, max_rows] so that made-up offsets cannot lead outside the buffers.
__global__ __launch_bounds__(1024) void k_worklist(const int32_t *__restrict__ eoff, int E,
                                                   int64_t max_rows, int32_t *__restrict__ ctl,
                                                   WorkItem *__restrict__ items, int max_items,
                                                   int runs_first)
{
    __shared__ int s_q[16], s_r[16], s_p[16];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    int r0 = 0, rows = 0;
    if (tid < E) {
        int64_t a = eoff[tid], b = eoff[tid + 1];
        a = a < 0 ? 0 : (a > max_rows ? max_rows : a);
        b = b < a ? a : (b > max_rows ? max_rows : b);
        r0 = (int)a;
        rows = (int)(b - a);
    }
    const int n = (rows + kItemRows - 1) / kItemRows;
    const int n4 = n & ~3;
    const int qincl = wave_inclusive_scan(n4, lane);
    const int rincl = wave_inclusive_scan(n - n4, lane);
    const int pairs = wave_sum(n - n4 >= 2 ? 2 : 0);  // items in this wave's runs of 2
    if (lane == 63) {
        s_q[wv] = qincl;
        s_r[wv] = rincl;
        s_p[wv] = pairs;
    }
    __syncthreads();
    int qbefore = qincl - n4, rbefore = rincl - (n - n4), qtotal = 0, rtotal = 0, ptotal = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        qbefore += (q < wv) ? s_q[q] : 0;
        rbefore += (q < wv) ? s_r[q] : 0;
        qtotal += s_q[q];
        rtotal += s_r[q];
        ptotal += s_p[q];
    }
    wave_fill_items(n, r0, rows, qbefore, rbefore, qtotal, runs_first != 0, tid, lane, max_items,
                    (int)max_rows, items);
    if (tid == 0) {
        ctl[0] = min(qtotal + rtotal, max_items);
        ctl[1] = runs_first ? min(qtotal, max_items) & ~3 : 0;
        ctl[2] = min(qtotal + ptotal, max_items);
    }
}

// ---- big cells: runs of 4 items on 8 wavefronts (packed, 16-bit) ------------
// An expert with hundreds of rows (a long prompt in one call) turns its
// projections from weight streaming into dense GEMMs bound by the matrix
// cores; the 4-wavefront cells above then move too many operand bytes per
// MFMA. A big cell is one run of 4 items (up to 256 rows) x 256 weight
// columns (gate/up: 128 columns of h from each matrix; down: 256 columns of
// y) on 512 threads, in 32-wide K-steps:
//  * a step's operands (A: 256 rows x 64 bytes; B: the 4 KB packed tiles of
//    slices w0, w0+1, already in MFMA lane order) go straight from memory into
//    one of 5 LDS buffers of 32 KB (the whole LDS; buffer loads with the LDS
//    flag, no registers), 4 steps ahead of the MFMAs, and are waited for 2
//    steps before use: these loads spend about as long in the memory system as
//    a step's MFMAs take (the down epilogue's router weights are loaded into
//    registers at the start instead of LDS);
//  * the loads keep the default cache policy: the operands of a step are read
//    by several workgroups at about the same time (the rows by every column
//    block of the run, the weights by the runs of the same expert), which then
//    hit in L2 (non-temporal weight loads were measured 10% slower);
//  * the MFMA operands of step s+1 are read from LDS into registers while the
//    MFMAs of step s run, each into the register of the operand it replaces
//    once that operand's last MFMA is issued; one barrier per step, as inline
//    asm with a memory clobber (__syncthreads()'s release fence would wait for
//    every load in flight);
//  * in LDS the 16-byte chunk j of A row r sits at chunk j ^ ((r >> 1) & 3):
//    the MFMA-order reads are then free of bank conflicts;
//  * wavefront (wr, wc) computes rows 64*wr.. of the run and packed slice
//    w0 + wc: the same 2 x 4 x 4 accumulators, MFMA sequence and epilogue as
//    a tall cell, so the results are the same bits.
// The buffers are separate LDS arrays and the step loop is unrolled by 5, so
// that the compiler can tell a buffer's reads from the loads in flight into
// the others and does not make the reads wait for those loads.
constexpr int kBigThreads = 512;
constexpr int kDeepAU4 = 4 * kItemRows * 4;   // A tile of one step: 256 rows x 4 chunks
constexpr int kDeepBufU4 = kDeepAU4 + 1024;   // + B: 16 KB = 32 KB per buffer
template <typename T, bool GATEUP, bool GATHERED>
__global__ __launch_bounds__(kBigThreads) void k_big(const GemmArgs p,
                                                      const int32_t *__restrict__ ctl,
                                                      const WorkItem *__restrict__ items)
{
    static_assert(sizeof(T) == 2, "big cells: 16-bit element types");
    static_assert(GATEUP || !GATHERED, "the down projection reads h row-major");
    constexpr int ES = 2;
    constexpr int BCOLS = big_cols(GATEUP);
    constexpr int NB = 5;                     // LDS buffers
    constexpr int VM = 4 * (NB - 3);          // loads of this wavefront still in flight
    __shared__ uint4 L0[kDeepBufU4], L1[kDeepBufU4], L2[kDeepBufU4], L3[kDeepBufU4],
        L4[kDeepBufU4];
    const int Kd = p.Kd, N = p.N;
    const int ncb = (N + BCOLS - 1) / BCOLS;
    const int nquads = min(ctl[1], ctl[0]) / 4;
    const int lb = xcd_logical_block(nquads * ncb);
    if (lb < 0) return;  // whole workgroup: no barrier reached
    const int qd = lb / ncb, cb = lb - qd * ncb;
    const WorkItem first = items[4 * qd];
    const WorkItem last = items[4 * qd + 3];
    // workgroup-uniform by construction; said so, so that the buffer
    // descriptors built from them stay in scalar registers
    const int expert = __builtin_amdgcn_readfirstlane(first.expert);
    const int row0 = __builtin_amdgcn_readfirstlane(first.row0);
    const int nvalid = __builtin_amdgcn_readfirstlane(
        max(0, min(4 * kItemRows, last.row0 + last.nrows - row0)));

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wr = wave & 3, wc = wave >> 2;
    const int nq = lane & 15, kg = lane >> 4;
    const WorkItem it = items[4 * qd + wr];
    // down: the router weight and token of the item's row 16 mt + 4 kg + r,
    // with (mt, r) = (nq >> 2, nq & 3), loaded now so that they have landed by
    // the epilogue; the 16 lanes of a K-group hold the 16 rows that each of
    // them stores (taken there with a shuffle), one register each
    float rsw = 0.f;
    int rtok = -1;
    if constexpr (!GATEUP) {
        const int rl = 16 * (nq >> 2) + 4 * kg + (nq & 3);
        if (rl < it.nrows) {
            rsw = p.sw[(int64_t)it.row0 + rl];
            rtok = p.stok[(int64_t)it.row0 + rl];
        }
    }

    // B: per step the packed tiles of slices w0, w0+1: gate/up 8 KB of gate,
    // then 8 KB of up; down 16 KB (tiles (w0, 0), (w0, 1), (w0+1, 0),
    // (w0+1, 1)). Wavefront w moves KB 2 w and 2 w + 1 of these 16.
    const PackedGeom z = packed_geom(Kd, N, GATEUP, ES);
    const int w0 = 2 * (cb & 1);
    const size_t gbase = ((size_t)expert * z.gs + (cb >> 1)) * z.nst * z.step_bytes;
    const uint32_t grange = (uint32_t)z.nst * z.step_bytes;
    __amdgpu_buffer_rsrc_t rb;
    uint32_t vb;
    if constexpr (GATEUP) {
        rb = make_rsrc(static_cast<const char *>(wave >> 2 ? p.B1 : p.B0) + gbase, grange);
        vb = (uint32_t)w0 * 4096u + (uint32_t)(wave & 3) * 2048u;
    } else {
        rb = make_rsrc(static_cast<const char *>(p.B0) + gbase, grange);
        vb = (uint32_t)w0 * 8192u + (uint32_t)wave * 2048u;
    }
    vb += (uint32_t)lane * 16u;
    const int bslot = kDeepAU4 + 128 * wave;

    // A: wavefront w moves rows 32 w .. 32 w + 31, 16 rows per instruction;
    // lane l takes row 32 w + 16 i + (l >> 2) and fills its LDS chunk l & 3
    // with the row's K chunk (l & 3) ^ ((l >> 3) & 3)
    const int arow = 32 * wave + (lane >> 2);
    const uint32_t achunk = (uint32_t)(8 * ((lane & 3) ^ ((lane >> 3) & 3)));  // elements
    __amdgpu_buffer_rsrc_t ra;
    uint32_t va[2];
    if constexpr (GATHERED) {
        ra = make_rsrc(p.A, (uint32_t)((size_t)p.a_rows * Kd * ES));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = arow + 16 * i;
            const int t = r < nvalid ? p.stok[row0 + r] : -1;
            va[i] = (unsigned)t < (unsigned)p.a_rows ? (uint32_t)t * (uint32_t)Kd * ES : 0x80000000u;
        }
    } else {
        ra = make_rsrc(static_cast<const T *>(p.A) + (size_t)row0 * Kd,
                       (uint32_t)((size_t)nvalid * Kd * ES));
#pragma unroll
        for (int i = 0; i < 2; ++i) va[i] = (uint32_t)(arow + 16 * i) * (uint32_t)Kd * ES;
    }

    float4_t acc[2][kMT][kNpl];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int c = 0; c < kNpl; ++c) acc[m][mt][c] = float4_t{0.f, 0.f, 0.f, 0.f};

    typedef __attribute__((address_space(3))) void *lds_ptr;
    // the operands of K-step s into LDS buffer L; K chunks past Kd (the next
    // row's data) and steps past the end are read at offsets past the
    // descriptors' ranges, which return zeros
    auto issue = [&](uint4 (&L)[kDeepBufU4], int s) {
        const uint32_t ka = (uint32_t)(32 * s) + achunk;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                ra, (lds_ptr)(L + (32 * wave + 16 * i) * 4), 16,
                (int)ka < Kd ? va[i] + ka * ES : 0x80000000u, 0, 0, 0);
        const uint32_t o = vb + (uint32_t)s * z.step_bytes;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr)(L + bslot + 64 * j), 16,
                                                     o + (uint32_t)j * 1024u, 0, 0, 0);
    };
    uint4 fa[kMT], fb[2][kNpl];
    auto read_a = [&](const uint4 (&L)[kDeepBufU4]) {
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
            const int row = 64 * wr + 16 * mt + nq;
            fa[mt] = L[row * 4 + (kg ^ ((row >> 1) & 3))];
        }
    };
    // B operand (matrix or slice half m, column quad c) of this wavefront
    auto read_b = [&](const uint4 (&L)[kDeepBufU4], int m, int c) {
        fb[m][c] = L[kDeepAU4 + (GATEUP ? 512 * m + 256 * wc : 512 * wc + 256 * m) + 64 * c + lane];
    };
    // step s: loads of step s+4 into Lf (read for step s-1, complete before
    // the last barrier), MFMAs of step s with step s+1's operands read from Ln
    // into the registers as they free up, then this wavefront's loads of step
    // s+2 landed, barrier
    auto stepfn = [&](int s, const uint4 (&Ln)[kDeepBufU4], uint4 (&Lf)[kDeepBufU4]) {
        issue(Lf, s + NB - 1);
#pragma unroll
        for (int c = 0; c < kNpl; ++c)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
                    acc[m][mt][c] = Elt<T>::mfma(fa[mt], fb[m][c], acc[m][mt][c]);
                read_b(Ln, m, c);
                // keep this order: a read hoisted above the MFMAs would hold a
                // second set of operand registers
                __builtin_amdgcn_sched_barrier(0);
            }
        read_a(Ln);
        __builtin_amdgcn_s_waitcnt(wait_vm(VM));
        asm volatile("s_barrier" ::: "memory");
    };

    const int nst = z.nst;
    issue(L0, 0);
    issue(L1, 1);
    issue(L2, 2);
    issue(L3, 3);
    __builtin_amdgcn_s_waitcnt(wait_vm(VM));  // steps 0 and 1 landed
    asm volatile("s_barrier" ::: "memory");
    read_a(L0);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int c = 0; c < kNpl; ++c) read_b(L0, m, c);
    // (no early exits from the unrolled loop: they made the compiler spill)
    int s = 0;
    for (; s + 5 <= nst; s += 5) {
        stepfn(s, L1, L4);
        stepfn(s + 1, L2, L0);
        stepfn(s + 2, L3, L1);
        stepfn(s + 3, L4, L2);
        stepfn(s + 4, L0, L3);
    }
    if (s < nst) stepfn(s, L1, L4);
    if (s + 1 < nst) stepfn(s + 1, L2, L0);
    if (s + 2 < nst) stepfn(s + 2, L3, L1);
    if (s + 3 < nst) stepfn(s + 3, L4, L2);
    __builtin_amdgcn_s_waitcnt(wait_vm(0));  // no load into LDS in flight at exit
    const int col = BCOLS * cb + (BCOLS / 2) * wc + kNpl * nq;
    if constexpr (GATEUP) {
        store_cells<T, true, kMT, false>(p, it, col, kg, acc, nullptr, 0);
    } else {
        // y = router weight x accumulator (fp32) on rows holding an entry, as
        // store_cells does, through a descriptor over the item's rows (the
        // shuffles run with every lane of the wavefront active). Non-temporal
        // here: at the shapes that take big cells y is far larger than the
        // caches, and sc1 stores evicted the operands that the other
        // workgroups share in L2 (measured: down 1.83 -> 1.67 ms on the
        // one-call long prompt)
        constexpr int HALF = 16 * kNpl;
        if (p.yexp) {
            // compact y (binary16 + block exponents), the same rows and stores
            const int col0 = BCOLS * cb + (BCOLS / 2) * wc;
            if (col0 >= N) return;  // wave-uniform
            const __amdgpu_buffer_rsrc_t ry16 =
                make_rsrc(static_cast<uint16_t *>(p.out) + (int64_t)it.row0 * N,
                          (uint32_t)(it.nrows * N * 2));
            int ev[kMT][4];
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    ev[mt][r] = 0;
                    const int src = 16 * kg + 4 * mt + r;
                    const float g = __shfl(rsw, src);
                    if (__shfl(rtok, src) < 0) continue;  // uniform over the DPP row
                    const int rl = 16 * mt + 4 * kg + r;
                    float v[2][4];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int c = 0; c < 4; ++c) v[m][c] = g * acc[m][mt][c][r];
                    ev[mt][r] = store_y16_row(p, ry16, rl, col, v, 0);
                }
            // this lane holds the token of row 16 (nq >> 2) + 4 kg + (nq & 3)
            store_y16_exponents<kMT>(p.yexp + (col0 / kY16Block) * p.estride, it.row0, ev,
                                     16 * (nq >> 2) + 4 * kg + (nq & 3), rtok >= 0);
            return;
        }
        const __amdgpu_buffer_rsrc_t ry =
            make_rsrc(static_cast<float *>(p.out) + (int64_t)it.row0 * N, (uint32_t)(it.nrows * N * 4));
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int src = 16 * kg + 4 * mt + r;
                const float g = __shfl(rsw, src);
                if (__shfl(rtok, src) < 0) continue;  // pad rows (and rows past the item)
                const int rl = 16 * mt + 4 * kg + r;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    if (col + m * HALF >= N) continue;  // col + HALF < N implies col < N
                    const float4 v = make_float4(g * acc[m][mt][0][r], g * acc[m][mt][1][r],
                                                 g * acc[m][mt][2][r], g * acc[m][mt][3][r]);
                    store_sc1<kNT>(ry, (uint32_t)((rl * N + col + m * HALF) * 4), v);
                }
            }
    }
}

// ---- split-K reductions (fixed split order) --------------------------------
__device__ __forceinline__ int rows_of_plan(const int32_t *meta, int64_t max_rows)
{
    const int64_t nr = meta[kMetaNr];
    return (int)(nr < 0 ? 0 : (nr > max_rows ? max_rows : nr));
}

// Both reductions are instantiated per split count NS, so that the NS planes'
// loads are issued together rather than one loop trip at a time (a split
// layer is latency-bound); the sums stay in split order.

// h[r][c..c+3] = D(silu(sum_s G_s) * sum_s U_s) for rows r < nr; pad rows
// (stok < 0, whose partial sums are not stored) get h = 0, as unsplit
template <typename T, int NS>
__global__ __launch_bounds__(256) void k_reduce_gateup(const float *__restrict__ part,
                                                       int64_t plane, int N,
                                                       const int32_t *__restrict__ stok,
                                                       const int32_t *__restrict__ meta,
                                                       int64_t max_rows, T *__restrict__ h)
{
    const int per = N / 4;
    const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = q / per;
    const int c = (int)(q - row * per) * 4;
    if (row >= rows_of_plan(meta, max_rows)) return;
    const float *P = part + row * 2 * N + c;
    float4 gs = make_float4(0.f, 0.f, 0.f, 0.f), us = gs;
    if (stok[row] >= 0) {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const float4 gv = *reinterpret_cast<const float4 *>(P + s * plane);
            const float4 uv = *reinterpret_cast<const float4 *>(P + s * plane + N);
            gs = make_float4(gs.x + gv.x, gs.y + gv.y, gs.z + gv.z, gs.w + gv.w);
            us = make_float4(us.x + uv.x, us.y + uv.y, us.z + uv.z, us.w + uv.w);
        }
    }
    const float h0 = silu(gs.x) * us.x, h1 = silu(gs.y) * us.y;
    const float h2 = silu(gs.z) * us.z, h3 = silu(gs.w) * us.w;
    T *H = h + row * N + c;
    if constexpr (sizeof(T) == 2)
        store_nt(reinterpret_cast<uint2 *>(H),
                 make_uint2(Elt<T>::pack2(h0, h1), Elt<T>::pack2(h2, h3)));
    else
        store_nt(reinterpret_cast<float4 *>(H), make_float4(h0, h1, h2, h3));
}

// y[r][c..c+3] = sw[r] * sum_s Y_s for rows r < nr with stok[r] >= 0
template <int NS>
__global__ __launch_bounds__(256) void k_reduce_down(const float *__restrict__ part, int64_t plane,
                                                     int N,
                                                     const int32_t *__restrict__ stok,
                                                     const float *__restrict__ sw,
                                                     const int32_t *__restrict__ meta,
                                                     int64_t max_rows, float *__restrict__ y)
{
    const int per = N / 4;
    const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = q / per;
    const int c = (int)(q - row * per) * 4;
    if (row >= rows_of_plan(meta, max_rows) || stok[row] < 0) return;
    const float *P = part + row * N + c;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        const float4 v = *reinterpret_cast<const float4 *>(P + s * plane);
        a = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
    }
    const float g = sw[row];
    store_nt(reinterpret_cast<float4 *>(y + row * N + c),
             make_float4(g * a.x, g * a.y, g * a.z, g * a.w));
}

// y in the compact format from the split planes: half a wavefront per (row,
// exponent block), lane l of it taking columns kY16Block * b + 4 l .. + 3; a
// unit's 32 lanes are all active or all not (the row decides), so the block
// maximum runs over all of them
template <int NS>
__global__ __launch_bounds__(256) void k_reduce_down_y16(
    const float *__restrict__ part, int64_t plane, int N, const int32_t *__restrict__ stok,
    const float *__restrict__ sw, const int32_t *__restrict__ meta, int64_t max_rows,
    uint16_t *__restrict__ y, int8_t *__restrict__ yexp, int nyb)
{
    // (exponents block-major: yexp[b * max_rows + row])
    const int64_t unit = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
    const int l = threadIdx.x & 31;
    const int64_t row = unit / nyb;
    const int b = (int)(unit - row * nyb);
    if (row >= rows_of_plan(meta, max_rows) || stok[row] < 0) return;
    const int c = b * kY16Block + 4 * l;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < N) {
        const float *P = part + row * N + c;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const float4 v = *reinterpret_cast<const float4 *>(P + s * plane);
            a = make_float4(a.x + v.x, a.y + v.y, a.z + v.z, a.w + v.w);
        }
    }
    const float g = sw[row];
    const float v[4] = {g * a.x, g * a.y, g * a.z, g * a.w};
    float M = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) M = __builtin_fmaxf(M, c < N ? __builtin_fabsf(v[q]) : 0.0f);
    M = row16_fmax(M);
    M = __builtin_fmaxf(M, __shfl_xor(M, 16));  // the unit's other 16 lanes
    const int e = y16_exponent(M);
    if (c < N) {
        const float scale = pow2f(e);
        float q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) q[k] = v[k] * scale;
        store_nt(reinterpret_cast<uint2 *>(y + row * N + c),
                 make_uint2(Elt<_Float16>::pack2(q[0], q[1]), Elt<_Float16>::pack2(q[2], q[3])));
    }
    if (l == 0) yexp[b * max_rows + row] = (int8_t)e;
}

// ---- host launchers --------------------------------------------------------
// the reductions' launch for a split count in [2, kMaxSplit] (any other count
// is refused)
template <typename T, int NS = 2>
hipError_t reduce_gateup(int nsplit, dim3 grid, hipStream_t s, const float *part, int64_t plane, int N,
                   const int32_t *stok, const int32_t *meta, int64_t max_rows, T *h)
{
    if constexpr (NS <= kMaxSplit) {
        if (nsplit != NS)
            return reduce_gateup<T, NS + 1>(nsplit, grid, s, part, plane, N, stok, meta, max_rows,
                                            h);
        hipLaunchKernelGGL((k_reduce_gateup<T, NS>), grid, dim3(256), 0, s, part, plane, N, stok,
                           meta, max_rows, h);
        return hipSuccess;
    }
    return hipErrorInvalidValue;
}

template <int NS = 2>
hipError_t reduce_down(int nsplit, dim3 grid, hipStream_t s, const float *part, int64_t plane, int N,
                 const int32_t *stok, const float *sw, const int32_t *meta, int64_t max_rows,
                 float *y)
{
    if constexpr (NS <= kMaxSplit) {
        if (nsplit != NS)
            return reduce_down<NS + 1>(nsplit, grid, s, part, plane, N, stok, sw, meta, max_rows,
                                       y);
        hipLaunchKernelGGL((k_reduce_down<NS>), grid, dim3(256), 0, s, part, plane, N, stok, sw,
                           meta, max_rows, y);
        return hipSuccess;
    }
    return hipErrorInvalidValue;
}

template <int NS = 2>
hipError_t reduce_down_y16(int nsplit, dim3 grid, hipStream_t s, const float *part, int64_t plane,
                           int N, const int32_t *stok, const float *sw, const int32_t *meta,
                           int64_t max_rows, uint16_t *y, int8_t *yexp, int nyb)
{
    if constexpr (NS <= kMaxSplit) {
        if (nsplit != NS)
            return reduce_down_y16<NS + 1>(nsplit, grid, s, part, plane, N, stok, sw, meta,
                                           max_rows, y, yexp, nyb);
        hipLaunchKernelGGL((k_reduce_down_y16<NS>), grid, dim3(256), 0, s, part, plane, N, stok,
                           sw, meta, max_rows, y, yexp, nyb);
        return hipSuccess;
    }
    return hipErrorInvalidValue;
}

hipError_t launch_worklist(const int32_t *eoff, int E, int64_t max_rows, void *scratch,
                           int64_t max_items, bool runs_first, hipStream_t s)
{
    int32_t *ctl = static_cast<int32_t *>(scratch);
    WorkItem *items = reinterpret_cast<WorkItem *>(static_cast<char *>(scratch) + kCtlBytes);
    hipLaunchKernelGGL(k_worklist, dim3(1), dim3(1024), 0, s, eoff, E, max_rows, ctl, items,
                       (int)max_items, runs_first ? 1 : 0);
    return hipGetLastError();
}

namespace {

unsigned reduce_blocks(int64_t rows, int N) { return (unsigned)((rows * (N / 4) + 255) / 256); }

// Narrow cells take a launch of 4-bit weights with fewer wide cells than this and, on
// average, fewer rows an item than that (both by the plan's bounds): they read an item's
// weights again for each 16 rows. Layers in a graph, us, narrow against wide cells (2,816
// x 704, 128 experts, top-8, bf16): 1 token 19 / 25, 4 tokens 29 / 33, 8 tokens 38 / 51;
// down cells of 16 to 64 tokens (966 to 1,002 by the bound) 66 to 106 / 64 to 99; gate/up
// cells of 8 to 64 tokens over 512 experts (303 to 1,929) are 4 to 9 us faster narrow.
constexpr int64_t kNarrowBelowGateUp = 2048, kNarrowBelowDown = 512, kNarrowBelowRows = 24;

// workgroups of a launch of narrow cells, or 0: wide cells
int64_t narrow_blocks(const FfnShape &z, int wf, int N, bool gateup)
{
    const int64_t gs = (N + group_cols(gateup) - 1) / group_cols(gateup);
    if (wf != kMx4 || z.max_items * gs >= (gateup ? kNarrowBelowGateUp : kNarrowBelowDown) ||
        z.max_rows >= kNarrowBelowRows * z.max_items)
        return 0;
    const int slice = group_cols(gateup) / kWavesPerBlock;
    return z.max_items * ((N + slice - 1) / slice);
}

// gate/up in the weight layout wf (fp32 has no 4-bit form: the caller refuses it)
template <typename T>
hipError_t gateup_any(const FfnShape &z, int dtype, int wf, const void *a, int a_rows,
                      bool gathered, const int32_t *stok, const void *wg, const void *wu, int d,
                      int f, const int32_t *meta, const void *scratch, void *h, hipStream_t s,
                      const WavePlan *wp = nullptr)
{
    GemmArgs p = gemm_args(z, scratch, true);
    p.A = a;
    p.a_rows = a_rows;
    p.B0 = wg;
    p.B1 = wu;
    p.stok = stok;
    p.out = h;
    p.Kd = d;
    p.N = f;
    if constexpr (sizeof(T) == 2) {
        if (wf == kPacked && z.big_gu && z.blocks_big_gu > 0) {
            p.skip_quads = 1;
            const dim3 bgrid((unsigned)z.blocks_big_gu);
            if (gathered)
                hipLaunchKernelGGL((k_big<T, true, true>), bgrid, dim3(kBigThreads), 0, s, p,
                                   ctl_of(scratch), items_of(scratch));
            else
                hipLaunchKernelGGL((k_big<T, true, false>), bgrid, dim3(kBigThreads), 0, s, p,
                                   ctl_of(scratch), items_of(scratch));
        }
    }
    const int64_t narrow = narrow_blocks(z, wf, f, true);
    if (narrow) p.nsplit = 1;
    hipError_t e =
        wf == kMx4      ? gateup_cells_mx4(dtype, p, narrow ? narrow : z.blocks_gu, narrow != 0,
                                           gathered, scratch, wp, s)
        : wf == kPacked ? gateup_cells<T, kPacked>(p, z.blocks_gu, gathered, scratch, wp, s)
                        : gateup_cells<T, kRowMajor>(p, z.blocks_gu, gathered, scratch, wp, s);
    if (e != hipSuccess) return e;
    if (p.nsplit > 1) {
        e = reduce_gateup<T>(p.nsplit, dim3(reduce_blocks(z.max_rows, f)), s, p.part, p.plane, f,
                             stok, meta, z.max_rows, static_cast<T *>(h));
        if (e != hipSuccess) return e;
    }
    return hipGetLastError();
}

template <typename T>
hipError_t down_any(const FfnShape &z, int dtype, int wf, const void *h, const void *wd, int d,
                    int f, const int32_t *stok, const float *sw, const int32_t *meta,
                    const void *scratch, void *y, int8_t *yexp, hipStream_t s)
{
    GemmArgs p = gemm_args(z, scratch, false);
    p.A = h;
    p.B0 = wd;
    p.stok = stok;
    p.sw = sw;
    p.out = y;
    p.Kd = f;
    p.N = d;
    int nyb = 0;
    if constexpr (sizeof(T) == 2) {
        p.yexp = yexp;
        p.estride = z.max_rows;
        nyb = (d + kY16Block - 1) / kY16Block;
        if (wf == kPacked && z.big_dn && z.blocks_big_dn > 0) {
            p.skip_quads = 1;
            hipLaunchKernelGGL((k_big<T, false, false>), dim3((unsigned)z.blocks_big_dn),
                               dim3(kBigThreads), 0, s, p, ctl_of(scratch), items_of(scratch));
        }
    }
    const int64_t narrow = narrow_blocks(z, wf, d, false);
    if (narrow) p.nsplit = 1;
    hipError_t e = wf == kMx4      ? down_cells_mx4(dtype, p, narrow ? narrow : z.blocks_dn,
                                                    narrow != 0, scratch, s)
                   : wf == kPacked ? down_cells<T, kPacked>(p, z.blocks_dn, scratch, s)
                                   : down_cells<T, kRowMajor>(p, z.blocks_dn, scratch, s);
    if (e != hipSuccess) return e;
    if (p.nsplit > 1) {
        e = p.yexp ? reduce_down_y16(p.nsplit,
                                     dim3((unsigned)((z.max_rows * nyb * 32 + 255) / 256)), s,
                                     p.part, p.plane, d, stok, sw, meta, z.max_rows,
                                     static_cast<uint16_t *>(y), p.yexp, nyb)
                   : reduce_down(p.nsplit, dim3(reduce_blocks(z.max_rows, d)), s, p.part,
                                 p.plane, d, stok, sw, meta, z.max_rows, static_cast<float *>(y));
        if (e != hipSuccess) return e;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gateup(const FfnShape &z, int dtype, int wf, const void *xs,
                         const int32_t *stok, const void *wg, const void *wu, int d, int f,
                         const int32_t *meta, const void *scratch, void *h, hipStream_t s)
{
    if (dtype == 1)
        return gateup_any<_Float16>(z, dtype, wf, xs, 0, false, stok, wg, wu, d, f, meta, scratch, h, s);
    if (dtype == 2)
        return gateup_any<__bf16>(z, dtype, wf, xs, 0, false, stok, wg, wu, d, f, meta, scratch, h, s);
    return gateup_any<float>(z, dtype, wf, xs, 0, false, stok, wg, wu, d, f, meta, scratch, h, s);
}

hipError_t launch_gateup_gathered(const FfnShape &z, int dtype, int wf, const void *x, int T,
                                  const int32_t *stok, const void *wg, const void *wu, int d, int f,
                                  const int32_t *meta, const void *scratch, void *h, hipStream_t s,
                                  const WavePlan *wp)
{
    if (dtype == 1)
        return gateup_any<_Float16>(z, dtype, wf, x, T, true, stok, wg, wu, d, f, meta, scratch, h, s,
                                    wp);
    if (dtype == 2)
        return gateup_any<__bf16>(z, dtype, wf, x, T, true, stok, wg, wu, d, f, meta, scratch, h, s,
                                  wp);
    return gateup_any<float>(z, dtype, wf, x, T, true, stok, wg, wu, d, f, meta, scratch, h, s, wp);
}

// every expert of a call of at most 64 entries pads to at most 64 rows (one
// work item) when tm divides 64
bool wave_plan_fits(int64_t nent, int tm) { return nent <= kWave && tm >= 1 && kWave % tm == 0; }

hipError_t launch_down(const FfnShape &z, int dtype, int wf, const void *h, const void *wd,
                       int d, int f, const int32_t *stok, const float *sw, const int32_t *meta,
                       const void *scratch, void *y, int8_t *yexp, hipStream_t s)
{
    if (dtype == 1)
        return down_any<_Float16>(z, dtype, wf, h, wd, d, f, stok, sw, meta, scratch, y, yexp, s);
    if (dtype == 2)
        return down_any<__bf16>(z, dtype, wf, h, wd, d, f, stok, sw, meta, scratch, y, yexp, s);
    return down_any<float>(z, dtype, wf, h, wd, d, f, stok, sw, meta, scratch, y, nullptr, s);
}

}  // namespace moe
