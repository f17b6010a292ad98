// The grouped FFN's kernels over weights in microscaled 4-bit floating point (wide cells
// in ffn_cells.hpp, layout in mx4.hip), and the narrow cells of small launches.
#include "ffn_cells.hpp"

namespace moe {

// ---- narrow cells -----------------------------------------------------------------
// A launch with too few wide cells to fill the GPU (a decode step: a few rows of each
// of some dozens of experts) is bound by how much of the weights is in flight. A narrow
// cell is one column slice of an item, its 4 wavefronts a quarter of the reduction each:
// 4 times as many workgroups, and no partial sums in memory (the wide cells' K splits
// need a second launch to add theirs). Rows go 16 at a time, straight from memory into
// registers -- each wavefront has its own part of them -- and there is no barrier until
// the 4 sums are added, in order, through LDS.
// Measured, decode layer (4 tokens, 2,816 x 704, 128 experts, top-8, bf16): gate/up 16 us
// for 59 MB, planning included (a workgroup knows its item after 2.8 us, half of them are
// done after 11, the last after 16), down 11 us for 30 MB, where wide cells took 16 + 5
// (the reduction) and 11. Figures of other sizes stand at kNarrowBelowGateUp in ffn.hip.
template <typename T, bool GATEUP, bool GATHERED, bool WP>
__global__ __launch_bounds__(256, 3) void k_narrow(const GemmArgs p,
                                                   const int32_t *__restrict__ ctl,
                                                   const WorkItem *__restrict__ items,
                                                   const WavePlan wp)
{
    static_assert(!WP || (GATEUP && GATHERED), "planned here: the gathered gate/up launch only");
    constexpr int SW = GATEUP ? 16 * kNpl : 32 * kNpl;  // columns of a slice
    constexpr int S = 4;  // steps of a wavefront in flight, one more (6: 3 to 5% slower)
    __shared__ float4_t s_sum[3][8][kWave];
    __shared__ float2 s_rinfo[kItemRows];
    __shared__ int s_tok[kItemRows];
    __shared__ WorkItem s_item;
    __shared__ int s_nb[2];
    static_assert(2 * kMaxExperts * 4 <= sizeof(s_sum), "plan counters fit the sums' LDS");
    const int slices = (p.N + SW - 1) / SW;
    int lb;
    WorkItem it;
    if constexpr (WP) {  // as in k_expert_gemm
        if (blockIdx.x < 8) {
            if (blockIdx.x == 0 && threadIdx.x < kWave) {
                int *ls = reinterpret_cast<int *>(s_sum);
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
            wave_plan_item(wp.ids, wp.nent, wp.E, wp.K, wp.tm, wp.nbits, wp.max_rows, slices,
                           blockIdx.x - 8, &n, &b, &w_it, s_tok);
            if (threadIdx.x == 0) {
                s_nb[0] = n;
                s_nb[1] = b;
                s_item = w_it;
            }
        }
        __syncthreads();
        lb = s_nb[1];
        if (lb < 0) return;  // whole workgroup
        it = s_item;
    } else {
        // (no workgroup shares another's weights: block order, so that the item is asked for
        // with the count and not after it; the grid is the list's capacity times the slices,
        // so there is an item to read, if one without meaning)
        lb = blockIdx.x;
        it = items[lb / slices];
        if (lb >= ctl[0] * slices) return;  // whole workgroup: no barrier reached
    }
    const int *ltok = WP ? s_tok : nullptr;
    const int slice = lb % slices;
    const int Kd = p.Kd;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nq = lane & 15, kg = lane >> 4;
    const int col = slice * SW + kNpl * nq;

    // this wavefront's steps [s0, s0 + n) of the slice's tiles; loads of later steps are
    // outside its range: zeros, no memory traffic
    const Mx4Quarter q4 = mx4_quarter(mx4_tiles(Kd, p.N, GATEUP), it.expert, slice, wave);
    constexpr uint32_t kStep = 4 * (GATEUP ? 1 : 2) * kMx4Tile;  // bytes from step to step
    const int s0 = q4.first, n = q4.count;
    const size_t tb = q4.at;
    const uint32_t r0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)q4.bytes[0]);
    const uint32_t r1 = (uint32_t)__builtin_amdgcn_readfirstlane((int)q4.bytes[1]);
    const char *b0c = static_cast<const char *>(p.B0);
    const __amdgpu_buffer_rsrc_t rb0 = make_rsrc(b0c + tb, r0);
    const __amdgpu_buffer_rsrc_t rb1 =
        GATEUP ? make_rsrc(static_cast<const char *>(p.B1) + tb, r0)
               : make_rsrc(b0c + tb + kMx4Tile, r1);
    const __amdgpu_buffer_rsrc_t ra =
        GATHERED ? make_rsrc(p.A, (uint32_t)((size_t)p.a_rows * Kd * 2))
                 : make_rsrc(static_cast<const T *>(p.A) + (size_t)it.row0 * Kd,
                             (uint32_t)((size_t)it.nrows * Kd * 2));
    struct Stage {
        Mx4Word b[2];
        uint4 a;
    };
    // (an expert's rows beyond 16 read its weights again, from L2)
    for (int row = 0; row < it.nrows; row += 16) {
        WorkItem part = it;
        part.row0 += row;
        part.nrows = min(16, it.nrows - row);
        Stage st[S];
        auto load_b = [&](Stage &q, int s) {
            q.b[0] = load_mx4(rb0, (uint32_t)s * kStep, lane);
            q.b[1] = load_mx4(rb1, (uint32_t)s * kStep, lane);
        };
#pragma unroll
        for (int j = 0; j < S - 1; ++j) load_b(st[j], j);
        __builtin_amdgcn_sched_barrier(0);
        // this lane's row and, of a step, its K-values 8 kg .. + 7 (past the item, or
        // without a token, it starts outside the range and reads zeros)
        uint32_t va = 0x80000000u;
        if constexpr (GATHERED) {
            const int t = nq < part.nrows ? (ltok ? ltok[row + nq] : p.stok[part.row0 + nq]) : -1;
            if ((unsigned)t < (unsigned)p.a_rows) va = (uint32_t)t * (uint32_t)Kd * 2;
        } else if (nq < part.nrows) {
            va = (uint32_t)(row + nq) * (uint32_t)Kd * 2;
        }
        const int k0 = 32 * s0 + 8 * kg;
        auto load_a = [&](Stage &q, int s) {
            q.a = Ld<16>::run(ra, va + (uint32_t)(k0 + 32 * s) * 2, 0u);
        };
#pragma unroll
        for (int j = 0; j < S - 1; ++j) load_a(st[j], j);
        if (!GATEUP && tid < 16) load_rinfo<!GATEUP>(p, part, tid, s_rinfo);
        float4_t acc[2][1][kNpl];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int c = 0; c < kNpl; ++c) acc[m][0][c] = float4_t{0.f, 0.f, 0.f, 0.f};
        auto step = [&](int s, const Stage &q, Stage &qf) {
            load_b(qf, s + S - 1);
            load_a(qf, s + S - 1);
            __builtin_amdgcn_sched_barrier(0);
            // (the weights past Kd are zeros; the row's values there are the next row's)
            const uint4 a = mask4(q.a, k0 + 32 * s < Kd ? 0xffffffffu : 0u);
#pragma unroll
            for (int f = 0; f < 8; ++f)
                acc[f & 1][0][f >> 1] = Elt<T>::mfma(a, mx4_operand<T>(q.b[f & 1], f >> 1),
                                                     acc[f & 1][0][f >> 1]);
            __builtin_amdgcn_sched_barrier(0);
        };
        int s = 0;
        for (; s + S <= n; s += S) {
#pragma unroll
            for (int j = 0; j < S; ++j) step(s + j, st[j], st[(j + S - 1) % S]);
        }
#pragma unroll
        for (int j = 0; j < S - 1; ++j)
            if (s + j < n) step(s + j, st[j], st[(j + S - 1) % S]);
        // the 4 wavefronts' sums, in order
        if (wave > 0) {
#pragma unroll
            for (int f = 0; f < 8; ++f) s_sum[wave - 1][f][lane] = acc[f & 1][0][f >> 1];
        }
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int f = 0; f < 8; ++f)
#pragma unroll
                for (int q = 0; q < 3; ++q) acc[f & 1][0][f >> 1] += s_sum[q][f][lane];
            store_cells<T, GATEUP, 1, false>(p, part, col, kg, acc, s_rinfo, 0);
        }
        __syncthreads();  // the sums and row values are read before they change
    }
}

template <typename T>
hipError_t gateup_mx4_t(const GemmArgs &p, int64_t blocks, bool narrow, bool gathered,
                        const void *scratch, const WavePlan *wp, hipStream_t s)
{
    if (!narrow) return gateup_cells<T, kMx4>(p, blocks, gathered, scratch, wp, s);
    const dim3 grid((unsigned)blocks), block(256);
    const int32_t *ctl = ctl_of(scratch);
    const WorkItem *items = items_of(scratch);
    if (gathered && wp && wp->ids)  // planned here: 8 workgroups before the cells', which
                                    // are dealt to the XCDs: a multiple of 8
        hipLaunchKernelGGL((k_narrow<T, true, true, true>), dim3((grid.x + 7) / 8 * 8 + 8), block,
                           0, s, p, ctl, items, *wp);
    else if (gathered)
        hipLaunchKernelGGL((k_narrow<T, true, true, false>), grid, block, 0, s, p, ctl, items,
                           WavePlan{});
    else
        hipLaunchKernelGGL((k_narrow<T, true, false, false>), grid, block, 0, s, p, ctl, items,
                           WavePlan{});
    return hipGetLastError();
}

template <typename T>
hipError_t down_mx4_t(const GemmArgs &p, int64_t blocks, bool narrow, const void *scratch,
                      hipStream_t s)
{
    if (!narrow) return down_cells<T, kMx4>(p, blocks, scratch, s);
    hipLaunchKernelGGL((k_narrow<T, false, false, false>), dim3((unsigned)blocks), dim3(256), 0, s,
                       p, ctl_of(scratch), items_of(scratch), WavePlan{});
    return hipGetLastError();
}

hipError_t gateup_cells_mx4(int dtype, const GemmArgs &p, int64_t blocks, bool narrow,
                            bool gathered, const void *scratch, const WavePlan *wp, hipStream_t s)
{
    return dtype == 1 ? gateup_mx4_t<_Float16>(p, blocks, narrow, gathered, scratch, wp, s)
                      : gateup_mx4_t<__bf16>(p, blocks, narrow, gathered, scratch, wp, s);
}

hipError_t down_cells_mx4(int dtype, const GemmArgs &p, int64_t blocks, bool narrow,
                          const void *scratch, hipStream_t s)
{
    return dtype == 1 ? down_mx4_t<_Float16>(p, blocks, narrow, scratch, s)
                      : down_mx4_t<__bf16>(p, blocks, narrow, scratch, s);
}

}  // namespace moe
