// The grouped FFN's kernels over weights in microscaled 4-bit floating point (cells in
// ffn_cells.hpp, layout in mx4.hip).
#include "ffn_cells.hpp"

namespace moe {

hipError_t gateup_cells_mx4(int dtype, const GemmArgs &p, int64_t blocks, bool gathered,
                            const void *scratch, const WavePlan *wp, hipStream_t s)
{
    return dtype == 1 ? gateup_cells<_Float16, kMx4>(p, blocks, gathered, scratch, wp, s)
                      : gateup_cells<__bf16, kMx4>(p, blocks, gathered, scratch, wp, s);
}

hipError_t down_cells_mx4(int dtype, const GemmArgs &p, int64_t blocks, const void *scratch,
                          hipStream_t s)
{
    return dtype == 1 ? down_cells<_Float16, kMx4>(p, blocks, scratch, s)
                      : down_cells<__bf16, kMx4>(p, blocks, scratch, s);
}

}  // namespace moe
