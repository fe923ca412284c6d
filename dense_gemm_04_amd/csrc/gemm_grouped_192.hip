// Products grouped by expert on tiles of 192 x 256: three quarters of a 256 x 256
// tile's work, for products whose last round of those would be mostly empty
// (pick_tile in gemm_grouped.hip; 8 x 8001 x 4096 x 2048 with B stored N x K 149 -> 143 us).

#include "grouped_tiled.hpp"
#include "ops.hpp"

namespace dg {

hipError_t launch_grouped_192(const GroupedArgs& a, hipStream_t s) {
    const int64_t tn = (a.N + 255) / 256, tm = row_tiles_bound(a.M, a.groups, 192);
    if (tm * tn > kMaxGrid) return hipErrorInvalidConfiguration;
    const bool epi = a.bias != nullptr || a.act != kActNone || a.row_scale != nullptr;
    auto fn = a.tb ? (epi ? &gemm_grouped_kernel<192, 256, 2, 4, false, true, true, false>
                          : &gemm_grouped_kernel<192, 256, 2, 4, false, true, false, false>)
                   : (epi ? &gemm_grouped_kernel<192, 256, 2, 4, false, false, true, false>
                          : &gemm_grouped_kernel<192, 256, 2, 4, false, false, false, false>);
    return launch_kernel(fn,
                         dim3((unsigned)(tm * tn)), dim3(512), s, a, tm, tn);
}

}  // namespace dg
