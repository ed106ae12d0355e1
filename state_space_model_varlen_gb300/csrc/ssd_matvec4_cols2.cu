// Products with 4-bit weights, passes of 16 columns.
#include "ssd_matvec4_mma.cuh"

namespace ssd {
cudaError_t launch_matvec4_cols2(const Matvec4Plan &q, int shared, bool whole, cudaStream_t stream) {
    return matvec4::run<2>(q, shared, whole, stream);
}
}  // namespace ssd
