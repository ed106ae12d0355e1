// Products with 4-bit weights, passes of 64 columns.
#include "ssd_matvec4_mma.cuh"

namespace ssd {
cudaError_t launch_matvec4_cols8(const Matvec4Plan &q, int shared, bool whole, cudaStream_t stream) {
    return matvec4::run<8>(q, shared, whole, stream);
}
}  // namespace ssd
