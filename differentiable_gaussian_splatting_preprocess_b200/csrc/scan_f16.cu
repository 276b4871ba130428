// Gated linear recurrence: kernels with float16 inputs and gates.
#include "scan_kernels.cuh"

namespace gs {
int scan_launch_f16(const ScanParams& p, const ScanMaps& maps, bool wide, int v, bool coupled, bool bwd,
                     cudaStream_t s) {
    return launch_half_type<__half, __half>(p, maps, wide, v, coupled, bwd, s);
}
}  // namespace gs
