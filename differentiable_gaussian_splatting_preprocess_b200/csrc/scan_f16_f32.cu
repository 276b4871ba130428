// Gated linear recurrence: kernels with float16 inputs and fp32 gates.
#include "scan_kernels.cuh"

namespace gs {
int scan_launch_f16_f32(const ScanParams& p, const ScanMaps& maps, bool wide, int v, bool coupled, bool bwd,
                         cudaStream_t s) {
    return launch_half_type<__half, float>(p, maps, wide, v, coupled, bwd, s);
}
}  // namespace gs
