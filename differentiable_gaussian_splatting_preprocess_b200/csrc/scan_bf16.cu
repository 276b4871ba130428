// Gated linear recurrence: kernels with bfloat16 inputs and gates.
#include "scan_kernels.cuh"

namespace gs {
int scan_launch_bf16(const ScanParams& p, const ScanMaps& maps, bool wide, int v, bool coupled, bool bwd,
                     cudaStream_t s) {
    return launch_half_type<__nv_bfloat16, __nv_bfloat16>(p, maps, wide, v, coupled, bwd, s);
}
}  // namespace gs
