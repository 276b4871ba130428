// Gated linear recurrence: kernels with bfloat16 inputs and fp32 gates.
#include "scan_kernels.cuh"

namespace gs {
int scan_launch_bf16_f32(const ScanParams& p, const ScanMaps& maps, bool wide, int v, bool coupled, bool bwd,
                         cudaStream_t s) {
    return launch_half_type<__nv_bfloat16, float>(p, maps, wide, v, coupled, bwd, s);
}
}  // namespace gs
