// Gated linear recurrence: kernels with fp32 inputs and gates.
#include "scan_kernels.cuh"

namespace gs {
int scan_launch_f32(const ScanParams& p, const ScanMaps& maps, bool wide, int v, bool coupled, bool bwd, cudaStream_t s) {
    if (wide && bwd) return launch_wide_bwd<float, float, 1, false>(p, maps, coupled, s);
    if (wide && v == 2)
        return p.group > 1 ? launch_wide_fwd<float, float, 2, true>(p, maps, coupled, s)
                           : launch_wide_fwd<float, float, 2, false>(p, maps, coupled, s);
    if (wide) return launch_wide_fwd<float, float, 1, false>(p, maps, coupled, s);
    if (v == 3) return launch_narrow<float, float, 3>(p, coupled, bwd, s);
    if (v == 4) return launch_narrow<float, float, 4>(p, coupled, bwd, s);
    return launch_narrow<float, float, 1>(p, coupled, bwd, s);
}
}  // namespace gs
