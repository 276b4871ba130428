// Gated linear recurrence: kernels with float16 inputs, gates of either type.
#include "scan_kernels.cuh"

namespace gs {
int scan_launch_f16(const ScanParams& p, const ScanMaps& maps, bool gate_f32, bool wide, int v, bool coupled, bool bwd, cudaStream_t s) {
    return gate_f32 ? launch_half_type<__half, float>(p, maps, wide, v, coupled, bwd, s)
                    : launch_half_type<__half, __half>(p, maps, wide, v, coupled, bwd, s);
}
}  // namespace gs
