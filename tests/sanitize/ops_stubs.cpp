// ops_stubs.cpp -- test infrastructure: stand-ins for the kernel launchers of
// the operators around the linear, beside host_stubs.cpp, so that
// mx_ops_api.cpp builds and runs on a CPU under the sanitizers.  No launcher
// touches memory; the last launch's sizes are kept for the checks.
#include <hip/hip_runtime.h>

#include "../../microscaling_quantized_linear_amd/csrc/mx_kernels.h"

extern "C" {
long mx_ops_launches = 0;
}

namespace mx {

static hipError_t counted() {
    ++mx_ops_launches;
    return hipSuccess;
}

hipError_t launch_add_rms_norm(const NormArgs &, int, int, hipStream_t) { return counted(); }
int64_t moe_sort_ws_bytes(int64_t E, int64_t pairs) {
    return pairs > 2048 ? (E + 4) * 4 * 2 : 0;
}
hipError_t launch_moe_sort(int64_t, int64_t, int64_t, const int32_t *, int32_t *, int32_t *,
                           int32_t *, void *, hipStream_t) {
    return counted();
}
hipError_t launch_moe_gather_sum(int64_t, int64_t, int64_t, int64_t, const uint16_t *, int64_t,
                                 const int32_t *, const float *, uint16_t *, int64_t,
                                 hipStream_t) {
    return counted();
}
const char *grouped_kernel_name(const GroupedArgs &) { return "grouped"; }
hipError_t launch_grouped(int, int, const GroupedArgs &, hipStream_t) { return counted(); }
hipError_t launch_stage_rows(const StageArgs &, int, hipStream_t) { return counted(); }
int64_t lora_splits(int64_t, int64_t, bool) { return 1; }
hipError_t launch_lora(const LoraArgs &, hipStream_t) { return counted(); }

}  // namespace mx
