// mode_stubs.cpp -- test infrastructure: the launcher stand-ins of ops_stubs.cpp
// and the launch plans of mx_plan.cpp, with a switch that changes the
// batch-invariant mode at the point where a call works out its workspace's
// size, as another thread could.
#include "../../include/mx.h"
#include "../../microscaling_quantized_linear_amd/csrc/mx_kernels.h"

#define lora_splits stub_lora_splits
#define launch_lora stub_launch_lora
#include "ops_stubs.cpp"
#undef lora_splits
#undef launch_lora

#define plan_gemv_w8 plain_plan_gemv_w8
#include "../../microscaling_quantized_linear_amd/csrc/mx_plan.cpp"
#undef plan_gemv_w8

extern "C" {
int mx_switch_to = -1;            // the mode to set there, -1: leave it
long mx_lora_written = 0;         // bytes of partial sums that the last launch writes
}

namespace mx {

static void switch_mode() {
    if (mx_switch_to >= 0) mx_set_batch_invariant(mx_switch_to);
}

// as many splits as the kernels make of K = 7168 in either mode
static int64_t splits_of(bool invariant) { return invariant ? 4 : 7; }

int64_t lora_splits(int64_t, int64_t, bool invariant) {
    switch_mode();
    return splits_of(invariant);
}

hipError_t launch_lora(const LoraArgs &a, hipStream_t) {
    mx_lora_written = (long)(splits_of(a.invariant) * a.M * ((a.R + 15) / 16 * 16) * 4);
    return hipSuccess;
}

GemvW8Plan plan_gemv_w8(int64_t tiles, int64_t steps, int64_t token_tiles, int waves, int group) {
    switch_mode();
    return plain_plan_gemv_w8(tiles, steps, token_tiles, waves, group);
}

}  // namespace mx
