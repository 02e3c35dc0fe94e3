#include "attn_step_kv8.h"

namespace m3 {
template hipError_t launch_kv8_step<__bf16>(const Kv8StepArgs&, uint32_t, uint32_t, hipStream_t);
}  // namespace m3
