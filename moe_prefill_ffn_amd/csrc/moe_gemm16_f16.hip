// The fp16 products' kernels.
#include "moe_gemm16_kernels.h"

namespace moe {

hipError_t launch_gemm16_f16(const Gemm16& g, hipStream_t st) { return launch_gemm16_typed<kF16>(g, st); }

}  // namespace moe
