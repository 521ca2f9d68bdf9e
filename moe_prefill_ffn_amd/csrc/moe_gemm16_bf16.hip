// The bf16 products' kernels.
#include "moe_gemm16_kernels.h"

namespace moe {

hipError_t launch_gemm16_bf16(const Gemm16& g, hipStream_t st) { return launch_gemm16_typed<kBF16>(g, st); }

}  // namespace moe
