// Products of rows in bf16 (linear_impl.hpp).
#include "linear_impl.hpp"

namespace gdn2 {

hipError_t launch_gemm_bf16(const GemmArgs &a, hipStream_t st) { return launch_gemm_type<Elt::kBf16>(a, st); }

} // namespace gdn2
