// Products of rows in f32 (linear_impl.hpp).
#include "linear_impl.hpp"

namespace gdn2 {

hipError_t launch_gemm_f32(const GemmArgs &a, hipStream_t st) { return launch_gemm_type<Elt::kF32>(a, st); }

} // namespace gdn2
