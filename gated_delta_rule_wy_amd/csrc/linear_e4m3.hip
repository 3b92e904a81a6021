// Products of rows in e4m3 (linear_impl.hpp).
#include "linear_impl.hpp"

namespace gdn2 {

hipError_t launch_gemm_e4m3(const GemmArgs &a, hipStream_t st) { return launch_gemm_type<Elt::kE4m3>(a, st); }

} // namespace gdn2
