// The recurrence over short runs of tokens, fp32 inputs.
#include "recurrent_impl.hpp"

namespace gdn2 {

hipError_t launch_recurrent_f32(const RecurrentArgs &a, hipStream_t st) { return rec_dk<float>(a, st); }

} // namespace gdn2
