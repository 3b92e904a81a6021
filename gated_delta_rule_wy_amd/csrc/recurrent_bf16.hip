// The recurrence over short runs of tokens, bf16 inputs.
#include "recurrent_impl.hpp"

namespace gdn2 {

hipError_t launch_recurrent_bf16(const RecurrentArgs &a, hipStream_t st) { return rec_dk<uint16_t>(a, st); }

hipError_t launch_recurrent(const RecurrentArgs &a, hipStream_t st)
{
    return a.bf16 ? launch_recurrent_bf16(a, st) : launch_recurrent_f32(a, st);
}

} // namespace gdn2
