// What the C ABI's entry points (api.hip, operators_api.hip) share.
#pragma once

#include "../../include/gdn2.h"
#include "gdn2_launch.hpp"

namespace gdn2 {

// Marks the start of a library call: decides whether its kernels are timed.
void prof_call();

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

inline bool head_dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// The convolution parameters of a *_prologue call: weights required, biases
// optional, history in / out each all-or-none.
int conv_args(const gdn2_short_conv *c, Prologue *p);

} // namespace gdn2
