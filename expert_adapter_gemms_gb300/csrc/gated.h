// Launchers of the gated block shared between its translation units.
#pragma once

#include "internal.h"

namespace moe_lora {

// The gated block (dh null: h [T, I]) or its backward's dy = [dg | du] [T, 2I], for at most
// kFewMaxTokens tokens.
constexpr int kFewMaxTokens = 32;
int launch_gated_few(int dtype, int act, const void* x, const void* W1, int T, int H, int I, const void* dh, void* out,
                     cudaStream_t stream);

}  // namespace moe_lora
