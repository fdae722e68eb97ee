// act_coef.h -- host side of the activations in products' epilogues (defined in
// gated_ffn.hip).
#pragma once

#include "act_math.h"

namespace meblock {

// Whether the activation and its parameter are ones that calls take.
bool act_ok(int act, float param);
// Its coefficients for the kernels.
meswish::Coef unit_coef(int act, float param);

}  // namespace meblock
