// How the tensor-core form of the gate's gradient holds 32-bit values in f16: blocks of
// kGateBlock rows share a power of two 2^e, and v = (hi + lo / kGateLo) 2^e.
#pragma once

#include "mma.cuh"

namespace moe {

constexpr int kGateBlock = 128;
constexpr float kGateLo = 2048.f;      // 2^11: lo has an exponent range of its own

}  // namespace moe
