// cgtp_act.h -- the activations of the node-side and dense operators in fp32, and
// their slopes (device code).
#pragma once

#include <hip/hip_runtime.h>

namespace cgtp {

// 1 ulp reciprocal and exp2: the error stays at that of the fp32 arguments
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// tanh from exp(2|z|): 1 - 2 / (e + 1), by its series where that would cancel
__device__ __forceinline__ float tanh_f(float z)
{
    const float t = fabsf(z), u = z * z;
    // z (1 - u/3 + 2u^2/15 - 17u^3/315 + 62u^4/2835 - 1382u^5/155925)
    const float near = z * (1.0f + u * (-0.33333334f + u * (0.13333334f + u * (-0.053968254f + u * (0.021869488f + u * -0.0088632355f)))));
    const float far = copysignf(1.0f - 2.0f * __builtin_amdgcn_rcpf(__expf(2.0f * t) + 1.0f), z);
    return t < 0.3f ? near : far;
}

enum : int { kNone = 0, kSilu = 1, kTanh = 2 };  // values of cgtp_act_t

template <int ACT>
__device__ __forceinline__ float act_of(float z)
{
    if constexpr (ACT == kNone) return z;
    if constexpr (ACT == kSilu) return z * sigmoid(z);
    return tanh_f(z);
}

// act'(z)
template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == kNone) return 1.0f;
    if constexpr (ACT == kSilu) {
        const float s = sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    }
    const float t = tanh_f(z);
    return 1.0f - t * t;
}

// the same with the activation known at run time (uniform over a launch)
__device__ __forceinline__ float act_of(int act, float z)
{
    return act == kNone ? z : act == kSilu ? act_of<kSilu>(z) : act_of<kTanh>(z);
}

__device__ __forceinline__ float act_slope(int act, float z)
{
    return act == kNone ? 1.0f : act == kSilu ? act_slope<kSilu>(z) : act_slope<kTanh>(z);
}

}  // namespace cgtp
