// swiglu.cuh -- silu(gate) * up in fp32, shared by the row quantisers and the
// whole-layer kernel.
#pragma once

namespace gbw {

// silu(g) = g / (1 + e^-g), for g < 0 as g e^g / (1 + e^g): the denominator stays
// in [1, 2].  (e^-g passes 2^126 for g < -87.3, from where __fdividef gives 0 for
// values that fp32, and the scale of an MXFP4 block, still hold.)
__device__ __forceinline__ float swiglu(float g, float u) {
  const float e = __expf(-fabsf(g));
  return __fdividef(g < 0.0f ? g * e : g, 1.0f + e) * u;
}

}  // namespace gbw
