// route.cuh -- the choice of one token's experts by one warp, shared by the
// routing kernels and the whole-layer kernel.
#pragma once

#include "common.cuh"

namespace gbw {

__device__ __forceinline__ float bf16_to_f32(uint32_t bits16) {
  return __uint_as_float(bits16 << 16);
}
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_to_f32(__ldg(p)); }
// from L2: the kernel before may still have been writing them when this one
// started (programmatic dependent launch)
__device__ __forceinline__ float load_logit(const float* p) { return __ldcg(p); }

__device__ __forceinline__ float no_nan(float v) {
  return v != v ? __int_as_float(0xFF800000) : v;
}

// Keys order as the values do, -0 equal to +0; 0 is below every value's key.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}

// exp(v - m) for v <= m; 1 for v == m also when both are infinite.
__device__ __forceinline__ float share(float v, float m) { return v == m ? 1.0f : expf(v - m); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The choice of one token: lane s < k gets the s-th expert and its weight.  A
// token without any logit above -inf gets weights of 0; with kNanRows (the whole
// layer, which shows nothing of its logits) weights of NaN when one of them is NaN.
template <typename TL, int NPL, bool kNanRows>
__device__ __forceinline__ void choose(const TL* row, int E, int k, int renorm, int lane, int& id,
                                       float& w) {
  uint32_t key[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) {
    const int e = j * 32 + lane;
    key[j] = e < E ? order_key(no_nan(load_logit(row + e))) : 0u;
  }
  float all = 0.0f, m = 0.0f, v = 0.0f;
  if (NPL <= 4) {
    // each lane's keys in falling order (equal ones by index), so that a
    // choice looks at one key of each lane
    int at[NPL];
#pragma unroll
    for (int j = 0; j < NPL; ++j) at[j] = j * 32 + lane;
#pragma unroll
    for (int i = 1; i < NPL; ++i)
#pragma unroll
      for (int j = i; j > 0; --j)
        if (key[j] > key[j - 1]) {
          const uint32_t tk = key[j];
          key[j] = key[j - 1];
          key[j - 1] = tk;
          const int ta = at[j];
          at[j] = at[j - 1];
          at[j - 1] = ta;
        }
    m = key_value(__reduce_max_sync(0xffffffffu, key[0]));
    if (!renorm) {
      float t = 0.0f;
#pragma unroll
      for (int j = 0; j < NPL; ++j)
        if (key[j]) t += share(key_value(key[j]), m);
      all = warp_sum(t);
    }
    for (int s = 0; s < k; ++s) {
      const uint32_t g = __reduce_max_sync(0xffffffffu, key[0]);
      const unsigned who = __ballot_sync(0xffffffffu, key[0] == g);
      int e;
      if (who & (who - 1))  // a tie: the lowest index
        e = (int)__reduce_min_sync(0xffffffffu, key[0] == g ? (unsigned)at[0] : 0xffffffffu);
      else
        e = __shfl_sync(0xffffffffu, at[0], __ffs(who) - 1);
      if (lane == s) { id = e; v = key_value(g); }
      if (at[0] == e) {
#pragma unroll
        for (int j = 0; j + 1 < NPL; ++j) {
          key[j] = key[j + 1];
          at[j] = at[j + 1];
        }
        key[NPL - 1] = 0u;
        at[NPL - 1] = -1;
      }
    }
  } else {
    for (int s = 0; s < k; ++s) {
      uint32_t lk = 0u;
      int le = 0;
#pragma unroll
      for (int j = 0; j < NPL; ++j)
        if (key[j] > lk) { lk = key[j]; le = j * 32 + lane; }
      const uint32_t g = __reduce_max_sync(0xffffffffu, lk);
      const int e = (int)__reduce_min_sync(0xffffffffu, lk == g ? (unsigned)le : 0xffffffffu);
      if (s == 0) {
        m = key_value(g);
        if (!renorm) {
          float t = 0.0f;
#pragma unroll
          for (int j = 0; j < NPL; ++j)
            if (key[j]) t += share(key_value(key[j]), m);
          all = warp_sum(t);
        }
      }
      if (lane == s) { id = e; v = key_value(g); }
#pragma unroll
      for (int j = 0; j < NPL; ++j)
        if (e == j * 32 + lane) key[j] = 0u;
    }
  }
  const float p = lane < k ? share(v, m) : 0.0f;
  const float total = renorm ? warp_sum(p) : all;
  w = m == __int_as_float(0xFF800000) ? 0.0f : p / total;
  if (kNanRows && m == __int_as_float(0xFF800000)) {  // rare, so read again
    bool nan = false;
    for (int e = lane; e < E; e += 32) {
      const float l = load_logit(row + e);
      nan |= l != l;
    }
    if (__any_sync(0xffffffffu, nan)) w = __int_as_float(0x7FC00000);
  }
}

}  // namespace gbw
