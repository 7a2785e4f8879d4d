// SiLU of the layer's convolutions (kda_prefill_conv, kda_tree_conv).
#pragma once

#include "kda_device.cuh"

namespace kda {

// z / (1 + 2^(-z log2 e)), the two functions of the special unit once each
// (the reciprocal is flushed from 2^126 on, as in kda_layer_prologue's: below
// z = -87.3, where silu is under 2^-119 in size, it is -0)
__device__ __forceinline__ float2 silu2(float2 z) {
  const float2 t = fmul2(z, make_float2(-1.4426950408889634f, -1.4426950408889634f));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = __fadd2_rn(e, make_float2(1.f, 1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(e.y));
  return fmul2(z, r);
}

// ... of a pair, rounded to BF16
__device__ __forceinline__ uint32_t silu_pair(float2 z) {
  const __nv_bfloat162 r = __float22bfloat162_rn(silu2(z));
  return *reinterpret_cast<const uint32_t *>(&r);
}

}  // namespace kda
