// Shared by the text side's attention kernels: 16-bit pairs and the prompt
// attention launcher.
#pragma once

#include <type_traits>

#include "kernels.cuh"

namespace vlm {

// A pair of 16-bit values (the first in the low half) and fp32.
template <typename T>
__device__ __forceinline__ float2 unpack16(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack16<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack16<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float lo, float hi) {
  return pack_f16x2(lo, hi);
}

// 32 bytes in one instruction where they are aligned to it: a warp's rows lie
// apart, so each store instruction costs one pass per lane.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// Causal attention of packed prompts (include/vlm.h, vlm_prompt_attention); the
// arguments are checked by the caller. Lengths are host arrays.
struct PromptAttn {
  int dtype, heads, kv_heads, head_dim;
  const int32_t *q_lens, *kv_lens;
  int n_seqs;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  float scale;
  void* out;
  int64_t out_stride;
  int32_t* status;
};
int launch_prompt_attention(const PromptAttn& p, cudaStream_t s);

}  // namespace vlm
