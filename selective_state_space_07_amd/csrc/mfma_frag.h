// Operands of the matrix cores as the SSD kernels use them (the linear-attention
// kernels take the vector types and the rounded form): 8 consecutive k-values
// per lane, multiplied as one 16x16x32 bfloat16 step or as eight 16x16x4 float32
// steps over the same 8 values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mscan {

typedef float f4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

// An MFMA operand: 8 k-values of one row (A) or one column (B).
template <int IO>
struct Frag;
template <>
struct Frag<1> {
  bf8 v;
};
template <>
struct Frag<0> {
  f4 lo, hi;
};

__device__ __forceinline__ Frag<1> frag8(const uint16_t* p) {  // 16-byte aligned
  return Frag<1>{__builtin_bit_cast(bf8, *reinterpret_cast<const u4*>(p))};
}
__device__ __forceinline__ Frag<0> frag8(const float* p) {  // 16-byte aligned
  return Frag<0>{*reinterpret_cast<const f4*>(p), *reinterpret_cast<const f4*>(p + 4)};
}
// 4 + 4 values (the permuted K order)
__device__ __forceinline__ Frag<1> frag44(const uint16_t* p0, const uint16_t* p1) {  // 8-byte aligned
  const u2 a = *reinterpret_cast<const u2*>(p0), b = *reinterpret_cast<const u2*>(p1);
  const u4 v = {a.x, a.y, b.x, b.y};
  return Frag<1>{__builtin_bit_cast(bf8, v)};
}
__device__ __forceinline__ Frag<0> frag44(const float* p0, const float* p1) {  // 16-byte aligned
  return Frag<0>{*reinterpret_cast<const f4*>(p0), *reinterpret_cast<const f4*>(p1)};
}
// from registers (float), rounded to the operand type
template <int IO>
__device__ __forceinline__ Frag<IO> frag_regs(f4 lo, f4 hi);
template <>
__device__ __forceinline__ Frag<1> frag_regs<1>(f4 lo, f4 hi) {
  bf8 v;
  v[0] = static_cast<__bf16>(lo.x);
  v[1] = static_cast<__bf16>(lo.y);
  v[2] = static_cast<__bf16>(lo.z);
  v[3] = static_cast<__bf16>(lo.w);
  v[4] = static_cast<__bf16>(hi.x);
  v[5] = static_cast<__bf16>(hi.y);
  v[6] = static_cast<__bf16>(hi.z);
  v[7] = static_cast<__bf16>(hi.w);
  return Frag<1>{v};
}
template <>
__device__ __forceinline__ Frag<0> frag_regs<0>(f4 lo, f4 hi) {
  return Frag<0>{lo, hi};
}
template <int IO>
__device__ __forceinline__ Frag<IO> frag_zero();
template <>
__device__ __forceinline__ Frag<1> frag_zero<1>() {
  const u4 z = {0u, 0u, 0u, 0u};
  return Frag<1>{__builtin_bit_cast(bf8, z)};
}
template <>
__device__ __forceinline__ Frag<0> frag_zero<0>() {
  return Frag<0>{f4{0.0f, 0.0f, 0.0f, 0.0f}, f4{0.0f, 0.0f, 0.0f, 0.0f}};
}

__device__ __forceinline__ f4 mma(const Frag<1>& a, const Frag<1>& b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f4 mma(const Frag<0>& a, const Frag<0>& b, f4 c) {
  // slot j of every lane group feeds step j: the eight steps cover all 32 k
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo.x, b.lo.x, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo.y, b.lo.y, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo.z, b.lo.z, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo.w, b.lo.w, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi.x, b.hi.x, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi.y, b.hi.y, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi.z, b.hi.z, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi.w, b.hi.w, c, 0, 0, 0);
  return c;
}

}  // namespace mscan
