// Elements of the arrays whose type is the caller's choice (fp32 or bf16), and
// checks of pointers and types, shared by the token scores and the embedding
// rows (internal to libdspark).
#pragma once

#include "common.cuh"

namespace dspark {

constexpr int kMaxItems = 1 << 24;
constexpr int kSms = 148;   // of a B200: grids are sized for them

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(uint16_t x) { return bf16_bits_to_float(x); }

// Two fp32 values as a pair of bf16, rounded to nearest even.
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  unsigned r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16(v, 0.f)); }

// A token id or row of an item that is out of range.
__device__ __forceinline__ void record_bad_item(unsigned* err, int item) {
  set_error(err, DSPARK_ERR_DEVICE_ASSERT, 0x70000000u | static_cast<unsigned>(item));
}

inline bool is_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool is_given(const void* p) { return p != nullptr && is_aligned16(p); }
inline bool is_element_type(dspark_dtype t) { return t == DSPARK_F32 || t == DSPARK_BF16; }

}  // namespace dspark
