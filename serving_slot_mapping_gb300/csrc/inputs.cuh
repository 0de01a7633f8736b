// Reads of tensors that a kernel before this one may have written, for kernels that
// start before it has ended (programmatic dependent launch).  Such reads come behind
// griddepcontrol.wait, and they are ordinary loads kept in their place: the loads of
// __ldg promise data that nobody writes while the kernel runs, which does not hold
// here (the compiler may move them ahead of the wait, and a line that the SM read
// before it may be old).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace pa {

__device__ __forceinline__ int32_t ld_input(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_input(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int64_t ld_input(const int64_t* p) {
  int64_t v;
  asm volatile("ld.global.b64 %0, [%1];" : "=l"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_input(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_input(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// The same for data that is read once.
__device__ __forceinline__ unsigned char ld_stream(const unsigned char* p) {
  uint32_t v;
  asm volatile("ld.global.cs.u8 %0, [%1];" : "=r"(v) : "l"(p));
  return (unsigned char)v;
}
__device__ __forceinline__ unsigned short ld_stream(const unsigned short* p) {
  unsigned short v;
  asm volatile("ld.global.cs.b16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_stream(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.cs.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_stream(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.cs.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// seq_lens[b], clamped to [0, max_len]; out of range it is recorded when err is given.
__device__ __forceinline__ int ld_seq_len(const int32_t* seq_lens, int b, int max_len, unsigned long long* err) {
  const int L = ld_input(seq_lens + b);
  if (L >= 0 && L <= max_len) return L;
  if (err != nullptr) record_error(err, ERR_SEQ_LEN, L);
  return L < 0 ? 0 : max_len;
}

}  // namespace pa
