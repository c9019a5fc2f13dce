// Operands from tiles that loads into LDS fill: device code for pipelines of
// such loads.
//
// The compiler cannot tell which stage a read of LDS meets and waits for every
// load into LDS that is open before it, so that a pipeline of any depth runs
// as one of a single stage.  These reads are written out, each block ending
// with its own wait; the caller waits for the loads of its stage, and for the
// other waves, before them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace aq {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void *lds_ptr_t;

// The LDS byte address of a pointer into a __shared__ array.
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)(uintptr_t)(lds_ptr_t) const_cast<void *>(p);
}

// NX 16-byte pieces of X and NW of the other operand, addresses in bytes.
__device__ __forceinline__ void lds_read(uint32_t xa, const uint32_t (&wa)[1], v4f &x, v4f (&w)[1]) {
  asm volatile(
      "ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x), "=&v"(w[0])
      : "v"(xa), "v"(wa[0])
      : "memory");
}
__device__ __forceinline__ void lds_read(uint32_t xa, const uint32_t (&wa)[2], v4f &x, v4f (&w)[2]) {
  asm volatile(
      "ds_read_b128 %0, %3\n\tds_read_b128 %1, %4\n\tds_read_b128 %2, %5\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x), "=&v"(w[0]), "=&v"(w[1])
      : "v"(xa), "v"(wa[0]), "v"(wa[1])
      : "memory");
}
__device__ __forceinline__ void lds_read(uint32_t xa, const uint32_t (&wa)[4], v4f &x, v4f (&w)[4]) {
  asm volatile(
      "ds_read_b128 %0, %5\n\tds_read_b128 %1, %6\n\tds_read_b128 %2, %7\n\t"
      "ds_read_b128 %3, %8\n\tds_read_b128 %4, %9\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x), "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]), "=&v"(w[3])
      : "v"(xa), "v"(wa[0]), "v"(wa[1]), "v"(wa[2]), "v"(wa[3])
      : "memory");
}
__device__ __forceinline__ void lds_read(const uint32_t (&xa)[2], const uint32_t (&wa)[1], v4f (&x)[2], v4f (&w)[1]) {
  asm volatile(
      "ds_read_b128 %0, %3\n\tds_read_b128 %1, %4\n\tds_read_b128 %2, %5\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(w[0])
      : "v"(xa[0]), "v"(xa[1]), "v"(wa[0])
      : "memory");
}
__device__ __forceinline__ void lds_read(const uint32_t (&xa)[2], const uint32_t (&wa)[2], v4f (&x)[2], v4f (&w)[2]) {
  asm volatile(
      "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %6\n\t"
      "ds_read_b128 %3, %7\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(w[0]), "=&v"(w[1])
      : "v"(xa[0]), "v"(xa[1]), "v"(wa[0]), "v"(wa[1])
      : "memory");
}
__device__ __forceinline__ void lds_read(const uint32_t (&xa)[2], const uint32_t (&wa)[4], v4f (&x)[2], v4f (&w)[4]) {
  asm volatile(
      "ds_read_b128 %0, %6\n\tds_read_b128 %1, %7\n\tds_read_b128 %2, %8\n\t"
      "ds_read_b128 %3, %9\n\tds_read_b128 %4, %10\n\tds_read_b128 %5, %11\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(w[0]), "=&v"(w[1]), "=&v"(w[2]), "=&v"(w[3])
      : "v"(xa[0]), "v"(xa[1]), "v"(wa[0]), "v"(wa[1]), "v"(wa[2]), "v"(wa[3])
      : "memory");
}
// (8-byte pieces of the other operand)
__device__ __forceinline__ void lds_read(const uint32_t (&xa)[2], const uint32_t (&wa)[2], v4f (&x)[2], v2u (&w)[2]) {
  asm volatile(
      "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b64 %2, %6\n\t"
      "ds_read_b64 %3, %7\n\t"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(x[0]), "=&v"(x[1]), "=&v"(w[0]), "=&v"(w[1])
      : "v"(xa[0]), "v"(xa[1]), "v"(wa[0]), "v"(wa[1])
      : "memory");
}

}  // namespace aq
