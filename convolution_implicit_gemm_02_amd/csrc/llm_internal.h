// llm_internal.h -- between the host side of the decoder-step operators (llm_host.cpp) and their kernels (llm_*.hip), and
// what those kernels share.  Not part of the public C ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/cbs_llm.h"

namespace cbs {

// Threads of a launch along its first axis: fewer than 2^32.
constexpr int64_t kMaxThreads = 0xffffffff;

// The host side has checked every argument before it launches.
hipError_t launch_rms_norm(const cbs_rms_desc &d, const cbs_rms_args &a, hipStream_t stream);
hipError_t launch_kv_write(const cbs_kv_desc &d, const cbs_kv_args &a, hipStream_t stream);
hipError_t launch_kv_read(const cbs_kv_desc &d, const cbs_kv_args &a, hipStream_t stream);

}  // namespace cbs

#ifdef __HIPCC__
namespace cbs {

typedef _Float16 f16_t;
typedef __bf16 bf16_t;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Element types by their CBS_ number, for code that picks the type at run time (wave-uniform).
__device__ __forceinline__ float load_as_f32(const void *p, int64_t i, int dtype) {
  switch (dtype) {
    case CBS_F16: return (float)((const f16_t *)p)[i];
    case CBS_BF16: return (float)((const bf16_t *)p)[i];
    default: return ((const float *)p)[i];
  }
}

__device__ __forceinline__ void store_f32_as(void *p, int64_t i, float v, int dtype) {
  switch (dtype) {
    case CBS_F16: ((f16_t *)p)[i] = (f16_t)v; break;
    case CBS_BF16: ((bf16_t *)p)[i] = (bf16_t)v; break;
    default: ((float *)p)[i] = v;
  }
}

// N elements from any element-aligned address: one wide access (global memory takes unaligned ones on this target).
template <typename T, int N>
struct Vec {
  T v[N];
};
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T *p) {
  Vec<T, N> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, N> &r) {
  __builtin_memcpy(p, &r, sizeof(r));
}

// The same past the caches, for what this kernel does not read again: written lines need not leave the L2 when it ends.
// us, cached and past: a norm of 4096 rows of 5120 bfloat16 40.5 and 27.8, of one row of 4096 4.5 and 3.6.
template <typename T, int N>
__device__ __forceinline__ void store_past(T *p, const Vec<T, N> &r) {
  if constexpr (sizeof(r) == 4) {
    typedef uint32_t U __attribute__((aligned(1)));
    __builtin_nontemporal_store(__builtin_bit_cast(uint32_t, r), (U *)p);
  } else {
    typedef uint32_t V __attribute__((ext_vector_type(sizeof(r) / 4)));
    typedef uint32_t U __attribute__((ext_vector_type(sizeof(r) / 4), aligned(1)));
    __builtin_nontemporal_store(__builtin_bit_cast(V, r), (U *)p);
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
// |v| as an integer keeps the order of magnitudes and puts a NaN above every number, so that a maximum over it does not lose one.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t wave_max_bits(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  return v;
}

// The step of a row of int8 codes whose largest magnitude is top, and a value's code.
__device__ __forceinline__ float code_step(float top) {
  const float s = __fdiv_rn(top, 127.0f);
  return s == 0.0f ? 1.0f : s;
}
__device__ __forceinline__ int code_of(float v, float step) {
  return (int)fminf(fmaxf(rintf(__fdiv_rn(v, step)), -127.0f), 127.0f);
}
// N of them, a multiple of four.  The quotient as a product with the step's reciprocal, corrected by its remainder (Markstein,
// IBM J. Res. Dev. 34, 1990): with a correctly rounded reciprocal that is the correctly rounded quotient, in a third of a division's
// instructions.  The remainder
// needs room below: steps under 2^-100 go the long way.  1.5 times 2^23 added rounds to a whole number, whose two's complement
// the low bits then are.
template <int N>
__device__ __forceinline__ Vec<int8_t, N> codes_of(const float (&v)[N], float step) {
  const float guess = __builtin_amdgcn_rcpf(step), by = __builtin_fmaf(__builtin_fmaf(-step, guess, 1.0f), guess, guess);
  uint32_t bits[N];
#pragma unroll
  for (int i = 0; i < N; i++) {
    const float q = v[i] * by;
    bits[i] = __float_as_uint(__builtin_fmaf(__builtin_fmaf(-q, step, v[i]), by, q) + 12582912.0f);
  }
  uint32_t words[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; i++)
    words[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(bits[4 * i + 3], bits[4 * i + 2], 0x0c0c0400u), __builtin_amdgcn_perm(bits[4 * i + 1], bits[4 * i], 0x0c0c0400u), 0x05040100u);
  Vec<int8_t, N> q = __builtin_bit_cast(Vec<int8_t, N>, words);
  if (__any(step < 0x1p-100f)) {
#pragma unroll
    for (int i = 0; i < N; i++) q.v[i] = (int8_t)code_of(v[i], step);
  }
  return q;
}

// N bytes a lane straight to LDS, lane l's at `to` + N l.
template <int N>
__device__ __forceinline__ void to_lds(unsigned char *to, const char *from) {
  const auto *f = (const __attribute__((address_space(1))) void *)from;
  auto *t = (__attribute__((address_space(3))) void *)to;
  if constexpr (N == 16) __builtin_amdgcn_global_load_lds(f, t, 16, 0, 0);
  else __builtin_amdgcn_global_load_lds(f, t, 4, 0, 0);
}
// Until n vector-memory operations of the wave are outstanding at most, and no LDS operation.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt is a 6-bit field");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}
// A barrier that waits for nothing else: __syncthreads() would wait for the loads on their way to LDS.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace cbs
#endif
