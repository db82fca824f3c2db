// net_common.cuh -- device helpers shared by the network operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "gs_internal.cuh"
#include "gs_net.h"

namespace gs {

// N elements that move as one access of up to 16 bytes (two for 32 bytes).
template <typename T, int N>
struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Pack {
  T v[N];
};

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, N>*>(p);
}
template <typename T, int N>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, N>& v) {
  *reinterpret_cast<Pack<T, N>*>(p) = v;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two values as the word of their bits.
template <typename T>
__device__ __forceinline__ uint32_t pair_word(float a, float b);
template <>
__device__ __forceinline__ uint32_t pair_word<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pair_word<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two fp32 operations in one instruction, each rounded as the single one is.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{ .reg .b64 a, b, c, r; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};"
      " fma.rn.f32x2 r, a, b, c; mov.b64 {%0, %1}, r; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 a, b, r; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5};"
      " add.rn.f32x2 r, a, b; mov.b64 {%0, %1}, r; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 a, b, r; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5};"
      " mul.rn.f32x2 r, a, b; mov.b64 {%0, %1}, r; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

inline int dtype_size(int32_t dtype) { return dtype == GS_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t dtype) { return dtype >= GS_BF16 && dtype <= GS_F32; }

// Element alignment of a pointer, and whether every row of a matrix starts on
// a multiple of `bytes`.
inline bool aligned_to(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
inline bool rows_aligned(const void* p, int64_t stride, int elem, size_t bytes) {
  return !p || (aligned_to(p, bytes) && (stride * elem) % (int64_t)bytes == 0);
}

// An output at its input's address: the same rows, or some would be written before
// others are read there.
inline bool in_place_ok(int64_t tokens, const void* in, int64_t in_stride, const void* out,
                        int64_t out_stride) {
  return in != out || !in || tokens < 2 || in_stride == out_stride;
}

// Kernels that begin while the one before on their stream ends: launched by
// launch_overlapped, a kernel touches global memory only after wait_for_previous,
// which returns when that kernel and all before it have ended and their writes are
// there.  Nor does it take what it reads for constant (__ldg, const __restrict__): that
// may be written while it is already running.  launch_dependents lets the next one be
// set up.  Back to back on 32640 x
// 1024 in bf16 it took the norms from 53.2 to 50.8 us forward and from 84.6 to 82.2
// backward.
__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, A... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

inline int device_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    return 152;
  return n;
}

// A checkpoint's arrays: whole groups of bytes, rows that do not overlap.
inline bool ckpt_ok(int64_t tokens, int32_t channels, const int8_t* q, int64_t q_stride,
                    const uint8_t* e, int64_t e_stride) {
  const int64_t groups = div_up(channels, GS_ACT8_GROUP);
  return q && e && aligned16(q) && q_stride % 16 == 0 && q_stride >= groups * GS_ACT8_GROUP &&
         (tokens < 2 || e_stride >= groups);
}

// ---- the 8-bit checkpoint's format ---------------------------------------
// Exponent of a group from the bits of its largest magnitude: 127 = 1.984375
// * 2^6, so a magnitude m * 2^p (1 <= m < 2) fits 127 steps of 2^(p - 6) when
// m <= 1.984375, and of 2^(p - 5) otherwise.  255 marks a group with an
// infinity or a NaN (magnitude bits >= 0x7f800000).
__device__ __forceinline__ uint32_t act8_exponent(uint32_t mag_bits) {
  if (mag_bits >= 0x7f800000u) return 255u;
  const int e = (int)(mag_bits >> 23) - 6 + ((mag_bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return e < 1 ? 1u : (uint32_t)e;
}
// 2^(127 - e): e = 255 gives 0 times a value, which the caller replaces by 0.
__device__ __forceinline__ float act8_inverse(uint32_t e) {
  return e == 255u ? 0.f : __uint_as_float((254u - e) << 23);
}
// The step 2^(e - 127); +inf for e = 255, so that 0 * step is the NaN that
// such a group reads back as.
__device__ __forceinline__ float act8_step(uint32_t e) { return __uint_as_float(e << 23); }

// Where rounding to 64 steps carried a value past the largest number of the type that
// it is read in (a magnitude above 127 / 128 of the power of two beyond fp16's, bf16's
// or fp32's range), it reads as that number.  Only groups with an exponent from here on
// can hold such a value: fp16 holds 127 * 2^9, bf16 and fp32 127 * 2^121.
template <typename T>
constexpr uint32_t kAct8Top = 249u;
template <>
constexpr uint32_t kAct8Top<__half> = 137u;
template <typename T>
__device__ __forceinline__ float largest();
template <>
__device__ __forceinline__ float largest<float>() { return __uint_as_float(0x7f7fffffu); }
template <>
__device__ __forceinline__ float largest<__nv_bfloat16>() { return __uint_as_float(0x7f7f0000u); }
template <>
__device__ __forceinline__ float largest<__half>() { return 65504.f; }
// v = q * step, q not 0: what half a step less would still hold was not beyond the type.
template <typename T>
__device__ __forceinline__ float act8_within(float v, float q, float step) {
  const float top = largest<T>();
  return fabsf(v) > top && (fabsf(q) - 0.5f) * step <= top ? copysignf(top, v) : v;
}

// q in the low byte of the result (anything where v is not finite): v * inv is exact
// (a power of two), and adding 1.5 * 2^23 rounds it to the nearest whole number, ties
// to even.
__device__ __forceinline__ uint32_t act8_round(float v, float inv) {
  return __float_as_uint(__fmaf_rn(v, inv, 12582912.f));
}
// The value of byte `i` of a word of checkpoint bytes, times the step: the byte
// (its sign bit flipped) is put into the significand of 2^23 + 128 + q.
__device__ __forceinline__ float act8_value(uint32_t flipped, int i, float step) {
  return (__uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7440 | i)) - 8388736.f) * step;
}

}  // namespace gs
