// The MX4 format and the device helpers its kernels share.
//
// An MX4 row of K values (K % 32 == 0) is K / 2 bytes of codes and K / 32
// scale bytes.  A code is sign, two exponent bits, one mantissa bit (the
// magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6); element 2j is the low half of byte
// j.  Scale byte b stands for 2^(b - 127); 255 marks a block with no value
// (NaN).  This is also the operand format of the block-scaled 4-bit tensor
// core instruction, so packed rows feed it without conversion.
//
// Quantisation of a block: with A its largest magnitude,
//     b = max(0, floor(log2 A) + 127 - 2),
// so that A / 2^(b - 127) lies in [4, 8); every element is divided by that
// power of two (exact), rounded to the nearest code (ties to the even code)
// and saturated at 6.  A block with an infinity or NaN gets b = 255, codes 0.
#pragma once
#include <atomic>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "colimoe_internal.cuh"

namespace colimoe {

constexpr int MXB = 32;  // values per scale byte

__host__ __device__ inline size_t type_bytes(int32_t t) { return t == COLI_F32 ? 4 : 2; }
__host__ __device__ inline bool float_type(int32_t t) { return t == COLI_F32 || t == COLI_BF16 || t == COLI_F16; }

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Scale byte of a block from the float bits of its largest magnitude (bits
// without sign; an infinity or NaN anywhere makes the largest bits >=
// 0x7f800000): the exponent field is floor(log2 A) + 127 for normal A and 0
// below, where the byte is 0 anyway.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - b) as a factor for b <= 252 (a normal float: exponent 254 - b);
// 0 for b = 255, so every code of the block becomes 0 unless the factor meets
// an infinity or NaN, whose elements the caller replaces by 0
__device__ __forceinline__ float mx4_inv(uint32_t b) { return b == 255u ? 0.f : __uint_as_float((254u - b) << 23); }
// 2^(b - 127); b = 0 is a subnormal float, 255 NaN
__device__ __forceinline__ float mx4_scale(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7fc00000u : b << 23);
}
// two scaled values -> one byte of codes (lo in the low half): round to
// nearest even, saturating, in one conversion instruction
__device__ __forceinline__ uint32_t mx4_pack2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
// value of a 4-bit code: exponent and mantissa bits put in a float's place are
// the code's value times 2^-126
__device__ __forceinline__ float mx4_code(uint32_t c) {
  return __uint_as_float(((c & 7u) << 22) | ((c & 8u) << 28)) * __uint_as_float(253u << 23);
}

// 8 consecutive elements of a lane, the block's 32 in 4 neighbouring lanes:
// returns the lane's 8 codes in one word and the block's scale byte.
__device__ __forceinline__ uint32_t mx4_quant8(const float* v, uint32_t* byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t b = mx4_scale_byte(m);
  *byte = b;
  if (b == 255u) return 0u;
  const float inv = mx4_inv(b);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= mx4_pack2(v[2 * i] * inv, v[2 * i + 1] * inv) << (8 * i);
  return w;
}

// 8 consecutive elements as they are in memory, so that a thread can have many
// loads in flight in few registers.  VEC: the address is 16-byte aligned and
// all 8 exist (one or two 16-byte loads); otherwise n guarded single loads,
// zero beyond.
template <typename T>
struct Raw8 {
  uint4 q[sizeof(T) / 2];
};
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load8(const T* p, int n) {
  Raw8<T> r;
  if (VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = n > 0 ? __ldcs(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0, 0, 0, 0);
  } else {
    constexpr int PER = 4 / sizeof(T);  // elements in a 32-bit word
    uint32_t w[2 * sizeof(T)] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= n) continue;
      if constexpr (PER == 1) w[i] = __float_as_uint(p[i]);
      else w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    }
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void floats8(const Raw8<T>& r, float* v) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    const uint32_t w[4] = {r.q[i].x, r.q[i].y, r.q[i].z, r.q[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        v[4 * i + j] = __uint_as_float(w[j]);
      } else {
        const T* h = reinterpret_cast<const T*>(&w[j]);
        v[2 * j] = to_f32(h[0]);
        v[2 * j + 1] = to_f32(h[1]);
      }
    }
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const float* v) {
  if (VEC) {
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        T h[2] = {from_f32<T>(v[2 * i]), from_f32<T>(v[2 * i + 1])};
        w[i] = *reinterpret_cast<uint32_t*>(h);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// rows of `ld` elements of type t at p keep 16-byte alignment
inline bool rows_aligned(const void* p, int64_t ld, int32_t t) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ((uint64_t)ld * type_bytes(t)) % 16 == 0;
}
// SMs of the current device (0 on failure), looked up once per device
inline int device_sms() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}
// launch with programmatic dependent launch (every kernel here begins with
// griddepcontrol.wait before it touches anything but weights)
template <typename... KA, typename... A>
cudaError_t launch_pdl(void (*kernel)(KA...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KA>(args)...);
}

}  // namespace colimoe
