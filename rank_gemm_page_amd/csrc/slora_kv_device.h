// Device code that the KV cache's kernels share: codes and how they are read, the
// page table, reductions over a workgroup.
#pragma once

#include "slora_device.h"
#include "slora_kv.h"

namespace slora {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef float float8v __attribute__((ext_vector_type(8)));

typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
// 16 bytes that nobody else reads: they do not displace what is in the caches.
__device__ __forceinline__ uint4 ld16_once(const void* p) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const uint4v*>(p)));
}

// ---------------------------------------------------------------------------
// Codes.  An int8 code c is kept as the byte c + 128: the byte with 0x64 above
// it is the fp16 number 1024 + c + 128, so two codes become fp16 with one byte
// permute and one packed subtraction.  An e4m3 code is its byte.

// nearest: the code of a value in units of a code; four: of four, a byte each.
template <int CODE> struct Code;

template <> struct Code<SLORA_KV_INT8> {
  static constexpr float kTop = 127.f;
  static constexpr uint32_t kZero = 0x80;
  static __device__ __forceinline__ half8 halves(uint32_t a, uint32_t b) {
    const half2v bias = {(_Float16)1152.f, (_Float16)1152.f};
    union { uint32_t u; half2v h; } p[4];
    p[0].u = __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u);
    p[1].u = __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u);
    p[2].u = __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u);
    p[3].u = __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u);
    half8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const half2v h = p[i].h - bias;
      r[2 * i] = h[0];
      r[2 * i + 1] = h[1];
    }
    return r;
  }
  static __device__ __forceinline__ float value(uint32_t byte) { return (float)(int)byte - 128.f; }
  // Added to 1.5 * 2^52, a number this small is rounded to an integer (ties to
  // even) that stands in the low bits.  A subnormal range may lie below its
  // largest value by half a unit, which takes codes up to half as much again:
  // they are held at the largest one.
  static __device__ __forceinline__ uint32_t nearest(double x) {
#pragma clang fp contract(off)
    return (uint32_t)min(max(__double2loint(x + (0x1.8p52 + 128.)), 1), 255);
  }
  static __device__ __forceinline__ uint32_t four(double a, double b, double c, double d) {
    return __builtin_amdgcn_perm(nearest(b), nearest(a), 0x0c0c0400u) |
           __builtin_amdgcn_perm(nearest(d), nearest(c), 0x04000c0cu);
  }
};

template <> struct Code<SLORA_KV_FP8> {
  static constexpr float kTop = 448.f;
  static constexpr uint32_t kZero = 0;
  static __device__ __forceinline__ half8 halves(uint32_t a, uint32_t b) {
    const half2v p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, false);
    const half2v p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, true);
    const half2v p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, false);
    const half2v p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, true);
    return half8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
  }
  static __device__ __forceinline__ float value(uint32_t byte) {
    return __builtin_amdgcn_cvt_pk_f32_fp8((int)byte, false)[0];
  }
  // The definition rounds the 64-bit product to fp32 and then to e4m3.  A
  // subnormal range's values are held at the last code as above.
  static __device__ __forceinline__ uint32_t nearest(double x) {
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(held(x), 0.f, 0, false) & 0xFF;
  }
  static __device__ __forceinline__ float held(double x) { return __builtin_amdgcn_fmed3f((float)x, -kTop, kTop); }
  static __device__ __forceinline__ uint32_t four(double a, double b, double c, double d) {
    const int low = __builtin_amdgcn_cvt_pk_fp8_f32(held(a), held(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(held(c), held(d), low, true);
  }
};

template <int CODE>
__device__ __forceinline__ float8v floats8(uint32_t a, uint32_t b) {
  float8v r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = Code<CODE>::value((a >> (8 * i)) & 0xFF);
    r[4 + i] = Code<CODE>::value((b >> (8 * i)) & 0xFF);
  }
  return r;
}

// Row stride of the page table per (sequence, layer, head), 64-bit.
__device__ __forceinline__ const int32_t* kv_row(const KvView& kv, int seq, int layer, int head) {
  return kv.table + (((int64_t)seq * kv.n_layers + layer) * kv.n_kv + head) * kv.max_blocks;
}

// ---------------------------------------------------------------------------
// Codes of a range that grew: nearest(code * (old range / new range)).  The ratio
// is at most 1, so that no code passes the last one.

template <int CODE> struct Again;

// (byte - 128) * ratio as one fma, whose product with 128 is exact
template <> struct Again<SLORA_KV_INT8> {
  static __device__ __forceinline__ uint32_t one(uint32_t byte, double ratio) {
#pragma clang fp contract(off)
    return (uint32_t)__double2loint(__builtin_fma((double)(float)byte, ratio, -128. * ratio) + (0x1.8p52 + 128.));
  }
  static __device__ __forceinline__ uint32_t four(uint32_t old, double r0, double r1, double r2, double r3) {
    const uint32_t a = one(old & 0xFF, r0), b = one((old >> 8) & 0xFF, r1), c = one((old >> 16) & 0xFF, r2);
    const uint32_t low = __builtin_amdgcn_perm(b, a, 0x0c0c0400u);
    return low | __builtin_amdgcn_perm(one(old >> 24, r3), c, 0x04000c0cu);
  }
};

template <> struct Again<SLORA_KV_FP8> {
  static __device__ __forceinline__ uint32_t four(uint32_t old, double r0, double r1, double r2, double r3) {
    const auto low = __builtin_amdgcn_cvt_pk_f32_fp8((int)old, false);
    const auto high = __builtin_amdgcn_cvt_pk_f32_fp8((int)old, true);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32((float)((double)low[0] * r0), (float)((double)low[1] * r1), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32((float)((double)high[0] * r2), (float)((double)high[1] * r3), w, true);
    return (uint32_t)w;
  }
};

template <int CODE>
__device__ __forceinline__ uint32_t again4(uint32_t old, double ratio) {
  return Again<CODE>::four(old, ratio, ratio, ratio, ratio);
}
template <int CODE>
__device__ __forceinline__ uint4 again16(uint4 o, double ratio) {
  return make_uint4(again4<CODE>(o.x, ratio), again4<CODE>(o.y, ratio), again4<CODE>(o.z, ratio),
                    again4<CODE>(o.w, ratio));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int m = 32; m; m >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  return v;
}
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t* lds) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) v = max(v, lds[w]);
  return v;
}

}  // namespace slora
